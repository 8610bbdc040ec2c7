"""Builds of the library in which a bounded wait of one source runs out where a test wants it: the wait that the kernels call
is replaced, by the preprocessor, by one that gives up in one place and is the kernels' own elsewhere."""
import os
import subprocess

from gqa_flash_attention_prefill_gb300 import build


def library(folder, source, header, place):
    """Path of a library whose `source` (a .cu of the package) gives up a wait where the expression `place` of bar, parity and
    timeout_ns is true; `header` defines wait_bounded."""
    build.build()
    text = f'''#include "{header}"
namespace gqa {{
__device__ int give_up_calls;
__device__ __forceinline__ bool wait_that_runs_out(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                                   unsigned int* status, unsigned long long timeout_ns) {{
  if (!({place})) return wait_bounded(bar, parity, abort_flag, status, timeout_ns);
  *abort_flag = 1u;
  atomicOr(status, 1u);  // GQA_DEV_TIMEOUT
  return false;
}}
}}  // namespace gqa
#define wait_bounded wait_that_runs_out
#include "{source}"
'''
    src = os.path.join(folder, source)
    obj, lib = src[:-3] + ".o", src[:-3] + ".so"
    with open(src, "w") as f:
        f.write(text.replace(f'#include "{source}"', f'#include "{os.path.join(build.CSRC, source)}"'))
    subprocess.run([build.nvcc(), "-c", src, "-o", obj] + build._flags(), check=True, capture_output=True, text=True)
    objs = [os.path.join(build.BUILD, s[:-3] + ".o") for s in build.SOURCES if s != source]
    subprocess.run([build.nvcc(), "-shared", "-o", lib, obj] + objs + build.ARCH, check=True, capture_output=True, text=True)
    return lib
