"""gqa_prefill_backward's refusals, each for its own reason: the arguments they start from pass every check, and nothing of
them stands on anything else; and the workspace that a call of a few tokens needs."""
import ctypes

import pytest
import torch

FAKE = 1 << 20  # a 256-byte-aligned non-null address; never dereferenced
STEP = 1 << 32  # between tensors: more than the workspace


@pytest.fixture(scope="module")
def lib():
    from gqa_flash_attention_prefill_gb300 import build
    import gqa_flash_attention_prefill_gb300 as pkg
    return pkg.load(build.build())


def size_of(lib, *shape):
    size = ctypes.c_size_t(0)
    assert lib.gqa_prefill_backward_workspace(*shape, ctypes.byref(size)) == 0
    return size.value


def call(lib, **over):
    a = dict(q=FAKE, k=FAKE + STEP, v=FAKE + 2 * STEP, cu=FAKE + 3 * STEP, pre=FAKE + 4 * STEP, kvi=FAKE + 5 * STEP, B=1, total_q=16,
             total_kv=16, hq=8, hkv=2, d=64, dtype=1, scale=0.125, window=0, out=FAKE + 6 * STEP, lse=FAKE + 7 * STEP,
             dout=FAKE + 8 * STEP, dlse=FAKE + 14 * STEP, sinks=FAKE + 15 * STEP, dq=FAKE + 9 * STEP, dk=FAKE + 10 * STEP,
             dv=FAKE + 11 * STEP, dsinks=FAKE + 16 * STEP, ws=FAKE + 12 * STEP, size=None, stream=None)
    a.update(over)
    if a["size"] is None:
        a["size"] = size_of(lib, a["B"], a["total_q"], a["total_kv"], a["hq"], a["hkv"], a["d"], a["dtype"])
    return lib.gqa_prefill_backward(*a.values())


Q, KV, LSE, H = 2 * 16 * 8 * 64, 2 * 16 * 2 * 64, 4 * 16 * 8, 4 * 8  # bytes


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real: no launch may follow")
def test_the_arguments_themselves_pass(lib):
    for d, hq, hkv in ((64, 8, 2), (128, 8, 2), (256, 8, 2), (64, 128, 1)):
        for dtype in (0, 1):
            assert call(lib, d=d, hq=hq, hkv=hkv, dtype=dtype) == -3  # no device
            assert call(lib, d=d, hq=hq, hkv=hkv, dtype=dtype, dlse=None, sinks=None, dsinks=None, window=7) == -3
    # What just does not overlap passes too.
    at = FAKE + 20 * STEP
    assert call(lib, dq=at, q=at + Q, out=at - Q) == -3
    assert call(lib, dk=at, dv=at + KV, dsinks=at + 2 * KV, ws=at + 2 * KV + 256) == -3


BASE = dict(q=(0, Q), k=(1, KV), v=(2, KV), cu=(3, 8), pre=(4, 4), kvi=(5, 8), out=(6, Q), lse=(7, LSE), dout=(8, Q), dlse=(14, LSE),
            sinks=(15, H), dq=(9, Q), dk=(10, KV), dv=(11, KV), dsinks=(16, H))


@pytest.mark.parametrize("result", ["dq", "dk", "dv", "dsinks", "ws"])
@pytest.mark.parametrize("other", sorted(BASE))
def test_overlaps(lib, result, other):
    """Each result over each other tensor: at its start, and by its last 16 bytes (4 of the small ones)."""
    if result == other:
        return
    at, size = BASE[other]
    start = FAKE + at * STEP
    step = 256 if result == "ws" else 16 if result in ("dq", "dk", "dv") else 4
    assert call(lib, **{result: start}) == -1
    last = (size - 1) // step * step  # the last aligned address inside
    assert call(lib, **{result: start + last}) == -1


def test_workspace_overlaps(lib):
    size = size_of(lib, 1, 16, 16, 8, 2, 64, 1)
    assert call(lib, dq=FAKE + 12 * STEP + size - 256) == -1
    assert call(lib, size=size - 1) == -1


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (64, 64, 8), (128, 32, 8), (256, 8, 4), (64, 128, 1)])
def test_a_call_that_cuts_nothing_needs_no_room_for_parts(lib, d, hq, hkv):
    """A unit of at most 8 tiles is never cut: an fp32 part of one alone is 128 rows of d values for each KV head."""
    g = hq // hkv
    n = 128 if d == 128 else 64
    tokens = 8 * n // g
    part = 4 * 128 * d * hkv
    few, many = (size_of(lib, 1, t, t, hq, hkv, d, 1) for t in (tokens, 32 * tokens))
    rows = 8 * n
    # A record for each of the units, statistics of 8 bytes a packed row, sums of the sinks' tiles, and the header.
    lists = 64 * (rows // 128 + 2 * (8 * n // 128 + 1) + 3) + 8 * hkv * (rows + 128) + 4 * hq * (rows // 128 + 1)
    assert few <= lists + 4096 and few < many
    assert many >= 2 * part
