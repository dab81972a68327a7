"""A status word that another stream sets and clears while calls run (B200).

The word is shared by calls that can run side by side, and one of them sets it
when a wait runs out.  Whatever a CTA reads, its threads go by one value: what
is written is right, the rest is left as it was, and nothing waits for threads
that have gone.
"""
import pytest
import torch

from grouped_gemm_splits_b200 import gl
from tests.gpu_util import offsets_on_device

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


def _while_it_changes(st, calls):
    """Run the calls on one stream while another one sets and clears ``st``; milliseconds of the calls' stream."""
    run, setter = torch.cuda.Stream(), torch.cuda.Stream()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    begin.record(run)
    for call in calls:
        with torch.cuda.stream(run):
            call()
        with torch.cuda.stream(setter):
            for _ in range(3):
                st.fill_(gl.GL_DEV_TIMEOUT)
                st.zero_()
    end.record(run)
    torch.cuda.synchronize()
    return begin.elapsed_time(end)


@pytest.mark.parametrize("ragged", [False, True])
def test_cast(ragged):
    rows, cols, n = 2048, 1024, 100
    x = _rand(rows, cols)
    off, st = offsets_on_device([700, 0, 1348], rows)
    kw = dict(row_offsets=off) if ragged else dict(G=1)
    want = gl.group_quantize_mxfp8(x, colwise=True, mma_scales=True, status=st,
                                   out={"scales_c": _bytes(rows, cols, 3 if ragged else 1)}, **kw)
    outs = [{k: torch.full_like(v, 0xA5) for k, v in want.items()} for _ in range(n)]
    ms = _while_it_changes(st, [lambda o=o: gl.group_quantize_mxfp8(x, colwise=True, mma_scales=True, status=st, out=o,
                                                                    **kw) for o in outs])
    assert ms < 1500
    for o in outs:
        for key, v in o.items():
            assert ((v == want[key]) | (v == 0xA5)).all(), key
    st.zero_()
    last = gl.group_quantize_mxfp8(x, colwise=True, mma_scales=True, status=st, out=outs[0], **kw)
    assert torch.equal(last["codes_r"], want["codes_r"]) and torch.equal(last["codes_c"], want["codes_c"])


def _bytes(rows, cols, G):
    return torch.full((gl.mxfp8_scale_bytes(rows, cols, G, True, True),), 0xA5, dtype=torch.uint8, device="cuda")
