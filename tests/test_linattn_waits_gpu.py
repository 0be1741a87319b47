"""The bounded waits of the linear-attention prompt kernel: a wait that runs out ends the launch with its error
words set, and leaves nothing behind for the next one."""
import pytest
import torch

from distilled_ssm_decode_b200 import ops
from linattn_util import check, decays, inputs, reference

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from distilled_ssm_decode_b200 import build
    build.build()


# One chunk and two: every copy of the launch has been issued when the wait runs out; nine: copies stop in the middle.
# (1, 3000): cut into segments, so the pass over the states stops as well.
@pytest.mark.parametrize("B,L,H,d", [(1, 100, 1, 128), (1, 256, 2, 128), (2, 1100, 80, 64), (1, 3000, 2, 64)])
def test_a_wait_that_runs_out_is_reported_and_leaves_nothing_behind(B, L, H, d):
    q, k, v, _ = (None if t is None else t.cuda() for t in inputs(B, L, H, H, d, d, BF16, L))
    dec = decays(H).cuda()
    dims = (BF16, B, L, H, H, d, d)
    ws = torch.zeros(ops.linattn_prefill_workspace_bytes(*dims), dtype=torch.uint8, device="cuda")
    with ops.linattn_hold():
        ops.linattn_prefill(q, k, v, dec, scale=0.25, workspace=ws)
        assert ops.linattn_error(ws, *dims) != 0
    o, st = ops.linattn_prefill(q, k, v, dec, scale=0.25, workspace=ws)
    assert ops.linattn_error(ws, *dims) == 0
    check(o, st, reference(q, k, v, dec, 0.25), L, d, BF16, True)


def test_the_default_call_tells_of_a_wait_that_ran_out():
    q, k, v, _ = (None if t is None else t.cuda() for t in inputs(1, 100, 2, 2, 64, 64, BF16, 3))
    dec = decays(2).cuda()
    with ops.linattn_hold():
        r = ops.linattn_prefill(q, k, v, dec)
        assert r.error() != 0
    r = ops.linattn_prefill(q, k, v, dec)
    o, st = r
    assert r.error() == 0 and len(r) == 2 and o is r[0] and st is r[1]


# fp32 takes the route without waits, cut (1, 3000) and in one piece; empty problems run nothing.
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("B,L", [(1, 3000), (2, 30), (2, 1), (2, 0), (0, 5)])
def test_every_call_that_succeeds_says_so(dtype, B, L):
    q, k, v, _ = (None if t is None else t.cuda() for t in inputs(B, L, 2, 2, 64, 64, dtype, 4))
    dec = decays(2).cuda()
    n = ops.linattn_prefill_workspace_bytes(dtype, B, L, 2, 2, 64, 64)
    ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")
    assert ops.linattn_prefill(q, k, v, dec, workspace=ws).error() == 0
    assert ops.linattn_prefill(q, k, v, dec).error() == 0
