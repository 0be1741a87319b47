"""Linear attention at the ends of fp32's range: whatever the decay, sums that fp32 holds come out finite, and small
ones keep their accuracy (fp64 definitions and bounds of linattn_util.py)."""
import pytest
import torch

from distilled_ssm_decode_b200 import ops
from linattn_util import check, decays, inputs, reference

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from distilled_ssm_decode_b200 import build
    build.build()


# Scores q.k of up to 3e35 (64 products of entries around 8e16; the sums with values around 1e-10 and their absolute
# values stay below 1e28), and of about 1e-29.
@pytest.mark.parametrize("qk,v", [(8e16, 1e-10), (1e-15, 1.0)])
@pytest.mark.parametrize("decay", [0.3, 0.75, 0.8, 0.8749, 0.875, 0.92, 1 - 2.0 ** -9, 1.0])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scores_at_the_ends_of_the_range(dtype, decay, qk, v):
    q, k, x, _ = inputs(2, 300, 2, 2, 64, 64, dtype, 17)
    q, k, x = (q * qk).cuda(), (k * qk).cuda(), (x * v).cuda()
    dec = decays(2, decay).cuda()
    o, st = ops.linattn_prefill(q, k, x, dec, scale=0.125)
    assert ops.linattn_prefill_uses_tensor_cores(q, k, x) == (dtype == BF16)
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(st).all())
    check(o, st, reference(q, k, x, dec, 0.125), 300, 64, dtype, dtype == BF16)
