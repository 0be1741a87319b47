"""Values that are not finite in a sequence's own tokens: where they get, and that everything else keeps its bits."""
import pytest
import torch

from distilled_ssm_decode_b200 import ops
from linattn_util import decays, inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from distilled_ssm_decode_b200 import build
    build.build()


@pytest.mark.parametrize("what", ["q", "k", "v"])
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("L", [300, 1500])              # in one piece, and cut into segments
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_value_that_is_not_finite_stays_in_its_place(dtype, L, bad, what):
    B, H, Hk, d = 2, 4, 2, 64
    x = dict(zip("qkvS", (t.cuda() for t in inputs(B, L, H, Hk, d, d, dtype, 6, carry=True))))
    dec = torch.tensor([1 - 2.0 ** -6, 0.8], device="cuda")
    call = lambda: ops.linattn_prefill(x["q"], x["k"], x["v"], dec, scale=0.25, state_in=x["S"])
    o0, s0 = call()
    b, t, h, e = 0, 150, 1, 5
    x[what][b, t, h, e] = bad
    o1, s1 = call()
    t0 = t - t % 128                                     # of a chunk's tokens, earlier ones may be reached
    hit_o, hit_s = torch.zeros_like(o0, dtype=torch.bool), torch.zeros_like(s0, dtype=torch.bool)
    may_o = hit_o.clone()
    G = H // Hk
    if what == "q":
        hit_o[b, t, h] = True
    elif what == "k":
        hit_s[b, h, e] = True
        hit_o[b, t:, h * G:(h + 1) * G] = True
        may_o[b, t0:t, h * G:(h + 1) * G] = True
    else:
        hit_s[b, h, :, e] = True
        hit_o[b, t:, h * G:(h + 1) * G, e] = True
        may_o[b, t0:t, h * G:(h + 1) * G, e] = True
    assert not torch.isfinite(o1[hit_o]).any() and not torch.isfinite(s1[hit_s]).any()
    assert torch.equal(o1[~hit_o & ~may_o], o0[~hit_o & ~may_o])
    assert torch.equal(s1[~hit_s], s0[~hit_s])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_keeps_a_value_that_is_not_finite_in_its_place(dtype):
    q, k, v, S = (t.cuda() for t in inputs(2, 1, 4, 2, 64, 64, dtype, 7, carry=True))
    dec = decays(2).cuda()
    S0, S1 = S.clone(), S.clone()
    o0 = ops.linattn_decode_step(q[:, 0], k[:, 0], v[:, 0], dec, S0)
    v[1, 0, 0, 9] = INF
    o1 = ops.linattn_decode_step(q[:, 0], k[:, 0], v[:, 0], dec, S1)
    hit_s, hit_o = torch.zeros_like(S, dtype=torch.bool), torch.zeros_like(o0, dtype=torch.bool)
    hit_s[1, 0, :, 9] = True
    hit_o[1, :2, 9] = True
    assert bool(torch.isinf(S1[hit_s]).all()) and not torch.isfinite(o1[hit_o]).any()
    assert torch.equal(S1[~hit_s], S0[~hit_s]) and torch.equal(o1[~hit_o], o0[~hit_o])
