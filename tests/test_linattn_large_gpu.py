"""Linear attention, norm and rotation where offsets pass 32 bits and where the batch is as large as the calls allow.
With a decay of 0.9 the tokens before the last 1024 reach an output by less than 0.9^1024 < 2^-155: the end of a long prompt is
the prompt of its last tokens."""
import pytest
import torch

from distilled_ssm_decode_b200 import ops
from linattn_util import check, decays, inputs, reference, rotate_bound

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from distilled_ssm_decode_b200 import build
    build.build()
    yield
    torch.cuda.empty_cache()


def _random(shape, dtype, seed):
    """Random values; the long axis repeats a block of tokens of an odd length."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(shape, dtype=dtype, device="cuda")
    n = 65521
    block = torch.randn((shape[0], min(n, shape[1]), *shape[2:]), generator=g, device="cuda").to(dtype)
    for t in range(0, shape[1], n):
        m = min(n, shape[1] - t)
        x[:, t:t + m] = block[:, :m]
    return x


@pytest.mark.parametrize("dtype,L", [(BF16, (1 << 22) + 205), (F32, (1 << 22) + 205)])
def test_prompt_of_more_than_2_31_entries(dtype, L):
    H, d, tail = 8, 64, 1024 + 300
    q, k, v = (_random((1, L, H, d), dtype, s) for s in (1, 2, 3))
    assert q.numel() > 1 << 31
    dec = decays(H, 0.9).cuda()
    r = ops.linattn_prefill(q, k, v, dec, scale=0.125)
    assert r.error() == 0
    ref = reference(*(x[:, -tail:].contiguous() for x in (q, k, v)), dec, 0.125)
    rows = (torch.arange(tail, device="cuda") >= 1024)[None, :, None, None]
    check(r[0][:, -tail:], r[1], ref, tail, d, dtype, dtype == BF16, rows)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_of_more_than_2_31_entries(dtype):
    L, H, hd = (1 << 22) + 205, 8, 64
    q = _random((1, L, H, hd), dtype, 4)
    k = q.new_empty((1, L, 0, hd))
    f = (10000.0 ** (-torch.arange(0, hd, 2, dtype=torch.float64) / hd)).float().cuda()
    w = torch.linspace(0.5, 1.5, hd, device="cuda")
    qo, _ = ops.qk_norm_rotate(q, k, ops.QKPrep(w, None, 1e-6, f), pos0=7)
    for part in (slice(0, 50), slice((1 << 22) - 50, (1 << 22) + 50), slice(L - 50, L)):
        pos = torch.arange(L, device="cuda")[part][None] + 7
        want, tol = rotate_bound(q[:, part], w, 1e-6, f, pos, False, dtype)
        assert bool(((qo[:, part].double() - want).abs() <= tol).all())


def test_decode_of_more_than_2_31_state_entries():
    B, H, d = 4100, 32, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    S = torch.randn((B, H, d, d), generator=g, device="cuda")
    assert S.numel() > 1 << 31
    q, k, v = (torch.randn((B, 1, H, d), generator=g, device="cuda").to(BF16) for _ in range(3))
    dec = decays(H).cuda()
    at = [0, 1, 4095, 4096, 4099]
    old = S[at].clone()
    o = ops.linattn_decode_step(q[:, 0], k[:, 0], v[:, 0], dec, S, scale=0.5)
    check(o[at][:, None], S[at], reference(q[at], k[at], v[at], dec, 0.5, None, old), 1, d, BF16, False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [1, 3, 9])
def test_the_largest_batch(dtype, L):
    B = 65535
    q, k, v, S = (t.cuda() for t in inputs(B, L, 2, 1, 8, 8, dtype, L, carry=True))
    dec = decays(1, 0.875).cuda()
    lens = (torch.arange(B, device="cuda") % (L + 1)).int()
    o = torch.zeros((B, L, 2, 8), dtype=dtype, device="cuda")
    r = ops.linattn_prefill(q, k, v, dec, lens=lens, state_in=S, o=o)
    assert r.error() == 0
    rows = (torch.arange(L, device="cuda")[None] < lens[:, None])[..., None, None]
    check(o, r[1], reference(q, k, v, dec, 1.0, lens, S), L, 8, dtype, dtype == BF16 and L > 8, rows)
    S1 = S.clone()
    o = ops.linattn_decode_step(q[:, 0], k[:, 0], v[:, 0], dec, S1)
    check(o[:, None], S1, reference(q[:, :1], k[:, :1], v[:, :1], dec, 1.0, None, S), 1, 8, dtype, False)
    with pytest.raises(ops.HyenaError):
        ops.linattn_prefill(*(torch.zeros((B + 1, 1, 1, 8), dtype=dtype, device="cuda") for _ in range(3)), dec)
