"""Linear attention against 64 bits where a sum hides nothing (linattn_precision.py says what is allowed and why), the
norm and rotation inside the token step with the rounding bound of each factor, and calls that overlap on different data."""
import pytest
import torch

from distilled_ssm_decode_b200 import ops
from linattn_precision import one_product_values, row_excess, state_excess
from linattn_util import U, decays, inputs, rotate_bound

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from distilled_ssm_decode_b200 import build
    build.build()


def _tc_call(q, k, v, *a, **kw):
    assert ops.linattn_prefill_uses_tensor_cores(q, k, v)
    r = ops.linattn_prefill(q, k, v, *a, **kw)
    assert r.error() == 0
    return r


# (1, 3000, ...) and (2, 5000, ...) are cut into segments; 64- and 128-column tiles; heads that leave lanes and columns idle
@pytest.mark.parametrize("B,L,Hk,dk,dv", [(2, 9, 2, 64, 64), (2, 33, 2, 128, 128), (2, 128, 2, 64, 64), (80, 100, 2, 128, 128),
                                          (2, 129, 2, 96, 80), (40, 300, 4, 64, 128), (1, 3000, 2, 64, 64), (2, 5000, 1, 128, 64)])
@pytest.mark.parametrize("decay", [1.0, 1 - 2.0 ** -9, 0.9, 0.7])
def test_state_keeps_every_term_of_a_weighted_key(B, L, Hk, dk, dv, decay):
    q, k, _, _ = inputs(B, L, Hk, Hk, dk, dv, BF16, L)
    q, k, v = q.cuda(), k.cuda(), one_product_values(B, L, Hk, dv, L).cuda()
    dec = decays(Hk, decay).cuda()
    _, st = _tc_call(q, k, v, dec)
    assert state_excess(st, k, v, dec) <= 1


@pytest.mark.parametrize("B,L,H,Hk,dk,dv", [(2, 9, 2, 2, 64, 64), (2, 129, 4, 2, 128, 128), (3, 300, 4, 4, 64, 64), (80, 260, 2, 2, 128, 128),
                                            (2, 300, 6, 2, 96, 80), (40, 140, 4, 4, 64, 128), (1, 3000, 4, 2, 64, 64)])
@pytest.mark.parametrize("decay", ["mixed", 1.0, 1 - 2.0 ** -12, 0.875, 0.8])
@pytest.mark.parametrize("padded", [False, True])
def test_no_row_of_the_outputs_loses_a_token(B, L, H, Hk, dk, dv, decay, padded):
    q, k, v, S = (t.cuda() for t in inputs(B, L, H, Hk, dk, dv, BF16, L + H, carry=True))
    S = S / 3
    dec = decays(Hk, decay).cuda()
    lens = torch.tensor([(L, L - 1, 1, 0, L // 2)[b % 5] for b in range(B)], dtype=torch.int32, device="cuda") if padded else None
    o, _ = _tc_call(q, k, v, dec, scale=0.125, lens=lens, state_in=S)
    assert row_excess(o, q, k, v, dec, 0.125, lens, S) <= 1


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hd,rot,interleaved", [(64, 64, False), (72, 32, True), (18, 6, False), (256, 256, False)])
@pytest.mark.parametrize("H,Hk", [(2, 2), (9, 1)])
def test_decode_with_norm_and_rotation_to_the_roundings(dtype, hd, rot, interleaved, H, Hk):
    """The bounds of the rotated factors (rotate_bound, fp32: they are not rounded to the activations' type) carried through
    S' = g S + k v^T (2 roundings) and o = scale S'^T q (hd products and sums, scale), and o's own rounding."""
    B, dv = 4, 40
    q, k, v, S = (t.cuda() for t in inputs(B, 1, H, Hk, hd, dv, dtype, hd + 1, carry=True))
    q, k, v = q[:, 0], k[:, 0], v[:, 0]
    g = torch.Generator().manual_seed(2)
    wq, wk = ((1 + 0.2 * torch.randn(hd, generator=g)).cuda() for _ in range(2))
    f = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    prep = ops.QKPrep(wq, wk, 1e-6, f, interleaved)
    dec = decays(Hk).cuda()
    pos = torch.tensor([0, 5, 70001, 3], dtype=torch.int32, device="cuda")
    q64, tq = rotate_bound(q, wq, 1e-6, f, pos, interleaved, F32)
    k64, tk = rotate_bound(k, wk, 1e-6, f, pos, interleaved, F32)
    v64, old = v.double(), dec.double()[:, None, None] * S.double()
    new = old + k64[..., :, None] * v64[..., None, :]
    ts = tk[..., :, None] * v64.abs()[..., None, :] + 2 * U * (old.abs() + (k64[..., :, None] * v64[..., None, :]).abs())
    heads = lambda x: x.unflatten(1, (Hk, H // Hk))
    o64 = 0.5 * (heads(q64) @ new).flatten(1, 2)
    to = 0.5 * (heads(tq) @ new.abs() + heads(q64.abs()) @ ts + (hd + 1) * U * (heads(q64.abs()) @ new.abs())).flatten(1, 2)
    to = 1.01 * to + (2.0 ** -8 if dtype == BF16 else U) * o64.abs() * 1.01
    o = ops.linattn_decode_step(q, k, v, dec, S, scale=0.5, prep=prep, positions=pos)
    assert bool(((S.double() - new).abs() <= 1.01 * ts).all()), float(((S.double() - new).abs() / ts).max())
    assert bool(((o.double() - o64).abs() <= to).all()), float(((o.double() - o64).abs() / to).max())


def _calls(dtype, seed):
    q, k, v, S = (t.cuda() for t in inputs(2, 3000, 4, 2, 64, 64, dtype, seed, carry=True))
    dec = decays(2).cuda()
    outs = []

    def step():
        r = ops.linattn_prefill(q, k, v, dec, state_in=S)              # cut into segments: states pass through the workspace
        st = r[1].clone()
        outs[:] = [r[0], r[1], ops.linattn_decode_step(q[:, 0], k[:, 0], v[:, 0], dec, st), st]
    return step, outs


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_two_streams_at_once_on_different_data(dtype):
    calls = [_calls(dtype, 41), _calls(dtype, 42)]
    want = []
    for step, outs in calls:
        step()
        torch.cuda.synchronize()
        want.append([x.clone() for x in outs])
    assert not torch.equal(want[0][1], want[1][1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, (step, _) in zip(streams, calls):
            with torch.cuda.stream(s):
                step()
    torch.cuda.synchronize()
    for (_, outs), w in zip(calls, want):
        for a, b in zip(outs, w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_two_graphs_replayed_at_once_on_different_data(dtype):
    calls = [_calls(dtype, 43), _calls(dtype, 44)]
    want, graphs = [], []
    for step, outs in calls:
        step()
        torch.cuda.synchronize()
        want.append([x.clone() for x in outs])
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, outs), w in zip(calls, want):
        for a, b in zip(outs, w):
            assert torch.equal(a, b)
