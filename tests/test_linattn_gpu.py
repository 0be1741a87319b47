"""Linear attention with a decay for each head (prompt and single-token forms) and the norm and
rotation of queries and keys, against their definitions in fp64 (bounds in linattn_util.py)."""
import pytest
import torch

from distilled_ssm_decode_b200 import ops
from linattn_util import check, decays, inputs, reference, rotate64, rotate_bound

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from distilled_ssm_decode_b200 import build
    build.build()


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _fused_cuda(q, k, v):
    """The same slices of one projection, on the device."""
    base = q._base.cuda()
    out, at = [], 0
    for t in (q, k, v):
        n = t.shape[2] * t.shape[3]
        out.append(base[..., at:at + n].unflatten(-1, t.shape[2:]))
        at += n
    return out


def _run(B, L, H, Hk, dk, dv, dtype, *, lens=None, carry=False, fused=False, kind="mixed", seed=0, scale=0.25):
    q, k, v, S = inputs(B, L, H, Hk, dk, dv, dtype, seed + L * 31 + dk, fused, carry)
    dec = decays(Hk, kind).cuda()
    qd, kd, vd = _fused_cuda(q, k, v) if fused else _cuda(q, k, v)
    Sd = None if S is None else S.cuda()
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    if lens is not None:          # what lies behind a row's tokens must not matter
        for b, n in enumerate(lens):
            for t in (qd, kd, vd):
                t[b, n:] = float("nan")
    o = torch.full((B, L, H, dv), 7.0, dtype=dtype, device="cuda")
    dims = (dtype, B, L, H, Hk, dk, dv)
    ws = torch.full((ops.linattn_prefill_workspace_bytes(*dims),), 255, dtype=torch.uint8, device="cuda")
    o, st = ops.linattn_prefill(qd, kd, vd, dec, scale=scale, lens=ln, state_in=Sd, o=o, workspace=ws)
    tc = ops.linattn_prefill_uses_tensor_cores(qd, kd, vd, o)
    assert tc == (dtype == BF16 and dk <= 128 and dk % 8 == 0 and dv % 8 == 0 and (L > 8 or L * H // Hk > 24))
    if tc:
        assert ops.linattn_error(ws, *dims) == 0, "a wait gave up"
    ref = reference(qd, kd, vd, dec, scale, ln, Sd)
    rows = None
    if lens is not None:
        rows = (torch.arange(L, device="cuda")[None] < ln[:, None])[..., None, None]
        assert bool((o.masked_select(~rows.expand_as(o)) == 7.0).all()), "rows behind a sequence were written"
    check(o, st, ref, L, dk, dtype, tc, rows)
    return qd, kd, vd, dec, Sd, o, st


@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prefill_lengths(L, dtype):
    _run(2, L, 3, 3, 64, 64, dtype, carry=L % 2 == 0)


@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 5), (8, 8), (17, 33), (24, 72), (64, 65), (96, 80), (128, 128), (72, 200),
                                   (128, 256), (130, 31), (192, 96), (256, 128)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prefill_widths(dk, dv, dtype):
    _run(2, 70, 2, 2, dk, dv, dtype, carry=True)


@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 1), (6, 2), (16, 8)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prefill_shared_heads_of_one_projection(H, Hk, dtype):
    _run(2, 150, H, Hk, 64, 48, dtype, fused=True, carry=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (96, 80), (20, 12)])
def test_prefill_padded_batch(dtype, dk, dv):
    _run(6, 200, 4, 2, dk, dv, dtype, lens=[200, 0, 1, 128, 129, 77], carry=True)
    _run(3, 40, 2, 2, dk, dv, dtype, lens=[0, 39, 40])


@pytest.mark.parametrize("kind", [0.0, 1.0, 0.5, 1e-30, 1 - 2.0 ** -12])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prefill_decays(kind, dtype):
    _run(1, 260, 2, 2, 64, 64, dtype, kind=kind, carry=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,H,d", [(1, 3000, 2, 64), (1, 4096, 1, 128), (2, 2500, 3, 32)])
def test_prefill_long_sequences_are_split(dtype, B, L, H, d):
    _run(B, L, H, H, d, d, dtype, carry=True)
    _run(B, L, H, H, d, d, dtype, lens=[L - 700 * i - 1 for i in range(B)])


# Work that fills the GPU in 128-column tiles, whole and cut, with query heads that share a state; and 64-column tiles of
# wide values where it does not.
@pytest.mark.parametrize("B,L,H,Hk,dk,dv", [(40, 150, 2, 2, 128, 128), (2, 2100, 8, 8, 128, 128), (38, 260, 4, 2, 64, 128),
                                            (40, 140, 6, 2, 104, 96), (1, 1500, 4, 2, 128, 192), (2, 300, 3, 1, 64, 128),
                                            (150, 130, 1, 1, 32, 64)])
@pytest.mark.parametrize("padded", [False, True])
def test_prefill_tiles_and_cuts(B, L, H, Hk, dk, dv, padded):
    lens = [(L, 0, 1, L - 1, 129, L // 2)[b % 6] for b in range(B)] if padded else None
    _run(B, L, H, Hk, dk, dv, BF16, lens=lens, carry=True, fused=True)


@pytest.mark.parametrize("L,H,Hk", [(1, 25, 1), (5, 10, 2), (8, 16, 4), (8, 3, 1), (8, 4, 1), (9, 1, 1), (1, 2, 2)])
def test_prefill_short_prompts_on_either_route(L, H, Hk):
    _run(3, L, H, Hk, 64, 128, BF16, carry=True)
    _run(200, L, H, Hk, 128, 128, BF16, lens=[b % (L + 1) for b in range(200)], carry=True)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_prefill_cut_prompt_with_short_rows(dk, dv):
    """A long padded prompt, cut, whose rows are mostly a few tokens: chunks of one piece of keys follow each other."""
    n = 48
    lens = [2049] + [(i * 7) % 37 for i in range(n - 1)]
    _run(n, 2049, 2, 2, dk, dv, BF16, lens=lens, carry=True)
    _run(2, 2049, 1, 1, dk, dv, BF16, lens=[2049, 3])


@pytest.mark.parametrize("kind", [0.75, 0.7499, 0.76])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prefill_decays_around_the_scaling_rule(kind, dtype):
    _run(2, 200, 4, 2, 64, 72, dtype, kind=kind, carry=True)


@pytest.mark.parametrize("decay", [1.0, 0.76, 0.3])
def test_prefill_large_values(decay):
    """Scores up to 1e9 and outputs beyond 1e12 stay finite and within the bounds."""
    q, k, v, _ = inputs(1, 140, 2, 2, 64, 64, BF16, 9)
    q, k, v = _cuda(q * 1e4, k * 1e4, v * 1e3)
    dec = decays(2, decay).cuda()
    o, st = ops.linattn_prefill(q, k, v, dec, scale=0.125)
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(st).all())
    check(o, st, reference(q, k, v, dec, 0.125), 140, 64, BF16, True)


def test_prefill_chunks_follow_each_other():
    """A prompt taken in pieces, each from the state of the one before, is the prompt taken whole (state: fp32 sums
    in another grouping; outputs: the bounds of both)."""
    q, k, v, S = _cuda(*inputs(2, 700, 4, 2, 64, 64, BF16, 31, carry=True))
    dec = decays(2).cuda()
    ref = reference(q, k, v, dec, 0.25, None, S)
    outs, st, t = [], S.clone(), 0
    for n in (1, 127, 128, 200, 244):
        x = [y[:, t:t + n].contiguous() for y in (q, k, v)]
        o, st = ops.linattn_prefill(*x, dec, scale=0.25, state_in=st, state=st)
        outs.append(o)
        t += n
    check(torch.cat(outs, 1), st, ref, 700, 64, BF16, True)


def test_prefill_lengths_outside_the_row_are_clamped():
    q, k, v, _ = _cuda(*inputs(2, 40, 2, 2, 32, 32, F32, 3))
    dec = decays(2).cuda()
    o1, s1 = ops.linattn_prefill(q, k, v, dec, lens=torch.tensor([-5, 1000], dtype=torch.int32, device="cuda"))
    o2, s2 = ops.linattn_prefill(q, k, v, dec, lens=torch.tensor([0, 40], dtype=torch.int32, device="cuda"))
    assert torch.equal(o1, o2) and torch.equal(s1, s2)
    assert not o1[0].any()


@pytest.mark.parametrize("B,L", [(2, 100), (1, 3000)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prefill_state_in_place_and_repeatable(B, L, dtype):
    """state_in may be state_out; the same call twice gives the same bits."""
    q, k, v, S = _cuda(*inputs(B, L, 2, 2, 64, 64, dtype, 5, carry=True))
    dec = decays(2).cuda()
    o1, s1 = ops.linattn_prefill(q, k, v, dec, state_in=S)
    o2, s2 = ops.linattn_prefill(q, k, v, dec, state_in=S, state=S)
    assert s2.data_ptr() == S.data_ptr()
    assert torch.equal(o1, o2) and torch.equal(s1, s2)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prefill_empty_problems(dtype):
    dec = decays(2).cuda()
    e = lambda *s: torch.empty(s, dtype=dtype, device="cuda")
    S = torch.randn((3, 2, 8, 8), device="cuda")
    o, st = ops.linattn_prefill(e(3, 0, 4, 8), e(3, 0, 2, 8), e(3, 0, 2, 8), dec)
    assert o.shape == (3, 0, 4, 8) and not st.any()
    _, st = ops.linattn_prefill(e(3, 0, 4, 8), e(3, 0, 2, 8), e(3, 0, 2, 8), dec, state_in=S)
    assert torch.equal(st, S)
    _, st = ops.linattn_prefill(e(3, 0, 4, 8), e(3, 0, 2, 8), e(3, 0, 2, 8), dec, state_in=S, state=S)
    assert st.data_ptr() == S.data_ptr()
    o, st = ops.linattn_prefill(e(0, 5, 4, 8), e(0, 5, 2, 8), e(0, 5, 2, 8), dec)
    assert o.numel() == 0 and st.numel() == 0


@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 5), (17, 30), (64, 64), (72, 104), (128, 128), (256, 200), (128, 33)])
@pytest.mark.parametrize("H,Hk", [(2, 2), (6, 2), (20, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_step(dk, dv, H, Hk, dtype):
    for B, fused in ((1, False), (5, True)):
        q, k, v, S = inputs(B, 1, H, Hk, dk, dv, dtype, dk * 7 + dv, fused, True)
        qd, kd, vd = _fused_cuda(q, k, v) if fused else _cuda(q, k, v)
        Sd, dec = S.cuda(), decays(Hk).cuda()
        ref = reference(qd, kd, vd, dec, 0.5, None, Sd)
        o = ops.linattn_decode_step(qd[:, 0], kd[:, 0], vd[:, 0], dec, Sd, scale=0.5)
        check(o[:, None], Sd, ref, 1, dk, dtype, False)


def test_decode_large_batch():
    q, k, v, S = _cuda(*inputs(300, 1, 2, 2, 128, 128, BF16, 11, False, True))
    dec = decays(2).cuda()
    ref = reference(q, k, v, dec, 1.0, None, S)
    o = ops.linattn_decode_step(q[:, 0], k[:, 0], v[:, 0], dec, S)
    check(o[:, None], S, ref, 1, 128, BF16, False)


def _prep(hd, rot, interleaved, weights=True, norm=True, eps=1e-6, seed=0):
    g = torch.Generator().manual_seed(seed)
    w = [(1 + 0.2 * torch.randn(hd, generator=g)).cuda() if weights else None for _ in range(2)]
    f = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().cuda() if rot else None
    return w[0], w[1], f, ops.QKPrep(w[0], w[1], eps, f, interleaved, norm)


@pytest.mark.parametrize("hd,rot", [(2, 2), (2, 0), (10, 4), (16, 8), (40, 20), (64, 64), (80, 32), (128, 128), (128, 0), (96, 2),
                                    (256, 256), (254, 130)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_qk_norm_rotate(hd, rot, interleaved, dtype):
    for B, L, H, Hk, fused in ((1, 1, 1, 1, False), (2, 37, 3, 1, True), (3, 5, 4, 4, False)):
        q, k, v, _ = inputs(B, L, H, Hk, hd, 2, dtype, hd + rot, fused)
        q, k = (_fused_cuda(q, k, v) if fused else _cuda(q, k, v))[:2]
        wq, wk, f, prep = _prep(hd, rot, interleaved)
        pos = (torch.randint(0, 1 << 30, (B, L), dtype=torch.int32) - (1 << 20)).cuda()
        for p, kw in ((pos, dict(positions=pos)),
                      (torch.arange(1000003, 1000003 + L, device="cuda").expand(B, L), dict(pos0=1000003))):
            qo, ko = ops.qk_norm_rotate(q, k, prep, **kw)
            for x, y, w in ((q, qo, wq), (k, ko, wk)):
                want, tol = rotate_bound(x, w, 1e-6, f, p, interleaved, dtype)
                assert bool(((y.double() - want).abs() <= tol).all()), float(((y.double() - want).abs() - tol).max())


# Every vector width (8, 4, none) and group of lanes, many heads (several rounds of a block), several tokens to a block, and
# bases and row strides that fit no vector.
@pytest.mark.parametrize("B,L,H,Hk,hd,rot", [(1, 5, 3, 1, 80, 40), (2, 700, 2, 1, 24, 8), (1, 3, 2, 2, 12, 4), (1, 3, 100, 1, 128, 128),
                                             (3, 500, 2, 2, 256, 8), (1, 1300, 7, 2, 64, 32), (2, 601, 1, 3, 40, 20),
                                             (1, 2, 1, 70, 256, 256), (5, 333, 4, 4, 96, 0)])
@pytest.mark.parametrize("shift", [0, 4, 1])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_qk_vectors(B, L, H, Hk, hd, rot, shift, interleaved, dtype):
    g = torch.Generator().manual_seed(hd + rot + shift)
    x = torch.randn((B, L, (H + Hk) * hd + 2 * shift), generator=g).to(dtype).cuda()
    q = x[..., shift:shift + H * hd].unflatten(-1, (H, hd))
    k = x[..., shift + H * hd:shift + (H + Hk) * hd].unflatten(-1, (Hk, hd))
    wq, wk, f, prep = _prep(hd, rot, interleaved)
    pos = torch.randint(0, 1 << 20, (B, L), generator=g, dtype=torch.int32).cuda()
    qo, ko = ops.qk_norm_rotate(q, k, prep, positions=pos)
    for a, y, w in ((q, qo, wq), (k, ko, wk)):
        want, tol = rotate_bound(a, w, 1e-6, f, pos, interleaved, dtype)
        assert bool(((y.double() - want).abs() <= tol).all()), float(((y.double() - want).abs() - tol).max())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_qk_options_and_in_place(dtype):
    x = torch.randn((2, 33, 5 * 64 + 40), device="cuda").to(dtype)
    q, k = x[..., :192].unflatten(-1, (3, 64)), x[..., 192:320].unflatten(-1, (2, 64))
    pos = torch.arange(33, device="cuda").expand(2, 33)
    for norm, weights, rot in ((False, False, 64), (True, False, 0), (True, True, 32), (False, True, 0)):
        wq, wk, f, prep = _prep(64, rot, False, weights, norm)
        qo, ko = ops.qk_norm_rotate(q, k, prep)
        for a, y, w in ((q, qo, wq), (k, ko, wk)):
            want, tol = rotate_bound(a, w, 1e-6, f, pos, False, dtype, norm)
            assert bool(((y.double() - want).abs() <= tol).all())
        z = x.clone()
        zq, zk = z[..., :192].unflatten(-1, (3, 64)), z[..., 192:320].unflatten(-1, (2, 64))
        ops.qk_norm_rotate(zq, zk, prep, q_out=zq, k_out=zk)
        assert torch.equal(zq, qo) and torch.equal(zk, ko)
        assert torch.equal(z[..., 320:], x[..., 320:])


def test_qk_zero_rows_and_one_sided():
    wq, wk, f, prep = _prep(32, 32, False)
    q = torch.zeros((2, 3, 2, 32), device="cuda")
    none = torch.empty((2, 3, 0, 32), device="cuda")
    qo, ko = ops.qk_norm_rotate(q, none, prep)
    assert not qo.any() and ko.numel() == 0
    qo, ko = ops.qk_norm_rotate(none, q, prep)
    assert not ko.any() and qo.numel() == 0
    e = torch.empty((2, 0, 2, 32), device="cuda")
    assert ops.qk_norm_rotate(e, e, prep)[0].shape == (2, 0, 2, 32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hd,rot,interleaved", [(64, 64, False), (72, 32, True), (18, 6, False), (256, 256, False)])
@pytest.mark.parametrize("H,Hk", [(2, 2), (9, 1)])
def test_decode_with_norm_and_rotation(dtype, hd, rot, interleaved, H, Hk):
    B, dv = 4, 40
    q, k, v, S = inputs(B, 1, H, Hk, hd, dv, dtype, hd, True, True)
    q, k, v = _fused_cuda(q, k, v)
    S, dec = S.cuda(), decays(Hk).cuda()
    wq, wk, f, prep = _prep(hd, rot, interleaved)
    pos = torch.tensor([0, 5, 70001, 3], dtype=torch.int32, device="cuda")
    for p, kw in ((pos, dict(positions=pos)), (torch.full((B,), 1234, device="cuda"), dict(pos0=1234))):
        qn = rotate64(q[:, 0], wq, 1e-6, f, p, interleaved)
        kn = rotate64(k[:, 0], wk, 1e-6, f, p, interleaved)
        o_ref, s_ref, mo, ms = reference(qn[:, None], kn[:, None], v, dec, 0.5, None, S)
        S2 = S.clone()
        o = ops.linattn_decode_step(q[:, 0], k[:, 0], v[:, 0], dec, S2, scale=0.5, prep=prep, **kw)
        # the norm and rotation add hd + 26 roundings of at most twice the entries' magnitude on each side
        extra = 4 * (hd + 26)
        check(o[:, None], S2, (o_ref, s_ref, mo * 1.5, ms * 1.5), 8 * extra, hd, dtype, False)


@pytest.mark.parametrize("dtype,tol", [(F32, 2e-5), (BF16, 2.0 ** -7)])
def test_prompt_then_tokens(dtype, tol):
    """As a layer uses them: norm and rotation of the prompt, the prompt form, then tokens whose norm and rotation run
    inside the step -- against the whole sequence in fp64.  bf16 rounds queries and keys of the prompt once more (two
    factors, 2^-8 / sqrt(3) each in rms), its operands and its outputs: sqrt(4 / 3) 2^-8 < 2^-7."""
    B, L, T, H, Hk, dk, dv = 3, 200, 5, 4, 2, 64, 48
    g = torch.Generator().manual_seed(1)
    x = torch.randn((B, L + T, (H + Hk) * dk + Hk * dv), generator=g).to(dtype).cuda()
    q = x[..., :H * dk].unflatten(-1, (H, dk))
    k = x[..., H * dk:(H + Hk) * dk].unflatten(-1, (Hk, dk))
    v = x[..., (H + Hk) * dk:].unflatten(-1, (Hk, dv))
    wq, wk, f, prep = _prep(dk, dk, False)
    dec = torch.tensor([1 - 2.0 ** -5, 1 - 2.0 ** -7], device="cuda")
    lens = [200, 131, 1]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    xp = x[:, :L].contiguous()
    sl = lambda a, lo, hi, h: a[..., lo:hi].unflatten(-1, (h, -1))
    qp, kp, vp = sl(xp, 0, H * dk, H), sl(xp, H * dk, (H + Hk) * dk, Hk), sl(xp, (H + Hk) * dk, x.shape[-1], Hk)
    qn, kn = ops.qk_norm_rotate(qp, kp, prep)
    o, S = ops.linattn_prefill(qn, kn, vp, dec, scale=dk ** -0.5, lens=n)
    outs = []
    for t in range(T):
        r = n.long() + t
        b = torch.arange(B, device="cuda")
        outs.append(ops.linattn_decode_step(q[b, r], k[b, r], v[b, r], dec, S, scale=dk ** -0.5, prep=prep,
                                            positions=n + t))
    pos = torch.arange(L + T, device="cuda").expand(B, L + T)
    q64, k64 = rotate64(q, wq, 1e-6, f, pos, False), rotate64(k, wk, 1e-6, f, pos, False)
    for b in range(B):
        m = lens[b] + T
        o_ref, s_ref, _, _ = reference(q64[b:b + 1, :m], k64[b:b + 1, :m], v[b:b + 1, :m].double(), dec, dk ** -0.5)
        got = torch.cat([o[b, :lens[b]], torch.stack([y[b] for y in outs])]).double()
        assert float((got - o_ref[0]).norm() / o_ref[0].norm()) <= tol
        assert float((S[b].double() - s_ref[0]).norm() / s_ref[0].norm()) <= tol


def _calls(dtype):
    q, k, v, S = _cuda(*inputs(2, 300, 4, 2, 64, 64, dtype, 21, carry=True))
    dec = decays(2).cuda()
    prep = _prep(64, 64, False)[3]
    ws = torch.empty(ops.linattn_prefill_workspace_bytes(dtype, 2, 300, 4, 2, 64, 64), dtype=torch.uint8, device="cuda")
    qo, ko, o, st = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty_like(S)
    od = torch.empty((2, 4, 64), dtype=dtype, device="cuda")

    def step():
        ops.qk_norm_rotate(q, k, prep, q_out=qo, k_out=ko)
        ops.linattn_prefill(qo, ko, v, dec, state_in=S, o=o, state=st, workspace=ws)
        ops.linattn_decode_step(q[:, 0], k[:, 0], v[:, 0], dec, st, prep=prep, pos0=300, o=od)
    return step, (q, k, v, S), (o, st, od)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_and_replayed_on_new_inputs(dtype):
    step, ins, outs = _calls(dtype)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in ins:
        x.copy_(torch.randn_like(x))
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in outs]
    step()
    torch.cuda.synchronize()
    for a, b in zip(got, outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_two_streams_at_once(dtype):
    (s1, _, o1), (s2, _, o2) = _calls(dtype), _calls(dtype)
    s1()
    want = [x.clone() for x in o1]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for st, f in zip(streams, (s1, s2)):
            with torch.cuda.stream(st):
                f()
    torch.cuda.synchronize()
    for o in (o1, o2):
        for a, b in zip(o, want):
            assert torch.equal(a, b)
