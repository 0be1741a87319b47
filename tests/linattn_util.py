"""fp64 forms of the linear-attention operators for the tests, straight from their definitions, and
the error bounds that the tests allow.

Bounds.  With u = 2^-24 (fp32) every product or sum the kernels make is off by at most u relative, so an
output is off by at most K u M, where M is the same formula with every factor replaced by its absolute
value and K the number of roundings on the longest way from an input to the output:
 - a state entry: per token its product, its weight (formed from two table entries) and its sum; per
   block of 8 tokens a decay and an update, per segment one more of each (CUDA-core route);
   so K <= 8 + 3 (8 + 2 L / 8).  On the tensor cores a chunk of 128 tokens is one sum of the bf16 terms of
   each weighted key (which together keep it to 2^-25) and one decay.  Three of a key's four terms can move a sum's
   last place; the fourth, below 2^-16 of its product, adds under 128 * 2^-16 of one rounding: K <= 8 + 3 * 128
   + 2 L / 128, taken twice because the units add with truncation.
 - an output: the dk products with a state entry and their sum, besides.
bf16 outputs add half a step, 2^-8 |o|.  On the tensor cores scores and states are rounded to bf16 as
operands: each term of the sums is off by at most 2^-8, so 2^-8 M more; and since independent roundings have
an rms of at most 2^-8 / sqrt(3) each, the 2-norm of operand and output roundings together stays below
sqrt(2 / 3) 2^-8 < 2^-8 of the outputs' for sums of independent terms.
"""
import torch

U = 2.0 ** -24


def decays(Hk, kind="mixed"):
    if kind == "mixed":
        base = [1 - 2.0 ** -4, 1.0, 0.5, 1 - 2.0 ** -9, 0.0, 1e-3, 0.875, 1 - 2.0 ** -6]
        return torch.tensor([base[i % len(base)] for i in range(Hk)])
    return torch.full((Hk,), float(kind))


def inputs(B, L, H, Hk, dk, dv, dtype, seed, fused=False, carry=False):
    """q, k, v (views of one projection if `fused`) and a state, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    if fused:
        x = torch.randn((B, L, (H + Hk) * dk + Hk * dv), generator=g).to(dtype)
        q = x[..., :H * dk].unflatten(-1, (H, dk))
        k = x[..., H * dk:(H + Hk) * dk].unflatten(-1, (Hk, dk))
        v = x[..., (H + Hk) * dk:].unflatten(-1, (Hk, dv))
    else:
        q, k, v = (torch.randn((B, L, n, w), generator=g).to(dtype) for n, w in ((H, dk), (Hk, dk), (Hk, dv)))
    S = torch.randn((B, Hk, dk, dv), generator=g) * 3 if carry else None
    return q, k, v, S


def _recur(q, k, v, decay, scale, lens, S):
    q, k, v, decay = q.double(), k.double(), v.double(), decay.double()
    B, L, H, dk = q.shape
    Hk, dv = v.shape[2:]
    S = torch.zeros((B, Hk, dk, dv), dtype=torch.float64, device=q.device) if S is None else S.double().clone()
    o = torch.zeros((B, L, H, dv), dtype=torch.float64, device=q.device)
    g = decay[:, None, None]
    for t in range(L):
        new = g * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        on = torch.ones(B, dtype=torch.bool, device=q.device) if lens is None else t < lens
        S = torch.where(on[:, None, None, None], new, S)
        y = torch.einsum("bhgd,bhdv->bhgv", q[:, t].unflatten(1, (Hk, H // Hk)), S).flatten(1, 2)
        o[:, t] = torch.where(on[:, None, None], scale * y, torch.zeros((), dtype=torch.float64, device=q.device))
    return o, S


def reference(q, k, v, decay, scale, lens=None, S=None):
    """(o, state, M_o, M_state) in fp64 by the token recurrence; rows of o behind lens are 0."""
    if lens is not None:          # what lies behind a row's tokens is not read
        behind = torch.arange(q.shape[1], device=q.device)[None] >= lens[:, None]
        q, k, v = (x.masked_fill(behind[..., None, None], 0.0) for x in (q, k, v))
    o, st = _recur(q, k, v, decay, scale, lens, S)
    mo, ms = _recur(q.abs(), k.abs(), v.abs(), decay, abs(scale), lens, None if S is None else S.abs())
    return o, st, mo, ms


def check(got_o, got_s, ref, L, dk, dtype, tc, rows=None):
    o, st, mo, ms = ref
    K = 2 * (8 + 3 * 128 + 2 * L / 128) if tc else 8 + 3 * (8 + 2 * L / 8)
    err = (got_s.double() - st).abs()
    assert bool((err <= K * U * ms + 1e-300).all()), f"state: {float((err / (ms + 1e-300)).max()):.3e} of M, K u = {K * U:.3e}"
    tol = (K + dk) * U * mo
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * o.abs() * (1 + 1e-6) + (2.0 ** -8 * mo * 1.01 if tc else 0.0)
    err = (got_o.double() - o).abs()
    if rows is not None:
        err, tol, o = err * rows, tol * rows, o * rows
    assert bool((err <= tol + 1e-300).all()), f"o: {float((err - tol).max()):.3e} over the bound, {float(err.max()):.3e} off"


def rotate64(x, w, eps, inv_freq, pos, interleaved, norm=True):
    """x [..., heads, hd], pos [...]"""
    x = x.double()
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if w is not None:
            x = x * w.double()
    if inv_freq is None or inv_freq.numel() == 0:
        return x
    rot = 2 * inv_freq.numel()
    ang = pos.double()[..., None, None] * inv_freq.double()
    c, s = torch.cos(ang), torch.sin(ang)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def rotate_bound(x, w, eps, inv_freq, pos, interleaved, dtype, norm=True):
    """The bound of an output of the norm and rotation: hd + 16 fp32 roundings in the norm (the sum of
    squares, mean, rsqrtf to 2 ulp, two products), 6 in the rotation (cos and sin to 2 ulp from an angle off by
    at most 2^-25 of half a turn: 2^-24 pi) of the absolute values, and the output's own rounding."""
    y = rotate64(x, w, eps, inv_freq, pos, interleaved, norm)
    n = rotate64(x, w, eps, None, pos, interleaved, norm).abs()
    m = n.clone()
    if inv_freq is not None and inv_freq.numel():
        rot = 2 * inv_freq.numel()
        if interleaved:
            t = n[..., 0:rot:2] + n[..., 1:rot:2]
            m[..., 0:rot:2], m[..., 1:rot:2] = t, t
        else:
            t = n[..., :rot // 2] + n[..., rot // 2:rot]
            m[..., :rot // 2], m[..., rot // 2:rot] = t, t
    return y, (x.shape[-1] + 16 + 6 + 4) * U * m + (2.0 ** -8 if dtype == torch.bfloat16 else U) * y.abs() * (1 + 1e-6)
