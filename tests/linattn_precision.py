"""Sharper checks of the linear-attention prompt form on the tensor cores than the sums of absolute values of
linattn_util.py allow, and a model of its arithmetic in which mistakes are planted (test_linattn_precision_cpu.py).

State.  With one token for each column of v, a state entry is one product g^(L-1-t) k v, so no sum hides what a factor
lost.  u = 2^-23 is what one addition in a tensor core can cut off.  Weight to fp32 1/2 u, the weighted key as four bf16 terms 1/4 u
(2^-25), their three additions 3 u: below 4 u within a chunk.  Every later chunk decays the entry once, and so does every later
segment of a cut prompt: a rounded factor and a rounding each, u.  A prompt has at most as many segments as chunks, so
(4 + 2 ceil(L / 128)) u.  A key cut to its first three terms is off by up to 2^-17 = 64 u, to two by 2^-9.

Outputs.  For a row (sequence, token, head) of dv entries: its rounding to bf16 is at most 2^-8 |o|.  Scores and the copy of
the state are rounded to bf16 as operands; each term of o is then off by at most 2^-8 of itself, independently of the others, so
their 2-norm is at most 2^-8 of the root of the terms' squared norms.  For values drawn independently that root is the
expectation of |o|, and with 64 entries and more |o| stays above 0.6 of it: (1 + 1 / 0.6) 2^-8 < 3 2^-8.  One lost token of
300 is 6% of a row, 15 times as much.
"""
import torch

from linattn_util import _recur

UA = 2.0 ** -23
ROW = 3 * 2.0 ** -8


def one_product_values(B, L, Hk, dv, seed):
    """v [B][L][Hk][dv] bf16 with one token for each column, spread over the prompt, the first and the last among them."""
    g = torch.Generator().manual_seed(seed)
    v = torch.zeros((B, L, Hk, dv))
    t = (torch.arange(dv) * (L - 1) + (dv - 1) // 2) // max(dv - 1, 1)
    x = 1 + torch.rand((B, Hk, dv), generator=g)
    for c in range(dv):
        v[:, t[c], :, c] = x[:, :, c]
    return v.to(torch.bfloat16)


def state_excess(got, k, v, decay):
    """The largest error of a state of one_product_values, in units of its bound."""
    L = k.shape[1]
    t = torch.arange(L, device=k.device, dtype=torch.float64)
    w = torch.pow(decay.double()[None, :], (L - 1 - t)[:, None])                                  # [L, Hk]
    ref = torch.einsum("blhd,blhv->bhdv", k.double() * w[None, :, :, None], v.double())
    bound = (4 + 2 * ((L + 127) // 128)) * UA * ref.abs() + 1e-36
    return float(((got.double() - ref).abs() / bound).max())


def row_excess(got, q, k, v, decay, scale, lens=None, S=None):
    """The largest row error of o, in units of its bound."""
    if lens is not None:
        behind = torch.arange(q.shape[1], device=q.device)[None] >= lens[:, None]
        q, k, v = (x.masked_fill(behind[..., None, None], 0.0) for x in (q, k, v))
    ref, _ = _recur(q, k, v, decay, scale, lens, S)
    err = (got.double() - ref).norm(dim=-1)
    if lens is not None:
        err = err * ~behind[..., None]
    return float((err / (ROW * ref.norm(dim=-1) + 1e-300)).max())


# ------------------------------------------------------------------ model of the kernel's roundings
def _bf(x):
    return x.float().to(torch.bfloat16).double()


def weighted_key(k, w, terms):
    """k w as the sum of the kernel's first `terms` bf16 terms (fp64; k holds bf16 numbers)."""
    w = w.float().double()
    w1 = _bf(w)
    w2 = _bf(w - w1)
    w3 = _bf(w - w1 - w2)
    t0 = _bf(k * w1)
    t1 = _bf(k * w2)
    parts = [t0, k * w1 - t0, t1, _bf(k * w3 + (k * w2 - t1))]
    return sum(parts[:terms])


def model(q, k, v, decay, scale, S=None, terms=4, lost=None, C=128):
    """(o, state) for one query head to a state, chunk by chunk, operands rounded as in the kernel, sums exact.  lost = (i, j):
    the score of row i and token j of every chunk is left out."""
    q, k, v, decay = q.double(), k.double(), v.double(), decay.double()
    B, L, H, dk = q.shape
    S = torch.zeros((B, H, dk, v.shape[3]), dtype=torch.float64) if S is None else S.double().clone()
    o = torch.empty((B, L, H, v.shape[3]), dtype=torch.float64)
    for t in range(0, L, C):
        n = min(C, L - t)
        i = torch.arange(n, dtype=torch.float64)
        qc, kc, vc = (x[:, t:t + n].transpose(1, 2) for x in (q, k, v))                            # [B, H, n, .]
        P = (qc @ kc.transpose(-1, -2)) * (torch.pow(decay[:, None, None], (i[:, None] - i[None, :]).clamp(min=0)) * (i[:, None] >= i[None, :]))
        P = _bf(P)
        if lost is not None and lost[0] < n:
            P[:, :, lost[0], lost[1]] = 0
        y = P @ vc + torch.pow(decay[:, None], i + 1)[..., None] * (qc @ _bf(S))
        o[:, t:t + n] = (scale * y).transpose(1, 2)
        w = torch.pow(decay[:, None], n - 1 - i)                                                   # [H, n]
        S = torch.pow(decay, n)[:, None, None] * S + weighted_key(kc, w[None, :, :, None].expand_as(kc), terms).transpose(-1, -2) @ vc
    return _bf(o), S.float()
