"""Cases for measuring the linear-attention operators: prompt form, single-token form, and the
norm and rotation of queries and keys in front of them.

    python -c "import perf.operators as o; print([c['name'] for c in o.listed()])"

`own` selects what run() does: False computes the operators in elementary torch operations (fp32,
rounded once at the end), True calls the library through distilled_ssm_decode_b200.ops.

Linear attention with a decay g_h for each key/value head (state S [dk][dv] per sequence and head):
    S_t = g S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t
Queries and keys: x * rsqrt(mean(x^2) + eps) * weight per head, then the rotation of the pairs of the
first rot entries by position * inv_freq.
"""
import torch

own = False

EPS = 1e-6
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    def prefill(name, B, L, H, Hk, dk, dv, dtype, ragged=False, carry=False):
        return dict(name=name, op="prefill", B=B, L=L, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, ragged=ragged, carry=carry)

    def decode(name, B, H, Hk, dk, dv, dtype, prep=False):
        return dict(name=name, op="decode", B=B, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, prep=prep)

    def qk(name, B, L, H, Hk, hd, rot, interleaved, dtype, pos0=0):
        return dict(name=name, op="qk", B=B, L=L, H=H, Hk=Hk, dk=hd, rot=rot, interleaved=interleaved, dtype=dtype, pos0=pos0)

    return [
        # one short chat turn on one sequence: latency counts
        prefill("prefill_short", 1, 37, 16, 16, 128, 128, "bf16"),
        # prompts of a generation batch (64 x 512 tokens, 2048 channels in 16 heads)
        prefill("prefill_batch", 64, 512, 16, 16, 128, 128, "bf16"),
        # a few medium prompts (8 x 4096 tokens, 1024 channels in 8 heads): fewer sequences than SMs
        prefill("prefill_medium", 8, 4096, 8, 8, 128, 128, "bf16"),
        # one long document (65536 tokens, 768 channels in 12 heads)
        prefill("prefill_long", 1, 65536, 12, 12, 64, 64, "bf16"),
        # a padded batch continued from stored states: queries share key/value heads, odd head sizes
        prefill("prefill_ragged_shared", 13, 1537, 12, 4, 96, 80, "bf16", ragged=True, carry=True),
        # fp32 activations (parity runs of a model)
        prefill("prefill_f32", 2, 1000, 8, 8, 64, 64, "f32"),
        # one sequence generating a token (4096 channels in 32 heads)
        decode("decode_one", 1, 32, 32, 128, 128, "bf16"),
        # a large serving batch: the state streams from memory
        decode("decode_batch", 256, 32, 32, 128, 128, "bf16"),
        # raw projections: norm and rotation inside the step, shared key/value heads, odd head sizes
        decode("decode_prep_shared_f32", 33, 24, 6, 72, 104, "f32", prep=True),
        # queries and keys of one token for each of 64 sequences
        qk("qk_token", 64, 1, 16, 16, 128, 128, False, "bf16", pos0=4095),
        # queries and keys of whole prompts
        qk("qk_prompt", 8, 4096, 8, 8, 128, 128, False, "bf16"),
        # partial rotation at far positions, interleaved pairs, one key head
        qk("qk_far_f32", 3, 1999, 7, 1, 80, 32, True, "f32", pos0=1000003),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["prefill", "decode", "qk"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hk = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    H = Hk * rng.choice([1, 1, 1, 2, 3, 4])
    if op == "prefill":
        dk, dv = (rng.choice([24, 32, 48, 64, 64, 96, 128, 128]) for _ in range(2))
        L = _log(rng, 1, 40000)
        # fp32 activations stay at a tenth of the tokens
        room = (3.0e5 if dtype == "bf16" else 3.0e4) / H
        L = max(1, min(L, int(room)))
        B = max(1, min(_log(rng, 1, 64), int(room / L)))
        return dict(op=op, B=B, L=L, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, ragged=rng.random() < 0.4, carry=rng.random() < 0.4)
    if op == "decode":
        dk, dv = (rng.choice([24, 40, 64, 72, 104, 128, 128, 256]) for _ in range(2))
        B = max(1, min(_log(rng, 1, 256), int(1.2e8 / (Hk * dk * dv))))
        return dict(op=op, B=B, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, prep=rng.random() < 0.5)
    hd = rng.choice([16, 40, 64, 80, 128, 128, 256])
    rot = rng.choice([0, hd // 4 * 2, hd, hd])
    L = _log(rng, 1, 30000)
    room = int(5.0e7 / ((H + Hk) * hd))
    L = max(1, min(L, room))
    B = max(1, min(_log(rng, 1, 64), room // L))
    return dict(op=op, B=B, L=L, H=H, Hk=Hk, dk=hd, rot=rot, interleaved=rng.random() < 0.4, dtype=dtype, pos0=rng.choice([0, 511, 70000, 1000003]))


# ------------------------------------------------------------------ inputs
def _projected(case, L, g, normed):
    """q, k, v as a model has them: slices of one projection [B][L][(H + Hk) dk + Hk dv]; queries and
    keys of unit mean square per entry when `normed` (else as a projection leaves them)."""
    B, H, Hk, dk, dv = case["B"], case["H"], case["Hk"], case["dk"], case.get("dv", 0)
    x = torch.randn((B, L, (H + Hk) * dk + Hk * dv), generator=g, device="cuda")
    if not normed:
        x *= 0.5 + torch.rand((B, L, 1), generator=g, device="cuda")
    x = x.to(_DT[case["dtype"]])
    q = x[..., :H * dk].unflatten(-1, (H, dk))
    k = x[..., H * dk:(H + Hk) * dk].unflatten(-1, (Hk, dk))
    v = x[..., (H + Hk) * dk:].unflatten(-1, (Hk, dv)) if dv else None
    return q, k, v


def _decay(Hk, g):
    """Decays 1 - 2^-e with e spread over [3, 9] across the heads, as retention-like layers use them."""
    e = 3.0 + 6.0 * torch.rand((Hk,), generator=g, device="cuda")
    return 1.0 - torch.exp2(-e)


def _plan(case, rot, interleaved, g):
    dk = case["dk"]
    freq = torch.exp2(-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(rot, 1) * 13.2877).float()
    return dict(wq=1.0 + 0.1 * torch.randn((dk,), generator=g, device="cuda"),
                wk=1.0 + 0.1 * torch.randn((dk,), generator=g, device="cuda"),
                inv_freq=freq, rot=rot, interleaved=interleaved)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(op=case["op"])
    if case["op"] == "qk":
        q, k, _ = _projected(case, case["L"], g, False)
        st.update(q=q, k=k, plan=_plan(case, case["rot"], case["interleaved"], g))
        # every sequence stands at its own place
        first = case["pos0"] + torch.randint(0, 512, (case["B"], 1), generator=g, device="cuda")
        st["pos"] = (first + torch.arange(case["L"], device="cuda")).to(torch.int32)
        return st
    B, Hk, dk, dv = case["B"], case["Hk"], case["dk"], case["dv"]
    st.update(decay=_decay(Hk, g), scale=dk ** -0.5, lens=None, S=None, plan=None, pos=None)
    if case["op"] == "decode":
        q, k, v = _projected(case, 1, g, not case["prep"])
        st.update(q=q[:, 0], k=k[:, 0], v=v[:, 0])
        if case["prep"]:
            st["plan"] = _plan(case, dk, False, g)
            st["pos"] = torch.randint(0, 32768, (B,), generator=g, device="cuda", dtype=torch.int32)
    else:
        q, k, v = _projected(case, case["L"], g, True)
        st.update(q=q, k=k, v=v, o=torch.zeros((B, case["L"], case["H"], dv), device="cuda", dtype=q.dtype))
        if case["ragged"]:
            # lengths from none to all of the padded prompt
            n = torch.randint(0, case["L"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            n[0] = case["L"]
            if B > 2:
                n[1], n[2] = 0, 1
            st["lens"] = n
    if case["op"] == "decode" or case["carry"]:
        # a state that has seen many tokens: entries of variance 1 / (1 - g^2)
        s = torch.randn((B, Hk, dk, dv), generator=g, device="cuda")
        st["S"] = s / torch.sqrt(1.0 - st["decay"] ** 2)[:, None, None]
    return st


# ------------------------------------------------------------------ plain forms
def _norm_rotate_plain(x, w, plan, pos):
    """x [..., heads, hd], pos [...]: fp32, angles in fp64 (positions may be far)."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    rot = plan["rot"]
    if rot == 0:
        return x
    ang = pos.double()[..., None, None] * plan["inv_freq"].double()
    c, s = torch.cos(ang).float(), torch.sin(ang).float()
    y, rest = x[..., :rot], x[..., rot:]
    if plan["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, rest], -1)


def _powers(decay, n):
    """decay^n for whole n >= 0 (a tensor), in fp64 and rounded once: [Hk, *n.shape]."""
    return torch.pow(decay.double().view(-1, *[1] * n.dim()), n.double()).float()


def _prefill_plain(st, C=128):
    """Chunks of C tokens: scores inside a chunk, states between chunks."""
    q, k, v, decay = st["q"].float(), st["k"].float(), st["v"].float(), st["decay"]
    B, L, H, dk = q.shape
    Hk, dv = v.shape[2], v.shape[3]
    dev = q.device
    nc = (L + C - 1) // C
    n = st["lens"].long() if st["lens"] is not None else torch.full((B,), L, device=dev)
    live = torch.arange(nc * C, device=dev)[None, :] < n[:, None]                                     # [B, T]
    cut = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, nc * C - L)).masked_fill(~live[..., None, None], 0.0)
    q = cut(q).view(B, nc, C, Hk, H // Hk, dk).permute(0, 3, 4, 1, 2, 5)                              # [B, Hk, G, nc, C, dk]
    k = cut(k).view(B, nc, C, Hk, dk).permute(0, 3, 1, 2, 4)                                          # [B, Hk, nc, C, dk]
    v = cut(v).view(B, nc, C, Hk, dv).permute(0, 3, 1, 2, 4)
    i = torch.arange(C, device=dev)
    D = _powers(decay, (i[:, None] - i[None, :]).clamp(min=0)) * (i[:, None] >= i[None, :])           # [Hk, C, C]
    # each chunk's own contribution, decayed to the chunk's end, and the state entering each chunk
    W = (k * _powers(decay, C - 1 - i)[:, None, :, None]).transpose(-1, -2) @ v                       # [B, Hk, nc, dk, dv]
    c = torch.arange(nc + 1, device=dev)
    gap = c[:, None] - 1 - c[None, :nc]
    M = _powers(decay, C * gap.clamp(min=0)) * (gap >= 0)                                             # [Hk, nc + 1, nc]
    S = (M @ W.flatten(-2)).view(B, Hk, nc + 1, dk, dv)
    if st["S"] is not None:
        S = S + _powers(decay, C * c)[None, :, :, None, None] * st["S"][:, :, None]
    o = ((q @ k[:, :, None].transpose(-1, -2)) * D[:, None, None]) @ v[:, :, None]
    o = o + _powers(decay, i + 1)[:, None, None, :, None] * (q @ S[:, :, None, :nc])
    o = (st["scale"] * o).permute(0, 3, 4, 1, 2, 5).reshape(B, nc * C, H, dv)[:, :L]
    o = torch.where(live[:, :L, None, None], o.to(st["o"].dtype), st["o"])
    # the state after the last token of each sequence: its last chunk, cut to the tokens it has
    last = (n - 1).clamp(min=0) // C
    m = n - last * C                                                                                  # 0..C tokens
    pick = last[:, None, None, None, None].expand(B, Hk, 1, 1, 1)
    one = lambda x: x.gather(2, pick.expand(-1, -1, 1, *x.shape[3:]))[:, :, 0]
    left = m[:, None] - 1 - i[None, :]                                                                # [B, C]
    w = (_powers(decay, left.clamp(min=0)) * (left >= 0)).transpose(0, 1)                             # [B, Hk, C]
    fin = (one(k) * w[..., None]).transpose(-1, -2) @ one(v)
    fin = fin + _powers(decay, m).transpose(0, 1)[..., None, None] * one(S[:, :, :nc])
    return o, fin


def _decode_plain(st):
    q, k, v, S = st["q"], st["k"], st["v"].float(), st["S"]
    if st["plan"] is not None:
        q = _norm_rotate_plain(q, st["plan"]["wq"], st["plan"], st["pos"])
        k = _norm_rotate_plain(k, st["plan"]["wk"], st["plan"], st["pos"])
    S.mul_(st["decay"][:, None, None]).add_(k.float()[..., :, None] * v[..., None, :])
    q = q.float().unflatten(1, (S.shape[1], -1))
    o = st["scale"] * (q @ S).flatten(1, 2)
    return o.to(st["v"].dtype), S


# ------------------------------------------------------------------ one pass
def run(state):
    st = state
    if own:
        from distilled_ssm_decode_b200 import ops
        if st["plan"] is not None and "prep" not in st:          # a program keeps this beside its weights
            p = st["plan"]
            st["prep"] = ops.QKPrep(p["wq"], p["wk"], EPS, p["inv_freq"] if p["rot"] else None, p["interleaved"])
        if st["op"] == "qk":
            return ops.qk_norm_rotate(st["q"], st["k"], st["prep"], positions=st["pos"])
        if st["op"] == "decode":
            o = ops.linattn_decode_step(st["q"], st["k"], st["v"], st["decay"], st["S"], scale=st["scale"],
                                        prep=st.get("prep"), positions=st["pos"])
            return o, st["S"]
        return ops.linattn_prefill(st["q"], st["k"], st["v"], st["decay"], scale=st["scale"], lens=st["lens"],
                                   state_in=st["S"], o=st["o"])
    if st["op"] == "qk":
        dt = st["q"].dtype
        return (_norm_rotate_plain(st["q"], st["plan"]["wq"], st["plan"], st["pos"]).to(dt),
                _norm_rotate_plain(st["k"], st["plan"]["wk"], st["plan"], st["pos"]).to(dt))
    return _decode_plain(st) if st["op"] == "decode" else _prefill_plain(st)


def work(case):
    """Inputs read once, outputs written once.  Operations: two products of dk x dv per token (state and
    output); for the norm and rotation about eight per entry."""
    a = 2 if case["dtype"] == "bf16" else 4
    B, H, Hk, dk = case["B"], case["H"], case["Hk"], case["dk"]
    if case["op"] == "qk":
        n = B * case["L"] * (H + Hk) * dk
        return {"bytes": 2 * n * a + 4 * B * case["L"], "flops": 8 * n}
    dv = case["dv"]
    state = 4 * B * Hk * dk * dv
    act = (H + Hk) * dk + (H + Hk) * dv
    if case["op"] == "decode":
        return {"bytes": B * act * a + 2 * state, "flops": 2 * B * (H + Hk) * dk * dv}
    # a padded batch: one full row, one empty, one of a single token, the rest half full on average
    T = case["L"] * (1 + max(0, B - 3 if B > 2 else B - 1) / 2) if case["ragged"] else B * case["L"]
    return {"bytes": int(T * act * a + (2 if case["carry"] else 1) * state), "flops": int(2 * T * (H + Hk) * dk * dv)}


# ------------------------------------------------------------------ 64 bits, from the definitions
def _rotated64(x, w, plan, pos):
    x = x.double()
    x = x / torch.sqrt(torch.mean(x ** 2, -1, keepdim=True) + EPS) * w.double()
    rot = plan["rot"]
    if rot:
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos.double()[..., None, None] * plan["inv_freq"].double())
        if plan["interleaved"]:
            z = torch.view_as_complex(x[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * turn
            x = torch.cat([torch.view_as_real(z).flatten(-2), x[..., rot:]], -1)
        else:
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
            x = torch.cat([z.real, z.imag, x[..., rot:]], -1)
    return x


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "qk":
        return (_rotated64(st["q"], st["plan"]["wq"], st["plan"], st["pos"]),
                _rotated64(st["k"], st["plan"]["wk"], st["plan"], st["pos"]))
    q, k, v = st["q"], st["k"], st["v"].double()
    if st["op"] == "decode":
        if st["plan"] is not None:
            q = _rotated64(q, st["plan"]["wq"], st["plan"], st["pos"])
            k = _rotated64(k, st["plan"]["wk"], st["plan"], st["pos"])
        q, k, v = q[:, None], k[:, None], v[:, None]
    q, k = q.double(), k.double()
    B, L, H, dk = q.shape
    Hk, dv = v.shape[2:]
    gam = st["decay"].double()[:, None, None]
    S = st["S"].double().clone() if st["S"] is not None else torch.zeros((B, Hk, dk, dv), dtype=torch.float64, device=q.device)
    o = torch.zeros((B, L, H, dv), dtype=torch.float64, device=q.device)
    q = q.unflatten(2, (Hk, H // Hk))
    for t in range(L):
        new = torch.addcmul(gam * S, k[:, t, :, :, None], v[:, t, :, None, :])
        if st["lens"] is None:
            S = new
            o[:, t] = (q[:, t] @ S).flatten(1, 2)
        else:
            on = (t < st["lens"])[:, None, None, None]
            S = torch.where(on, new, S)
            o[:, t] = torch.where(on, q[:, t] @ S, 0.0).flatten(1, 2)
    o *= st["scale"]
    return (o[:, 0], S) if st["op"] == "decode" else (o, S)
