"""Argument checks of the linear-attention entry points (host only: every call fails validation, has
nothing to do, or is stopped by the launch-failure hook, so nothing is enqueued)."""
import ctypes

import pytest
import torch

OK, ERR_ARG, ERR_SHAPE, ERR_ALIGN, ERR_WS, ERR_UNSUP, ERR_CUDA = 0, -1, -2, -3, -4, -5, -6
FAKE = 1 << 40          # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from distilled_ssm_decode_b200 import build, ops
    build.build()
    return ops.lib()


def _p(x):
    return ctypes.c_void_p(x)


def prefill(lib, dtype=1, B=2, L=16, H=4, Hk=2, dk=8, dv=8, ldq=None, ldk=None, ldv=None, q=FAKE, state=FAKE, si=0, dec=FAKE,
            lens=0, wsp=FAKE, ws=1 << 40):
    ldq, ldk, ldv = (d if x is None else x for x, d in ((ldq, H * dk), (ldk, Hk * dk), (ldv, Hk * dv)))
    return lib.hyena_linattn_prefill(_p(q), _p(FAKE), _p(FAKE), dtype, B, L, H, Hk, dk, dv, ldq, ldk, ldv, _p(dec), 1.0,
                                     _p(lens), _p(si), _p(FAKE), _p(state), _p(wsp), ws, None)


def test_prefill_refusals(lib):
    assert prefill(lib, dtype=2) == ERR_ARG
    for bad in (dict(B=-1), dict(L=-1), dict(H=0), dict(Hk=0), dict(H=3), dict(dk=0), dict(dv=0), dict(ldq=31), dict(ldk=15),
                dict(ldv=15)):
        assert prefill(lib, **bad) == ERR_SHAPE, bad
    for big in (dict(dk=257), dict(B=65536), dict(H=1 << 20, Hk=1 << 20, dv=1 << 12), dict(L=0x7fffff01)):
        assert prefill(lib, **big) == ERR_UNSUP, big
    for null in (dict(q=0), dict(state=0), dict(dec=0), dict(wsp=0)):
        assert prefill(lib, **null) == ERR_ARG, null
    for off in (dict(q=FAKE + 1), dict(state=FAKE + 4), dict(si=FAKE + 8), dict(dec=FAKE + 2), dict(lens=FAKE + 2),
                dict(wsp=FAKE + 16), dict(dtype=0, q=FAKE + 2)):
        assert prefill(lib, **off) == ERR_ALIGN, off
    assert prefill(lib, ws=0) == ERR_WS
    assert prefill(lib, B=0) == OK
    assert prefill(lib, L=0, si=FAKE) == OK           # state_in is state_out: nothing to copy


def test_prefill_workspace(lib):
    f = lib.hyena_linattn_prefill_workspace_bytes
    assert f(1, 64, 512, 16, 16, 128, 128) > 0
    # split sequences keep one state per segment
    assert f(0, 1, 65536, 4, 4, 64, 64) >= 2 * 4 * 64 * 64 * 4
    assert f(1, 0, 16, 2, 2, 8, 8) > 0 and f(1, 2, 0, 2, 2, 8, 8) > 0        # empty problems
    assert f(1, 1, 16, 3, 2, 8, 8) == 0 and f(5, 1, 16, 2, 2, 8, 8) == 0


def test_route_query_and_error_words(lib):
    f = lib.hyena_linattn_prefill_uses_tensor_cores

    def route(dtype=1, dk=64, dv=64, ldq=256, ldk=128, ldv=128, q=FAKE, o=FAKE, H=4):
        return f(dtype, 2, 16, H, 2, dk, dv, ldq, ldk, ldv, _p(q), _p(FAKE), _p(FAKE), _p(o))
    assert route() == 1 and route(dk=8, dv=200, ldv=400) == 1 and route(ldq=264) == 1
    for other in (dict(dtype=0), dict(dk=60), dict(dv=60), dict(dk=136, ldq=1000, ldk=1000), dict(ldq=260), dict(q=FAKE + 8),
                  dict(o=FAKE + 2)):
        assert route(**other) == 0, other
    assert route(dtype=3) == ERR_ARG and route(H=3) == ERR_SHAPE and route(ldq=100) == ERR_SHAPE
    for args in ((1, 2, 16, 4, 2, 64, 64), (1, 1, 65536, 12, 12, 64, 64), (0, 1, 300, 1, 1, 8, 8)):
        off, n = lib.hyena_linattn_prefill_error_offset(*args), lib.hyena_linattn_prefill_workspace_bytes(*args)
        assert off % 256 == 0 and (n - off) % 4 == 0 and n > off
    assert lib.hyena_linattn_prefill_error_offset(1, 2, 16, 4, 3, 64, 64) == 0


def decode(lib, dtype=1, B=2, H=4, Hk=2, dk=8, dv=8, ldq=None, q=FAKE, state=FAKE, prep=None, pos=0):
    return lib.hyena_linattn_decode_step(_p(q), _p(FAKE), _p(FAKE), dtype, B, H, Hk, dk, dv, H * dk if ldq is None else ldq, Hk * dk,
                                         Hk * dv, _p(FAKE), 1.0, prep, _p(pos), 0, _p(state), _p(FAKE), None)


def _prep(**kw):
    from distilled_ssm_decode_b200.ops import _CQKPrep
    d = dict(norm=1, eps=1e-6, q_weight=FAKE, k_weight=FAKE, rot_dim=8, inv_freq=FAKE, interleaved=0)
    d.update(kw)
    c = _CQKPrep(*(d[n] for n, _ in _CQKPrep._fields_))
    _prep.keep = c
    return ctypes.c_void_p(ctypes.addressof(c))


BAD_PREPS = [(dict(rot_dim=10), ERR_SHAPE), (dict(rot_dim=3), ERR_SHAPE), (dict(rot_dim=-2), ERR_SHAPE), (dict(norm=2), ERR_ARG),
             (dict(interleaved=-1), ERR_ARG), (dict(eps=-1.0), ERR_ARG), (dict(eps=float("nan")), ERR_ARG),
             (dict(inv_freq=None), ERR_ARG), (dict(q_weight=FAKE + 2), ERR_ALIGN), (dict(k_weight=FAKE + 1), ERR_ALIGN),
             (dict(inv_freq=FAKE + 2), ERR_ALIGN)]


def test_decode_refusals(lib):
    assert decode(lib, dtype=-1) == ERR_ARG
    assert decode(lib, H=5) == ERR_SHAPE
    assert decode(lib, ldq=8) == ERR_SHAPE
    assert decode(lib, dk=300) == ERR_UNSUP
    assert decode(lib, q=0) == ERR_ARG
    assert decode(lib, state=0) == ERR_ARG
    assert decode(lib, state=FAKE + 8) == ERR_ALIGN
    assert decode(lib, state=FAKE + 2, dv=7) == ERR_ALIGN
    assert decode(lib, pos=FAKE + 1) == ERR_ALIGN
    assert decode(lib, B=0) == OK
    assert decode(lib, dk=7, prep=_prep(rot_dim=0)) == ERR_SHAPE        # pairs need an even width
    for kw, want in BAD_PREPS:
        assert decode(lib, prep=_prep(**kw)) == want, kw


def qk(lib, dtype=1, B=2, L=3, H=2, Hk=1, hd=8, ldq=16, ldk=8, ldqo=16, ldko=8, q=FAKE, k=FAKE, qo=2 * FAKE, ko=2 * FAKE, pos=0,
       prep=None):
    return lib.hyena_qk_norm_rotate(_p(q), _p(k), dtype, B, L, H, Hk, hd, ldq, ldk, prep or _prep(), _p(pos), 0, _p(qo), _p(ko),
                                    ldqo, ldko, None)


def test_qk_refusals(lib):
    assert qk(lib, dtype=9) == ERR_ARG
    assert lib.hyena_qk_norm_rotate(_p(FAKE), _p(FAKE), 1, 1, 1, 1, 1, 8, 8, 8, None, None, 0, _p(FAKE), _p(FAKE), 8, 8,
                                    None) == ERR_ARG
    for bad in (dict(B=-1), dict(L=-1), dict(H=-1), dict(Hk=-1), dict(hd=0), dict(hd=7), dict(ldq=15), dict(ldk=7), dict(ldqo=8),
                dict(ldko=0)):
        assert qk(lib, **bad) == ERR_SHAPE, bad
    assert qk(lib, hd=258, ldq=1000, ldk=1000, ldqo=1000, ldko=1000) == ERR_UNSUP
    for null in (dict(q=0), dict(k=0), dict(qo=0), dict(ko=0)):
        assert qk(lib, **null) == ERR_ARG, null
    assert qk(lib, q=2 * FAKE, ldq=32) == ERR_ARG          # in place over rows of another stride
    for off in (dict(q=FAKE + 1), dict(ko=FAKE + 1), dict(pos=FAKE + 2)):
        assert qk(lib, **off) == ERR_ALIGN, off
    for kw, want in BAD_PREPS:
        assert qk(lib, prep=_prep(**kw)) == want, kw
    assert qk(lib, B=0) == OK and qk(lib, L=0) == OK
    assert qk(lib, H=0, Hk=0, q=0, k=0, qo=0, ko=0) == OK


def test_qk_positions_stay_in_32_bits(lib):
    f = lambda L, pos0, pos: lib.hyena_qk_norm_rotate(_p(FAKE), _p(FAKE), 1, 1, L, 1, 1, 8, 8, 8, _prep(), _p(pos), pos0,
                                                      _p(2 * FAKE), _p(2 * FAKE), 8, 8, None)
    assert f(2, 0x7fffffff, 0) == ERR_ARG and f(0x7fffffff, 2, 0) == ERR_ARG
    assert lib.hyena_test_fail_next_launches(2) == OK          # the largest that fits passes the checks
    try:
        assert f(1, 0x7fffffff, 0) == ERR_CUDA and f(2, 0x7fffffff, FAKE) == ERR_CUDA
    finally:
        lib.hyena_test_fail_next_launches(0)


def test_launch_failures_are_reported(lib):
    assert lib.hyena_test_fail_next_launches(4) == OK
    try:
        assert prefill(lib) == ERR_CUDA
        assert prefill(lib, L=0) == ERR_CUDA
        assert decode(lib) == ERR_CUDA
        assert qk(lib, H=0, q=0, qo=0) == ERR_CUDA
    finally:
        lib.hyena_test_fail_next_launches(0)


def test_binding_refuses_cpu_tensors_and_bad_layouts():
    from distilled_ssm_decode_b200 import ops
    x = torch.zeros((1, 2, 2, 8))
    with pytest.raises(TypeError, match="CUDA tensor"):
        ops.linattn_prefill(x, x, x, torch.ones(2))
    with pytest.raises(TypeError, match="CUDA tensor"):
        ops.linattn_decode_step(x[0], x[0], x[0], torch.ones(2), torch.zeros((2, 2, 8, 8)))
    with pytest.raises(TypeError, match="CUDA tensor"):
        ops.qk_norm_rotate(x, x, ops.QKPrep())
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ops.linattn_prefill(x.half(), x, x, torch.ones(2))
    with pytest.raises(TypeError):
        ops.QKPrep(wq=torch.ones(8))


def test_binding_row_strides():
    """The stride rule on views, without a GPU: a stand-in that claims to be on the device."""
    from distilled_ssm_decode_b200 import ops

    class T(torch.Tensor):
        is_cuda = True
    x = torch.zeros((2, 5, 3 * 8 + 7)).as_subclass(T)
    q = x[..., 4:28].unflatten(-1, (3, 8))
    rows = lambda t, dim=4: ops._rows(t, "t", dim, torch.float32, t.device)
    assert rows(q) == 31
    assert rows(q[:, 0], 3) == 5 * 31
    assert rows(q[:1, :1]) == 24 or rows(q[:1, :1]) >= 24
    with pytest.raises(ValueError, match="contiguous"):
        rows(q.transpose(2, 3))
    with pytest.raises(ValueError, match="contiguous"):
        rows(q[..., ::2, :])
    with pytest.raises(ValueError, match="token stride"):
        rows(q[:, :3])
    with pytest.raises(ValueError, match="overlap"):
        rows(x[:, :1, :24].unflatten(-1, (3, 8)).expand(2, 4, 3, 8)[:1])
    with pytest.raises(ValueError, match="dimensions"):
        rows(q, 3)
