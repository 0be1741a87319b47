"""More argument checks of the linear-attention entry points (host only, as in test_linattn_cpu.py)."""
import ctypes

import pytest
import torch

OK, ERR_ARG, ERR_ALIGN, ERR_CUDA = 0, -1, -3, -6
FAKE = 1 << 40          # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from distilled_ssm_decode_b200 import build, ops
    build.build()
    return ops.lib()


def test_hold_hook_validates_its_argument(lib):
    assert lib.hyena_test_linattn_hold(2) == ERR_ARG and lib.hyena_test_linattn_hold(-1) == ERR_ARG
    assert lib.hyena_test_linattn_hold(0) == OK


class _OnDevice(torch.Tensor):
    """A stand-in that claims to be on the device: the checks before the library call run without a GPU."""
    is_cuda = True


@pytest.mark.parametrize("pos0", [1 << 31, (1 << 32) + 5, -(1 << 31) - 1])
def test_binding_refuses_positions_beyond_32_bits(monkeypatch, pos0):
    """They reached the library cut to their low 32 bits: another position's angles."""
    from distilled_ssm_decode_b200 import ops
    monkeypatch.setattr(ops, "_run", lambda *a: pytest.fail("the library was called"))
    x = torch.zeros((2, 3, 2, 8)).as_subclass(_OnDevice)
    prep = ops.QKPrep()
    with pytest.raises(ValueError, match="pos0"):
        ops.qk_norm_rotate(x, x, prep, pos0=pos0)
    with pytest.raises(ValueError, match="pos0"):
        ops.linattn_decode_step(x[:, 0], x[:, 0], x[:, 0], torch.ones(2), torch.zeros((2, 2, 8, 8)), prep=prep, pos0=pos0)


@pytest.mark.parametrize("shape", [((1 << 32) + 2, 1, 1, 1), (1, (1 << 32) + 9, 1, 1), (1, 1, 1 << 31, 1)])
def test_binding_refuses_sizes_beyond_32_bits(shape):
    """As above: (2^32 + 2) rows became 2."""
    from distilled_ssm_decode_b200 import ops
    x = torch.zeros((1, 1, 1, 1)).expand(shape).as_subclass(_OnDevice)
    with pytest.raises(ValueError, match="32 bits"):
        ops._rows(x, "q", 4, torch.float32, x.device)
    if shape[1] == 1:
        with pytest.raises(ValueError, match="32 bits"):
            ops._rows(x[:, 0], "q", 3, torch.float32, x.device)


def test_route_query_gives_the_calls_alignment_errors(lib):
    """The query's documented answer: 1, 0, or the error that the call would return for these arguments."""
    p = ctypes.c_void_p

    def both(dtype=1, **at):
        q, k, v, o = (at.get(n, FAKE) for n in "qkvo")
        r = lib.hyena_linattn_prefill_uses_tensor_cores(dtype, 2, 16, 4, 2, 64, 64, 256, 128, 128, p(q), p(k), p(v), p(o))
        c = lib.hyena_linattn_prefill(p(q), p(k), p(v), dtype, 2, 16, 4, 2, 64, 64, 256, 128, 128, p(FAKE), 1.0, None, None,
                                      p(o), p(FAKE), p(FAKE), 1 << 40, None)
        return r, c
    for n in "qkvo":
        assert both(**{n: FAKE + 1}) == (ERR_ALIGN, ERR_ALIGN), n
        assert both(dtype=0, **{n: FAKE + 2}) == (ERR_ALIGN, ERR_ALIGN), n
    assert lib.hyena_test_fail_next_launches(2) == OK
    try:
        assert both() == (1, ERR_CUDA) and both(q=FAKE + 2) == (0, ERR_CUDA)
    finally:
        lib.hyena_test_fail_next_launches(0)


def test_a_prefill_result_is_a_pair_also_when_copied():
    import copy
    import pickle
    from distilled_ssm_decode_b200 import ops
    o, s = torch.ones(2), torch.zeros(3)
    r = ops.LinattnPrefill(o, s, torch.zeros(1), (torch.float32, 0, 0, 1, 1, 1, 1))
    assert r == (o, s) and r.error() == 0
    for c in (copy.copy(r), copy.deepcopy(r), pickle.loads(pickle.dumps(r))):
        assert len(c) == 2 and torch.equal(c[0], o) and torch.equal(c[1], s)
