"""More argument checks of the linear-attention entry points (host only, as in test_linattn_cpu.py)."""
import pytest

OK, ERR_ARG = 0, -1


@pytest.fixture(scope="module")
def lib():
    from distilled_ssm_decode_b200 import build, ops
    build.build()
    return ops.lib()


def test_hold_hook_validates_its_argument(lib):
    assert lib.hyena_test_linattn_hold(2) == ERR_ARG and lib.hyena_test_linattn_hold(-1) == ERR_ARG
    assert lib.hyena_test_linattn_hold(0) == OK
