"""The linear-attention operators through the bounds-checked build (libhyena_b200_dbg.so): ragged little
shapes and one split prompt; no global access may be out of range, and the results hold."""
import pytest
import torch

from distilled_ssm_decode_b200 import ops
import test_linattn_gpu as T

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def dbg():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from distilled_ssm_decode_b200 import build
    path = build.build(debug_bounds=True)
    with ops.using_library(path):
        st, _ = ops.bounds_check()
        assert st == 0
        yield


def _clean():
    torch.cuda.synchronize()
    st, rec = ops.bounds_check()
    assert st == 0, f"out-of-range access recorded: file {rec[0]}, line {rec[1]}, index {rec[2]}, extent {rec[3]}"


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [1, 3, 65, 130])
@pytest.mark.parametrize("dk,dv", [(1, 3), (24, 8), (64, 80), (128, 128), (200, 72)])
def test_prefill_in_bounds(dtype, L, dk, dv):
    T._run(2, L, 4, 2, dk, dv, dtype, carry=True, fused=True)
    T._run(3, L, 2, 2, dk, dv, dtype, lens=[0, L, (L + 1) // 2])
    _clean()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_split_prefill_in_bounds(dtype):
    T._run(2, 1500, 2, 1, 64, 64, dtype, lens=[1499, 700], carry=True)
    _clean()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(1, 1), (18, 20), (128, 128), (256, 33)])
def test_decode_and_norm_in_bounds(dtype, dk, dv):
    T.test_decode_step(dk, dv, 6, 2, dtype)
    if dk % 2 == 0:
        T.test_qk_norm_rotate(dk, dk // 4 * 2, True, dtype)
        T.test_qk_norm_rotate(dk, dk, False, dtype)
        T.test_decode_with_norm_and_rotation(dtype, dk, dk // 4 * 2, False, 2, 2)
    _clean()


@pytest.mark.parametrize("B,L,H,Hk,dk,dv", [(40, 150, 2, 2, 128, 128), (2, 2100, 8, 8, 128, 128), (38, 260, 4, 2, 64, 128),
                                            (1, 1500, 4, 2, 128, 192)])
def test_tiles_and_cuts_in_bounds(B, L, H, Hk, dk, dv):
    T.test_prefill_tiles_and_cuts(B, L, H, Hk, dk, dv, True)
    _clean()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [0, 4, 1])
@pytest.mark.parametrize("B,L,H,Hk,hd,rot", [(2, 700, 2, 1, 24, 8), (1, 3, 100, 1, 128, 128), (2, 601, 1, 3, 40, 20)])
def test_norm_in_vectors_in_bounds(B, L, H, Hk, hd, rot, shift, dtype):
    T.test_qk_vectors(B, L, H, Hk, hd, rot, shift, False, dtype)
    T.test_qk_vectors(B, L, H, Hk, hd, rot, shift, True, dtype)
    _clean()
