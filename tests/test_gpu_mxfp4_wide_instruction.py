"""The 32 x 32 x 64 block-scaled MFMA on e2m1 operands, which carries the MoE tiles and the dense
tiles from 64 x 128 on: operand and result layout, byte select, exact sums, and scales of NaN.
(The 16 x 16 x 128 form has the same tests in test_gpu_mxfp4_instructions.py.)"""

import ctypes
import os

import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LIB = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native",
                   "libmxfp4_wide_probe.so")


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(LIB):
        pytest.fail(f"{LIB} is not built (run __graft_entry__.build())")
    h = ctypes.CDLL(LIB)
    h.tq4test_mfma_fp4_wide_probe.argtypes = [ctypes.c_void_p] * 6 + [ctypes.c_int, ctypes.c_void_p]
    return h


def _mfma(lib, ca, cb, sa, sb, c, sel=0):
    t = [torch.from_numpy(np.ascontiguousarray(v)).cuda()
         for v in (O.pack_nibbles(ca), O.pack_nibbles(cb), sa, sb, c)]
    d = torch.empty(32, 32, device="cuda")
    assert lib.tq4test_mfma_fp4_wide_probe(*(v.data_ptr() for v in t), d.data_ptr(), sel,
                                           torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    return d.cpu().numpy()


def _operands(seed, span):
    rng = np.random.default_rng(seed)
    codes = [rng.integers(0, 16, (32, 64)).astype(np.uint8) for _ in range(2)]
    scales = [rng.integers(127 - span, 128 + span, (32, 2)).astype(np.uint8) for _ in range(2)]
    return codes + scales


@pytest.mark.parametrize("sel", [0, 1, 2, 3])
@pytest.mark.parametrize("span", [0, 1, 3])
def test_layout_and_exact_sums(lib, sel, span):
    """Scales within 2^(4 span): sums of 64 products below 2^(4 span + 12) units."""
    ca, cb, sa, sb = _operands(sel, span)
    c = np.random.default_rng(9).integers(-1000, 1000, (32, 32)).astype(np.float32)
    d = _mfma(lib, ca, cb, sa, sb, c, sel)
    want = c + O.mxfp4_values(ca, sa) @ O.mxfp4_values(cb, sb).T
    assert np.array_equal(d, want.astype(np.float32)) and np.array_equal(d, want)


@pytest.mark.parametrize("k", [0, 1, 31, 32, 33, 63])
def test_one_value_of_k_at_a_time(lib, k):
    ca, cb, sa, sb = _operands(20 + k, 3)
    keep = np.arange(64) == k
    ca = ca * keep.astype(np.uint8)
    d = _mfma(lib, ca, cb, sa, sb, np.zeros((32, 32), np.float32), 2)
    va, vb = O.mxfp4_values(ca, sa), O.mxfp4_values(cb, sb)
    assert np.array_equal(d, np.outer(va[:, k], vb[:, k]))


def test_far_scales_round_to_fp32(lib):
    ca, cb, sa, sb = _operands(5, 20)
    d = _mfma(lib, ca, cb, sa, sb, np.zeros((32, 32), np.float32))
    va, vb = O.mxfp4_values(ca, sa), O.mxfp4_values(cb, sb)
    # three fp32 additions, each off by less than 2^-23 of what is summed
    assert np.all(np.abs(d - va @ vb.T) <= 3 * 2.0 ** -23 * (np.abs(va) @ np.abs(vb).T))


def test_a_long_accumulator_stays_exact(lib):
    ca, cb, sa, sb = _operands(6, 0)
    c = (np.random.default_rng(1).integers(-2 ** 23, 2 ** 23, (32, 32)) * 0.25).astype(np.float32)
    d = _mfma(lib, ca, cb, sa, sb, c)
    assert np.array_equal(d, c + O.mxfp4_values(ca, sa) @ O.mxfp4_values(cb, sb).T)


def test_zero_operands_and_the_smallest_scale(lib):
    ca, cb, sa, sb = _operands(7, 1)
    c = np.random.default_rng(2).standard_normal((32, 32)).astype(np.float32)
    assert np.array_equal(_mfma(lib, ca * 0, cb, sa, sb, c), c)
    assert np.array_equal(_mfma(lib, ca, cb, sa * 0, sb, c), c)      # 2^-127 is below c's last bit
    # zero codes under zero scale bytes, as behind k, against the largest scale
    assert np.array_equal(_mfma(lib, ca * 0, cb, sa * 0, np.full_like(sb, 254), c), c)


@pytest.mark.parametrize("block", [0, 1])
@pytest.mark.parametrize("sel", [0, 2])
def test_a_nan_scale_makes_its_row_nan(lib, block, sel):
    ca, cb, sa, sb = _operands(8, 1)
    c = np.zeros((32, 32), np.float32)
    good = _mfma(lib, ca, cb, sa, sb, c, sel)
    for zero in (False, True):
        a, s = ca.copy(), sa.copy()
        s[19, block] = 255
        if zero:
            a[19, 32 * block:32 * block + 32] = 0
        d = _mfma(lib, a, cb, s, sb, c, sel)
        assert np.isnan(d[19]).all() and np.array_equal(np.delete(d, 19, 0), np.delete(good, 19, 0))
        d = _mfma(lib, cb, a, sb, s, c, sel)
        assert np.isnan(d[:, 19]).all() and np.isfinite(np.delete(d, 19, 1)).all()
