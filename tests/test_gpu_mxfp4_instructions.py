"""The instructions that the MXFP4 operators rest on: what one block-scaled MFMA does with
e2m1 operands, and how the conversions to e2m1 round.  The layers' exactness and
their NaN rows rest on these facts."""

import ctypes
import os

import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LIB = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "libmxfp4_probe.so")


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(LIB):
        pytest.fail(f"{LIB} is not built (run __graft_entry__.build())")
    h = ctypes.CDLL(LIB)
    h.tq4test_mfma_fp4_probe.argtypes = [ctypes.c_void_p] * 6 + [ctypes.c_int, ctypes.c_void_p]
    h.tq4test_cvt_fp4_probe.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    return h


def _mfma(lib, ca, cb, sa, sb, c, sel=0):
    t = [torch.from_numpy(np.ascontiguousarray(v)).cuda()
         for v in (O.pack_nibbles(ca), O.pack_nibbles(cb), sa, sb, c)]
    d = torch.empty(16, 16, device="cuda")
    assert lib.tq4test_mfma_fp4_probe(*(v.data_ptr() for v in t), d.data_ptr(), sel,
                                      torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    return d.cpu().numpy()


def _operands(seed, span):
    rng = np.random.default_rng(seed)
    codes = [rng.integers(0, 16, (16, 128)).astype(np.uint8) for _ in range(2)]
    scales = [rng.integers(127 - span, 128 + span, (16, 4)).astype(np.uint8) for _ in range(2)]
    return codes + scales


@pytest.mark.parametrize("sel", [0, 1, 2, 3])
@pytest.mark.parametrize("span", [0, 1, 3])
def test_layout_and_exact_sums(lib, sel, span):
    """Scales within 2^(4 span): sums of 128 products below 2^(4 span + 13) units."""
    ca, cb, sa, sb = _operands(sel, span)
    c = np.random.default_rng(9).integers(-1000, 1000, (16, 16)).astype(np.float32)
    d = _mfma(lib, ca, cb, sa, sb, c, sel)
    want = c + O.mxfp4_values(ca, sa) @ O.mxfp4_values(cb, sb).T
    assert np.array_equal(d, want.astype(np.float32)) and np.array_equal(d, want)


def test_far_scales_round_to_fp32(lib):
    ca, cb, sa, sb = _operands(5, 20)
    d = _mfma(lib, ca, cb, sa, sb, np.zeros((16, 16), np.float32))
    va, vb = O.mxfp4_values(ca, sa), O.mxfp4_values(cb, sb)
    # five fp32 additions, each off by less than 2^-23 of what is summed
    assert np.all(np.abs(d - va @ vb.T) <= 5 * 2.0 ** -23 * (np.abs(va) @ np.abs(vb).T))


def test_a_long_accumulator_stays_exact(lib):
    ca, cb, sa, sb = _operands(6, 0)
    c = (np.random.default_rng(1).integers(-2 ** 23, 2 ** 23, (16, 16)) * 0.25).astype(np.float32)
    d = _mfma(lib, ca, cb, sa, sb, c)
    assert np.array_equal(d, c + O.mxfp4_values(ca, sa) @ O.mxfp4_values(cb, sb).T)


def test_zero_operands_and_the_smallest_scale(lib):
    ca, cb, sa, sb = _operands(7, 1)
    c = np.random.default_rng(2).standard_normal((16, 16)).astype(np.float32)
    assert np.array_equal(_mfma(lib, ca * 0, cb, sa, sb, c), c)
    assert np.array_equal(_mfma(lib, ca, cb, sa * 0, sb, c), c)      # 2^-127 is below c's last bit
    # zero codes under zero scale bytes, as behind k, against the largest scale
    assert np.array_equal(_mfma(lib, ca * 0, cb, sa * 0, np.full_like(sb, 254), c), c)


def test_a_nan_scale_makes_its_row_nan(lib):
    ca, cb, sa, sb = _operands(8, 1)
    c = np.zeros((16, 16), np.float32)
    good = _mfma(lib, ca, cb, sa, sb, c)
    for zero in (False, True):
        a, s = ca.copy(), sa.copy()
        s[3, 1] = 255
        if zero:
            a[3, 32:64] = 0
        d = _mfma(lib, a, cb, s, sb, c)
        assert np.isnan(d[3]).all() and np.array_equal(np.delete(d, 3, 0), np.delete(good, 3, 0))
        d = _mfma(lib, cb, a, sb, s, c)
        assert np.isnan(d[:, 3]).all() and np.isfinite(np.delete(d, 3, 1)).all()


@pytest.mark.parametrize("byte", [0, 1, 27, 100, 126, 127, 128, 200, 253, 254])
def test_conversions_round_by_the_rule(lib, byte):
    """Every finite bf16 value: nearest level, ties to the even code, 6 at most."""
    v = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    v = v[(v & 0x7FFF) < 0x7F80]
    n = len(v) // 2
    a = torch.from_numpy(v[:2 * n].view(np.int16).copy()).cuda()
    s = torch.full((n,), byte << 23, dtype=torch.int32, device="cuda")
    out = torch.empty(2, n, dtype=torch.uint8, device="cuda")
    assert lib.tq4test_cvt_fp4_probe(a.data_ptr(), s.data_ptr(), n, out[0].data_ptr(),
                                     out[1].data_ptr(),
                                     torch.cuda.current_stream().cuda_stream) == 0
    u = np.abs(O.f64_from_bf16_bits(v)) * 2.0 ** (127 - byte)
    want = np.zeros(len(v), int)
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        want += (u >= mid) if i % 2 else (u > mid)
    want |= (v >> 12) & 8
    for row in out.cpu().numpy():
        assert np.array_equal(O.unpack_nibbles(row[None])[0], want)
