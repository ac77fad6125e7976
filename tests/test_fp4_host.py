"""4-bit matrices without a GPU: the oracle's pins, the arithmetic that the quantiser's kernels
rest on, buffer sizes, and the refusals of the C ABI and the binding, none of which launches."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

from oracle import fp4_oracle as F

FAKE = 1 << 20  # an aligned address that is never dereferenced: every call fails its checks first


@pytest.fixture(scope="module")
def H():
    from conftest import build_library
    build_library()
    import pruning_hinm_spmm_b200 as H
    return H


# ----------------------------------------------------------------------------- oracle
def test_oracle_codes_and_ties():
    x = np.array([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.26, 0.2501, 7.0, 5.1, 0, -0.0, 4.9]])
    codes = F.nearest(np.abs(x), F.E2M1) + 8 * np.signbit(x)
    assert codes.tolist() == [[0, 2, 2, 4, 4, 6, 6, 7, 8, 9, 1, 7, 7, 0, 8, 6]]
    assert len(F.E4M3) == 127 and F.E4M3[-1] == 448.0 and F.E4M3[1] == 2.0 ** -9
    assert F.nearest(np.array([0.5 * (448 + 416), 2.0 ** -10]), F.E4M3).tolist() == [126, 0]


def test_oracle_scales():
    x = np.zeros((1, 32))
    x[0, 5], x[0, 20] = 6.0 * 448, 3.0
    c, s = F.quantize(x, F.NV)
    assert s.tolist() == [[126, F.nearest(np.array(0.5), F.E4M3)]] and c[0, 0, 5] == 7 and c[0, 1, 4] == 7
    c, s = F.quantize(x, F.MX)
    assert s.tolist() == [[11 - 2 + 127]] and c[0, 0, 5] == 7  # 2688 / 2^9 = 5.25 -> 6
    assert np.isnan(F.rounded(np.array([[1.0, np.nan]]), F.MX)).all()
    assert np.isnan(F.rounded(np.array([[1.0, np.inf]]), F.NV)).all()
    assert F.pow2_scale([2688.0]) == 1.0 and F.pow2_scale([2689.0]) == 2.0 and F.pow2_scale([0.0]) == 2.0 ** -126
    assert F.pow2_scale([np.inf, np.nan, 1.0]) == 2.0 ** -11


def test_oracle_layout():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((130, 70))
    c, s = F.quantize(x, F.NV)
    v, b = F.pack(c, s, F.NV, 70)
    assert v.shape == (130, 64) and b.shape == (2, 2, 512)
    assert v[129, 3] == c[129, 0, 6] | c[129, 0, 7] << 4
    assert b[1, 0, 16 * 1 + 0 + 3] == s[129, 3] and b[0, 1, 16 * 31 + 4 * 3 + 0] == s[127, 4]


def _rn32(x):
    """Fraction rounded to fp32 (nearest even), away from under- and overflow."""
    if x == 0:
        return Fraction(0)
    sign, x = (-1 if x < 0 else 1), abs(x)
    e = 0
    while x >= 2 ** 24:
        x, e = x / 2, e + 1
    while x < 2 ** 23:
        x, e = x * 2, e - 1
    n = x.numerator // x.denominator
    r = x - n
    n += 1 if r > Fraction(1, 2) or (r == Fraction(1, 2) and n % 2) else 0
    return sign * Fraction(n) * Fraction(2) ** e


def test_residual_quotient_is_on_the_exact_quotients_side():
    """The quantiser's x / s: q0 = x r, q = q0 + (x - q0 s) r, r = fl32(1 / s), each step rounded
    to fp32 (fused).  For every significand of a scale and every border between two codes, q is
    below, on or above the border exactly when x / s is, for x on the border and 40 fp32 numbers
    either side of it; the quotient is the correctly rounded one."""
    borders = [Fraction(k, 4) for k in (1, 3, 5, 7, 10, 14, 20)]
    for m in range(8, 16):
        s = Fraction(m, 8)
        r = _rn32(1 / s)
        for b in borders:
            mid = b * s
            ulp = Fraction(2) ** -23
            while 2 ** 24 * ulp <= mid:
                ulp *= 2
            while 2 ** 23 * ulp > mid:
                ulp /= 2
            for j in range(-40, 41):
                x = mid + j * (ulp if j >= 0 or mid != 2 ** 23 * ulp else ulp / 2)
                assert _rn32(x) == x
                q0 = _rn32(x * r)
                q = _rn32(q0 + _rn32(x - q0 * s) * r)
                assert q == _rn32(x / s)
                assert (q > b) == (x / s > b) and (q < b) == (x / s < b)


def test_residual_division_by_6_is_correctly_rounded():
    """max / 6 the same way, over every significand (the quotient scales with the exponent)."""
    a = np.arange(1 << 23, 1 << 24, dtype=np.int64).astype(np.float64)
    c = float(np.float32(1 / 6))
    q0 = (a * c).astype(np.float32)               # 48 bits: one rounding
    rem = a - 6.0 * q0.astype(np.float64)         # exact
    assert (rem == rem.astype(np.float32)).all()
    got = (q0.astype(np.longdouble) + rem.astype(np.longdouble) * np.longdouble(c)).astype(np.float32)
    assert (got == (a / 6.0).astype(np.float32)).all()


# ----------------------------------------------------------------------------- sizes
@pytest.mark.parametrize("fmt", [F.NV, F.MX])
def test_sizes(H, fmt):
    chunk = 64 if fmt == F.NV else 128
    for b, r, d in [(1, 1, 1), (1, 128, 128), (3, 129, 130), (2, 1000, 4096)]:
        D, t = -(-d // 128) * 128, -(-r // 128)
        assert H.hinm_fp4_size(fmt, b, r, d) == (b * r * D // 2, b * t * (D // chunk) * 512)
    # ragged: a tile (or 128 of the depth) more for each group
    assert H.hinm_fp4_size(fmt, 1, 300, 130, H.HINM_RAGGED_ROWS, 5) == (300 * 128, (2 + 5) * (256 // chunk) * 512)
    D = 128 * (300 // 128 + 5)
    assert H.hinm_fp4_size(fmt, 1, 130, 300, H.HINM_RAGGED_DEPTH, 5) == (130 * D // 2, 2 * (D // chunk) * 512)
    assert H.hinm_fp4_size(fmt, 1, 0, 64, H.HINM_RAGGED_ROWS, 1)[0] == 0


@pytest.mark.parametrize("groups", [1, 3, 40])
def test_group_tiles_do_not_meet(groups):
    """Group e's tiles start at offsets[e] / 128 + e: for any sizes no two groups share a tile and all
    lie in rows / 128 + groups tiles."""
    rng = np.random.default_rng(groups)
    for _ in range(200):
        n = rng.integers(0, [1, 2, 130, 300][rng.integers(4)], groups)
        o = np.concatenate([[0], np.cumsum(n)])
        first = o[:-1] // 128 + np.arange(groups)
        last = first + -(-n // 128)
        assert (last[:-1] <= first[1:]).all()
        assert last[-1] <= o[-1] // 128 + groups


# ----------------------------------------------------------------------------- refusals
def _fp4(H, **kw):
    d = dict(layout_version=1, format=0, batch=1, rows=128, depth=128, ragged=0, groups=0, offsets=None,
             values=FAKE, scales=FAKE, tensor_scale=None)
    d.update(kw)
    return H.hinm_fp4(*d.values())


def test_size_refusals(H):
    v = ctypes.c_size_t()
    size = lambda *a: H.lib().hinm_fp4_size(*a, ctypes.byref(v), ctypes.byref(v))  # noqa: E731
    assert size(0, 1, 1, 1, 0, 0) == H.HINM_OK
    assert size(2, 1, 1, 1, 0, 0) == H.HINM_ERR_INVALID_ARG
    assert size(0, 1, 1, 1, 3, 1) == H.HINM_ERR_INVALID_ARG
    for bad in [(0, 0, 1, 1, 0, 0), (0, 1, 0, 1, 0, 0), (0, 1, 1, 0, 0, 0), (0, 1, -1, 1, 0, 0), (0, 1, 1, 1, 0, 2),
                (0, 1, 1, 1, 1, 0), (0, 1, 1, 1, 1, 513), (0, 2, 1, 1, 1, 1), (0, 1, 0, 1, 2, 1),
                (0, 70000, 1, 1, 0, 0), (0, 1, 1, 4000001, 0, 0), (0, 60000, 60000, 1, 0, 0)]:
        assert size(*bad) == H.HINM_ERR_SHAPE, bad
    assert H.lib().hinm_fp4_size(0, 1, 1, 1, 0, 0, None, ctypes.byref(v)) == H.HINM_ERR_INVALID_ARG


def test_quantize_refusals(H):
    L, E = H.lib(), H
    def call(q=None, src=FAKE, dtype=0, ld=128, bs=0, axis=1, bits=None, fn="hinm_fp4_quantize", **kw):
        return getattr(L, fn)(src, dtype, ld, bs, axis, bits,
                              ctypes.byref(_fp4(H, **kw) if q is None else q), None)
    for fn in ("hinm_fp4_quantize", "hinm_fp4_tensor_scale"):
        k = dict(fn=fn, tensor_scale=FAKE)
        assert call(layout_version=2, **k) == E.HINM_ERR_INVALID_ARG
        assert call(format=5, **k) == E.HINM_ERR_INVALID_ARG
        assert call(rows=0, **k) == E.HINM_ERR_SHAPE
        assert call(src=None, **k) == E.HINM_ERR_INVALID_ARG
        assert call(dtype=3, **k) == E.HINM_ERR_INVALID_ARG
        assert call(axis=2, **k) == E.HINM_ERR_INVALID_ARG
        assert call(ld=127, **k) == E.HINM_ERR_SHAPE
        assert call(ld=127, rows=127, axis=0, depth=500, src=FAKE + 1, **k) == E.HINM_ERR_ALIGNMENT
        assert call(src=FAKE + 2, dtype=2, **k) == E.HINM_ERR_ALIGNMENT
        assert call(bits=FAKE + 2, **k) == E.HINM_ERR_ALIGNMENT
        assert call(batch=2, bs=128 * 128 - 1, **k) == E.HINM_ERR_SHAPE
        assert call(ragged=1, groups=2, **k) == E.HINM_ERR_INVALID_ARG          # no offsets
        assert call(ragged=1, groups=2, offsets=FAKE, bits=FAKE, **k) == E.HINM_ERR_UNSUPPORTED
        assert call(ragged=1, groups=2, offsets=FAKE + 2, **k) == E.HINM_ERR_ALIGNMENT
    assert call(format=1, tensor_scale=FAKE) == E.HINM_ERR_INVALID_ARG           # MX has no such scale
    assert call(values=None) == E.HINM_ERR_INVALID_ARG
    assert call(scales=FAKE + 8) == E.HINM_ERR_ALIGNMENT
    assert call(fn="hinm_fp4_tensor_scale") == E.HINM_ERR_INVALID_ARG             # nowhere to write
    assert call(fn="hinm_fp4_tensor_scale", format=1) == E.HINM_ERR_UNSUPPORTED
    assert L.hinm_fp4_quantize(FAKE, 0, 128, 0, 1, None, None, None) == E.HINM_ERR_INVALID_ARG
    d = lambda dst=FAKE, ld=128, axis=1, **kw: L.hinm_fp4_dequantize(  # noqa: E731
        ctypes.byref(_fp4(H, **kw)), axis, dst, 0, ld, 0, None)
    assert d(dst=None) == E.HINM_ERR_INVALID_ARG and d(ld=5) == E.HINM_ERR_SHAPE and d(axis=-1) == E.HINM_ERR_INVALID_ARG
    assert d(values=None) == E.HINM_ERR_INVALID_ARG
    assert b"" != L.hinm_last_error()


def test_product_refusals(H):
    L, E = H.lib(), H
    def mm(a={}, b={}, Y=FAKE, dtype=0, ld=128, tr=0, bias=None, act=0, fn="hinm_fp4_matmul"):
        return getattr(L, fn)(ctypes.byref(_fp4(H, **a)), ctypes.byref(_fp4(H, **b)), Y, dtype, ld, tr, bias, act, None)
    assert mm(b=dict(depth=256)) == E.HINM_ERR_SHAPE
    assert mm(b=dict(format=1)) == E.HINM_ERR_INVALID_ARG
    assert mm(a=dict(batch=2)) == E.HINM_ERR_SHAPE
    assert mm(b=dict(ragged=1, groups=2, offsets=FAKE)) == E.HINM_ERR_UNSUPPORTED
    assert mm(ld=127) == E.HINM_ERR_SHAPE and mm(tr=1, ld=127) == E.HINM_ERR_SHAPE
    assert mm(Y=None) == E.HINM_ERR_INVALID_ARG and mm(Y=FAKE + 1) == E.HINM_ERR_ALIGNMENT
    assert mm(Y=FAKE + 2, dtype=2) == E.HINM_ERR_ALIGNMENT
    assert mm(dtype=9) == E.HINM_ERR_INVALID_ARG and mm(act=4) == E.HINM_ERR_INVALID_ARG
    assert mm(bias=FAKE + 1) == E.HINM_ERR_ALIGNMENT
    assert mm(a=dict(values=None)) == E.HINM_ERR_INVALID_ARG and mm(b=dict(scales=FAKE + 4)) == E.HINM_ERR_ALIGNMENT
    g = dict(fn="hinm_fp4_grouped_matmul")
    rag = dict(ragged=1, groups=2, offsets=FAKE)
    assert mm(**g) == E.HINM_ERR_UNSUPPORTED
    assert mm(a=dict(batch=3), b=rag, **g) == E.HINM_ERR_SHAPE
    assert mm(a=rag, b=rag, **g) == E.HINM_ERR_UNSUPPORTED
    assert mm(a=dict(batch=2), b=dict(rag, depth=64), **g) == E.HINM_ERR_SHAPE
    assert mm(a=dict(batch=2), b=dict(rag, rows=0), **g) == E.HINM_OK    # no tokens: nothing to do
    wg = lambda a={}, b={}, Y=FAKE, ld=128, bs=128 * 128: L.hinm_fp4_grouped_weight_grad(  # noqa: E731
        ctypes.byref(_fp4(H, **a)), ctypes.byref(_fp4(H, **b)), Y, 2, ld, bs, None)
    dep = dict(ragged=2, groups=2, offsets=FAKE)
    assert wg() == E.HINM_ERR_UNSUPPORTED and wg(a=dep, b=rag) == E.HINM_ERR_UNSUPPORTED
    assert wg(a=dep, b=dict(dep, groups=3)) == E.HINM_ERR_SHAPE
    assert wg(a=dep, b=dict(dep, depth=64)) == E.HINM_ERR_SHAPE
    assert wg(a=dep, b=dep, bs=128 * 128 - 1) == E.HINM_ERR_SHAPE
    assert wg(a=dep, b=dep, Y=None) == E.HINM_ERR_INVALID_ARG


def test_binding_refuses_before_any_call(H):
    """Tensors that are not on the current device, and arguments that do not fit."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current CUDA device"):
        H.hinm_fp4_quantize(x, H.HINM_FP4_NV)
    q = H.Fp4Matrix.allocate(H.HINM_FP4_MX, 1, 4, 32, "cpu")
    assert q.values.numel() == 4 * 64 and q.tensor_scale is None and q.groups == 0
    with pytest.raises(ValueError, match="current CUDA device"):
        H.hinm_fp4_dequantize(q)
    with pytest.raises(ValueError, match="current CUDA device"):
        H.hinm_fp4_matmul(q, q)
    with pytest.raises(ValueError, match="dtype"):
        H._dtype_code(torch.zeros(2, dtype=torch.int32), "src")
    with pytest.raises(ValueError, match="contiguous"):
        H._matrix(torch.zeros(8, 8).t(), "src")
    with pytest.raises(ValueError, match="dimensions"):
        H._matrix(torch.zeros(8), "src")
    with pytest.raises(ValueError, match="does not"):
        H._fp4_check_source(q, 1, 32, 5, 0)
    with pytest.raises(H.HinmError):
        H.Fp4Matrix.allocate(H.HINM_FP4_NV, 1, 4, 0, "cpu")


def test_matrices_are_copied_and_saved_without_their_c_struct(H):
    import copy
    import pickle
    torch = pytest.importorskip("torch")
    q = H.Fp4Matrix(format=H.HINM_FP4_MX, batch=1, rows=2, depth=128, values=torch.arange(128, dtype=torch.uint8),
                    scales=torch.arange(512).to(torch.uint8))
    object.__setattr__(q, "_c", ((0, 1, 2, None, None), H.hinm_fp4()))  # as after a call
    for other in (copy.copy(q), copy.deepcopy(q), pickle.loads(pickle.dumps(q))):
        assert other._c == (None, None) and other.rows == 2 and torch.equal(other.values, q.values)
    assert q._c[0] is not None


# ----------------------------------------------------------------------------- cuts of a product
def test_every_cut_is_reached_by_some_size(H):
    """The sizes that the GPU tests take for each kernel of the product exist."""
    import fp4_cuts
    missing = [c for c in fp4_cuts.CUTS if fp4_cuts.find(H, *c) is None]
    assert not missing, missing


def test_cut_of_a_product(H):
    import fp4_cuts
    cut = lambda *a: fp4_cuts.cut(H, *a)  # noqa: E731
    assert cut("plain", 11008, 4096, 4096, 1, False) == (256, 1, 1, 0)
    assert cut("plain", 4096, 1, 4096, 1, True)[::2] == (64, 4)
    assert cut("plain", 300, 64, 300, 1, True)[3] == 0 and cut("plain", 300, 65, 300, 1, True)[3] == 1
    assert cut("rows", 300, 0, 300, 4, True) == (0, 0, 0, 0)          # no tokens: nothing to multiply
    L, out = H.lib(), (ctypes.c_int32 * 4)()
    call = lambda a, b, o=out: L.hinm_selftest_fp4_cut(ctypes.byref(a), ctypes.byref(b), 0, o)  # noqa: E731
    assert call(_fp4(H), _fp4(H)) == H.HINM_OK and out[0] == 64
    assert call(_fp4(H, rows=0), _fp4(H)) == H.HINM_ERR_SHAPE
    assert call(_fp4(H), _fp4(H, depth=256)) == H.HINM_ERR_SHAPE
    assert call(_fp4(H), _fp4(H, batch=2)) == H.HINM_ERR_UNSUPPORTED
    assert call(_fp4(H, ragged=1, groups=2), _fp4(H, ragged=1, groups=2)) == H.HINM_ERR_UNSUPPORTED
    assert call(_fp4(H, batch=3), _fp4(H, ragged=1, groups=2)) == H.HINM_ERR_UNSUPPORTED
    assert L.hinm_selftest_fp4_cut(None, None, 0, out) == H.HINM_ERR_INVALID_ARG
    assert call(_fp4(H), _fp4(H), None) == H.HINM_ERR_INVALID_ARG
    assert call(_fp4(H, batch=2), _fp4(H, batch=2)) == H.HINM_ERR_UNSUPPORTED
    # as many tokens as there may be: their number and the groups' do not overflow
    assert cut("rows", 64, 0x7FFFFF00, 1, 512, True)[3] == 1
    assert cut("rows", 64, 0x7FFFFF00, 1, 512, False)[3] == 0
