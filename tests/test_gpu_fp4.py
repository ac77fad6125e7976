"""The 4-bit matrices on the GPU, through the binding, against the 64-bit oracle.

Codes, scales and read-back values are whole decisions: they match exactly.  Products: the sum over
K terms in fp32, in any order, is within K 2^-24 sum|a b| of the exact one (each addition rounds by
at most half a step, 2^-24 relative to a partial sum that sum|a b| bounds); the scales' product,
the multiplication with it and the bias (fused) add 3 roundings; an activation has a slope of at most
1.13 and adds its own error (SiLU: exp 2 ulp, sum 1/2, division 2; GELU: erf 2 ulp of a factor up to 2,
2 products: 16 half steps cover either), and the store rounds once to Y's type by half a step of it.
Where every partial sum is a whole number below 2^24 the products match bit for bit.
"""
import numpy as np
import pytest

from oracle import fp4_oracle as F

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FORMATS = pytest.mark.parametrize("fmt", [F.NV, F.MX], ids=["nv", "mx"])


@pytest.fixture(scope="module")
def H():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import pruning_hinm_spmm_b200 as H
    yield H
    assert H.hinm_device_status() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = gen(seed)
    x = torch.randn(shape, generator=g, device="cuda") * scale
    x = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.02, x * 20, x)
    return x.to(dtype)


def np64(t):
    return t.detach().double().cpu().numpy()


def ints(o):
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def to_type(v, dtype):
    """64-bit values as the library stores them: rounded to fp32, then to dtype."""
    with np.errstate(over="ignore"):
        return torch.from_numpy(np.asarray(v).astype(np.float32)).to(dtype)


def same(got, want):
    """Equal values, NaN where NaN."""
    got, want = got.cpu(), want.cpu()
    return got.shape == want.shape and bool(((got == want) | (got.isnan() & want.isnan())).all())


def check_stored(q, fmt, codes, sc, depth, matrix=0):
    """The stored bytes of one matrix of q's batch: all value bytes, and the scale bytes of its rows."""
    R = codes.shape[0]
    v, s = F.pack(codes, sc, fmt, depth)
    D = v.shape[1]
    got = q.values.cpu().numpy()[:q.batch * R * D].reshape(q.batch, R, D)[matrix]
    np.testing.assert_array_equal(got, v)
    gs = q.scales.cpu().numpy()[:q.batch * s.size].reshape((q.batch,) + s.shape)[matrix]
    r = np.arange(R)
    cols = 16 * (r % 32) + 4 * (r // 32 % 4)
    for b in range(4):
        np.testing.assert_array_equal(gs[r // 128, :, cols + b], s[r // 128, :, cols + b])


# ----------------------------------------------------------------------------- quantisation
@FORMATS
@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,depth", [(1, 1), (1, 40), (5, 16), (7, 17), (33, 64), (64, 63), (128, 128), (129, 200),
                                        (40, 1003), (200, 96)])
def test_quantize_and_back(H, fmt, axis, dtype, rows, depth):
    shape = (rows, depth) if axis == 1 else (depth, rows)
    x = rand(rows * 31 + depth, *shape, dtype=DT[dtype], scale=0.3)
    g = None if fmt == F.MX else torch.tensor([0.0113], device="cuda")
    gv = 1.0 if fmt == F.MX else float(g)
    q = H.hinm_fp4_quantize(x, fmt, axis=axis, tensor_scale=g)
    xs = np64(x) if axis == 1 else np64(x).T
    codes, sc = F.quantize(xs, fmt, gv)
    check_stored(q, fmt, codes, sc, depth)
    want = F.values(codes, sc, fmt, depth, gv)
    for out in ("bf16", "fp32"):
        y = H.hinm_fp4_dequantize(q, axis=axis, dtype=DT[out])
        assert same(y, to_type(want if axis == 1 else want.T, DT[out]))


@FORMATS
def test_every_bf16_maximum(H, fmt):
    """Blocks whose largest element is each positive bf16 number, alone or with smaller ones."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    B = F.BLOCK[fmt]
    x = bits[:, None] * torch.linspace(1, -1, B, device="cuda", dtype=torch.float32)[None]
    x = x.to(torch.bfloat16)
    x[:, 0] = bits
    q = H.hinm_fp4_quantize(x, fmt)
    codes, sc = F.quantize(np64(x), fmt)
    got = q.values.cpu().numpy()[:x.shape[0] * 64].reshape(-1, 64)[:, :B // 2]
    np.testing.assert_array_equal(got, (codes[:, 0, 0::2] | codes[:, 0, 1::2] << 4).astype(np.uint8))
    assert same(H.hinm_fp4_dequantize(q, dtype=torch.float32), to_type(F.values(codes, sc, fmt, B), torch.float32))


@pytest.mark.parametrize("axis", [1, 0])
def test_borders_between_codes(H, axis):
    """NV: every scale with every border between two codes, and the fp32 numbers next to them."""
    rows = []
    for s in F.E4M3[1:]:
        for side in (-1, 0, 1):
            b = np.float32(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * s)
            b = b if side == 0 else np.nextafter(b, np.float32(side * np.inf), dtype=np.float32)
            rows.append(np.concatenate([[np.float32(6 * s)], b, -b, [0.0]]))
    x = np.stack(rows).astype(np.float32)
    codes, sc = F.quantize(x, F.NV)
    t = torch.from_numpy(x).cuda()
    q = H.hinm_fp4_quantize(t if axis == 1 else t.t().contiguous(), F.NV, axis=axis)
    check_stored(q, F.NV, codes, sc, 16)


@FORMATS
@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cols", [64, 61])
def test_mask_zeros_and_values_that_are_not_finite(H, fmt, axis, dtype, cols):
    R = 70
    x = rand(3, R, cols, dtype=DT[dtype])
    keep = torch.rand(R, cols, generator=gen(4), device="cuda") < 0.5
    keep[5] = False                    # a row whose mask leaves nothing
    keep[:, 7] = False
    keep[20, :32] = False
    x[~keep] = float("nan")            # masked places may hold anything
    x[30][~keep[30]] = float("inf")
    x[9, 0], keep[9, 0] = float("nan"), True
    x[10, 33], keep[10, 33] = float("-inf"), True
    x[11] = 0.0
    pad = torch.zeros(R, -(-cols // 32) * 32, dtype=torch.long, device="cuda")
    pad[:, :cols] = keep
    words = (pad.view(R, -1, 32) << torch.arange(32, device="cuda")).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    m = np.where(keep.cpu().numpy(), np64(x), 0.0)
    g = H.hinm_fp4_quantize(x, fmt, axis=axis, bitmask=words, tensor_scale="amax" if fmt == F.NV else None)
    gv = F.pow2_scale(m) if fmt == F.NV else 1.0
    if fmt == F.NV:
        assert float(g.tensor_scale) == gv
    want = F.rounded(m if axis == 1 else m.T, fmt, gv)
    y = H.hinm_fp4_dequantize(g, axis=axis, dtype=DT[dtype])
    assert same(y, to_type(want if axis == 1 else want.T, DT[dtype]))
    if axis == 1:  # (down the columns, the blocks of row 5 hold rows 9 and 10 as well)
        assert y[5].eq(0).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 1, 4096), (1, 300, 500), (3, 257, 129), (2, 512, 1024), (70, 8, 64)])
def test_tensor_scale(H, dtype, shape):
    x = rand(sum(shape), *shape, dtype=DT[dtype], scale=3.0)
    x[0, 0, 0] = float("inf")
    x[-1, -1, -1] = float("nan") if shape != (1, 1, 1) else 0.0
    if shape[0] > 1:
        x[1] = 0.0
    q = H.Fp4Matrix.allocate(F.NV, shape[0], shape[1], shape[2], "cuda")
    got = H.hinm_fp4_tensor_scale(x, q)
    assert got.tolist() == [F.pow2_scale(np64(x[b])) for b in range(shape[0])]
    # a given scale is kept, and "amax" after it writes into another tensor
    mine = torch.full((shape[0],), 0.5, device="cuda")
    H.hinm_fp4_quantize(x, F.NV, tensor_scale=mine, out=q)
    H.hinm_fp4_quantize(x, F.NV, tensor_scale="amax", out=q)
    assert mine.eq(0.5).all() and q.tensor_scale.tolist() == [F.pow2_scale(np64(x[b])) for b in range(shape[0])]


@FORMATS
@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("offset,extra", [(0, 8), (8, 24), (1, 2), (16, 48)])
def test_strided_source_and_destination(H, fmt, axis, offset, extra):
    R, C = 50, 96
    big = torch.full((R, C + extra + offset), 9.0, dtype=torch.bfloat16, device="cuda")
    x = rand(8, R, C)
    big[:, offset:offset + C] = x
    view = big[:, offset:offset + C]
    a, b = H.hinm_fp4_quantize(view, fmt, axis=axis), H.hinm_fp4_quantize(x, fmt, axis=axis)
    assert torch.equal(a.values, b.values)
    want = H.hinm_fp4_dequantize(b, axis=axis)
    back = torch.full_like(big, -3.0)
    H.hinm_fp4_dequantize(a, axis=axis, out=back[:, offset:offset + C])
    assert torch.equal(back[:, offset:offset + C], want)
    assert back[:, :offset].eq(-3).all() and back[:, offset + C:].eq(-3).all()


@FORMATS
@pytest.mark.parametrize("axis", [1, 0])
def test_batch(H, fmt, axis):
    E, R, C = 3, 130, 72
    x = rand(12, E, R, C, scale=0.1)
    q = H.hinm_fp4_quantize(x, fmt, axis=axis, tensor_scale="amax" if fmt == F.NV else None)
    for e in range(E):
        m = np64(x[e]) if axis == 1 else np64(x[e]).T
        gv = F.pow2_scale(m) if fmt == F.NV else 1.0
        codes, sc = F.quantize(m, fmt, gv)
        check_stored(q, fmt, codes, sc, m.shape[1], e)
    y = H.hinm_fp4_dequantize(q, axis=axis)
    assert y.shape == x.shape
    m = np64(x[2]) if axis == 1 else np64(x[2]).T
    want = F.rounded(m, fmt, F.pow2_scale(m) if fmt == F.NV else 1.0)
    assert same(y[2], to_type(want if axis == 1 else want.T, torch.bfloat16))


GROUPS = [[0, 5], [0, 0, 3, 3, 40], [2, 2, 130, 300, 300], [0, 128, 256, 384], [0, 1, 2, 3, 4, 300], [7, 7, 7]]
MANY = [[0, 700, 701, 1500, 2000], [11, 11, 1290]]


@FORMATS
@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("depth,o", [(d, o) for d in (64, 200) for o in GROUPS] + [(900, o) for o in MANY], ids=str)
def test_ragged_rows(H, fmt, axis, o, depth):
    T = o[-1] + 9
    x = rand(T, T, depth)
    x[o[-1]:] = float("nan")            # behind the last group: not read
    x[:o[0]] = float("inf")
    src = x if axis == 1 else x.t().contiguous()
    q = H.Fp4Matrix.allocate(fmt, 1, T, depth, "cuda", H.HINM_RAGGED_ROWS, ints(o))
    q.values.fill_(0xA5)
    H.hinm_fp4_quantize(src, fmt, axis=axis, ragged=H.HINM_RAGGED_ROWS, offsets=ints(o), out=q,
                        tensor_scale="amax" if fmt == F.NV else None)
    real = np64(x)[o[0]:o[-1]]
    gv = F.pow2_scale(real) if fmt == F.NV else 1.0
    if fmt == F.NV:
        assert float(q.tensor_scale) == gv
    chunk = 64 if fmt == F.NV else 128
    D = -(-depth // 128) * 128
    vals = q.values.cpu().numpy()[:T * D // 2].reshape(T, -1)
    scs = q.scales.cpu().numpy()[:(T // 128 + len(o) - 1) * (D // chunk) * 512].reshape(-1, D // chunk, 512)
    for e in range(len(o) - 1):
        n = o[e + 1] - o[e]
        if n == 0:
            continue
        codes, sc = F.quantize(np64(x)[o[e]:o[e + 1]], fmt, gv)
        v, s = F.pack(codes, sc, fmt, depth)
        np.testing.assert_array_equal(vals[o[e]:o[e + 1]], v)
        r = np.arange(n)
        for b in range(4):
            at = 16 * (r % 32) + 4 * (r // 32 % 4) + b
            np.testing.assert_array_equal(scs[o[e] // 128 + e + r // 128, :, at], s[r // 128, :, at])
    assert (vals[o[-1]:] == 0xA5).all() and (vals[:o[0]] == 0xA5).all()
    out = torch.full_like(src, 5.0)
    H.hinm_fp4_dequantize(q, axis=axis, out=out)
    got = out if axis == 1 else out.t()
    assert got[o[-1]:].eq(5).all() and got[:o[0]].eq(5).all()
    if real.size:
        assert same(got[o[0]:o[-1]], to_type(F.rounded(real, fmt, gv), torch.bfloat16))


@FORMATS
@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("rows,o", [(r, o) for r in (24, 131) for o in GROUPS] + [(516, o) for o in MANY], ids=str)
def test_ragged_depth(H, fmt, axis, o, rows):
    T = o[-1] + 9
    x = rand(T + 1, T, rows)             # tokens x rows: axis 0
    x[o[-1]:] = float("nan")
    src = x if axis == 0 else x.t().contiguous()
    q = H.hinm_fp4_quantize(src, fmt, axis=axis, ragged=H.HINM_RAGGED_DEPTH, offsets=ints(o),
                            tensor_scale="amax" if fmt == F.NV else None)
    real = np64(x)[o[0]:o[-1]]
    gv = F.pow2_scale(real) if fmt == F.NV else 1.0
    G = len(o) - 1
    D = 128 * (T // 128 + G)
    vals = q.values.cpu().numpy()[:rows * D // 2].reshape(rows, -1)
    for e in range(G):
        n = o[e + 1] - o[e]
        if n == 0:
            continue
        codes, sc = F.quantize(np64(x)[o[e]:o[e + 1]].T, fmt, gv)
        v, _ = F.pack(codes, sc, fmt, n)
        at = 64 * (o[e] // 128 + e)
        np.testing.assert_array_equal(vals[:, at:at + v.shape[1]], v)   # zeros up to 128 among them
    out = torch.full_like(src, 5.0)
    H.hinm_fp4_dequantize(q, axis=axis, out=out)
    got = out if axis == 0 else out.t()
    assert got[o[-1]:].eq(5).all() and got[:o[0]].eq(5).all()
    for e in range(G):
        if o[e + 1] > o[e]:
            want = F.rounded(np64(x)[o[e]:o[e + 1]].T, fmt, gv).T
            assert same(got[o[e]:o[e + 1]], to_type(want, torch.bfloat16))


def mask_words(keep):
    """bool [..., rows, cols] -> hinm_mask's words."""
    cols = keep.shape[-1]
    pad = torch.zeros(*keep.shape[:-1], -(-cols // 32) * 32, dtype=torch.long, device="cuda")
    pad[..., :cols] = keep
    words = (pad.unflatten(-1, (-1, 32)) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


@FORMATS
@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols,offset,extra", [(640, 1216, 0, 0), (645, 1219, 0, 0), (645, 1219, 3, 2),
                                                    (512, 1024, 1, 7), (700, 1000, 8, 16)])
@pytest.mark.parametrize("masked", [False, True])
def test_many_blocks(H, fmt, axis, dtype, rows, cols, offset, extra, masked):
    """Several blocks of threads in each direction; rows that start at any element."""
    big = torch.full((rows, offset + cols + extra), float("nan"), dtype=DT[dtype], device="cuda")
    x = big[:, offset:offset + cols]
    x.copy_(rand(rows + cols, rows, cols, dtype=DT[dtype]))
    keep = torch.ones(rows, cols, dtype=torch.bool, device="cuda")
    if masked:
        keep = torch.rand(rows, cols, generator=gen(6), device="cuda") < 0.3
        x[~keep] = float("nan")
    q = H.hinm_fp4_quantize(x, fmt, axis=axis, bitmask=mask_words(keep) if masked else None,
                            tensor_scale="amax" if fmt == F.NV else None)
    m = np.where(keep.cpu().numpy(), np64(x), 0.0)
    m = m if axis == 1 else m.T
    gv = F.pow2_scale(m) if fmt == F.NV else 1.0
    if fmt == F.NV:
        assert float(q.tensor_scale) == gv
    codes, sc = F.quantize(m, fmt, gv)
    check_stored(q, fmt, codes, sc, m.shape[1])
    want = F.values(codes, sc, fmt, m.shape[1], gv)
    back = torch.full_like(big, -3.0)
    H.hinm_fp4_dequantize(q, axis=axis, out=back[:, offset:offset + cols])
    assert same(back[:, offset:offset + cols], to_type(want if axis == 1 else want.T, DT[dtype]))
    assert back[:, :offset].eq(-3).all() and back[:, offset + cols:].eq(-3).all()


@FORMATS
@pytest.mark.parametrize("axis", [1, 0])
def test_masked_batch(H, fmt, axis):
    E, R, C = 3, 150, 75
    x = rand(2, E, R, C, dtype=torch.float32)
    keep = torch.rand(E, R, C, generator=gen(3), device="cuda") < 0.5
    x[~keep] = float("inf")
    keep[1] = False                     # an expert without any weight
    q = H.hinm_fp4_quantize(x, fmt, axis=axis, bitmask=mask_words(keep), tensor_scale="amax" if fmt == F.NV else None)
    y = H.hinm_fp4_dequantize(q, axis=axis, dtype=torch.float32)
    assert y[1].eq(0).all()
    for e in range(E):
        m = np.where(keep[e].cpu().numpy(), np64(x[e]), 0.0)
        m = m if axis == 1 else m.T
        want = F.rounded(m, fmt, F.pow2_scale(m) if fmt == F.NV else 1.0)
        assert same(y[e], to_type(want if axis == 1 else want.T, torch.float32))


# ----------------------------------------------------------------------------- products
def operands(H, seed, M, N, K, fmt, scale="amax"):
    """A and B as 4-bit matrices and their values in 64 bits with the scales in them."""
    out = []
    for i, rows in enumerate((M, N)):
        x = rand(seed + i, rows, K, scale=0.05 if i == 0 else 1.0)
        q = H.hinm_fp4_quantize(x, fmt, tensor_scale=scale if fmt == F.NV else None)
        out += [q, np64(H.hinm_fp4_dequantize(q, dtype=torch.float32))]
    return out[0], out[2], out[1], out[3]


def check_product(y, a, b, bias=None, act=0, dtype=None):
    """y [M, N] against a b^T in 64 bits within the bound of the header."""
    dtype = dtype or y.dtype
    K = a.shape[1]
    want = a @ b.T
    mag = np.abs(a) @ np.abs(b).T
    h = 2.0 ** -24
    err = (K + 3) * h * mag
    if bias is not None:
        want = want + bias[:, None]
        err = err + h * (mag + np.abs(bias)[:, None])
    z = F.activate(want, act)
    if act:
        err = 1.13 * err + 16 * h * np.abs(want)
    err = err + torch.finfo(dtype).eps / 2 * (np.abs(z) + err) + 2.0 ** -24 * (dtype == torch.float16)
    got = np64(y)
    bad = ~(np.abs(got - z) <= err)
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - z) - err).max()))


SHAPES = [(1, 1, 1), (1, 1, 300), (128, 16, 128), (130, 17, 65), (256, 1, 4096), (100, 64, 700), (300, 65, 512),
          (129, 129, 129), (257, 200, 1000), (512, 256, 1024), (640, 513, 384), (1000, 777, 1547), (64, 1024, 2048)]


@FORMATS
@pytest.mark.parametrize("transposed", [False, True], ids=["MN", "NM"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul(H, fmt, transposed, M, N, K):
    A, B, a, b = operands(H, M + N + K, M, N, K, fmt)
    for dtype in DT.values():
        y = H.hinm_fp4_matmul(A, B, dtype=dtype, transposed=transposed)
        check_product(y.t() if transposed else y, a, b)


@FORMATS
@pytest.mark.parametrize("M,N,K", [(4096, 1024, 512), (2304, 4096, 768), (1100, 2500, 260), (256, 20000, 130)])
def test_matmul_large(H, fmt, M, N, K):
    """Sizes that take pairs of CTAs and several rounds of tiles."""
    A, B, a, b = operands(H, 5, M, N, K, fmt)
    for transposed in (False, True):
        y = H.hinm_fp4_matmul(A, B, dtype=torch.float32, transposed=transposed)
        check_product(y.t() if transposed else y, a, b)


@pytest.mark.parametrize("transposed", [False, True], ids=["MN", "NM"])
@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,N,K", [(200, 3, 2048), (384, 320, 256), (70, 100, 96), (2304, 2100, 128)])
def test_bias_and_activation(H, transposed, act, dtype, M, N, K):
    A, B, a, b = operands(H, act, M, N, K, F.NV)
    bias = torch.randn(M, generator=gen(1), device="cuda")
    y = H.hinm_fp4_matmul(A, B, dtype=DT[dtype], transposed=transposed, bias=bias, activation=act)
    check_product(y.t() if transposed else y, a, b, np64(bias), act)


def whole(seed, rows, K):
    """Values that both formats hold exactly whatever the blocks: 0, +-1 .. +-6 with a 6 in every block of
    16 along both dimensions."""
    v = torch.tensor([0, 1, 2, 3, 4, 6, -1, -2, -3, -4, -6], device="cuda")
    x = v[torch.randint(len(v), (rows, K), generator=gen(seed), device="cuda")].float()
    r, c = torch.arange(rows, device="cuda")[:, None], torch.arange(K, device="cuda")[None]
    x[(r + c) % 16 == 0] = 6.0
    return x.bfloat16()


@FORMATS
@pytest.mark.parametrize("M,N,K", [(256, 1, 2048), (300, 70, 640), (512, 512, 512), (2560, 2304, 320), (129, 257, 4096)])
def test_whole_numbers_bit_for_bit(H, fmt, M, N, K):
    x, w = whole(2, N, K), whole(1, M, K)
    A, B = H.hinm_fp4_quantize(w, fmt), H.hinm_fp4_quantize(x, fmt)
    assert torch.equal(H.hinm_fp4_dequantize(A), w) and torch.equal(H.hinm_fp4_dequantize(B), x)
    want = w.double() @ x.double().t()
    for transposed in (False, True):
        y = H.hinm_fp4_matmul(A, B, dtype=torch.float32, transposed=transposed)
        assert torch.equal(y, (want.t() if transposed else want).float())
        for _ in range(2):  # and the same every time
            assert torch.equal(H.hinm_fp4_matmul(A, B, dtype=torch.float32, transposed=transposed), y)


@pytest.mark.parametrize("transposed", [False, True], ids=["MN", "NM"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset,pad", [(0, 0), (3, 5), (8, 8), (16, 48)])
@pytest.mark.parametrize("M,N", [(200, 40), (256, 384), (190, 300)])
def test_strided_output(H, transposed, dtype, offset, pad, M, N):
    A, B, a, b = operands(H, 9, M, N, 256, F.MX)
    r, c = (N, M) if transposed else (M, N)
    big = torch.full((r, c + offset + pad), 7.0, dtype=DT[dtype], device="cuda")
    view = big[:, offset:offset + c]
    H.hinm_fp4_matmul(A, B, Y_out=view, transposed=transposed)
    check_product(view.t() if transposed else view, a, b)
    assert big[:, :offset].eq(7).all() and big[:, offset + c:].eq(7).all()


@FORMATS
@pytest.mark.parametrize("M,N,K", [(300, 40, 300), (512, 640, 512)])
def test_nan_stays_in_its_row_and_column(H, fmt, M, N, K):
    w, x = rand(1, M, K), rand(2, N, K)
    w[17, 5] = float("nan")
    x[33, K - 1] = float("inf")
    A, B = H.hinm_fp4_quantize(w, fmt), H.hinm_fp4_quantize(x, fmt)
    y = H.hinm_fp4_matmul(A, B, dtype=torch.float32)
    nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    nan[17], nan[:, 33] = True, True
    assert torch.equal(y.isnan(), nan)


@pytest.mark.parametrize("transposed", [False, True], ids=["MN", "NM"])
@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("M,N,K", [(300, 40, 300), (256, 4, 4096), (512, 640, 512), (2304, 2112, 256)])
def test_nan_passes_every_activation(H, transposed, act, M, N, K):
    w, x = rand(1, M, K), rand(2, N, K)
    w[17, 5] = float("nan")
    A, B = H.hinm_fp4_quantize(w, F.MX), H.hinm_fp4_quantize(x, F.MX)
    bias = torch.zeros(M, device="cuda")
    bias[20] = float("nan")
    y = H.hinm_fp4_matmul(A, B, transposed=transposed, bias=bias, activation=act)
    y = y.t() if transposed else y
    nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    nan[17], nan[20] = True, True
    assert torch.equal(y.isnan(), nan)


def test_places_past_32_bits(H):
    """A source, a matrix and a product of more than 2^31 elements: their last rows against the same
    rows alone.  (More than 2^32 bytes: 4.6 GB each.)"""
    R, C = 70016, 32768
    assert R * C > 2 ** 31
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    for r in range(0, R, 8752):
        x[r:r + 8752] = rand(r, 8752, C)
    tail = slice(R - 200, R)
    q = H.hinm_fp4_quantize(x, F.MX)
    few = H.hinm_fp4_quantize(x[tail].contiguous(), F.MX)
    assert torch.equal(q.values[-200 * C // 2:], few.values[:200 * C // 2])
    y = H.hinm_fp4_dequantize(q)
    assert torch.equal(y[tail], H.hinm_fp4_dequantize(few))
    del q, y
    q = H.hinm_fp4_quantize(x, F.NV, axis=0)       # the transpose: 32768 rows of depth 70016
    y = H.hinm_fp4_dequantize(q, axis=0)
    few = H.hinm_fp4_quantize(x[R - 256:].contiguous(), F.NV, axis=0)   # whole blocks of the depth
    assert torch.equal(y[R - 256:], H.hinm_fp4_dequantize(few, axis=0))
    del q, y, x
    A, B, a, b = operands(H, 9, R, C, 128, F.MX)
    Y = H.hinm_fp4_matmul(A, B)
    check_product(Y[tail, -300:], a[tail], b[-300:])
    check_product(Y[:100, :300], a[:100], b[:300])
    H.hinm_fp4_matmul(B, A, Y_out=Y, transposed=True)    # the same products, by the other path
    check_product(Y[tail, -300:], a[tail], b[-300:])


# ----------------------------------------------------------------------------- products by expert
EXPERTS = [
    ([0, 3, 3, 10], 96, 64), ([0, 0, 0, 1], 130, 200), ([0, 70, 200, 201, 201, 460], 260, 130),
    ([5, 40, 300], 64, 256), ([0, 0, 0], 40, 64), ([0, 600, 600, 1500], 512, 384), ([0] + [1] * 30 + [7], 128, 512),
    ([0, 1000, 1001, 1700, 3000], 300, 520),
]


@FORMATS
@pytest.mark.parametrize("transposed", [False, True], ids=["MN", "NM"])
@pytest.mark.parametrize("o,M,K", EXPERTS, ids=str)
@pytest.mark.parametrize("biased", [False, True])
def test_grouped_matmul(H, fmt, transposed, o, M, K, biased):
    E, T = len(o) - 1, o[-1] + 6
    w, x = rand(1, E, M, K, scale=0.05), rand(2, T, K)
    x[o[-1]:] = float("nan")
    amax = "amax" if fmt == F.NV else None
    A = H.hinm_fp4_quantize(w, fmt, tensor_scale=amax)
    B = H.hinm_fp4_quantize(x, fmt, ragged=H.HINM_RAGGED_ROWS, offsets=ints(o), tensor_scale=amax)
    a = np64(H.hinm_fp4_dequantize(A, dtype=torch.float32)).reshape(E, M, K)
    b = np64(H.hinm_fp4_dequantize(B, dtype=torch.float32))
    bias = torch.randn(E, M, generator=gen(3), device="cuda") if biased else None
    act = 2 if biased else 0
    for dtype in (torch.bfloat16, torch.float32):
        Y = torch.full((T, M) if transposed else (M, T), 4.0, dtype=dtype, device="cuda")
        H.hinm_fp4_grouped_matmul(A, B, Y_out=Y, transposed=transposed, bias=bias, activation=act)
        y = Y.t() if transposed else Y
        for e in range(E):
            if o[e + 1] > o[e]:
                check_product(y[:, o[e]:o[e + 1]], a[e], b[o[e]:o[e + 1]], np64(bias)[e] if biased else None, act)
        assert y[:, o[-1]:].eq(4).all() and y[:, :o[0]].eq(4).all()


@FORMATS
@pytest.mark.parametrize("o,M,N", [([0, 3, 3, 10], 96, 64), ([2, 130, 130, 700], 260, 129), ([0, 0, 0], 40, 64),
                                   ([0, 128, 256], 128, 512), ([0, 1000, 1001, 1700, 3000], 300, 520)], ids=str)
def test_grouped_weight_grad(H, fmt, o, M, N):
    E, T = len(o) - 1, o[-1] + 6
    d, x = rand(1, T, M, scale=1e-3), rand(2, T, N)
    d[o[-1]:], x[o[-1]:] = float("nan"), float("nan")
    q = [H.hinm_fp4_quantize(t, fmt, axis=0, ragged=H.HINM_RAGGED_DEPTH, offsets=ints(o),
                             tensor_scale="amax" if fmt == F.NV else None) for t in (d, x)]
    dq, xq = (np64(H.hinm_fp4_dequantize(t, axis=0, dtype=torch.float32)) for t in q)
    for dtype in (torch.bfloat16, torch.float32):
        big = torch.full((E, M, N + 3), 4.0, dtype=dtype, device="cuda")
        H.hinm_fp4_grouped_weight_grad(q[0], q[1], Y_out=big[:, :, :N])
        for e in range(E):
            if o[e + 1] > o[e]:
                check_product(big[e, :, :N], dq[o[e]:o[e + 1]].T, xq[o[e]:o[e + 1]].T)
            else:
                assert big[e, :, :N].eq(0).all()
        assert big[:, :, N:].eq(4).all()


def test_no_tokens_at_all(H):
    o = ints([0, 0, 0])
    A = H.hinm_fp4_quantize(rand(1, 2, 64, 64), F.MX)
    B = H.hinm_fp4_quantize(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), F.MX,
                            ragged=H.HINM_RAGGED_ROWS, offsets=o)
    assert H.hinm_fp4_grouped_matmul(A, B).shape == (64, 0)
    d = [H.hinm_fp4_quantize(torch.empty(0, n, dtype=torch.bfloat16, device="cuda"), F.NV, axis=0,
                             ragged=H.HINM_RAGGED_DEPTH, offsets=o, tensor_scale="amax") for n in (32, 48)]
    y = H.hinm_fp4_grouped_weight_grad(d[0], d[1], Y_out=torch.full((2, 32, 48), 3.0, device="cuda"))
    assert y.eq(0).all()


def test_many_experts(H):
    E, M, K = 512, 32, 64
    n = torch.randint(0, 4, (E,), generator=torch.Generator().manual_seed(1))
    o = [0] + n.cumsum(0).tolist()
    w, x = whole(1, E * M, K).view(E, M, K), whole(2, o[-1], K)
    A = H.hinm_fp4_quantize(w, F.NV)
    B = H.hinm_fp4_quantize(x, F.NV, ragged=H.HINM_RAGGED_ROWS, offsets=ints(o))
    y = H.hinm_fp4_grouped_matmul(A, B, dtype=torch.float32, transposed=True)
    e = torch.repeat_interleave(torch.arange(E), n).cuda()
    assert torch.equal(y, torch.einsum("tk,tmk->tm", x.double(), w.double()[e]).float())


@pytest.mark.parametrize("o", [[0, 9, 5, 20], [0, 5, 30], [-4, 5, 20], [3, 2, 20]], ids=str)
def test_bad_offsets_are_reported(H, o):
    """Offsets that decrease or leave the matrix: the status word says so, nothing outside the matrices
    is touched and the products write nothing."""
    T, E, M, K = 20, len(o) - 1, 48, 64
    x, w = rand(1, T, K), rand(2, E, M, K)
    A = H.hinm_fp4_quantize(w, F.MX)
    good = H.hinm_fp4_quantize(x, F.MX, ragged=H.HINM_RAGGED_ROWS, offsets=ints([0] * E + [T]))
    assert H.hinm_device_status() == 0
    good.offsets = ints(o)
    Y = torch.full((T, M), 2.0, dtype=torch.bfloat16, device="cuda")
    H.hinm_fp4_grouped_matmul(A, good, Y_out=Y, transposed=True)
    assert H.hinm_device_status() == H.HINM_ERR_INVALID_ARG and Y.eq(2).all()
    d = [H.hinm_fp4_quantize(t, F.MX, axis=0, ragged=H.HINM_RAGGED_DEPTH, offsets=ints([0] * E + [T]))
         for t in (rand(3, T, M), x)]
    d[1].offsets = ints(o)
    G = torch.full((E, M, K), 2.0, device="cuda")
    H.hinm_fp4_grouped_weight_grad(d[0], d[1], Y_out=G)
    assert H.hinm_device_status() == H.HINM_ERR_INVALID_ARG and G.eq(2).all()
    for axis, ragged in ((1, H.HINM_RAGGED_ROWS), (0, H.HINM_RAGGED_DEPTH)):  # in bounds whatever comes
        q = H.hinm_fp4_quantize(x, F.NV, axis=axis, ragged=ragged, offsets=ints(o), tensor_scale="amax")
        out = torch.full_like(x, 1.0)
        H.hinm_fp4_dequantize(q, axis=axis, out=out)
        H.hinm_device_status()


# ----------------------------------------------------------------------------- together
@FORMATS
@pytest.mark.parametrize("M,K,N", [(256, 192, 96), (144, 320, 400)])
def test_linear_layer_and_its_gradients(H, fmt, M, K, N):
    """Y = W X, dX = W^T dY, dW = dY X^T in the library's own layout, each product of operands quantised
    along its summed dimension: against the formula in 64 bits on the rounded operands."""
    W, X, dY = rand(1, M, K, scale=0.05), rand(2, K, N), rand(3, M, N, scale=1e-3)
    amax = "amax" if fmt == F.NV else None
    q = lambda t, axis: H.hinm_fp4_quantize(t, fmt, axis=axis, tensor_scale=amax)  # noqa: E731
    r = lambda t, axis: (lambda m: F.rounded(m, fmt, F.pow2_scale(m) if fmt == F.NV else 1.0))(  # noqa: E731
        np64(t) if axis == 1 else np64(t).T)
    check_product(H.hinm_fp4_matmul(q(W, 1), q(X, 0)), r(W, 1), r(X, 0))
    check_product(H.hinm_fp4_matmul(q(W, 0), q(dY, 0)), r(W, 0), r(dY, 0))
    check_product(H.hinm_fp4_matmul(q(dY, 1), q(X, 1), dtype=torch.float32), r(dY, 1), r(X, 1))


@FORMATS
def test_gradients_against_differences(H, fmt):
    """On values that 4 bits hold exactly, rounding is the identity along either axis, so the loss
    sum(dY * (W X)) is linear in each operand: its differences are the gradients, exactly."""
    M, K, N = 96, 80, 64
    W, X, dY = whole(1, M, K), whole(2, K, N), whole(3, M, N)
    q = lambda t, axis: H.hinm_fp4_quantize(t.contiguous(), fmt, axis=axis)  # noqa: E731
    loss = lambda w, x: float((H.hinm_fp4_matmul(q(w, 1), q(x, 0), dtype=torch.float32).double()  # noqa: E731
                               * dY.double()).sum())
    dX = H.hinm_fp4_matmul(q(W, 0), q(dY, 0), dtype=torch.float32)
    dW = H.hinm_fp4_matmul(q(dY, 1), q(X, 1), dtype=torch.float32)
    base = loss(W, X)
    for i, j, to in [(0, 1, 3.0), (79, 63, -2.0), (40, 17, 0.0), (33, 2, 4.0)]:
        X2 = X.clone()
        step = to - float(X[i, j]) if (i + j) % 16 else 0.0  # the 6 of a block stays
        X2[i, j] += step
        assert loss(W, X2) - base == step * float(dX[i, j])
    for i, j, to in [(0, 1, 3.0), (95, 79, -2.0), (50, 17, 0.0)]:
        W2 = W.clone()
        step = to - float(W[i, j]) if (i + j) % 16 else 0.0
        W2[i, j] += step
        assert loss(W2, X) - base == step * float(dW[i, j])


@FORMATS
def test_expert_layer_forward_and_backward(H, fmt):
    """Two expert products with an activation between them, token by token, then the gradients of the
    second: dX by expert and dW by expert, from the same offsets on the device."""
    E, D, M = 4, 192, 320
    o = [0, 37, 37, 300, 311]
    T, off = o[-1] + 3, ints(o)
    amax = "amax" if fmt == F.NV else None
    x, w1, w2 = rand(1, T, D), rand(2, E, M, D, scale=0.05), rand(3, E, D, M, scale=0.05)
    rag = dict(ragged=H.HINM_RAGGED_ROWS, offsets=off, tensor_scale=amax)
    q1, q2 = (H.hinm_fp4_quantize(w, fmt, tensor_scale=amax) for w in (w1, w2))
    h = H.hinm_fp4_grouped_matmul(q1, H.hinm_fp4_quantize(x, fmt, **rag), transposed=True,
                                  activation=H.HINM_ACT_SILU)
    y = H.hinm_fp4_grouped_matmul(q2, H.hinm_fp4_quantize(h, fmt, **rag), transposed=True)
    rr = lambda m, all_: F.rounded(m, fmt, F.pow2_scale(all_) if fmt == F.NV else 1.0)  # noqa: E731
    hs = np64(h)
    dy = rand(5, T, D, scale=1e-2)
    dh = H.hinm_fp4_grouped_matmul(H.hinm_fp4_quantize(w2, fmt, axis=0, tensor_scale=amax),
                                   H.hinm_fp4_quantize(dy, fmt, **rag), transposed=True)
    dep = dict(axis=0, ragged=H.HINM_RAGGED_DEPTH, offsets=off, tensor_scale=amax)
    dw = H.hinm_fp4_grouped_weight_grad(H.hinm_fp4_quantize(dy, fmt, **dep), H.hinm_fp4_quantize(h, fmt, **dep))
    assert y[o[-1]:].eq(0).all() and dh[o[-1]:].eq(0).all()
    for e in range(E):
        s = slice(o[e], o[e + 1])
        if o[e + 1] == o[e]:
            assert dw[e].eq(0).all()
            continue
        xs, dys, live = np64(x)[s], np64(dy)[s], slice(0, o[-1])
        check_product(h[s].t(), rr(np64(w1[e]), np64(w1[e])), rr(xs, np64(x)[live]), act=2)
        check_product(y[s].t(), rr(np64(w2[e]), np64(w2[e])), rr(hs[s], hs[live]))
        check_product(dh[s].t(), rr(np64(w2[e]).T, np64(w2[e])), rr(dys, np64(dy)[live]))
        check_product(dw[e], rr(dys.T, np64(dy)[live]), rr(hs[s].T, hs[live]))


def test_pruned_weight_in_4_bits(H):
    """The path's own mask (importance, boundary search, mask) on the weight that is quantised: what it
    prunes is 0 and takes no part in the scales."""
    M, K, N, T = 256, 512, 64, 128
    W, X = rand(1, M, K, scale=0.02), rand(2, K, N)
    I, stats = H.hinm_importance_stats(W, X, T)
    counts, _, rank = H.hinm_boundary_search(I, None, T, 0.5, stats=stats)
    bits, _ = H.hinm_mask(I, None, counts, T, rank)
    q = H.hinm_fp4_quantize(W, F.NV, bitmask=bits, tensor_scale="amax")
    keep = ((bits.cpu().numpy().view(np.uint32)[..., None] >> np.arange(32)) & 1).reshape(M, -1)[:, :K]
    m = np.where(keep > 0, np64(W), 0.0)
    assert same(H.hinm_fp4_dequantize(q), to_type(F.rounded(m, F.NV, F.pow2_scale(m)), torch.bfloat16))
    assert 0.4 < keep.mean() < 0.6
    B = H.hinm_fp4_quantize(X, F.NV, axis=0, tensor_scale="amax")
    check_product(H.hinm_fp4_matmul(q, B), F.rounded(m, F.NV, F.pow2_scale(m)),
                  F.rounded(np64(X).T, F.NV, F.pow2_scale(np64(X))))


# ----------------------------------------------------------------------------- streams and graphs
def test_another_stream(H):
    A, B, a, b = operands(H, 3, 300, 40, 512, F.NV)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    x = rand(7, 64, 512)
    torch.cuda.synchronize()
    y1 = H.hinm_fp4_matmul(A, B, Y_out=torch.empty(300, 40, device="cuda"), stream=s1)  # two at once
    with torch.cuda.stream(s2):
        q = H.hinm_fp4_quantize(x, F.NV, tensor_scale="amax")
        y2 = H.hinm_fp4_matmul(A, q, dtype=torch.float32)
    torch.cuda.synchronize()
    check_product(y1, a, b)
    check_product(y2, a, F.rounded(np64(x), F.NV, F.pow2_scale(np64(x))))


def test_what_a_call_makes_belongs_to_its_stream(H):
    """A call on a given stream while the current one is busy: its new tensors are filled on the stream
    that writes them."""
    o = [0, 30, 30, 60]
    x, w = rand(1, 70, 256), rand(2, 3, 96, 256)
    s = torch.cuda.Stream()
    ragged = dict(ragged=H.HINM_RAGGED_ROWS, offsets=ints(o))
    A = H.hinm_fp4_quantize(w, F.NV, tensor_scale="amax")
    want = H.hinm_fp4_quantize(x, F.NV, tensor_scale="amax", **ragged)
    want_x = H.hinm_fp4_dequantize(want)
    want_y = H.hinm_fp4_grouped_matmul(A, want)
    for busy in (False, True):                     # (the first time, memory for the stream is found)
        torch.cuda.synchronize()
        if busy:
            torch.cuda._sleep(20_000_000)          # some 10 ms of the current stream
        q = H.hinm_fp4_quantize(x, F.NV, tensor_scale="amax", stream=s, **ragged)
        back = H.hinm_fp4_dequantize(q, stream=s)
        y = H.hinm_fp4_grouped_matmul(A, q, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(q.tensor_scale, want.tensor_scale)
    assert torch.equal(back, want_x) and torch.equal(y, want_y)


def test_a_refused_call_leaves_the_matrix_as_it_was(H):
    x = rand(1, 64, 256)
    off = ints([0, 20, 64])
    rag = dict(ragged=H.HINM_RAGGED_ROWS, offsets=off)
    q = H.hinm_fp4_quantize(x, F.NV, tensor_scale="amax", **rag)
    want, g = H.hinm_fp4_dequantize(q), q.tensor_scale
    bad = [dict(rag, tensor_scale=torch.ones(1, dtype=torch.float64, device="cuda")),
           dict(rag, tensor_scale=torch.ones(1)), dict(rag, tensor_scale="max"),
           dict(rag, offsets=off.long()), dict(rag, offsets=off.cpu()), dict(rag, offsets=ints([0, 64])),
           dict(rag, offsets=None), dict(rag, ragged=H.HINM_RAGGED_DEPTH)]
    for k in bad:
        with pytest.raises(ValueError):
            H.hinm_fp4_quantize(-x, F.NV, out=q, **k)
    with pytest.raises(ValueError):
        H.hinm_fp4_quantize(-x[:60], F.NV, out=q, **dict(rag, offsets=ints([0, 20, 60])))
    assert q.offsets is off and q.tensor_scale is g
    assert torch.equal(H.hinm_fp4_dequantize(q), want)


def test_graph_replay(H):
    """A captured expert layer: new tokens and new offsets in the same buffers, replayed."""
    E, M, K, T = 4, 160, 256, 64
    w = rand(1, E, M, K, scale=0.05)
    A = H.hinm_fp4_quantize(w, F.NV, tensor_scale="amax")
    x, off = rand(2, T, K), ints([0, 10, 10, 40, 64])
    rag = dict(ragged=H.HINM_RAGGED_ROWS, offsets=off, tensor_scale="amax")
    q = H.hinm_fp4_quantize(x, F.NV, **rag)
    Y = torch.zeros(T, M, dtype=torch.bfloat16, device="cuda")

    def step():
        H.hinm_fp4_quantize(x, F.NV, out=q, **rag)
        H.hinm_fp4_grouped_matmul(A, q, Y_out=Y, transposed=True, activation=H.HINM_ACT_GELU)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed, o in [(3, [0, 10, 10, 40, 64]), (4, [0, 64, 64, 64, 64]), (5, [0, 1, 2, 3, 4])]:
        x.copy_(rand(seed, T, K))
        off.copy_(ints(o))
        Y.zero_()
        g.replay()
        got = Y.clone()
        Y.zero_()
        step()
        assert torch.equal(got, Y) and bool(got[:o[-1]].ne(0).any())
        assert got[o[-1]:].eq(0).all()
    del g


def test_buffers_that_move_are_seen(H):
    """A matrix whose tensors are exchanged, or whose memory moves, is described anew."""
    x = rand(1, 32, 64)
    q = H.hinm_fp4_quantize(x, F.MX)
    want = H.hinm_fp4_dequantize(q)
    q.values = q.values.clone()
    H.hinm_fp4_quantize(-x, F.MX, out=q)
    assert torch.equal(H.hinm_fp4_dequantize(q), -want)
    q.values.data = torch.zeros_like(q.values)
    assert H.hinm_fp4_dequantize(q).eq(0).all()
    q.values = q.values[:100]
    with pytest.raises(ValueError, match="values"):
        H.hinm_fp4_dequantize(q)
