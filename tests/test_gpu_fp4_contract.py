"""What the header promises of the 4-bit calls beyond their values: what is reported, how exact the
activations are in the tails, and every cut of a product, whichever sizes the library takes it for."""
import numpy as np
import pytest

import fp4_cuts
from oracle import fp4_oracle as F

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
FORMATS = pytest.mark.parametrize("fmt", [F.NV, F.MX], ids=["nv", "mx"])


@pytest.fixture(scope="module")
def H():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import pruning_hinm_spmm_b200 as H
    yield H
    assert H.hinm_device_status() == 0


def rand(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def ints(o):
    return torch.tensor(o, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------------- offsets
BAD = [[0, 9, 5, 300], [0, 5, 310], [-4, 5, 300], [3, 2, 300], [0, 200, 100, 300], [0, 300, 299], [0, 301],
       list(range(0, 200)) + [150, 300]]
GOOD = [[0, 9, 9, 300], [5, 5, 5], [0, 300], [300, 300], [0, 0, 0, 299], list(range(0, 200)) + [300]]


@FORMATS
@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("ragged", ["rows", "depth"])
@pytest.mark.parametrize("o,bad", [(o, True) for o in BAD] + [(o, False) for o in GOOD],
                         ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("other", [40, 129])
def test_every_call_reports_bad_offsets_by_itself(H, fmt, axis, ragged, o, bad, other):
    """300 tokens: the scale, the codes and the way back each set the status word; good offsets never do."""
    T, form = 300, H.HINM_RAGGED_ROWS if ragged == "rows" else H.HINM_RAGGED_DEPTH
    tokens_first = (ragged == "rows") == (axis == 1)
    x = rand(1, *((T, other) if tokens_first else (other, T)))
    rows, depth = (T, other) if ragged == "rows" else (other, T)
    want = H.HINM_ERR_INVALID_ARG if bad else 0
    q = H.Fp4Matrix.allocate(fmt, 1, rows, depth, "cuda", form, ints(o))
    q.values.zero_()
    q.scales.zero_()
    assert H.hinm_device_status() == 0
    if fmt == F.NV:
        H.hinm_fp4_tensor_scale(x, q, axis=axis)
        assert H.hinm_device_status() == want
        q.tensor_scale.fill_(1.0)
    H.hinm_fp4_quantize(x, fmt, axis=axis, ragged=form, offsets=q.offsets, out=q,
                        tensor_scale=q.tensor_scale)
    assert H.hinm_device_status() == want
    H.hinm_fp4_dequantize(q, axis=axis, out=torch.empty_like(x))
    assert H.hinm_device_status() == want
    wide = torch.empty(x.shape[0], x.shape[1] + 3, dtype=x.dtype, device="cuda")[:, 3:]  # rows that start anywhere
    wide.copy_(x)
    H.hinm_fp4_quantize(wide, fmt, axis=axis, ragged=form, offsets=q.offsets, out=q, tensor_scale=q.tensor_scale)
    assert H.hinm_device_status() == want
    H.hinm_fp4_dequantize(q, axis=axis, out=wide)
    assert H.hinm_device_status() == want


@pytest.mark.parametrize("E,R,C", [(300, 64, 600), (513, 257, 131), (1500, 40, 64), (1200, 128, 300)])
def test_scales_of_many_matrices(H, E, R, C):
    """More matrices than the grid has blocks for, each of one block or of several."""
    x = rand(1, E, R, C) * torch.exp2(torch.arange(E, device="cuda") % 40 - 20)[:, None, None].bfloat16()
    x[E // 2] = 0
    q = H.Fp4Matrix.allocate(F.NV, E, R, C, "cuda")
    got = H.hinm_fp4_tensor_scale(x, q).double().cpu().numpy()
    amax = x.abs().amax((1, 2)).double().cpu().numpy()
    assert got.tolist() == [F.pow2_scale([a]) for a in amax]


# ----------------------------------------------------------------------------- activations
def silu64(z):
    e = np.exp(-np.abs(z))
    return np.where(z < 0, z * e, z) / (1 + e)


def arguments():
    """Both tails to where the result is 0 or the argument, both sides of 0 from the smallest number on."""
    line = np.linspace(-115.0, 115.0, 5000)
    small = np.logspace(-45, 38.5, 900)
    z = np.concatenate([line, np.linspace(-16, 3, 2000), small, -small, [0.0, -0.0, 3.4e38, -3.4e38]])
    return z.astype(np.float32)


def of_bias(H, z, dtype, act, N, K, transposed):
    """act(z) for each z, as the bias of a product of zeros: [len(z)] rows of N equal columns."""
    M = len(z)
    A = H.hinm_fp4_quantize(torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), F.MX)
    B = H.hinm_fp4_quantize(rand(1, N, K), F.MX)
    y = H.hinm_fp4_matmul(A, B, dtype=dtype, transposed=transposed, bias=torch.from_numpy(z).cuda(), activation=act)
    y = y.t() if transposed else y
    assert ((y == y[:, :1]) | (y.isnan() & y[:, :1].isnan())).all()
    return y[:, 0].double().cpu().numpy()


def check_tails(got, want, dtype, own):
    """own: the activation's own error relative to the value.  Besides it the store rounds by half a step,
    relative where the value is normal in dtype and of the smallest subnormal where it is not; 2^-140 stands
    for what goes under in fp32 on the way.  What is at least half a step past dtype's largest number is
    infinite: that number is (2 - eps) 2^e, steps there are eps 2^e, so the border is (2 - eps / 2) 2^e (fp16:
    65520)."""
    info = torch.finfo(dtype)
    store = 0.0 if dtype == torch.float32 else info.eps / 2
    over = np.abs(want) >= (2 - info.eps / 2) * 2.0 ** np.floor(np.log2(info.max))
    assert np.array_equal(np.isinf(got), over)
    err = np.abs(want) * (own + store * (1 + own)) + 2.0 ** -140 + info.tiny * info.eps / 2
    bad = ~over & ~(np.abs(got - want) <= err)
    assert not bad.any(), (int(bad.sum()), want[bad][:5], got[bad][:5])


# (rows x columns: the accumulator's rows along Y's rows, along its columns, tokens in the lanes; shared depth)
LAYOUTS = pytest.mark.parametrize("N,K,transposed,M", [(1, 32, False, None), (70, 32, False, None), (5, 32, True, None),
                                                       (100, 32, True, None), (2, 4096, False, 640), (2, 4096, True, 640)])
DTYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])


@DTYPES
@LAYOUTS
def test_silu_in_both_tails(H, dtype, N, K, transposed, M):
    z = arguments()[::1 if M is None else 13][:M]
    own = 2.0 ** -20 if dtype == torch.float32 else 2.0 ** -16
    z64 = z.astype(np.float64)
    check_tails(of_bias(H, z, dtype, H.HINM_ACT_SILU, N, K, transposed), silu64(z64), dtype, own)
    ends = of_bias(H, np.array([np.inf, np.nan], np.float32), dtype, H.HINM_ACT_SILU, N, K, transposed)
    assert ends[0] == np.inf and np.isnan(ends[1])


def gelu64(z):
    """z Phi(z) with Phi's small side as erfc: 1 + erf would have lost it."""
    from math import erfc
    small = np.array([0.5 * erfc(abs(float(v)) * np.sqrt(0.5)) for v in z])
    return z * np.where(z < 0, small, 1 - small)


@DTYPES
@LAYOUTS
def test_gelu_in_both_tails(H, dtype, N, K, transposed, M):
    z = arguments()[::1 if M is None else 13][:M]
    z64 = z.astype(np.float64)
    own = (np.minimum(z64 * z64, 240.0) + 16) * 2.0 ** -23   # (past 15.4 GELU is 0 or z itself)
    check_tails(of_bias(H, z, dtype, H.HINM_ACT_GELU, N, K, transposed), gelu64(z64), dtype, own)
    ends = of_bias(H, np.array([np.inf, np.nan], np.float32), dtype, H.HINM_ACT_GELU, N, K, transposed)
    assert ends[0] == np.inf and np.isnan(ends[1])


# ----------------------------------------------------------------------------- every cut of a product
def spread(n, E):
    """Offsets of E groups in n tokens: the first group empty, the second at most 100, one more empty where
    there are four, the rest uneven, a few tokens behind the last."""
    live = n - min(3, n // 8)
    sizes = np.zeros(E, dtype=np.int64)
    sizes[1] = min(100, max(1, live // 7))
    rest = [e for e in range(2, E) if not (e == 3 and E >= 4)]
    left = live - sizes[1]
    if not rest:
        sizes[1] = live
    for i, e in enumerate(rest):
        sizes[e] = left - (left // 3) if i + 1 < len(rest) and left > 1 else left
        left -= sizes[e]
    return [0] + np.cumsum(sizes).tolist()


def whole(seed, rows, K):
    """0, +-1 .. +-6, which both formats hold whatever the blocks (a 6 in every whole block along either
    dimension, and in the last column): sums of fewer than 2^24 / 36 products are exact in fp32 in any order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.tensor([0, 1, 2, 3, 4, 6, -1, -2, -3, -4, -6], device="cuda")
    x = v[torch.randint(len(v), (rows, K), generator=g, device="cuda")].float()
    r, c = torch.arange(rows, device="cuda")[:, None], torch.arange(K, device="cuda")[None]
    x[((r + c) % 16 == 0) | (c == K - 1)] = 6.0
    return x.bfloat16()


class Product:
    """One product of a kind and its result in 64 bits, from bf16 operands w (of each expert) and x."""

    def __init__(self, H, fmt, kind, M, N, K, E, make):
        self.H, self.kind, self.M, self.N, self.E = H, kind, M, N, E
        scale = "amax" if fmt == F.NV else None
        q = lambda t, **k: H.hinm_fp4_quantize(t, fmt, tensor_scale=scale, **k)  # noqa: E731
        back = lambda m, **k: H.hinm_fp4_dequantize(m, dtype=torch.float32, **k).double()  # noqa: E731
        if kind == "plain":
            self.A, self.B = q(make(1, M, K)), q(make(2, N, K))
            self.parts = [(slice(0, N), back(self.A), back(self.B))]
        elif kind == "rows":
            self.o = spread(N, E)
            w, x = make(1, E * M, K).view(E, M, K), make(2, N, K)
            x[self.o[-1]:] = float("nan")
            self.A = q(w)
            self.B = q(x, ragged=H.HINM_RAGGED_ROWS, offsets=ints(self.o))
            a, b = back(self.A), back(self.B)
            self.parts = [(slice(s, e), a[i], b[s:e]) for i, (s, e) in enumerate(zip(self.o, self.o[1:]))]
        else:
            self.o = spread(K, E)
            d, x = make(1, K, M), make(2, K, N)
            if make is whole:  # a group's last block may be a part of one
                last = [e - 1 for e in self.o[1:] if e > 0]
                d[last], x[last] = 6.0, 6.0
            d[self.o[-1]:], x[self.o[-1]:] = float("nan"), float("nan")
            r = dict(axis=0, ragged=H.HINM_RAGGED_DEPTH, offsets=ints(self.o))
            self.A, self.B = q(d, **r), q(x, **r)
            a, b = back(self.A, axis=0), back(self.B, axis=0)
            self.parts = [(i, a[s:e].t(), b[s:e].t()) for i, (s, e) in enumerate(zip(self.o, self.o[1:]))]

    def run(self, dtype, transposed, bias, act, offset, pad):
        """The outputs of each part as [M][columns], out of a tensor whose other places stay as they were."""
        H, M, N = self.H, self.M, self.N
        shape = (self.E, M, N) if self.kind == "depth" else (N, M) if transposed else (M, N)
        big = torch.full(shape[:-1] + (shape[-1] + offset + pad,), 7.0, dtype=dtype, device="cuda")
        y = big[..., offset:offset + shape[-1]]
        if self.kind == "plain":
            H.hinm_fp4_matmul(self.A, self.B, Y_out=y, transposed=transposed, bias=bias, activation=act)
        elif self.kind == "rows":
            H.hinm_fp4_grouped_matmul(self.A, self.B, Y_out=y, transposed=transposed, bias=bias, activation=act)
        else:
            H.hinm_fp4_grouped_weight_grad(self.A, self.B, Y_out=y)
        assert big[..., :offset].eq(7).all() and big[..., offset + shape[-1]:].eq(7).all()
        if self.kind == "depth":
            return [y[i] for i, _, _ in self.parts]
        yt = y.t() if transposed else y
        if self.kind == "rows":
            assert yt[:, self.o[-1]:].eq(7).all()
        return [yt[:, s] for s, _, _ in self.parts]


def check_sum(y, a, b, bias, act):
    """As the products' bound: K + 3 roundings of sum |a b|, the bias's, the activation's slope (at most 1.13)
    and own error (16 half steps), the store."""
    h = 2.0 ** -24
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    err = (a.shape[1] + 3) * h * mag
    if bias is not None:
        want = want + bias.double()[:, None]
        err = err + h * (mag + bias.abs().double()[:, None])
    z = want
    if act == 2:
        z = want * torch.sigmoid(want)
    if act == 3:
        z = want * 0.5 * torch.special.erfc(-want * 0.5 ** 0.5)
    if act:
        err = 1.13 * err + 16 * h * want.abs() + (2.0 ** -16 * z.abs() if y.dtype != torch.float32 else 0)
    err = err + torch.finfo(y.dtype).eps / 2 * (z.abs() + err)
    bad = ~((y.double() - z).abs() <= err)
    assert not bad.any(), (int(bad.sum()), y.double()[bad][:4], z[bad][:4])


@FORMATS
@pytest.mark.parametrize("kind,transposed,columns,pairs,shared,lanes", fp4_cuts.CUTS, ids=str)
def test_every_cut(H, fmt, kind, transposed, columns, pairs, shared, lanes):
    sizes = fp4_cuts.find(H, kind, transposed, columns, pairs, shared, lanes)
    assert sizes, "no size takes this cut on this device"
    M, N, K, E = sizes
    c = fp4_cuts.cut(H, kind, M, N, K, E, transposed, fmt)
    assert (c[0], c[1], c[2] > 1, c[3]) == (columns, pairs, bool(shared), lanes)
    grad = kind == "depth"
    # whole numbers: bit for bit, and the same again
    p = Product(H, fmt, kind, M, N, K, E, whole)
    first = p.run(torch.float32, transposed, None, 0, 0, 0)
    for y, (_, a, b) in zip(first, p.parts):
        assert torch.equal(y.double(), a @ b.t())
    for y, z in zip(p.run(torch.float32, transposed, None, 0, 0, 0), first):
        assert torch.equal(y, z)
    # any numbers; bias and activation; rows of Y that start on 32 bytes, and anywhere
    p = Product(H, fmt, kind, M, N, K, E, lambda s, *d: rand(s, *d, scale=0.05 if s == 1 else 1.0))
    g = torch.Generator(device="cuda").manual_seed(3)
    bias = None if grad else torch.randn((E, M) if kind == "rows" else (M,), generator=g, device="cuda")
    width = (N if grad or not transposed else M)
    for dtype, act, offset, pad in ((torch.bfloat16, 3, 0, -width % 16), (torch.float32, 2, 3, 2),
                                    (torch.float16, 2, 0, 0), (torch.float32, 3, 0, -width % 8),
                                    (torch.bfloat16, 0, 1, 0)):
        act = 0 if grad else act
        for i, (y, (_, a, b)) in enumerate(zip(p.run(dtype, transposed, bias, act, offset, pad), p.parts)):
            row = bias if bias is None or kind == "plain" else bias[i]
            check_sum(y, a, b, row, act)


@FORMATS
def test_a_scale_that_is_not_a_number_stays_in_its_row_in_every_cut(H, fmt):
    for kind, transposed, columns, pairs, shared, lanes in fp4_cuts.CUTS:
        if kind != "plain":
            continue
        M, N, K, _ = fp4_cuts.find(H, kind, transposed, columns, pairs, shared, lanes)
        w, x = rand(1, M, K), rand(2, N, K)
        w[M // 2, 5], x[N // 3, K - 1] = float("nan"), float("inf")
        y = H.hinm_fp4_matmul(H.hinm_fp4_quantize(w, fmt), H.hinm_fp4_quantize(x, fmt), transposed=transposed)
        y = y.t() if transposed else y
        nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
        nan[M // 2], nan[:, N // 3] = True, True
        assert torch.equal(y.isnan(), nan)


@FORMATS
def test_products_of_pairs_at_once_and_replayed(H, fmt):
    """The pairs' kernel, which takes the whole GPU, on two streams at once, and out of a graph whose operands
    change under it."""
    sizes = [fp4_cuts.find(H, kind, False, 256, 1, 0, False) for kind in ("plain", "rows", "depth")]
    products = [Product(H, fmt, kind, *size, whole) for kind, size in zip(("plain", "rows", "depth"), sizes)]
    want = [[a @ b.t() for _, a, b in p.parts] for p in products]
    streams = [torch.cuda.Stream() for _ in products]
    got = []
    torch.cuda.synchronize()
    for _ in range(3):
        for p, s in zip(products, streams):
            with torch.cuda.stream(s):
                got.append((p, p.run(torch.float32, False, None, 0, 0, 0)))
    torch.cuda.synchronize()
    for p, ys in got:
        for y, z in zip(ys, want[products.index(p)]):
            assert torch.equal(y.double(), z)
    M, N, K, _ = sizes[0]
    x, w = whole(5, N, K), products[0].A
    q = H.hinm_fp4_quantize(x, fmt)
    Y = torch.empty(M, N, device="cuda")
    H.hinm_fp4_quantize(x, fmt, out=q)
    H.hinm_fp4_matmul(w, q, Y_out=Y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H.hinm_fp4_quantize(x, fmt, out=q)
        H.hinm_fp4_matmul(w, q, Y_out=Y)
    for seed in (6, 7):
        x.copy_(whole(seed, N, K))
        Y.zero_()
        g.replay()
        assert torch.equal(Y.double(), products[0].parts[0][1] @ x.double().t())
    del g


@FORMATS
@pytest.mark.parametrize("axis", [1, 0])
def test_batches_of_a_larger_tensor(H, fmt, axis):
    """Matrices and rows a stride apart, on the way in and back."""
    big = torch.full((7, 90, 150), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = big[1::2, 5:85:2, 8:136]        # every other matrix and row
    view.copy_(rand(3, 3, 40, 128))
    scale = "amax" if fmt == F.NV else None
    a = H.hinm_fp4_quantize(view, fmt, axis=axis, tensor_scale=scale)
    b = H.hinm_fp4_quantize(view.contiguous(), fmt, axis=axis, tensor_scale=scale)
    want = H.hinm_fp4_dequantize(b, axis=axis)
    out = torch.full_like(big, 5.0)
    H.hinm_fp4_dequantize(a, axis=axis, out=out[1::2, 5:85:2, 8:136])
    assert torch.equal(out[1::2, 5:85:2, 8:136], want)
    out[1::2, 5:85:2, 8:136] = 5.0
    assert out.eq(5).all()


# ----------------------------------------------------------------------------- waits
def test_a_product_that_lasts_longer_than_a_wait_may(H):
    """Waits inside the kernels are limited to 2 s each.  A product of 1.9e16 operations takes longer than that
    (2.1 s at the tensor cores' nominal rate), by tiles of 10 ms: right, and no wait ran out.  Every code is 1
    with the scale 1, so that every output is the depth."""
    M, K = 61440, 2_500_096
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 100 GB")
    A = H.Fp4Matrix.allocate(F.MX, 1, M, K, "cuda")
    A.values.fill_(0x22)
    A.scales.fill_(127)
    Y = torch.empty(M, M, device="cuda")
    assert H.hinm_device_status() == 0
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    H.hinm_fp4_matmul(A, A, Y_out=Y)
    end.record()
    torch.cuda.synchronize()
    assert H.hinm_device_status() == 0
    assert start.elapsed_time(end) > 2000
    assert float(Y.min()) == K and float(Y.max()) == K
    del A, Y
    torch.cuda.empty_cache()
