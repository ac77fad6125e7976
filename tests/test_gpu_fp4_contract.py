"""What the header promises of the 4-bit calls beyond their values: what is reported, how exact the
activations are in the tails, and every cut of a product, whichever sizes the library takes it for."""
import numpy as np
import pytest

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
