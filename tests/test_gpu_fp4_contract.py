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
