"""The 4-bit binding without a GPU: CPU tensors stand for device ones, and the C calls either refuse
(before any launch) or are replaced by ones that only note what they are given."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture()
def H(monkeypatch):
    from conftest import build_library
    build_library()
    import pruning_hinm_spmm_b200 as H
    # CPU tensors are on "device" -1
    monkeypatch.setattr(H, "_current", lambda t, name, stream=None: (-1, 0))
    return H


class Noted:
    """The C library with some of the 4-bit calls replaced: they note the matrix's pointers."""

    def __init__(self, real, *names):
        self.real, self.names, self.calls = real, names, []

    def __getattr__(self, name):
        if name not in self.names:
            return getattr(self.real, name)

        def call(src, dtype, ld, bs, axis, bits, q, stream):
            self.calls.append((name, q._obj.tensor_scale, q._obj.offsets))
            return 0
        return call


def fields(q):
    return {k: v for k, v in vars(q).items() if not k.startswith("_")}


BF16 = torch.bfloat16
CASES = {  # what only the C checks refuse: source, further arguments
    "a bitmask with ragged rows": lambda H: (torch.zeros(64, 256, dtype=BF16), dict(
        ragged=H.HINM_RAGGED_ROWS, offsets=torch.tensor([0, 20, 64], dtype=torch.int32),
        bitmask=torch.zeros(64 * 8, dtype=torch.int32))),
    "rows without a stride": lambda H: (torch.zeros(1, 256, dtype=BF16).expand(64, 256), {}),
    "rows that overlap": lambda H: (torch.zeros(64 * 256, dtype=BF16).as_strided((64, 256), (100, 1)), {}),
    "values out of place": lambda H: (torch.zeros(64, 256, dtype=BF16), {}),
}


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("scale", ["amax", "given", None])
@pytest.mark.parametrize("case", list(CASES))
def test_a_call_that_c_refuses_leaves_the_matrix_as_it_was(H, monkeypatch, case, scale, given):
    x, kw = CASES[case](H)
    ragged = kw.get("ragged", H.HINM_RAGGED_NONE)
    off = torch.tensor([0, 30, 64], dtype=torch.int32) if ragged else None
    q = H.Fp4Matrix.allocate(H.HINM_FP4_NV, 1, 64, 256, "cpu", ragged, off)
    if given:
        q.tensor_scale, q.given_scale = torch.full((1,), 0.5), True
    noted = Noted(H._lib)
    if case == "values out of place":  # the scale's own call does not look at them: it must not run
        noted = Noted(H._lib, "hinm_fp4_tensor_scale")
        q.values = torch.zeros(q.values.numel() + 24, dtype=torch.uint8)[8:]
    monkeypatch.setattr(H, "_lib", noted)
    q.scales.fill_(7)
    was, before = fields(q), q.tensor_scale.clone()
    with pytest.raises((H.HinmError, ValueError)):
        H.hinm_fp4_quantize(x, H.HINM_FP4_NV, out=q, tensor_scale=torch.ones(1) if scale == "given" else scale, **kw)
    now = fields(q)
    assert now.keys() == was.keys() and all(now[k] is was[k] for k in was)
    assert torch.equal(q.tensor_scale, before) and q.scales.eq(7).all() and not noted.calls


def test_an_accepted_call_takes_the_new_offsets_and_scale(H, monkeypatch):
    noted = Noted(H._lib, "hinm_fp4_tensor_scale", "hinm_fp4_quantize")
    monkeypatch.setattr(H, "_lib", noted)
    off, off2 = (torch.tensor([0, n, 64], dtype=torch.int32) for n in (20, 30))
    g, x = torch.full((1,), 0.25), torch.zeros(64, 256, dtype=BF16)
    rag = dict(ragged=H.HINM_RAGGED_ROWS)
    q = H.hinm_fp4_quantize(x, H.HINM_FP4_NV, offsets=off, tensor_scale="amax", **rag)
    mine = q.tensor_scale
    r = H.hinm_fp4_quantize(x, H.HINM_FP4_NV, offsets=off2, tensor_scale=g, out=q, **rag)
    assert r is q and q.offsets is off2 and q.tensor_scale is g
    H.hinm_fp4_quantize(x, H.HINM_FP4_NV, offsets=off2, out=q, **rag)
    assert q.tensor_scale is None
    at = [t.data_ptr() for t in (mine, off, g, off2)]
    assert noted.calls == [("hinm_fp4_tensor_scale", at[0], at[1]), ("hinm_fp4_quantize", at[0], at[1]),
                           ("hinm_fp4_quantize", at[2], at[3]), ("hinm_fp4_quantize", None, at[3])]


def test_amax_never_writes_into_a_scale_that_the_caller_gave(H, monkeypatch):
    """However the matrix came by it: "amax" takes a tensor of its own, once, and leaves the caller's."""
    import copy
    import dataclasses
    import pickle
    noted = Noted(H._lib, "hinm_fp4_tensor_scale", "hinm_fp4_quantize")
    monkeypatch.setattr(H, "_lib", noted)
    x = torch.zeros(64, 256, dtype=BF16)
    amax = lambda q: H.hinm_fp4_quantize(x, H.HINM_FP4_NV, tensor_scale="amax", out=q)  # noqa: E731
    g = torch.full((1,), 0.5)
    built = H.Fp4Matrix.allocate(H.HINM_FP4_NV, 1, 64, 256, "cpu", tensor_scale=False)
    ways = {
        "constructor": H.Fp4Matrix(format=H.HINM_FP4_NV, batch=1, rows=64, depth=256, values=built.values,
                                   scales=built.scales, tensor_scale=g),
        "assigned": H.Fp4Matrix.allocate(H.HINM_FP4_NV, 1, 64, 256, "cpu"),
        "assigned to amax's": amax(H.Fp4Matrix.allocate(H.HINM_FP4_NV, 1, 64, 256, "cpu")),
        "quantised with": H.hinm_fp4_quantize(x, H.HINM_FP4_NV, tensor_scale=g),
    }
    ways["assigned"].tensor_scale = g
    ways["assigned to amax's"].tensor_scale = g
    first = amax(H.Fp4Matrix.allocate(H.HINM_FP4_NV, 1, 64, 256, "cpu"))
    theirs = first.tensor_scale          # the scale of another matrix, taken over by its copies
    copies = {"replace": dataclasses.replace(first, values=first.values.clone()), "copy": copy.copy(first)}
    for name, q in {**ways, **copies}.items():
        kept = g if name in ways else theirs
        assert q.tensor_scale is kept, name
        amax(q)
        made = q.tensor_scale
        assert made is not kept and not q.given_scale, name
        assert noted.calls[-2:] == [(f, made.data_ptr(), None) for f in
                                    ("hinm_fp4_tensor_scale", "hinm_fp4_quantize")], name
        amax(q)
        assert q.tensor_scale is made, name  # its own is written again, where it is
    for q in (copy.deepcopy(first), pickle.loads(pickle.dumps(first))):
        amax(q)
        assert q.tensor_scale is not theirs
    own = H.Fp4Matrix.allocate(H.HINM_FP4_NV, 1, 64, 256, "cpu")
    ones = own.tensor_scale
    assert amax(own).tensor_scale is ones    # (allocate's ones are the matrix's own)
