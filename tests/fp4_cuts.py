"""The smallest of a set of odd sizes for which the library takes a given cut of a 4-bit product.

The cut is the library's own answer (hinm_selftest_fp4_cut), so that the tests reach every kernel whatever
its choice rests on; when no size takes a cut any more, the search says so.
"""
import itertools

MS = (65, 130, 257, 333, 700, 1001, 1500, 2003, 2500, 3003, 4001, 5001)
NS = (1, 3, 20, 64, 100, 201, 333, 420, 701, 1001, 1500, 2003, 3003, 4001)
KS = (64, 300, 1000, 2050, 4000, 8050, 16300)
GROUPS = {"plain": (1,), "rows": (4, 16), "depth": (2, 4)}  # kinds of product and their numbers of experts

# kind, transposed, columns of a tile, pairs, shared depth, tokens in the lanes
CUTS = ([(kind, False, c, p, s, False) for kind in GROUPS
         for c, p, s in ((64, 0, 0), (64, 0, 1), (128, 0, 0), (128, 0, 1), (192, 0, 0), (256, 1, 0))]
        + [(kind, True, c, p, s, True) for kind in ("plain", "rows")
           for c, p, s in ((64, 0, 0), (64, 0, 1), (128, 0, 0), (128, 0, 1), (192, 0, 0), (256, 1, 0))]
        + [(kind, True, 64, 0, s, False) for kind in ("plain", "rows") for s in (0, 1)]
        + [("rows", True, 128, 0, 0, False), ("rows", True, 128, 0, 1, False)])


def _matrix(H, fmt, batch, rows, depth, ragged, groups):
    class Offsets:  # only counted
        @staticmethod
        def numel():
            return groups + 1
    return H.Fp4Matrix(format=fmt, batch=batch, rows=rows, depth=depth, values=None, scales=None, ragged=ragged,
                       offsets=Offsets if ragged else None)


def cut(H, kind, M, N, K, E, transposed, fmt=0):
    """(columns, pairs, CTAs a depth, tokens in the lanes) of a product of M x K by K x N; E experts."""
    if kind == "plain":
        a, b = (1, 0, 0), (1, 0, 0)
    elif kind == "rows":
        a, b = (E, 0, 0), (1, H.HINM_RAGGED_ROWS, E)
    else:
        a = b = (1, H.HINM_RAGGED_DEPTH, E)
    A = _matrix(H, fmt, a[0], M, K, *a[1:])
    B = _matrix(H, fmt, b[0], N, K, *b[1:])
    return H.hinm_selftest_fp4_cut(A, B, transposed)


def find(H, kind, transposed, columns, pairs, shared, lanes):
    """(M, N, K, experts), the fewest operations."""
    sizes = sorted(itertools.product(MS, NS, KS, GROUPS[kind]), key=lambda s: s[0] * s[1] * s[2])
    for M, N, K, E in sizes:
        if kind != "plain" and (N < 20 or kind == "depth" and K < 300):
            continue  # (tokens for uneven groups)
        c = cut(H, kind, M, N, K, E, transposed)
        if c[0] == columns and c[1] == pairs and (c[2] > 1) == bool(shared) and c[3] == lanes:
            return M, N, K, E
    return None
