"""Tree attention on scores and values at the ends of their ranges, against oracle/tree.py.

Tolerances as in test_gpu_tree.py, but for a softcap c: c tanh(s / c) is worked out to 2^-20 of itself (its quotient and
product, tanh or the fit: 2^-24 and two or three steps of 2^-24 each), whatever c is, which adds 2^-20 of the largest
|score| to what a score may be off. Where every score is exact, equal ones are the only ones with weight and a score is
off by nothing."""

import numpy as np
import pytest

from grouped_query_attention_gb300 import GroupQueryAttention
from oracle import tree as ot
from test_gpu_tree import CASES, check, make, operator, run_gpu, run_oracle, tolerance

pytestmark = pytest.mark.gpu

FORMS = {   # as test_gpu_tree.CASES: the tensor-core pipeline with one and two row tiles a piece, the warp MMAs
    "one_tile": CASES["tile_32"],
    "two_tiles": ("f16", 1, 40, 8, 2, 64, 900, (877,), None, -1, 0, 0, 0, "tree", 0),
    "split": ("f16", 1, 11, 4, 2, 128, 3000, (2990,), None, -1, 0, 0, 0, "tree", 0),
    "mma_h256": CASES["h256"], "mma_f32": CASES["tile_32_f32"], "mma_h256_f32": CASES["h256_f32"],
}


def capped_check(d, softcap):
    d["softcap"] = softcap
    out, mag, reach, rk, rv = run_oracle(d)
    d["softcap"] = float(2.0 * min(softcap, reach.max()))   # tolerance(): 2^-21 of it
    got = run_gpu(d, operator(dict(d, softcap=softcap)))
    assert got[3].block_status() == 0
    check(d, got, (out, mag, reach, rk, rv))


@pytest.mark.parametrize("name", list(FORMS))
@pytest.mark.parametrize("softcap", [1e4, 5e5, 1e6, 3e7, 1e8, 1e10, 1e30])
def test_softcaps_far_above_the_scores(name, softcap):
    """c tanh(s / c) is s."""
    capped_check(make(FORMS[name], seed=3), softcap)


@pytest.mark.parametrize("name", list(FORMS))
@pytest.mark.parametrize("softcap", [1e-3, 1e-10, 1e-38, 1e-45])
def test_softcaps_far_below_the_scores(name, softcap):
    """Every score is c, -c or (of a zero product) 0: all visible rows weigh the same."""
    d = make(FORMS[name], seed=3)
    d["k"][:, 0] = 0
    capped_check(d, softcap)


@pytest.mark.parametrize("name", list(FORMS))
@pytest.mark.parametrize("softcap", [1e38, 2.4e38, 3.4e38])
def test_the_largest_softcaps(name, softcap):
    """c log2(e) is no float any more."""
    capped_check(make(FORMS[name], seed=3), softcap)


def exact_scores(d, scale, softcap=0.0):
    """Queries and keys of whole numbers times a power of two: equal scores are equal in every bit, unequal ones are worlds
    apart, and the output is the mean of the values of the largest."""
    d["softcap"] = 0.0
    d["q"], d["pk"], d["k"] = (np.sign(np.nan_to_num(d[x])).astype(d[x].dtype) for x in ("q", "pk", "k"))
    d["q"][..., 1::2] = 0
    pk, pv = d["pk"].copy(), d["pv"].copy()
    out, mag, reach = ot.forward(d["q"], d["k"], d["v"], d["parents"], d["totals"] - 1, d["news"], pk, pv, d["N"], d["Nkv"],
                                 scale=scale, softcap=softcap, window=d["window"])
    op = GroupQueryAttention(d["N"], d["Nkv"], scale=scale, softcap=softcap, local_window_size=d["window"])
    got = run_gpu(d, op)
    assert op.block_status() == 0
    check(d, got, (out, mag, 0 * reach, pk, pv))


MMA = [x for x in FORMS if x.startswith("mma")]


@pytest.mark.parametrize("power", [17, 20, 22, 23, 24, 25, 27, 31, 40, 60])
@pytest.mark.parametrize("name,sign", [(x, 1) for x in MMA] + [(x, -1) for x in FORMS])
def test_scores_of_any_size_on_warp_mmas(name, sign, power):
    """(Negative scales take every call there.)"""
    exact_scores(make(FORMS[name], seed=5), sign * 2.0 ** power)


@pytest.mark.parametrize("power", [17, 19, 20, 22, 23, 24, 25, 27, 31, 40, 60])
@pytest.mark.parametrize("name", ["one_tile", "two_tiles", "split", "h64_window"])
def test_scores_of_any_size(name, power):
    """(... of the tensor-core pipeline.)"""
    case = ("f16", 2, 20, 4, 2, 64, 500, (490, 333), None, 100, 0, 0, 0, "tree", 0) if name == "h64_window" else FORMS[name]
    exact_scores(make(case, seed=5), 2.0 ** power)


@pytest.mark.parametrize("name", list(FORMS))
@pytest.mark.parametrize("softcap", [3e7, 1e9, 1e12])
def test_scores_as_large_as_a_large_softcap(name, softcap):
    """Scores up to about 4 c, where floats are 2 to 2^16 apart."""
    exact_scores(make(FORMS[name], seed=4), 2.0 ** round(np.log2(softcap / 16)), softcap)


# ------------------------------------------------------------------ values that are not finite

SPLIT = {"split_f32": ("f32", 1, 5, 4, 2, 64, 5000, (4999,), None, -1, 0, 0, 0, "tree", 0)}


def spoiled_check(d, where, op=None, scale=0.0):
    """where: [(tensor, index)] set to +inf. Elements that see one are not finite, all others as without it."""
    clean = dict(d, pv=d["pv"].copy(), v=d["v"].copy())
    for name, at in where:
        clean[name][at] = 1.0
    for x in ("pv", "v"):
        d[x] = clean[x].copy()
    for name, at in where:
        d[name][at] = np.inf

    def forward(x):
        return ot.forward(x["q"], x["k"], x["v"], x["parents"], x["totals"] - 1, x["news"], x["pk"].copy(), x["pv"].copy(),
                          x["N"], x["Nkv"], scale=scale, softcap=x["softcap"], window=x["window"], sink=x["sink"],
                          smooth=bool(x["smooth"]))

    with np.errstate(invalid="ignore"):
        spoiled = ~np.isfinite(forward(d)[0])
    ref, mag, reach = forward(clean)
    assert spoiled.any() and not spoiled.all()
    got = run_gpu(d, op or operator(d, scale=scale))[0].astype(np.float64)
    assert not np.isfinite(got[spoiled]).any(), (~spoiled & ~np.isfinite(got)).sum()
    bad = ~spoiled & ~(np.abs(got - ref) <= tolerance(clean, ref, mag, reach))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist())


@pytest.mark.parametrize("name", ["split", "split_f32", "mma_h256", "one_tile", "two_tiles", "mma_f32"])
def test_infinite_values_of_a_split_range(name):
    """A cached value in the middle: the heads that read it are spoiled in its coordinate, in whichever worker's piece
    it lies."""
    d = make({**CASES, **FORMS, **SPLIT}[name], seed=8)
    spoiled_check(d, [("pv", (0, 0, int(d["totals"][0]) // 2, 7))])


@pytest.mark.parametrize("name", ["split", "split_f32", "mma_h256", "one_tile", "two_tiles", "mma_f32", "forest", "forest_window_f32"])
@pytest.mark.parametrize("what", ["cached", "node"])
def test_infinite_values_of_no_weight(name, what):
    """The same beside a key of such a score that the weight of every other one is far below the smallest float: an
    infinite value times that is infinite still."""
    d = make({**CASES, **FORMS, **SPLIT}[name], seed=9)
    last = int(d["totals"][0]) - d["S"] - 1
    d["q"][:] = np.where(np.isnan(d["q"]), d["q"], 1)
    d["k"][:], d["pk"][:] = np.where(np.isnan(d["k"]), d["k"], 0), np.where(np.isnan(d["pk"]), d["pk"], 0)
    d["pk"][0, 0, last] = 1                               # score H scale, the others 0
    scale = 400.0 / d["H"]
    row = last // 2 if d["window"] < 0 else last - 1
    spoiled_check(d, [("pv", (0, 0, row, 7)) if what == "cached" else ("v", (0, 2, 9))], scale=scale)


WINDOWED = {   # fp16: one, two row tiles a piece, many pieces; warp MMAs: fp16 heads of 256, fp32
    "one_tile": ("f16", 2, 24, 4, 2, 64, 900, (900, 700), None, 300, 0, 0, 0, "chain", 0),
    "two_tiles": ("f16", 2, 70, 8, 2, 128, 900, (900, 700), (70, 33), 300, 5.0, 1, 0, "chain", 0),
    "all_nodes": ("f16", 1, 512, 2, 1, 64, 2000, (1990,), None, 600, 0, 0, 0, "chain", 0),
    "pieces": ("f16", 2, 40, 16, 4, 96, 3000, (3000, 2700), None, 1250, 0, 0, 0, "tree", 0),
    "h256": ("f16", 1, 20, 4, 2, 256, 500, (490,), None, 200, 0, 0, 1, "chain", 0),
    "f32": ("f32", 2, 20, 4, 2, 128, 500, (490, 333), None, 100, 0, 1, 0, "tree", 0),
    "f32_pieces": ("f32", 1, 33, 8, 2, 64, 6000, (5999,), None, 3000, 0, 0, 0, "chain", 0),
}


@pytest.mark.parametrize("name", WINDOWED)
@pytest.mark.parametrize("behind", [0, 1, 3, 9, "last"])
def test_cached_values_at_a_windows_edge(name, behind):
    """A cached value that nodes of a depth up to `behind` see (the root sees furthest back): they are spoiled, in that
    coordinate, and nobody else. One head of one sequence."""
    d = make(WINDOWED[name], seed=6)
    b = d["B"] - 1
    n = d["S"] if d["news"] is None else int(d["news"][b])
    depth = max(len(ot.ancestors(d["parents"], b, i)) - 1 for i in range(n))
    off = min(depth, 1 << 20 if behind == "last" else behind)
    row = int(d["totals"][b]) - n - d["window"] + off
    spoiled_check(d, [("pv", (b, d["Nkv"] - 1, row, 5)), ("pv", (b, 0, max(0, row - 1), d["H"] - 1))])


@pytest.mark.parametrize("name", WINDOWED)
def test_nan_keys_at_a_windows_edge(name):
    """A cached key of NaN: rows that see it are NaN, the others as they were."""
    d = make(WINDOWED[name], seed=7)
    b = d["B"] - 1
    n = d["S"] if d["news"] is None else int(d["news"][b])
    row = int(d["totals"][b]) - n - d["window"] + 2
    ref, mag, reach, _, _ = run_oracle(d)
    tol = tolerance(d, ref, mag, reach)
    d["pk"][b, 0, row, 3] = np.nan
    got = run_gpu(d)[0].astype(np.float64).reshape(d["B"], d["S"], d["N"], d["H"])
    ref, tol = ref.reshape(got.shape), tol.reshape(got.shape)
    G, seen = d["N"] // d["Nkv"], 0
    for i in range(n):
        sees = len(ot.ancestors(d["parents"], b, i)) - 1 <= 2
        seen += sees
        if sees:
            assert np.isnan(got[b, i, :G]).all()
        else:
            assert (np.abs(got - ref) <= tol)[b, i].all()
        assert (np.abs(got - ref) <= tol)[b, i, G:].all()
    assert 0 < seen < n
