"""GPU tests of the drafted-token operators against the fp64 definitions of oracle/tree.py.

Tolerances, derived from the roundings (u = 2^-24, the half step of fp32):
  caches, moved rows, paths, lengths, tokens: equal.
  output: its own rounding, half a step of its type, and what the sums carry. A score is a sum of H products in fp32
    (at most (H + 20) 2 u of max|q| sum|k| scale with its factors; the parts of fp32 operands lose 2^-20 of a product
    more), and an error d of the scores changes a probability by 2 d at most; a softcap's tanh adds 2^-21 of the cap to
    d. exp2, its argument and the fp32 sums 2^-19. Each fp16 probability enters the product with V rounded (2^-11; its
    sum is of the same rounded ones, so it weighs |v - out|), and one below 2^-29 of the largest is off by 2^-40
    of it; fp32 products lose 2^-20. All of these weigh sum_j p_j |v_j|, the first also |out|.
"""

import numpy as np
import pytest
import torch

from grouped_query_attention_gb300 import GroupQueryAttention, GqaError, capi
from oracle import tree as ot

pytestmark = pytest.mark.gpu

NP = {"f16": np.float16, "f32": np.float32}


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def random_tree(rng, S, kind):
    if kind == "chain":
        return np.arange(-1, S - 1)
    if kind == "star":
        return np.array([-1] + [0] * (S - 1))
    par = np.array([-1] + [int(rng.integers(0, i)) for i in range(1, S)])
    if kind == "forest":
        par[rng.random(S) < 0.2] = -1
    return par


CASES = {
    # name: dtype, B, S, N, Nkv, H, C, totals, news (None: S), window, softcap, sink, smooth, kind, one tree
    "root": ("f16", 3, 1, 8, 2, 128, 200, (1, 64, 197), None, -1, 0, 0, 0, "chain", 0),
    "root_f32": ("f32", 3, 1, 8, 2, 128, 200, (1, 65, 200), None, -1, 0, 0, 0, "chain", 1),
    "h16": ("f16", 2, 2, 3, 3, 16, 50, (2, 50), None, -1, 0, 0, 0, "chain", 0),
    "h16_f32": ("f32", 2, 2, 3, 3, 16, 50, (2, 50), None, -1, 0, 0, 0, "chain", 0),
    "h48_g3": ("f16", 2, 9, 6, 2, 48, 70, (33, 70), None, -1, 0, 0, 0, "tree", 0),
    "h80_f32_ragged": ("f32", 2, 7, 10, 2, 80, 90, (40, 90), (7, 2), -1, 0, 1, 0, "tree", 0),
    "h96_ragged": ("f16", 4, 5, 6, 2, 96, 300, (300, 5, 77, 0), (5, 5, 1, 0), -1, 0, 0, 0, "tree", 0),
    "h192": ("f16", 2, 20, 4, 2, 192, 100, (100, 37), None, -1, 0, 0, 0, "star", 0),
    "h256_f32": ("f32", 2, 17, 4, 1, 256, 140, (140, 17), None, -1, 0, 0, 0, "tree", 0),
    "h256": ("f16", 1, 33, 8, 2, 256, 400, (391,), None, -1, 0, 0, 0, "tree", 0),
    "h256_window_f32": ("f32", 1, 6, 4, 2, 256, 400, (391,), None, 70, 0, 0, 1, "tree", 0),
    "g12": ("f16", 2, 3, 12, 1, 64, 100, (100, 17), None, -1, 0, 1, 0, "tree", 0),
    "g7_f32": ("f32", 1, 9, 7, 1, 96, 200, (123,), None, 64, 0, 0, 0, "tree", 0),
    "tile_16": ("f16", 2, 4, 8, 2, 128, 500, (500, 333), None, -1, 0, 0, 0, "tree", 0),
    "tile_32": ("f16", 2, 8, 8, 2, 128, 500, (500, 333), None, -1, 0, 0, 0, "tree", 0),
    "tile_64": ("f16", 2, 16, 8, 2, 128, 500, (500, 333), None, -1, 0, 0, 0, "tree", 0),
    "tile_16_f32": ("f32", 2, 4, 8, 2, 128, 500, (500, 333), None, -1, 0, 0, 0, "tree", 0),
    "tile_32_f32": ("f32", 2, 8, 8, 2, 128, 500, (500, 333), None, -1, 0, 0, 0, "tree", 0),
    "tile_64_f32": ("f32", 2, 16, 8, 2, 128, 500, (500, 333), None, -1, 0, 0, 0, "tree", 0),
    "tiles_3": ("f16", 2, 37, 8, 2, 64, 300, (300, 37), None, -1, 0, 0, 0, "tree", 1),
    "tiles_5_f32": ("f32", 1, 75, 8, 2, 64, 300, (222,), None, -1, 0, 0, 0, "tree", 0),
    "window": ("f16", 3, 12, 8, 2, 64, 400, (400, 150, 12), None, 100, 0, 0, 0, "tree", 0),
    "window_0_f32": ("f32", 2, 5, 4, 2, 64, 100, (100, 33), None, 0, 0, 0, 0, "tree", 0),
    "window_2": ("f16", 2, 30, 4, 2, 64, 100, (100, 33), None, 2, 0, 0, 0, "chain", 0),
    "softcap_sink": ("f16", 2, 6, 8, 2, 128, 300, (300, 130), None, -1, 5.0, 1, 0, "tree", 0),
    "softcap_f32": ("f32", 2, 7, 8, 4, 64, 100, (100, 50), None, 40, 5.0, 1, 0, "tree", 0),
    "smooth": ("f16", 2, 6, 8, 2, 128, 300, (300, 6), None, -1, 0, 0, 1, "tree", 0),
    "long_split": ("f16", 2, 11, 4, 2, 128, 9000, (9000, 5001), None, -1, 0, 0, 0, "tree", 0),
    "long_split_f32": ("f32", 1, 5, 2, 1, 64, 20000, (19999,), None, -1, 0, 0, 0, "tree", 0),
    "long_rows": ("f16", 1, 100, 8, 1, 128, 3000, (2999,), None, -1, 0, 0, 0, "tree", 0),
    "forest": ("f16", 2, 40, 4, 2, 64, 200, (200, 44), None, -1, 0, 0, 0, "forest", 0),
    "forest_window_f32": ("f32", 2, 40, 4, 2, 64, 200, (200, 44), None, 5, 0, 0, 0, "forest", 0),
    "many_nodes": ("f16", 1, 512, 4, 2, 128, 700, (650,), None, -1, 0, 0, 0, "tree", 0),
    "many_nodes_ragged": ("f16", 2, 300, 4, 2, 64, 700, (650, 120), (299, 120), -1, 0, 0, 0, "chain", 1),
    "empty_slots": ("f16", 4, 2, 4, 2, 64, 64, (0, 10, 0, 64), (0, 0, 0, 2), -1, 0, 0, 0, "chain", 1),
    "no_cached_rows": ("f16", 2, 64, 8, 2, 128, 64, (64, 30), (64, 30), -1, 0, 0, 0, "tree", 0),
    "group_of_40": ("f16", 1, 7, 40, 1, 128, 300, (300,), None, -1, 0, 0, 0, "tree", 0),
    "many_units": ("f16", 4, 16, 16, 4, 128, 6000, (6000, 5500, 4100, 5999), None, -1, 0, 0, 0, "tree", 0),
    "many_units_two_tiles": ("f16", 4, 40, 16, 4, 128, 6000, (6000, 5500, 4100, 5999), (40, 13, 40, 33), -1, 0, 0, 0, "tree", 0),
    "many_units_h64": ("f16", 3, 12, 20, 4, 64, 12000, (12000, 9000, 11111), None, -1, 8.0, 1, 0, "tree", 0),
    "many_units_window": ("f16", 4, 50, 16, 4, 96, 6000, (6000, 5500, 4100, 5999), None, 2500, 20.0, 0, 0, "chain", 0),
    "many_pieces": ("f16", 150, 10, 16, 4, 128, 40, tuple(10 + 31 * i % 31 for i in range(150)), None, -1, 0, 0, 0, "tree", 0),
    "many_pieces_two_tiles": ("f16", 150, 10, 64, 4, 64, 140, tuple(10 + 37 * i % 131 for i in range(150)), None, -1, 0, 0, 0, "tree", 0),
    "many_sequences": ("f16", 150, 3, 4, 2, 64, 40, tuple(3 + 37 * i % 38 for i in range(150)), None, -1, 0, 0, 0, "tree", 0),
}


def make(case, seed=0):
    dtype, B, S, N, Nkv, H, C, totals, news, window, softcap, sink, smooth, kind, one = case
    rng = np.random.default_rng(seed)
    t = NP[dtype]
    d = dict(dtype=dtype, B=B, S=S, N=N, Nkv=Nkv, H=H, C=C, window=window, softcap=softcap, smooth=smooth,
             totals=np.array(totals, np.int32), news=None if news is None else np.array(news, np.int32))
    d["parents"] = np.stack([random_tree(rng, S, kind) for _ in range(1 if one else B)]).astype(np.int32)
    d["q"] = (2 * rng.standard_normal((B, S, N * H))).astype(t)
    d["k"], d["v"] = (rng.standard_normal((B, S, Nkv * H)).astype(t) for _ in range(2))
    d["pk"], d["pv"] = (rng.standard_normal((B, Nkv, C, H)).astype(t) for _ in range(2))
    d["sink"] = rng.standard_normal(N).astype(t) if sink else None
    for b in range(B):   # what does not count holds anything
        n = S if news is None else news[b]
        for x in ("q", "k", "v"):
            d[x][b, n:] = np.nan
        for x in ("pk", "pv"):
            d[x][b, :, totals[b] - n:] = np.nan
        if not one:
            d["parents"][b, n:] = 1 << 30
    return d


def run_oracle(d):
    pk, pv = d["pk"].copy(), d["pv"].copy()
    out, mag, reach = ot.forward(d["q"], d["k"], d["v"], d["parents"], d["totals"] - 1, d["news"], pk, pv, d["N"], d["Nkv"],
                                 softcap=d["softcap"], window=d["window"], sink=d["sink"], smooth=bool(d["smooth"]))
    return out, mag, reach, pk, pv


def operator(d, **attrs):
    return GroupQueryAttention(d["N"], d["Nkv"], softcap=float(d["softcap"]), local_window_size=d["window"],
                               smooth_softmax=1 if d["smooth"] else -1, **attrs)


def run_gpu(d, op=None, total=None, output=None):
    op = op or operator(d)
    pk, pv = dev(d["pk"]), dev(d["pv"])
    out = op.tree_forward(dev(d["q"]), dev(d["k"]), dev(d["v"]), dev(d["parents"]), dev(d["totals"] - 1),
                          max(1, int(d["totals"].max())) if total is None else total, pk, pv, new_lens=dev(d["news"]),
                          head_sink=dev(d["sink"]), output=output)
    torch.cuda.synchronize()
    return out.cpu().numpy(), pk.cpu().numpy(), pv.cpu().numpy(), op


def tolerance(d, out, mag, reach):
    f16, H = d["dtype"] == "f16", d["H"]
    s = ((H + 20) * 2.0 ** -23 + (0 if f16 else 2.0 ** -20)) * reach + d["softcap"] * 2.0 ** -21
    s = np.repeat(s, H, axis=-1).reshape(out.shape)
    p = 2.0 ** -11 if f16 else 2.0 ** -20
    half = 2.0 ** -11 if f16 else 2.0 ** -24
    most = np.nanmax(np.abs(np.concatenate([d["pv"].astype(np.float64).ravel(), d["v"].astype(np.float64).ravel()])))
    tiny = max(1, int(d["totals"].max())) * most * 2.0 ** -40 if f16 else 0.0
    return half * np.abs(out) + (p * (1 + half) + 2 * s + 2.0 ** -19) * mag + (p if f16 else 0) * np.abs(out) + tiny + 2.0 ** -25


def check(d, got, want=None):
    out, pk, pv = got[:3]
    ref, mag, reach, rk, rv = want or run_oracle(d)
    assert np.array_equal(pk, rk, equal_nan=True) and np.array_equal(pv, rv, equal_nan=True)
    bad = ~(np.abs(out.astype(np.float64) - ref) <= tolerance(d, ref, mag, reach))
    assert not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[:3].tolist(), np.nanmax(np.abs(out - ref)))


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    d = make(CASES[name])
    got = run_gpu(d)
    check(d, got)
    assert got[3].block_status() == 0


@pytest.mark.parametrize("name", ["tile_16", "tile_64_f32", "long_split", "h96_ragged", "window", "many_nodes_ragged"])
def test_forward_with_a_loose_bound_is_the_same_on_every_run(name):
    d = make(CASES[name], seed=1)
    want = run_oracle(d)
    op = operator(d)
    first = run_gpu(d, op, total=d["C"])
    check(d, first, want)
    again = run_gpu(d, op, total=d["C"])
    assert np.array_equal(first[0], again[0])


@pytest.mark.parametrize("name", ["tile_16", "tile_32", "tile_64", "tiles_3", "h96_ragged", "window", "forest", "softcap_sink",
                                  "many_units_h64", "tile_32_f32"])
@pytest.mark.parametrize("scale", [-0.1, 0.3])
def test_forward_of_other_scales(name, scale):
    """A negative scale takes fp16 calls to the warp MMAs."""
    d = make(CASES[name])
    pk, pv = d["pk"].copy(), d["pv"].copy()
    out, mag, reach = ot.forward(d["q"], d["k"], d["v"], d["parents"], d["totals"] - 1, d["news"], pk, pv, d["N"], d["Nkv"],
                                 scale=scale, softcap=d["softcap"], window=d["window"], sink=d["sink"], smooth=bool(d["smooth"]))
    check(d, run_gpu(d, operator(d, scale=scale)), (out, mag, reach, pk, pv))


def test_bad_lengths_leave_everything():
    d = make(CASES["tile_16"])
    op = operator(d)
    for totals, news in (([501, 333], None), ([3, 333], None), ([-1, 333], None), ([500, 333], [5, 4]), ([500, 333], [-1, 4]),
                         ([-2 ** 31, 333], [0, 4])):
        e = dict(d, totals=np.array([500, 333], np.int32))
        want = run_oracle(e)
        x = dict(d, totals=np.array(totals, np.int64).astype(np.int32), news=None if news is None else np.array(news, np.int32))
        if totals[0] == -2 ** 31:   # seqlens_k = 2^31 - 1: one more wraps
            assert int((x["totals"] - 1)[0]) == 2 ** 31 - 1
        out = torch.full((2, 4, 8 * 128), 7.0, dtype=torch.float16, device="cuda")
        got = run_gpu(x, op, total=500, output=out)
        assert op.block_status() == capi.GQA_DEVICE_BAD_SEQLEN
        assert (got[0][0] == 7).all() and np.array_equal(got[1][0], d["pk"][0], equal_nan=True)
        assert np.array_equal(got[1][1], want[3][1], equal_nan=True)
        tol = tolerance(e, *want[:3])[1]
        assert (np.abs(got[0][1] - want[0][1]) <= tol).all()


def test_bad_parents_are_roots_and_reported():
    d = make(CASES["tile_64"])
    d["parents"][0, 5], d["parents"][1, 3], d["parents"][1, 0] = 5, -7, 0
    got = run_gpu(d)
    check(d, got)
    assert got[3].block_status() == capi.GQA_DEVICE_BAD_TREE


def test_infinite_and_nan_values_reach_only_who_sees_them():
    """A node with NaN rows spoils itself and its descendants, nobody else."""
    for name in ("tile_64", "tile_64_f32"):
        d = make(CASES[name])
        d["k"][0, 7], d["v"][1, 4] = np.nan, np.inf
        got = run_gpu(d)
        finite = dict(d, k=np.nan_to_num(d["k"]), v=np.nan_to_num(d["v"], posinf=1.0))
        ref, mag, reach, _, _ = run_oracle(finite)
        tol = tolerance(finite, ref, mag, reach)
        for b, node in ((0, 7), (1, 4)):
            for i in range(16):
                spoiled = node in ot.ancestors(d["parents"], b, i)
                row = got[0][b, i].astype(np.float64)
                assert (~np.isfinite(row)).all() if spoiled else (np.abs(row - ref[b, i]) <= tol[b, i]).all()


@pytest.mark.parametrize("name", ["tile_64", "tile_64_f32", "h256", "window"])
def test_a_nan_score_is_not_lost(name):
    """The root's key is NaN: every node sees it, the root (whose other keys are in other units) too."""
    d = make(CASES[name])
    d["k"][:, 0] = np.nan
    assert np.isnan(run_gpu(d)[0]).all()


@pytest.mark.parametrize("seed", range(24))
def test_forward_random(seed):
    """Sizes, masks and types drawn over the range of a call."""
    rng = np.random.default_rng([seed, 17])
    H = int(rng.choice([16, 64, 80, 96, 128, 128, 256]))
    Nkv, B = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 3, 5]))
    N, S = Nkv * int(rng.choice([1, 2, 3, 4, 7, 8])), int(rng.choice([1, 2, 5, 11, 33, 70, 130]))
    C = S + int(rng.choice([0, 1, 40, 127, 128, 300, 900]))
    news = tuple(int(x) for x in rng.integers(0, S + 1, B)) if rng.random() < 0.5 else None
    totals = tuple(int(rng.integers(S if news is None else news[b], C + 1)) for b in range(B))
    case = (str(rng.choice(["f16", "f16", "f32"])), B, S, N, Nkv, H, C, totals, news, int(rng.choice([-1, -1, 0, 3, 60, C])),
            float(rng.choice([0, 0, 2.0, 30.0])), int(rng.integers(0, 2)), int(rng.integers(0, 2)),
            str(rng.choice(["tree", "chain", "star", "forest"])), int(rng.integers(0, 2)))
    d = make(case, seed)
    got = run_gpu(d, total=C if rng.random() < 0.5 else None)
    check(d, got)
    assert got[3].block_status() == 0


@pytest.mark.parametrize("dtype,H,rows", [("f16", 128, 17_500_000), ("f32", 128, 9_000_000)])
def test_rows_behind_two_gigabytes(dtype, H, rows):
    """Offsets of a cache past 2^31 elements (fp16) and 2^32 bytes (fp32): a window at its end, and the move of its rows."""
    rng = np.random.default_rng(8)
    S, N, W = 6, 4, 200
    t = NP[dtype]
    tail = [rng.standard_normal((1, 1, 400, H)).astype(t) for _ in range(2)]
    q, k, v = (rng.standard_normal((1, S, n * H)).astype(t) for n in (N, 1, 1))
    par = np.array([[-1, 0, 0, 1, 3, 2]], np.int32)
    op = GroupQueryAttention(N, 1, local_window_size=W)
    big = [torch.empty((1, 1, rows, H), dtype=getattr(torch, "float16" if dtype == "f16" else "float32"), device="cuda") for _ in range(2)]
    for b, x in zip(big, tail):
        b[:, :, rows - 400:] = dev(x)
    out = op.tree_forward(dev(q), dev(k), dev(v), dev(par), dev(np.array([rows - 1], np.int32)), rows, *big)
    d = dict(dtype=dtype, H=H, softcap=0, totals=np.array([400]), v=v, pv=tail[1])
    want, mag, reach = ot.forward(q, k, v, par, np.array([399]), None, *tail, N, 1, window=W)
    assert (np.abs(out.cpu().numpy() - want) <= tolerance(d, want, mag, reach)).all()
    path, lens = np.array([[0, 1, 3, 4, -1, -1]], np.int32), np.array([4], np.int32)
    got = op.tree_accept([tuple(big)], dev(path), dev(lens), dev(np.array([rows - 1], np.int32)))
    ot.accept(tail, path, lens, np.array([399]))
    assert got.tolist() == [rows - S + 3] and op.block_status() == 0
    for b, x in zip(big, tail):
        assert np.array_equal(b[:, :, rows - 400:].cpu().numpy(), x)


def test_a_second_stream_and_a_graph():
    d = make(CASES["tile_32"])
    want = run_oracle(d)
    op = operator(d)
    args = [dev(d[x]) for x in ("q", "k", "v", "parents")] + [dev(d["totals"] - 1), 500]
    pk, pv, out = dev(d["pk"]), dev(d["pv"]), torch.empty((2, 8, 8 * 128), dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        op.tree_forward(*args, pk, pv, output=out)
    side.synchronize()
    check(d, (out.cpu().numpy(), pk.cpu().numpy(), pv.cpu().numpy()), want)
    graphs = []
    for _ in range(2):   # two graphs of one operator, replayed side by side
        o, k2, v2 = torch.zeros_like(out), dev(d["pk"]), dev(d["pv"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            op.tree_forward(*args, k2, v2, output=o)
        graphs.append((g, o, k2, v2, torch.cuda.Stream()))
    for _ in range(3):
        for g, *_, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, o, k2, v2, _ in graphs:
        check(d, (o.cpu().numpy(), k2.cpu().numpy(), v2.cpu().numpy()), want)


@pytest.mark.parametrize("name,tile", [("tile_64", 0), ("long_rows", 0), ("many_units", 3), ("many_units_two_tiles", 2)])
def test_expired_waits_are_reported_and_leave_the_next_call_alone(name, tile):
    """The copy of a key tile is withheld: the waits for it run out, the call says so, the next one is right."""
    d = make(CASES[name])
    op = operator(d)
    capi.gqa_set_wait_limit(op.handle, 2_000_000, tile)
    run_gpu(d, op)
    assert op.block_status() == capi.GQA_DEVICE_TIMEOUT
    capi.gqa_set_wait_limit(op.handle, 0)
    check(d, run_gpu(d, op))
    assert op.block_status() == 0


def test_python_refusals():
    d = make(CASES["tile_16"])
    op = operator(d)
    q, k, v, par, seq, pk, pv = (dev(x) for x in (d["q"], d["k"], d["v"], d["parents"], d["totals"] - 1, d["pk"], d["pv"]))
    with pytest.raises(ValueError, match="contiguous"):
        op.tree_forward(q, k, v, par, seq, 500, pk.transpose(1, 2).contiguous().transpose(1, 2), pv)
    with pytest.raises(GqaError):
        op.tree_forward(q, k, v, par.long().float(), seq, 500, pk, pv)
    with pytest.raises(GqaError):
        op.tree_forward(q, k, v, par, seq, 501, pk, pv)
    with pytest.raises(ValueError):
        op.tree_forward(q, k, v, par, seq, 2 ** 31, pk, pv)
    with pytest.raises(GqaError):
        op.tree_forward(q, k, v, par, seq, 500, pk, pk)


# ------------------------------------------------------------------ verification

def peaked(rng, shape, std=3.0):
    x = np.exp(std * rng.standard_normal(shape))
    return x / x.sum(-1, keepdims=True)


def make_verify(B, S, V, drafts=True, kind="tree", news=None, dtype=np.float32, seed=0, std=3.0, noise=0.5):
    rng = np.random.default_rng(seed)
    logits = std * rng.standard_normal((B, S, V))
    p = np.exp(logits)
    q = np.exp(logits + noise * rng.standard_normal((B, S, V)))
    p, q = (p / p.sum(-1, keepdims=True)).astype(dtype), (q / q.sum(-1, keepdims=True)).astype(dtype)
    par = np.stack([random_tree(rng, S, kind) for _ in range(B)]).astype(np.int32)
    tok = np.zeros((B, S), np.int32)
    for b in range(B):
        for i in range(S):
            a = max(0, par[b, i])
            if drafts:
                row = q[b, a].astype(np.float64)
                tok[b, i] = rng.choice(V, p=row / row.sum())
            else:
                rank = int((par[b, 1:i] == par[b, i]).sum())
                tok[b, i] = np.argsort(-q[b, a].astype(np.float64), kind="stable")[min(rank, V - 1)]
    return dict(tokens=tok, parents=par, target_probs=p, accept_uniforms=rng.random((B, S)).astype(np.float32),
                sample_uniforms=rng.random(B).astype(np.float32), draft_probs=q if drafts else None,
                new_lens=None if news is None else np.array(news, np.int32))


def run_verify(v, op=None, **kw):
    op = op or GroupQueryAttention(1, 1)
    got = op.tree_verify(*(dev(v[x]) for x in ("tokens", "parents", "target_probs", "accept_uniforms", "sample_uniforms")),
                         draft_probs=dev(v["draft_probs"]), new_lens=dev(v["new_lens"]), **kw)
    return [x.cpu().numpy() for x in got]


def same(got, want):
    for a, b in zip(got, want):
        assert np.array_equal(a, b), (a, b)


VERIFY = {
    "one": dict(B=1, S=1, V=1), "root_only": dict(B=3, S=1, V=1000), "chain": dict(B=5, S=6, V=32768, kind="chain"),
    "chain_odd": dict(B=3, S=4, V=32769, kind="chain"), "small": dict(B=7, S=9, V=17), "two_words": dict(B=9, S=5, V=2),
    "tree": dict(B=4, S=40, V=5003), "tree_large": dict(B=2, S=12, V=100003), "star": dict(B=16, S=30, V=301, kind="star"),
    "far_drafts": dict(B=8, S=30, V=1001, kind="star", noise=4.0), "flat": dict(B=8, S=10, V=40001, std=0.1),
    "certain": dict(B=4, S=33, V=4099, drafts=False), "certain_star": dict(B=16, S=30, V=50, drafts=False, kind="star"),
    "certain_large": dict(B=2, S=8, V=131072, drafts=False), "half": dict(B=4, S=10, V=20002, dtype=np.float16),
    "half_odd": dict(B=4, S=10, V=4097, dtype=np.float16), "half_certain": dict(B=4, S=10, V=9001, dtype=np.float16, drafts=False),
    "ragged": dict(B=6, S=7, V=6000, news=(7, 0, 1, 3, 7, 2)), "forest": dict(B=6, S=20, V=300, kind="forest"),
    "many_nodes": dict(B=2, S=512, V=100, kind="tree"), "many_chain": dict(B=2, S=512, V=100, kind="chain", noise=0.01),
    "many_star": dict(B=2, S=512, V=100, kind="star", drafts=False),
}


@pytest.mark.parametrize("name", VERIFY)
def test_verify(name):
    for seed in range(3):
        v = make_verify(**VERIFY[name], seed=seed)
        op = GroupQueryAttention(1, 1)
        same(run_verify(v, op), ot.verify(**v))
        assert op.block_status() == 0


@pytest.mark.parametrize("drafts", [True, False])
def test_verify_vocabulary_past_a_warps_mask(drafts):
    """More than 2^20 tokens: a warp's run has more turns than the 64 bits that mark those with a token turned down."""
    for seed in range(2):
        v = make_verify(2, 6, 1100003, drafts=drafts, kind="star", seed=seed)
        v["accept_uniforms"][:, 1:] = 1.0 - 2.0 ** -24   # (turns most drafts down)
        if not drafts:
            v["tokens"][:, 1:3] = [[0, 1100002], [524287, 7]]
        same(run_verify(v), ot.verify(**v))


def test_verify_rows_behind_two_billion_elements():
    """A chain of certain rows (every draft passes), the last of which lies behind 2^31 elements: it holds two tokens."""
    S, V = 512, 4200003
    tokens = torch.from_numpy(np.random.default_rng(8).integers(0, V, (1, S)).astype(np.int32)).cuda()
    p = torch.zeros((1, S, V), dtype=torch.float16, device="cuda")
    p[0, torch.arange(S - 1), tokens[0, 1:].long()] = 1.0
    p[0, S - 1, 7], p[0, S - 1, V - 1] = 0.25, 0.75
    op = GroupQueryAttention(1, 1)
    for draft in (None, p):
        for u, want in ((0.125, 7), (0.5, V - 1)):
            path, lens, token = op.tree_verify(tokens, dev(np.arange(-1, S - 1, dtype=np.int32)[None]), p,
                                               torch.full((1, S), 0.75, device="cuda"), torch.full((1,), u, device="cuda"),
                                               draft_probs=draft)
            assert torch.equal(path[0].cpu(), torch.arange(S, dtype=torch.int32)) and (int(lens), int(token)) == (S, want)
    assert op.block_status() == 0


def test_verify_takes_one_tree_for_all():
    v = make_verify(4, 9, 500, kind="star")
    v["parents"] = v["parents"][:1]
    same(run_verify(v), ot.verify(**v))


@pytest.mark.parametrize("drafts", [True, False])
def test_verify_extreme_numbers(drafts):
    """Uniforms at the ends of their range, and outside it: 0 accepts what is possible, 1 - 2^-24 and 1 draw the last
    token, NaN turns every draft down."""
    for u in (0.0, 1.0 - 2.0 ** -24, 1.0, np.nan):
        v = make_verify(4, 8, 3001, drafts=drafts, std=1.0)
        v["accept_uniforms"][:] = u
        v["sample_uniforms"][:] = u
        same(run_verify(v), ot.verify(**v))


@pytest.mark.parametrize("drafts", [True, False])
def test_verify_improper_probabilities(drafts):
    """Negative, infinite and NaN probabilities count as none; tokens outside the vocabulary are turned down; a row
    without a positive probability is reported."""
    v = make_verify(5, 6, 600, drafts=drafts, kind="star")
    rng = np.random.default_rng(5)
    for x in (v["target_probs"], v["draft_probs"]):
        if x is not None:
            x[rng.random(x.shape) < 0.1] = np.nan
            x[rng.random(x.shape) < 0.1] = np.inf
            x[rng.random(x.shape) < 0.1] = -0.5
    v["tokens"][0, 1:3], v["tokens"][1, 2] = -1, 600
    v["target_probs"][3] = np.nan
    op = GroupQueryAttention(1, 1)
    got = run_verify(v, op)
    same(got, ot.verify(**v))
    assert got[2][3] == -1 and op.block_status() == capi.GQA_DEVICE_BAD_PROBS


def test_verify_equal_rows_leave_nothing():
    """Where draft and target agree every draft passes; a number of 1 turns it down and nothing is left to draw from,
    which takes the target's own row."""
    v = make_verify(3, 5, 2000, kind="star")
    v["draft_probs"] = v["target_probs"].copy()
    same(run_verify(v), ot.verify(**v))
    v["accept_uniforms"][:] = 1.0
    got = run_verify(v)
    same(got, ot.verify(**v))
    assert (got[1] == 1).all() and (got[2] >= 0).all()


def test_verify_reports_bad_trees_and_lengths():
    v = make_verify(4, 6, 100, news=(6, 7, -1, 6))
    v["parents"][0, 3], v["parents"][3, 0] = 3, 0
    op = GroupQueryAttention(1, 1)
    got = run_verify(v, op)
    same(got, ot.verify(**v))
    assert (got[0][1:3] == -1).all() and op.block_status() == capi.GQA_DEVICE_BAD_TREE | capi.GQA_DEVICE_BAD_SEQLEN


def test_verify_in_a_graph_draws_anew():
    v = make_verify(6, 8, 5000)
    op = GroupQueryAttention(1, 1)
    run_verify(v, op)
    t = {k: dev(x) for k, x in v.items() if x is not None}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = op.tree_verify(**t)
    for seed in range(3):
        w = make_verify(6, 8, 5000, seed=seed)
        for k in t:
            t[k].copy_(dev(w[k]))
        g.replay()
        same([x.cpu().numpy() for x in got], ot.verify(**w))


# ------------------------------------------------------------------ accepted rows

@pytest.mark.parametrize("dtype,L,B,S,Nkv,H,C", [("f16", 1, 1, 8, 8, 128, 64), ("f32", 3, 4, 17, 3, 80, 50),
                                                 ("f16", 128, 2, 5, 1, 16, 9), ("f16", 2, 3, 512, 2, 64, 600),
                                                 ("f32", 2, 2, 33, 2, 256, 33)])
def test_accept(dtype, L, B, S, Nkv, H, C):
    rng = np.random.default_rng(3)
    caches = [rng.standard_normal((B, Nkv, C, H)).astype(NP[dtype]) for _ in range(2 * L)]
    path, lens, totals, news = np.full((B, S), -1, np.int32), np.zeros(B, np.int32), [], []
    for b in range(B):
        n = int(rng.integers(1, S + 1))
        k = int(rng.integers(0, n + 1))
        path[b, :k] = np.sort(rng.choice(n, k, replace=False))
        lens[b] = k
        news.append(n)
        totals.append(n + int(rng.integers(0, C - n + 1)))
    seq, news = np.array(totals, np.int32) - 1, np.array(news, np.int32)
    op = GroupQueryAttention(Nkv, Nkv)
    t = [dev(c) for c in caches]
    got = op.tree_accept(list(zip(t[::2], t[1::2])), dev(path), dev(lens), dev(seq), new_lens=dev(news))
    want = ot.accept(caches, path, lens, seq, news)
    assert np.array_equal(got.cpu().numpy(), want) and op.block_status() == 0
    for a, c in zip(t, caches):
        assert np.array_equal(a.cpu().numpy(), c)


def test_accept_skips_bad_paths_and_lengths():
    C, S = 20, 4
    path = np.array([[0, 2, 1, -1], [0, 0, 1, 2], [0, 4, -1, -1], [-1, 0, -1, -1], [0, 1, 2, 3], [0, 1, 2, 3], [1, 3, -1, -1]], np.int32)
    lens = np.array([3, 2, 2, 2, 5, 2, 2], np.int32)
    seq = np.array([10, 10, 10, 10, 10, 20, 10], np.int32)
    rng = np.random.default_rng(4)
    caches = [rng.standard_normal((7, 2, C, 32)).astype(np.float32) for _ in range(2)]
    t = [dev(c) for c in caches]
    op = GroupQueryAttention(2, 2)
    got = op.tree_accept([tuple(t)], dev(path), dev(lens), dev(seq))
    want = ot.accept(caches, path, lens, seq)
    assert got.cpu().tolist() == want.tolist() == [-1] * 6 + [8]
    assert op.block_status() == capi.GQA_DEVICE_BAD_TREE | capi.GQA_DEVICE_BAD_SEQLEN
    for a, c in zip(t, caches):
        assert np.array_equal(a.cpu().numpy(), c)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_drafting_loop(dtype):
    """Three rounds of drafting over two layers: rotated nodes, tree attention, verification of the drafts, the accepted
    rows moved together. What is left in the caches is what storing the accepted tokens one by one gives, and a plain
    step of the framework on it agrees with the oracle."""
    rng = np.random.default_rng(6)
    B, S, N, Nkv, H, C, V, layers = 3, 9, 8, 2, 64, 128, 500, 2
    t = NP[dtype]
    op = GroupQueryAttention(N, Nkv)
    angles = np.arange(C)[:, None] * 1e4 ** (-np.arange(32) / 32)
    cos, sin = np.cos(angles).astype(np.float32), np.sin(angles).astype(np.float32)
    seq = np.array([20, 5, 40], np.int32)
    ref = [rng.standard_normal((B, Nkv, C, H)).astype(t) for _ in range(2 * layers)]
    gpu = [dev(c) for c in ref]
    caches = list(zip(gpu[::2], gpu[1::2]))
    kept = [[[np.array(c[b, :, i]) for i in range(seq[b] + 1)] for b in range(B)] for c in ref]   # rows, one by one
    lens_k = dev(seq)
    for step in range(3):
        v = make_verify(B, S, V, seed=step)
        par = v["parents"]
        depth = np.array([[len(ot.ancestors(par, b, i)) - 1 for i in range(S)] for b in range(B)])
        seq_in = lens_k.cpu().numpy() + S                       # the nodes' rows are live during the step
        pos = (lens_k.cpu().numpy()[:, None] + 1 + depth).astype(np.int32)
        stored = []
        for layer in range(layers):
            q, k, val = (rng.standard_normal((B, S, n * H)).astype(t) for n in (N, Nkv, Nkv))
            gq, gk = op.rotary_axes(dev(q), dev(k), dev(pos[None]), dev(cos), dev(sin), [32])
            out = op.tree_forward(gq, gk, dev(val), dev(par), dev(seq_in), int(seq_in.max()) + 1, *caches[layer])
            d = dict(dtype=dtype, H=H, softcap=0, totals=seq_in + 1, v=val, pv=ref[2 * layer + 1])
            want, mag, reach = ot.forward(gq.cpu().numpy(), gk.cpu().numpy(), val, par, seq_in, None, ref[2 * layer],
                                          ref[2 * layer + 1], N, Nkv)
            assert (np.abs(out.cpu().numpy() - want) <= tolerance(d, want, mag, reach)).all()
            stored += [gk.cpu().numpy(), val]
        path, plens, token = op.tree_verify(*(dev(v[x]) for x in ("tokens", "parents", "target_probs", "accept_uniforms",
                                                                  "sample_uniforms")), draft_probs=dev(v["draft_probs"]))
        lens_k = op.tree_accept(caches, path, plens, dev(seq_in))
        rp, rl, rt = ot.verify(**v)
        same([x.cpu().numpy() for x in (path, plens, token)], (rp, rl, rt))
        ot.accept(ref, rp, rl, seq_in)
        for c, x in zip(kept, stored):
            for b in range(B):
                c[b] += [x[b, i].reshape(Nkv, H) for i in rp[b, :rl[b]]]
    total = lens_k.cpu().numpy() + 1
    for a, c, rows in zip(gpu, ref, kept):
        assert np.array_equal(a.cpu().numpy(), c)
        for b in range(B):
            assert len(rows[b]) == total[b] and np.array_equal(a[b, :, :total[b]].cpu().numpy(), np.stack(rows[b], 1))
    # a plain decode step goes on from there
    q, k, val = (rng.standard_normal((B, 1, n * H)).astype(t) for n in (N, Nkv, Nkv))
    out = op(dev(q), dev(k), dev(val), lens_k + 1, int(total.max()) + 1, *caches[0], past_key=caches[0][0], past_value=caches[0][1])
    d = dict(dtype=dtype, H=H, softcap=0, totals=total + 1, v=val, pv=ref[1])
    want, mag, reach = ot.forward(q, k, val, np.array([[-1]]), total, None, ref[0], ref[1], N, Nkv)
    atol, rtol = (2e-3, 1e-2) if dtype == "f16" else (1e-4, 1e-4)   # the framework's own for this entry
    assert (np.abs(out.cpu().numpy() - want) <= atol + rtol * np.abs(want)).all()
    assert op.block_status() == 0
