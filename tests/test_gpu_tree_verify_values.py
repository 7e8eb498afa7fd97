"""Verification of drafted tokens where the numbers are hard. Paths and tokens are equal to those of the 64-bit
definition (oracle/tree.py); where a border is placed on purpose, it stands further from the numbers that meet it than
the 64-bit sums round (math.fsum and one product: 2^-52)."""

import math

import numpy as np
import pytest
import torch

from grouped_query_attention_gb300 import GroupQueryAttention, capi
from oracle import tree as ot
from test_gpu_tree import NP, dev, make_verify, run_verify, same

pytestmark = pytest.mark.gpu


def star(tokens, rows, draft, u, us, dtype=np.float32):
    """A root with children of these tokens; the root's rows (B, V) or (V,), every other node's uniform."""
    tokens = np.atleast_2d(np.asarray(tokens, np.int32))
    B, S = tokens.shape[0], tokens.shape[1] + 1

    def spread(row):
        row = np.broadcast_to(np.asarray(row, np.float64), (B, np.asarray(row).shape[-1]))
        x = np.full((B, S, row.shape[-1]), 1.0 / row.shape[-1])
        x[:, 0] = row
        return x.astype(dtype)

    return dict(tokens=np.concatenate([np.zeros((B, 1), np.int32), tokens], 1),
                parents=np.array([[-1] + [0] * (S - 1)], np.int32), target_probs=spread(rows),
                draft_probs=None if draft is None else spread(draft),
                accept_uniforms=np.broadcast_to(np.float32(u), (B, S)).copy(),
                sample_uniforms=np.broadcast_to(np.float32(us), (B,)).copy(), new_lens=None)


# ------------------------------------------------------------------ many drafts turned down

@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("V", [3000, 40001])
@pytest.mark.parametrize("qt,refused", [(0.99, 2), (0.99, 9), (0.9, 16), (0.6, 45), (0.97, 300)])
def test_a_certain_target_behind_many_refusals(qt, refused, V, dtype):
    """The target is certain of one token, the draft almost: what is left is that token after every refusal, and its
    child, the last one, passes. Without that child it is drawn."""
    t, rng = V // 3, np.random.default_rng(9)
    p, q = np.zeros(V), rng.random(V)
    q[t] = 0.0
    q *= (1.0 - qt) / q.sum()
    p[t], q[t] = 1.0, qt
    others = rng.choice(np.delete(np.arange(V), t), refused, replace=V < refused)
    for children, nodes, token in ((list(others) + [t], 2, None), (others, 1, t)):
        v = star(children, p, q, 0.5, 0.25, NP[dtype])
        got = run_verify(v)
        same(got, ot.verify(**v))
        assert got[1].tolist() == [nodes] and (token is None or got[2].tolist() == [token])


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("noise", [0.5, 0.05, 0.005])
def test_close_drafts_turned_down_by_force(noise, drafts):
    """Uniforms near 1 turn down drafts of rows that hardly differ: remainders of 0.2 to 0.002 of the rows, one behind
    the other."""
    for seed in range(4):
        v = make_verify(4, 12, 2003, drafts=drafts, kind="star", noise=noise, std=2.0, seed=seed)
        v["accept_uniforms"][:] = 1.0 - 2.0 ** -24 if seed % 2 else 1.0
        same(run_verify(v), ot.verify(**v))


def test_refusals_on_the_way_down():
    """Nodes of a path that turn several close drafts down before one passes, then the next node anew."""
    rng = np.random.default_rng(12)
    for seed in range(6):
        v = make_verify(3, 60, 1009, kind="tree", noise=0.02, std=2.0, seed=seed)
        v["accept_uniforms"][:] = np.where(rng.random((3, 60)) < 0.7, 1.0, rng.random((3, 60)))
        same(run_verify(v), ot.verify(**v))


# ------------------------------------------------------------------ next to nothing

TINY = 2.0 ** -149


def test_draws_from_rows_of_the_smallest_floats():
    """Rows of a few smallest floats: the place u sum is between two of their multiples."""
    row = np.zeros(700)
    row[[5, 300, 301, 699]] = np.array([3, 5, 7, 1]) * TINY
    us = np.array([0.1, 0.19, 0.2, 0.21, 0.5, 0.53, 0.5333, 0.54, 0.9, 0.93, 0.935, 0.96], np.float32)
    for draft in (None, np.full(700, 1.0 / 700)):
        v = star(np.full((12, 1), 7), row, draft, 1.0, us)
        if draft is not None:
            v["new_lens"] = np.full(12, 1, np.int32)     # the draw alone: round 0
        want = ot.verify(**v)
        assert set(want[2].tolist()) == {5, 300, 301, 699}
        same(run_verify(v), want)


def test_tests_of_the_smallest_floats():
    """u q(x) < r(x) where both are a few smallest floats."""
    u = np.linspace(0.05, 0.95, 19, dtype=np.float32)
    for pu, qu in ((1, 1), (1, 2), (2, 3), (5, 7), (1, 3)):
        p, q = np.full(600, 1.0 / 600), np.full(600, 1.0 / 600)
        p[17], q[17] = pu * TINY, qu * TINY
        v = star(np.full((19, 1), 17), p, q, 0.0, 0.5)
        v["accept_uniforms"][:, 1] = u
        want = ot.verify(**v)
        assert (want[1] == 2).tolist() == [float(x) * qu < pu for x in u]
        same(run_verify(v), want)


@pytest.mark.parametrize("tiny", [1e-38, 1e-41, 2.0 ** -149, 1e-30, 1e-20])
def test_remainders_of_almost_nothing(tiny):
    """Target and draft agree but for tokens of almost no probability: what a refusal leaves is those."""
    V = 5000
    p, q = np.zeros(V), np.zeros(V)
    p[100] = q[100] = 1.0
    p[[7, 2000, 4999]] = np.array([2.0, 5.0, 3.0]) * tiny
    q[[7, 3000]] = np.array([1.0, 4.0]) * tiny
    for children in ([3000], [3000, 100], [3000, 100, 7, 2000], [3000, 3000, 3000, 4999], [3000, 4999, 2000, 7, 100]):
        for u in (0.05, 0.3, 0.7, 1.0):
            us = np.array([0.05, 0.15, 0.5, 0.8], np.float32)
            v = star(np.tile(children, (4, 1)), p, q, u, us)
            same(run_verify(v), ot.verify(**v))


# ------------------------------------------------------------------ the last bits

def bordered(rest, least, most, rng, below):
    """A uniform u and a float x: u (sum(rest) + x) lies a relative distance in [least, most] below x, or above it."""
    base = math.fsum(rest)
    while True:
        u = np.float32(rng.uniform(0.2, 0.8))
        x = np.float32(float(u) * base / (1.0 - float(u)))   # u (base + x) = x, but for its rounding
        for c in (x, np.nextafter(x, np.float32(np.inf)), np.nextafter(x, np.float32(0))):
            edge = float(u) * (base + float(c))
            if least <= (float(c) - edge) / edge * (1 if below else -1) <= most:
                return u, c


def test_sums_of_certain_drafts_keep_their_bits():
    """A first token of almost everything is turned down; the sum of the rest, 2^-15 of the row, meets a token's
    probability at 2^-38 to 2^-36 of it."""
    rng = np.random.default_rng(21)
    B, V = 64, 900
    v = star(np.tile([0, 1], (B, 1)), np.zeros((B, V)), None, 1.0, 0.5)
    for b in range(B):
        rest = (rng.random(V - 2) * 2.0 ** -25).astype(np.float32)
        u, x = bordered(rest.astype(np.float64), 2.0 ** -38, 2.0 ** -36, rng, b % 2)
        v["target_probs"][b, 0, 1], v["target_probs"][b, 0, 2:] = x, rest
        v["target_probs"][b, 0, 0] = 1.0 - 2.0 ** -15
        v["accept_uniforms"][b, 2] = u
    want = ot.verify(**v)
    assert want[1].tolist() == [1, 2] * (B // 2)
    same(run_verify(v), want)


def test_sums_of_large_vocabularies_keep_their_bits():
    """A CTA a sequence (153 of them, 149 empty) and 2^20 tokens: 512 numbers a chain of the sum, two of about 1 and then
    510 of 2^-26 and a bit that a float sum of them near 2^-17 cannot hold (each loses 2^-42, all the same way: 2^-35 of
    the whole). The sum meets a token's probability at 2^-38 to 2^-36 of it."""
    rng = np.random.default_rng(22)
    B, V, live = 153, 1 << 20, 8
    rows = np.full((live, 3, V), 2.0 ** -26 * (1 + 0.49 * 2.0 ** -15), np.float32)
    u = np.ones((B, 3), np.float32)
    for b in range(live):
        rest = rows[b, 0].reshape(16, -1)              # a warp's run
        rest[:, :256] = 0.75 + 0.25 * rng.random((16, 256))
        rows[b, 0, [0, V - 1]] = 0.0                   # token 0 is turned down first, so that the sum counts
        u[b, 2], rows[b, 0, V - 1] = bordered(rows[b, 0].astype(np.float64), 2.0 ** -38, 2.0 ** -36, rng, b % 2)
    p = torch.zeros((B, 3, V), device="cuda")
    p[:live] = dev(rows)
    tokens, par = np.tile(np.array([[0, 0, V - 1]], np.int32), (B, 1)), np.array([[-1, 0, 0]], np.int32)
    us, news = np.full(B, 0.001, np.float32), np.where(np.arange(B) < live, 3, 0).astype(np.int32)
    got = GroupQueryAttention(1, 1).tree_verify(dev(tokens), dev(par), p, dev(u), dev(us), new_lens=dev(news))
    want = ot.verify(tokens[:live], par, rows, u[:live], us[:live])
    assert want[1].tolist() == [1, 2] * (live // 2)
    same([x[:live].cpu().numpy() for x in got], want)


# ------------------------------------------------------------------ numbers that are no probabilities

@pytest.mark.parametrize("drafts", [True, False])
def test_numbers_too_large_for_a_probability(drafts):
    """Numbers from 2^40 on count as none, whatever their sum; below it they count. A row without another is reported."""
    rng = np.random.default_rng(31)
    p = rng.random((6, 3000)) / 3000
    p[:4, [3, 200, 1700, 2999]] = np.array([[2e38], [3e11], [2.0 ** 40], [1e30]])
    p[4] = 0.0
    p[4, [3, 200]] = 2e38
    q = np.full(3000, 1.0 / 3000)
    q[[3, 77]] = 3e38
    q[1000] = 1e11
    v = star(np.tile([3, 77, 1000, 2999], (6, 1)), p, q if drafts else None, 1.0, [0.05, 0.1, 0.5, 0.7, 0.7, 0.9])
    op = GroupQueryAttention(1, 1)
    got = run_verify(v, op)
    same(got, ot.verify(**v))
    assert got[2].min() == got[2][4] == -1 and op.block_status() == capi.GQA_DEVICE_BAD_PROBS


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("size", [1e-6, 1.0, 1e3, 1e6, 1e10])
def test_rows_that_are_not_normalised(size, drafts):
    """Rows whose sums are far from 1: the tests are those of the definition, the draw takes a share of what is left."""
    for seed in range(3):
        v = make_verify(5, 14, 700, drafts=drafts, kind="star", seed=seed, std=1.0)
        v["target_probs"] = (v["target_probs"] * np.float32(size * 30)).astype(np.float32)
        if drafts:
            v["draft_probs"] = (v["draft_probs"] * np.float32(size * (1 + 40 * seed))).astype(np.float32)
        same(run_verify(v), ot.verify(**v))
