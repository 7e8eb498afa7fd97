"""Cases of the multi-axis rotary embedding, of attention over the block-scaled int8 cache (with the row's
attention weights where asked) and of the eviction from that cache.

A case is one pass through one of them, as a serving loop calls it:

rotary  q, k of a batch of tokens -> (optional RMS norm) -> rotated at positions of several axes.
step    S new rows per sequence are quantised into the cache, then their queries attend to it; with `weights`
        the attention weight every cache row received is added to its running sum.
evict   a full cache is reduced to the `keep` rows per KV head with the largest running sums (the first and the
        most recent rows are always kept), and the newest token attends to what is left.

The int8 codes themselves are not among the outputs: every code of the cache enters the attention output that is
returned with the block scales.
"""

import math

import torch

own = False

DT = {"f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases

def _rotary(name, dtype, B, S, N, Nkv, H, sections, interleaved=False, norm=False, R=32768):
    return dict(name=name, op="rotary", dtype=dtype, B=B, S=S, N=N, Nkv=Nkv, H=H, sections=sections,
                interleaved=interleaved, norm=norm, R=R)


def _step(name, dtype, B, S, N, Nkv, H, C, bs, lo, hi, ragged=False, window=-1, softcap=0.0, sink=False,
          weights=False):
    return dict(name=name, op="step", dtype=dtype, B=B, S=S, N=N, Nkv=Nkv, H=H, C=C, bs=bs, lo=lo, hi=hi,
                ragged=ragged, window=window, softcap=softcap, sink=sink, weights=weights)


def _evict(name, dtype, B, N, Nkv, H, C, bs, lo, hi, keep, recent, first):
    return dict(name=name, op="evict", dtype=dtype, B=B, N=N, Nkv=Nkv, H=H, C=C, bs=bs, lo=lo, hi=hi, keep=keep,
                recent=recent, first=first)


def listed():
    return [
        # one token for each of 16 sequences: the smallest call of a decode step
        _rotary("rotary_decode_f16", "f16", 16, 1, 32, 8, 128, "16,24,24"),
        # a batch of prompts with q/k norms, the attention shape of the fp16 prefill workload
        _rotary("rotary_prompt_norm_f16", "f16", 4, 4096, 32, 8, 128, "16,24,24", norm=True),
        # fp32 image-patch tokens, interleaved axes, part of an odd-sized head rotated
        _rotary("rotary_partial_f32", "f32", 3, 1025, 12, 4, 96, "12,10,10", interleaved=True),
        # the decode workload: 16 sequences of 1k to 8k tokens
        _step("step_decode_f16", "f16", 16, 1, 32, 8, 128, 8192, 64, 1025, 8192),
        # the large fp32 decode workload, keeping the running sums an eviction needs
        _step("step_decode_weights_f32", "f32", 32, 1, 32, 8, 128, 16384, 128, 4097, 16384, weights=True),
        # one long document, few heads: the work has to be split over the keys
        _step("step_long_f16", "f16", 1, 1, 16, 2, 64, 200192, 32, 200001, 200001),
        # a few drafted tokens per sequence, a different number for each
        _step("step_draft_f16", "f16", 5, 4, 24, 8, 96, 4096, 16, 37, 3001, ragged=True, weights=True),
        # the chunked prefill workload: 512 new tokens on 2k to 6k cached ones, window, softcap and sink
        _step("step_chunk_f16", "f16", 8, 512, 64, 8, 128, 8192, 64, 2560, 6656, window=4096, softcap=50.0,
              sink=True),
        # fresh prompts whose attention weights seed the running sums
        _step("step_prompt_weights_f16", "f16", 2, 4096, 32, 8, 128, 4096, 64, 4096, 4096, weights=True),
        # a ragged batch of fp32 prompts
        _step("step_prompt_f32", "f32", 3, 1500, 16, 4, 128, 2048, 128, 700, 1500, ragged=True),
        # a decode batch whose caches reached their capacity
        _evict("evict_decode_f16", "f16", 16, 32, 8, 128, 8192, 64, 6000, 8192, 2048, 256, 4),
        # long prompts reduced to a small decode cache
        _evict("evict_long_f32", "f32", 2, 16, 4, 128, 131072, 128, 100003, 131072, 4096, 512, 16),
    ]


def _loguniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotary", "step", "step", "decode", "decode", "evict"])
    dtype = rng.choice(["f16", "f16", "f32"])
    H = rng.choice([64, 80, 96, 128, 128, 128, 256])
    Nkv = rng.choice([1, 2, 3, 4, 8])
    N = Nkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    bs = rng.choice([16, 32, 64, 128, 256])
    if kind == "rotary":
        B = _loguniform(rng, 1, 16)
        S = _loguniform(rng, 1, max(1, min(4096, (1 << 26) // (B * (N + Nkv) * H))))
        axes = rng.choice([1, 2, 3, 4])
        pairs = rng.choice([H // 2, H // 4 // 8 * 8 or 8])
        cuts = sorted(rng.randrange(1, pairs) for _ in range(axes - 1))
        sec = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
        inter = rng.random() < 0.5
        if inter:   # every axis after the first has room among the pairs it takes
            sec = [pairs // axes] * axes
            sec[0] += pairs - sum(sec)
        return {k: v for k, v in _rotary("", dtype, B, S, N, Nkv, H, ",".join(map(str, sec)), inter,
                                         rng.random() < 0.5, rng.choice([4096, 32768])).items() if k != "name"}
    if kind == "evict":
        B = _loguniform(rng, 1, 16)
        T = _loguniform(rng, 300, min(131072, (1 << 27) // (B * Nkv * H)))
        C = (T + rng.randrange(0, 200) + bs - 1) // bs * bs
        keep = max(3, int(T * rng.uniform(0.05, 0.9)))
        recent = rng.randrange(1, keep)
        first = rng.randrange(0, min(16, keep - recent) + 1)
        return {k: v for k, v in _evict("", dtype, B, N, Nkv, H, C, bs, max(2, int(T * rng.uniform(0.02, 1.0))), T,
                                        keep, recent, first).items() if k != "name"}
    if kind == "decode":
        S = rng.choice([1, 1, 1, 2, 3, 5])
        B = _loguniform(rng, 1, 32)
        T = _loguniform(rng, S + 8, min(131072, (1 << 28) // (B * Nkv * H)))
    else:
        S = _loguniform(rng, 8, 2048)
        B = _loguniform(rng, 1, 8)
        T = S + rng.choice([0, _loguniform(rng, 1, 6000)])
        # pairs over all heads at most a quarter of the chunked workload's
        while B > 1 and B * N * S * T > 1 << 29:
            B -= 1
        while B * N * S * T > 1 << 29:
            N -= Nkv if N > Nkv else 0
            if N == Nkv and N * S * T > 1 << 29:
                S, T = max(8, S // 2), max(8, T // 2)
    C = (T + rng.randrange(0, 100) + bs - 1) // bs * bs
    ragged = rng.random() < 0.4
    lo = S if ragged else max(S, int(T * rng.uniform(0.1, 1.0)))
    return {k: v for k, v in _step("", dtype, B, S, N, Nkv, H, C, bs, lo, T, ragged,
                                   rng.choice([-1, -1, -1, rng.randrange(1, T + 1)]),
                                   rng.choice([0.0, 0.0, 0.0, 30.0]), rng.random() < 0.25,
                                   rng.random() < 0.4).items() if k != "name"}


# ------------------------------------------------------------------------------------------------ inputs

def _lengths(case, B):
    """Total lengths evenly spread over [lo, hi] (prepare() shuffles them)."""
    lo, hi = case["lo"], case["hi"]
    return [hi] if B == 1 else [lo + round((hi - lo) * b / (B - 1)) for b in range(B)]


def _new_rows(case, totals):
    """Rows each sequence adds: S, or for a ragged batch a different number each (at most its total)."""
    S = case["S"]
    if not case["ragged"]:
        return [S] * len(totals)
    return [min(t, S - (S - 1) * b // max(1, len(totals) - 1)) for b, t in enumerate(sorted(totals, reverse=True))]


def _sections(case):
    return [int(x) for x in case["sections"].split(",")]


def _cache(case, gen, dev):
    B, Nkv, H, C, bs = (case[k] for k in ("B", "Nkv", "H", "C", "bs"))
    st = {}
    for name in ("k", "v"):
        st[name + "_codes"] = torch.randint(-127, 128, (B, Nkv, C, H), dtype=torch.int8, device=dev, generator=gen)
        # scales of blocks of unit-variance rows, a few times larger for some blocks
        s = torch.rand((B, Nkv, C // bs), device=dev, generator=gen)
        st[name + "_scales"] = 0.01 + 0.02 * s + 0.05 * (s > 0.97)
    return st


def _data(case, seed):
    """The inputs of a case as tensors and plain values."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    t = DT[case["dtype"]]
    B, N, Nkv, H = (case[k] for k in ("B", "N", "Nkv", "H"))

    def normal(*shape, std=1.0):
        return (torch.randn(shape, device=dev, generator=gen) * std).to(t)

    if case["op"] == "rotary":
        S, sec = case["S"], _sections(case)
        st = dict(query=normal(B, S, N * H), key=normal(B, S, Nkv * H))
        # text runs on all axes alike; an image keeps its time and walks over its rows and columns
        base = torch.randint(0, case["R"] - 2 * S if case["R"] > 2 * S else 1, (B, 1), device=dev, generator=gen)
        i = torch.arange(S, device=dev)[None]
        w = max(1, math.isqrt(S))
        axis = [base + i * 0 if a == 0 and S > 1 else base + (i // w if a % 2 else i % w) for a in range(len(sec))]
        st["positions"] = torch.stack([x.expand(B, S) for x in axis]).to(torch.int32).contiguous()
        pairs = sum(sec)
        ang = (torch.arange(case["R"], device=dev, dtype=torch.float64)[:, None]
               * (1e6 ** (-torch.arange(pairs, device=dev, dtype=torch.float64) / pairs))[None])
        st["cos"], st["sin"] = ang.cos().to(t), ang.sin().to(t)
        st["q_w"] = (1 + 0.1 * torch.randn(H, device=dev, generator=gen)).to(t) if case["norm"] else None
        st["k_w"] = (1 + 0.1 * torch.randn(H, device=dev, generator=gen)).to(t) if case["norm"] else None
        return st

    totals = _lengths(case, B)
    new = _new_rows(case, totals) if case["op"] == "step" else [1] * B
    order = torch.randperm(B, device=dev, generator=gen)
    if case["op"] == "step" and case["ragged"]:
        totals = sorted(totals, reverse=True)
    st = _cache(case, gen, dev)
    st["total"] = torch.tensor(totals, dtype=torch.int32, device=dev)[order].contiguous()
    st["new"] = torch.tensor(new, dtype=torch.int32, device=dev)[order].contiguous()
    st["seqlens_k"] = st["total"] - 1
    st["T"] = max(totals)
    S = case["S"] if case["op"] == "step" else 1
    st["query"] = normal(B, S, N * H, std=2.0)
    if case["op"] == "step":
        st["key"] = normal(B, S, Nkv * H)
        st["value"] = normal(B, S, Nkv * H)
        st["sink"] = normal(N) if case["sink"] else None
        if case["weights"]:
            st["past_weights"] = torch.rand((B, Nkv, case["C"]), device=dev, generator=gen)
            st["present_weights"] = torch.zeros((B, Nkv, case["C"]), device=dev)
    else:
        w = torch.rand((B, Nkv, case["C"]), device=dev, generator=gen) ** 8 * 50
        st["weights"] = torch.where(w < 1e-6, torch.zeros_like(w), w)   # rows nothing ever attended to
        keep, bs = case["keep"], case["bs"]
        rows = (keep + bs - 1) // bs * bs
        st["to_k_codes"] = torch.zeros((B, Nkv, rows, H), dtype=torch.int8, device=dev)
        st["to_v_codes"] = torch.zeros((B, Nkv, rows, H), dtype=torch.int8, device=dev)
        st["to_k_scales"] = torch.zeros((B, Nkv, rows // bs), device=dev)
        st["to_v_scales"] = torch.zeros((B, Nkv, rows // bs), device=dev)
        st["to_weights"] = torch.zeros((B, Nkv, rows), device=dev)
    return st


def prepare(case, seed):
    st = _data(case, seed)
    st["case"] = case
    if own:
        from grouped_query_attention_gb300 import BlockCache, GroupQueryAttention
        st["op"] = GroupQueryAttention(case["N"], case["Nkv"], softcap=case.get("softcap", 0.0),
                                       local_window_size=case.get("window", -1))
        if case["op"] != "rotary":
            st["cache"] = BlockCache(st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"], case["bs"])
        if case["op"] == "evict":
            st["into"] = BlockCache(st["to_k_codes"], st["to_v_codes"], st["to_k_scales"], st["to_v_scales"],
                                    case["bs"])
    return st


# ------------------------------------------------------------------------------------------------ plain forms

def _axis_of_pair(sec, interleaved, dev):
    d = torch.arange(sum(sec), device=dev)
    if not interleaved:
        ends = torch.tensor(sec, device=dev).cumsum(0)
        return torch.searchsorted(ends, d, right=True)
    a = len(sec)
    counts = torch.tensor([0] + sec[1:], device=dev)
    r = d % a
    return torch.where(d < a * counts[r], r, torch.zeros_like(r))


def _plain_rotary(st):
    case = st["case"]
    B, S, H = case["B"], case["S"], case["H"]
    sec = _sections(case)
    pairs = sum(sec)
    axis = _axis_of_pair(sec, case["interleaved"], st["cos"].device)
    pos = st["positions"].long()[axis].permute(1, 2, 0)                       # (B, S, pairs)
    d = torch.arange(pairs, device=pos.device)
    c = st["cos"][pos, d].float()[:, :, None]
    s = st["sin"][pos, d].float()[:, :, None]

    def turn(x, n, w):
        x = x.view(B, S, n, H).float()
        if w is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        a, b = x[..., :pairs], x[..., pairs:2 * pairs]
        y = torch.cat((a * c - b * s, b * c + a * s, x[..., 2 * pairs:]), dim=-1)
        return y.to(st["query"].dtype).view(B, S, n * H)

    return {"query": turn(st["query"], case["N"], st["q_w"]), "key": turn(st["key"], case["Nkv"], st["k_w"])}


def _plain_append(st, name, codes, scales):
    """Quantise the new rows of `st[name]` into the blocks they touch (codes, scales in place)."""
    case = st["case"]
    B, S, Nkv, H, C, bs = (case[k] for k in ("B", "S", "Nkv", "H", "C", "bs"))
    nb = C // bs
    nt = min((S + bs - 2) // bs + 1, nb)
    total, past = st["total"].long(), (st["total"] - st["new"]).long()
    blk = (past // bs).clamp(max=nb - nt)[:, None] + torch.arange(nt, device=past.device)   # (B, nt)
    rows = blk[:, :, None] * bs + torch.arange(bs, device=past.device)                      # (B, nt, bs)
    bi = torch.arange(B, device=past.device)[:, None]
    old = rows < past[:, None, None]
    fresh = ~old & (rows < total[:, None, None])
    src = (rows - past[:, None, None]).clamp(0, S - 1)
    x = st[name].view(B, S, Nkv, H)[bi[:, :, None], src].permute(0, 1, 3, 2, 4).float()     # (B, nt, Nkv, bs, H)
    fresh, old = fresh[:, :, None, :, None], old[:, :, None, :, None]
    amax = torch.where(fresh, x.abs(), torch.zeros_like(x)).amax((-1, -2))                  # (B, nt, Nkv)
    c = codes.view(B, Nkv, nb, bs, H)[bi, :, blk]
    s0 = scales[bi, :, blk]
    had = torch.where(old.any(3).any(-1), s0, torch.zeros_like(s0))
    s = torch.where(fresh.any(3).any(-1), torch.maximum(had, amax / 127), s0)
    # the nearest code of x / s: quotients in 64 bits, they lie next to a border now and then
    v = torch.where(fresh, x.double(), c.double() * s0.double()[..., None, None])
    q = torch.where(s[..., None, None] > 0, v / s.double()[..., None, None], torch.zeros_like(v))
    q = q.round().clamp(-127, 127).to(torch.int8)
    codes.view(B, Nkv, nb, bs, H)[bi, :, blk] = torch.where(fresh | old, q, c)
    scales[bi, :, blk] = s


def _plain_attend(st, codes, scales, total, new, T, sink, window, softcap, weights=None):
    """Attention of the last new[b] rows of each sequence over cache rows [0, T)."""
    case = st["case"]
    B, N, Nkv, H, bs = (case[k] for k in ("B", "N", "Nkv", "H", "bs"))
    G = N // Nkv
    q = st["query"]
    S = q.shape[1]
    k, v = (codes[i][:, :, :T].float() * scales[i].repeat_interleave(bs, dim=2)[:, :, :T, None] for i in (0, 1))
    qr = q.view(B, S, Nkv, G, H).permute(0, 2, 3, 1, 4).reshape(B, Nkv, G * S, H).float()
    s = torch.matmul(qr, k.transpose(-1, -2)).view(B, Nkv, G, S, T) * (1.0 / math.sqrt(H))
    if softcap > 0:
        s = softcap * torch.tanh(s / softcap)
    i, j = torch.arange(S, device=q.device), torch.arange(T, device=q.device)
    p = (total - new)[:, None] + i                                                          # (B, S) cache rows
    see = (j <= p[:, :, None]) & (i[None, :, None] < new[:, None, None])
    if window >= 0:
        see &= j >= p[:, :, None] - window
    s = s.masked_fill(~see[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    if sink is not None:
        sk = sink.float().view(1, Nkv, G, 1, 1)
        m = torch.maximum(m, sk)
    e = torch.exp(s - m)
    den = e.sum(-1, keepdim=True)
    if sink is not None:
        den = den + torch.exp(sk - m)
    e = torch.where(den > 0, e / den, torch.zeros_like(e))
    out = torch.matmul(e.view(B, Nkv, G * S, T), v).view(B, Nkv, G, S, H)
    out = out * (i[None] < new[:, None])[:, None, None, :, None]
    if weights is not None:
        past, present = weights
        got = e.sum((2, 3))
        had = torch.where(j < (total - new)[:, None, None], past[:, :, :T], torch.zeros_like(got))
        present[:, :, :T] = torch.where(j < total[:, None, None], had + got, present[:, :, :T])
    return out.permute(0, 3, 1, 2, 4).reshape(B, S, N * H).to(q.dtype)


def _plain_step(st):
    case = st["case"]
    _plain_append(st, "key", st["k_codes"], st["k_scales"])
    _plain_append(st, "value", st["v_codes"], st["v_scales"])
    w = (st["past_weights"], st["present_weights"]) if case["weights"] else None
    out = _plain_attend(st, (st["k_codes"], st["v_codes"]), (st["k_scales"], st["v_scales"]), st["total"], st["new"],
                        st["T"], st["sink"], case["window"], case["softcap"], w)
    return _step_outputs(st, out)


def _step_outputs(st, out):
    got = {"output": out, "key_scales": st["k_scales"], "value_scales": st["v_scales"]}
    if st["case"]["weights"]:
        got["weights"] = st["present_weights"]
    return got


def _plain_evict(st):
    case = st["case"]
    B, Nkv, H, C, bs, keep = (case[k] for k in ("B", "Nkv", "H", "C", "bs", "keep"))
    recent, first = case["recent"], case["first"]
    total = st["total"].long()
    j = torch.arange(C, device=total.device)
    forced = (j < first) | (j >= (total - recent)[:, None])                                # (B, C)
    live = j < total[:, None]
    w = torch.where(forced[:, None], torch.full_like(st["weights"], float("inf")), st["weights"])
    w = torch.where(live[:, None], w, torch.full_like(w, float("-inf")))
    n = total.clamp(max=keep)                                                              # rows that stay
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[:, :, :keep]
    slot = torch.arange(keep, device=total.device)
    order = torch.where(slot < n[:, None, None], order, torch.full_like(order, C))
    kept = order.sort(-1).values                                                           # (B, Nkv, keep)
    stays = kept < C
    at = kept.clamp(max=C - 1)
    rows = st["to_weights"].shape[-1]
    pad = rows - keep
    for name in ("k", "v"):
        c = st[name + "_codes"].gather(2, at[..., None].expand(-1, -1, -1, H))
        s = st[name + "_scales"].gather(2, at // bs)
        s = torch.where(stays, s, torch.zeros_like(s))
        sb = torch.nn.functional.pad(s, (0, pad)).view(B, Nkv, rows // bs, bs).amax(-1)    # scale of a new block
        to = st["to_" + name + "_codes"]
        sr = sb.repeat_interleave(bs, dim=2)[:, :, :keep]
        quot = c.double() * s.double()[..., None] / sr.double()[..., None]
        quot = torch.where(sr[..., None] > 0, quot, torch.zeros_like(quot)).round().to(torch.int8)
        to[:, :, :keep] = torch.where(stays[..., None], quot, to[:, :, :keep])
        used = (torch.arange(rows // bs, device=total.device) * bs < n[:, None])[:, None]
        st["to_" + name + "_scales"][:] = torch.where(used, sb, st["to_" + name + "_scales"])
    st["to_weights"][:, :, :keep] = torch.where(stays, st["weights"].gather(2, at), st["to_weights"][:, :, :keep])
    kept = torch.where(stays, kept, torch.full_like(kept, -1)).to(torch.int32)
    n32 = n.to(torch.int32)
    out = _plain_attend(st, (st["to_k_codes"], st["to_v_codes"]), (st["to_k_scales"], st["to_v_scales"]), n32,
                        st["new"], min(keep, st["T"]), None, -1, 0.0)
    return _evict_outputs(st, out, kept, n32 - 1)


def _evict_outputs(st, out, kept, seqlens):
    return {"output": out, "kept": kept, "seqlens_k": seqlens, "weights": st["to_weights"],
            "key_scales": st["to_k_scales"], "value_scales": st["to_v_scales"]}


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if not own:
        return {"rotary": _plain_rotary, "step": _plain_step, "evict": _plain_evict}[case["op"]](state)
    op = state["op"]
    if case["op"] == "rotary":
        q, k = op.rotary_axes(state["query"], state["key"], state["positions"], state["cos"], state["sin"],
                              _sections(case), interleaved=case["interleaved"], q_norm_weight=state["q_w"],
                              k_norm_weight=state["k_w"])
        return {"query": q, "key": k}
    if case["op"] == "step":
        out = op.block_forward(state["query"], state["key"], state["value"], state["seqlens_k"], state["T"],
                               state["cache"], new_lens=state["new"] if case["ragged"] else None,
                               head_sink=state["sink"], past_weights=state.get("past_weights"),
                               present_weights=state.get("present_weights"))
        return _step_outputs(state, out)
    kept, seqlens = op.block_evict(state["cache"], state["weights"], state["seqlens_k"], state["T"], case["keep"],
                                   state["into"], state["to_weights"], recent=case["recent"], first=case["first"])
    out = op.block_forward(state["query"], None, None, seqlens, min(case["keep"], state["T"]), state["into"])
    return _evict_outputs(state, out, kept, seqlens)


# ------------------------------------------------------------------------------------------------ work of a pass

def _pairs(case, total, new):
    """Visible (query, key) pairs of one head of a sequence, and the cache rows its queries reach."""
    W = case.get("window", -1)
    past = total - new
    pairs = 0
    if W < 0:
        pairs = new * past + new * (new + 1) // 2
        return pairs, total
    pairs = sum(min(p, W) + 1 for p in range(past, total))
    return pairs, total - max(0, past - W)


def work(case):
    B, N, Nkv, H = (case[k] for k in ("B", "N", "Nkv", "H"))
    e = 2 if case["dtype"] == "f16" else 4
    if case["op"] == "rotary":
        S, sec = case["S"], _sections(case)
        n = B * S * (N + Nkv) * H
        return {"bytes": 2 * n * e + 4 * len(sec) * B * S + 2 * e * sum(sec) * min(B * S, case["R"]),
                "flops": (3 if not case["norm"] else 7) * n}
    totals = sorted(_lengths(case, B), reverse=True)
    bs = case["bs"]
    if case["op"] == "step":
        news = _new_rows(case, totals)
        both = [_pairs(case, t, n) for t, n in zip(totals, news)]
        rows = sum(r for _, r in both)
        byt = sum(news) * (2 * N + 2 * Nkv) * H * e + rows * Nkv * (2 * H + 8 / bs) + sum(news) * Nkv * 2 * H
        if case["weights"]:
            byt += 8 * Nkv * sum(totals)
        return {"bytes": byt, "flops": 4 * H * N * sum(p for p, _ in both)}
    kept = sum(min(t, case["keep"]) for t in totals)
    byt = Nkv * (4 * sum(totals) + kept * (2 * 2 * H + 4 + 4 + 4 + 16 / bs)) + 2 * B * N * H * e
    return {"bytes": byt, "flops": 4 * H * N * kept}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = _data(case, seed)
    return {"rotary": _exact_rotary, "step": _exact_step, "evict": _exact_evict}[case["op"]](case, st)


def _exact_rotary(case, st):
    """Pairs as complex numbers, each multiplied by the table's value at its own axis' position."""
    sec = _sections(case)
    n = sum(sec)
    axes = []
    for d in range(n):
        if case["interleaved"]:
            r = d % len(sec)
            axes.append(r if r > 0 and d // len(sec) < sec[r] else 0)
        else:
            axes.append(next(a for a in range(len(sec)) if d < sum(sec[:a + 1])))
    unit = torch.complex(st["cos"].double(), st["sin"].double())
    got = {}
    for name, heads, w in (("query", case["N"], st["q_w"]), ("key", case["Nkv"], st["k_w"])):
        x = st[name].double().reshape(case["B"], case["S"], heads, case["H"])
        if w is not None:
            x = x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / case["H"] + 1e-6) * w.double()
        y = x.clone()
        for d in range(n):
            u = unit[st["positions"][axes[d]].long(), d][:, :, None]
            z = torch.complex(x[..., d], x[..., d + n]) * u
            y[..., d], y[..., d + n] = z.real, z.imag
        got[name] = y.reshape(case["B"], case["S"], heads * case["H"])
    return got


def _exact_rows(case, st, b, name, total, new):
    """Values and block scales of one sequence's cache after its new rows are stored."""
    bs, Nkv, H = case["bs"], case["Nkv"], case["H"]
    short = {"key": "k", "value": "v"}[name]
    val = st[short + "_codes"][b, :, :total].double()
    sc = st[short + "_scales"][b].double().clone()
    past = total - new
    if past:
        val[:, :past] *= sc[:, torch.arange(past, device=sc.device) // bs, None]
    if new:
        val[:, past:] = st[name][b, :new].double().view(new, Nkv, H).transpose(0, 1)
        for blk in range(past // bs, (total - 1) // bs + 1):
            a, z = blk * bs, min((blk + 1) * bs, total)
            here = val[:, max(a, past):z].abs().amax((1, 2)).float() / 127       # a scale is held in 32 bits
            s = torch.maximum(here.double(), sc[:, blk]) if past > a else here.double()
            sc[:, blk] = s
            s = s[:, None, None]
            val[:, a:z] = torch.where(s > 0, (val[:, a:z] / s).round().clamp(-127, 127) * s, 0.0)
    return val, sc


def _exact_attend(case, q, k, v, total, new, sink, window, softcap):
    """q (S, N, H), k and v (Nkv, total, H) -> output (S, N, H), weight of each cache row (Nkv, total)."""
    Nkv, H = case["Nkv"], case["H"]
    G = case["N"] // Nkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    got = torch.zeros((Nkv, total), dtype=torch.float64, device=q.device)
    pos = torch.arange(total - new, total, device=q.device)
    gap = pos[:, None] - torch.arange(total, device=q.device)[None]
    hide = gap < 0 if window < 0 else (gap < 0) | (gap > window)
    for h in range(case["N"]):
        g = h // G
        z = q[:new, h].double() @ k[g].T / math.sqrt(H)
        if softcap > 0:
            z = torch.tanh(z / softcap) * softcap
        z = torch.where(hide, -math.inf, z)
        if sink is not None:
            z = torch.cat((z, sink[h].double().expand(new, 1)), dim=1)
        z = torch.softmax(z, dim=1)[:, :total]
        out[:new, h] = z @ v[g]
        got[g] += z.sum(0)
    return out, got


def _exact_step(case, st):
    B, S, N, H, C = (case[k] for k in ("B", "S", "N", "H", "C"))
    out = torch.zeros((B, S, N, H), dtype=torch.float64, device=st["query"].device)
    ks, vs = st["k_scales"].double().clone(), st["v_scales"].double().clone()
    w = torch.zeros((B, case["Nkv"], C), dtype=torch.float64, device=out.device)
    for b in range(B):
        total, new = int(st["total"][b]), int(st["new"][b])
        k, ks[b] = _exact_rows(case, st, b, "key", total, new)
        v, vs[b] = _exact_rows(case, st, b, "value", total, new)
        out[b], got = _exact_attend(case, st["query"][b].view(S, N, H), k, v, total, new, st["sink"], case["window"],
                                    case["softcap"])
        if case["weights"]:
            past = total - new
            w[b, :, :past] = st["past_weights"][b, :, :past].double()
            w[b, :, :total] += got
    res = {"output": out.view(B, S, N * H), "key_scales": ks, "value_scales": vs}
    if case["weights"]:
        res["weights"] = w
    return res


def _exact_evict(case, st):
    B, N, Nkv, H, bs, keep = (case[k] for k in ("B", "N", "Nkv", "H", "bs", "keep"))
    dev = st["query"].device
    rows = st["to_weights"].shape[-1]
    out = torch.zeros((B, 1, N, H), dtype=torch.float64, device=dev)
    w = torch.zeros((B, Nkv, rows), dtype=torch.float64, device=dev)
    scales = {n: torch.zeros((B, Nkv, rows // bs), dtype=torch.float64, device=dev) for n in ("k", "v")}
    kept = torch.full((B, Nkv, keep), -1, dtype=torch.int32, device=dev)
    for b in range(B):
        total = int(st["total"][b])
        n = min(total, keep)
        vals = {m: torch.zeros((Nkv, n, H), dtype=torch.float64, device=dev) for m in ("k", "v")}
        for g in range(Nkv):
            if total <= keep:
                idx = torch.arange(total, device=dev)
            else:
                inner = st["weights"][b, g, case["first"]:total - case["recent"]].double()
                best = torch.sort(-inner, stable=True).indices[:keep - case["first"] - case["recent"]]
                idx = torch.cat((torch.arange(case["first"], device=dev), best.sort().values + case["first"],
                                 torch.arange(total - case["recent"], total, device=dev)))
            kept[b, g, :n] = idx.int()
            w[b, g, :n] = st["weights"][b, g, idx].double()
            for m in ("k", "v"):
                s = st[m + "_scales"][b, g, idx // bs].double()
                x = st[m + "_codes"][b, g, idx].double() * s[:, None]
                for blk in range((n + bs - 1) // bs):
                    a, z = blk * bs, min((blk + 1) * bs, n)
                    top = s[a:z].max()
                    scales[m][b, g, blk] = top
                    x[a:z] = torch.where(top > 0, (x[a:z] / top).round() * top, 0.0)
                vals[m][g] = x
        out[b], _ = _exact_attend(case, st["query"][b].view(1, N, H), vals["k"], vals["v"], n, 1, None, -1, 0.0)
    return {"output": out.view(B, 1, N * H), "kept": kept, "seqlens_k": (st["total"].clamp(max=keep) - 1),
            "weights": w, "key_scales": scales["k"], "value_scales": scales["v"]}
