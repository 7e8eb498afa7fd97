"""Cases of speculative decoding over the float cache: attention for a tree of drafted tokens, verification of the
drafts against the target's probabilities, and moving the accepted rows of the caches together.

A case is one pass through one of them, as a serving loop calls it:

tree    S drafted nodes per sequence are stored behind its cached rows, then every node attends to the cached rows,
        its ancestors and itself.
verify  the drafted tokens are tested one by one from the root on, with given random numbers, and the token behind the
        last accepted one is drawn from what the target's probabilities leave.
accept  the accepted nodes' rows of every layer's cache move together behind the cached rows.
"""

import math
import random

import torch

own = False

DT = {"f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases

def _tree(name, dtype, B, S, N, Nkv, H, C, lo, hi, shape="tree", ragged=False, window=-1, softcap=0.0, sink=False):
    return dict(name=name, op="tree", dtype=dtype, B=B, S=S, N=N, Nkv=Nkv, H=H, C=C, lo=lo, hi=hi, shape=shape,
                ragged=ragged, window=window, softcap=softcap, sink=sink)


def _verify(name, dtype, B, S, V, shape="tree", drafts=True, ragged=False):
    return dict(name=name, op="verify", dtype=dtype, B=B, S=S, V=V, shape=shape, drafts=drafts, ragged=ragged)


def _accept(name, dtype, L, B, S, Nkv, H, C, ragged=False):
    return dict(name=name, op="accept", dtype=dtype, L=L, B=B, S=S, Nkv=Nkv, H=H, C=C, ragged=ragged)


def listed():
    return [
        # one user, five drafted tokens in a row on a short conversation: the smallest step
        _tree("tree_chain_f16", "f16", 1, 5, 32, 8, 128, 2048, 1030, 1030, shape="chain"),
        # the decode workload's caches (16 sequences of 1k to 8k tokens) with a tree of 16 nodes each
        _tree("tree_decode_f16", "f16", 16, 16, 32, 8, 128, 8192, 1040, 8192),
        # wide trees on the chunked prefill workload's caches: window, softcap and sink
        _tree("tree_wide_f16", "f16", 8, 64, 64, 8, 128, 8192, 2112, 6208, window=4096, softcap=50.0, sink=True),
        # one long document, few heads: the work has to be split over the keys
        _tree("tree_long_f16", "f16", 1, 26, 16, 2, 64, 200192, 200026, 200026),
        # a different number of drafts for each sequence, an odd head size
        _tree("tree_ragged_f16", "f16", 5, 13, 24, 8, 96, 4096, 37, 3001, ragged=True),
        # fp32 tensors over fp32 caches
        _tree("tree_decode_f32", "f32", 8, 8, 32, 8, 128, 16384, 4104, 16384),
        # one user, four drafted tokens in a row, a small vocabulary
        _verify("verify_chain", "f32", 1, 5, 32768, shape="chain"),
        # a batch of drafted chains of different lengths
        _verify("verify_chain_batch", "f32", 64, 8, 131072, shape="chain", ragged=True),
        # trees drawn from the draft's probabilities, an odd vocabulary
        _verify("verify_tree", "f32", 16, 64, 100003),
        # trees of the draft's most likely tokens (no draft probabilities), half-precision probabilities
        _verify("verify_tree_top_f16", "f16", 32, 32, 131072, drafts=False),
        # one layer of one user
        _accept("accept_one_layer", "f16", 1, 1, 8, 8, 128, 2048),
        # all layers of a batch
        _accept("accept_layers", "f16", 32, 16, 64, 8, 128, 256, ragged=True),
    ]


def _loguniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "tree", "verify", "verify", "accept"])
    dtype = rng.choice(["f16", "f16", "f32"])
    H = rng.choice([64, 80, 96, 128, 128, 128, 256])
    Nkv = rng.choice([1, 2, 3, 4, 8])
    shape = rng.choice(["tree", "tree", "chain"])
    ragged = rng.random() < 0.4
    if kind == "verify":
        V = _loguniform(rng, 1000, 262144)
        B = _loguniform(rng, 1, 64)
        S = _loguniform(rng, 1, max(1, min(100, (1 << 27) // (B * V))))
        case = _verify("", rng.choice(["f32", "f32", "f16"]), B, S, V, shape, rng.random() < 0.6, ragged)
    elif kind == "accept":
        B = _loguniform(rng, 1, 16)
        S = _loguniform(rng, 1, 128)
        C = S + _loguniform(rng, 1, 1000)
        L = _loguniform(rng, 1, max(1, min(60, (1 << 26) // (B * Nkv * C * H))))
        case = _accept("", dtype, L, B, S, Nkv, H, C, ragged)
    else:
        N = Nkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
        B = _loguniform(rng, 1, 32)
        S = _loguniform(rng, 1, 256)
        T = S + _loguniform(rng, 1, min(131072, (1 << 26) // (B * Nkv * H)))
        # (row, key) pairs over all heads at most a quarter of the wide trees'
        while B > 1 and B * N * S * T > 1 << 25:
            B -= 1
        while S > 1 and B * N * S * T > 1 << 25:
            S -= 1
        C = T + rng.randrange(0, 100)
        lo = S if rng.random() < 0.2 else max(S, int(T * rng.uniform(0.1, 1.0)))
        case = _tree("", dtype, B, S, N, Nkv, H, C, lo, T, shape, ragged, rng.choice([-1, -1, -1, rng.randrange(1, T + 1)]),
                     rng.choice([0.0, 0.0, 0.0, 30.0]), rng.random() < 0.25)
    del case["name"]
    return case


# ------------------------------------------------------------------------------------------------ inputs

def _parents(rnd, S, shape):
    """Parents of S nodes, each before its children, node 0 the root. A tree grows near its root and its latest nodes."""
    par = [-1]
    for i in range(1, S):
        par.append(i - 1 if shape == "chain" else rnd.randrange(i) if rnd.random() < 0.6 else rnd.randrange(max(0, i - 4), i))
    return par


def _ancestors(par):
    """ancestors-or-self of every node, as rows of truth values."""
    rows = []
    for i, a in enumerate(par):
        row = list(rows[a]) if a >= 0 else [False] * len(par)
        row[i] = True
        rows.append(row)
    return rows


def _counts(case):
    """Nodes of every sequence: S, or for a ragged batch a different number each."""
    B, S = case["B"], case["S"]
    return [S - (S - 1) * b // max(1, B - 1) if case["ragged"] else S for b in range(B)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rnd = random.Random(int(seed))
    t = DT[case["dtype"]]
    B, S = case["B"], case["S"]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, device=dev, generator=gen) * std).to(t)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    st = {"case": case}
    order = rnd.sample(range(B), B)
    new = _counts(case)
    st["new"] = ints([new[b] for b in order])
    if case["op"] != "accept":
        trees = [_parents(rnd, S, case["shape"]) for _ in range(B)]
        st["parents"] = ints(trees)
    if case["op"] == "tree":
        N, Nkv, H, C, lo, hi = (case[k] for k in ("N", "Nkv", "H", "C", "lo", "hi"))
        totals = [hi] if B == 1 else [max(lo + round((hi - lo) * b / (B - 1)), new[b]) for b in range(B)]
        st["total"] = ints([totals[b] for b in order])
        st["seqlens_k"] = st["total"] - 1
        st["T"] = max(totals)
        # what a program without tree attention keeps in place of the parents
        st["ancestors"] = torch.tensor([_ancestors(x) for x in trees], device=dev)
        st["query"] = normal(B, S, N * H, std=2.0)
        st["key"], st["value"] = normal(B, S, Nkv * H), normal(B, S, Nkv * H)
        st["present_key"], st["present_value"] = normal(B, Nkv, C, H), normal(B, Nkv, C, H)
        st["sink"] = normal(N) if case["sink"] else None
    elif case["op"] == "verify":
        V = case["V"]
        # the draft's logits are the target's with an error
        logits = torch.randn((B, S, V), device=dev, generator=gen) * 3.0
        draft = torch.softmax(logits + 0.7 * torch.randn(logits.shape, device=dev, generator=gen), dim=-1)
        st["target_probs"] = torch.softmax(logits, dim=-1).to(t)
        del logits
        if case["drafts"]:   # every child drawn from its parent's row
            cum = draft.double().cumsum(-1)
            at = st["parents"].long().clamp(min=0)
            x = torch.rand((B, S, 1), device=dev, generator=gen, dtype=torch.float64)
            rows = cum.gather(1, at[:, :, None].expand(B, S, V)) if S * V * B < 1 << 24 else None
            if rows is None:
                tok = torch.stack([torch.searchsorted(cum[b, at[b]], x[b] * cum[b, at[b], -1:]) for b in range(B)])
            else:
                tok = torch.searchsorted(rows, x * rows[..., -1:])
            st["tokens"] = tok[..., 0].clamp(max=V - 1).to(torch.int32)
            st["draft_probs"] = draft.to(t)
            del cum, rows
        else:                # the first, second, ... most likely token of the parent's row
            par = st["parents"].cpu().tolist()
            rank = [[sum(1 for y in row[1:i] if y == row[i]) for i in range(S)] for row in par]
            top = draft.topk(min(V, 1 + max(map(max, rank))), dim=-1).indices
            at = st["parents"].long().clamp(min=0)
            st["tokens"] = top[torch.arange(B, device=dev)[:, None], at, ints(rank).long()].to(torch.int32)
            st["draft_probs"] = None
        st["accept_uniforms"] = torch.rand((B, S), device=dev, generator=gen)
        st["sample_uniforms"] = torch.rand((B,), device=dev, generator=gen)
    else:
        L, Nkv, H, C = (case[k] for k in ("L", "Nkv", "H", "C"))
        new = [new[b] for b in order]
        lens = [1 + rnd.randrange(n) for n in new]
        paths = [[0] + sorted(rnd.sample(range(1, n), k - 1)) + [-1] * (S - k) for n, k in zip(new, lens)]
        st["path"], st["path_lens"] = ints(paths), ints(lens)
        st["total"] = ints([n + rnd.randrange(0, C - S + 1) for n in new])
        st["seqlens_k"] = st["total"] - 1
        st["keys"], st["values"] = normal(L, B, Nkv, C, H), normal(L, B, Nkv, C, H)
        st["caches"] = list(zip(st["keys"].unbind(0), st["values"].unbind(0)))
    if own:
        from grouped_query_attention_gb300 import GroupQueryAttention
        st["gqa"] = GroupQueryAttention(case.get("N", 1) if case["op"] == "tree" else case.get("Nkv", 1),
                                        case.get("Nkv", 1), softcap=case.get("softcap", 0.0),
                                        local_window_size=case.get("window", -1))
    return st


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_tree(st):
    case = st["case"]
    B, S, N, Nkv, H = (case[k] for k in ("B", "S", "N", "Nkv", "H"))
    G, T, W = N // Nkv, st["T"], case["window"]
    q, total, new = st["query"], st["total"].long(), st["new"].long()
    past = total - new
    dev = q.device
    i, j, bi = torch.arange(S, device=dev), torch.arange(T, device=dev), torch.arange(B, device=dev)[:, None]
    live = i < new[:, None]                                                                 # (B, S)
    # store the nodes (a padding node writes node 0's row once more)
    src = torch.where(live, i, torch.zeros_like(i))
    rows = past[:, None] + src
    st["present_key"][bi, :, rows] = st["key"].view(B, S, Nkv, H)[bi, src]
    st["present_value"][bi, :, rows] = st["value"].view(B, S, Nkv, H)[bi, src]
    # visible rows: the cached ones and the ancestors, within the window by depth
    depth = st["ancestors"].sum(-1) - 1
    rel = j - past[:, None]                                                                 # (B, T)
    node = rel.clamp(0, S - 1)
    anc = st["ancestors"].gather(2, node[:, None].expand(B, S, T))
    at = torch.where(rel < 0, rel, depth.gather(1, node))[:, None]                          # depth of a key, past ones below 0
    see = torch.where((rel < 0)[:, None], torch.ones_like(anc), anc & (rel < new[:, None])[:, None]) & live[:, :, None]
    if W >= 0:
        see = see & (at >= depth[:, :, None] - W)
    k, v = st["present_key"][:, :, :T].float(), st["present_value"][:, :, :T].float()
    qr = q.view(B, S, Nkv, G, H).permute(0, 2, 3, 1, 4).reshape(B, Nkv, G * S, H).float()
    s = torch.matmul(qr, k.transpose(-1, -2)).view(B, Nkv, G, S, T) * (1.0 / math.sqrt(H))
    if case["softcap"] > 0:
        s = case["softcap"] * torch.tanh(s / case["softcap"])
    s = s.masked_fill(~see[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    if st["sink"] is not None:
        sk = st["sink"].float().view(1, Nkv, G, 1, 1)
        m = torch.maximum(m, sk)
    e = torch.exp(s - m)
    den = e.sum(-1, keepdim=True)
    if st["sink"] is not None:
        den = den + torch.exp(sk - m)
    e = torch.where(den > 0, e / den, torch.zeros_like(e))
    # rows behind a sequence's last hold anything: their weight is zero, and so is what they add
    v = torch.where((j < total[:, None])[:, None, :, None], v, torch.zeros_like(v))
    out = torch.matmul(e.view(B, Nkv, G * S, T), v).view(B, Nkv, G, S, H) * live[:, None, None, :, None]
    return {"output": out.permute(0, 3, 1, 2, 4).reshape(B, S, N * H).to(q.dtype),
            "present_key": st["present_key"], "present_value": st["present_value"]}


def _plain_verify(st):
    case = st["case"]
    B, S, V = case["B"], case["S"], case["V"]
    p, q = st["target_probs"], st["draft_probs"]
    par, tok, new, u = st["parents"].long(), st["tokens"].long(), st["new"].long(), st["accept_uniforms"].double()
    dev = p.device
    bi = torch.arange(B, device=dev)
    cur = torch.zeros(B, dtype=torch.long, device=dev)
    count = (new > 0).long()
    path = torch.full((B, S + 1), -1, dtype=torch.int32, device=dev)
    path[:, 0] = torch.where(new > 0, 0, -1)
    # what is left of the target's row behind the children turned down so far, and its sum (a fresh row's is 1)
    left, z = p[:, 0].double(), torch.ones(B, dtype=torch.float64, device=dev)
    # the sequential sweep of the definition: a node is tested when its parent is the last accepted one
    for i in range(1, S):
        test = (par[:, i] == cur) & (i < new)
        x = tok[:, i]
        qx = q[bi, cur, x].double() if q is not None else torch.ones_like(z)
        took = test & (u[:, i] * qx * z < left[bi, x])
        lost = test & ~took
        if q is not None:
            rest = (left / torch.where(z > 0, z, torch.ones_like(z))[:, None] - q[bi, cur].double()).clamp(min=0)
        else:
            rest = left.scatter(1, x[:, None], 0.0)
        left = torch.where(lost[:, None], rest, left)
        z = torch.where(lost, left.sum(-1), z)
        path[bi, torch.where(took, count, S)] = torch.where(took, i, -1).to(torch.int32)
        count = count + took
        cur = torch.where(took, i, cur)
        left = torch.where(took[:, None], p[bi, cur].double(), left)
        z = torch.where(took, 1.0, z)
    left = torch.where((left.sum(-1) > 0)[:, None], left, p[bi, cur].double())
    cum = left.cumsum(-1)
    token = (cum <= st["sample_uniforms"].double()[:, None] * cum[:, -1:]).sum(-1).clamp(max=V - 1)
    return {"path": path[:, :S].contiguous(), "path_lens": count.to(torch.int32),
            "next_token": torch.where(new > 0, token, -1).to(torch.int32)}


def _plain_accept(st):
    S = st["case"]["S"]
    dev = st["path"].device
    past = (st["total"] - st["new"]).long()
    i, bi = torch.arange(S, device=dev), torch.arange(st["case"]["B"], device=dev)[:, None]
    keep = i < st["path_lens"].long()[:, None]
    # (positions behind the path write the root's row to itself)
    src = past[:, None] + torch.where(keep, st["path"].long(), torch.zeros_like(i))
    dst = past[:, None] + torch.where(keep, i, torch.zeros_like(i))
    st["keys"][:, bi, :, dst] = st["keys"][:, bi, :, src]
    st["values"][:, bi, :, dst] = st["values"][:, bi, :, src]
    return {"seqlens_k": (past + st["path_lens"] - 1).to(torch.int32), "keys": st["keys"], "values": st["values"]}


# ------------------------------------------------------------------------------------------------ the pass

def run(st):
    case = st["case"]
    ragged = st["new"] if case["ragged"] else None
    if not own:
        return {"tree": _plain_tree, "verify": _plain_verify, "accept": _plain_accept}[case["op"]](st)
    gqa = st["gqa"]
    if case["op"] == "tree":
        out = gqa.tree_forward(st["query"], st["key"], st["value"], st["parents"], st["seqlens_k"], st["T"],
                               st["present_key"], st["present_value"], new_lens=ragged, head_sink=st["sink"])
        return {"output": out, "present_key": st["present_key"], "present_value": st["present_value"]}
    if case["op"] == "verify":
        path, lens, token = gqa.tree_verify(st["tokens"], st["parents"], st["target_probs"], st["accept_uniforms"],
                                            st["sample_uniforms"], draft_probs=st["draft_probs"], new_lens=ragged)
        return {"path": path, "path_lens": lens, "next_token": token}
    seqlens = gqa.tree_accept(st["caches"], st["path"], st["path_lens"], st["seqlens_k"], new_lens=ragged)
    return {"seqlens_k": seqlens, "keys": st["keys"], "values": st["values"]}


def _lengths(case):
    B, lo, hi = case["B"], case["lo"], case["hi"]
    new = _counts(case)
    return [hi] if B == 1 else [max(lo + round((hi - lo) * b / (B - 1)), new[b]) for b in range(B)]


def work(case):
    esize = 2 if case["dtype"] == "f16" else 4
    B, S = case["B"], case["S"]
    new = _counts(case)
    if case["op"] == "verify":
        # one row of each sequence's probabilities, to draw from
        rows = 2 if case["drafts"] else 1
        return {"bytes": B * (rows * case["V"] * esize + 16 * S + 12), "flops": B * rows * case["V"]}
    if case["op"] == "accept":
        # half the nodes on average, read and written
        rows = sum((1 + n) / 2 for n in new)
        return {"bytes": case["L"] * rows * 4 * case["Nkv"] * case["H"] * esize + 12 * B * S, "flops": 0}
    N, Nkv, H, W = (case[k] for k in ("N", "Nkv", "H", "window"))
    byts = flops = 0
    for t, n in zip(_lengths(case), new):
        seen = t - n if W < 0 else min(t - n, W)
        byts += (seen + 2 * n) * 2 * Nkv * H * esize + 2 * n * N * H * esize + (S - n) * N * H * esize
        flops += 4.0 * N * H * n * (seen + (n if case["shape"] == "chain" else math.log2(n + 1)) / 2)
    return {"bytes": byts, "flops": flops}


# ------------------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"tree": _exact_tree, "verify": _exact_verify, "accept": _exact_accept}[case["op"]](case, st)


def _exact_tree(case, st):
    B, S, N, Nkv, H, W = (case[k] for k in ("B", "S", "N", "Nkv", "H", "window"))
    G = N // Nkv
    out = torch.zeros((B, S, Nkv, G, H), dtype=torch.float64, device="cuda")
    keys, values = st["present_key"].clone(), st["present_value"].clone()
    par, total, new = (st[k].cpu().tolist() for k in ("parents", "total", "new"))
    for b in range(B):
        t, n = total[b], new[b]
        past = t - n
        see = torch.zeros((n, t), dtype=torch.bool)
        level = []
        for i in range(n):
            level.append(0 if par[b][i] < 0 else level[par[b][i]] + 1)
            see[i, max(0, past + level[i] - W) if W >= 0 else 0:past] = True
            a = i
            while a >= 0:
                see[i, past + a] = W < 0 or level[i] - level[a] <= W
                a = par[b][a]
        hide = ~see.cuda()
        for g in range(Nkv):
            keys[b, g, past:t] = st["key"][b, :n].view(n, Nkv, H)[:, g]
            values[b, g, past:t] = st["value"][b, :n].view(n, Nkv, H)[:, g]
            k, v = keys[b, g, :t].double(), values[b, g, :t].double()
            for h in range(G):
                s = st["query"][b, :n].view(n, N, H)[:, g * G + h].double() @ k.T / math.sqrt(H)
                if case["softcap"] > 0:
                    s = case["softcap"] * torch.tanh(s / case["softcap"])
                s[hide] = -math.inf
                if st["sink"] is not None:
                    s = torch.cat((s, st["sink"][g * G + h].double().expand(n, 1)), dim=1)
                out[b, :n, g, h] = torch.softmax(s, dim=1)[:, :t] @ v
    return {"output": out.view(B, S, N * H), "present_key": keys.double(), "present_value": values.double()}


def _exact_verify(case, st):
    import numpy as np
    B, S = case["B"], case["S"]
    par, tok, new, u, us = (st[k].cpu().numpy() for k in ("parents", "tokens", "new", "accept_uniforms", "sample_uniforms"))
    path, lens, token = np.full((B, S), -1), np.zeros(B, int), np.zeros(B, int)
    for b in range(B):
        node, taken = 0, [0]
        while True:
            p = st["target_probs"][b, node].cpu().numpy().astype(np.float64)
            q = None if st["draft_probs"] is None else st["draft_probs"][b, node].cpu().numpy().astype(np.float64)
            rest, norm, follow = p, 1.0, None
            for c in np.flatnonzero(par[b, :new[b]] == node):
                x = tok[b, c]
                if np.float64(u[b, c]) * (1.0 if q is None else q[x]) * norm < rest[x]:
                    follow = int(c)
                    break
                if q is None:
                    rest = rest.copy()
                    rest[x] = 0.0
                else:
                    rest = np.maximum(rest / (norm if norm > 0 else 1.0) - q, 0.0)
                norm = rest.sum()
            if follow is None:
                break
            node = follow
            taken.append(node)
        rest = rest if rest.sum() > 0 else p
        cum = np.cumsum(rest)
        token[b] = min(np.searchsorted(cum, np.float64(us[b]) * cum[-1], side="right"), case["V"] - 1)
        path[b, :len(taken)], lens[b] = taken, len(taken)
    return {"path": path.astype(np.int32), "path_lens": lens.astype(np.int32), "next_token": token.astype(np.int32)}


def _exact_accept(case, st):
    keys, values = st["keys"].double(), st["values"].double()
    path, lens, total, new = (st[k].cpu().tolist() for k in ("path", "path_lens", "total", "new"))
    for b in range(case["B"]):
        past = total[b] - new[b]
        for i in range(lens[b]):   # rows only move forward, past rows that are read later
            keys[:, b, :, past + i] = keys[:, b, :, past + path[b][i]]
            values[:, b, :, past + i] = values[:, b, :, past + path[b][i]]
    seqlens = torch.tensor([t - n + k - 1 for t, n, k in zip(total, new, lens)], dtype=torch.int32)
    return {"seqlens_k": seqlens, "keys": keys, "values": values}
