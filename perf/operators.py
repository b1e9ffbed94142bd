"""Operators on a paged KV cache that grows by drafted trees and shrinks by eviction.

Four operators: attention of a tree of drafted tokens over the cache (``tree_attend``), the move of
the accepted path's rows to consecutive positions (``tree_commit``), decode attention that adds each
position's attention weight to a running sum (``dense_decode`` / ``indexed_attend`` with ``mass``),
and eviction by that sum (``evict``). ``run`` computes them in plain torch operations, or, where
``own`` is true, by the calls that a user makes of the library.

A case names the operator (``op``) and its sizes; lengths, page tables and padded nodes follow from
the case, everything else from the seed.
"""

import math
import random

import torch

own = False

DEV = "cuda"
NONE = -2  # parent of an unused node


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------


def _tree(name, batch, length, n, h_q=32, h_kv=8, d=128, page=16, window=-1, budget=0, store=False):
    return {"name": name, "op": "tree", "batch": batch, "length": length, "n": n, "h_q": h_q,
            "h_kv": h_kv, "d": d, "page": page, "window": window, "budget": budget, "store": store}


def _commit(name, batch, length, n, accepted, h_kv=8, d=128, page=16, rank=32):
    return {"name": name, "op": "commit", "batch": batch, "length": length, "n": n,
            "accepted": accepted, "h_kv": h_kv, "d": d, "page": page, "rank": rank}


def _mass(name, batch, length, budget=0, h_q=32, h_kv=8, d=128, page=16, window=-1):
    return {"name": name, "op": "mass", "batch": batch, "length": length, "budget": budget,
            "h_q": h_q, "h_kv": h_kv, "d": d, "page": page, "window": window}


def _evict(name, batch, length, keep, recent, h_kv=8, d=128, page=16, rank=32):
    return {"name": name, "op": "evict", "batch": batch, "length": length, "keep": keep,
            "recent": recent, "h_kv": h_kv, "d": d, "page": page, "rank": rank}


def listed():
    return [
        # one user, a short chain of drafts on a short chat: latency
        _tree("tree_b1_short", 1, 701, 5, store=True),
        # a small batch of chats, a medium tree, ragged lengths, the nodes' rows stored by the call
        _tree("tree_b8_8k", 8, 8190, 26, store=True),
        # long contexts with the widest tree: as much arithmetic per byte as the path gets
        _tree("tree_b16_32k", 16, 32768, 64),
        # a sliding-window layer of the hybrid stack (head dim 256)
        _tree("tree_b8_window", 8, 16001, 31, h_q=16, d=256, window=1024),
        # a sparse layer: the context is the selected positions of a 64K cache
        _tree("tree_b16_indexed", 16, 65536, 16, budget=2048),
        # the accepted path of one user's tree
        _commit("commit_b1", 1, 701, 8, 3),
        # the accepted paths of a large batch of wide trees
        _commit("commit_b64", 64, 2047, 64, 9),
        # the weights of one short sequence's step: latency
        _mass("mass_b1_2k", 1, 1999),
        # the weights over long contexts
        _mass("mass_b16_32k", 16, 32768),
        # a sparse layer's step: the weights of its selected positions
        _mass("mass_b16_indexed", 16, 65536, budget=2048),
        # one sequence cut to its budget
        _evict("evict_b1_4k", 1, 4127, 2048, 64),
        # a batch of long contexts cut to a quarter
        _evict("evict_b16_64k", 16, 65536, 16384, 256),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "commit", "mass", "mass", "evict"])
    d = rng.choice([128, 128, 256])
    page = rng.choice([16, 16, 32, 64])
    h_kv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 8])
    batch = _log_int(rng, 1, 16)
    # (batch * length * h_kv * d up to the largest listed case of the operator)
    cap = 16 * 32768 * 8 * 128 // (batch * h_kv * d)
    length = _log_int(rng, 64, min(cap, 65536))
    if op == "tree":
        n = _log_int(rng, 1, 64)
        if n * g > 256:
            n = 256 // g
        kind = rng.choice(["full", "full", "window", "indexed"])
        window = _log_int(rng, 16, length) if kind == "window" else -1
        budget = _log_int(rng, 16, min(length, 4096)) if kind == "indexed" else 0
        return _tree("", batch, length, n, g * h_kv, h_kv, d, page, window, budget,
                     rng.random() < 0.3 and length <= 8192)
    if op == "commit":
        n = _log_int(rng, 1, 64)
        return _commit("", _log_int(rng, 1, 64), min(length, 2048), n, rng.randint(1, min(n, 16)),
                       h_kv, d, page, 64 if d == 256 else rng.choice([16, 32, 64]))
    if op == "mass":
        kind = rng.choice(["full", "indexed", "window"])
        window = _log_int(rng, 16, length) if kind == "window" else -1
        budget = _log_int(rng, 16, min(length, 4096)) if kind == "indexed" else 0
        return _mass("", batch, length, budget, g * h_kv, h_kv, d, page, window)
    keep = _log_int(rng, 16, min(length, 16384))
    return _evict("", batch, length, keep, rng.randint(0, keep // 2), h_kv, d, page,
                  64 if d == 256 else rng.choice([16, 32, 64]))


def _lens(case):
    """Committed lengths: the first sequence has the full length, the others down to half of it."""
    L = case["length"]
    return [L - (b * 7919) % (L // 2 + 1) for b in range(case["batch"])]


def _accepted(case):
    return [1 + (case["accepted"] - 1 + 5 * b) % case["accepted"] for b in range(case["batch"])]


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, *shape):
    """bf16 values of a standard normal distribution."""
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    return x.normal_(generator=g)


def _pages(case, g, extra, copies=1):
    """Scattered page tables: every sequence's pages are a random part of one pool."""
    per = -(-(case["length"] + extra) // case["page"])
    total = case["batch"] * per * copies + 3
    perm = torch.randperm(total, generator=g, device=DEV, dtype=torch.int64)
    bt = perm[:case["batch"] * per].to(torch.int32).view(case["batch"], per).contiguous()
    return bt, total, perm


def prepare(case, seed):
    g = _gen(seed)
    B, Hk, D, ps = case["batch"], case["h_kv"], case["d"], case["page"]
    lens = _lens(case)
    s = {"case": case, "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    op = case["op"]
    extra = case["n"] if op in ("tree", "commit") else 0
    bt, total, perm = _pages(case, g, extra, 2 if op == "evict" else 1)
    s["block_table"] = bt
    s["k"] = _normal(g, total, ps, Hk, D)
    s["v"] = _normal(g, total, ps, Hk, D)
    if op in ("tree", "mass"):
        n = case["n"] if op == "tree" else 1
        # queries with a spread of logits of a few units, as trained heads have
        q = _normal(g, B, n, case["h_q"], D) * 2
        s["q"] = q if op == "tree" else q[:, 0].contiguous()
        if case["budget"]:
            # ascending positions, one of each cell of the context (a selection's positions)
            bud = case["budget"]
            cells = torch.tensor([[max(1, L // bud)] for L in lens], device=DEV)
            have = torch.tensor([[min(bud, L)] for L in lens], device=DEV)
            i = torch.arange(bud, device=DEV)[None, None]
            u = torch.rand((B, Hk, bud), generator=g, device=DEV, dtype=torch.float64)
            pos = i * cells[:, :, None] + (u * cells[:, :, None]).long()
            s["idx"] = torch.where(i < have[:, :, None], pos, -1).to(torch.int32).contiguous()
            s["count"] = have.expand(B, Hk).to(torch.int32).contiguous()
    if op == "tree":
        n = case["n"]
        i = torch.arange(n, device=DEV)[None]
        back = (torch.rand((B, n), generator=g, device=DEV) ** 2 * 6).long() + 1
        par = torch.clamp(i - back, min=-1)
        size = torch.tensor([[n - (b % 3 if n > 4 else 0)] for b in range(B)], device=DEV)
        s["parents"] = torch.where(i < size, par, NONE).to(torch.int32).contiguous()
        if case["store"]:
            s["k_new"] = _normal(g, B, n, Hk, D)
            s["v_new"] = _normal(g, B, n, Hk, D)
    if op == "mass":
        # the sums of a few earlier steps, of the size of one step's weights
        s["mass"] = torch.rand((B, Hk, bt.shape[1] * ps), generator=g, device=DEV)
        s["mass"] *= 2.0 * case["h_q"] / Hk / (case["budget"] or case["length"])
    if op in ("commit", "evict"):
        r = case["rank"]
        s["codes"] = torch.randint(0, 120, (total, Hk, ps, r), generator=g, device=DEV,
                                   dtype=torch.uint8)
    if op == "commit":
        n, m = case["n"], case["accepted"]
        have = torch.tensor(_accepted(case), dtype=torch.int32, device=DEV)
        order = torch.rand((B, n), generator=g, device=DEV).argsort(1)[:, :m].sort(1).values
        i = torch.arange(m, device=DEV)[None]
        # the first have[b] of a random ascending choice of nodes
        s["path"] = torch.where(i < have[:, None], order, -1).to(torch.int32).contiguous()
        s["n_path"] = have
    if op == "evict":
        # heavy-tailed sums: a few positions hold most of the weight
        u = torch.rand((B, Hk, bt.shape[1] * ps), generator=g, device=DEV)
        s["mass"] = 1e-3 / (u + 1e-6)
        per = -(-case["keep"] // ps)
        used = B * bt.shape[1]
        s["dst"] = perm[used:used + B * per].to(torch.int32).view(B, per).contiguous()
        s["mass_out"] = torch.zeros_like(s["mass"])
    return s


# ------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------


def _rows(cache, table, pos):
    """Rows ``[B, H, P, D]`` of logical positions ``pos`` ``[B, H, P]`` (long, in range)."""
    ps = cache.shape[1]
    b = torch.arange(pos.shape[0], device=DEV)[:, None, None]
    h = torch.arange(pos.shape[1], device=DEV)[None, :, None]
    return cache[table[b, pos // ps].long(), pos % ps, h]


def _ancestors(par):
    """visible[b, i, j]: node j is node i or one of its ancestors (unused nodes: nothing), by
    squaring the one-step relation."""
    B, n = par.shape
    used = par > NONE
    eye = torch.eye(n, dtype=torch.bool, device=DEV)[None] & used[:, :, None]
    step = (par[:, :, None] == torch.arange(n, device=DEV)[None, None]) | eye
    reach = step.float()
    # (log2 64 squarings reach every ancestor)
    reach = ((reach @ reach) > 0).float()
    reach = ((reach @ reach) > 0).float()
    reach = ((reach @ reach) > 0).float()
    reach = ((reach @ reach) > 0).float()
    reach = ((reach @ reach) > 0).float()
    reach = ((reach @ reach) > 0).float()
    return (reach > 0) & used[:, :, None]


def _plain_tree(s):
    c = s["case"]
    k, v, bt, q, par = s["k"], s["v"], s["block_table"], s["q"], s["parents"].long()
    B, n, Hq, D = q.shape
    H, ps = c["h_kv"], c["page"]
    G = Hq // H
    L = s["seq_lens"].long()
    b = torch.arange(B, device=DEV)[:, None]
    node_pos = L[:, None] + torch.arange(n, device=DEV)[None]
    used = par > NONE
    if "k_new" in s:
        page, slot = bt[b, node_pos // ps].long(), node_pos % ps
        k[page[used], slot[used]] = s["k_new"][used]
        v[page[used], slot[used]] = s["v_new"][used]
    vis = _ancestors(par)
    depth = vis.sum(2) - 1
    if c["budget"]:
        pos = s["idx"].long().clamp(min=0)
        ok = (torch.arange(c["budget"], device=DEV)[None, None] < s["count"][:, :, None])
        ok = ok[:, :, None, :].expand(B, H, n, -1)
    else:
        pos = torch.arange(int(c["length"]), device=DEV)[None, None].expand(B, H, -1)
        lo = L[:, None] + depth - c["window"] + 1 if c["window"] > 0 else torch.zeros_like(depth)
        ok = (pos[:, :, None, :] < L[:, None, None, None]) & (pos[:, :, None, :] >= lo[:, None, :, None])
    tree = vis[:, None].expand(B, H, n, n)
    if c["window"] > 0:
        tree = tree & (depth[:, None, None, :] > depth[:, None, :, None] - c["window"])
    every = torch.cat([pos, node_pos[:, None].expand(B, H, n)], 2)
    ok = torch.cat([ok & used[:, None, :, None], tree], 3)
    qf = q.float().view(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    x = (qf @ _rows(k, bt, every).float().transpose(2, 3)).view(B, H, n, G, -1) / math.sqrt(D)
    x = torch.where(ok[:, :, :, None, :], x, -math.inf)
    top = x.amax(4, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(4, keepdim=True)
    o = p.view(B, H, n * G, -1) @ _rows(v, bt, every).float()
    o = o.view(B, H, n, G, D) / torch.where(total > 0, total, 1.0)
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D).to(torch.bfloat16)


def _plain_commit(s):
    k, v, sc, bt = s["k"], s["v"], s["codes"], s["block_table"]
    ps = k.shape[1]
    path, L = s["path"].long(), s["seq_lens"].long()
    b, i = torch.nonzero(torch.arange(path.shape[1], device=DEV)[None] < s["n_path"][:, None],
                         as_tuple=True)
    src, dst = L[b] + path[b, i], L[b] + i
    sp, ss, dp, ds = bt[b, src // ps].long(), src % ps, bt[b, dst // ps].long(), dst % ps
    k[dp, ds] = k[sp, ss]
    v[dp, ds] = v[sp, ss]
    sc[dp, :, ds] = sc[sp, :, ss]
    return s["seq_lens"] + s["n_path"]


def _plain_mass(s):
    c = s["case"]
    q, L = s["q"], s["seq_lens"].long()
    B, Hq, D = q.shape
    H = c["h_kv"]
    if c["budget"]:
        pos = s["idx"].long().clamp(min=0)
        ok = torch.arange(c["budget"], device=DEV)[None, None] < s["count"][:, :, None]
    else:
        pos = torch.arange(int(c["length"]), device=DEV)[None, None].expand(B, H, -1)
        ok = pos < L[:, None, None]
        if c["window"] > 0:
            ok = ok & (pos >= L[:, None, None] - c["window"])
    x = q.float().view(B, H, Hq // H, D) @ _rows(s["k"], s["block_table"], pos).float().transpose(2, 3)
    x = torch.where(ok[:, :, None], x / math.sqrt(D), -math.inf)
    p = torch.exp(x - x.amax(3, keepdim=True))
    p = p / p.sum(3, keepdim=True)
    o = p @ _rows(s["v"], s["block_table"], pos).float()
    w = torch.where(ok, p.sum(2), 0.0)
    s["mass"].scatter_add_(2, pos, w)
    return o.reshape(B, Hq, D).to(torch.bfloat16)


def _plain_evict(s):
    c = s["case"]
    k, v, sc, m = s["k"], s["v"], s["codes"], s["mass"]
    B, H, cap = m.shape
    ps, keep = k.shape[1], c["keep"]
    L = s["seq_lens"].long()[:, None, None]
    at = torch.arange(cap, device=DEV)[None, None].expand(B, H, -1)
    # the last `recent` positions come first, then the sums in descending order (stable: ties to
    # the lower position), then what lies behind the sequence
    key = torch.where(at >= L - c["recent"], math.inf, m)
    key = torch.where(at < L, key, -math.inf)
    best = torch.sort(key, dim=2, descending=True, stable=True).indices[:, :, :keep]
    best = torch.where(best < L, best, cap).sort(2).values
    if best.shape[2] < keep:
        best = torch.cat([best, torch.full((B, H, keep - best.shape[2]), cap, device=DEV)], 2)
    ok = best < cap
    idx = torch.where(ok, best, -1).to(torch.int32)
    count = ok.sum(2).to(torch.int32)
    b, h, i = torch.nonzero(ok, as_tuple=True)
    src = best[b, h, i]
    sp, ss = s["block_table"][b, src // ps].long(), src % ps
    dp, ds = s["dst"][b, i // ps].long(), i % ps
    k[dp, ds, h] = k[sp, ss, h]
    v[dp, ds, h] = v[sp, ss, h]
    sc[dp, h, ds] = sc[sp, h, ss]
    out = torch.where(at < L, 0.0, s["mass_out"])
    out[b, h, i] = m[b, h, src]
    s["mass_out"].copy_(out)
    return idx, count, torch.clamp(s["seq_lens"], max=keep)


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import token_level_sparse_fp8_b200 as J
    if op == "tree":
        if own:
            o = J.tree_attend(s["q"], s["k"], s["v"], s["block_table"], s["seq_lens"], s["parents"],
                              k_new=s.get("k_new"), v_new=s.get("v_new"), idx=s.get("idx"),
                              count=s.get("count"), window=c["window"])
        else:
            o = _plain_tree(s)
        return [o, s["k"], s["v"]] if c["store"] else [o]
    if op == "commit":
        if own:
            lens = J.tree_commit(s["k"], s["v"], s["block_table"], s["seq_lens"], s["path"],
                                 s["n_path"], score_cache=s["codes"])
        else:
            lens = _plain_commit(s)
        return [lens, s["k"], s["v"], s["codes"]]
    if op == "mass":
        if not own:
            o = _plain_mass(s)
        elif c["budget"]:
            o = J.indexed_attend(s["q"], s["k"], s["v"], s["block_table"], s["idx"], s["count"],
                                 mass=s["mass"])
        else:
            o = J.dense_decode(s["q"], s["k"], s["v"], s["block_table"], s["seq_lens"],
                               window=c["window"], mass=s["mass"])
        return [o, s["mass"]]
    if own:
        idx, count, lens = J.evict(s["mass"], s["k"], s["v"], s["block_table"], s["seq_lens"],
                                   c["keep"], recent=c["recent"], score_cache=s["codes"],
                                   dst_block_table=s["dst"], mass_out=s["mass_out"])
    else:
        idx, count, lens = _plain_evict(s)
    return [idx, count, lens, s["k"], s["v"], s["codes"], s["mass_out"]]


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------


def work(case):
    lens, B, H, D = _lens(case), case["batch"], case["h_kv"], case["d"]
    row = 4 * D  # bytes of one K row and one V row
    op = case["op"]
    if op in ("tree", "mass"):
        n = case["n"] if op == "tree" else 1
        w = case["window"]
        extra = n if op == "tree" else 0
        ctx = [min(L, case["budget"]) if case["budget"] else min(L, w) if w > 0 else L for L in lens]
        q = B * n * case["h_q"] * D
        rows = H * sum(c + extra for c in ctx)
        b = rows * row + 2 * 2 * q
        if op == "tree":
            b += 4 * B * n + (B * n * H * row if case["store"] else 0)
            # (stored nodes are read from the new rows, once, and written once)
        else:
            b += rows * 8
        if case["budget"]:
            b += 4 * H * sum(ctx)
        return {"bytes": b, "flops": 4 * n * case["h_q"] * D * sum(c + extra for c in ctx)}
    if op == "commit":
        moved = H * sum(_accepted(case))
        return {"bytes": 2 * moved * (row + case["rank"]) + 4 * sum(_accepted(case)), "flops": 0}
    kept = H * sum(min(L, case["keep"]) for L in lens)
    return {"bytes": 4 * H * sum(lens) + 2 * kept * (row + case["rank"]) + 4 * kept
            + 4 * B * H * case["keep"] + 4 * H * sum(lens), "flops": 0}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------


def _gather64(cache, table, b, h, pos):
    ps = cache.shape[1]
    return cache[table[b].long()[pos // ps], pos % ps, h].double()


def exact(case, seed):
    s = prepare(case, seed)
    op, H, D, ps = case["op"], case["h_kv"], case["d"], case["page"]
    lens, bt = _lens(case), s["block_table"]
    B = case["batch"]
    if op == "tree":
        n, G, w = case["n"], case["h_q"] // H, case["window"]
        par = s["parents"].tolist()
        o = torch.zeros((B, n, case["h_q"], D), dtype=torch.float64, device=DEV)
        for b in range(B):
            L = lens[b]
            anc, dep = [], []
            for i, p in enumerate(par[b]):
                if p == NONE:
                    anc.append([])
                    dep.append(0)
                else:
                    anc.append((anc[p] if p >= 0 else []) + [i])
                    dep.append(dep[p] + 1 if p >= 0 else 0)
                if p != NONE and case["store"]:
                    page, slot = int(bt[b, (L + i) // ps]), (L + i) % ps
                    s["k"][page, slot] = s["k_new"][b, i]
                    s["v"][page, slot] = s["v_new"][b, i]
            for h in range(H):
                lo = max(0, L - w) if w > 0 else 0
                if case["budget"]:
                    ctx = s["idx"][b, h, :int(s["count"][b, h])].long()
                else:
                    ctx = torch.arange(lo, L, device=DEV)
                every = torch.cat([ctx, L + torch.arange(n, device=DEV)])
                see = torch.zeros((n, len(every)), dtype=torch.bool)
                c = len(ctx)
                for i in range(n):
                    if not anc[i]:
                        continue
                    # (a window w: the w positions up to the node's own, L + its depth)
                    first = max(lo, L + dep[i] - w + 1) if w > 0 else lo
                    see[i, first - lo:c] = True
                    for a in anc[i]:
                        see[i, c + a] = w <= 0 or dep[i] - dep[a] < w
                see = see.to(DEV)
                qh = s["q"][b, :, h * G:(h + 1) * G].double()
                x = torch.einsum("ngd,td->ngt", qh, _gather64(s["k"], bt, b, h, every)) * D ** -0.5
                x = x.masked_fill(~see[:, None], -math.inf)
                some = see.any(1)
                p = torch.softmax(x[some], 2)
                o[b, some, h * G:(h + 1) * G] = torch.einsum(
                    "ngt,td->ngd", p, _gather64(s["v"], bt, b, h, every))
        return [o, s["k"], s["v"]] if case["store"] else [o]
    if op == "commit":
        acc, path = _accepted(case), s["path"].tolist()
        k0, v0, c0 = s["k"].clone(), s["v"].clone(), s["codes"].clone()
        tab = bt.tolist()
        for b in range(B):
            for i in range(acc[b]):
                src, dst = lens[b] + path[b][i], lens[b] + i
                a, z = (tab[b][src // ps], src % ps), (tab[b][dst // ps], dst % ps)
                s["k"][z] = k0[a]
                s["v"][z] = v0[a]
                s["codes"][z[0], :, z[1]] = c0[a[0], :, a[1]]
        return [torch.tensor([x + y for x, y in zip(lens, acc)], dtype=torch.int32), s["k"], s["v"],
                s["codes"]]
    if op == "mass":
        G = case["h_q"] // H
        o = torch.zeros((B, case["h_q"], D), dtype=torch.float64, device=DEV)
        m = s["mass"].double()
        for b in range(B):
            for h in range(H):
                if case["budget"]:
                    pos = s["idx"][b, h, :int(s["count"][b, h])].long()
                else:
                    lo = max(0, lens[b] - case["window"]) if case["window"] > 0 else 0
                    pos = torch.arange(lo, lens[b], device=DEV)
                x = s["q"][b, h * G:(h + 1) * G].double() @ _gather64(s["k"], bt, b, h, pos).T
                p = torch.softmax(x * D ** -0.5, 1)
                o[b, h * G:(h + 1) * G] = p @ _gather64(s["v"], bt, b, h, pos)
                m[b, h, pos] += p.sum(0)
        return [o, m]
    keep, recent = case["keep"], case["recent"]
    idx = torch.full((B, H, keep), -1, dtype=torch.int32, device=DEV)
    for b in range(B):
        L = lens[b]
        n = min(L, keep)
        for h in range(H):
            if L <= keep:
                pos = torch.arange(L, device=DEV)
            else:
                m = s["mass"][b, h, :L - recent].double()
                want = keep - recent
                edge = torch.sort(m).values[len(m) - want] if want else math.inf
                above = m > edge
                tied = torch.nonzero(m == edge)[:want - int(above.sum()), 0]
                above[tied] = True
                pos = torch.cat([torch.nonzero(above)[:, 0], torch.arange(L - recent, L, device=DEV)])
            idx[b, h, :n] = pos.to(torch.int32)
            i = torch.arange(n, device=DEV)
            sp, dp = bt[b].long()[pos // ps], s["dst"][b].long()[i // ps]
            s["k"][dp, i % ps, h] = s["k"][sp, pos % ps, h]
            s["v"][dp, i % ps, h] = s["v"][sp, pos % ps, h]
            s["codes"][dp, h, i % ps] = s["codes"][sp, h, pos % ps]
            s["mass_out"][b, h, :L] = 0
            s["mass_out"][b, h, :n] = s["mass"][b, h, pos]
    count = torch.tensor([[min(L, keep)] * H for L in lens], dtype=torch.int32)
    return [idx, count, torch.tensor([min(L, keep) for L in lens], dtype=torch.int32), s["k"], s["v"],
            s["codes"], s["mass_out"].double()]
