"""Cache operators at the edges of their range: precision, odd states of the layer, bad pages, sizes
that take the rarer branches of the kernels. Float64 references as in test_gpu_cache_ops.py.

Tolerances, fixed before the first run. With A = sum_t p_t |v_t| from the oracle and T visible
positions: weights as two bf16 parts are off by at most 2^-14 of themselves, fp32 scores by
X / 2 = d 2^-23 scale max_t sum_i |q_i k_ti| + 2^-20 as a factor on each weight and on their sum, the
sums over T positions (two products each, and the sum of weights) by 3 T 2^-23 A, the bf16 output by
half a step (2^-8 of its value).
"""

import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from test_gpu_cache_ops import (NAN, Paged, _built, _clean_flags, cuda, f64, jssa,  # noqa: F401
                                random_tree)

pytestmark = pytest.mark.gpu


def weight_slack(q, k, scale, positions):
    """Factor on A from scores, split weights and sums; ``q`` [..., d], ``k`` [..., d], NaN left out."""
    d = q.shape[-1]
    k = np.abs(np.where(np.isfinite(k), k, 0)).reshape(-1, d)
    top = float((np.abs(q).reshape(-1, d) @ k.T).max())
    return 2.0 ** -14 + 2 * (d * 2.0 ** -23 * abs(scale) * top + 2.0 ** -20) + 3 * positions * 2.0 ** -23


def check_close(got, ref, mag, slack):
    assert np.isfinite(got).all()
    tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * slack * mag
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) - tol))


# ------------------------------------------------------------------------------------------------
# tree attention
# ------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("n,g,d", [(7, 4, 128), (40, 4, 128), (9, 4, 256), (64, 2, 256)])
def test_tree_attend_weights_are_not_rounded_once(n, g, d):
    # the weights keep more than a bf16's digits, as in the decode kernels: outputs near zero show it
    J = jssa()
    c = Paged([230, 64], n, 1, d, seed=50 + n)
    q, kn, vn = c.normal(2, n, g, d), c.normal(2, n, 1, d), c.normal(2, n, 1, d)
    parents = [random_tree(c.rng, n, b) for b in range(2)]
    scale = 1 / math.sqrt(d)
    out = J.tree_attend(q.cuda(), c.k, c.v, c.bt, c.seq_lens, cuda(parents), kn.cuda(), vn.cuda())
    ref, mag = C.tree_attend(f64(q), f64(c.k), f64(c.v), c.table, c.lens, parents, scale)
    check_close(f64(out), ref, mag, weight_slack(f64(q), f64(c.k), scale, 230 + n))
    assert J.device_error() == 0


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n", [6, 64])
def test_tree_attend_visible_infinities(n, d):
    # an infinite value that every row sees reaches that element of every row, and no other
    J = jssa()
    c = Paged([200], n, 1, d, seed=60 + n)
    q, kn, vn = c.normal(1, n, 4, d), c.normal(1, n, 1, d), c.normal(1, n, 1, d)
    parents = cuda([random_tree(c.rng, n)])
    for t, e, x in ((3, 5, math.inf), (90, 7, -math.inf)):
        c.v[c.table[0, t // 16], t % 16, 0, e] = x
    out = J.tree_attend(q.cuda(), c.k, c.v, c.bt, c.seq_lens, parents, kn.cuda(), vn.cuda())[0].float()
    assert bool((out[..., 5] == math.inf).all()) and bool((out[..., 7] == -math.inf).all())
    out[..., 5] = out[..., 7] = 0.0
    assert bool(torch.isfinite(out).all())


# ------------------------------------------------------------------------------------------------
# the layer
# ------------------------------------------------------------------------------------------------


def make_layer(lens, h_kv=2, d=128, r=32, budget=64, extra=80, seed=70, track_mass=True):
    J = jssa()
    c = Paged(lens, extra, h_kv, d, seed=seed)
    c.k.nan_to_num_(0.0), c.v.nan_to_num_(0.0)
    m = torch.linalg.qr(torch.randn((h_kv, d, r), generator=torch.Generator().manual_seed(seed)))[0]
    layer = J.PagedLayer(c.k, c.v, c.bt, c.seq_lens, m.transpose(1, 2).contiguous().cuda(), budget,
                         track_mass=track_mass)
    layer.prefill_scores()
    return c, layer


def test_captured_calls_of_every_size_keep_their_memory():
    # graphs of calls whose workspaces grow from one to the next; what is allocated afterwards must not
    # share memory with any of them
    c, layer = make_layer([900, 333], extra=80)
    g, nodes = 4, (8, 64)
    q = {n: c.normal(2, n, 2 * g, 128).cuda() for n in nodes}
    kn, vn = ({n: c.normal(2, n, 2, 128).cuda() for n in nodes} for _ in range(2))
    par = {n: cuda([random_tree(c.rng, n) for _ in range(2)]) for n in nodes}
    q1 = q[8][:, 0].contiguous()
    calls = [lambda: layer.step(q1)[0].clone(), lambda: layer.dense(q1, window=64),
             lambda: layer.dense(q1)]
    for n in nodes:
        for sparse in (False, True):
            calls.append(lambda n=n, sparse=sparse: layer.draft(q[n], kn[n], vn[n], par[n], sparse=sparse))
    k0, v0, codes = c.k.clone(), c.v.clone(), layer.score_cache.clone()

    def reset():
        c.k.copy_(k0), c.v.copy_(v0), layer.score_cache.copy_(codes), layer.mass.zero_()

    want = []
    for f in calls:
        reset()
        want.append((f().clone(), layer.mass.clone()))
    graphs, outs = [], []
    for f in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(f())
        graphs.append(graph)
    for f in calls:
        reset()
        f()
    torch.cuda.synchronize()
    patterns = [torch.full((1 << k,), 90 + k, dtype=torch.uint8, device="cuda")
                for k in range(12, 25) for _ in range(3)]
    for graph, out, (ref, mass) in zip(graphs, outs, want):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(layer.mass, mass)
    for i, p in enumerate(patterns):
        assert bool((p == 90 + 12 + i // 3).all())
    assert jssa().device_error() & ~16 == 0


@pytest.mark.parametrize("sparse", [False, True])
def test_draft_with_lengths_outside_the_table(sparse):
    # a negative length counts as 0, one past the table as the table's: flagged, and the layer lives on
    J = jssa()
    c, layer = make_layer([40, 25], extra=80, seed=71)
    cap = c.table.shape[1] * 16
    q, kn, vn = c.normal(2, 5, 8, 128), c.normal(2, 5, 2, 128), c.normal(2, 5, 2, 128)
    par = [random_tree(c.rng, 5) for _ in range(2)]
    want = None
    for bad, as_if, flag in ((-40, 0, 4), (0, 0, 0), (10 ** 6, cap, 4 | 2), (cap, cap, 2)):
        layer.seq_lens.copy_(cuda([bad, 25]))
        out = layer.draft(q.cuda(), kn.cuda(), vn.cuda(), cuda(par), sparse=sparse)
        assert J.device_error() & ~16 == flag
        # the stored rows and codes, and the output, are those of the length it counts as
        got = [out, c.k.clone(), c.v.clone(), layer.score_cache.clone()]
        if bad != as_if:
            want = got
        else:
            assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert layer.seq_lens.tolist() == [cap, 25]


@pytest.mark.parametrize("sparse", [False, True])
def test_draft_leaves_dropped_nodes_out(sparse):
    # a node that names itself, a later or an unused one takes no part, nor do the nodes below it: no
    # rows, no codes, no share in the query that selects the context
    J = jssa()
    c, layer = make_layer([300, 120], extra=80, seed=72)
    par = [[-1, 0, 2, 5, 1, 4, -2, 6, 3, 0], [-1, -3, 1, 2, 0, 0, 9, 6, 7, 8]]
    n = len(par[0])
    q, kn, vn = c.normal(2, n, 8, 128), c.normal(2, n, 2, 128), c.normal(2, n, 2, 128)
    used = [C.used_nodes(p) for p in par]
    for b in range(2):  # (of the size that decides the selection, had they a share)
        q[b, torch.as_tensor(~used[b])] *= 20
    before = [c.k.clone(), c.v.clone(), layer.score_cache.clone()]
    out = layer.draft(q.cuda(), kn.cuda(), vn.cuda(), cuda(par), sparse=sparse)
    assert J.device_error() & ~16 == 2
    for b, L in enumerate(c.lens):
        for i in range(n):
            page, slot = c.table[b, (L + i) // 16], (L + i) % 16
            now = [c.k[page, slot], c.v[page, slot], layer.score_cache[page, :, slot]]
            was = [before[0][page, slot], before[1][page, slot], before[2][page, :, slot]]
            if used[b][i]:
                assert torch.equal(now[0].cpu(), kn[b, i]) and not torch.equal(now[2], was[2])
            else:
                assert all(torch.equal(x, y) for x, y in zip(now, was))
    idx = count = None
    if sparse:
        mean = torch.stack([q[b, torch.as_tensor(used[b])].double().mean(0) for b in range(2)])
        idx, count = J.score_topk(mean.to(torch.bfloat16).cuda(), layer.basis, layer.score_cache, c.bt,
                                  c.seq_lens, layer.budget)
        same = (idx[..., None] == layer.idx[:, :, None]).any(-1).float().mean()
        assert float(same) > 0.95  # (a mean rounded from float32 or float64 may differ by a bf16 step)
        idx, count = layer.idx.cpu().numpy(), layer.count.cpu().numpy()
    scale = 1 / math.sqrt(128)
    ref, mag = C.tree_attend(f64(q), f64(c.k), f64(c.v), c.table, c.lens, par, scale, -1, idx, count)
    check_close(f64(out), ref, mag, weight_slack(f64(q), f64(c.k), scale, 310))


def test_draft_selects_without_the_padding():
    # what an unused node's query holds reaches nothing
    J = jssa()
    c, layer = make_layer([500, 120], extra=80, seed=73)
    par = cuda([[-1, 0, 0, -2, -7], [-1, -1, -5, -5, -5]])
    q, kn, vn = c.normal(2, 5, 8, 128).cuda(), c.normal(2, 5, 2, 128).cuda(), c.normal(2, 5, 2, 128).cuda()
    want = layer.draft(q, kn, vn, par, sparse=True).clone()
    idx = layer.idx.clone()
    for bad in (NAN, math.inf, 3e38):
        q[0, 3:], q[1, 2:] = bad, bad
        out = layer.draft(q, kn, vn, par, sparse=True)
        assert torch.equal(layer.idx, idx) and torch.equal(out, want)
    assert J.device_error() & ~16 == 0


@pytest.mark.parametrize("d,r", [(128, 32), (256, 64)])
@pytest.mark.parametrize("n", [0, 1, 33, 64])
def test_draft_sizes(n, d, r):
    # the slots and the mean query of trees of every width, no nodes among them
    J = jssa()
    c, layer = make_layer([77, 0, 200], h_kv=1, d=d, r=r, extra=80, seed=74)
    par = [random_tree(c.rng, n, unused=min(n, b)) for b in range(3)]
    q, kn, vn = c.normal(3, n, 3, d), c.normal(3, n, 1, d), c.normal(3, n, 1, d)
    par = torch.as_tensor(np.asarray(par).reshape(3, n))
    slots, mean = J.api._tree_prepare(q.cuda(), cuda(par), c.bt, c.seq_lens, c.k.shape[0], 16, True)
    used = [C.used_nodes(par[b].tolist()) for b in range(3)]
    for b, L in enumerate(c.lens):
        pos = L + np.arange(n)
        want = np.where(used[b], c.table[b][pos // 16] * 16 + pos % 16, -1) if n else np.zeros(0)
        assert np.array_equal(slots.view(3, n)[b].cpu().numpy(), want)
        rows = q[b, torch.as_tensor(used[b])].double()
        ref = rows.mean(0).numpy() if len(rows) else np.zeros((3, d))
        # one rounding to bf16, fp32 sums of n terms
        tol = 2.0 ** -8 * np.abs(ref) + (n + 1) * 2.0 ** -23 * (rows.abs().mean(0).numpy() if len(rows) else 0)
        assert np.all(np.abs(f64(mean[b]) - ref) <= tol)
    for sparse in (False, True):
        out = layer.draft(q.cuda(), kn.cuda(), vn.cuda(), cuda(par), sparse=sparse)
        idx = layer.idx.cpu().numpy() if sparse else None
        cnt = layer.count.cpu().numpy() if sparse else None
        if not n:
            assert out.shape == (3, 0, 3, d)
            continue
        ref, mag = C.tree_attend(f64(q), f64(c.k), f64(c.v), c.table, c.lens, par.tolist(), d ** -0.5, -1,
                                 idx, cnt)
        check_close(f64(out), ref, mag, weight_slack(f64(q), f64(c.k), d ** -0.5, 264))
    assert J.device_error() & ~16 == 0


def test_a_refused_draft_changes_nothing():
    J = jssa()
    c, layer = make_layer([300, 120], extra=80, seed=75)
    q, kn, vn = c.normal(2, 6, 8, 128).cuda(), c.normal(2, 6, 2, 128).cuda(), c.normal(2, 6, 2, 128).cuda()
    par = cuda([random_tree(c.rng, 6) for _ in range(2)])
    layer.idx.fill_(3), layer.count.fill_(4)
    state = [c.k, c.v, layer.score_cache, layer.seq_lens, layer.idx, layer.count, layer.mass]
    before = [t.clone() for t in state]
    for sparse in (False, True):
        wide = c.normal(2, 6, 2, 256).cuda()
        for args, kw in [
            ((q, kn, vn, par.long()), {}), ((q, kn, vn, par.cpu()), {}), ((q, kn, vn, par[:, :5]), {}),
            ((q[:, :5], kn, vn, par), {}), ((q.float(), kn, vn, par), {}), ((q, kn, vn.float(), par), {}),
            ((q, kn, vn[:, :, :1], par), {}), ((q, kn[:1], vn, par), {}), ((q, kn, None, par), {}),
            ((q, wide, wide, par), {}), ((q[0], kn, vn, par), {}),
            ((q, kn.transpose(1, 2).contiguous().transpose(1, 2), vn, par), {}),
            ((q, kn, vn, par), dict(out=torch.empty_like(q)[:1])),
            ((q.repeat(1, 1, 5, 1), kn, vn, par), {}),  # 20 query heads per KV head
            ((q[:, :, :3].contiguous(), kn, vn, par), {}),  # 3 query heads, 2 KV heads
            *([((q, kn, vn, par), dict(window=32))] if sparse else []),
        ]:
            with pytest.raises((ValueError, TypeError, J.JSSAError)):
                layer.draft(*args, sparse=sparse, **kw)
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(state, before))
    assert J.device_error() == 0


# ------------------------------------------------------------------------------------------------
# eviction and commit over unusable pages
# ------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("L,keep", [(100, 40), (3000, 700)])
@pytest.mark.parametrize("how", ["in place", "mass apart", "pages apart", "both apart"])
def test_evict_leaves_rows_of_unusable_pages_alone(how, L, keep):
    # a row that cannot be read or written stays as it was: K, V, code and mass
    J = jssa()
    ps, h_kv = 16, 2
    c = Paged([1, 1], 0, h_kv, 128, ps, pages=-(-L // ps), seed=keep)
    lens = cuda([L, L - 7])
    c.k.copy_(c.normal(*c.k.shape)), c.v.copy_(c.normal(*c.v.shape))
    n0, per = c.k.shape[0], -(-keep // ps)
    if "pages" in how or "both" in how:
        c.k, c.v = (torch.cat([t, torch.zeros((2 * per, *t.shape[1:]), dtype=t.dtype, device="cuda")])
                    for t in (c.k, c.v))
    codes = torch.randint(0, 256, (c.k.shape[0], h_kv, ps, 32), dtype=torch.uint8, device="cuda")
    mass = torch.rand((2, h_kv, c.table.shape[1] * ps), device="cuda") ** 6
    src = c.table.copy()
    src[0, 3], src[1, 1], src[1, 5] = -1, 10 ** 6, c.k.shape[0]
    if c.k.shape[0] == n0:
        dst = src
    else:
        dst = (n0 + np.arange(2 * per)).reshape(2, per)
        dst[0, 1] = -5
        dst = dst[:, :-1]  # (one page short: the last rows have no place)
    apart = how in ("mass apart", "both apart")
    mass_out = torch.full_like(mass, 5.0) if apart else mass
    start = [t.clone() for t in (c.k, c.v, codes, mass, mass_out)]
    bt = cuda(src)
    idx, count, _ = J.evict(mass, c.k, c.v, bt, lens, keep, 9, codes,
                            None if dst is src else cuda(dst), mass_out if apart else None)
    assert J.device_error() == (1 if dst is src else 3)
    k1, v1, s1, _, m1 = (t.clone().cpu() for t in start)
    k0, v0, s0, m0, _ = (t.cpu() for t in start)

    def place(table, b, t):
        page = table[b, t // ps] if t // ps < table.shape[1] else -1
        return (page, t % ps) if 0 <= page < c.k.shape[0] else None

    for b, n in enumerate([L, L - 7]):
        for h in range(h_kv):
            want = C.kept_positions(m0[b, h].numpy(), n, keep, 9)
            assert np.array_equal(idx[b, h].cpu().numpy(), want)
            for i, t in enumerate(want):
                a, z = place(src, b, t), place(dst, b, i)
                if a is None or z is None:
                    continue
                k1[z[0], z[1], h], v1[z[0], z[1], h] = k0[a[0], a[1], h], v0[a[0], a[1], h]
                s1[z[0], h, z[1]], m1[b, h, i] = s0[a[0], h, a[1]], m0[b, h, t]
            m1[b, h, keep:n] = 0
    for got, ref in zip((c.k, c.v, codes, mass_out), (k1, v1, s1, m1)):
        assert torch.equal(got.cpu(), ref)
    if apart:
        assert torch.equal(mass.cpu(), m0)


@pytest.mark.parametrize("node", [1, 2])
def test_commit_flags_an_accepted_node_on_an_unusable_page(node):
    # a node that keeps its position is an entry like any other
    J = jssa()
    c = Paged([15, 40], 20, 1, seed=80)
    table = c.table.copy()
    table[0, 1] = -1  # (positions 16.. of the first sequence: its nodes 1..)
    path = np.array([[0, 0, 0], [0, 1, 2]])
    path[0, 1] = node
    k0 = c.k.clone()
    out = J.tree_commit(c.k, c.v, cuda(table), c.seq_lens, cuda(path), cuda([2, 3]))
    assert J.device_error() == 1 and out.tolist() == [17, 43]
    assert torch.equal(torch.nan_to_num(c.k, nan=7.0), torch.nan_to_num(k0, nan=7.0))


# ------------------------------------------------------------------------------------------------
# rarer branches: groups, head dims, many splits, long contexts, non-finite values in later tiles
# ------------------------------------------------------------------------------------------------


def _ref_attend(q, k, v, table, positions, h, g, scale, mass=None):
    """Float64 on the GPU: (outputs [g, d], sum of weight * |v|, weights summed over the group) of the
    query heads of KV head ``h`` over ``positions`` (a tensor)."""
    ps = k.shape[1]
    page = table.long()[positions // ps]
    kk, vv = k[page, positions % ps, h].double(), v[page, positions % ps, h].double()
    p = torch.softmax(q[h * g:(h + 1) * g].double() @ kk.T * scale, 1)
    return p @ vv, p @ vv.abs(), p.sum(0)


def check_mass_call(out, mass, before, q, k, v, bt, positions, g, scale):
    """``positions(b, h)``: the attended positions. Outputs and masses of a call against float64: a
    weight is off by the slack without its split, which the masses do not have."""
    batch, h_kv, d = q.shape[0], k.shape[2], k.shape[3]
    for b in range(batch):
        for h in range(h_kv):
            pos = positions(b, h)
            got, old = mass[b, h].double(), before[b, h].double()
            if len(pos) == 0:
                assert torch.count_nonzero(out[b, h * g:(h + 1) * g]).item() == 0
                assert torch.equal(got, old)
                continue
            o, a, w = _ref_attend(q[b], k, v, bt[b], pos, h, g, scale)
            qa = q[b, h * g:(h + 1) * g].double().abs()
            top = float((qa @ k[bt[b].long()[pos // k.shape[1]], pos % k.shape[1], h].double().abs().T).max())
            slack = 2 * (d * 2.0 ** -23 * scale * top + 2.0 ** -20) + 3 * len(pos) * 2.0 ** -23
            tol = 2.0 ** -8 * o.abs() + (1 + 2.0 ** -8) * (slack + 2.0 ** -14) * a
            assert bool(((out[b, h * g:(h + 1) * g].double() - o).abs() <= tol).all())
            assert bool(((got[pos] - old[pos] - w).abs() <= slack * w + 2.0 ** -22 * (old[pos] + w)).all())
            rest = torch.ones(len(got), dtype=torch.bool, device="cuda")
            rest[pos] = False
            assert torch.equal(got[rest], old[rest])


def paged_normal(lens, h_kv, d, seed, extra=0, ps=16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    per = -(-(max(lens) + extra) // ps)
    total = len(lens) * per + 2
    bt = torch.randperm(total, generator=gen, device="cuda")[:len(lens) * per].view(len(lens), per).int()
    k, v = (torch.empty((total, ps, h_kv, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
            for _ in range(2))
    return gen, bt, k, v


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("budget", [70, 1100])
def test_indexed_mass_groups_and_head_dims(budget, g, d):
    J = jssa()
    lens, h_kv = [0, 5, 90, 1700], 2
    gen, bt, k, v = paged_normal(lens, h_kv, d, seed=g + d)
    q = torch.empty((4, h_kv * g, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) * 2
    idx = torch.full((4, h_kv, budget), -1, dtype=torch.int32, device="cuda")
    count = torch.zeros((4, h_kv), dtype=torch.int32, device="cuda")
    for b, L in enumerate(lens):
        for h in range(h_kv):
            m = min(L, budget - h)
            count[b, h] = m
            idx[b, h, :m] = torch.randperm(L, generator=gen, device="cuda")[:m].sort().values.int()
    mass = torch.rand((4, h_kv, bt.shape[1] * 16 + 3), generator=gen, device="cuda")
    before = mass.clone()
    out = J.indexed_attend(q, k, v, bt, idx, count, mass=mass)
    check_mass_call(out, mass, before, q, k, v, bt,
                    lambda b, h: idx[b, h, :int(count[b, h])].long(), g, d ** -0.5)
    assert J.device_error() == 0


@pytest.mark.parametrize("d,r,g,h_kv", [(128, 16, 1, 2), (128, 64, 3, 2), (128, 32, 8, 1), (256, 64, 2, 2),
                                        (256, 64, 4, 1)])
def test_decode_step_with_mass(d, r, g, h_kv):
    J = jssa()
    lens, budget = [1, 40, 3000], 96
    gen, bt, k, v = paged_normal(lens, h_kv, d, seed=r + g)
    basis = torch.linalg.qr(torch.randn((h_kv, d, r), generator=gen, device="cuda"))[0].transpose(1, 2).contiguous()
    layer = J.PagedLayer(k, v, bt, cuda(lens), basis, budget, track_mass=True)
    layer.prefill_scores()
    plain = J.PagedLayer(k.clone(), v.clone(), bt, cuda(lens), basis, budget)
    plain.score_cache.copy_(layer.score_cache)
    new = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)  # noqa: E731
    layer.mass.copy_(torch.rand(layer.mass.shape, generator=gen, device="cuda"))
    for _ in range(2):
        q, kn, vn = new(3, h_kv * g, d), new(3, h_kv, d), new(3, h_kv, d)
        before = layer.mass.clone()
        out, idx, count = layer.step(q, kn, vn)
        _, idx2, count2 = plain.step(q, kn, vn)
        assert torch.equal(idx, idx2) and torch.equal(count, count2)
        assert torch.equal(layer.k_cache, plain.k_cache) and torch.equal(layer.score_cache, plain.score_cache)
        check_mass_call(out, layer.mass, before, q, layer.k_cache, layer.v_cache, bt,
                        lambda b, h: idx[b, h, :int(count[b, h])].long(), g, d ** -0.5)
    assert J.device_error() & ~16 == 0


@pytest.mark.parametrize("d,g", [(128, 1), (128, 4), (256, 3)])
def test_dense_mass_over_many_splits(d, g):
    # one pair over 42K positions: more partials than the second kernel keeps weights of
    J = jssa()
    gen, bt, k, v = paged_normal([42001], 1, d, seed=d + g)
    q = torch.empty((1, g, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) * 2
    mass = torch.rand((1, 1, bt.shape[1] * 16), generator=gen, device="cuda")
    for window in (-1, 40000):
        before = mass.clone()
        out = J.dense_decode(q, k, v, bt, cuda([42001]), window=window, mass=mass)
        lo = 0 if window < 0 else 42001 - window
        check_mass_call(out, mass, before, q, k, v, bt,
                        lambda b, h: torch.arange(lo, 42001, device="cuda"), g, d ** -0.5)
    assert J.device_error() == 0


@pytest.mark.parametrize("batch,L,n,g,h_kv,d,window", [
    (1, 131072, 9, 4, 1, 128, -1), (1, 131072, 64, 4, 1, 128, -1), (1, 70001, 5, 2, 2, 256, -1),
    (2, 131072, 40, 4, 1, 128, 100000), (1, 131000, 3, 8, 1, 256, 4096),
])
def test_tree_attend_over_the_longest_contexts(batch, L, n, g, h_kv, d, window):
    J = jssa()
    lens = [L - 1009 * b for b in range(batch)]
    gen, bt, k, v = paged_normal(lens, h_kv, d, seed=n, extra=n)
    rng = np.random.default_rng(n)
    q = torch.empty((batch, n, h_kv * g, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) * 2
    parents = [random_tree(rng, n, b) for b in range(batch)]
    out = J.tree_attend(q, k, v, bt, cuda(lens), cuda(parents), window=window)
    for b in range(batch):
        for i in range(n):
            pos = C.tree_positions(parents[b], i, lens[b], window)
            if not pos:
                assert torch.count_nonzero(out[b, i]).item() == 0
                continue
            pos = torch.as_tensor(np.asarray(pos)).cuda()
            for h in range(h_kv):
                o, a, _ = _ref_attend(q[b, i], k, v, bt[b], pos, h, g, d ** -0.5)
                qa = q[b, i, h * g:(h + 1) * g].double().abs()
                top = float((qa @ k[bt[b].long()[pos // 16], pos % 16, h].double().abs().T).max())
                # (a row's sums run over tiles of 64 positions, a CTA's share of them, and the CTAs' partials)
                slack = 2.0 ** -14 + 2 * (d * 2.0 ** -23 * d ** -0.5 * top + 2.0 ** -20) + 3 * len(pos) * 2.0 ** -23
                tol = 2.0 ** -8 * o.abs() + (1 + 2.0 ** -8) * slack * a
                assert bool(((out[b, i, h * g:(h + 1) * g].double() - o).abs() <= tol).all())
    assert J.device_error() == 0


@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("n,g,d", [(33, 4, 128), (64, 4, 128), (64, 8, 128), (40, 3, 128), (40, 3, 256), (64, 4, 256)])
def test_masked_values_in_later_tiles_do_not_leak(n, g, d, bad):
    # as test_masked_values_do_not_leak, with nodes in the fifth and sixth tile of their pair, and with
    # more rows than one group holds
    J = jssa()
    L = 300
    c = Paged([L], n, 1, d, seed=n)
    parents = [random_tree(c.rng, n)]
    anc = C.ancestors(parents[0])
    depth = [len(a) - 1 for a in anc]
    q, kn, vn = c.normal(1, n, g, d), c.normal(1, n, 1, d), c.normal(1, n, 1, d)
    run = lambda **kw: J.tree_attend(  # noqa: E731
        q.cuda(), c.k, c.v, c.bt, c.seq_lens, cuda(parents), kn.cuda(), vn.cuda(), **kw)[0].float()
    ref = run()
    for node in (2, n - 9):
        was = vn[0, node, 0, 7].clone()
        vn[0, node, 0, 7] = bad
        out = run()
        vn[0, node, 0, 7] = was
        sees = torch.as_tensor([node in a for a in anc])
        assert bool(sees.any()) and not bool(sees.all())
        assert torch.equal(out[~sees], ref[~sees])
        hit = out[sees][..., 7]
        assert bool((torch.isnan(hit) if math.isnan(bad) else hit == bad).all())
        out[..., 7] = ref[..., 7]
        assert bool(torch.isfinite(out).all())
        # (V of that tile is cleared and added by hand: the other elements are the same sums)
        assert torch.equal(out, ref)
    # a window that starts in a tile with a bad value, seen by the shallow nodes only
    window = 150
    ref = run(window=window)
    t = L + 2 - window
    c.v[c.table[0, t // 16], t % 16, 0, 2] = bad
    out = run(window=window)
    sees = torch.as_tensor([dep <= 1 for dep in depth])
    assert torch.equal(out[~sees], ref[~sees])
    assert not bool(torch.isfinite(out[sees][..., 2]).any())
