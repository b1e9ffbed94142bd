"""Tree attention, commit, attention mass and eviction on the GPU against the float64 oracle.

Tolerances, fixed before the first run:
* moved rows, index sets, counts and lengths: exact;
* attention outputs, elementwise, with A = sum_t p_t |v_t| from the oracle: the bf16 weights may be
  off by half a step each (2^-8 A), the bf16 output by half a step (2^-8 |o|), scores and sums in
  fp32 by X = 2 (d 2^-23 max_t scale sum|q||k| + 2^-20), as a factor on A;
* mass: the same relative X on each step's weights, and fp32 additions (2^-23 of the entry).
"""

import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as C

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from token_level_sparse_fp8_b200 import build
    build.build()


@pytest.fixture(autouse=True)
def _clean_flags():
    J = jssa()
    J.device_error(clear=True)
    yield
    J.device_error(clear=True)


def jssa():
    import token_level_sparse_fp8_b200 as J
    return J


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def cuda(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a)).to(dtype).cuda()


class Paged:
    """A paged cache whose unused slots hold NaN, with scattered pages; ``head_major`` lays the
    pages out as [page, head, slot, d]."""

    def __init__(self, lens, extra=0, h_kv=2, d=128, ps=16, seed=0, head_major=False, pages=None):
        self.lens, self.ps, self.h_kv, self.d = list(lens), ps, h_kv, d
        self.rng = rng = np.random.default_rng(seed)
        per = pages or max(1, max(-(-(n + extra) // ps) for n in lens))
        total = per * len(lens) + 3
        self.table = rng.permutation(total)[:per * len(lens)].reshape(len(lens), per)
        shape = (total, h_kv, ps, d) if head_major else (total, ps, h_kv, d)
        self.k, self.v = (torch.full(shape, NAN, dtype=torch.bfloat16) for _ in range(2))
        if head_major:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        for b, n in enumerate(lens):
            for t in range(n):
                for c in (self.k, self.v):
                    c[self.table[b, t // ps], t % ps] = self.normal(h_kv, d)
        self.k, self.v = self.k.cuda(), self.v.cuda()  # (strides are kept)
        self.bt, self.seq_lens = cuda(self.table), cuda(lens)

    def normal(self, *shape):
        return torch.from_numpy(self.rng.standard_normal(shape)).to(torch.bfloat16)

    def put(self, b, t, k, v):
        self.k[self.table[b, t // self.ps], t % self.ps] = k.to(self.k.device)
        self.v[self.table[b, t // self.ps], t % self.ps] = v.to(self.v.device)


def fp32_slack(q, k, d, scale):
    """X of the module's tolerances; ``k`` without NaN."""
    top = float(np.abs(q).sum(-1).max()) * float(np.nanmax(np.abs(np.where(np.isfinite(k), k, 0))))
    return 2 * (d * 2.0 ** -23 * abs(scale) * top + 2.0 ** -20)


def check_out(out, ref, mag, slack):
    got = f64(out)
    assert np.isfinite(got).all()
    tol = 2.0 ** -8 * (mag + np.abs(ref)) + slack * mag
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) - tol))


def random_tree(rng, n, unused=0):
    par = [int(max(-1, i - 1 - rng.integers(0, 4))) for i in range(n)]
    for i in range(n - unused, n):
        par[i] = -2 - i
    return par


def run_tree(c, n, g, parents, window=-1, budget=0, stored=False, seed=1, scale=None):
    """A tree step over ``c``; the nodes' rows come through k_new or are put into the cache."""
    J = jssa()
    B, h_q = len(c.lens), c.h_kv * g
    q, kn, vn = c.normal(B, n, h_q, c.d) * 2, c.normal(B, n, c.h_kv, c.d), c.normal(B, n, c.h_kv, c.d)
    idx = count = None
    if budget:
        idx = np.full((B, c.h_kv, budget), -1)
        count = np.zeros((B, c.h_kv), dtype=np.int64)
        for b, L in enumerate(c.lens):
            for h in range(c.h_kv):
                m = min(L, budget) - (h if L > 1 else 0)
                count[b, h] = max(m, 0)
                idx[b, h, :count[b, h]] = np.sort(c.rng.permutation(L)[:count[b, h]])
    if stored:
        for b, L in enumerate(c.lens):
            used = C.used_nodes(parents[b])
            for i in range(n):
                if used[i]:
                    c.put(b, L + i, kn[b, i], vn[b, i])
    before = c.k.clone(), c.v.clone()
    kw = {} if stored else dict(k_new=kn.cuda(), v_new=vn.cuda())
    if budget:
        kw.update(idx=cuda(idx), count=cuda(count))
    scale = 1 / math.sqrt(c.d) if scale is None else scale
    out = J.tree_attend(q.cuda(), c.k, c.v, c.bt, c.seq_lens, cuda(parents), window=window,
                        scale=scale, **kw)
    # the cache: used nodes' rows written, nothing else
    for b, L in enumerate(c.lens):
        used = C.used_nodes(parents[b])
        for i in range(n):
            if used[i] and not stored:
                p, s = c.table[b, (L + i) // c.ps], (L + i) % c.ps
                before[0][p, s], before[1][p, s] = kn[b, i].cuda(), vn[b, i].cuda()
    for x, y in zip(before, (c.k, c.v)):
        assert torch.equal(torch.nan_to_num(x, nan=7.0), torch.nan_to_num(y, nan=7.0))
    ref, mag = C.tree_attend(f64(q), f64(c.k), f64(c.v), c.table, c.lens, parents, scale, window,
                             idx, count)
    check_out(out, ref, mag, fp32_slack(f64(q), f64(c.k), c.d, scale))
    return out, q, parents


# ------------------------------------------------------------------------------------------------
# tree attention
# ------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("lens,n,g,h_kv,ps", [
    ([0, 1, 63, 64, 65, 200], 1, 1, 1, 16),      # single tokens, empty context, tile edges
    ([0, 5, 64, 130, 257], 5, 3, 2, 16),         # odd group, rows below a warp
    ([0, 1, 2, 61], 64, 1, 2, 64),               # the widest tree, longer than the context
    ([190, 60, 1], 33, 4, 2, 8),                 # 132 rows: just past one 128-row tile
    ([77, 128], 64, 8, 1, 32),                   # 512 rows
    ([70], 32, 8, 1, 16),                        # 256 rows
])
@pytest.mark.parametrize("stored", [False, True])
def test_tree_attend(lens, n, g, h_kv, ps, d, stored):
    c = Paged(lens, n, h_kv, d, ps, seed=n + d)
    parents = [random_tree(c.rng, n, unused=min(n - 1, b % 3)) for b in range(len(lens))]
    run_tree(c, n, g, parents, stored=stored)
    assert jssa().device_error() == 0


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 5000])
def test_tree_attend_window(window, d):
    c = Paged([0, 3, 64, 200, 133], 20, 2, d, 16, seed=window)
    parents = [list(range(-1, 19))] + [random_tree(c.rng, 20, b) for b in range(1, 5)]
    run_tree(c, 20, 4, parents, window=window)
    assert jssa().device_error() == 0


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("budget", [1, 64, 130])
def test_tree_attend_indexed(budget, d):
    c = Paged([0, 1, 64, 200, 131], 9, 2, d, 16, seed=budget)
    run_tree(c, 9, 4, [random_tree(c.rng, 9, b % 3) for b in range(5)], budget=budget)
    assert jssa().device_error() == 0


def test_tree_attend_all_nodes_unused_and_no_nodes():
    J = jssa()
    c = Paged([40, 9], 4)
    out, _, _ = run_tree(c, 4, 2, [[-2] * 4, [-1, 0, -7, -9]])
    assert torch.count_nonzero(out[0]).item() == 0 and torch.count_nonzero(out[1, 2:]).item() == 0
    q = torch.zeros((2, 0, 4, 128), dtype=torch.bfloat16, device="cuda")
    par = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    assert J.tree_attend(q, c.k, c.v, c.bt, c.seq_lens, par).shape == (2, 0, 4, 128)


def test_tree_attend_other_strides():
    c = Paged([100, 31], 12, 2, 128, 16, seed=9, head_major=True)
    assert c.k.stride(1) == 128 and c.k.stride(2) == 16 * 128
    run_tree(c, 12, 4, [random_tree(c.rng, 12) for _ in range(2)])
    big = torch.full((c.k.shape[0], 2 * c.ps, 3, 128), NAN, dtype=torch.bfloat16, device="cuda")
    c2 = Paged([100, 31], 12, 2, 128, 16, seed=9)
    for name in ("k", "v"):
        wide = big.clone()[:, ::2, 1:3]
        wide.copy_(getattr(c2, name))
        setattr(c2, name, wide)
    run_tree(c2, 12, 4, [random_tree(c2.rng, 12) for _ in range(2)])


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf])
def test_masked_values_do_not_leak(bad, d):
    # node 1's row is not finite: its subtree sees that, its siblings and the rest do not; the same
    # for a context position that only some nodes' windows hold
    J = jssa()
    c = Paged([37], 6, 1, d, seed=4)
    parents = [[-1, -1, 0, 1, 2, 0]]
    q, kn, vn = c.normal(1, 6, 4, d), c.normal(1, 6, 1, d), c.normal(1, 6, 1, d)
    ref = J.tree_attend(q.cuda(), c.k, c.v, c.bt, c.seq_lens, cuda(parents), kn.cuda(), vn.cuda())
    vn[0, 1, 0, 3], kn[0, 1, 0, 5] = bad, bad
    out = J.tree_attend(q.cuda(), c.k, c.v, c.bt, c.seq_lens, cuda(parents), kn.cuda(), vn.cuda())
    clean = [0, 2, 4, 5]
    assert torch.equal(out[0, clean], ref[0, clean])
    vn[0, 1, 0, 3], kn[0, 1, 0, 5] = bad, 0.5  # (a finite key: the value alone reaches the output)
    out = J.tree_attend(q.cuda(), c.k, c.v, c.bt, c.seq_lens, cuda(parents), kn.cuda(), vn.cuda())
    assert torch.equal(out[0, clean], ref[0, clean])
    got = out[0, [1, 3]].float()
    assert bool((torch.isnan(got[..., 3]) if math.isnan(bad) else got[..., 3] == bad).all())
    assert bool(torch.isfinite(got[..., :3]).all()) and bool(torch.isfinite(got[..., 4:]).all())
    # window 8: node 0 sees positions 30.., its child (depth 1) 31..
    kn[0, 1], vn[0, 1] = 0.25, 0.25
    ref = J.tree_attend(q.cuda(), c.k, c.v, c.bt, c.seq_lens, cuda(parents), kn.cuda(), vn.cuda(),
                        window=8)
    c.v[c.table[0, 30 // 16], 30 % 16, 0, 2] = bad
    out = J.tree_attend(q.cuda(), c.k, c.v, c.bt, c.seq_lens, cuda(parents), kn.cuda(), vn.cuda(),
                        window=8)
    deep = [2, 3, 4, 5]
    assert torch.equal(out[0, deep], ref[0, deep])
    assert not bool(torch.isfinite(out[0, :2, :, 2].float()).any())


def test_tree_attend_flags_bad_inputs():
    J = jssa()
    c = Paged([40, 40, 40], 8, 2, seed=6)
    q = c.normal(3, 8, 4, 128)
    kn, vn = c.normal(3, 8, 2, 128).cuda(), c.normal(3, 8, 2, 128).cuda()
    good = [random_tree(c.rng, 8) for _ in range(3)]
    run = lambda par, table, lens, **kw: J.tree_attend(  # noqa: E731
        q.cuda(), c.k, c.v, cuda(table), cuda(lens), cuda(par), kn, vn, **kw)
    scale = 1 / math.sqrt(128)
    # a parent behind the node, itself, or unused: the node is unused and flagged
    par = [[-1, 0, 2, 5, 1, 4, -2, 6], good[1], good[2]]
    out = run(par, c.table, c.lens)
    assert J.device_error() == 2
    ref, mag = C.tree_attend(f64(q), f64(c.k), f64(c.v), c.table, c.lens, par, scale)
    check_out(out, ref, mag, fp32_slack(f64(q), f64(c.k), 128, scale))
    assert torch.count_nonzero(out[0, [2, 3, 6, 7]]).item() == 0
    # pages outside the pool: their positions take no part
    table = c.table.copy()
    table[0, 1], table[1, 0] = -1, c.k.shape[0]
    out = run(good, table, c.lens)
    assert J.device_error() == 1
    ref, mag = C.tree_attend(f64(q), f64(c.k), f64(c.v), table, c.lens, good, scale)
    check_out(out, ref, mag, fp32_slack(f64(q), f64(c.k), 128, scale))
    # nodes past the end of the block table, and index-set entries outside it
    full = [c.table.shape[1] * 16 - 3, 40, 40]
    c.k.nan_to_num_(0.5), c.v.nan_to_num_(0.5)
    out = run(good, c.table, full)
    assert J.device_error() == 2
    ref, mag = C.tree_attend(f64(q), f64(c.k), f64(c.v), c.table, full, good, scale)
    check_out(out, ref, mag, fp32_slack(f64(q), f64(c.k), 128, scale))
    idx = np.tile(np.array([3, 5, -1, 10 ** 6]), (3, 2, 1))
    cnt = np.full((3, 2), 9)  # (clamped to the budget)
    out = run(good, c.table, c.lens, idx=cuda(idx), count=cuda(cnt))
    assert J.device_error() == 2
    ref, mag = C.tree_attend(f64(q), f64(c.k), f64(c.v), c.table, c.lens, good, scale, -1, idx,
                             np.minimum(cnt, 4))
    check_out(out, ref, mag, fp32_slack(f64(q), f64(c.k), 128, scale))
    # lengths outside the table are clamped
    out = run(good, c.table, [-5, 40, 40])
    assert J.device_error() == 4
    ref, mag = C.tree_attend(f64(q), f64(c.k), f64(c.v), c.table, [0, 40, 40], good, scale)
    check_out(out, ref, mag, fp32_slack(f64(q), f64(c.k), 128, scale))
    run(good, c.table, [10 ** 6, 40, 40])
    assert J.device_error() == 4 | 2


def _tree_ref64(q, k, v, bt, lens, parents, window, scale):
    """The tree in torch float64 on the GPU, one sequence and head at a time (long contexts)."""
    B, n, h_q, d = q.shape
    h_kv, ps = k.shape[2], k.shape[1]
    g = h_q // h_kv
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for b in range(B):
        L = int(lens[b])
        pos = torch.arange(L + n, device="cuda")
        page = bt[b].long()[pos // ps]
        anc = C.ancestors(parents[b])
        see = torch.zeros((n, L + n), dtype=torch.bool)
        for i in range(n):
            dep = len(anc[i]) - 1
            if anc[i]:
                see[i, (max(0, L + dep - window + 1) if window > 0 else 0):L] = True
                see[i, [L + a for a in anc[i] if window <= 0 or len(anc[a]) - 1 > dep - window]] = True
        see = see.cuda()
        for h in range(h_kv):
            kk = torch.nan_to_num(k[page, pos % ps, h].double())
            vv = torch.nan_to_num(v[page, pos % ps, h].double())
            x = torch.einsum("ngd,td->ngt", q[b, :, h * g:(h + 1) * g].double(), kk) * scale
            x = x.masked_fill(~see[:, None], -math.inf)
            some = see.any(1)
            p = torch.softmax(x[some], 2)
            out[b, some, h * g:(h + 1) * g] = torch.einsum("ngt,td->ngd", p, vv)
            mag[b, some, h * g:(h + 1) * g] = torch.einsum("ngt,td->ngd", p, vv.abs())
    return out, mag


@pytest.mark.parametrize("batch,L,n,g,h_kv,d,window", [
    (1, 20011, 7, 4, 2, 128, -1),     # few rows, many splits
    (3, 9000, 64, 4, 2, 128, -1),     # 256 rows
    (2, 5003, 64, 8, 2, 128, -1),     # 512 rows
    (2, 7001, 64, 2, 2, 256, -1),     # one full tile at head dim 256
    (2, 3001, 50, 8, 1, 256, -1),     # four row tiles at head dim 256
    (4, 9000, 31, 4, 2, 128, 1024),
    (40, 700, 12, 4, 8, 128, -1),     # more (sequence, head) pairs than SMs
    (300, 40, 4, 4, 4, 128, -1),      # many pairs of a single tile
    (300, 50, 2, 2, 4, 256, -1),
    (150, 90, 40, 4, 4, 128, 30),     # many short pairs of two tiles, 160 rows, windowed
])
def test_tree_attend_long(batch, L, n, g, h_kv, d, window):
    J = jssa()
    gen = torch.Generator(device="cuda").manual_seed(L)
    rng = np.random.default_rng(L)
    lens = [L - int(x) for x in [0, *rng.integers(0, L // 2, batch - 1)]]
    ps, per = 16, -(-(L + n) // 16)
    total = batch * per + 1
    bt = torch.randperm(total, generator=gen, device="cuda")[:batch * per].view(batch, per).int()
    k, v = (torch.empty((total, ps, h_kv, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
            for _ in range(2))
    q = torch.empty((batch, n, h_kv * g, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) * 2
    parents = [random_tree(rng, n, b % 4 if n > 8 else 0) for b in range(batch)]
    scale = 1 / math.sqrt(d)
    out = J.tree_attend(q, k, v, bt, cuda(lens), cuda(parents), window=window)
    ref, mag = _tree_ref64(q, k, v, bt, lens, parents, window, scale)
    slack = 2 * (d * 2.0 ** -23 * scale * float(q.abs().sum(-1).max()) * float(k.abs().max()) + 2.0 ** -20)
    check_out(out, f64(ref), f64(mag), slack)
    again = J.tree_attend(q, k, v, bt, cuda(lens), cuda(parents), window=window)
    assert torch.equal(out, again)  # no atomics: the same bits
    assert J.device_error() == 0


def test_tree_attend_large_logits():
    # row maxima that jump by hundreds from tile to tile (the running maximum is rescaled often)
    c = Paged([300], 5, 1, 128, seed=12)
    with torch.no_grad():
        for t in range(300):
            c.k[c.table[0, t // 16], t % 16] *= 1 + t // 40
    run_tree(c, 5, 4, [random_tree(c.rng, 5)], scale=1.0)


def test_tree_attend_captured_on_a_stream():
    J = jssa()
    c = Paged([333, 64], 11, 2, seed=14)
    par = cuda([random_tree(c.rng, 11) for _ in range(2)])
    q, q2 = (c.normal(2, 11, 8, 128).cuda() for _ in range(2))
    kn, vn = c.normal(2, 11, 2, 128).cuda(), c.normal(2, 11, 2, 128).cuda()
    want = J.tree_attend(q, c.k, c.v, c.bt, c.seq_lens, par, kn, vn)
    want2 = J.tree_attend(q2, c.k, c.v, c.bt, c.seq_lens, par, kn, vn)
    graphs, outs = [], []
    for x in (q, q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(J.tree_attend(x, c.k, c.v, c.bt, c.seq_lens, par, kn, vn))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for s, g in zip(streams, graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want2)
        for o in outs:
            o.zero_()


# ------------------------------------------------------------------------------------------------
# commit
# ------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("d,code", [(128, 16), (128, 32), (128, 64), (256, 64), (128, 0), (256, "bf16")])
@pytest.mark.parametrize("head_major", [False, True])
def test_tree_commit(d, code, head_major):
    J = jssa()
    lens = [0, 5, 31, 16, 100]
    c = Paged(lens, 64, 3, d, 16, seed=d, head_major=head_major)
    c.k.nan_to_num_(), c.v.nan_to_num_()
    c.k.copy_(c.normal(*c.k.shape)), c.v.copy_(c.normal(*c.v.shape))
    sc = None
    if code == "bf16":
        sc = c.normal(c.k.shape[0], 3, 16, 32).cuda()
    elif code:
        sc = torch.randint(0, 256, (c.k.shape[0], 3, 16, code), dtype=torch.uint8, device="cuda")
    path = np.full((5, 64), -1)
    n_path = [0, 1, 64, 7, 3]
    path[1, :1] = [63]
    path[2] = np.arange(64)[::-1]      # any order
    path[3, :7] = [0, 1, 3, 4, 9, 20, 63]
    path[4, :3] = [5, 5, 0]            # a node twice
    k0, v0, s0 = c.k.clone(), c.v.clone(), None if sc is None else sc.clone()
    out = J.tree_commit(c.k, c.v, c.bt, c.seq_lens, cuda(path), cuda(n_path), sc)
    assert out.tolist() == [a + b for a, b in zip(lens, n_path)] and c.seq_lens.tolist() == lens
    k1, v1, s1 = k0.clone(), v0.clone(), None if sc is None else s0.clone()
    for b, L in enumerate(lens):
        for i in range(n_path[b]):
            src, dst = L + path[b, i], L + i
            a, z = (c.table[b, src // 16], src % 16), (c.table[b, dst // 16], dst % 16)
            k1[z], v1[z] = k0[a], v0[a]
            if sc is not None:
                s1[z[0], :, z[1]] = s0[a[0], :, a[1]]
    assert torch.equal(c.k, k1) and torch.equal(c.v, v1)
    assert sc is None or torch.equal(sc, s1)
    assert J.device_error() == 0


def test_tree_commit_flags_bad_inputs():
    J = jssa()
    c = Paged([10, 40, 20], 8, 1, seed=3)
    c.k.copy_(c.normal(*c.k.shape)), c.v.copy_(c.normal(*c.v.shape))
    k0 = c.k.clone()
    path = cuda([[2, 64, -1, 3], [4, 5, 6, 7], [1, 2, 3, 4]])
    table = c.table.copy()
    table[1, 44 // 16:] = -1
    out = J.tree_commit(c.k, c.v, cuda(table), c.seq_lens, path, cuda([4, 4, 99]))
    assert J.device_error() == 3 and out.tolist() == [14, 44, 24]
    k1 = k0.clone()
    for b, L, moves in ((0, 10, [(2, 0)]), (2, 20, [(1, 0), (2, 1), (3, 2), (4, 3)])):
        for s, t in moves:
            k1[c.table[b, (L + t) // 16], (L + t) % 16] = k0[c.table[b, (L + s) // 16], (L + s) % 16]
    k1[c.table[0, 13 // 16], 13 % 16] = k0[c.table[0, 13 // 16], 13 % 16]
    assert torch.equal(c.k, k1)


# ------------------------------------------------------------------------------------------------
# attention mass
# ------------------------------------------------------------------------------------------------


def check_mass(got, ref, before, slack):
    tol = slack * (ref - before) + 2.0 ** -22 * np.abs(ref)
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) - tol))
    assert np.array_equal(got[ref == before], before[ref == before])


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("g", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("window", [-1, 1, 70])
def test_dense_mass(g, d, window):
    J = jssa()
    c = Paged([0, 1, 63, 64, 65, 333], 0, 2, d, seed=g)
    q = c.normal(6, 2 * g, d) * 2
    cap = c.table.shape[1] * 16
    mass = torch.rand((6, 2, cap + 5), device="cuda")
    m0 = f64(mass)
    scale = 1 / math.sqrt(d)
    out = J.dense_decode(q.cuda(), c.k, c.v, c.bt, c.seq_lens, window=window, mass=mass)
    plain = J.dense_decode(q.cuda(), c.k, c.v, c.bt, c.seq_lens, window=window)
    ref, mref = C.mass_step(f64(q), f64(c.k), f64(c.v), c.table, c.lens, scale, m0, window)
    slack = fp32_slack(f64(q), f64(c.k), d, scale)
    check_mass(f64(mass), mref, m0, slack)
    assert np.max(np.abs(f64(out) - ref)) <= 1e-2 and torch.equal(out[0], torch.zeros_like(out[0]))
    assert float((out.float() - plain.float()).abs().max()) <= 2 ** -6  # (merged in another order)
    # a second step adds to the first
    m1 = f64(mass)
    J.dense_decode(q.cuda(), c.k, c.v, c.bt, c.seq_lens, window=window, mass=mass)
    check_mass(f64(mass), m1 + (mref - m0), m1, slack)
    assert J.device_error() == 0


@pytest.mark.parametrize("d,g", [(128, 4), (256, 2), (128, 3)])
def test_dense_mass_long(d, g):
    # many splits and several position blocks per pair
    J = jssa()
    gen = torch.Generator(device="cuda").manual_seed(d)
    L, h_kv, ps = 9001, 2, 16
    per = -(-L // ps)
    bt = torch.randperm(2 * per, generator=gen, device="cuda").view(2, per).int()
    k, v = (torch.empty((2 * per, ps, h_kv, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
            for _ in range(2))
    q = torch.empty((2, h_kv * g, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) * 2
    lens = [L, 1030]
    mass = torch.zeros((2, h_kv, per * ps), device="cuda")
    out = J.dense_decode(q, k, v, bt, cuda(lens), mass=mass)
    scale = 1 / math.sqrt(d)
    slack = 2 * (d * 2.0 ** -23 * scale * float(q.abs().sum(-1).max()) * float(k.abs().max()) + 2.0 ** -20)
    for b in range(2):
        pos = torch.arange(lens[b], device="cuda")
        page = bt[b].long()[pos // ps]
        for h in range(h_kv):
            p = torch.softmax(q[b, h * g:(h + 1) * g].double() @ k[page, pos % ps, h].double().T * scale, 1)
            w = p.sum(0)
            got = mass[b, h].double()
            assert bool(((got[:lens[b]] - w).abs() <= (slack + 2.0 ** -22) * w).all())
            assert torch.count_nonzero(got[lens[b]:]).item() == 0
            o = p @ v[page, pos % ps, h].double()
            a = p @ v[page, pos % ps, h].double().abs()
            err = (out[b, h * g:(h + 1) * g].double() - o).abs()
            assert bool((err <= 2.0 ** -8 * o.abs() + (2.0 ** -14 + slack) * a).all())


@pytest.mark.parametrize("budget", [1, 64, 100, 1500])
def test_indexed_mass(budget):
    J = jssa()
    c = Paged([0, 1, 90, 1700], 0, 2, 128, seed=budget)
    g, d = 4, 128
    q = c.normal(4, 8, d) * 2
    idx, count = np.full((4, 2, budget), -1), np.zeros((4, 2), dtype=np.int64)
    for b, L in enumerate(c.lens):
        for h in range(2):
            count[b, h] = min(L, budget)
            idx[b, h, :count[b, h]] = np.sort(c.rng.permutation(L)[:count[b, h]])
    mass = torch.rand((4, 2, c.table.shape[1] * 16), device="cuda")
    m0, scale = f64(mass), 1 / math.sqrt(d)
    out = J.indexed_attend(q.cuda(), c.k, c.v, c.bt, cuda(idx), cuda(count), mass=mass)
    ref, mref = C.mass_step(f64(q), f64(c.k), f64(c.v), c.table, c.lens, scale, m0, -1, idx, count)
    check_mass(f64(mass), mref, m0, fp32_slack(f64(q), f64(c.k), d, scale))
    assert np.max(np.abs(f64(out) - ref)) <= 1e-2
    assert J.device_error() == 0


def test_mass_skips_unusable_pages():
    J = jssa()
    c = Paged([100], 0, 1, 128, seed=2)
    q = c.normal(1, 4, 128)
    table = c.table.copy()
    table[0, 2] = 10 ** 6
    mass = torch.zeros((1, 1, c.table.shape[1] * 16), device="cuda")
    J.dense_decode(q.cuda(), c.k, c.v, cuda(table), c.seq_lens, mass=mass)
    assert J.device_error() == 1
    assert torch.count_nonzero(mass[0, 0, 32:48]).item() == 0
    assert abs(float(mass.sum()) - 4.0) < 1e-5


def test_mass_calls_share_nothing():
    # two captured calls replayed at once on two streams, and an eager call with a given workspace
    J = jssa()
    c = Paged([700, 64], 0, 2, seed=8)
    q = [c.normal(2, 8, 128).cuda() for _ in range(2)]
    zero = torch.zeros((2, 2, c.table.shape[1] * 16), device="cuda")
    want, mass, graphs = [], [zero.clone() for _ in q], []
    ws = J.Workspace("cuda")
    for x in q:
        m = zero.clone()
        want.append((J.dense_decode(x, c.k, c.v, c.bt, c.seq_lens, mass=m, ws=ws), m))
    outs = []
    for x, m in zip(q, mass):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(J.dense_decode(x, c.k, c.v, c.bt, c.seq_lens, mass=m))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(4):
        for m in mass:
            m.zero_()
        for s, g in zip(streams, graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (o, m), got, gm in zip(want, outs, mass):
            assert torch.equal(o, got) and torch.equal(m, gm)


# ------------------------------------------------------------------------------------------------
# eviction
# ------------------------------------------------------------------------------------------------


def run_evict(c, mass, keep, recent, code=32, in_place=False, table=None):
    J = jssa()
    B, cap = len(c.lens), mass.shape[2]
    c.k.copy_(c.normal(*c.k.shape)), c.v.copy_(c.normal(*c.v.shape))
    sc = None
    if code:
        sc = torch.randint(0, 256, (c.k.shape[0], c.h_kv, c.ps, code), dtype=torch.uint8, device="cuda")
    dst = mass_out = None
    if not in_place:
        per = -(-keep // c.ps)
        n0 = c.k.shape[0]
        grow = lambda t: torch.cat([t, torch.zeros((B * per + 1, *t.shape[1:]), dtype=t.dtype, device="cuda")])  # noqa: E731
        c.k, c.v = grow(c.k), grow(c.v)
        sc = None if sc is None else grow(sc)
        dst = n0 + c.rng.permutation(B * per).reshape(B, per)
        mass_out = torch.full_like(mass, 7.0)
    k0, v0, s0, m0 = c.k.clone(), c.v.clone(), None if sc is None else sc.clone(), mass.clone()
    idx, count, lens = J.evict(mass, c.k, c.v, c.bt, c.seq_lens, keep, recent, sc,
                               None if dst is None else cuda(dst), mass_out)
    k1, v1, s1 = k0.clone(), v0.clone(), None if sc is None else s0.clone()
    m1 = m0.clone() if in_place else torch.full_like(mass, 7.0)
    to = c.table if in_place else dst
    hm = mass.cpu().numpy() if not in_place else m0.cpu().numpy()
    for b, L in enumerate(c.lens):
        assert int(lens[b]) == min(L, keep)
        for h in range(c.h_kv):
            want = C.kept_positions(hm[b, h], L, keep, recent)
            assert int(count[b, h]) == len(want)
            got = idx[b, h].cpu().numpy()
            assert np.array_equal(got[:len(want)], want) and np.all(got[len(want):] == -1)
            w = torch.as_tensor(want).cuda()
            i = torch.arange(len(want), device="cuda")
            sp, dp = c.bt[b].long()[w // c.ps], torch.as_tensor(to[b]).cuda()[i // c.ps]
            k1[dp, i % c.ps, h] = k0[sp, w % c.ps, h]
            v1[dp, i % c.ps, h] = v0[sp, w % c.ps, h]
            if sc is not None:
                s1[dp, h, i % c.ps] = s0[sp, h, w % c.ps]
            m1[b, h, :L] = 0
            m1[b, h, :len(want)] = m0[b, h, w]
    assert torch.equal(c.k, k1) and torch.equal(c.v, v1)
    assert sc is None or torch.equal(sc, s1)
    got = mass if in_place else mass_out
    assert torch.equal(torch.nan_to_num(got, nan=-3.0), torch.nan_to_num(m1, nan=-3.0))
    assert in_place or torch.equal(torch.nan_to_num(mass), torch.nan_to_num(m0))
    assert c.seq_lens.tolist() == c.lens and J.device_error() == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (16, 0), (16, 5), (100, 100), (257, 31), (1000, 8)])
def test_evict(keep, recent, in_place):
    c = Paged([0, 1, 15, 16, 17, 300, 999], 0, 2, 128, pages=63, seed=keep)
    mass = torch.rand((7, 2, 63 * 16), device="cuda") ** 8
    run_evict(c, mass, keep, recent, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("d,code,head_major,ps", [(128, 16, False, 8), (128, 64, True, 16), (256, 64, False, 32),
                                                   (256, 0, True, 16), (128, 0, False, 64)])
def test_evict_layouts(d, code, head_major, ps, in_place):
    c = Paged([500, 130, 64], 0, 3, d, ps, pages=512 // ps, seed=ps, head_major=head_major)
    mass = torch.rand((3, 3, 512 + 8), device="cuda")
    run_evict(c, mass, 128, 16, code, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_ties_and_odd_values(in_place):
    c = Paged([200] * 6, 0, 1, 128, seed=5)
    m = torch.zeros((6, 1, 208))
    m[1] = 1.0
    m[2, 0, ::3] = 2.0
    m[3] = torch.randint(0, 3, (208,)).float()
    m[3, 0, [7, 50]] = NAN
    m[3, 0, [9, 60]] = math.inf
    m[3, 0, [11, 61]] = -math.inf
    m[4] = torch.where(torch.arange(208) % 2 == 0, 0.0, -0.0)  # the same value: ties
    m[5] = torch.arange(208).float() * 1e-41                   # denormals
    run_evict(c, m.cuda(), 70, 6, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,L,keep", [(1, 40000, 9000), (3, 20011, 2048), (40, 3000, 500)])
def test_evict_long(batch, L, keep, in_place):
    c = Paged([1] * batch, 0, 2 if batch < 40 else 4, 128, pages=-(-L // 16), seed=L)
    c.lens = [L - 17 * b for b in range(batch)]
    c.seq_lens = cuda(c.lens)
    mass = torch.rand((batch, c.h_kv, c.table.shape[1] * 16), device="cuda") ** 16
    run_evict(c, mass, keep, 64, in_place=in_place)


def test_evict_into_unusable_pages():
    J = jssa()
    c = Paged([100, 100], 0, 1, 128, seed=1)
    c.k.copy_(c.normal(*c.k.shape)), c.v.copy_(c.normal(*c.v.shape))
    mass = torch.rand((2, 1, c.table.shape[1] * 16), device="cuda")
    k0 = c.k.clone()
    idx, count, lens = J.evict(mass, c.k, c.v, c.bt, c.seq_lens, 32, 4,
                               dst_block_table=cuda([[-1, -1], [10 ** 6, -1]]),
                               mass_out=torch.zeros_like(mass))
    assert J.device_error() == 1 and torch.equal(c.k, k0) and count.tolist() == [[32], [32]]


def test_arguments_are_checked():
    J = jssa()
    c = Paged([40, 20], 8, 2)
    q = c.normal(2, 8, 4, 128).cuda()
    par = cuda([list(range(-1, 7))] * 2)
    mass = torch.zeros((2, 2, c.table.shape[1] * 16), device="cuda")
    with pytest.raises(ValueError):
        J.tree_attend(q, c.k, c.v, c.bt, c.seq_lens, par[:, :7].contiguous())
    with pytest.raises(ValueError):
        J.tree_attend(q, c.k, c.v, c.bt[:1].contiguous(), c.seq_lens, par)
    with pytest.raises(TypeError):
        J.tree_attend(q.half(), c.k, c.v, c.bt, c.seq_lens, par)
    with pytest.raises(ValueError):
        J.tree_attend(q, c.k, c.v, c.bt, c.seq_lens, par, k_new=c.normal(2, 8, 2, 128).cuda())
    with pytest.raises(ValueError):
        J.tree_attend(q, c.k, c.v, c.bt, c.seq_lens, par.cpu())
    with pytest.raises(J.JSSAError):
        J.tree_attend(q.repeat(1, 9, 1, 1), c.k, c.v, c.bt, c.seq_lens, par.repeat(1, 9))
    with pytest.raises(ValueError):
        J.evict(mass[:, :1].contiguous(), c.k, c.v, c.bt, c.seq_lens, 8)
    with pytest.raises(ValueError):
        J.evict(mass[..., :-1].contiguous(), c.k, c.v, c.bt, c.seq_lens, 8)
    with pytest.raises(J.JSSAError):
        J.evict(mass, c.k, c.v, c.bt, c.seq_lens, 8, 9)
    with pytest.raises(J.JSSAError):
        J.evict(mass, c.k, c.v, c.bt, c.seq_lens, 8, lens=c.seq_lens)
    with pytest.raises(ValueError):
        J.dense_decode(q[:, 0].contiguous(), c.k, c.v, c.bt, c.seq_lens, mass=mass[:1])
    with pytest.raises(ValueError):
        J.tree_commit(c.k, c.v, c.bt, c.seq_lens, par[:1].contiguous(), cuda([1, 1]))
    assert torch.count_nonzero(mass).item() == 0


# ------------------------------------------------------------------------------------------------
# together, through PagedLayer
# ------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("sparse", [False, True])
def test_draft_commit_step_evict(sparse):
    # a layer's life: a drafted tree, its accepted path, steps that keep the mass, an eviction, and
    # another tree over the shortened cache
    J = jssa()
    from parity import check_output
    lens, h_kv, g, d, r, budget, n = [300, 77], 2, 4, 128, 32, 64, 9
    c = Paged(lens, 40, h_kv, d, seed=20)
    c.k.nan_to_num_(0.0), c.v.nan_to_num_(0.0)
    m = torch.linalg.qr(torch.randn((h_kv, d, r), generator=torch.Generator().manual_seed(1)))[0]
    layer = J.PagedLayer(c.k, c.v, c.bt, c.seq_lens, m.transpose(1, 2).contiguous().cuda(), budget,
                         track_mass=True)
    layer.prefill_scores()
    rng, scale = c.rng, 1 / math.sqrt(d)
    for rounds in range(2):
        parents = [random_tree(rng, n, unused=b) for b in range(2)]
        q, kn, vn = c.normal(2, n, h_kv * g, d), c.normal(2, n, h_kv, d), c.normal(2, n, h_kv, d)
        now = layer.seq_lens.tolist()
        out = layer.draft(q.cuda(), kn.cuda(), vn.cuda(), cuda(parents), sparse=sparse)
        idx = layer.idx.cpu().numpy() if sparse else None
        cnt = layer.count.cpu().numpy() if sparse else None
        ref, mag = C.tree_attend(f64(q), f64(c.k), f64(c.v), c.table, now, parents, scale, -1, idx, cnt)
        check_out(out, ref, mag, fp32_slack(f64(q), f64(c.k), d, scale))
        # the accepted path: the deepest node of each tree
        anc = [C.ancestors(p) for p in parents]
        paths = [max(a, key=len) for a in anc]
        path = np.full((2, n), -1)
        for b, p in enumerate(paths):
            path[b, :len(p)] = p
        layer.commit(cuda(path), cuda([len(p) for p in paths]))
        assert layer.seq_lens.tolist() == [a + len(p) for a, p in zip(now, paths)]
        # the committed rows' scoring codes are those of a fresh store
        codes = layer.score_cache.clone()
        layer.prefill_scores()
        for b, L in enumerate(layer.seq_lens.tolist()):
            t = torch.arange(L, device="cuda")
            pg = c.bt[b].long()[t // 16]
            assert torch.equal(codes[pg, :, t % 16], layer.score_cache[pg, :, t % 16])
        for b, p in enumerate(paths):
            for i, node in enumerate(p):
                t = now[b] + i
                assert torch.equal(c.k[c.table[b, t // 16], t % 16].cpu(), kn[b, node])
        # decode steps that keep the mass
        before = layer.mass.clone()
        for _ in range(2):
            layer.seq_lens += 1
            qs, ks, vs = c.normal(2, h_kv * g, d), c.normal(2, h_kv, d), c.normal(2, h_kv, d)
            m0 = f64(layer.mass)
            o, idx, cnt = layer.step(qs.cuda(), ks.cuda(), vs.cuda())
            ref, mref = C.mass_step(f64(qs), f64(c.k), f64(c.v), c.table, layer.seq_lens.tolist(),
                                    scale, m0, -1, idx.cpu().numpy(), cnt.cpu().numpy())
            check_output(f64(o), ref)
            check_mass(f64(layer.mass), mref, m0, fp32_slack(f64(qs), f64(c.k), d, scale))
            m0 = f64(layer.mass)
            o = layer.dense(qs.cuda())
            ref, mref = C.mass_step(f64(qs), f64(c.k), f64(c.v), c.table, layer.seq_lens.tolist(),
                                    scale, m0)
            check_output(f64(o), ref)
            check_mass(f64(layer.mass), mref, m0, fp32_slack(f64(qs), f64(c.k), d, scale))
        assert float((layer.mass - before).sum()) == pytest.approx(2 * 2 * 2 * h_kv * g, rel=1e-4)
        # eviction
        mass, k0, now = layer.mass.cpu().numpy(), c.k.clone(), layer.seq_lens.tolist()
        idx, count = layer.evict(64, 8)
        for b in range(2):
            for h in range(h_kv):
                want = C.kept_positions(mass[b, h], now[b], 64, 8)
                assert np.array_equal(idx[b, h, :len(want)].cpu().numpy(), want)
                for i in (0, len(want) // 2, len(want) - 1):
                    t = want[i]
                    assert torch.equal(c.k[c.table[b, i // 16], i % 16, h],
                                       k0[c.table[b, t // 16], t % 16, h])
        assert layer.seq_lens.tolist() == [min(64, x) for x in now]
        assert torch.count_nonzero(layer.mass[:, :, 64:]).item() == 0
    assert J.device_error() & ~16 == 0


@pytest.mark.parametrize("d,n,g", [(128, 12, 4), (128, 64, 4), (256, 12, 4)])
def test_tree_wait_timeout_then_recovery(d, n, g):
    # a wait limit of one clock cycle: waits of a correct launch run out, the flag is raised, the
    # call drains and returns; with the default limit the next call is correct and clean
    J = jssa()
    c = Paged([1500, 70], n, 2, d, seed=21)
    parents = [random_tree(c.rng, n) for _ in range(2)]
    q, kn, vn = c.normal(2, n, 2 * g, d).cuda(), c.normal(2, n, 2, d).cuda(), c.normal(2, n, 2, d).cuda()
    want = J.tree_attend(q, c.k, c.v, c.bt, c.seq_lens, cuda(parents), kn, vn)
    assert J.device_error(clear=True) == 0
    J.set_wait_limit(1)
    try:
        J.tree_attend(q, c.k, c.v, c.bt, c.seq_lens, cuda(parents), kn, vn)
        torch.cuda.synchronize()
    finally:
        J.set_wait_limit(0)
    assert J.device_error(clear=True) & 32
    out = J.tree_attend(q, c.k, c.v, c.bt, c.seq_lens, cuda(parents), kn, vn)
    assert torch.equal(out, want) and J.device_error(clear=True) == 0


@pytest.mark.parametrize("pages,mass_apart", [("same", True), ("other", False)])
@pytest.mark.parametrize("batch,L,keep", [(2, 700, 150), (1, 30000, 5000)])
def test_evict_half_in_place(pages, mass_apart, batch, L, keep):
    # the pages move in place but not the mass, or the other way round
    J = jssa()
    c = Paged([1] * batch, 0, 2, 128, pages=-(-L // 16), seed=keep)
    c.lens = [L - 30 * b for b in range(batch)]
    lens = cuda(c.lens)
    c.k.copy_(c.normal(*c.k.shape)), c.v.copy_(c.normal(*c.v.shape))
    mass = torch.rand((batch, 2, c.table.shape[1] * 16), device="cuda") ** 6
    m0, k0 = mass.clone(), c.k.clone()
    mass_out = torch.full_like(mass, 5.0) if mass_apart else mass
    dst, n0 = None, c.k.shape[0]
    table = c.table
    if pages == "other":
        per = -(-keep // 16)
        c.k, c.v = (torch.cat([t, torch.zeros((batch * per, *t.shape[1:]), dtype=t.dtype, device="cuda")])
                    for t in (c.k, c.v))
        table = n0 + np.arange(batch * per).reshape(batch, per)
        dst = cuda(table)
    idx, count, _ = J.evict(mass, c.k, c.v, c.bt, lens, keep, 9, dst_block_table=dst, mass_out=mass_out)
    for b, n in enumerate(c.lens):
        for h in range(2):
            want = C.kept_positions(m0[b, h].cpu().numpy(), n, keep, 9)
            assert np.array_equal(idx[b, h].cpu().numpy(), want)
            w, i = torch.as_tensor(want).cuda(), torch.arange(keep, device="cuda")
            to = torch.as_tensor(table[b]).cuda()[i // 16]
            assert torch.equal(c.k[to, i % 16, h], k0[c.bt[b].long()[w // 16], w % 16, h])
            assert torch.equal(mass_out[b, h, :keep], m0[b, h, w])
            assert torch.count_nonzero(mass_out[b, h, keep:n]).item() == 0
    if pages == "other":
        assert torch.equal(c.k[:n0], k0)
    if mass_apart:
        assert torch.equal(mass, m0)
    assert J.device_error() == 0


def test_calls_at_once_on_two_streams():
    # eager calls of every operator on two streams, each on its own data, nothing waited for
    J = jssa()
    cs = [Paged([900, 333], 16, 2, seed=30 + i) for i in range(2)]
    for c in cs:
        c.k.nan_to_num_(0.25), c.v.nan_to_num_(0.25)
    work = []
    for c in cs:
        work.append(dict(q=c.normal(2, 16, 8, 128).cuda(), kn=c.normal(2, 16, 2, 128).cuda(),
                         vn=c.normal(2, 16, 2, 128).cuda(),
                         par=cuda([random_tree(c.rng, 16) for _ in range(2)]),
                         path=cuda([[0, 2, 5, 9], [1, 3, 4, 15]]), n=cuda([4, 3])))

    def run(c, w, mass):
        o = [J.tree_attend(w["q"], c.k, c.v, c.bt, c.seq_lens, w["par"], w["kn"], w["vn"])]
        lens = J.tree_commit(c.k, c.v, c.bt, c.seq_lens, w["path"], w["n"])
        o.append(J.dense_decode(w["q"][:, 0].contiguous(), c.k, c.v, c.bt, lens, mass=mass))
        o += list(J.evict(mass, c.k, c.v, c.bt, lens, 100, 7))
        return o + [mass, c.k.clone(), c.v.clone()]

    def fresh(c):
        return torch.zeros((2, 2, c.table.shape[1] * 16), device="cuda")

    start = [(c.k.clone(), c.v.clone()) for c in cs]
    want = [run(c, w, fresh(c)) for c, w in zip(cs, work)]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, (k, v) in zip(cs, start):
            c.k.copy_(k), c.v.copy_(v)
        masses = [fresh(c) for c in cs]
        streams = [torch.cuda.Stream() for _ in cs]
        got = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for s, c, w, m in zip(streams, cs, work, masses):
            with torch.cuda.stream(s):
                got.append(run(c, w, m))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert J.device_error() == 0


def test_step_captured_and_replayed():
    # one graph of a whole round: draft, commit, a step with its mass, an eviction
    J = jssa()
    lens, h_kv, g, n = [200, 90], 2, 4, 8
    c = Paged(lens, 60, h_kv, 128, seed=40)
    c.k.nan_to_num_(0.0), c.v.nan_to_num_(0.0)
    m = torch.linalg.qr(torch.randn((h_kv, 128, 32), generator=torch.Generator().manual_seed(2)))[0]
    layer = J.PagedLayer(c.k, c.v, c.bt, c.seq_lens, m.transpose(1, 2).contiguous().cuda(), 64,
                         track_mass=True)
    layer.prefill_scores()
    q, kn, vn = (x.cuda() for x in (c.normal(2, n, h_kv * g, 128), c.normal(2, n, h_kv, 128),
                                    c.normal(2, n, h_kv, 128)))
    par = cuda([random_tree(c.rng, n) for _ in range(2)])
    path, n_path = cuda([[0, 1], [0, 3]]), cuda([2, 1])
    k1, v1 = kn[:, 0].contiguous(), vn[:, 0].contiguous()
    q1 = q[:, 0].contiguous()
    state = [c.k, c.v, layer.score_cache, layer.mass, layer.seq_lens]

    def once():
        a = layer.draft(q, kn, vn, par, sparse=True)
        layer.commit(path, n_path)
        layer.seq_lens += 1
        b = layer.step(q1, k1, v1)[0].clone()
        idx, count = layer.evict(60, 8)
        return [a, b, idx, count]

    start = [t.clone() for t in state]
    want = [t.clone() for t in once()] + [t.clone() for t in state]

    def reset():
        for t, s in zip(state, start):
            t.copy_(s)

    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()  # (workspaces of the layer)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = once()
    for _ in range(2):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, outs + state))


def test_draft_refuses_too_many_nodes():
    J = jssa()
    c = Paged([40], 80, 1, 128, seed=41)
    layer = J.PagedLayer(c.k, c.v, c.bt, c.seq_lens, torch.zeros((1, 32, 128), device="cuda"), 16)
    codes = layer.score_cache.clone()
    kn = c.normal(1, 65, 1, 128).cuda()
    with pytest.raises(ValueError):
        layer.draft(c.normal(1, 65, 4, 128).cuda(), kn, kn, cuda([list(range(-1, 64))]))
    assert torch.equal(layer.score_cache, codes)
    with pytest.raises(ValueError):
        layer.evict(8)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.05])
@pytest.mark.parametrize("g", [5, 6, 7])
def test_tree_attend_odd_groups_and_scales(g, scale, d):
    # a zero scale (the mean of the visible values) and a negative one; group sizes that are no power of 2
    c = Paged([150, 0, 63], 23, 2, d, seed=g)
    run_tree(c, 23, g, [random_tree(c.rng, 23, b) for b in range(3)], scale=scale)
    assert jssa().device_error() == 0
