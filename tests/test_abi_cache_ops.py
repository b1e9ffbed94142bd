"""Host-side refusals of the cache-maintenance entry points (nothing is launched)."""

import ctypes

import pytest

OK, NULL, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE = 0, -1, -2, -3, -4, -5
F = ctypes.c_float(0.1)
STRIDES = (16 * 2 * 128, 2 * 128, 128)


@pytest.fixture(scope="module")
def lib():
    from token_level_sparse_fp8_b200 import build, _lib
    build.build()
    return _lib.load()


def _tree(lib, **kw):
    a = dict(q=0x1000, k_new=None, v_new=None, k=0x2000, v=0x3000, strides=STRIDES, bt=0x4000,
             max_pages=8, lens=0x5000, parents=0x6000, idx=None, count=None, batch=2, n=8, h_q=8,
             h_kv=2, d=128, budget=0, num_pages=20, ps=16, window=-1, out=0x7000, ws=0x8000,
             ws_bytes=1 << 40)
    a.update(kw)
    return lib.jssa_tree_attend(a["q"], a["k_new"], a["v_new"], a["k"], a["v"], *a["strides"],
                                a["bt"], a["max_pages"], a["lens"], a["parents"], a["idx"],
                                a["count"], a["batch"], a["n"], a["h_q"], a["h_kv"], a["d"],
                                a["budget"], a["num_pages"], a["ps"], a["window"], F, a["out"],
                                a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), SHAPE), (dict(n=65), UNSUPPORTED), (dict(n=0), OK), (dict(batch=0), OK),
    (dict(batch=-1), SHAPE), (dict(batch=-1, n=0), SHAPE), (dict(d=96), UNSUPPORTED),
    (dict(h_q=7), SHAPE), (dict(h_q=18), UNSUPPORTED), (dict(ps=24), UNSUPPORTED),
    (dict(q=None), NULL), (dict(parents=None), NULL), (dict(lens=None), NULL), (dict(k=None), NULL),
    (dict(bt=None), NULL), (dict(out=None), NULL), (dict(k_new=0x9000), NULL),
    (dict(idx=0x9000, budget=64), NULL), (dict(idx=0x9000, count=0x9100, budget=0), SHAPE),
    (dict(idx=0x9000, count=0x9100, budget=64, window=4), SHAPE),
    (dict(q=0x1008), ALIGN), (dict(out=0x7002), ALIGN), (dict(k=0x2008), ALIGN),
    (dict(k_new=0x9008, v_new=0x9100), ALIGN), (dict(strides=(4097, 256, 128)), ALIGN),
    (dict(strides=(0, 256, 128)), SHAPE), (dict(batch=40000), UNSUPPORTED),
])
def test_tree_attend_refuses(lib, kw, status):
    assert _tree(lib, **kw) == status


def _evict(lib, **kw):
    a = dict(mass=0x1000, ms=128, k=0x2000, v=0x3000, strides=STRIDES, sc=0x4000, sb=32, bt=0x5000,
             max_pages=8, dst=0x6000, dst_pages=8, lens=0x7000, batch=2, h_kv=2, d=128,
             num_pages=20, ps=16, keep=16, recent=4, idx=0x8000, count=0x9000, mo=0xA000,
             lo=0xB000)
    a.update(kw)
    return lib.jssa_evict(a["mass"], a["ms"], a["k"], a["v"], *a["strides"], a["sc"], a["sb"],
                          a["bt"], a["max_pages"], a["dst"], a["dst_pages"], a["lens"], a["batch"],
                          a["h_kv"], a["d"], a["num_pages"], a["ps"], a["keep"], a["recent"],
                          a["idx"], a["count"], a["mo"], a["lo"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(keep=0), SHAPE), (dict(recent=-1), SHAPE), (dict(recent=17), SHAPE), (dict(batch=0), OK),
    (dict(batch=-1), SHAPE), (dict(h_kv=0), SHAPE), (dict(d=576), UNSUPPORTED),
    (dict(sb=24), UNSUPPORTED), (dict(sb=128), UNSUPPORTED), (dict(ms=127), SHAPE),
    (dict(mass=None), NULL), (dict(mo=None), NULL), (dict(idx=None), NULL), (dict(count=None), NULL),
    (dict(dst=None), NULL), (dict(lens=None), NULL), (dict(lo=None), NULL), (dict(k=None), NULL),
    (dict(lo=0x7000), SHAPE), (dict(dst=0x5000, dst_pages=4), SHAPE), (dict(dst_pages=0), SHAPE),
    (dict(sc=0x4008), ALIGN), (dict(mass=0x1002), ALIGN), (dict(v=0x3008), ALIGN),
    (dict(batch=40000), UNSUPPORTED),
])
def test_evict_refuses(lib, kw, status):
    assert _evict(lib, **kw) == status


def _commit(lib, **kw):
    a = dict(k=0x2000, v=0x3000, strides=STRIDES, sc=0x4000, sb=32, bt=0x5000, max_pages=8,
             lens=0x7000, path=0x8000, n_path=0x9000, max_path=8, batch=2, h_kv=2, d=128,
             num_pages=20, ps=16, lo=0xB000)
    a.update(kw)
    return lib.jssa_tree_commit(a["k"], a["v"], *a["strides"], a["sc"], a["sb"], a["bt"],
                                a["max_pages"], a["lens"], a["path"], a["n_path"], a["max_path"],
                                a["batch"], a["h_kv"], a["d"], a["num_pages"], a["ps"], a["lo"],
                                None)


@pytest.mark.parametrize("kw,status", [
    (dict(max_path=65), UNSUPPORTED), (dict(max_path=-1), SHAPE), (dict(batch=0), OK),
    (dict(path=None), NULL), (dict(n_path=None), NULL), (dict(lo=0x7000), SHAPE),
    (dict(lo=None), NULL), (dict(sb=8), UNSUPPORTED), (dict(v=None), NULL), (dict(sc=0x4004), ALIGN),
    (dict(d=64), UNSUPPORTED), (dict(ps=0), SHAPE),
])
def test_tree_commit_refuses(lib, kw, status):
    assert _commit(lib, **kw) == status


def test_mass_forms_refuse(lib):
    base = (0x1000, 0x2000, 0x3000, *STRIDES, 0x4000, 8)
    big = 1 << 40

    def dense(mass=0x6000, stride=128, h_q=8, batch=2, ws=0x9000, n=big):
        return lib.jssa_dense_decode_mass(*base, 0x5000, batch, h_q, 2, 128, 20, 16, -1, F, mass,
                                          stride, 0x8000, ws, n, None)

    def indexed(mass=0x6000, stride=128, idx=0x5000, budget=32, ws=0x9000, n=big):
        return lib.jssa_indexed_attend_mass(*base, idx, 0x5100, 2, 8, 2, 128, budget, 20, 16, F,
                                            mass, stride, 0x8000, ws, n, None)

    assert dense(mass=None) == NULL and dense(mass=0x6002) == ALIGN and dense(stride=127) == SHAPE
    assert dense(h_q=18) == UNSUPPORTED and dense(batch=0) == OK and dense(batch=40000) == UNSUPPORTED
    assert dense(ws=None) == WORKSPACE and dense(n=64) == WORKSPACE and dense(ws=0x9008) == ALIGN
    assert indexed(mass=None) == NULL and indexed(idx=None) == NULL and indexed(budget=0) == SHAPE
    assert indexed(stride=64) == SHAPE and indexed(n=64) == WORKSPACE
    st = lib.jssa_decode_mass(0x1000, None, None, 0x2000, 0x3000, *STRIDES, 0x4000, 0x5000, 0x6000, 8,
                              0x7000, 2, 8, 2, 128, 32, 20, 16, 32, F, None, 128, 0x8000, 0x9000,
                              0xA000, 0xB000, big, None)
    assert st == NULL


def test_workspace_sizes(lib):
    from token_level_sparse_fp8_b200 import api, _lib
    # the scores of every attended position: G floats per (sequence, KV head)
    n = api.workspace_size(_lib.FN_DENSE_DECODE_MASS, 2, 8, 2, 128, 64, 16, 0)
    assert n >= 2 * 2 * 64 * 16 * 4 * 4
    assert n > api.workspace_size(_lib.FN_DENSE_DECODE_MASS, 2, 8, 2, 128, 64, 16, 128)
    assert api.workspace_size(_lib.FN_DECODE_MASS, 2, 8, 2, 128, 64, 16, 128) >= (
        api.workspace_size(_lib.FN_INDEXED_ATTEND_MASS, 2, 8, 2, 128, 64, 16, 128)
        + api.workspace_size(_lib.FN_SCORE_TOPK, 2, 8, 2, 128, 64, 16, 128))
    with pytest.raises(_lib.JSSAError):
        api.workspace_size(_lib.FN_TREE_ATTEND, 2, 8, 2, 128, 64, 16, 65)
