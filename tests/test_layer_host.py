"""Host-side behaviour of the Python binding around the cache operators (no GPU, no launch)."""

import weakref

import pytest
import torch

from token_level_sparse_fp8_b200 import api


@pytest.fixture
def cpu_workspace(monkeypatch):
    """A workspace over host memory whose calls into the library do nothing."""
    state = {"capturing": False}
    monkeypatch.setattr(api, "call", lambda *a: None)
    monkeypatch.setattr(api, "_stream", lambda device: 0)
    monkeypatch.setattr(api, "_capturing", lambda: state["capturing"], raising=False)
    return api.Workspace("cpu"), state


def test_workspace_keeps_what_a_captured_graph_holds(cpu_workspace):
    ws, state = cpu_workspace
    state["capturing"] = True
    ws.get(1000)
    held = weakref.ref(ws.buf)
    ws.get(500)
    state["capturing"] = False
    ws.get(5000)  # replaces the buffer
    assert held() is not None and ws.buf.numel() == 5000
    dropped = weakref.ref(ws.buf)
    ws.get(9000)
    assert dropped() is None  # no graph was given that one
    assert held() is not None


def _decode_args(d=128, h_kv=2, r=32, batch=2):
    """Arguments of a decode step on host memory: (q, k_new, v_new, k, v, codes, basis, table, lens)."""
    bf = torch.bfloat16
    k = torch.zeros((6, 16, h_kv, d), dtype=bf)
    return dict(q=torch.zeros((batch, 4 * h_kv, d), dtype=bf), k_new=torch.zeros((batch, h_kv, d), dtype=bf),
                v_new=torch.zeros((batch, h_kv, d), dtype=bf), k_cache=k, v_cache=k.clone(),
                score_cache=torch.zeros((6, h_kv, 16, r), dtype=torch.uint8),
                basis=torch.zeros((h_kv, r, d)), block_table=torch.zeros((batch, 3), dtype=torch.int32),
                seq_lens=torch.ones((batch,), dtype=torch.int32))


@pytest.fixture
def no_launch(monkeypatch):
    """Arguments may be on the host; a call that gets as far as the library fails the test."""
    def launched(*a, **k):
        raise AssertionError("the call was not refused")

    monkeypatch.setattr(api, "_need", lambda *a, **k: None)
    for name in ("call", "_call_on", "_ws", "_scratch", "_caches", "_table", "_arg", "_same_device"):
        monkeypatch.setattr(api, name, launched)


@pytest.mark.parametrize("with_mass", [False, True])
@pytest.mark.parametrize("q_dim,cache_dim", [(256, 128), (128, 256)])
def test_attention_refuses_another_head_dim(no_launch, q_dim, cache_dim, with_mass):
    # rows of another length would be read past their ends
    a = _decode_args(cache_dim)
    q = torch.zeros((2, 8, q_dim), dtype=torch.bfloat16)
    mass = torch.zeros((2, 2, 48)) if with_mass else None
    idx, count = torch.zeros((2, 2, 8), dtype=torch.int32), torch.ones((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="head dim"):
        api.dense_decode(q, a["k_cache"], a["v_cache"], a["block_table"], a["seq_lens"], mass=mass)
    with pytest.raises(ValueError, match="head dim"):
        api.indexed_attend(q, a["k_cache"], a["v_cache"], a["block_table"], idx, count, mass=mass)
    with pytest.raises(ValueError, match="head dim"):
        api.decode(**{**a, "q": q}, budget=8, mass=mass)


@pytest.mark.parametrize("with_mass", [False, True])
@pytest.mark.parametrize("name,shape", [
    ("v_cache", (5, 16, 2, 128)), ("score_cache", (5, 2, 16, 32)), ("score_cache", (6, 2, 8, 32)),
    ("score_cache", (6, 2, 16, 16)), ("basis", (1, 32, 128)), ("basis", (2, 32, 64)),
    ("k_new", (1, 2, 128)), ("v_new", (2, 1, 128)),
])
def test_decode_refuses_other_shapes(no_launch, name, shape, with_mass):
    a = _decode_args()
    a[name] = torch.zeros(shape, dtype=a[name].dtype)
    with pytest.raises(ValueError, match="shape|agree"):
        api.decode(**a, budget=8, mass=torch.zeros((2, 2, 48)) if with_mass else None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), -2), (dict(batch=-1), -2), (dict(n=65), -3), (dict(n=0, mean=None), 0), (dict(batch=0), 0),
    (dict(parents=None), -1), (dict(bt=None), -1), (dict(lens=None), -1), (dict(slots=None), -1),
    (dict(q=None), -1), (dict(q=0x1008), -4), (dict(mean=0x6008), -4), (dict(d=96), -3), (dict(h_q=0), -2),
    (dict(h_q=1 << 20), -3), (dict(ps=24), -3), (dict(max_pages=0), -2), (dict(num_pages=0), -2),
])
def test_tree_prepare_refuses(kw, status):
    from token_level_sparse_fp8_b200 import _lib, build
    build.build()
    a = dict(q=0x1000, parents=0x2000, bt=0x3000, max_pages=8, lens=0x4000, batch=2, n=8, h_q=8, d=128,
             num_pages=20, ps=16, slots=0x5000, mean=0x6000)
    a.update(kw)
    assert _lib.load().jssa_tree_prepare(
        a["q"], a["parents"], a["bt"], a["max_pages"], a["lens"], a["batch"], a["n"], a["h_q"], a["d"],
        a["num_pages"], a["ps"], a["slots"], a["mean"], None) == status


def test_host_pipeline_refuses_a_layer_that_keeps_the_mass():
    # its steps would leave the mass behind, and a later eviction would go by stale sums
    class Layer:
        mass = torch.zeros((1, 1, 16))

    with pytest.raises(ValueError, match="mass"):
        api.HostPipeline(Layer(), (1, 4, 128), (1, 1, 128))


def test_decode_accepts_caches_with_more_pages(monkeypatch):
    # a pool of codes or values that is larger than K's holds every row the call names
    reached = []
    monkeypatch.setattr(api, "_need", lambda *a, **k: None)
    monkeypatch.setattr(api, "_ws", lambda *a, **k: reached.append(1) or (_ for _ in ()).throw(KeyError))
    a = _decode_args()
    a["v_cache"] = torch.zeros((9, 16, 2, 128), dtype=torch.bfloat16)
    a["score_cache"] = torch.zeros((7, 2, 16, 32), dtype=torch.uint8)
    with pytest.raises(KeyError):
        api.decode(**a, budget=8)
    assert reached
