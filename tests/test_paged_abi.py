"""Host-side refusals of the paged cache's entry points (no GPU needed: nothing here launches)."""
import ctypes

import pytest
import torch

FAKE = 1 << 20


@pytest.fixture(scope="module")
def hstu():
    import hstu_sequential_transduction_layer_b200 as m
    return m


def P(i):
    return FAKE + (i << 40)          # far apart: no overlap by chance


def cache_of(hstu, **kw):
    f = dict(num_pages=100, page_size=64, num_heads=2, head_dim=64, dtype=hstu.HSTU_BF16, k=P(1),
             v=P(2), positions=P(3), timestamps=P(4), weights=P(5))
    f.update(kw)
    return hstu.HstuPagedCache(**f)


def shape_of(hstu, **kw):
    f = dict(num_seqs=3, total_tokens=3, max_seq_len=500, d_model=128, num_heads=2, d_qk=64, d_v=64,
             dtype=hstu.HSTU_BF16, n_pos_buckets=16, n_time_buckets=8)
    f.update(kw)
    return hstu.make_shape(**f)


BAD_CACHES = [dict(num_pages=0), dict(num_pages=1 << 31), dict(page_size=24), dict(page_size=8),
              dict(page_size=2048), dict(page_size=0), dict(num_heads=0), dict(head_dim=0),
              dict(dtype=5), dict(k=None), dict(v=None), dict(k=P(1) + 8), dict(v=P(2) + 2),
              dict(positions=P(3) + 2), dict(timestamps=P(4) + 4), dict(weights=P(5) + 1)]


def append(hstu, cache=None, T=10, B=3, M=4, **kw):
    a = dict(uvqk=P(6), off=P(7), ts=P(8), table=P(9), lens=P(10), nxt=P(11))
    a.update(kw)
    c = cache or cache_of(hstu)
    return hstu.library().hstu_cache_append(ctypes.byref(c), B, T, a["uvqk"], a["off"], a["ts"],
                                            a["table"], M, a["lens"], a["nxt"], None)


def attend(hstu, cache=None, shape=None, M=9, append=1, scale=0.1, **kw):
    a = dict(uvqk=P(6), table=P(9), lens=P(10), nxt=P(11), now=P(8), pos=P(12), tim=P(13), ali=None,
             av=P(14), ws=P(15), ws_bytes=1 << 30)
    a.update(kw)
    c, s = cache or cache_of(hstu), shape or shape_of(hstu)
    return hstu.library().hstu_paged_attention_fwd(
        ctypes.byref(s), ctypes.byref(c), a["uvqk"], a["table"], M, a["lens"], a["nxt"], a["now"],
        a["pos"], a["tim"], a["ali"], scale, append, a["av"], a["ws"], a["ws_bytes"], None)


def layer(hstu, cache=None, shape=None, M=9, **kw):
    a = dict(X=P(6), table=P(9), lens=P(10), nxt=P(11), now=P(8), W1=P(16), b1=P(17), W2=P(18),
             b2=P(19), lnw=P(20), lnb=P(21), pos=P(12), tim=P(13), ali=None, out=P(14), ws=P(15),
             ws_bytes=1 << 30)
    a.update(kw)
    c, s = cache or cache_of(hstu), shape or shape_of(hstu)
    return hstu.library().hstu_paged_layer_fwd(
        ctypes.byref(s), ctypes.byref(c), a["X"], a["table"], M, a["lens"], a["nxt"], a["now"],
        a["W1"], a["b1"], a["W2"], a["b2"], a["lnw"], a["lnb"], a["pos"], a["tim"], a["ali"], 0.1, 1,
        a["out"], a["ws"], a["ws_bytes"], None)


def evict(hstu, cache=None, B=3, M=9, budget=100, recent=10, **kw):
    a = dict(table=P(9), lens=P(10), nxt=P(11), new=P(14), ws=P(15), ws_bytes=1 << 30)
    a.update(kw)
    c = cache or cache_of(hstu)
    return hstu.library().hstu_cache_evict(ctypes.byref(c), B, a["table"], M, a["lens"], a["nxt"],
                                           budget, recent, a["new"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("call", [append, attend, layer, evict], ids=lambda f: f.__name__)
def test_bad_caches(hstu, call):
    for bad in BAD_CACHES:
        assert call(hstu, cache=cache_of(hstu, **bad)) == hstu.HSTU_ERR_INVALID_ARG, bad
    for hd, dtype in ((32, hstu.HSTU_BF16), (96, hstu.HSTU_BF16), (16, hstu.HSTU_F32),
                      (256, hstu.HSTU_F32)):
        assert call(hstu, cache=cache_of(hstu, head_dim=hd, dtype=dtype)) == hstu.HSTU_ERR_UNSUPPORTED


def test_append_refusals(hstu):
    E = hstu.HSTU_ERR_INVALID_ARG
    assert append(hstu, T=-1) == E
    assert append(hstu, B=-1) == E
    assert append(hstu, B=0) == E                         # tokens without sequences
    for name in ("uvqk", "off", "table", "lens"):
        assert append(hstu, **{name: None}) == E, name
    assert append(hstu, ts=None) == E                     # the cache keeps timestamps
    assert append(hstu, uvqk=P(6) + 2) == E
    assert append(hstu, uvqk=P(1) + 4096) == E            # reads the cache's own K
    assert append(hstu, M=0) == E and append(hstu, M=-3) == E
    assert append(hstu, M=1 << 24) == hstu.HSTU_ERR_UNSUPPORTED          # 2^30 slots a row
    assert append(hstu, T=0) == hstu.HSTU_OK              # nothing to do
    assert append(hstu, T=0, B=0, table=None, lens=None) == hstu.HSTU_OK


def test_attention_refusals(hstu):
    E, U = hstu.HSTU_ERR_INVALID_ARG, hstu.HSTU_ERR_UNSUPPORTED
    assert attend(hstu, shape=shape_of(hstu, total_tokens=4)) == E        # one token a sequence
    assert attend(hstu, shape=shape_of(hstu, num_heads=3, d_model=192)) == E     # not the cache's heads
    assert attend(hstu, shape=shape_of(hstu, d_qk=128, d_v=128)) == E
    assert attend(hstu, shape=shape_of(hstu, d_qk=64, d_v=128)) == U
    assert attend(hstu, shape=shape_of(hstu, dtype=hstu.HSTU_F32)) == E
    assert attend(hstu, shape=shape_of(hstu, max_seq_len=0)) == E
    assert attend(hstu, shape=shape_of(hstu, num_seqs=1 << 30, total_tokens=1 << 30)) == U
    for name in ("uvqk", "table", "lens", "av", "ws"):
        assert attend(hstu, **{name: None}) == E, name
    assert attend(hstu, now=None) == E                    # the time table needs the tokens' times
    assert attend(hstu, now=None, tim=None) == E          # and so does a cache that stores them
    assert attend(hstu, cache=cache_of(hstu, timestamps=None)) == E
    assert attend(hstu, ali=P(22)) == E                   # ALiBi together with tables
    assert attend(hstu, shape=shape_of(hstu, n_pos_buckets=0)) == E
    assert attend(hstu, scale=float("nan")) == E and attend(hstu, scale=float("inf")) == E
    assert attend(hstu, uvqk=P(6) + 8) == E and attend(hstu, av=P(14) + 4) == E
    assert attend(hstu, ws=P(15) + 128) == E
    assert attend(hstu, av=P(6)) == E                     # aliasing
    assert attend(hstu, av=P(15)) == E
    assert attend(hstu, av=P(2) + 1024) == E
    assert attend(hstu, uvqk=P(1) + 1024) == E
    assert attend(hstu, ws=P(5)) == E
    assert attend(hstu, M=0) == E
    assert attend(hstu, M=1 << 24) == U
    assert attend(hstu, shape=shape_of(hstu, max_seq_len=1 << 31)) == U
    assert attend(hstu, shape=shape_of(hstu, num_seqs=1 << 20, total_tokens=1 << 20, max_seq_len=1 << 20)) == U
    assert attend(hstu, cache=cache_of(hstu, num_pages=(1 << 31) - 1)) == U   # rows beyond 32 bits
    assert attend(hstu, ws_bytes=hstu.paged_attention_workspace_size(shape_of(hstu)) - 1) == E
    empty = shape_of(hstu, num_seqs=0, total_tokens=0)
    assert attend(hstu, shape=empty, uvqk=None, av=None, ws=None, table=None, lens=None) == hstu.HSTU_OK


def test_layer_refusals(hstu):
    E = hstu.HSTU_ERR_INVALID_ARG
    for name in ("X", "W1", "W2", "lnw", "lnb", "out", "ws", "table", "lens"):
        assert layer(hstu, **{name: None}) == E, name
    assert layer(hstu, W1=P(16) + 2) == E
    assert layer(hstu, out=P(6)) == E
    assert layer(hstu, out=P(1)) == E and layer(hstu, X=P(2)) == E
    assert layer(hstu, ws_bytes=hstu.paged_layer_workspace_size(shape_of(hstu)) - 1) == E
    assert hstu.paged_layer_workspace_size(shape_of(hstu, d_model=0)) == 0


def test_evict_refusals(hstu):
    E = hstu.HSTU_ERR_INVALID_ARG
    assert evict(hstu, budget=-1) == E and evict(hstu, recent=-1) == E
    assert evict(hstu, budget=10, recent=11) == E
    assert evict(hstu, cache=cache_of(hstu, weights=None)) == E
    assert evict(hstu, cache=cache_of(hstu, positions=None)) == E
    for name in ("table", "lens", "new", "ws"):
        assert evict(hstu, **{name: None}) == E, name
    size = hstu.cache_evict_workspace_size(type("C", (), {"ref": ctypes.byref(cache_of(hstu))}), 3, 9)
    assert size >= 3 * 9 * 64 * 4
    assert evict(hstu, ws_bytes=size - 1) == E
    assert evict(hstu, ws=P(15) + 16) == E
    assert evict(hstu, new=P(10) + 8) == E                # part of cache_lens
    assert evict(hstu, new=P(11)) == E                    # next_positions
    assert evict(hstu, new=P(3)) == E and evict(hstu, ws=P(1)) == E
    assert evict(hstu, B=0, table=None, lens=None, new=None, ws=None) == hstu.HSTU_OK


def test_binding_refuses_tensors_that_do_not_fit(hstu):
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hstu.PagedCache(k, k)                              # not on a GPU
    with pytest.raises(ValueError):
        hstu._arg("x", k, torch.float32, k.numel(), k.device)
    with pytest.raises(ValueError):
        hstu._arg("x", k, torch.bfloat16, k.numel() - 1, k.device)
    with pytest.raises(ValueError):
        hstu._arg("x", k.transpose(0, 1), torch.bfloat16, k.numel(), k.device)
    with pytest.raises(ValueError):
        hstu._arg("x", k, torch.bfloat16, k.numel(), torch.device("cuda", 0))
    assert hstu._arg("x", None, torch.bfloat16, 3, k.device) is None
