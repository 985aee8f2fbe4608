"""The paged cache's host side and what can be read off its kernels' source (no GPU needed)."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import paged
from tests.paged_util import Case
from tests.test_paged_abi import P, append, attend, cache_of, evict, layer, shape_of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def hstu():
    import hstu_sequential_transduction_layer_b200 as m
    return m


def kernel_body(name):
    """A kernel's definition, comments taken out."""
    path = os.path.join(ROOT, "hstu_sequential_transduction_layer_b200", "csrc", "paged_kernels.cuh")
    text = re.sub(r"//[^\n]*", "", open(path).read())
    at = re.search(r"__global__[^;{]*\b%s\(" % name, text).start()
    return text[at:text.index("\n}\n", at)]


def test_a_cluster_has_started_before_its_shared_memory_is_touched():
    """A CTA's shared memory may be accessed by its cluster only once it runs: the selection waits for a
    cluster barrier before the search, whose first step stores to the other CTAs, and arrives on it
    behind the return of sequences that are short enough (all of the cluster's CTAs return there)."""
    body = kernel_body("evict_select_kernel")
    arrive, wait = body.find("cluster_arrive()"), body.find("cluster_wait()")
    search = body.index("for (; pass < 3 && in_bin != want; pass++)")
    assert 0 <= arrive < wait < search
    assert body.index("return;") < arrive
    assert "map_shared_rank" not in body[:wait]


def test_what_a_call_writes_is_apart_from_its_index_arrays(hstu):
    """The kernels read lengths, tables and biases while they write: an output, a workspace or a cache
    array on top of one of them is refused."""
    E = hstu.HSTU_ERR_INVALID_ARG
    where = {"table": P(9), "lens": P(10), "nxt": P(11)}
    for name, at in where.items():
        assert evict(hstu, ws=at) == E, name
        assert evict(hstu, **{name: P(5) + 64}) == E, name             # in the weights
        assert append(hstu, **{name: P(1) + 64}) == E, name
    assert evict(hstu, new=P(9)) == E
    assert evict(hstu, new=P(9) + 8) == E
    for name in ("off", "ts"):
        assert append(hstu, **{name: P(4) + 64}) == E, name
    where.update(now=P(8), pos=P(12), tim=P(13))
    for name, at in where.items():
        for call, out in ((attend, "av"), (layer, "out")):
            assert call(hstu, **{out: at}) == E, (call, name)
            assert call(hstu, ws=at) == E, (call, name)
            assert call(hstu, **{name: P(2) + 64}) == E, (call, name)
    for call, out in ((attend, "av"), (layer, "out")):
        slopes = dict(pos=None, tim=None, ali=P(22))
        assert call(hstu, **slopes, **{out: P(22)}) == E
        assert call(hstu, **slopes, ws=P(22)) == E


def test_index_arrays_are_naturally_aligned(hstu):
    E = hstu.HSTU_ERR_INVALID_ARG
    for call in (append, attend, layer, evict):
        assert call(hstu, table=P(9) + 2) == E, call
        assert call(hstu, lens=P(10) + 4) == E, call
        assert call(hstu, nxt=P(11) + 4) == E, call
    assert append(hstu, off=P(7) + 4) == E and append(hstu, ts=P(8) + 1) == E
    assert evict(hstu, new=P(14) + 4) == E
    for call in (attend, layer):
        assert call(hstu, now=P(8) + 4) == E
        assert call(hstu, pos=P(12) + 2) == E and call(hstu, tim=P(13) + 1) == E
        assert call(hstu, pos=None, tim=None, ali=P(22) + 2) == E


def test_evict_without_a_page_by_hand():
    # the row's first page is missing: its 16 slots stay, so of 20 kept slots four hold tokens.  Of slots
    # 16..35 the most attended are 18, 35, 20 and 34: the three beyond slot 20 fill 16, 17 and 19
    c = Case(10, [36], 1, 64, 16, bias="none")
    c.table[0, 0] = -1
    second, third = int(c.table[0, 1]), int(c.table[0, 2])
    c.cache["weights"][second, 0], c.cache["weights"][third, 0, :4] = 0.0, 0.0
    c.cache["weights"][second, 0, [2, 4, 5]] = [4.0, 2.0, 1.0]
    c.cache["weights"][third, 0, [2, 3]] = [2.0, 3.0]
    before = {name: c.cache[name].copy() for name in ("k", "v", "weights", "positions")}
    assert paged.evict(c.cache, c.table, c.lens, c.next, 20, 0).tolist() == [20]
    for name, a in before.items():
        rows = a[second].copy() if name == "positions" else a[second].swapaxes(0, 1).copy()
        far = a[third] if name == "positions" else a[third].swapaxes(0, 1)
        rows[0], rows[1], rows[3] = rows[4].copy(), far[2], far[3]
        got = c.cache[name][second] if name == "positions" else c.cache[name][second].swapaxes(0, 1)
        assert np.array_equal(got, rows, equal_nan=True), name
        others = [p for p in range(len(a)) if p != second]
        assert np.array_equal(a[others], c.cache[name][others], equal_nan=True), name


def test_a_caches_tensors_are_not_exchanged(hstu):
    # the struct that the kernels get holds their addresses: an exchanged tensor would not be seen, and
    # the old one's memory would be written after its release
    cache = object.__new__(hstu.PagedCache)
    for name in ("k", "v", "positions", "timestamps", "weights"):
        with pytest.raises(AttributeError):
            setattr(cache, name, None)


def test_workspace_sizes_of_calls_that_are_refused(hstu):
    """0, as for every shape that its call refuses; a wrapped product would look like a small workspace."""
    def size(B, M, **kw):
        return hstu.cache_evict_workspace_size(type("C", (), {"ref": ctypes.byref(cache_of(hstu, **kw))}), B, M)
    assert size(3, 9) > 0
    for B, M in ((1 << 27, 1), (1 << 34, 1 << 23), ((1 << 63) - 1, 1), (1, 1 << 24), (1, 1 << 31), (-1, 1), (1, -1)):
        assert size(B, M) == 0, (B, M)
    for f in (hstu.paged_attention_workspace_size, hstu.paged_layer_workspace_size):
        assert f(shape_of(hstu)) > 0
        for kw in (dict(total_tokens=4), dict(num_seqs=1 << 62), dict(num_seqs=1 << 30, total_tokens=1 << 30),
                   dict(dtype=hstu.HSTU_F32, d_qk=96, d_v=96), dict(dtype=hstu.HSTU_F32, d_qk=64, d_v=32)):
            assert f(shape_of(hstu, **kw)) == 0, kw


def test_a_caches_arrays_are_apart(hstu):
    """Positions on top of times, weights on top of keys and the like are refused; K and V may be one
    array where they are only read."""
    E = hstu.HSTU_ERR_INVALID_ARG
    slots, kv = 100 * 64, 100 * 64 * 2 * 64 * 2
    for call in (append, attend, layer, evict):
        for over in (dict(v=P(1) + kv - 16), dict(v=P(1)), dict(positions=P(1) + 4), dict(positions=P(2) + kv - 4),
                     dict(timestamps=P(3) + 4 * slots - 8), dict(weights=P(4) + 8 * slots - 4), dict(weights=P(1)),
                     dict(weights=P(3)), dict(positions=P(5) + 8 * slots - 4)):
            assert call(hstu, cache=cache_of(hstu, **over)) == E, (call, over)
    assert attend(hstu, cache=cache_of(hstu, v=P(1)), append=0) != E
    assert attend(hstu, cache=cache_of(hstu, weights=P(1)), append=0) == E
    assert append(hstu, cache=cache_of(hstu, v=P(1) + kv, k=P(1)), T=0) == hstu.HSTU_OK      # side by side
