"""The paged cache on the GPU against its fp64 oracle (oracle/paged.py): filling, attention of one new
token a sequence, eviction, the layer over new tokens, and a serving loop of all of them.  Copied
values are compared bit for bit; AV and weights against bounds derived from the values
(tests/paged_util.py)."""
import copy

import numpy as np
import pytest
import torch

import oracle
from oracle import paged
from tests.gpu_util import assert_bf16_close, assert_f32_close, dev, host
from tests.paged_util import Case, check_av, check_cache, same, values
from workloads import random_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hstu():
    import hstu_sequential_transduction_layer_b200 as m
    return m


def attention_case(hstu, c, append=True):
    g = c.on_device(hstu)
    av, want = c.want_attention(append)
    ab, wb = c.bounds()
    c.attend(hstu, g, append)
    assert hstu.device_status() == hstu.HSTU_OK
    check_av(g["av"], av, ab)
    check_cache(g["cache"], want, wb)
    return g


EDGES = [0, 1, 7, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257]


@pytest.mark.parametrize("ps", [16, 64, 1024])
@pytest.mark.parametrize("dtype,H,hd", [("bf16", 2, 64), ("bf16", 3, 128), ("fp32", 2, 32),
                                        ("fp32", 1, 64), ("fp32", 2, 128)])
def test_attention_lengths_around_every_edge(hstu, dtype, H, hd, ps):
    attention_case(hstu, Case(11, EDGES, H, hd, ps, dtype))


@pytest.mark.parametrize("bias", ["rab", "pos", "time", "alibi", "none"])
@pytest.mark.parametrize("thinned", [False, True])
@pytest.mark.parametrize("append", [False, True])
def test_attention_biases(hstu, bias, thinned, append):
    c = Case(12, [300, 0, 77, 1], 4, 64, 32, bias=bias, thinned=thinned)
    attention_case(hstu, c, append)


@pytest.mark.parametrize("weights,positions", [(False, True), (True, False), (False, False)])
def test_attention_without_the_optional_arrays(hstu, weights, positions):
    c = Case(13, [40, 131], 2, 64, 16, weights=weights, positions=positions)
    c.next[:] = [40, 135]            # a cache without positions: slot i holds position i
    if not positions:
        g = c.on_device(hstu)
        c.attend(hstu, g)            # next_positions None: the cached lengths
        c.next[:] = c.lens
        av, _ = c.want_attention()
        check_av(g["av"], av, c.bounds()[0])
    else:
        attention_case(hstu, c)


@pytest.mark.parametrize("H,hd,lens", [
    (8, 64, [2111, 1, 0, 900, -1, 513]),                    # ragged, one row inactive
    (1, 64, [5000]),                                        # one head, one long sequence
    (16, 128, [700, 650]),
    (5, 64, [n % 41 for n in range(150)]),                  # many short sequences
    (2, 128, [-1, -1]),                                     # nothing active
    (1, 64, [3])])
def test_attention_batches(hstu, H, hd, lens):
    c = Case(14, lens, H, hd, 16, bias="rab", P=1000, Tb=9, spread=40000)
    g = attention_case(hstu, c)
    for b, n in enumerate(lens):
        if n < 0:
            assert (g["av"][b] == 0).all()


def test_attention_time_far_apart_and_in_the_future(hstu):
    # differences beyond 2^32 seconds, and tokens newer than the new one: bucket of 0
    c = Case(15, [64], 2, 64, 16, bias="time", Tb=60)
    p, o = c.table[0, np.arange(64) // 16], np.arange(64) % 16
    c.cache["timestamps"][p, o] = c.now[0] - np.array([(1 << min(i, 61)) - (i % 3) for i in range(64)])
    c.cache["timestamps"][p[:5], o[:5]] = c.now[0] + 10 ** np.arange(5)
    attention_case(hstu, c)


def test_attention_position_beyond_2_24_and_behind(hstu):
    c = Case(16, [33], 2, 64, 16, bias="pos", P=50)
    p, o = c.table[0, np.arange(33) // 16], np.arange(33) % 16
    c.next[0] = (1 << 31) - 1
    c.cache["positions"][p, o] = (1 << 31) - 1 - np.arange(33) * 2
    c.cache["positions"][p[0], o[0]] = 3
    attention_case(hstu, c)


def test_attention_repeats_bit_for_bit_and_ignores_its_neighbours(hstu):
    c = Case(17, [1500, 3, 64, 800], 4, 64, 16)
    g, h = c.on_device(hstu), c.on_device(hstu)
    c.attend(hstu, g)
    c.attend(hstu, h)
    assert torch.equal(g["av"], h["av"])
    same_w = (g["cache"].weights == h["cache"].weights) | g["cache"].weights.isnan()
    assert same_w.all()
    # another batch around sequence 0 (its own pool of pages): close, as sums are split elsewhere
    alone = c.on_device(hstu)
    for k in ("uvqk", "table", "lens", "next", "now", "av"):
        alone[k] = alone[k][:1].contiguous()
    s = alone["shape"]
    alone["shape"] = hstu.make_shape(1, 1, s.max_seq_len, s.d_model, 4, 64, 64, hstu.HSTU_BF16,
                                     s.n_pos_buckets, s.n_time_buckets)
    c.attend(hstu, alone)
    want, _ = c.want_attention()
    check_av(alone["av"], want[:1], c.bounds()[0][:1])


def test_attention_infinite_and_nan_keys_stay_in_their_sequence(hstu):
    c = Case(18, [70, 70], 2, 64, 16)
    p, o = c.table[0, 9 // 16], 9
    c.cache["k"][p, 0, o, 5] = np.inf
    c.uvqk.reshape(2, 4, 2, 64)[0, 2, 0, 5] = 1.0
    g = c.on_device(hstu)
    c.attend(hstu, g)
    got = g["av"].reshape(2, 2, 64)
    av, _ = c.want_attention()
    av = av.reshape(2, 2, 64)
    # score +inf: AV of that head is infinite (by V's sign), all else as ever
    fine = np.isfinite(av)
    assert (torch.isfinite(got).cpu().numpy() == fine).all() and not fine[0, 0].any()
    assert fine[0, 1].all() and fine[1].all()
    ab = c.bounds()[0].reshape(2, 2, 64)
    assert (np.abs(got.double().cpu().numpy()[fine] - av[fine]) <= ab[fine]).all()


def test_attention_bad_lengths_and_pages_are_reported(hstu):
    c = Case(19, [40, 50, 60], 2, 64, 16, extra=0)          # page 4 has no room in sequence 2's row
    g = c.on_device(hstu)
    g["table"][0, 1] = 1 << 30                               # no page: slots 16..31 are left out
    g["lens"][1] = 10 ** 12                                  # clamped to the table
    before = copy.deepcopy(c)
    c.attend(hstu, g, append=False)
    assert hstu.device_status() == hstu.HSTU_ERR_DEVICE_BAD_OFFSETS
    assert hstu.device_status() == hstu.HSTU_OK
    av, _ = before.want_attention(append=False)
    check_av(g["av"][2:], av[2:], before.bounds()[0][2:])
    # sequence 0 without its second page
    k = before.cache["v"][before.table[0, 1]]
    keep = k.copy()
    k[:] = 0.0
    kk = before.cache["k"][before.table[0, 1]]
    kk[:] = 0.0
    av0, _ = before.want_attention(append=False)
    check_av(g["av"][:1], av0[:1], before.bounds()[0][:1] + 1e-6)
    del keep
    # a full row: the token is scored, not stored
    c = Case(20, [32], 2, 64, 16, extra=0)
    g = c.on_device(hstu)
    c.attend(hstu, g, append=True)
    assert hstu.device_status() == hstu.HSTU_ERR_DEVICE_BAD_OFFSETS


def test_attention_a_shared_prefix(hstu):
    # two sequences read the same first page; nothing sums weights
    c = Case(21, [40, 40], 2, 64, 16, weights=False)
    c.table[1, 0] = c.table[0, 0]
    attention_case(hstu, c)


def test_attention_far_into_a_large_pool(hstu):
    # element offsets beyond 2^31 in K and V
    H, hd, ps = 32, 128, 64
    pages = (1 << 31) // (H * hd * ps) + 40
    k = torch.empty((pages, H, ps, hd), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = Case(22, [150], H, hd, ps, bias="none", positions=False, weights=False)
    small = c.on_device(hstu)
    far = [pages - 1, pages - 20, pages - 7]
    for i in range(3):
        k[far[i]], v[far[i]] = small["cache"].k[c.table[0, i]], small["cache"].v[c.table[0, i]]
    small["table"][0, :3] = torch.tensor(far, dtype=torch.int32)
    small["cache"] = hstu.PagedCache(k, v)
    c.attend(hstu, small)
    assert hstu.device_status() == hstu.HSTU_OK
    av, want = c.want_attention()
    check_av(small["av"], av, c.bounds()[0])
    same(k[far[2]], want["k"][c.table[0, 2]], "appended page")
    same(v[far[2]], want["v"][c.table[0, 2]], "appended page")


def test_attention_captured_and_replayed(hstu):
    # two graphs share one workspace; each step's graph advances the lengths itself
    c = Case(23, [700, 20, 0], 4, 64, 16, extra=12)
    ws = torch.empty(hstu.paged_attention_workspace_size(c.on_device(hstu)["shape"]), dtype=torch.uint8,
                     device="cuda")
    gs = [c.on_device(hstu) for _ in range(3)]
    for g in gs:
        s = g["shape"]
        g["shape"] = hstu.make_shape(3, 3, 712, s.d_model, 4, 64, 64, hstu.HSTU_BF16,
                                     s.n_pos_buckets, s.n_time_buckets)
    graphs = []
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for g in gs[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            c.attend(hstu, g, workspace=ws)
            g["lens"].add_(1)
            g["next"].add_(1)
        graphs.append(graph)
    torch.cuda.synchronize()
    ws.fill_(255)                                            # whatever it held before
    eager = gs[2]
    for step in range(8):
        for graph in graphs:
            graph.replay()
        c.attend(hstu, eager)
        eager["lens"].add_(1)
        eager["next"].add_(1)
        torch.cuda.synchronize()
        for g in gs[:2]:
            assert torch.equal(g["av"], eager["av"]), step
            assert torch.equal(g["cache"].k.isnan(), eager["cache"].k.isnan())
    assert hstu.device_status() == hstu.HSTU_OK


@pytest.mark.parametrize("lens", [[(i * 7) % 23 - 1 for i in range(900)], [i % 4 - 1 for i in range(5000)],
                                  [0] * 385, [200] + [-1] * 800 + [333], [-1] * 700 + [17]])
def test_attention_more_sequences_than_threads(hstu, lens):
    # lengths are scanned in groups of more than one; empty groups and groups of inactive ones
    attention_case(hstu, Case(25, lens, 1, 64, 16, "fp32", bias="pos"))


def test_attention_wide_models(hstu):
    attention_case(hstu, Case(26, [61, 18, 130], 33, 128, 32))
    attention_case(hstu, Case(27, [70, 9], 48, 32, 16, "fp32", bias="alibi"))


def test_attention_lengths_beyond_the_announced_longest_are_clamped(hstu):
    c = Case(28, [100, 40], 2, 64, 16, extra=30)
    g = c.on_device(hstu)
    s = g["shape"]
    g["shape"] = hstu.make_shape(2, 2, 81, s.d_model, 2, 64, 64, hstu.HSTU_BF16, s.n_pos_buckets,
                                 s.n_time_buckets)
    k = g["cache"].k.clone()
    c.attend(hstu, g)
    assert hstu.device_status() == hstu.HSTU_ERR_DEVICE_BAD_OFFSETS
    c.lens[0] = 80                       # and its new token is not stored
    av, _ = c.want_attention(append=False)
    check_av(g["av"], av, c.bounds()[0])
    p = int(c.table[0, 80 // 16])
    assert torch.equal(g["cache"].k[p], k[p])
    same(g["cache"].k[c.table[1, 40 // 16]][:, 40 % 16], c.uvqk.reshape(2, 4, 2, 64)[1, 3], "stored row")


def test_positions_outside_their_range_are_reported(hstu):
    for bad in (1 << 31, -1, 1 << 40):
        c = Case(29, [20], 1, 64, 16, bias="pos")
        g = c.on_device(hstu)
        g["next"][0] = bad
        c.attend(hstu, g)
        assert hstu.device_status() == hstu.HSTU_ERR_DEVICE_BAD_OFFSETS
        assert torch.isfinite(g["av"]).all()
        off = torch.tensor([0, 3], device="cuda")
        g["lens"][0] = 3
        hstu.hstu_cache_append(g["cache"], c.dev(values(c.rng, (3, 256), "bf16"), torch.bfloat16), off,
                               None, g["table"], g["lens"], g["next"])
        assert hstu.device_status() == hstu.HSTU_ERR_DEVICE_BAD_OFFSETS


def test_attention_on_two_streams_at_once(hstu):
    cases = [Case(24 + i, [1200, 300, 40], 4, 64, 16) for i in range(2)]
    gs = [c.on_device(hstu) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, g, st in zip(cases, gs, streams):
            c.attend(hstu, g, append=False, stream=st)
    torch.cuda.synchronize()
    assert hstu.device_status() == hstu.HSTU_OK
    for c, g in zip(cases, gs):
        check_av(g["av"], c.want_attention()[0], c.bounds()[0])


def test_calls_on_a_stream_of_their_own_allocate_there(hstu):
    # new workspaces and outputs belong to the call's stream, given as an object or as its address
    c = Case(30, [400, 90], 4, 64, 16, extra=4)
    st, busy = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    for address in (False, True):
        g = c.on_device(hstu)
        torch.cuda.synchronize()
        stream = st.cuda_stream if address else st
        with torch.cuda.stream(st):
            for _ in range(3):
                busy = busy @ busy * 1e-3                    # the stream is behind the host
        c.attend(hstu, g, append=False, stream=stream)
        for _ in range(8):                                   # what the current stream allocates meanwhile
            torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
        new = hstu.hstu_cache_evict(g["cache"], g["table"], g["lens"], g["next"], 64, 8, stream=stream)
        torch.cuda.synchronize()
        assert hstu.device_status() == hstu.HSTU_OK
        check_av(g["av"], c.want_attention(append=False)[0], c.bounds()[0])
        assert new.tolist() == [64, 64]


# ------------------------------------------------------------------------------------------------
# Append
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,H,hd,ps,lens,counts", [
    ("bf16", 2, 64, 16, [0, 5, 16, 31, 40], [0, 1, 17, 1, 100]),
    ("bf16", 3, 128, 64, [0, 63, 200], [300, 2, 0]),
    ("fp32", 2, 32, 16, [7, 0], [9, 33]),
    ("fp32", 1, 128, 32, [1], [31]),
    ("bf16", 8, 64, 64, [0, 0, 0, 1], [0, 0, 700, 0]),
    ("fp32", 65, 128, 16, [3, 0], [20, 1]),
    ("bf16", 2, 128, 256, [0], [1]),
    ("bf16", 1, 64, 16, [0] * 300, [i % 7 for i in range(300)])])
def test_append(hstu, dtype, H, hd, ps, lens, counts):
    c = Case(31, lens, H, hd, ps, dtype, thinned=True, extra=max(counts))
    T = sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    rows, ts = values(c.rng, (T, 4 * H * hd), dtype), c.rng.integers(0, 1 << 40, T)
    g = c.on_device(hstu)
    hstu.hstu_cache_append(g["cache"], c.dev(rows, c.torch_dtype()), c.dev(off, torch.int64),
                           c.dev(ts, torch.int64), g["table"], g["lens"], g["next"])
    assert hstu.device_status() == hstu.HSTU_OK
    paged.append(c.cache, rows, off, ts, c.table, c.lens, c.next)
    check_cache(g["cache"], c.cache)


def test_append_reports_what_does_not_fit(hstu):
    c = Case(32, [10, -1, 3], 2, 64, 16, bias="none", extra=0)     # one page a row
    rows = values(c.rng, (30, 512), "bf16")
    off = np.array([0, 12, 20, 30], np.int64)                       # 2: 10 tokens, 13 slots left
    g = c.on_device(hstu)
    hstu.hstu_cache_append(g["cache"], c.dev(rows, torch.bfloat16), c.dev(off, torch.int64), None,
                           g["table"], g["lens"])
    assert hstu.device_status() == hstu.HSTU_ERR_DEVICE_BAD_OFFSETS
    # sequence 0 keeps the six that fit, the inactive one none
    paged.append(c.cache, np.concatenate([rows[:6], rows[20:]]), np.array([0, 6, 6, 16]), None,
                 c.table, c.lens)
    check_cache(g["cache"], c.cache)


def test_append_bad_offsets_are_reported(hstu):
    c = Case(33, [3, 4], 2, 64, 16, bias="none", extra=20)
    g = c.on_device(hstu)
    rows = c.dev(values(c.rng, (8, 512), "bf16"), torch.bfloat16)
    for off in ([0, 9, 8], [0, 4, 7], [2, 4, 8], [0, -3, 8], [0, 1 << 40, 8]):
        hstu.hstu_cache_append(g["cache"], rows, torch.tensor(off, device="cuda"), None, g["table"],
                               g["lens"])
        assert hstu.device_status() == hstu.HSTU_ERR_DEVICE_BAD_OFFSETS, off


# ------------------------------------------------------------------------------------------------
# Evict
# ------------------------------------------------------------------------------------------------

def evict_case(hstu, c, budget, recent, alias=False):
    g = c.on_device(hstu)
    new = hstu.hstu_cache_evict(g["cache"], g["table"], g["lens"], g["next"], budget, recent,
                                new_lens=g["lens"] if alias else None)
    assert hstu.device_status() == hstu.HSTU_OK
    want = paged.evict(c.cache, c.table, c.lens, c.next, budget, recent)
    same(new, want, "new_lens")
    check_cache(g["cache"], c.cache)
    return g


@pytest.mark.parametrize("lens,budget,recent", [
    ([33, 32, 31, -1, 0], 32, 5), ([1, 2, 3], 1, 0), ([1, 2, 3], 1, 1), ([100, 7], 0, 0),
    ([700, 699, 650, 20], 650, 64), ([2100, 1024, 1025], 1024, 100), ([3000], 200, 200),
    ([40, 41, 90], 64, 3)])
@pytest.mark.parametrize("thinned", [False, True])
def test_evict(hstu, lens, budget, recent, thinned):
    evict_case(hstu, Case(41, lens, 3, 64, 16, thinned=thinned), budget, recent, alias=thinned)


@pytest.mark.parametrize("dtype,H,hd,ps", [("bf16", 8, 128, 64), ("fp32", 2, 32, 32),
                                           ("fp32", 1, 128, 16), ("bf16", 1, 64, 1024)])
def test_evict_types(hstu, dtype, H, hd, ps):
    evict_case(hstu, Case(42, [333, 150, 20], H, hd, ps, dtype, bias="none"), 111, 10)


@pytest.mark.parametrize("kind", ["zero", "two values", "inf", "nan", "tiny", "negative", "cancel"])
def test_evict_ties_and_odd_weights(hstu, kind):
    c = Case(43, [500, 90, 1300], 2, 64, 16, thinned=True)
    w, rng = c.cache["weights"], c.rng
    live = ~np.isnan(w)
    n = live.sum()
    w[live] = {"zero": np.zeros(n), "two values": rng.integers(0, 2, n) * 1.0,
               "inf": np.where(rng.random(n) < 0.6, np.inf, 1.0),
               "nan": np.where(rng.random(n) < 0.5, np.nan, rng.random(n).astype(np.float32)),
               "tiny": rng.integers(0, 3, n) * 2.0 ** -149,
               "negative": rng.integers(-3, 3, n) * 1.0,
               "cancel": np.where(rng.random(n) < 0.5, -0.0, 0.0)}[kind]
    evict_case(hstu, c, 80, 30)


def test_evict_a_long_history(hstu):
    evict_case(hstu, Case(44, [20011, 5], 1, 64, 64, bias="none"), 7001, 500)


@pytest.mark.parametrize("kind", ["random", "zero", "two values"])
@pytest.mark.parametrize("others", [1, 9])
def test_evict_long_histories(hstu, kind, others):
    # few sequences: a cluster of sixteen CTAs; more of them: eight, whose shared memory does not hold
    # all keys, so that some go through the workspace
    c = Case(48, [70001] + [100] * others, 1, 64, 1024, bias="none")
    live = ~np.isnan(c.cache["weights"])
    if kind != "random":
        c.cache["weights"][live] = 0.0 if kind == "zero" else c.rng.integers(0, 2, live.sum())
    evict_case(hstu, c, 30011, 1000)


@pytest.mark.parametrize("n", [400, 3000])
def test_evict_many_sequences(hstu, n):
    evict_case(hstu, Case(45, [i % 50 for i in range(n)], 1, 64, 16, bias="none"), 20, 4)


def test_evict_close_weights(hstu):
    # keys that differ in the last bits only: every pass of the search is needed
    c = Case(49, [4000, 900], 1, 64, 64, bias="none")
    live = ~np.isnan(c.cache["weights"])
    c.cache["weights"][live] = (np.float32(1.0) + c.rng.integers(0, 1500, live.sum()) * np.float32(2.0 ** -23))
    evict_case(hstu, c, 801, 16)


def test_evict_captured_with_a_dirty_workspace(hstu):
    c = Case(46, [400, 130, 20], 2, 64, 16)
    g = c.on_device(hstu)
    ws = torch.full((hstu.cache_evict_workspace_size(g["cache"], 3, c.M),), 255, dtype=torch.uint8,
                    device="cuda")
    new = torch.zeros(3, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=st):
        hstu.hstu_cache_evict(g["cache"], g["table"], g["lens"], g["next"], 64, 8, new_lens=new,
                              workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    want = paged.evict(c.cache, c.table, c.lens, c.next, 64, 8)
    same(new, want, "new_lens")
    check_cache(g["cache"], c.cache)


def test_evict_bad_lengths_and_pages_are_reported(hstu):
    c = Case(47, [60, 60], 2, 64, 16)
    g = c.on_device(hstu)
    g["table"][0, 2] = -1
    g["lens"][1] = 1 << 50
    new = hstu.hstu_cache_evict(g["cache"], g["table"], g["lens"], g["next"], 30, 4)
    assert hstu.device_status() == hstu.HSTU_ERR_DEVICE_BAD_OFFSETS
    assert new.tolist() == [30, 30]


# ------------------------------------------------------------------------------------------------
# The layer, and a serving loop
# ------------------------------------------------------------------------------------------------

def history_case(seed, lens, H, hd, dtype, alibi=False):
    return random_case(seed, lens, H * hd, H, hd, P=64, Tb=16, dtype=dtype, alibi=alibi)


@pytest.mark.parametrize("dtype,H,hd,alibi", [("bf16", 2, 64, False), ("bf16", 8, 64, False),
                                              ("bf16", 4, 128, True), ("fp32", 2, 32, False)])
def test_layer_decodes_the_rows_of_the_forward(hstu, dtype, H, hd, alibi):
    """Histories are filled from their f1 output, the last tokens go through the layer one at a time:
    their rows are the whole forward's."""
    steps, d = 3, H * hd
    inp = history_case(51, [150, 3, 67], H, hd, dtype, alibi)
    p, f = inp.layers[0], "bf16" if dtype == "bf16" else "f32"
    want = oracle.layer_fwd_inputs(inp)
    off, B = inp.seq_offsets, 3
    W = {k: dev(getattr(p, k), f) for k in ("W1", "b1", "W2", "b2", "ln_w", "ln_b")}
    tab = [dev(inp.pos_table, "f32"), dev(inp.time_table, "f32"), dev(inp.alibi_slopes, "f32")]
    code = hstu.HSTU_BF16 if dtype == "bf16" else hstu.HSTU_F32
    P = 0 if alibi else 64
    Tb = 0 if alibi else 16
    lens = inp.lengths.astype(np.int64) - steps
    hist = np.concatenate([np.arange(off[b], off[b] + lens[b]) for b in range(B)])
    hoff = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    X = dev(inp.X, f)
    ts = torch.from_numpy(np.ascontiguousarray(inp.timestamps)).cuda() if inp.timestamps is not None \
        else torch.zeros(inp.T, dtype=torch.int64, device="cuda")
    uvqk = torch.empty((len(hist), 4 * d), dtype=X.dtype, device="cuda")
    s = hstu.make_shape(B, len(hist), 150, d, H, hd, hd, code, P, Tb)
    rows = torch.from_numpy(hist).cuda()
    hstu.hstu_f1_fwd(s, X[rows].contiguous(), W["W1"], W["b1"], uvqk)
    ps, M = 16, 10
    cache = hstu.PagedCache.allocate(B * M, ps, H, hd, X.dtype)
    table = torch.randperm(B * M, generator=torch.Generator().manual_seed(1)).int().reshape(B, M).cuda()
    clen = torch.zeros(B, dtype=torch.int64, device="cuda")
    hstu.hstu_cache_append(cache, uvqk, torch.from_numpy(hoff).cuda(), ts[rows].contiguous(), table, clen)
    clen = torch.from_numpy(lens).cuda()
    shape = hstu.make_shape(B, B, 151, d, H, hd, hd, code, P, Tb)
    for k in range(steps):
        at = torch.from_numpy(off[:B] + lens + k).cuda()
        y = hstu.hstu_paged_layer_fwd(shape, cache, X[at].contiguous(), table, clen, clen,
                                      ts[at].contiguous(), W["W1"], W["b1"], W["W2"], W["b2"],
                                      W["ln_w"], W["ln_b"], *tab, inp.scale)
        clen += 1
        assert hstu.device_status() == hstu.HSTU_OK
        close = assert_bf16_close if dtype == "bf16" else assert_f32_close
        close(host(y), want[off[:B] + lens + k], f"step {k}")


def test_layer_inactive_rows_do_not_disturb_the_batch(hstu):
    inp = history_case(52, [1, 1, 1], 2, 64, "bf16")
    p = inp.layers[0]
    W = [dev(getattr(p, k)) for k in ("W1", "b1", "W2", "b2", "ln_w", "ln_b")]
    tab = [dev(inp.pos_table, "f32"), dev(inp.time_table, "f32"), None]
    X, now = dev(inp.X), torch.from_numpy(np.ascontiguousarray(inp.timestamps)).cuda()
    out = []
    for rows in ([0, 1, 2], [0, -1, 2]):
        cache = hstu.PagedCache.allocate(3, 16, 2, 64)
        lens = torch.tensor([0 if r >= 0 else -1 for r in rows], device="cuda")
        table = torch.arange(3, dtype=torch.int32, device="cuda").reshape(3, 1)
        s = hstu.make_shape(3, 3, 1, 128, 2, 64, 64, hstu.HSTU_BF16, 64, 16)
        out.append(hstu.hstu_paged_layer_fwd(s, cache, X, table, lens, None, now, *W, *tab, inp.scale))
        assert hstu.device_status() == hstu.HSTU_OK
        out.append(cache.k)
    assert torch.equal(out[0][[0, 2]], out[2][[0, 2]]) and torch.isfinite(out[2].float()).all()
    assert torch.equal(out[1][[0, 2]], out[3][[0, 2]]) and (out[3][1] == 0).all()


def test_layer_captured_equals_eager(hstu):
    inp = history_case(53, [1, 1], 2, 64, "bf16")
    p = inp.layers[0]
    W = [dev(getattr(p, k)) for k in ("W1", "b1", "W2", "b2", "ln_w", "ln_b")]
    tab = [dev(inp.pos_table, "f32"), dev(inp.time_table, "f32"), None]
    s = hstu.make_shape(2, 2, 30, 128, 2, 64, 64, hstu.HSTU_BF16, 64, 16)
    table = torch.arange(4, dtype=torch.int32, device="cuda").reshape(2, 2)
    now = torch.from_numpy(np.ascontiguousarray(inp.timestamps)).cuda()
    runs = []
    for captured in (False, True):
        cache, X = hstu.PagedCache.allocate(4, 16, 2, 64), dev(inp.X)
        lens = torch.tensor([0, 0], device="cuda")
        ws = torch.empty(hstu.paged_layer_workspace_size(s), dtype=torch.uint8, device="cuda")

        def step():   # the output is the next step's input
            y = hstu.hstu_paged_layer_fwd(s, cache, X, table, lens, None, now, *W, *tab, inp.scale,
                                          workspace=ws)
            X.copy_(y)
            lens.add_(1)
        if captured:
            graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
            with torch.cuda.graph(graph, stream=st):
                step()
            for _ in range(20):
                graph.replay()
        else:
            for _ in range(20):
                step()
        torch.cuda.synchronize()
        runs.append((X.clone(), cache.k.clone(), cache.weights.clone(), lens.clone()))
    assert hstu.device_status() == hstu.HSTU_OK
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_calls_back_to_back_see_each_others_writes(hstu):
    # every kernel's launch overlaps the one before it: unwaited steps equal steps waited for one by one
    runs = []
    for wait in (False, True):
        c = Case(62, [900, 30, 2000, 500], 4, 128, 16, extra=70)
        g = c.on_device(hstu)
        s = g["shape"]
        g["shape"] = hstu.make_shape(4, 4, 2071, s.d_model, 4, 128, 128, hstu.HSTU_BF16,
                                     s.n_pos_buckets, s.n_time_buckets)
        ws = torch.empty(hstu.paged_attention_workspace_size(g["shape"]), dtype=torch.uint8, device="cuda")
        es = torch.empty(hstu.cache_evict_workspace_size(g["cache"], 4, c.M), dtype=torch.uint8, device="cuda")
        out = []
        torch.cuda.synchronize()
        for step in range(60):
            c.attend(hstu, g, workspace=ws)
            out.append(g["av"].clone())
            if wait:
                torch.cuda.synchronize()
            g["lens"].add_(1)
            g["next"].add_(1)
            g["uvqk"].copy_((out[-1][:, :1] * 1e-3).to(torch.bfloat16) + g["uvqk"].roll(7, 1))
            if step % 20 == 19:
                hstu.hstu_cache_evict(g["cache"], g["table"], g["lens"], g["next"], 800, 50,
                                      new_lens=g["lens"], workspace=es)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert hstu.device_status() == hstu.HSTU_OK
        runs.append((torch.stack(out), g["cache"].k, g["cache"].weights, g["cache"].positions, g["lens"]))
    for a, b in zip(*runs):
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("dtype,H,hd,bias", [("bf16", 4, 64, "rab"), ("fp32", 2, 32, "alibi")])
def test_serving_loop(hstu, dtype, H, hd, bias):
    """Fill, then token after token with an eviction whenever a sequence outgrows its budget, against
    the oracle step by step.  The oracle continues from the device's weights (fp32 sums), so that
    the evictions' choices are compared exactly."""
    B, ps, budget, recent, room = 3, 16, 48, 8, 64
    c = Case(61, [0] * B, H, hd, ps, dtype, bias=bias, extra=room)
    g = c.on_device(hstu)
    counts = [45, 3, 30]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    rows = values(c.rng, (sum(counts), 4 * H * hd), dtype)
    ts = 1_600_000_000 + np.arange(sum(counts))
    hstu.hstu_cache_append(g["cache"], c.dev(rows, c.torch_dtype()), c.dev(off, torch.int64),
                           c.dev(ts, torch.int64), g["table"], g["lens"], g["next"])
    paged.append(c.cache, rows, off, ts, c.table, c.lens, c.next)
    check_cache(g["cache"], c.cache)
    for name in ("lens", "next"):
        g[name] += c.dev(np.array(counts), torch.int64)
    c.lens += counts
    c.next += counts
    g["shape"] = hstu.make_shape(B, B, room, max(64, H * hd), H, hd, hd, g["shape"].dtype,
                                 g["shape"].n_pos_buckets, g["shape"].n_time_buckets)
    c.scale = 1 / 64
    for step in range(25):
        c.uvqk = values(c.rng, (B, 4 * H * hd), dtype)
        c.now = np.array([1_600_001_000 + 50 * step] * B)
        g["uvqk"], g["now"] = c.dev(c.uvqk, c.torch_dtype()), c.dev(c.now, torch.int64)
        ab, wb = c.bounds()
        av, want = c.want_attention()
        c.attend(hstu, g)
        assert hstu.device_status() == hstu.HSTU_OK
        check_av(g["av"], av, ab, f"step {step}")
        check_cache(g["cache"], want, wb)
        c.cache = want
        c.cache["weights"] = g["cache"].weights.double().cpu().numpy()
        for name in ("lens", "next"):
            g[name] += 1
        c.lens += 1
        c.next += 1
        if step % 5 == 4:
            hstu.hstu_cache_evict(g["cache"], g["table"], g["lens"], g["next"], budget, recent,
                                  new_lens=g["lens"])
            c.lens = paged.evict(c.cache, c.table, c.lens, c.next, budget, recent)
            same(g["lens"], c.lens, "lengths")
            check_cache(g["cache"], c.cache)
    assert hstu.device_status() == hstu.HSTU_OK
