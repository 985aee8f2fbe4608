"""The paged cache on the GPU in calls beside the everyday ones (tests/test_paged_gpu.py): behind other
work, behind a CUDA error of an earlier call, with rows that name no page, without the optional
arrays, and with many tiles of one history a warp.  Against the fp64 oracle (oracle/paged.py)."""
import copy
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import paged
from tests.paged_util import Case, check_av, check_cache, same, values

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def hstu():
    import hstu_sequential_transduction_layer_b200 as m
    return m


@pytest.mark.parametrize("lens,ps,budget", [([5000, 70, 5000, 3000], 64, 2500), ([40000], 1024, 20000)])
def test_evict_behind_other_work(hstu, lens, ps, budget):
    # the CTAs of a cluster start when products on another stream leave the SMs room for them
    c = Case(71, lens, 1, 64, ps, bias="none")
    want = copy.deepcopy(c)
    new = paged.evict(want.cache, c.table, c.lens, c.next, budget, 100)
    other, busy = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    for _ in range(4):
        g = c.on_device(hstu)
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            for _ in range(20):
                torch.mm(busy, busy)
        got = hstu.hstu_cache_evict(g["cache"], g["table"], g["lens"], g["next"], budget, 100)
        torch.cuda.synchronize()
        assert hstu.device_status() == hstu.HSTU_OK
        same(got, new, "new_lens")
        check_cache(g["cache"], want.cache)


def leave_an_error(hstu):
    """A CUDA call of the library's that fails, as may any before the call that is tested: its status is
    asked for on a stream that is being captured, which CUDA refuses (and the capture is given up)."""
    cuda, graph = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    handle = ctypes.c_void_p(st.cuda_stream)
    assert cuda.cuStreamBeginCapture_v2(handle, 1) == 0                  # 1: this thread's calls
    assert hstu.library().hstu_get_device_status(handle) == hstu.HSTU_ERR_CUDA
    assert cuda.cuStreamEndCapture(handle, ctypes.byref(graph)) != 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("lens,ps,budget", [([40000, 60], 1024, 20000), ([900, 40, 1000], 16, 500)])
def test_evict_behind_an_earlier_error(hstu, lens, ps, budget):
    # one selection only: a second one would find the lengths cut (cache_lens are the new ones) and
    # leave the kept tokens where they are
    c = Case(72, lens, 1, 64, ps, bias="none")
    g = c.on_device(hstu)
    leave_an_error(hstu)
    before = hstu.launch_count()
    hstu.hstu_cache_evict(g["cache"], g["table"], g["lens"], g["next"], budget, 100, new_lens=g["lens"])
    assert hstu.launch_count() - before == 2
    assert hstu.device_status() == hstu.HSTU_OK
    same(g["lens"], paged.evict(c.cache, c.table, c.lens, c.next, budget, 100), "lengths")
    check_cache(g["cache"], c.cache)


def test_attention_and_append_behind_an_earlier_error(hstu):
    c = Case(73, [100, 700], 2, 64, 16, extra=2)
    av, want = c.want_attention()
    ab, wb = c.bounds()
    g = c.on_device(hstu)
    leave_an_error(hstu)
    c.attend(hstu, g)
    check_av(g["av"], av, ab)
    check_cache(g["cache"], want, wb)
    c.cache, weights = want, g["cache"].weights.double().cpu().numpy()
    c.cache["weights"] = weights
    rows, off, ts = values(c.rng, (2, 512), "bf16"), np.array([0, 1, 2]), np.array([7, 9])
    leave_an_error(hstu)
    hstu.hstu_cache_append(g["cache"], c.dev(rows, torch.bfloat16), c.dev(off, torch.int64),
                           c.dev(ts, torch.int64), g["table"], g["lens"] + 1, g["next"] + 1)
    assert hstu.device_status() == hstu.HSTU_OK
    paged.append(c.cache, rows, off, ts, c.table, c.lens + 1, c.next + 1)
    check_cache(g["cache"], c.cache)


def test_evict_a_long_history_captured_first(hstu):
    # in a process of its own: nothing has been asked of the device before the capture
    code = """
import numpy as np, torch
import hstu_sequential_transduction_layer_b200 as hstu
from oracle import paged
from tests.paged_util import Case, check_cache, same
c = Case(74, [40000], 1, 64, 1024, bias="none")
g = c.on_device(hstu)
ws = torch.empty(hstu.cache_evict_workspace_size(g["cache"], 1, c.M), dtype=torch.uint8, device="cuda")
graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(graph, stream=st):
    hstu.hstu_cache_evict(g["cache"], g["table"], g["lens"], g["next"], 9000, 100, new_lens=g["lens"],
                          workspace=ws)
graph.replay()
torch.cuda.synchronize()
assert hstu.device_status() == hstu.HSTU_OK
same(g["lens"], paged.evict(c.cache, c.table, c.lens, c.next, 9000, 100), "lengths")
check_cache(g["cache"], c.cache)
print("done")
"""
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "done", out.stderr[-2000:]


@pytest.mark.parametrize("lens,budget,recent,missing", [
    ([60, 60], 30, 4, [(0, 2)]),                       # a page above the budget, and one across it
    ([200, 60], 100, 20, [(0, 1), (0, 4), (1, 0)]),    # below it: more slots without a page than gaps
    ([200, 150], 90, 0, [(0, 0), (0, 2), (0, 9), (0, 12), (1, 5)]),
    ([100, 40], 30, 30, [(0, 0), (0, 1), (1, 1)]),     # only recent tokens stay: none moves for a missing page
    ([64, 50], 16, 3, [(0, 0)]),                       # every kept slot is on the missing page
    ([50, 200], 0, 0, [(0, 0), (1, 3)]),
    ([70, 300], 40, 8, [(0, j) for j in range(5)])])   # a history without any page
@pytest.mark.parametrize("entry", [-1, 1 << 30, "pages"])
def test_evict_rows_without_a_page(hstu, lens, budget, recent, missing, entry):
    c = Case(75, lens, 2, 64, 16, thinned=True)
    for b, j in missing:
        c.table[b, j] = len(c.cache["k"]) if entry == "pages" else entry
    g = c.on_device(hstu)
    new = hstu.hstu_cache_evict(g["cache"], g["table"], g["lens"], g["next"], budget, recent)
    assert hstu.device_status() == hstu.HSTU_ERR_DEVICE_BAD_OFFSETS
    assert hstu.device_status() == hstu.HSTU_OK
    same(new, paged.evict(c.cache, c.table, c.lens, c.next, budget, recent), "new_lens")
    check_cache(g["cache"], c.cache)          # pages of nobody included


@pytest.mark.parametrize("aliased", [False, True])
def test_evict_lengths_beyond_the_table(hstu, aliased):
    # sequence 0 fills its row, sequence 1's row is the table's and its tail names no page, sequence 2
    # is cut to what the row holds although the budget is larger
    c = Case(76, [96, 70, 96], 2, 64, 16, extra=0)
    c.lens[:] = [97, 1 << 50, 96]
    for budget in (40, 96, 500):
        d = copy.deepcopy(c)
        g = d.on_device(hstu)
        new = hstu.hstu_cache_evict(g["cache"], g["table"], g["lens"], g["next"], budget, 10,
                                    new_lens=g["lens"] if aliased else None)
        assert hstu.device_status() == hstu.HSTU_ERR_DEVICE_BAD_OFFSETS
        # the slots behind sequence 1's tokens hold NaN weights at position -5: they go first
        same(new, paged.evict(d.cache, d.table, d.lens, d.next, budget, 10), "new_lens")
        check_cache(g["cache"], d.cache)


@pytest.mark.parametrize("kind", ["random", "nan", "zero"])
def test_evict_a_long_history_without_some_pages(hstu, kind):
    # slots whose keys go through the workspace, and ties among the tokens that are left
    c = Case(77, [70001] + [100] * 9, 1, 64, 1024, bias="none")
    live = ~np.isnan(c.cache["weights"])
    if kind != "random":
        c.cache["weights"][live] = np.nan if kind == "nan" else 0.0
    c.table[0, [0, 13, 40, 66, 68]] = -1
    g = c.on_device(hstu)
    new = hstu.hstu_cache_evict(g["cache"], g["table"], g["lens"], g["next"], 30011, 1000)
    assert hstu.device_status() == hstu.HSTU_ERR_DEVICE_BAD_OFFSETS
    same(new, paged.evict(c.cache, c.table, c.lens, c.next, 30011, 1000), "new_lens")
    check_cache(g["cache"], c.cache)


@pytest.mark.parametrize("weights,bias", [(True, "rab"), (False, "rab"), (True, "alibi"), (False, "none")])
@pytest.mark.parametrize("append", [True, False])
def test_attention_without_positions_stores_the_token(hstu, weights, bias, append):
    # slot i holds position i; with and without weights, and (ALiBi, no bias) without timestamps
    c = Case(78, [40, 131, 0, -1], 2, 64, 16, weights=weights, positions=False, bias=bias)
    c.next[:] = c.lens
    g = c.on_device(hstu)
    c.attend(hstu, g, append)                # next_positions None: the cached lengths
    assert hstu.device_status() == hstu.HSTU_OK
    av, want = c.want_attention(append)
    ab, wb = c.bounds()
    check_av(g["av"], av, ab)
    check_cache(g["cache"], want, wb)


@pytest.mark.parametrize("dtype,H,hd,ps,bias", [("bf16", 8, 64, 16, "rab"), ("bf16", 4, 128, 64, "alibi"),
                                                ("fp32", 8, 32, 16, "time"), ("fp32", 2, 128, 32, "rab")])
def test_attention_many_tiles_a_warp(hstu, dtype, H, hd, ps, bias):
    """Eight tiles and more a warp, nearly all of one history: the producer refills stages inside a history
    and looks ahead along it."""
    c = Case(79, [2000 + 41 * i for i in range(25)], H, hd, ps, dtype, bias=bias, thinned=True, P=4000, Tb=32,
             spread=40000)
    tile = 4096 // (hd * (2 if dtype == "bf16" else 4))
    warps = torch.cuda.get_device_properties(0).multi_processor_count * 11
    assert H * sum(n // tile + 1 for n in c.lens.tolist()) >= 8 * warps
    g = c.on_device(hstu)
    av, want = c.want_attention()
    ab, wb = c.bounds()
    c.attend(hstu, g)
    assert hstu.device_status() == hstu.HSTU_OK
    check_av(g["av"], av, ab)
    check_cache(g["cache"], want, wb)


def test_layer_behind_an_earlier_error(hstu):
    H, hd, B = 2, 32, 3
    c = Case(80, [20, 5, 0], H, hd, 16, "fp32", bias="none")
    w = {k: c.dev(0.1 * c.rng.standard_normal(s), torch.float32)
         for k, s in (("W1", (64, 256)), ("b1", 256), ("W2", (64, 64)), ("b2", 64), ("ln_w", 64), ("ln_b", 64))}
    X = c.dev(values(c.rng, (B, 64), "fp32"), torch.float32)
    out = []
    for behind in (False, True):
        g = c.on_device(hstu)
        if behind:
            leave_an_error(hstu)
        out.append(hstu.hstu_paged_layer_fwd(g["shape"], g["cache"], X, g["table"], g["lens"], g["next"], None,
                                             w["W1"], w["b1"], w["W2"], w["b2"], w["ln_w"], w["ln_b"], None, None,
                                             None, c.scale))
        assert hstu.device_status() == hstu.HSTU_OK
        out.append(g["cache"].k.nan_to_num(7.0))
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])


@pytest.mark.parametrize("dtype,H,hd,ps,lens", [("bf16", 4, 64, 16, [900, 30, 2000, 500]), ("bf16", 8, 128, 64, [1300] * 9),
                                                ("fp32", 3, 128, 16, [700, 701, 1]), ("bf16", 1, 64, 1024, [3000])])
def test_calls_with_nothing_in_between(hstu, dtype, H, hd, ps, lens):
    """Each kernel's launch overlaps the one before it, with no other kernel between them: a fill, scores that
    sum weights, an eviction by them, more scores equal the same calls waited for one by one."""
    B, grow = len(lens), 40
    runs = []
    for wait in (False, True):
        c = Case(81, lens, H, hd, ps, dtype, extra=grow + 1)
        g = c.on_device(hstu)
        s = g["shape"]
        g["shape"] = hstu.make_shape(B, B, max(lens) + grow + 2, s.d_model, H, hd, hd, s.dtype, s.n_pos_buckets,
                                     s.n_time_buckets)
        off = torch.arange(B + 1, device="cuda") * grow
        rows = c.dev(values(c.rng, (B * grow, 4 * H * hd), dtype), c.torch_dtype())
        ts = g["now"].repeat_interleave(grow)
        more, seen = g["lens"] + grow, g["next"] + grow
        ws = torch.empty(hstu.paged_attention_workspace_size(g["shape"]), dtype=torch.uint8, device="cuda")
        es = torch.empty(hstu.cache_evict_workspace_size(g["cache"], B, c.M), dtype=torch.uint8, device="cuda")
        av = [torch.empty_like(g["av"]) for _ in range(17)]
        cut = torch.empty_like(more)
        torch.cuda.synchronize()

        def attend(k, lens, append=False):
            hstu.hstu_paged_attention_fwd(g["shape"], g["cache"], g["uvqk"], g["table"], lens, seen, g["now"], g["pos"],
                                          g["tim"], g["slopes"], c.scale, av[k], append=append, workspace=ws)
        for repeat in range(4):
            steps = [lambda: hstu.hstu_cache_append(g["cache"], rows, off, ts, g["table"], g["lens"], g["next"])]
            steps += [lambda k=k: attend(4 * repeat + k, more, k == 2) for k in range(3)]
            steps += [lambda: hstu.hstu_cache_evict(g["cache"], g["table"], more, seen, 600, 50, new_lens=cut, workspace=es),
                      lambda: attend(4 * repeat + 3, cut, True)]
            for step in steps:
                step()
                if wait:
                    torch.cuda.synchronize()
        attend(16, more)
        torch.cuda.synchronize()
        assert hstu.device_status() == hstu.HSTU_OK
        cache = g["cache"]
        runs.append([*av, cut, cache.k, cache.v, cache.weights, cache.positions, cache.timestamps])
    for a, b in zip(*runs):
        if a.is_floating_point():
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
        else:
            assert torch.equal(a, b)
