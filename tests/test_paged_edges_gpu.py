"""The paged cache on the GPU in calls beside the everyday ones (tests/test_paged_gpu.py): behind other
work, behind a CUDA error of an earlier call, with rows that name no page, without the optional
arrays, and with many tiles of one history a warp.  Against the fp64 oracle (oracle/paged.py)."""
import copy

import numpy as np
import pytest
import torch

from oracle import paged
from tests.paged_util import Case, check_cache, same

pytestmark = pytest.mark.gpu


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
