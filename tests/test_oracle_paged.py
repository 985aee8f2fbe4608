"""The paged cache's fp64 oracle, pinned on the CPU: its attention against the candidate oracle (one
candidate a user, pinned to the causal layer itself), its append against that attention, its
eviction against hand-worked cases."""
import copy

import numpy as np
import pytest

import oracle
from oracle import paged
from tests.paged_util import Case


def _contiguous(c, b):
    """Sequence b's cached U|V|Q|K rows (U and Q zero: never read)."""
    n, H, hd, ps = int(c.lens[b]), c.H, c.hd, c.ps
    rows = np.zeros((n, 4, H, hd))
    for j in range(n):
        p, o = c.table[b, j // ps], j % ps
        rows[j, 1], rows[j, 3] = c.cache["v"][p, :, o], c.cache["k"][p, :, o]
    return rows.reshape(n, 4 * H * hd)


@pytest.mark.parametrize("bias", ["rab", "pos", "time", "alibi", "none"])
def test_attention_is_one_candidate_against_a_contiguous_history(bias):
    c = Case(3, [0, 1, 17, 40, 130], 2, 64, 16, bias=bias)
    av, after = c.want_attention()
    for b, n in enumerate(c.lens):
        n = int(n)
        hist = _contiguous(c, b)
        ts = None
        if c.tim is not None:
            ts = np.array([c.cache["timestamps"][c.table[b, j // c.ps], j % c.ps] for j in range(n)],
                          np.int64)
        want = oracle.candidate_attention(
            np.array([0, n], np.int64), hist, np.array([0, 1], np.int64), c.uvqk[b:b + 1],
            num_heads=2, d_qk=64, d_v=64, hist_timestamps=ts,
            cand_timestamps=c.now[b:b + 1] if c.tim is not None else None, pos_table=c.pos,
            time_table=c.tim, alibi_slopes=c.slopes, scale=c.scale)
        assert np.abs(av[b] - want[0]).max() <= 1e-12 * max(1.0, np.abs(want).max())
        # the new token is the row after the last
        p, o = c.table[b, n // c.ps], n % c.ps
        assert (after["k"][p, :, o] == c.uvqk[b].reshape(4, 2, 64)[3]).all()
        assert after["positions"][p, o] == n


def test_weights_are_the_magnitudes_that_make_up_av():
    # V = 1 and positive weights: AV is their sum, each |a| lands on its token
    c = Case(4, [50], 1, 64, 16, bias="none")
    c.cache["v"][~np.isnan(c.cache["v"])] = 1.0
    c.uvqk = np.abs(c.uvqk)
    c.cache["k"] = np.abs(c.cache["k"])
    c.uvqk.reshape(1, 4, 64)[0, 1] = 1.0
    before = copy.deepcopy(c.cache["weights"])
    av, after = c.want_attention()
    p = c.table[0, np.arange(51) // 16]
    o = np.arange(51) % 16
    gained = after["weights"][p, 0, o] - np.nan_to_num(before[p, 0, o])
    assert abs(gained.sum() - av[0, 0]) <= 1e-12


def test_append_then_attend_token_by_token_is_the_forward():
    # a history decoded one token at a time gives the causal attention's rows
    c = Case(5, [0], 2, 64, 16, bias="pos", extra=30)
    rows = Case(6, [0] * 30, 2, 64, 16, bias="none").uvqk
    n = 12
    paged.append(c.cache, rows[:n], np.array([0, n]), None, c.table, c.lens, c.next)
    got = []
    for t in range(n, 30):
        got.append(paged.attention(c.cache, rows[t:t + 1], c.table, np.array([t]), np.array([t]), None,
                                   c.pos, None, None, 0.5)[0])
    want = oracle.attention(np.array([0, 30], np.int64), rows, num_heads=2, d_qk=64, d_v=64,
                            pos_table=c.pos, scale=0.5)
    assert np.abs(np.array(got) - want[n:]).max() <= 1e-12


def test_evict_by_hand():
    c = Case(7, [8], 2, 64, 16, bias="none")
    p = c.table[0, 0]
    c.cache["weights"][p, 0, :8] = [5, 1, 4, 0, 3, 9, 0, 2]
    c.cache["weights"][p, 1, :8] = [0, 1, 0, 0, 0, 0, 0, 0]
    k = c.cache["k"][p].copy()
    # recent = 1 protects position 7; of the others 5, 0, 2 are the largest: slots 0, 2, 5, 7 stay
    assert paged.evict(c.cache, c.table, c.lens, c.next, 4, 1).tolist() == [4]
    assert c.cache["positions"][p, :4].tolist() == [0, 5, 2, 7]
    assert (c.cache["k"][p, :, :4] == k[:, [0, 5, 2, 7]]).all()
    assert (c.cache["k"][p, :, 4:8] == k[:, 4:8]).all()


def test_evict_ties_go_to_the_lower_slot_and_nan_goes_first():
    c = Case(8, [6], 1, 64, 16, bias="none")
    p = c.table[0, 0]
    c.cache["weights"][p, 0, :6] = [1, np.nan, 1, 1, 1, np.inf]
    assert paged.evict(c.cache, c.table, c.lens, c.next, 3, 0).tolist() == [3]
    assert c.cache["positions"][p, :3].tolist() == [0, 5, 2]


def test_evict_leaves_short_and_inactive_sequences():
    c = Case(9, [5, -1, 4], 1, 64, 16, bias="none")
    before = copy.deepcopy(c.cache)
    assert paged.evict(c.cache, c.table, c.lens, c.next, 5, 2).tolist() == [5, -1, 4]
    for name in ("k", "v", "weights", "positions"):
        assert np.array_equal(before[name], c.cache[name], equal_nan=True)
