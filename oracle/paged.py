"""The paged cache's operators in fp64, written out plainly: a cache is a dict of numpy arrays k, v
[num_pages, H, page_size, hd], positions, timestamps [num_pages, page_size] and weights [num_pages, H,
page_size] (positions, timestamps and weights may be None), changed in place.  Test infrastructure
only.

The attention is Eq. 2 of the layer ("Actions Speak Louder than Words" paper notes, section 3.1) for
one new row; paging and eviction are this library's own.
"""
import math

import numpy as np


def _place(cache, table, b, i):
    ps = cache["k"].shape[2]
    return int(table[b, i // ps]), i % ps


def append(cache, uvqk, offsets, timestamps, table, lens, next_positions=None):
    H, hd = cache["k"].shape[1], cache["k"].shape[3]
    rows = uvqk.reshape(-1, 4, H, hd)
    for b in range(len(lens)):
        for i in range(int(offsets[b + 1] - offsets[b])):
            t = int(offsets[b]) + i
            p, o = _place(cache, table, b, int(lens[b]) + i)
            cache["v"][p, :, o], cache["k"][p, :, o] = rows[t, 1], rows[t, 3]
            if cache["positions"] is not None:
                cache["positions"][p, o] = (lens if next_positions is None else next_positions)[b] + i
            if cache["timestamps"] is not None:
                cache["timestamps"][p, o] = timestamps[t]
            if cache["weights"] is not None:
                cache["weights"][p, :, o] = 0.0


def silu(x):
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def attention(cache, uvqk, table, lens, next_positions, now, pos_table, time_table, slopes, scale,
              add=True):
    """AV [B, H*hd]; `add`: the new tokens join the cache.  lens[b] < 0: inactive."""
    H, hd = cache["k"].shape[1], cache["k"].shape[3]
    B = len(lens)
    rows = uvqk.reshape(B, 4, H, hd)
    av = np.zeros((B, H, hd))
    for b in range(B):
        n = int(lens[b])
        if n < 0:
            continue
        p_new = int(n if next_positions is None else next_positions[b])
        for j in range(n + 1):
            if j < n:
                p, o = _place(cache, table, b, j)
                k, v = cache["k"][p, :, o], cache["v"][p, :, o]
                dist = max(p_new - (j if cache["positions"] is None else int(cache["positions"][p, o])), 0)
                dt = int(now[b]) - int(cache["timestamps"][p, o]) if time_table is not None else 0
            else:
                k, v, dist, dt = rows[b, 3], rows[b, 1], 0, 0
            x = (rows[b, 2] * k).sum(-1)
            if pos_table is not None:
                x = x + pos_table[:, min(dist, pos_table.shape[1] - 1)]
            if time_table is not None:
                bucket = (1 + max(dt, 0)).bit_length() - 1
                x = x + time_table[:, min(bucket, time_table.shape[1] - 1)]
            if slopes is not None:
                x = x - slopes * dist
            a = scale * silu(x)
            av[b] += a[:, None] * v
            if j < n and cache["weights"] is not None:
                cache["weights"][p, :, o] += np.abs(a)
        if add:
            p, o = _place(cache, table, b, n)
            cache["k"][p, :, o], cache["v"][p, :, o] = rows[b, 3], rows[b, 1]
            if cache["positions"] is not None:
                cache["positions"][p, o] = p_new
            if cache["timestamps"] is not None and now is not None:
                cache["timestamps"][p, o] = now[b]
            if cache["weights"] is not None:
                cache["weights"][p, :, o] = np.abs(a)
    return av.reshape(B, H * hd)


def evict(cache, table, lens, next_positions, budget, recent):
    """New lengths; the kept tokens of the slots >= budget move into the gaps below.  A length beyond the
    table is the table's.  A slot whose entry is no page holds no token: below budget it stays one of
    the kept slots, from there on it is cut."""
    num_pages, ps = len(cache["k"]), cache["k"].shape[2]
    out = np.array(lens)
    for b in range(len(lens)):
        n = min(int(lens[b]), table.shape[1] * ps)
        out[b] = n
        if n <= budget:
            continue
        p_next = int(n if next_positions is None else next_positions[b])
        rank = []
        for j in range(n):
            p, o = _place(cache, table, b, j)
            if not 0 <= p < num_pages:
                rank.append((-1 if j < budget else 3, 0, 0.0, j))
                continue
            total = 0.0
            for w in cache["weights"][p, :, o]:
                total += float(w)
            total = float(np.float32(total))
            first = 0 if cache["positions"][p, o] >= p_next - recent else 1
            bad = math.isnan(total)
            rank.append((first, 1 if bad and first else 0, 0.0 if bad or not first else -total, j))
        kept = sorted(r[3] for r in sorted(rank)[:budget])
        stay = set(kept)
        gaps = [j for j in range(budget) if j not in stay]
        for to, frm in zip(gaps, [j for j in kept if j >= budget]):
            (pt, ot), (pf, of) = _place(cache, table, b, to), _place(cache, table, b, frm)
            for name in ("k", "v", "weights"):
                cache[name][pt, :, ot] = cache[name][pf, :, of]
            for name in ("positions", "timestamps"):
                if cache[name] is not None:
                    cache[name][pt, ot] = cache[name][pf, of]
        out[b] = budget
    return out
