"""Seeded paged-cache cases for the tests: fp64 numpy arrays holding values the device type can
represent, their device copies, and error bounds of the fp32 arithmetic."""
import copy

import numpy as np
import torch

from oracle import paged
from tests.gpu_util import round_bf16

U = 2.0 ** -24          # half a unit in the last place of fp32, relative


def values(rng, shape, dtype):
    x = rng.standard_normal(shape)
    x = x / (1.0 + np.exp(-x))          # as f1 leaves U, V, Q, K
    return round_bf16(x) if dtype == "bf16" else x.astype(np.float32).astype(np.float64)


class Case:
    """Caches of len(lens) sequences (lens[b] < 0: inactive) in a pool whose unused slots hold NaN.
    `extra`: room for this many more tokens a sequence."""

    def __init__(self, seed, lens, H, hd, ps, dtype="bf16", bias="rab", thinned=False,
                 weights=True, positions=True, extra=1, P=96, Tb=24, spread=500):
        rng = np.random.default_rng(seed)
        self.rng, self.dtype, self.H, self.hd, self.ps = rng, dtype, H, hd, ps
        self.lens = np.array(lens, np.int64)
        B = len(lens)
        need = [0 if n < 0 else -(-(n + extra) // ps) for n in lens]
        self.M = max(1, max(need))
        pages = sum(need) + 3
        order = rng.permutation(pages)
        self.table = np.full((B, self.M), -7, np.int32)
        nan = np.nan
        c = {"k": np.full((pages, H, ps, hd), nan), "v": np.full((pages, H, ps, hd), nan),
             "positions": np.full((pages, ps), -5, np.int64) if positions else None,
             "timestamps": np.full((pages, ps), -9, np.int64) if bias in ("rab", "time") else None,
             "weights": np.full((pages, H, ps), nan) if weights else None}
        at = 0
        self.next = np.zeros(B, np.int64)
        self.now = np.zeros(B, np.int64)
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            if n < 0:
                continue
            steps = rng.integers(1, 6, n) if thinned else np.ones(n, np.int64)
            pos = np.cumsum(steps) - 1 if n else np.zeros(0, np.int64)
            ts = 1_600_000_000 + np.cumsum(rng.integers(0, spread, n + 1))
            self.next[b] = pos[-1] + 1 + (3 if thinned else 0) if n else 0
            self.now[b] = ts[n]
            mix = rng.permutation(n) if thinned else np.arange(n)
            for j in range(n):
                p, o = self.table[b, j // ps], j % ps
                c["k"][p, :, o] = values(rng, (H, hd), dtype)
                c["v"][p, :, o] = values(rng, (H, hd), dtype)
                if positions:
                    c["positions"][p, o] = pos[mix[j]]
                if c["timestamps"] is not None:
                    c["timestamps"][p, o] = ts[mix[j]]
                if weights:
                    c["weights"][p, :, o] = np.float32(np.abs(rng.standard_normal(H)) * 1e-2)
        self.cache = c
        self.uvqk = values(rng, (B, 4 * H * hd), dtype)
        f = lambda n: (0.3 * rng.standard_normal((H, n))).astype(np.float32).astype(np.float64)  # noqa: E731
        self.pos = f(P) if bias in ("rab", "pos") else None
        self.tim = f(Tb) if bias in ("rab", "time") else None
        self.slopes = (2.0 ** (-8.0 * np.arange(1, H + 1) / H)).astype(np.float32).astype(np.float64) \
            if bias == "alibi" else None
        self.scale = float(np.float32(1.0 / max(1, max(lens))))

    def bounds(self):
        """|error| bounds of AV [B, H*hd] and of the weights' sums, from the values themselves: a dot
        product of hd terms and three bias terms, SiLU (slope at most 1.1; 8 roundings), a sum of n
        products.  Every sum is bounded as if taken one term after the other."""
        H, hd, ps = self.H, self.hd, self.ps
        av = np.zeros((len(self.lens), H, hd))
        wb = None if self.cache["weights"] is None else np.zeros_like(self.cache["weights"])
        for b, n in enumerate(self.lens):
            if n < 0:
                continue
            n = int(n)
            u, v1, q, k1 = self.uvqk[b].reshape(4, H, hd)
            j = np.arange(n)
            p, o = self.table[b, j // ps], j % ps
            K = np.concatenate([self.cache["k"][p, :, o], k1[None]])
            V = np.concatenate([self.cache["v"][p, :, o], v1[None]])
            mag = (np.abs(K) * np.abs(q)).sum(-1)                     # [n + 1, H]
            for t in (self.pos, self.tim):
                if t is not None:
                    mag = mag + np.abs(t).max(1)
            if self.slopes is not None:
                mag = mag + self.slopes * (float(self.next[b]) + 1)
            ex = (hd + 8) * U * mag
            ea = abs(self.scale) * (1.1 * ex + 8 * U * mag)
            amax = abs(self.scale) * mag                              # |SiLU(x)| <= |x| <= mag
            # terms: one product each, n + 1 of them summed
            av[b] = (ea[..., None] * np.abs(V)).sum(0) + (n + 16) * U * (amax[..., None] * np.abs(V)).sum(0)
            if wb is not None:
                w = np.nan_to_num(self.cache["weights"][p, :, o])
                wb[p, :, o] = ea[:n] + 2 * U * (np.abs(w) + amax[:n])
                if n // ps < self.M and self.table[b, n // ps] >= 0:
                    wb[self.table[b, n // ps], :, n % ps] = ea[n]
        return av.reshape(len(self.lens), H * hd), wb

    def want_attention(self, append=True):
        """(AV, cache after the call) by the oracle."""
        c = copy.deepcopy(self.cache)
        av = paged.attention(c, self.uvqk, self.table, self.lens, self.next, self.now, self.pos,
                             self.tim, self.slopes, self.scale, append)
        return av, c

    # ---------------------------------------------------------------- device side
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype == "bf16" else torch.float32

    def dev(self, a, dt):
        return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda()

    def on_device(self, hstu):
        c = self.cache
        d = self.torch_dtype()
        cache = hstu.PagedCache(self.dev(c["k"], d), self.dev(c["v"], d),
                                self.dev(c["positions"], torch.int32),
                                self.dev(c["timestamps"], torch.int64),
                                self.dev(c["weights"], torch.float32))
        B, H, hd = len(self.lens), self.H, self.hd
        g = {"cache": cache, "uvqk": self.dev(self.uvqk, d), "table": self.dev(self.table, torch.int32),
             "lens": self.dev(self.lens, torch.int64), "next": self.dev(self.next, torch.int64),
             "now": self.dev(self.now, torch.int64), "pos": self.dev(self.pos, torch.float32),
             "tim": self.dev(self.tim, torch.float32), "slopes": self.dev(self.slopes, torch.float32)}
        g["shape"] = hstu.make_shape(B, B, max(1, int(self.lens.max()) + 1), max(64, H * hd), H, hd, hd,
                                     hstu.HSTU_BF16 if self.dtype == "bf16" else hstu.HSTU_F32,
                                     0 if self.pos is None else self.pos.shape[1],
                                     0 if self.tim is None else self.tim.shape[1])
        g["av"] = torch.full((B, H * hd), float("nan"), device="cuda")
        return g

    def attend(self, hstu, g, append=True, **kw):
        return hstu.hstu_paged_attention_fwd(g["shape"], g["cache"], g["uvqk"], g["table"], g["lens"],
                                             g["next"] if self.cache["positions"] is not None else None,
                                             g["now"], g["pos"], g["tim"], g["slopes"], self.scale,
                                             g["av"], append=append, **kw)


def same(t, want, what):
    """Bit-exact equality of a device array with fp64 or integer values (NaN equals NaN)."""
    got = t.double().cpu().numpy() if t.is_floating_point() else t.long().cpu().numpy()
    ok = (got == want) | ((got != got) & (want != want)) if t.is_floating_point() else got == want
    assert ok.all(), f"{what}: {np.argwhere(~ok)[:5].tolist()} differ of {ok.size} ({(~ok).sum()})"


def check_cache(cache, want, weight_bound=None):
    same(cache.k, want["k"], "k")
    same(cache.v, want["v"], "v")
    if want["positions"] is not None:
        same(cache.positions, want["positions"], "positions")
    if want["timestamps"] is not None:
        same(cache.timestamps, want["timestamps"], "timestamps")
    if want["weights"] is not None:
        if weight_bound is None:
            same(cache.weights, want["weights"], "weights")
            return
        got = cache.weights.double().cpu().numpy()
        nan = np.isnan(want["weights"])
        assert (np.isnan(got) == nan).all(), "weights: slots that hold no token were written"
        bad = np.abs(got - want["weights"]) > weight_bound
        assert not bad[~nan].any(), f"weights: {np.argwhere(bad & ~nan)[:5].tolist()}"


def check_av(av, want, bound, what="AV"):
    got = av.double().cpu().numpy()
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - want) - bound
    assert (over <= 0).all(), f"{what}: off by {np.abs(got - want).max():.3e}, " \
        f"{(over > 0).sum()} values beyond their bounds, first {np.argwhere(over > 0)[:3].tolist()}"
