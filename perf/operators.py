"""Cases of the paged-cache operators: attention of one new token a user over a paged key-value
cache, filling the cache from a forward's U|V|Q|K, and eviction by accumulated attention weight.

`own = False` computes the operators from their formulas with elementary torch operations; `own =
True` calls the library.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------

def _attention(name, dtype, heads, head_dim, page_size, users, shortest, longest, power, bias, P=0,
               Tb=0, gap=60, weights=False, thinned=False, append=True):
    c = dict(op="attention", dtype=dtype, heads=heads, head_dim=head_dim, page_size=page_size,
             users=users, shortest=shortest, longest=longest, power=power, bias=bias, P=P, Tb=Tb,
             gap=gap, weights=weights, thinned=thinned, append=append)
    return dict(c, name=name) if name else c


def _append(name, dtype, heads, head_dim, page_size, users, cached, shortest, longest, power):
    c = dict(op="append", dtype=dtype, heads=heads, head_dim=head_dim, page_size=page_size,
             users=users, cached=cached, shortest=shortest, longest=longest, power=power)
    return dict(c, name=name) if name else c


def _evict(name, dtype, heads, head_dim, page_size, users, shortest, longest, budget, recent):
    c = dict(op="evict", dtype=dtype, heads=heads, head_dim=head_dim, page_size=page_size,
             users=users, shortest=shortest, longest=longest, power=0.0, budget=budget,
             recent=recent)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the first actions of a new user, fp32 heads of the smallest configuration: latency
        _attention("attention_new_user_fp32", "fp32", 2, 32, 16, 1, 17, 17, 0.0, "rab", 64, 32),
        # one user of the long-sequence benchmark's model at its full history: the split over length
        _attention("attention_one_user_8k", "bf16", 8, 64, 64, 1, 8191, 8191, 0.0, "rab", 8192, 128),
        # a batch of short ragged histories (two-layer retrieval model), small pages, weights kept
        _attention("attention_retrieval_batch", "bf16", 4, 64, 16, 128, 16, 1024, 1.5, "rab", 128,
                   64, gap=300, weights=True),
        # the long-sequence model's batch after evictions: gaps in the positions, weights kept
        _attention("attention_long_thinned", "bf16", 8, 64, 64, 24, 4000, 8192, 0.0, "rab", 8192,
                   128, weights=True, thinned=True),
        # ranking with ALiBi, wide heads; the token is scored and not stored
        _attention("attention_alibi_rank", "bf16", 8, 128, 32, 64, 256, 4096, 0.0, "alibi",
                   append=False),
        # the widest model, ragged histories: bandwidth
        _attention("attention_large", "bf16", 32, 128, 128, 32, 512, 8192, 1.2, "rab", 8192, 128,
                   gap=3600, weights=True),
        # a few new actions a user onto short histories
        _append("append_few_actions", "bf16", 4, 64, 16, 61, 100, 0, 9, 0.0),
        # whole histories of the long-sequence benchmark into an empty cache
        _append("append_whole_histories", "bf16", 8, 64, 64, 8, 0, 8192, 8192, 0.0),
        # ragged pieces of the widest model's histories, continuing inside a page
        _append("append_large_pieces", "bf16", 32, 128, 128, 16, 77, 1, 700, 0.0),
        # a serving loop's regular eviction: one page above the budget
        _evict("evict_one_page", "bf16", 8, 64, 64, 48, 4097, 4160, 4096, 64),
        # histories cut to half at once
        _evict("evict_half", "bf16", 8, 64, 64, 8, 8192, 8192, 4096, 128),
        # one very long history cut to a quarter
        _evict("evict_one_long_user", "bf16", 8, 64, 16, 1, 32771, 32771, 8192, 1000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "evict"])
    dtype = "fp32" if rng.random() < 0.2 else "bf16"
    heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 16, 32])
    head_dim = rng.choice([32, 64, 128] if dtype == "fp32" else [64, 128])
    page_size = rng.choice([16, 32, 64, 128, 256])
    row = 2 * heads * head_dim * (4 if dtype == "fp32" else 2)
    if op == "attention":
        longest = _log_int(rng, 1, 32768)
        users = _log_int(rng, 1, max(1, min(256, int(1.2e9 / (row * longest)))))
        shortest = rng.randint(0, longest)
        bias = rng.choice(["rab", "rab", "pos", "time", "alibi", "none"])
        return _attention(None, dtype, heads, head_dim, page_size, users, shortest, longest,
                          rng.choice([0.0, 1.2, 1.5]), bias,
                          _log_int(rng, 1, 8192) if bias in ("rab", "pos") else 0,
                          _log_int(rng, 1, 128) if bias in ("rab", "time") else 0,
                          gap=rng.choice([60, 300, 3600]), weights=rng.random() < 0.5,
                          thinned=rng.random() < 0.5, append=rng.random() < 0.7)
    if op == "append":
        longest = _log_int(rng, 1, 8192)
        users = _log_int(rng, 1, max(1, min(256, int(2.5e8 / (row * longest)))))
        return _append(None, dtype, heads, head_dim, page_size, users, rng.randint(0, 300),
                       rng.randint(0, longest), longest, rng.choice([0.0, 1.2]))
    longest = _log_int(rng, 2, 32768)
    users = _log_int(rng, 1, max(1, min(64, int(3e8 / (row * longest)))))
    budget = rng.randint(1, longest)
    return _evict(None, dtype, heads, head_dim, page_size, users, rng.randint(0, longest), longest,
                  budget, rng.randint(0, budget))


def _lengths(case):
    """Tokens a user, fixed by the case: p(n) ~ n^-power on [shortest, longest] (power 0: uniform)."""
    lo, hi, B = case["shortest"], case["longest"], case["users"]
    u = np.random.default_rng([B, lo, hi, case["page_size"]]).random(B)
    if case["power"] == 0.0:
        return np.minimum(hi, lo + np.floor(u * (hi - lo + 1))).astype(np.int64)
    e = 1.0 - case["power"]
    a, b = max(lo, 1) ** e, (hi + 1) ** e
    return np.clip(np.floor((a + u * (b - a)) ** (1.0 / e)), lo, hi).astype(np.int64)


def work(case):
    n = _lengths(case)
    B, H, hd, ps = case["users"], case["heads"], case["head_dim"], case["page_size"]
    es = 4 if case["dtype"] == "fp32" else 2
    row = 2 * H * hd * es                            # K and V of one token
    if case["op"] == "attention":
        N = int(n.sum())
        token = row + (8 * H if case["weights"] else 0)
        token += 4 if case["bias"] in ("rab", "pos", "alibi") else 0
        token += 8 if case["bias"] in ("rab", "time") else 0
        user = H * hd * es + row + H * hd * 4 + (row if case["append"] else 0)
        pages = int(-(-n // ps).sum())
        tables = 4 * H * (min(case["P"], int(n.max()) + 1) + case["Tb"])
        return {"bytes": N * token + B * user + 4 * pages + tables, "flops": (N + B) * H * (4 * hd + 12)}
    if case["op"] == "append":
        T = max(1, int(n.sum()))
        return {"bytes": T * (2 * row + 20 + 4 * H) + 16 * B, "flops": 0}
    cut = n[n > case["budget"]]
    front = np.minimum(case["budget"], cut - case["recent"])      # slots that may become gaps
    gaps = front * (1.0 - (case["budget"] - case["recent"]) / np.maximum(cut - case["recent"], 1))
    moved = float(gaps.sum())
    return {"bytes": int(cut.sum()) * (4 * H + 4) + moved * 2 * (row + 4 * H + 12) + 16 * B,
            "flops": int(cut.sum()) * H}


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, H, hd, ps, B = (DTYPES[case["dtype"]], case["heads"], case["head_dim"], case["page_size"],
                        case["users"])
    n = _lengths(case)
    attention, append, evict = (case["op"] == o for o in ("attention", "append", "evict"))
    cached = np.full(B, case["cached"], np.int64) if append else n
    room = cached + (n if append else 0) + (1 if attention else 0)
    need = -(-room // ps)
    M = max(1, int(need.max()))
    pages = int(need.sum()) + 5

    def act(*shape):       # K, V, Q as f1 leaves them: SiLU of a projection
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        return (x * torch.sigmoid(x)).to(dt)

    # pages are handed out in no order; entries past a user's own are -1
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = np.cumsum(need) - need
    idx = np.arange(M)[None] + at[:, None]
    used = torch.from_numpy(np.arange(M)[None] < need[:, None]).cuda()
    table = torch.where(used, order[torch.from_numpy(np.minimum(idx, pages - 1)).cuda()], -1)
    # positions 0, 1, ... or, after evictions, an unordered subset; integer seconds, growing
    slots = torch.arange(M * ps, device="cuda")
    if case.get("thinned"):
        pos = torch.cumsum(1 + (torch.rand((B, M * ps), generator=g, device="cuda") < 0.3).long()
                           * torch.randint(0, 9, (B, M * ps), generator=g, device="cuda"), 1)
    else:
        pos = slots.expand(B, -1).contiguous()
    lens = torch.from_numpy(cached).cuda()
    live = slots[None] < lens[:, None]
    steps = -torch.log1p(-torch.rand((B, M * ps), generator=g, device="cuda", dtype=torch.float64))
    ts = (1.6e9 + torch.cumsum(steps * case.get("gap", 60), 1)).floor().long()
    last = (lens - 1).clamp(min=0)[:, None]
    nxt = torch.where(lens > 0, pos.gather(1, last)[:, 0] + 1, 0)
    now = ts.gather(1, last)[:, 0] + case.get("gap", 60)
    if case.get("thinned"):
        mix = torch.rand((B, M * ps), generator=g, device="cuda").masked_fill(~live, 2.0).argsort(1)
        pos, ts = pos.gather(1, mix), ts.gather(1, mix)
    s = {"case": case, "page_table": table, "cache_lens": lens, "next_positions": nxt,
         "timestamps": torch.zeros((pages, ps), dtype=torch.int64, device="cuda"),
         "positions": torch.zeros((pages, ps), dtype=torch.int32, device="cuda"), "weights": None}
    owned = used.repeat_interleave(ps, 1)
    flat = (table.long().repeat_interleave(ps, 1) * ps + slots % ps)[owned]
    s["positions"].view(-1)[flat] = pos[owned].int()
    s["timestamps"].view(-1)[flat] = ts[owned]
    s["k"], s["v"] = act(pages, H, ps, hd), act(pages, H, ps, hd)
    if case.get("weights") or append or evict:
        # sums of |a| over many steps: spread over decades; tokens no step has seen yet hold 0
        w = torch.randn((pages, H, ps), generator=g, device="cuda")
        s["weights"] = torch.exp(w) * 1e-3
        s["weights"][(torch.rand((pages, ps), generator=g, device="cuda") < 0.05)[:, None, :]
                     .expand(-1, H, -1)] = 0.0
    if attention:
        s["uvqk"] = act(B, 4 * H * hd)
        s["now"] = now
        s["scale"] = 1.0 / max(1, case["longest"])
        tab = lambda c: 0.02 * torch.randn((H, c), generator=g, device="cuda") if c else None  # noqa: E731
        s["pos_table"], s["time_table"] = tab(case["P"]), tab(case["Tb"])
        s["slopes"] = None
        if case["bias"] == "alibi":
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
        s["av"] = torch.empty((B, H * hd), device="cuda")
    elif append:
        T = int(n.sum())
        s["uvqk"] = act(T, 4 * H * hd)
        s["seq_offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).cuda()
        s["new_times"] = now.repeat_interleave(torch.from_numpy(n).cuda(), output_size=T)
    else:
        s["weights_before"], s["positions_before"] = s["weights"].clone(), s["positions"].clone()
        s["new_lens"] = torch.empty_like(lens)
    if own:
        import hstu_sequential_transduction_layer_b200 as hstu
        s["cache"] = hstu.PagedCache(s["k"], s["v"], s["positions"], s["timestamps"], s["weights"])
        if attention:
            s["shape"] = hstu.make_shape(B, B, int(n.max()) + 1, H * hd, H, hd, hd,
                                         hstu.HSTU_F32 if dt == torch.float32 else hstu.HSTU_BF16,
                                         case["P"], case["Tb"])
            size = hstu.paged_attention_workspace_size(s["shape"])
        elif evict:
            size = hstu.cache_evict_workspace_size(s["cache"], B, M)
        if not append:
            s["workspace"] = torch.empty(max(256, size), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op == "evict":
        # what the last pass moved goes back, so that every pass evicts from a full cache
        s["weights"].copy_(s["weights_before"])
        s["positions"].copy_(s["positions_before"])
    if own:
        _own(s, op)
    else:
        {"attention": _plain_attention, "append": _plain_append, "evict": _plain_evict}[op](s)
    out = {"k": s["k"], "v": s["v"], "positions": s["positions"], "timestamps": s["timestamps"]}
    if s["weights"] is not None:
        out["weights"] = s["weights"]
    if op == "attention":
        out["av"] = s["av"]
    if op == "evict":
        out["new_lens"] = s["new_lens"]
    return out


def _own(s, op):
    import hstu_sequential_transduction_layer_b200 as hstu
    c = s["case"]
    if op == "attention":
        hstu.hstu_paged_attention_fwd(s["shape"], s["cache"], s["uvqk"], s["page_table"],
                                      s["cache_lens"], s["next_positions"], s["now"],
                                      s["pos_table"], s["time_table"], s["slopes"], s["scale"],
                                      s["av"], append=c["append"], workspace=s["workspace"])
    elif op == "append":
        hstu.hstu_cache_append(s["cache"], s["uvqk"], s["seq_offsets"], s["new_times"],
                               s["page_table"], s["cache_lens"], s["next_positions"])
    else:
        hstu.hstu_cache_evict(s["cache"], s["page_table"], s["cache_lens"], s["next_positions"],
                              c["budget"], c["recent"], s["new_lens"], workspace=s["workspace"])


def _slots(s):
    """Page and slot of every (user, index), and which indices are cached."""
    ps, table = s["case"]["page_size"], s["page_table"].long().clamp(min=0)
    i = torch.arange(table.shape[1] * ps, device="cuda")
    return table[:, i // ps], (i % ps).expand(table.shape[0], -1), i[None] < s["cache_lens"][:, None]


def _plain_attention(s):
    c, B = s["case"], s["uvqk"].shape[0]
    H, hd, ps = c["heads"], c["head_dim"], c["page_size"]
    _, v1, q, k1 = s["uvqk"].view(B, 4, H, hd).unbind(1)
    page, slot, live = _slots(s)
    x = (s["k"][page, :, slot].float() * q.float()[:, None]).sum(-1)            # [B, L, H]
    x1 = (q.float() * k1.float()).sum(-1)                                       # [B, H]
    far = (s["next_positions"][:, None] - s["positions"][page, slot]).clamp(min=0)
    if s["slopes"] is not None:
        x = x - s["slopes"] * far[..., None].float()
    if s["pos_table"] is not None:
        x = x + s["pos_table"].t()[far.clamp(max=c["P"] - 1)]
        x1 = x1 + s["pos_table"][:, 0]
    if s["time_table"] is not None:
        ago = (s["now"][:, None] - s["timestamps"][page, slot]).clamp(min=0)
        bucket = torch.frexp((1 + ago).double())[1].long() - 1
        x = x + s["time_table"].t()[bucket.clamp(max=c["Tb"] - 1)]
        x1 = x1 + s["time_table"][:, 0]
    a = s["scale"] * x / (1 + torch.exp(-x)) * live[..., None]
    a1 = s["scale"] * x1 / (1 + torch.exp(-x1))
    av = (a[..., None] * s["v"][page, :, slot].float()).sum(1) + a1[..., None] * v1.float()
    s["av"].copy_(av.reshape(B, H * hd))
    h = torch.arange(H, device="cuda")
    if s["weights"] is not None:
        at = (page[..., None] * H + h) * ps + slot[..., None]
        s["weights"].view(-1).index_add_(0, at.reshape(-1), a.abs().reshape(-1))
    if c["append"]:
        n = s["cache_lens"]
        p, o = page.gather(1, n[:, None])[:, 0], n % ps
        s["k"][p, :, o], s["v"][p, :, o] = k1, v1
        s["positions"][p, o], s["timestamps"][p, o] = s["next_positions"].int(), s["now"]
        if s["weights"] is not None:
            s["weights"][p, :, o] = a1.abs()


def _plain_append(s):
    c, T = s["case"], s["uvqk"].shape[0]
    ps = c["page_size"]
    _, v, _, k = s["uvqk"].view(T, 4, c["heads"], c["head_dim"]).unbind(1)
    off = s["seq_offsets"]
    user = torch.searchsorted(off, torch.arange(T, device="cuda"), right=True) - 1
    i = torch.arange(T, device="cuda") - off[user]
    at = s["cache_lens"][user] + i
    p, o = s["page_table"].long()[user, at // ps], at % ps
    s["k"][p, :, o], s["v"][p, :, o] = k, v
    s["positions"][p, o] = (s["next_positions"][user] + i).int()
    s["timestamps"][p, o] = s["new_times"]
    s["weights"][p, :, o] = torch.zeros((), device="cuda")


def _plain_evict(s):
    c, n = s["case"], s["cache_lens"]
    budget = c["budget"]
    page, slot, live = _slots(s)
    score = s["weights"][page, :, slot].double().sum(-1).float()                # [B, L]
    recent = s["positions"][page, slot] >= (s["next_positions"] - c["recent"])[:, None]
    # kept first: the recent ones, then by weight; unused slots last; equal ones by slot
    score = torch.where(recent, math.inf, score).masked_fill(~live, -math.inf)
    rank = score.sort(dim=1, descending=True, stable=True)[1].argsort(1)
    i = torch.arange(score.shape[1], device="cuda")[None]
    cut = (n > budget)[:, None]
    keep = rank < budget
    gap, mover = cut & ~keep & (i < budget), cut & live & keep & (i >= budget)
    # the j-th gap takes the j-th kept slot past the budget
    to = torch.where(gap, i, 1 << 40).sort(dim=1)[0]
    frm = torch.where(mover, i, 1 << 40).sort(dim=1)[0]
    j, b = (to < 1 << 40).nonzero(as_tuple=True)[::-1]
    to, frm = to[b, j], frm[b, j]
    pt, st, pf, sf = page[b, to], slot[b, to], page[b, frm], slot[b, frm]
    for name in ("k", "v", "weights"):
        s[name][pt, :, st] = s[name][pf, :, sf]
    for name in ("positions", "timestamps"):
        s[name][pt, st] = s[name][pf, sf]
    s["new_lens"].copy_(n.clamp(max=budget))


# ------------------------------------------------------------------------------------------------
# The definition in 64 bits, user by user
# ------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    H, hd, ps, B = case["heads"], case["head_dim"], case["page_size"], case["users"]
    table, lens = s["page_table"].tolist(), s["cache_lens"].tolist()
    nxt = s["next_positions"].tolist()
    out = {"positions": s["positions"].clone(), "timestamps": s["timestamps"].clone(),
           "k": None, "v": None}
    w = s["weights"]
    if w is not None:
        out["weights"] = w.double()
    place = lambda b, i: (table[b][i // ps], i % ps)  # noqa: E731
    if case["op"] == "append":
        off = s["seq_offsets"].tolist()
        k, v = s["k"].double(), s["v"].double()
        rows = s["uvqk"].double().reshape(-1, 4, H, hd)
        for b in range(B):
            r, m = off[b], off[b + 1] - off[b]
            i = 0
            while i < m:             # up to the end of each page
                p, o = place(b, lens[b] + i)
                e = min(ps - o, m - i)
                k[p, :, o:o + e] = rows[r + i:r + i + e, 3].transpose(0, 1)
                v[p, :, o:o + e] = rows[r + i:r + i + e, 1].transpose(0, 1)
                first = nxt[b] + i
                out["positions"][p, o:o + e] = torch.arange(first, first + e, device="cuda").int()
                out["timestamps"][p, o:o + e] = s["new_times"][r + i:r + i + e]
                out["weights"][p, :, o:o + e] = 0.0
                i += e
        return dict(out, k=k, v=v)
    if case["op"] == "evict":
        k, v = s["k"].double(), s["v"].double()
        tm, ps_in = s["timestamps"], s["positions"]
        out["new_lens"] = s["cache_lens"].clone()
        for b in range(B):
            n, m = lens[b], case["budget"]
            if n <= m:
                continue
            out["new_lens"][b] = m
            pg = torch.tensor(table[b], device="cuda")[:-(-n // ps)]
            sums = w[pg].double().sum(1).reshape(-1)[:n].float().cpu().numpy()
            recent = (ps_in[pg].reshape(-1)[:n] >= nxt[b] - case["recent"]).cpu().numpy()
            order = np.lexsort((np.arange(n), -sums.astype(np.float64), ~recent))
            keep = np.zeros(n, bool)
            keep[order[:m]] = True
            to = np.flatnonzero(~keep[:m])
            frm = m + np.flatnonzero(keep[m:])
            tp, fp = pg[torch.from_numpy(to // ps).cuda()], pg[torch.from_numpy(frm // ps).cuda()]
            to, fo = torch.from_numpy(to % ps).cuda(), torch.from_numpy(frm % ps).cuda()
            for x, y in ((k, s["k"]), (v, s["v"]), (out["weights"], w)):
                x[tp, :, to] = y[fp, :, fo].double()
            for x, y in ((out["positions"], ps_in), (out["timestamps"], tm)):
                x[tp, to] = y[fp, fo]
        return dict(out, k=k, v=v)
    out["av"] = torch.zeros((B, H * hd), dtype=torch.float64, device="cuda")
    powers = 2.0 ** torch.arange(1, 62, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = lens[b]
        pg = torch.tensor(table[b], device="cuda")[:-(-n // ps)]
        u, v1, q, k1 = s["uvqk"][b].double().reshape(4, H, hd)
        K = torch.cat([s["k"][pg].double().transpose(0, 1).reshape(H, -1, hd)[:, :n], k1[:, None]], 1)
        V = torch.cat([s["v"][pg].double().transpose(0, 1).reshape(H, -1, hd)[:, :n], v1[:, None]], 1)
        x = torch.matmul(K, q[..., None])[..., 0]
        here = s["next_positions"][b:b + 1].int()
        dist = here - torch.cat([s["positions"][pg].reshape(-1)[:n], here])
        dt = s["now"][b] - torch.cat([s["timestamps"][pg].reshape(-1)[:n], s["now"][b:b + 1]])
        if case["bias"] == "alibi":
            x = x - s["slopes"].double()[:, None] * dist
        if case["P"]:
            x = x + s["pos_table"].double()[:, dist.clamp(0, case["P"] - 1).long()]
        if case["Tb"]:
            bucket = ((1.0 + dt.clamp(min=0).double())[:, None] >= powers).sum(1)
            x = x + s["time_table"].double()[:, bucket.clamp(max=case["Tb"] - 1)]
        a = float(np.float32(s["scale"])) * x * torch.sigmoid(x)
        out["av"][b] = torch.matmul(a[:, None], V).reshape(-1)
        if w is not None:
            for j, p in enumerate(pg.tolist()):
                e = min(ps, n - j * ps)
                out["weights"][p, :, :e] += a[:, j * ps:j * ps + e].abs()
        if case["append"]:
            p, o = place(b, n)
            out["positions"][p, o], out["timestamps"][p, o] = here[0], s["now"][b]
            if w is not None:
                out["weights"][p, :, o] = a[:, n].abs()
    return out
