"""What is measured of the window attention, the paged decode attention and the cache's pages.

``listed()`` names the cases, ``prepare`` makes a case's inputs from a seed, ``run`` makes one
pass (the plain torch form, or with ``own`` the library's calls), ``exact`` gives the outputs in
64 bits and ``work`` the bytes and operations that a pass cannot do without.

Kinds of cases:

* ``fwd``     sliding-window attention with sink tokens over a contiguous cache, out and log-sum-exp;
* ``train``   the same forward followed by its backward pass, as one layer of a training step;
* ``decode``  attention of the newest token(s) over a paged cache;
* ``append``  new tokens put into a paged cache (pages taken, rows written);
* ``beam``    rows forked, one token appended to parents and children (shared last pages are
  copied), parents freed: one step of a search that branches;
* ``compact`` a fragmented pool's live pages moved to its lowest ids.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _window(name, kind, T, h_q, h_kv, d_qk, d_v, window, sink, batch=1, q_pos0=0):
    return {"name": name, "kind": kind, "batch": batch, "seqlen_q": T, "q_pos0": q_pos0, "h_q": h_q,
            "h_kv": h_kv, "d_qk": d_qk, "d_v": d_v, "window": window, "sink": sink}


def _paged(name, kind, batch, h_q, h_kv, d_qk, d_v, page, max_len, min_len, new=1, window=0, sink=0):
    return {"name": name, "kind": kind, "batch": batch, "h_q": h_q, "h_kv": h_kv, "d_qk": d_qk, "d_v": d_v,
            "page": page, "max_len": max_len, "min_len": min_len, "new": new, "window": window, "sink": sink}


def listed():
    return [
        # a short prompt through one small layer (the tiny workload's heads, an odd length): latency
        _window("prefill_tiny", "fwd", 1000, 4, 1, 64, 64, 128, 4),
        # a batch of prompts through a layer without head groups and a ragged window
        _window("prefill_mha", "fwd", 8192, 16, 16, 128, 128, 1000, 16, batch=2),
        # a long prompt at the grouped 192/128 heads, window 512 and one block of sinks
        _window("prefill_gqa", "fwd", 16384, 64, 4, 192, 128, 512, 64),
        # training steps: a tiny layer; grouped heads; a full-attention layer (the window covers everything)
        _window("train_tiny", "train", 1000, 4, 1, 64, 64, 128, 4),
        _window("train_gqa", "train", 8192, 64, 4, 192, 128, 512, 64),
        _window("train_full", "train", 4096, 16, 16, 128, 128, 4096, 0),
        # one conversation, its newest token: latency
        _paged("decode_one", "decode", 1, 16, 16, 128, 128, 64, 1000, 1000),
        # a serving batch of ragged lengths at the grouped heads
        _paged("decode_ragged", "decode", 64, 64, 4, 192, 128, 64, 32768, 1),
        # four drafted tokens at a time, sliding window with sinks, small pages
        _paged("decode_window", "decode", 48, 32, 8, 128, 128, 16, 16000, 2000, new=4, window=4096, sink=16),
        # prompts of ragged lengths written into their pages
        _paged("append_prompts", "append", 16, 64, 4, 192, 128, 64, 0, 0, new=4096),
        # a search that branches: 32 rows forked, a token each, parents freed
        _paged("beam_step", "beam", 64, 64, 4, 192, 128, 64, 4000, 100),
        # half of a pool's rows have ended: the rest is moved together
        _paged("compact_pool", "compact", 96, 64, 4, 192, 128, 64, 6000, 500),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    kind = rng.choice(["fwd", "train", "decode", "append", "beam", "compact"])
    d_qk, d_v = rng.choice([(64, 64), (128, 128), (192, 128), (128, 64), (64, 128)])
    h_kv = rng.choice([1, 2, 4, 8])
    h_q = h_kv * rng.choice([1, 2, 4, 6, 8, 16])
    if kind in ("fwd", "train"):
        T = _log(rng, 200, 16384 if kind == "fwd" else 8192)
        window = _log(rng, 1, T) if rng.random() < 0.8 else T
        batch = rng.choice([1, 1, 2, 3])
        # bounds the scores of the plain form to those of the largest listed case
        while batch * T * h_q * min(T, max(window, 64) * 2) > (8e8 if kind == "fwd" else 4e8):
            T, window = T * 2 // 3, min(window, T * 2 // 3)
        T = max(T, 1)
        q_pos0 = rng.choice([0, 0, rng.randrange(0, 2 * window + 1)])
        c = _window("", kind, T, h_q, h_kv, d_qk, d_v, max(window, 1), _log(rng, 1, 128) - 1,
                    batch, q_pos0)
    else:
        page = rng.choice([16, 32, 64, 128])
        batch = _log(rng, 1, 64) if kind == "decode" else 2 * _log(rng, 1, 32)
        cap = min(16384, int(4e9 / (batch * h_kv * (d_qk + d_v) * 2)))
        max_len = _log(rng, 64, max(cap, 65))
        window = rng.choice([0, 0, _log(rng, 1, max_len)]) if kind == "decode" else 0
        new = rng.choice([1, 1, 2, 4]) if kind == "decode" else _log(rng, 1, 2048) if kind == "append" else 1
        if kind == "append":
            max_len = min(max_len, 2048)
        c = _paged("", kind, batch, h_q, h_kv, d_qk, d_v, page, max_len, 1 + rng.randrange(max_len // 2), new,
                   window, _log(rng, 1, 64) - 1 if window else 0)
    del c["name"]
    return c


def _lens(c):
    """The rows' lengths: spread between min_len and max_len, the first the longest (the same for every seed)."""
    rng = random.Random(7)
    return [c["max_len"]] + [rng.randint(c["min_len"], c["max_len"]) for _ in range(c["batch"] - 1)]


def _news(c):
    """Tokens appended to each row."""
    rng = random.Random(8)
    return [c["new"]] + [rng.randint(1, c["new"]) for _ in range(c["batch"] - 1)]


def _pages(c, n):
    return -(-n // c["page"])


def _scale(c):
    return 1.0 / math.sqrt(c["d_qk"])


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = {"c": c}
    if c["kind"] in ("fwd", "train"):
        Tk = c["q_pos0"] + c["seqlen_q"]
        x["q"] = _randn((c["batch"], c["seqlen_q"], c["h_q"], c["d_qk"]), g)
        x["k"] = _randn((c["batch"], c["h_kv"], Tk, c["d_qk"]), g)
        x["v"] = _randn((c["batch"], c["h_kv"], Tk, c["d_v"]), g)
        if c["kind"] == "train":
            x["d_out"] = _randn((c["batch"], c["seqlen_q"], c["h_q"], c["d_v"]), g)
        return x
    # a pool whose pages are handed out in random order; ref counts the rows that hold a page
    rng = random.Random(seed)
    B, P = c["batch"], c["page"]
    lens = _lens(c)
    if c["kind"] == "append":
        lens = [min(n, c["max_len"]) for n in lens]
    if c["kind"] == "beam":                          # the second half of the rows is empty
        lens[B // 2:] = [0] * (B - B // 2)
    tail = c["new"] if c["kind"] in ("append", "beam") else 0
    cols = _pages(c, c["max_len"] + tail) + 1
    used = sum(_pages(c, n) for n in lens)
    n_pages = used + B * (_pages(c, tail) + 2) if tail else used + max(2, used // 8)
    order = list(range(n_pages))
    rng.shuffle(order)
    table, at = [], 0
    for n in lens:
        k = _pages(c, n)
        table.append(order[at:at + k] + [-1] * (cols - k))
        at += k
    if c["kind"] == "compact":                       # every second row has ended
        for b in range(1, B, 2):
            lens[b], table[b] = 0, [-1] * cols
    ref = [0] * n_pages
    for row in table:
        for p in row:
            if p >= 0:
                ref[p] += 1
    x["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    x["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x["ref"] = torch.tensor(ref, dtype=torch.int32, device="cuda")
    x["k_pages"] = _randn((n_pages, c["h_kv"], P, c["d_qk"]), g)
    x["v_pages"] = _randn((n_pages, c["h_kv"], P, c["d_v"]), g)
    if c["kind"] == "decode":
        x["q"] = _randn((B, c["new"], c["h_q"], c["d_qk"]), g)
    if c["kind"] in ("append", "beam"):
        news = _news(c) if c["kind"] == "append" else [1] * B
        x["n_new"] = torch.tensor(news, dtype=torch.int32, device="cuda")
        x["k_new"] = _randn((B, c["h_kv"], c["new"], c["d_qk"]), g)
        x["v_new"] = _randn((B, c["h_kv"], c["new"], c["d_v"]), g)
    if c["kind"] == "beam":
        half = torch.arange(B // 2, dtype=torch.int32, device="cuda")
        x["src"], x["dst"] = half, half + B // 2
    return x


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------

def _plain_window_parts(x):
    """Blocks of queries, the keys that each block can see (sinks last) and who sees which."""
    c = x["c"]
    B, Tq, q0, Hkv, G = c["batch"], c["seqlen_q"], c["q_pos0"], c["h_kv"], c["h_q"] // c["h_kv"]
    Tk, W = q0 + Tq, min(c["window"], q0 + Tq)
    S = min(Tq, max(64, W))
    n = -(-Tq // S)
    dev = x["q"].device
    t = q0 + torch.arange(n * S, device=dev).view(n, S)
    span = min(W - 1 + S, q0 + n * S)
    u = (q0 + (torch.arange(n, device=dev) + 1) * S - span).unsqueeze(1) + torch.arange(span, device=dev)
    ns = min(c["sink"], Tk)
    sinks = torch.arange(ns, device=dev).expand(n, ns)
    u_all = torch.cat([u, sinks], 1)                                           # [n, span + ns]
    tt, uu = t.unsqueeze(2), u_all.unsqueeze(1)
    near = (uu <= tt) & (uu > tt - W) & (uu >= 0)
    far = (uu <= tt - W)
    is_sink = (torch.arange(span + ns, device=dev) >= span).view(1, 1, -1)
    vis = torch.where(is_sink, far, near)                                      # [n, S, keys]
    at = u_all.clamp(0, Tk - 1)
    q = torch.nn.functional.pad(x["q"].float(), (0, 0, 0, 0, 0, n * S - Tq))
    q = q.view(B, n, S, Hkv, G, -1).permute(0, 3, 1, 4, 2, 5)                  # [B, Hkv, n, G, S, d]
    k = x["k"].float()[:, :, at]                                               # [B, Hkv, n, keys, d]
    v = x["v"].float()[:, :, at]
    s = torch.matmul(q.reshape(B, Hkv, n, G * S, -1), k.transpose(-1, -2)).view(B, Hkv, n, G, S, -1)
    s.mul_(_scale(c)).masked_fill_(~vis.view(1, 1, n, 1, S, -1), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    p.div_(z)
    return q, k, v, p, (m + z.log()).squeeze(-1), at, n, S


def _rows(y, c, n, S):
    """[B, Hkv, n, G, S, d] back to [B, Tq, Hq, d]."""
    B, Hkv, G, d = c["batch"], c["h_kv"], c["h_q"] // c["h_kv"], y.shape[-1]
    return y.permute(0, 2, 4, 1, 3, 5).reshape(B, n * S, Hkv * G, d)[:, :c["seqlen_q"]]


def _plain_window(x, backward):
    c = x["c"]
    B, Hkv, G = c["batch"], c["h_kv"], c["h_q"] // c["h_kv"]
    q, k, v, p, lse, at, n, S = _plain_window_parts(x)
    pf = p.view(B, Hkv, n, G * S, -1)
    o = torch.matmul(pf, v)                                                    # [B, Hkv, n, G*S, d_v]
    out = {"out": _rows(o.view(B, Hkv, n, G, S, -1), c, n, S).to(torch.bfloat16),
           "lse": _rows(lse.unsqueeze(-1), c, n, S).squeeze(-1).contiguous()}
    if not backward:
        return out
    do = torch.nn.functional.pad(x["d_out"].float(), (0, 0, 0, 0, 0, n * S - c["seqlen_q"]))
    do = do.view(B, n, S, Hkv, G, -1).permute(0, 3, 1, 4, 2, 5).reshape(B, Hkv, n, G * S, -1)
    dv = torch.matmul(pf.transpose(-1, -2), do)                                # [B, Hkv, n, keys, d_v]
    delta = (do * o).sum(-1, keepdim=True)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_(delta).mul_(pf).mul_(_scale(c))
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q.reshape(B, Hkv, n, G * S, -1))
    i = at.reshape(-1)
    gk = torch.zeros(x["k"].shape, dtype=torch.float32, device=i.device).index_add_(2, i, dk.flatten(2, 3))
    gv = torch.zeros(x["v"].shape, dtype=torch.float32, device=i.device).index_add_(2, i, dv.flatten(2, 3))
    out["dq"] = _rows(dq.view(B, Hkv, n, G, S, -1), c, n, S).to(torch.bfloat16)
    out["dk"], out["dv"] = gk.to(torch.bfloat16), gv.to(torch.bfloat16)
    return out


def _plain_decode(x):
    c = x["c"]
    B, Tq, Hkv, G = c["batch"], c["new"], c["h_kv"], c["h_q"] // c["h_kv"]
    cols = _pages(c, c["max_len"])
    pages = x["table"][:, :cols].clamp(min=0).long()
    k = x["k_pages"][pages].transpose(1, 2).reshape(B, Hkv, -1, c["d_qk"])     # [B, Hkv, L, d]
    v = x["v_pages"][pages].transpose(1, 2).reshape(B, Hkv, -1, c["d_v"])
    t = (x["lens"].long() - Tq).unsqueeze(1) + torch.arange(Tq, device=k.device)
    tt, u = t.unsqueeze(2), torch.arange(k.shape[2], device=k.device).view(1, 1, -1)
    W = c["window"] if c["window"] else k.shape[2]
    vis = (u <= tt) & ((u > tt - W) | (u < c["sink"]))                         # [B, Tq, L]
    q = x["q"].float().view(B, Tq, Hkv, G, -1).permute(0, 2, 1, 3, 4)          # [B, Hkv, Tq, G, d]
    s = torch.matmul(q.reshape(B, Hkv, Tq * G, -1), k.float().transpose(-1, -2)).mul_(_scale(c))
    s = s.view(B, Hkv, Tq, G, -1).masked_fill_(~vis.view(B, 1, Tq, 1, -1), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = (s - m.clamp(min=torch.finfo(torch.float32).min)).exp_()
    z = p.sum(-1, keepdim=True)
    p = p / z.clamp(min=torch.finfo(torch.float32).tiny)
    v = v.float().masked_fill_(~vis.any(1).view(B, 1, -1, 1), 0.0)
    o = torch.matmul(p.view(B, Hkv, Tq * G, -1), v).view(B, Hkv, Tq, G, -1)
    lse = (m + z.log()).squeeze(-1)
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(B, Tq, Hkv * G, -1).to(torch.bfloat16),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, Tq, Hkv * G)}


def _plain_append(c, k_pages, v_pages, table, lens, ref, k_new, v_new, n_new):
    """Pages for the new tokens (a shared last page is copied), their rows written; in place."""
    P, B = c["page"], c["batch"]
    L, n = lens.long(), n_new.long()
    first, last = (L + P - 1) // P, (L + n + P - 1) // P
    partial = (L % P != 0) & (n > 0)
    tail = table.gather(1, (L // P).clamp(max=table.shape[1] - 1).unsqueeze(1)).squeeze(1).clamp(min=0).long()
    same = (tail.unsqueeze(0) == tail.unsqueeze(1)) & partial.unsqueeze(0) & partial.unsqueeze(1)
    earlier = torch.tril(same, -1).sum(1)
    copy = partial & (ref[tail].long() - earlier > 1)
    want = last - first + copy
    start = want.cumsum(0) - want
    free = torch.argsort((ref > 0).to(torch.int8), stable=True)                # free pages, lowest first
    col = torch.arange(table.shape[1], device=table.device).unsqueeze(0)
    begin = torch.where(copy, L // P, first)
    fresh = (col >= begin.unsqueeze(1)) & (col < last.unsqueeze(1))
    at = (start.unsqueeze(1) + col - begin.unsqueeze(1)).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[at].to(torch.int32), table))
    ref.index_add_(0, tail, -copy.to(torch.int32))
    ref.index_add_(0, table.clamp(min=0).long().flatten(), fresh.to(torch.int32).flatten())
    now = table.gather(1, (L // P).clamp(max=table.shape[1] - 1).unsqueeze(1)).squeeze(1).clamp(min=0).long()
    src, dst = torch.where(copy, tail, now), now                               # a row that copies nothing rewrites its own page
    keep = (torch.arange(P, device=L.device) < (L % P).unsqueeze(1)) & copy.unsqueeze(1)
    for_k, for_v = k_pages[src], v_pages[src]
    k_pages[dst] = torch.where(keep.view(B, 1, P, 1), for_k, k_pages[dst])
    v_pages[dst] = torch.where(keep.view(B, 1, P, 1), for_v, v_pages[dst])
    i = torch.minimum(torch.arange(k_new.shape[2], device=L.device).unsqueeze(0), (n - 1).unsqueeze(1))
    pos = L.unsqueeze(1) + i                                                   # the last token again behind a row's end
    page, row = table.gather(1, pos // P).long(), pos % P
    b = torch.arange(B, device=L.device).unsqueeze(1)
    k_pages[page, :, row] = k_new[b, :, i]
    v_pages[page, :, row] = v_new[b, :, i]
    lens.add_(n_new)


def _plain_beam(x, table, lens, ref):
    c = x["c"]
    src, dst = x["src"].long(), x["dst"].long()
    held = table[src]
    table[dst], lens[dst] = held, lens[src]
    ref.index_add_(0, held.clamp(min=0).long().flatten(), (held >= 0).to(torch.int32).flatten())
    _plain_append(c, x["k_pages"], x["v_pages"], table, lens, ref, x["k_new"], x["v_new"], x["n_new"])
    held = table[src]
    ref.index_add_(0, held.clamp(min=0).long().flatten(), -(held >= 0).to(torch.int32).flatten())
    table[src], lens[src] = -1, 0


def _plain_compact(x, table, ref):
    live = ref > 0
    n_live = live.sum()
    ids = torch.arange(ref.numel(), device=ref.device)
    holes = torch.argsort((live | (ids >= n_live)).to(torch.int8), stable=True)   # holes below n_live first
    moves = live & (ids >= n_live)
    rank = (moves.cumsum(0) - 1).clamp(min=0)
    remap = torch.where(moves, holes[rank], ids)
    # a page that stays is copied onto itself, a free one onto a page that is no target
    src = torch.argsort((~moves).to(torch.int8), stable=True)
    count = int(moves.sum())                                                   # how many pages to index with
    src = src[:count]
    x["k_pages"][remap[src]] = x["k_pages"][src]
    x["v_pages"][remap[src]] = x["v_pages"][src]
    table.copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()].to(torch.int32), table))
    new_ref = torch.zeros_like(ref).index_add_(0, torch.where(live, remap, 0), torch.where(live, ref, 0))
    ref.copy_(new_ref)
    return torch.where(live, remap, -1).to(torch.int32), n_live.to(torch.int32).view(1)


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def _run_plain(x):
    kind = x["c"]["kind"]
    if kind in ("fwd", "train"):
        return _plain_window(x, kind == "train")
    if kind == "decode":
        return _plain_decode(x)
    table, lens, ref = x["table"].clone(), x["lens"].clone(), x["ref"].clone()
    out = {"k_pages": x["k_pages"], "v_pages": x["v_pages"], "table": table, "lens": lens, "ref": ref}
    if kind == "append":
        _plain_append(x["c"], x["k_pages"], x["v_pages"], table, lens, ref, x["k_new"], x["v_new"], x["n_new"])
    elif kind == "beam":
        _plain_beam(x, table, lens, ref)
    else:
        out["remap"], out["n_live"] = _plain_compact(x, table, ref)
    return out


def _run_own(x):
    from dynamic_block_sparse_scoring_b200 import abi
    c = x["c"]
    if c["kind"] in ("fwd", "train"):
        cfg = abi.window_config(batch=c["batch"], seqlen_q=c["seqlen_q"], seqlen_kv=c["q_pos0"] + c["seqlen_q"],
                                q_pos0=c["q_pos0"], h_q=c["h_q"], h_kv=c["h_kv"], d_qk=c["d_qk"], d_v=c["d_v"],
                                window=c["window"], sink=c["sink"], scale=_scale(c))
        out, lse = abi.window_forward(cfg, x["q"], x["k"], x["v"])
        if c["kind"] == "fwd":
            return {"out": out, "lse": lse}
        dq, dk, dv = abi.window_backward(cfg, x["q"], x["k"], x["v"], out, lse, x["d_out"])
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    cfg = abi.paged_config(batch=c["batch"], seqlen_q=c["new"], h_q=c["h_q"], h_kv=c["h_kv"], d_qk=c["d_qk"],
                           d_v=c["d_v"], page_size=c["page"], n_pages=x["k_pages"].shape[0],
                           max_pages=x["table"].shape[1], window=c["window"], sink=c["sink"], scale=_scale(c))
    if c["kind"] == "decode":
        out, lse = abi.paged_attention(cfg, x["q"], x["k_pages"], x["v_pages"], x["table"], x["lens"])
        return {"out": out, "lse": lse}
    table, lens, ref = x["table"].clone(), x["lens"].clone(), x["ref"].clone()
    out = {"k_pages": x["k_pages"], "v_pages": x["v_pages"], "table": table, "lens": lens, "ref": ref}
    if c["kind"] == "beam":
        abi.pages_fork(cfg, x["src"], x["dst"], table, lens, ref)
    if c["kind"] in ("append", "beam"):
        abi.paged_append(cfg, x["k_new"], x["v_new"], x["k_pages"], x["v_pages"], table, lens, ref, x["n_new"])
    if c["kind"] == "beam":
        abi.pages_free(cfg, x["src"], table, lens, ref)
    if c["kind"] == "compact":
        out["remap"], out["n_live"] = abi.pages_compact(cfg, x["k_pages"], x["v_pages"], table, lens, ref)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    """Row blocks one after another from the definitions; the pages' cases move whole values only (None)."""
    x = prepare(case, seed)
    c = case
    if c["kind"] not in ("fwd", "train", "decode"):
        return None
    Hkv, G, scale = c["h_kv"], c["h_q"] // c["h_kv"], _scale(c)

    def attend(q, k, v, t, u, W, ns, do=None):
        # q [rows, d] at positions t [rows]; keys k, v at positions u
        s = (q @ k.T) * scale
        vis = (u[None] <= t[:, None]) & ((u[None] > t[:, None] - W) | (u[None] < ns))
        s = torch.where(vis, s, torch.full_like(s, -math.inf))
        lse = torch.logsumexp(s, 1)
        p = torch.where(vis, torch.exp(s - lse[:, None]), torch.zeros_like(s))
        o = p @ torch.where(vis.any(0)[:, None], v, torch.zeros_like(v))
        if do is None:
            return o, lse, None
        ds = p * (do @ v.T - (do * o).sum(1, keepdim=True)) * scale
        return o, lse, (ds @ k, ds.T @ q, p.T @ do)

    if c["kind"] == "decode":
        B, Tq = c["batch"], c["new"]
        lens = x["lens"].tolist()
        W = c["window"] if c["window"] else 1 << 40
        out = torch.zeros(B, Tq, c["h_q"], c["d_v"], dtype=torch.float64, device="cuda")
        lse = torch.full((B, Tq, c["h_q"]), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(B):
            n = lens[b]
            if n == 0:
                continue
            pages = x["table"][b, :_pages(c, n)].long()
            t = torch.arange(n - Tq, n, device="cuda").repeat_interleave(G)
            u = torch.arange(n, device="cuda")
            for h in range(Hkv):
                k = x["k_pages"][pages, h].reshape(-1, c["d_qk"])[:n].double()
                v = x["v_pages"][pages, h].reshape(-1, c["d_v"])[:n].double()
                q = x["q"][b, :, h * G:(h + 1) * G].reshape(Tq * G, -1).double()
                o, e, _ = attend(q, k, v, t, u, W, c["sink"])
                out[b, :, h * G:(h + 1) * G] = o.view(Tq, G, -1)
                lse[b, :, h * G:(h + 1) * G] = e.view(Tq, G)
        return {"out": out, "lse": lse}

    train = c["kind"] == "train"
    B, Tq, q0 = c["batch"], c["seqlen_q"], c["q_pos0"]
    Tk = q0 + Tq
    ns, W = min(c["sink"], Tk), c["window"]
    out = torch.empty(B, Tq, c["h_q"], c["d_v"], dtype=torch.float64, device="cuda")
    lse = torch.empty(B, Tq, c["h_q"], dtype=torch.float64, device="cuda")
    dq = torch.zeros(x["q"].shape, dtype=torch.float64, device="cuda")
    dk = torch.zeros(x["k"].shape, dtype=torch.float64, device="cuda")
    dv = torch.zeros(x["v"].shape, dtype=torch.float64, device="cuda")
    step = max(16, min(512, 8192 // G))
    for b in range(B):
        for h in range(Hkv):
            k, v = x["k"][b, h].double(), x["v"][b, h].double()
            hs = slice(h * G, (h + 1) * G)
            for i0 in range(0, Tq, step):
                i1 = min(i0 + step, Tq)
                lo = max(0, q0 + i0 - W + 1)
                u = torch.arange(lo, q0 + i1, device="cuda")
                if ns and lo:
                    u = torch.cat([torch.arange(min(ns, lo), device="cuda"), u])
                t = torch.arange(q0 + i0, q0 + i1, device="cuda").repeat_interleave(G)
                q = x["q"][b, i0:i1, hs].reshape((i1 - i0) * G, -1).double()
                do = x["d_out"][b, i0:i1, hs].reshape((i1 - i0) * G, -1).double() if train else None
                o, e, grads = attend(q, k[u], v[u], t, u, W, ns, do)
                out[b, i0:i1, hs], lse[b, i0:i1, hs] = o.view(i1 - i0, G, -1), e.view(i1 - i0, G)
                if train:
                    dq[b, i0:i1, hs] = grads[0].view(i1 - i0, G, -1)
                    dk[b, h].index_add_(0, u, grads[1])
                    dv[b, h].index_add_(0, u, grads[2])
    if not train:
        return {"out": out, "lse": lse}
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# ---------------------------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------------------------

def _visible(t, W, ns):
    """Keys that the query at position t sees."""
    lo = max(0, t - W + 1)
    return t + 1 - lo + min(ns, lo)


def work(case):
    c = case
    B, row = c["batch"], (c["d_qk"] + c["d_v"]) * 2
    if c["kind"] in ("fwd", "train"):
        Tq, Tk = c["seqlen_q"], c["q_pos0"] + c["seqlen_q"]
        pairs = B * c["h_q"] * sum(_visible(t, c["window"], c["sink"]) for t in range(c["q_pos0"], Tk))
        q_side, k_side = B * Tq * c["h_q"] * row, B * c["h_kv"] * Tk * row
        nbytes = q_side + k_side + 4 * B * Tq * c["h_q"]
        flops = 2 * (c["d_qk"] + c["d_v"]) * pairs
        if c["kind"] == "train":
            nbytes += q_side + k_side                                          # d_out, dq; dk, dv
            flops += 2 * (3 * c["d_qk"] + 2 * c["d_v"]) * pairs
        return {"bytes": nbytes, "flops": flops}
    lens = _lens(c)
    if c["kind"] == "decode":
        W, Tq = c["window"] or 1 << 40, c["new"]
        keys = sum(n - max(0, n - Tq - W + 1) + min(c["sink"], max(0, n - Tq - W + 1)) for n in lens)
        pairs = c["h_q"] * sum(_visible(n - Tq + i, W, c["sink"]) for n in lens for i in range(Tq) if n - Tq + i >= 0)
        return {"bytes": keys * c["h_kv"] * row + B * Tq * c["h_q"] * (row + 4),
                "flops": 2 * (c["d_qk"] + c["d_v"]) * pairs}
    page = c["h_kv"] * c["page"] * row
    ints = 4 * sum(_pages(c, n) for n in lens)
    if c["kind"] == "append":
        return {"bytes": 2 * sum(_news(c)) * c["h_kv"] * row + 2 * ints, "flops": 0}
    if c["kind"] == "beam":
        half = lens[:B // 2]
        copied = sum(n % c["page"] for n in half)                              # rows of shared last pages
        return {"bytes": 2 * (copied + B) * c["h_kv"] * row + 2 * ints, "flops": 0}
    live = sum(_pages(c, n) for n in lens[::2])
    used = sum(_pages(c, n) for n in lens)
    n_pages = used + max(2, used // 8)
    # a live page's id is anywhere in the pool: so many of them lie above the live count
    return {"bytes": 2 * page * (live * (n_pages - live) // n_pages) + 2 * ints, "flops": 0}
