"""Work for the operators around a paged 8-bit key/value cache that forks share: what one pass of each has to do, in plain
torch operations and through the library.

Operators:
  shared   attention of requests that are forks of a few sessions: the blocks that a group of requests shares are attended
           to once for all of its tokens, the rest of each request's keys by itself, and the two are joined
  rope     the rows of a q/k/v product -> per-head RMS norm of q and k (where weights are given), rotary positions of q and
           k, and q, k, v as contiguous arrays
  fork     a batch of forks and releases of slots: block tables, page counts, freed pages, open blocks
  compact  the pages in use moved to the lowest indices, the block tables and the free stack rewritten, for a pool that
           may then be cut
"""
import math

import numpy as np
import torch

own = False

B = 64                       # tokens per block
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------

def _shared(name, groups, reqs, prefix, extra, new, heads, d, dtype, seed):
    return {"name": name, "op": "shared", "groups": groups, "req_lo": reqs[0], "req_hi": reqs[1], "prefix_lo": prefix[0],
            "prefix_hi": prefix[1], "extra_lo": extra[0], "extra_hi": extra[1], "new_lo": new[0], "new_hi": new[1],
            "q_heads": heads[0], "kv_heads": heads[1], "d": d, "dtype": dtype, "lens_seed": seed}


def _rope(name, requests, new, ctx, heads, d, dtype, rotary, layout, norm, scaling, factor, base, seed):
    return {"name": name, "op": "rope", "n": requests, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "q_heads": heads[0], "kv_heads": heads[1], "d": d, "dtype": dtype, "rotary": rotary, "layout": layout,
            "norm": norm, "scaling": scaling, "factor": factor, "base": base, "original": 8192, "lens_seed": seed}


def _fork(name, sources, forks, ctx, heads, d, dtype, seed):
    return {"name": name, "op": "fork", "sources": sources, "n": forks, "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "q_heads": heads[0], "kv_heads": heads[1], "d": d, "dtype": dtype, "lens_seed": seed}


def _compact(name, pages, used, slots, after, heads, d, seed):
    return {"name": name, "op": "compact", "pages": pages, "used": used, "slots": slots, "after": after,
            "q_heads": heads[0], "kv_heads": heads[1], "d": d, "dtype": "bf16", "lens_seed": seed}


def listed():
    return [
        # one token for each of 8 forks of a short session: the latency of a step
        _shared("forks_8_tokens", 1, (8, 8), (4096, 4096), (0, 300), (1, 1), (16, 4), 128, "bf16", 1),
        # a decode step of 64 forks of one 41,802-token conversation, each some tokens past the fork
        _shared("forks_64_tokens", 1, (64, 64), (41802, 41802), (0, 500), (1, 1), (16, 2), 256, "bf16", 2),
        # a decode step of several conversations, each with 1 to 16 branches
        _shared("families_12_tokens", 12, (1, 16), (500, 16384), (0, 1500), (1, 1), (32, 8), 128, "bf16", 3),
        # 16 branches of 20 to 200 tokens that continue a 12,000-token prefix
        _shared("branches_16_prompts", 1, (16, 16), (12000, 12000), (0, 0), (20, 200), (16, 4), 128, "bf16", 4),
        # the largest: 8 long continuations of one long conversation
        _shared("branches_8_turns", 1, (8, 8), (37802, 37802), (0, 0), (1000, 1000), (16, 4), 128, "bf16", 5),
        # branches of the small fp32 layer
        _shared("branches_fp32", 2, (3, 5), (900, 2048), (0, 100), (1, 40), (2, 2), 64, "fp32", 6),
        # the token of one conversation, a quarter of the head rotated, with the norm of q and k
        _rope("rope_token", 1, (1, 1), (41802, 41802), (16, 2), 256, "bf16", 64, "half", True, "none", 1.0, 1e7, 7),
        # a batch of long prompts, whole heads in interleaved pairs, positions stretched for a long context
        _rope("rope_prompts", 8, (4000, 8000), (0, 100000), (32, 8), 128, "bf16", 128, "interleaved", False, "parts", 8.0, 1e4, 8),
        # 16 branches of one session, forked at once
        _fork("fork_16", 1, 16, (12000, 12000), (16, 4), 128, "bf16", 9),
        # 256 slots handed to forks of 12 sessions, or emptied; most held something before
        _fork("fork_256", 12, 256, (500, 41802), (16, 2), 256, "bf16", 10),
        # a small pool
        _compact("compact_small", 300, 0.5, 8, 1.0, (16, 2), 256, 11),
        # a pool of 2.6 GB, cut to three quarters
        _compact("compact_large", 20000, 0.6, 128, 0.75, (32, 8), 128, 12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared"] * 5 + ["rope"] * 3 + ["fork"] * 2 + ["compact"] * 2)
    kv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    while kv * g > 64:
        g = rng.choice([1, 2, 4, 8])
    base = {"op": op, "q_heads": kv * g, "kv_heads": kv, "d": rng.choice([64, 128, 256]),
            "dtype": "fp32" if rng.random() < 0.2 else "bf16", "lens_seed": rng.randrange(1 << 30)}
    c = dict(base)
    if op == "rope":
        single = rng.random() < 0.4
        c["n"] = _log_int(rng, 1, 256) if single else _log_int(rng, 1, 12)
        new = 1 if single else _log_int(rng, 2, 8000)
        c["new_lo"], c["new_hi"] = (1 if rng.random() < 0.5 else new), new
        c["ctx_lo"], c["ctx_hi"] = 0, _log_int(rng, 64, 1000000)
        c["rotary"] = 16 * rng.randint(1, c["d"] // 16) if rng.random() < 0.5 else c["d"]
        c["layout"] = rng.choice(["half", "interleaved"])
        c["norm"] = rng.random() < 0.5
        c["scaling"] = rng.choice(["none", "linear", "parts"])
        c["factor"] = 1.0 if c["scaling"] == "none" else float(rng.choice([2, 3, 4, 8, 16, 40]))
        c["base"] = float(rng.choice([10000, 150000, 500000, 1000000, 10000000]))
        c["original"] = rng.choice([2048, 4096, 8192, 32768])
        while work(c)["bytes"] > work(listed()[7])["bytes"]:
            c["n"] = max(1, c["n"] * 3 // 4)
            c["new_hi"] = max(1, c["new_hi"] * 3 // 4)
            c["new_lo"] = min(c["new_lo"], c["new_hi"])
        return c
    if op == "fork":
        c["n"], c["sources"] = _log_int(rng, 1, 256), _log_int(rng, 1, 16)
        c["ctx_lo"], c["ctx_hi"] = 0, _log_int(rng, 64, 41802)
        return c
    if op == "compact":
        c["dtype"] = "bf16"
        c["pages"] = min(_log_int(rng, 4, 40000), int(2.6e9 / (2 * kv * B * c["d"])))
        c["used"] = rng.uniform(0.05, 1.0)
        c["slots"] = _log_int(rng, 1, 256)
        c["after"] = 1.0 if rng.random() < 0.5 else rng.uniform(c["used"], 1.0)
        return c
    single = rng.random() < 0.5
    c["groups"] = 1 if rng.random() < 0.5 else _log_int(rng, 2, 24)
    top = _log_int(rng, 1, 64 if c["groups"] == 1 else 16)
    c["req_lo"], c["req_hi"] = (1 if rng.random() < 0.5 else top), top
    new = 1 if single else _log_int(rng, 2, 1500)
    c["new_lo"], c["new_hi"] = (1 if rng.random() < 0.5 else new), new
    top = _log_int(rng, 64, 41802)
    c["prefix_lo"], c["prefix_hi"] = (top if rng.random() < 0.5 else 0), top
    c["extra_lo"], c["extra_hi"] = 0, 0 if rng.random() < 0.3 else _log_int(rng, 1, 2000)
    cap = 0.9 * work(listed()[4])["flops"] * (0.05 if c["dtype"] == "fp32" else 1.0)
    while True:   # within the largest listed case, and what the plain form's arrays take
        w = work(c)
        most = c["groups"] * c["req_hi"]
        rows, suffix = most * c["new_hi"], c["extra_hi"] + 2 * c["new_hi"] + 192
        scores = max(c["req_hi"] * c["new_hi"] * g * c["prefix_hi"] * 4.0, rows * c["q_heads"] * suffix * 4.0)
        keys = max(c["prefix_hi"], most * suffix) * c["kv_heads"] * c["d"] * 8.0
        if w["flops"] <= cap and w["bytes"] <= 2.0e9 and scores <= 8e9 and keys <= 1.2e10:
            return c
        if c["new_hi"] > 1:
            c["new_hi"] = max(1, c["new_hi"] * 3 // 4)
            c["new_lo"] = min(c["new_lo"], c["new_hi"])
        elif c["groups"] > 1:
            c["groups"] = max(1, c["groups"] * 3 // 4)
        elif c["req_hi"] > 1:
            c["req_hi"] = max(1, c["req_hi"] * 3 // 4)
            c["req_lo"] = min(c["req_lo"], c["req_hi"])
        else:
            c["prefix_hi"] = c["prefix_hi"] * 3 // 4
            c["prefix_lo"] = min(c["prefix_lo"], c["prefix_hi"])


def _spread(rs, n, lo, hi):
    """n whole numbers of [lo, hi], over their logarithm."""
    if lo == hi:
        return np.full(n, lo, dtype=np.int64)
    x = np.exp(rs.uniform(math.log(lo + 1), math.log(hi + 1), n)) - 1
    return np.clip(np.rint(x).astype(np.int64), lo, hi)


def _lens(case):
    """The lengths of a case, a function of it alone."""
    rs = np.random.RandomState(case["lens_seed"] % (1 << 31))
    if case["op"] == "shared":
        reqs = _spread(rs, case["groups"], case["req_lo"], case["req_hi"])
        prefix = _spread(rs, case["groups"], case["prefix_lo"], case["prefix_hi"])
        n = int(reqs.sum())
        extra = _spread(rs, n, case["extra_lo"], case["extra_hi"])
        new = _spread(rs, n, case["new_lo"], case["new_hi"])
        group = np.repeat(np.arange(case["groups"]), reqs)
        ctx = prefix[group] + extra
        held = prefix // B                                   # blocks that a group's forks were handed
        first = ctx // B                                     # block of a request's first new token
        # shared blocks: up to the first block of a request's own, or that a request's first new token lies in
        start = np.array([first[group == i].min() if (group == i).sum() == 1 else min(held[i], first[group == i].min())
                          for i in range(case["groups"])])
        return {"reqs": reqs, "group": group, "ctx": ctx, "new": new, "held": held, "start": start}
    if case["op"] == "rope":
        return {"ctx": _spread(rs, case["n"], case["ctx_lo"], case["ctx_hi"]),
                "new": _spread(rs, case["n"], case["new_lo"], case["new_hi"])}
    if case["op"] == "fork":
        ctx = _spread(rs, case["sources"], case["ctx_lo"], case["ctx_hi"])
        n, k = case["n"], case["sources"]
        src = rs.randint(0, k, n)
        src[rs.uniform(size=n) < (0.1 if k > 1 else 0.0)] = -1               # a release
        had = rs.randint(0, k, n)                                            # what the slot was forked from before
        had_own = _spread(rs, n, 0, 300)                                     # and its tokens since
        had_len = np.where(rs.uniform(size=n) < 0.8, ctx[had] // B * B + had_own, 0)
        return {"ctx": ctx, "src": src, "had": had, "had_len": had_len}
    n = case["pages"]
    used = min(n, max(1, int(round(case["used"] * n))))
    after = min(n, max(used, int(round(case["after"] * n))))
    cuts = np.sort(rs.randint(0, used + 1, case["slots"] - 1)) if case["slots"] > 1 else np.zeros(0, dtype=np.int64)
    return {"used": used, "after": after, "edges": np.concatenate([[0], cuts, [used]])}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def _to(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = {"case": case, "op": case["op"], "shape": (case["q_heads"], case["kv_heads"], case["d"]), "lens": _lens(case)}
    {"shared": _prepare_shared, "rope": _prepare_rope, "fork": _prepare_fork, "compact": _prepare_compact}[case["op"]](st, rs, gen)
    return st


def _values(gen, dt, *size):   # activations, with heads of unequal size
    x = torch.randn(size, generator=gen, device=DEV)
    return (x * (0.5 + torch.rand((size[-2], 1), generator=gen, device=DEV))).to(dt)


def _prepare_shared(st, rs, gen):
    case, L = st["case"], st["lens"]
    hq, hkv, d = st["shape"]
    dt = DT[case["dtype"]]
    ctx, new, group, held = L["ctx"], L["new"], L["group"], L["held"]
    n, end = len(ctx), L["ctx"] + L["new"]
    n_slots, max_blocks = n + 3, int(end.max()) // B + 2
    own_blocks = end // B - np.minimum(held[group], end // B)
    n_pages = int(held.sum() + own_blocks.sum()) + 5
    pages = rs.permutation(n_pages).astype(np.int32)
    slots = rs.permutation(n_slots)[:n].astype(np.int32)
    buf = rs.randint(0, 2, n).astype(np.int32)
    state = np.zeros((n_slots, 2), dtype=np.int32)
    table = np.full((n_slots, max_blocks), -1, dtype=np.int32)
    shared_at = np.concatenate([[0], np.cumsum(held)])
    at = int(shared_at[-1])
    rows = np.concatenate([[0], np.cumsum(new)])
    units = []
    for i in range(n):
        h, b1 = int(held[group[i]]), int(end[i]) // B
        p0 = int(shared_at[group[i]])
        table[slots[i], :h] = pages[p0:p0 + h]
        table[slots[i], h:b1] = pages[at:at + b1 - h]
        at += max(b1 - h, 0)
        b0 = int(ctx[i]) // B
        block = np.arange(b0, (int(end[i]) + B - 1) // B)
        lo, hi = np.maximum(ctx[i], block * B), np.minimum(end[i], block * B + B)
        closes = hi == block * B + B
        to = buf[i] ^ int(b1 != b0)
        u = np.stack([np.full_like(block, slots[i]), block, np.where(closes, table[slots[i], np.minimum(block, max_blocks - 1)], -1),
                      lo - block * B, hi - lo, rows[i] + lo - ctx[i], np.full_like(block, buf[i]), np.where(closes, -1, to)], 1)
        units.append(u)
        state[slots[i]] = int(end[i]), to
    units = np.concatenate(units).astype(np.int32)
    total = int(rows[-1])
    bounds = np.concatenate([[0], np.cumsum(L["reqs"])])
    st.update(n=n, total=total, n_units=len(units), n_pages=n_pages, n_slots=n_slots, max_blocks=max_blocks,
              max_new=int(new.max()), max_len=int(end.max()), max_suffix=int((end - B * L["start"][group]).max()),
              scale=1.0 / math.sqrt(d), slots=_to(slots), buf=_to(buf), ctx=_to(ctx), new_dev=_to(new),
              state=_to(state), table=_to(table), rows=_to(rows.astype(np.int32)), units=_to(units),
              counts=_to(np.array([len(units), 0], dtype=np.int32)), bounds=_to(bounds.astype(np.int32)),
              groups=torch.zeros((len(held), 4), dtype=torch.int32, device=DEV),
              starts=torch.zeros(len(units), dtype=torch.int32, device=DEV))
    shape = (n_pages, hkv, B, d)
    # a block's largest of 64 d normal values is near 4: 8-bit steps of about 4 / 127
    for name in ("k", "v"):
        st[name] = (torch.randn(shape, generator=gen, device=DEV) * 32).round_().clamp_(-127, 127).to(torch.int8)
        st[name + "_scale"] = 0.02 + 0.03 * torch.rand(shape[:2], generator=gen, device=DEV)
    # queries of heads that look at few keys and of heads that look at many
    temp = 0.5 + 2.5 * torch.rand((hq, 1), generator=gen, device=DEV)
    st["q"] = (torch.randn((total, hq, d), generator=gen, device=DEV) * temp).to(dt)
    st["out"] = torch.zeros((total, hq, d), dtype=dt, device=DEV)
    st["k_new"], st["v_new"] = _values(gen, dt, total, hkv, d), _values(gen, dt, total, hkv, d)
    # the open blocks as they came: [slot][buffer][key / value][head][offset][d]
    st["tail"] = torch.randn((n_slots, 2, 2, hkv, B, d), generator=gen, device=DEV).to(dt)


def _prepare_rope(st, rs, gen):
    case, L = st["case"], st["lens"]
    hq, hkv, d = st["shape"]
    dt = DT[case["dtype"]]
    order = rs.permutation(len(L["ctx"]))
    pos = np.concatenate([L["ctx"][i] + np.arange(L["new"][i]) for i in order]).astype(np.int32)
    n = len(pos)
    # the rows of a product of the hidden states with the q, k and v weights
    st["qkv"] = _values(gen, dt, n, hq + 2 * hkv, d).view(n, -1)
    st["positions"] = _to(pos)
    for name in ("q_weight", "k_weight"):
        w = (1 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(dt)
        st[name] = w if case["norm"] else None
    for name, h in (("q_out", hq), ("k_out", hkv), ("v_out", hkv)):
        st[name] = torch.zeros((n, h, d), dtype=dt, device=DEV)
    f = case["factor"]
    st["eps"] = float(np.float32(1e-6))
    st["magnitude"] = float(np.float32(0.1 * math.log(f) + 1)) if case["scaling"] == "parts" else 1.0


def _prepare_fork(st, rs, gen):
    case, L = st["case"], st["lens"]
    hq, hkv, d = st["shape"]
    n, k = case["n"], case["sources"]
    n_slots = n + k + 2
    max_blocks = int(max(L["ctx"].max(), L["had_len"].max())) // B + 1
    had_blocks = L["had_len"] // B
    from_src = np.minimum(had_blocks, L["ctx"][L["had"]] // B)
    src_blocks = L["ctx"] // B
    n_pages = int(src_blocks.sum() + (had_blocks - from_src).sum()) + 7
    pages = rs.permutation(n_pages).astype(np.int32)
    where = rs.permutation(n_slots).astype(np.int32)
    src_slot, dst_slot = where[:k], where[k:k + n]
    table = np.full((n_slots, max_blocks), -1, dtype=np.int32)
    state = np.zeros((n_slots, 2), dtype=np.int32)
    refs = np.zeros(n_pages + 1, dtype=np.int32)
    at = 0
    for i in range(k):
        m = int(src_blocks[i])
        table[src_slot[i], :m] = pages[at:at + m]
        state[src_slot[i]] = int(L["ctx"][i]), rs.randint(0, 2)
        at += m
    for i in range(n):
        m, o = int(from_src[i]), int(had_blocks[i] - from_src[i])
        table[dst_slot[i], :m] = table[src_slot[L["had"][i]], :m]
        table[dst_slot[i], m:m + o] = pages[at:at + o]
        state[dst_slot[i]] = int(L["had_len"][i]), rs.randint(0, 2)
        at += o
    for s in range(n_slots):
        np.add.at(refs, table[s, :state[s, 0] // B], 1)
    free = np.zeros(n_pages + 1, dtype=np.int32)             # one more than the cache has: see _fork_plain
    free[:n_pages - at] = pages[at:]
    src = np.where(L["src"] >= 0, src_slot[np.maximum(L["src"], 0)], -1).astype(np.int32)
    st.update(n=n, n_slots=n_slots, n_pages=n_pages, max_blocks=max_blocks, table=_to(table), state=_to(state),
              refs_full=_to(refs), free_full=_to(free), n_free=_to(np.array([n_pages - at], dtype=np.int32)),
              src=_to(src), dst=_to(dst_slot),
              tail=torch.randn((n_slots, 2, 2, hkv, B, d), generator=gen, device=DEV).to(DT[case["dtype"]]))


def _prepare_compact(st, rs, gen):
    case, L = st["case"], st["lens"]
    hq, hkv, d = st["shape"]
    n, used = case["pages"], L["used"]
    pages = rs.permutation(n).astype(np.int32)
    # the slots hold runs of the pages in use, the first page of each slot shared with the slot before
    n_slots = case["slots"]
    edges = L["edges"]
    max_blocks = int(np.diff(edges).max()) + 2
    table = np.full((n_slots, max_blocks), -1, dtype=np.int32)
    state = np.zeros((n_slots, 2), dtype=np.int32)
    refs = np.zeros(n, dtype=np.int32)
    for s in range(n_slots):
        own_pages = pages[edges[s]:edges[s + 1]]
        if s and len(own_pages) and edges[s] > 0:
            own_pages = np.concatenate([pages[edges[s] - 1:edges[s]], own_pages])
        table[s, :len(own_pages)] = own_pages
        state[s] = len(own_pages) * B + rs.randint(0, B), rs.randint(0, 2)
        np.add.at(refs, own_pages, 1)
    free = np.zeros(n, dtype=np.int32)
    free[:n - used] = pages[used:]
    moves = int((refs[used:] > 0).sum())
    shape = (n, hkv, B, d)
    after = L["after"]
    st.update(n_pages=n, n_slots=n_slots, max_blocks=max_blocks, moves=moves, used=used, after=after, table=_to(table),
              state=_to(state), refs=_to(refs), free=_to(free), n_free=_to(np.array([n - used], dtype=np.int32)),
              k=torch.randint(-127, 128, shape, generator=gen, device=DEV, dtype=torch.int8),
              v=torch.randint(-127, 128, shape, generator=gen, device=DEV, dtype=torch.int8),
              k_scale=0.02 + 0.03 * torch.rand(shape[:2], generator=gen, device=DEV),
              v_scale=0.02 + 0.03 * torch.rand(shape[:2], generator=gen, device=DEV),
              # the books after the call, beside those before it
              table_out=torch.full((n_slots, max_blocks), -1, dtype=torch.int32, device=DEV),
              refs_out=torch.zeros(after, dtype=torch.int32, device=DEV),
              free_out=torch.zeros(after, dtype=torch.int32, device=DEV),
              n_free_out=torch.zeros(1, dtype=torch.int32, device=DEV),
              counts=torch.zeros(4, dtype=torch.int32, device=DEV))


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------

def _groups_plain(st):
    """[first row, rows, slot whose table is read, shared blocks] per group of requests; the shared blocks per unit."""
    L, dev = st["lens"], st["slots"].device
    table, rows = st["table"], st["rows"].long()
    reqs = L["reqs"].tolist()
    first = st["ctx"] // B
    at, starts = 0, []
    for i, m in enumerate(reqs):
        s = st["slots"][at:at + m].long()
        same = (table[s] == table[s[:1]]).all(0).int().cumprod(0).sum()
        shared = torch.minimum(same, first[at:at + m].min())
        st["groups"][i] = torch.stack([rows[at], rows[at + m] - rows[at], s[0], shared]).int()
        starts.append(shared.expand(m))
        at += m
    start = torch.cat(starts)
    req = torch.bucketize(st["units"][:, 5].long(), rows[1:], right=True)
    st["starts"].copy_(start[req])
    return start


def _shared_plain(st):
    """softmax(scale q k^T) v over [a group's shared blocks; the request's other complete blocks before the query's own, all
    from 8 bits; the query's own block as it came]."""
    hq, hkv, d = st["shape"]
    g, n, dev, L = hq // hkv, st["n"], st["q"].device, st["lens"]
    start = _groups_plain(st)
    total, T = st["total"], st["max_new"]
    rows, slots = st["rows"].long(), st["slots"].long()
    q_all = st["q"].float() * st["scale"]
    # the shared blocks, once for all rows of a group
    m1 = torch.full((total, hkv, g), float("-inf"), device=dev)
    l1 = torch.zeros((total, hkv, g), device=dev)
    o1 = torch.zeros((total, hkv, g, d), device=dev)
    r0, at = 0, 0
    for i, m in enumerate(L["reqs"].tolist()):
        r1 = r0 + int(L["new"][at:at + m].sum())
        p = int(L["start"][i])
        if p and r1 > r0:
            page = st["table"][slots[at], :p].long()
            for h in range(hkv):
                k = (st["k"][page, h].float() * st["k_scale"][page, h][:, None, None]).view(p * B, d)
                v = (st["v"][page, h].float() * st["v_scale"][page, h][:, None, None]).view(p * B, d)
                s = q_all[r0:r1, h * g:(h + 1) * g].reshape(-1, d) @ k.t()
                top = s.amax(1, keepdim=True)
                s -= top
                s.exp_()
                m1[r0:r1, h] = top.view(-1, g)
                l1[r0:r1, h] = s.sum(1).view(-1, g)
                o1[r0:r1, h] = (s @ v).view(-1, g, d)
        r0, at = r1, at + m
    # the rest of each request's keys
    new, ctx, buf = st["new_dev"], st["ctx"], st["buf"].long()
    t = torch.arange(T, device=dev)
    pick = (rows[:-1, None] + t).clamp_(max=total - 1)                                  # [n][T]
    q = q_all[pick].view(n, T, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, T * g, d)
    qpos = ctx[:, None] + t
    qblk = qpos // B
    nb = max(1, (st["max_suffix"] - 1) // B)
    blk = start[:, None] + torch.arange(nb, device=dev)                                 # [n][nb]
    pages = st["table"][slots[:, None], blk.clamp(max=st["max_blocks"] - 1)].long().clamp_(min=0)
    k = (st["k"][pages].float() * st["k_scale"][pages][..., None, None]).transpose(1, 2).reshape(n, hkv, nb * B, d)
    v = (st["v"][pages].float() * st["v_scale"][pages][..., None, None]).transpose(1, 2).reshape(n, hkv, nb * B, d)
    see = blk.repeat_interleave(B, 1)[:, None, :] < qblk[..., None]                     # [n][T][nb 64]
    base = ctx // B * B
    R = T + B - 1
    r = torch.arange(R, device=dev)
    kpos = base[:, None] + r                                                            # [n][R]
    in_tail = (kpos < ctx[:, None])[..., None, None]
    fresh = (rows[:-1, None] + kpos - ctx[:, None]).clamp_(0, total - 1)
    tail = st["tail"][slots, buf].permute(1, 0, 3, 2, 4)[:, :, r.clamp(max=B - 1)]      # [2][n][R][hkv][d]
    kr = torch.where(in_tail, tail[0], st["k_new"][fresh]).float().transpose(1, 2)      # [n][hkv][R][d]
    vr = torch.where(in_tail, tail[1], st["v_new"][fresh]).float().transpose(1, 2)
    see_r = (kpos[:, None, :] // B == qblk[..., None]) & (kpos[:, None, :] <= qpos[..., None])
    s = torch.cat([q @ k.transpose(2, 3), q @ kr.transpose(2, 3)], 3)
    mask = torch.cat([see, see_r], 2)[:, None, :, None, :].expand(n, 1, T, g, nb * B + R).reshape(n, 1, T * g, -1)
    s.masked_fill_(~mask, float("-inf"))
    top = s.amax(3, keepdim=True)
    s -= top.clamp(min=-1e30)
    s.exp_()
    o2 = s[..., :nb * B] @ v + s[..., nb * B:] @ vr
    req = torch.repeat_interleave(torch.arange(n, device=dev), new, output_size=total)
    tok = torch.arange(total, device=dev) - rows[req]
    part = lambda x: x.view(n, hkv, T, g, -1)[req, :, tok]   # noqa: E731  [total][hkv][g][...]
    m2, l2, o2 = part(top)[..., 0], part(s.sum(3))[..., 0], part(o2)
    top = torch.maximum(m1, m2)
    f1, f2 = (m1 - top).exp(), (m2 - top).exp()
    o = (o1 * f1[..., None] + o2 * f2[..., None]) / (l1 * f1 + l2 * f2)[..., None]
    st["out"].copy_(o.view(total, hq, d))


def _inv_freq(case):
    """Angle per position of each pair, 64 bits."""
    rd = case["rotary"]
    f = case["base"] ** (-torch.arange(0, rd, 2, dtype=torch.float64, device=DEV) / rd)
    if case["scaling"] == "linear":
        f = f / case["factor"]
    elif case["scaling"] == "parts":   # turns within the trained length: many keep their pace, few are stretched
        turns = case["original"] * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / case["factor"] * (1 - keep)
    return f


def _rope_plain(st):
    case = st["case"]
    hq, hkv, d = st["shape"]
    rd, n = case["rotary"], st["qkv"].shape[0]
    angle = st["positions"].double()[:, None] * _inv_freq(case)
    cos, sin = (angle.cos() * st["magnitude"]).float()[:, None], (angle.sin() * st["magnitude"]).float()[:, None]
    q, k, v = st["qkv"].view(n, hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
    for x, w, out in ((q, st["q_weight"], st["q_out"]), (k, st["k_weight"], st["k_out"])):
        x = x.float()
        if w is not None:
            x = x * (1 / (x.square().mean(2, keepdim=True) + st["eps"]).sqrt()) * w.float()
        y = x.clone()
        if case["layout"] == "half":
            a, b = x[..., :rd // 2], x[..., rd // 2:rd]
            y[..., :rd // 2], y[..., rd // 2:rd] = a * cos - b * sin, a * sin + b * cos
        else:
            a, b = x[..., 0:rd:2], x[..., 1:rd:2]
            y[..., 0:rd:2], y[..., 1:rd:2] = a * cos - b * sin, a * sin + b * cos
        out.copy_(y)
    st["v_out"].copy_(v)


def _fork_plain(st):
    """Pages first gain the forks' names, then lose those that the slots held; pages that no slot names any more are pushed
    on the free stack in the order of their numbers."""
    src, dst, table, state = st["src"].long(), st["dst"].long(), st["table"], st["state"]
    refs, free, P = st["refs_full"], st["free_full"], st["n_pages"]
    fork = src >= 0
    src0 = src.clamp(min=0)
    length = torch.where(fork, state[src0, 0], torch.zeros_like(state[src0, 0]))
    block = torch.arange(st["max_blocks"], device=src.device)
    to = torch.where(block < (length // B)[:, None], table[src0], torch.full_like(table[src0], P)).long()
    old = torch.where(block < (state[dst, 0] // B)[:, None], table[dst], torch.full_like(table[dst], P)).long()
    ones = torch.ones(to.numel(), dtype=torch.int32, device=src.device)
    after = refs.clone()
    after.index_add_(0, to.view(-1), ones)
    after.index_add_(0, old.view(-1), ones, alpha=-1)
    freed = (after[:P] == 0) & (refs[:P] > 0)
    at = st["n_free"].long() + freed.long().cumsum(0) - 1
    free[torch.where(freed, at, torch.full_like(at, P))] = torch.arange(P, dtype=torch.int32, device=src.device)
    st["n_free"] += freed.sum().int()
    refs.copy_(after)
    table[dst] = torch.where(to < P, to.int(), table[dst])
    new_buf = torch.where(fork, state[src0, 1], state[dst, 1])
    # the open rows
    off = torch.arange(B, device=src.device)
    take = (off < (length % B)[:, None])[:, None, None, :, None]
    st["tail"][dst, new_buf.long()] = torch.where(take, st["tail"][src0, new_buf.long()], st["tail"][dst, new_buf.long()])
    state[dst] = torch.stack([length, new_buf], 1)


def _compact_plain(st):
    """The i-th page in use at or past the number of pages in use moves to the i-th free page below it."""
    refs, P, used, m, after = st["refs"], st["n_pages"], st["used"], st["moves"], st["after"]
    dev = refs.device
    page = torch.arange(P, device=dev)
    busy = refs > 0
    count = busy.sum()
    hole, mover = ~busy & (page < count), busy & (page >= count)
    from_ = torch.zeros(P + 1, dtype=torch.long, device=dev)
    to = torch.zeros(P + 1, dtype=torch.long, device=dev)
    to[torch.where(hole, hole.long().cumsum(0) - 1, torch.full_like(page, P))] = page
    from_[torch.where(mover, mover.long().cumsum(0) - 1, torch.full_like(page, P))] = page
    from_, to = from_[:m], to[:m]
    now = page.clone()
    now[from_] = to
    for name in ("k", "v", "k_scale", "v_scale"):
        st[name][to] = st[name][from_]
    block = torch.arange(st["max_blocks"], device=dev)
    valid = block < (st["state"][:, :1] // B)
    st["table_out"].copy_(torch.where(valid, now[st["table"].long().clamp(min=0)].int(), st["table_out"]))
    moved = refs.clone()
    moved[to] = refs[from_]
    moved[from_] = 0
    st["refs_out"].copy_(moved[:after])
    left = after - 1 - torch.arange(after, device=dev, dtype=torch.int32)
    st["free_out"].copy_(torch.where(left >= count, left, st["free_out"]))
    st["n_free_out"].copy_(after - count)
    st["counts"][:3] = torch.stack([count, torch.zeros_like(count), mover.sum()]).int()


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def _handles(st):
    """The library's handles over the program's buffers, made once, as a program makes them."""
    if "handles" not in st:
        from chunked_gated_deltanet_gb300 import gdn
        case, (hq, hkv, d) = st["case"], st["shape"]
        h = {"gdn": gdn, "desc": gdn.make_attn_desc(hq, hkv, d, gdn.GDN_FP32 if case["dtype"] == "fp32" else gdn.GDN_BF16,
                                                    st.get("scale"))}
        cache = lambda **b: gdn.KvCache(h["desc"], st["n_pages"], st["n_slots"], st["max_blocks"], DEV, **b)   # noqa: E731
        if st["op"] == "shared":
            h["cache"] = cache(**{b: st[b] for b in ("k", "v", "k_scale", "v_scale", "tail", "state", "table")})
            h["plan"] = gdn.KvPlan(st["rows"], st["units"], st["counts"])
            h["groups"] = gdn.KvGroups(st["groups"], st["starts"])
            h["ws"] = gdn.kv_shared_workspace(h["desc"], st["total"], st["max_len"], st["max_suffix"], DEV)
        elif st["op"] == "rope":
            layout = gdn.GDN_ROPE_HALF if case["layout"] == "half" else gdn.GDN_ROPE_INTERLEAVED
            scaling = {"none": gdn.GDN_ROPE_NONE, "linear": gdn.GDN_ROPE_LINEAR, "parts": gdn.GDN_ROPE_PARTS}[case["scaling"]]
            h["rope"] = gdn.make_rope_desc(case["rotary"], layout, case["base"], scaling, case["factor"], case["original"],
                                           32.0, 1.0, st["magnitude"], st["eps"])
            h["table"] = gdn.rope_table(h["rope"], DEV)
            n = st["qkv"].shape[0]
            h["qkv"] = st["qkv"].view(n, hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
        elif st["op"] == "fork":
            P = st["n_pages"]
            h["cache"] = cache(tail=st["tail"], state=st["state"], table=st["table"], refs=st["refs_full"][:P],
                               free=st["free_full"][:P], n_free=st["n_free"])
        else:
            h["cache"] = cache(**{b: st[b] for b in ("k", "v", "k_scale", "v_scale", "state", "table", "refs", "free", "n_free")})
            h["ws"] = gdn.kv_compact_workspace(st["n_pages"], DEV)
        st["handles"] = h
    return st["handles"]


def _run_own(st):
    h = _handles(st)
    gdn, desc = h["gdn"], h["desc"]
    if st["op"] == "shared":
        gdn.gdn_kv_group(desc, h["cache"], h["plan"], st["bounds"], h["groups"])
        gdn.gdn_kv_attention_shared(desc, h["cache"], h["plan"], h["groups"], st["q"], st["k_new"], st["v_new"], st["out"],
                                    h["ws"], st["max_new"], st["max_len"], st["max_suffix"])
    elif st["op"] == "rope":
        q, k, v = h["qkv"]
        gdn.gdn_rope(desc, h["rope"], h["table"], st["positions"], q, k, st["q_out"], st["k_out"], v, st["v_out"],
                     st["q_weight"], st["k_weight"])
    elif st["op"] == "fork":
        gdn.gdn_kv_fork_batch(desc, h["cache"], st["src"], st["dst"])
    else:
        gdn.gdn_kv_compact(desc, h["cache"], h["ws"], st["counts"], table_out=st["table_out"], refs_out=st["refs_out"],
                           free_out=st["free_out"], n_free_out=st["n_free_out"])


def run(st):
    if own:
        _run_own(st)
    else:
        {"shared": _shared_plain, "rope": _rope_plain, "fork": _fork_plain, "compact": _compact_plain}[st["op"]](st)
    if st["op"] == "shared":
        return {"out": st["out"], "groups": st["groups"], "starts": st["starts"]}
    if st["op"] == "rope":
        return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"]}
    if st["op"] == "fork":
        return {"table": st["table"], "state": st["state"], "refs": st["refs_full"][:st["n_pages"]],
                "free": st["free_full"][:st["n_pages"]], "n_free": st["n_free"], "tail": st["tail"]}
    return {"k": st["k"], "v": st["v"], "k_scale": st["k_scale"], "v_scale": st["v_scale"], "table": st["table_out"],
            "refs": st["refs_out"], "free": st["free_out"], "n_free": st["n_free_out"], "counts": st["counts"]}


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------

def work(case):
    L = _lens(case)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["d"]
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "shared":
        ctx, new, group = L["ctx"], L["new"], L["group"]
        end, start = ctx + new, L["start"][group]
        pos = lambda m: m * (m + 1) / 2.0   # noqa: E731  keys seen by the queries at positions 0 .. m - 1
        keys = float((pos(end) - pos(ctx)).sum())
        total = float(new.sum())
        held = float(L["start"].sum()) + float(np.maximum((end - 1) // B - start, 0).sum())
        old = float((ctx % B).sum())
        n_units = float(((end + B - 1) // B - ctx // B).sum())
        table = 4.0 * float(start.sum())   # the requests' entries for the shared blocks, compared
        return {"bytes": 2 * hkv * (held * (B * d + 4) + old * d * e + total * d * e) + 2 * total * hq * d * e + 36 * n_units + table,
                "flops": 4.0 * d * hq * keys}
    if case["op"] == "rope":
        n = float(L["new"].sum())
        per_head = 3.0 * case["rotary"] + (4.0 * d if case["norm"] else 0.0)
        return {"bytes": 2 * n * (hq + 2 * hkv) * d * e + 4 * n, "flops": n * (hq + hkv) * per_head}
    if case["op"] == "fork":
        src = L["src"]
        length = np.where(src >= 0, L["ctx"][np.maximum(src, 0)], 0)
        from_src = np.unique(src[src >= 0])
        entries = float((length // B).sum())                                  # written
        read = float((L["ctx"][from_src] // B).sum()) + float((L["had_len"] // B).sum())
        row = 2.0 * hkv * d * e
        rows = float((length % B).sum()) + float((L["ctx"][from_src] % B).sum())
        return {"bytes": 4 * (entries + read) + 8 * read + row * rows + 24 * case["n"], "flops": 0}
    n, used = case["pages"], L["used"]
    moves = used * (1.0 - used / n)   # pages in use past the last one that stays, on average
    page = 2.0 * hkv * (B * d + 4)
    return {"bytes": 2 * moves * page + 8.0 * used + 4.0 * (n + 2 * L["after"]), "flops": 0}


# ---------------------------------------------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"shared": _exact_shared, "rope": _exact_rope, "fork": _exact_fork, "compact": _exact_compact}[case["op"]](st)


def _exact_fork(st):
    """Of the outputs only the open rows are no whole numbers."""
    tail, state = st["tail"].double(), st["state"].tolist()
    for s, t in zip(st["src"].tolist(), st["dst"].tolist()):
        if s >= 0:
            tokens, buf = state[s]
            tail[t, buf, :, :, :tokens % B] = tail[s, buf, :, :, :tokens % B]
    return {"table": None, "state": None, "refs": None, "free": None, "n_free": None, "tail": tail}


def _exact_compact(st):
    """Of the outputs only the scales are no whole numbers."""
    used = (st["refs"] > 0).tolist()
    count = sum(used)
    to = [p for p in range(count) if not used[p]]
    from_ = [p for p in range(count, len(used)) if used[p]]
    res = dict.fromkeys(("k", "v", "table", "refs", "free", "n_free", "counts"))
    for name in ("k_scale", "v_scale"):
        x = st[name].double()
        x[to] = x[from_]
        res[name] = x
    return res


def _exact_shared(st):
    hq, hkv, d = st["shape"]
    g, L = hq // hkv, st["lens"]
    ctx, new = L["ctx"], L["new"]
    if float((new * (ctx + new)).sum()) * hq * d * 4 > 3.0e12:
        return None
    table, slots, bufs = st["table"].cpu().numpy(), st["slots"].tolist(), st["buf"].tolist()
    starts = np.concatenate([[0], np.cumsum(new)])
    out = torch.zeros((st["total"], hq, d), dtype=torch.float64, device=DEV)
    for i in range(len(ctx)):
        c, m, b0 = int(ctx[i]), int(new[i]), int(ctx[i]) // B
        row = slice(starts[i], starts[i + 1])
        raw = [torch.cat([st["tail"][slots[i], bufs[i], w, :, :c % B].transpose(0, 1), st[name][row]], 0).double()
               for w, name in ((0, "k_new"), (1, "v_new"))]
        page = torch.from_numpy(np.maximum(table[slots[i], :(c + m - 1) // B], 0).astype(np.int64)).to(DEV)
        for h in range(hkv):
            k8 = (st["k"][page, h].double() * st["k_scale"][page, h].double()[:, None, None]).reshape(-1, d)
            v8 = (st["v"][page, h].double() * st["v_scale"][page, h].double()[:, None, None]).reshape(-1, d)
            for b in range(b0, (c + m - 1) // B + 1):   # the queries of one block
                lo, hi = max(c, b * B), min(c + m, b * B + B)
                keys = torch.cat([k8[:b * B], raw[0][(b - b0) * B:hi - b0 * B, h]])
                vals = torch.cat([v8[:b * B], raw[1][(b - b0) * B:hi - b0 * B, h]])
                r = slice(int(starts[i]) + lo - c, int(starts[i]) + hi - c)
                qs = st["q"][r].double().view(hi - lo, hkv, g, d)[:, h].reshape(-1, d)
                logit = (qs @ keys.t()).mul_(st["scale"]).view(hi - lo, g, -1)
                late = torch.arange(hi, device=DEV)[None, :] > torch.arange(lo, hi, device=DEV)[:, None]
                p = torch.softmax(logit.masked_fill_(late[:, None, :], float("-inf")), -1)
                out[r].view(hi - lo, hkv, g, d)[:, h] = (p.view(-1, hi) @ vals).view(hi - lo, g, d)
    return {"out": out, "groups": None, "starts": None}


def _exact_rope(st):
    case = st["case"]
    hq, hkv, d = st["shape"]
    rd, n = case["rotary"], st["qkv"].shape[0]
    half = rd // 2
    x = st["qkv"].view(n, hq + 2 * hkv, d).double()
    pace = []
    for i in range(half):
        f = math.exp(-2.0 * i / rd * math.log(case["base"]))
        slow = f / case["factor"]
        if case["scaling"] == "linear":
            f = slow
        elif case["scaling"] == "parts":
            turns = case["original"] * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / 31.0))
            f = keep * f + (1 - keep) * slow
        pace.append(f)
    angle = st["positions"].double().outer(torch.tensor(pace, dtype=torch.float64, device=DEV))
    turn = torch.polar(torch.full_like(angle, st["magnitude"]), angle)[:, None, :]        # m e^{i a}
    res = {}
    for name, lo, hi in (("q", 0, hq), ("k", hq, hq + hkv)):
        y = x[:, lo:hi]
        w = st[name + "_weight"]
        if w is not None:
            y = y / torch.sqrt((y * y).sum(2, keepdim=True) / d + st["eps"]) * w.double()
        y = y.contiguous()
        if case["layout"] == "half":
            z = torch.complex(y[..., :half].contiguous(), y[..., half:rd].contiguous()) * turn
            y = torch.cat([z.real, z.imag, y[..., rd:]], 2)
        else:
            z = torch.view_as_complex(y[..., :rd].reshape(n, hi - lo, half, 2)) * turn
            y = torch.cat([torch.view_as_real(z).reshape(n, hi - lo, rd), y[..., rd:]], 2)
        res[name] = y
    res["v"] = x[:, hq + hkv:]
    return res
