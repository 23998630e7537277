"""Work for the operators of a paged key/value cache held in 8 bits: what one pass of each has to do, in plain
torch operations and through the library.

The cache keeps keys and values in blocks of 64 tokens. A complete block is held as int8, with one fp32 scale per
block and head (absmax / 127); the open block at a session's end is kept as it came, in the session's tail. A query
at position p reads the complete blocks before its own from the 8-bit cache and its own block, up to p, as it came.

Operators:
  plan    block tables and the map of 64-token units (slot, block, page, rows) of a batch, from request lengths
  append  new keys and values into the cache: complete blocks quantised, the open block into the tail
  attend  attention of the new tokens over the cache, for prompts (many new tokens) and for single tokens
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

def _plan(name, n, new, ctx, seed):
    return {"name": name, "op": "plan", "n": n, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "shared": False, "lens_seed": seed, "q_heads": 16, "kv_heads": 2, "d": 128, "dtype": "bf16"}


def _case(name, op, n, new, ctx, heads, d, dtype, seed, shared=False):
    return {"name": name, "op": op, "n": n, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "shared": shared, "lens_seed": seed, "q_heads": heads[0], "kv_heads": heads[1], "d": d, "dtype": dtype}


def listed():
    return [
        # one token of one conversation: the latency of a step's bookkeeping
        _plan("plan_token", 1, (1, 1), (41802, 41802), 1),
        # one decode step of 256 sessions
        _plan("plan_tokens_256", 256, (1, 1), (1, 16384), 2),
        # a batch of prompts, from very short to long
        _plan("plan_prompts_1024", 1024, (1, 4000), (0, 8192), 3),
        # the new key and value of each of 64 sessions (a decode step)
        _case("append_tokens_64", "append", 64, (1, 1), (1, 16384), (16, 2), 256, "bf16", 4),
        # prompts of an 8-session batch
        _case("append_prompts_8", "append", 8, (4096, 32768), (0, 700), (32, 8), 128, "bf16", 5),
        # one token at the end of a 41,802-token conversation: few heads, one long axis
        _case("token_long", "attend", 1, (1, 1), (41802, 41802), (16, 2), 256, "bf16", 6),
        # a decode step of 64 sessions of uneven length
        _case("tokens_64", "attend", 64, (1, 1), (500, 16384), (32, 8), 128, "bf16", 7),
        # a decode step in fp32, one key/value head per query head
        _case("tokens_fp32", "attend", 16, (1, 1), (100, 4096), (8, 8), 64, "fp32", 8),
        # a 290-token question over a long conversation, starting inside a block
        _case("question", "attend", 1, (290, 290), (41802, 41802), (16, 2), 256, "bf16", 9),
        # branches of 20 to 200 tokens that share a 12,000-token prefix's pages
        _case("branches_16", "attend", 16, (20, 200), (12000, 12000), (16, 4), 128, "bf16", 10, True),
        # the largest turn of a conversation near its end
        _case("turn_4000", "attend", 1, (4000, 4000), (37802, 37802), (16, 4), 128, "bf16", 11),
        # a fresh prompt of the small fp32 layer
        _case("prompt_fp32", "attend", 1, (2048, 2048), (0, 0), (2, 2), 64, "fp32", 12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attend", "attend", "attend", "attend"])
    kv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    while kv * g > 64:
        g = rng.choice([1, 2, 4, 8])
    c = {"op": op, "shared": False, "lens_seed": rng.randrange(1 << 30), "q_heads": kv * g, "kv_heads": kv,
         "d": rng.choice([64, 128, 256]), "dtype": "fp32" if rng.random() < 0.2 else "bf16"}
    if op == "plan":
        c["n"] = _log_int(rng, 1, 1024)
        c["new_lo"], c["new_hi"] = (1, 1) if rng.random() < 0.5 else (1, _log_int(rng, 16, 4000))
        c["ctx_lo"], c["ctx_hi"] = 0, _log_int(rng, 64, 32768)
        return c
    single = rng.random() < 0.5
    if op == "append":
        c["n"] = _log_int(rng, 1, 256) if single else _log_int(rng, 1, 16)
        c["new_lo"], c["new_hi"] = (1, 1) if single else (1, _log_int(rng, 64, 16384))
        c["ctx_lo"], c["ctx_hi"] = 0, _log_int(rng, 64, 2048)
    else:
        c["n"] = _log_int(rng, 1, 128) if single else _log_int(rng, 1, 12)
        new = 1 if single else _log_int(rng, 2, 4000)
        c["new_lo"], c["new_hi"] = (1 if rng.random() < 0.5 else new), new
        ctx = _log_int(rng, 64, 40000)
        c["ctx_lo"], c["ctx_hi"] = (ctx if rng.random() < 0.5 else 0), ctx
        c["shared"] = c["n"] > 1 and c["ctx_lo"] == c["ctx_hi"]
    cap = 0.9 * work(listed()[10])["flops"] * (0.05 if c["dtype"] == "fp32" else 1.0)
    while True:   # within the largest listed case, and what the plain form's padded arrays take
        w = work(c)
        n, new, ctx = c["n"], c["new_hi"], c["ctx_hi"]
        scores = n * new * c["q_heads"] * (ctx + 2 * new + 128) * 4.0 if op == "attend" else 0.0
        keys = n * (ctx + 2 * new) * c["kv_heads"] * c["d"] * 8.0 if op == "attend" else n * new * kv * c["d"] * 8.0
        if w["flops"] <= cap and w["bytes"] <= 2.0e9 and scores <= 1.2e10 and keys <= 2.0e10:
            return c
        if c["new_hi"] > 1:
            c["new_hi"] = max(1, c["new_hi"] * 3 // 4)
            c["new_lo"] = min(c["new_lo"], c["new_hi"])
        elif c["n"] > 1:
            c["n"] = max(1, c["n"] * 3 // 4)
            c["shared"] = c["shared"] and c["n"] > 1
        else:
            c["ctx_hi"] = c["ctx_hi"] * 3 // 4
            c["ctx_lo"] = min(c["ctx_lo"], c["ctx_hi"])


def _lens(case):
    """(tokens already in the cache, new tokens) per request: a function of the case alone."""
    rs = np.random.RandomState(case["lens_seed"] % (1 << 31))
    n = case["n"]

    def spread(lo, hi):   # over the logarithm
        if lo == hi:
            return np.full(n, lo, dtype=np.int64)
        x = np.exp(rs.uniform(math.log(lo + 1), math.log(hi + 1), n)) - 1
        return np.clip(np.rint(x).astype(np.int64), lo, hi)

    new = spread(case["new_lo"], case["new_hi"])
    ctx = spread(case["ctx_lo"], case["ctx_hi"])
    return ctx, new


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    ctx, new = _lens(case)
    n, hq, hkv, d = case["n"], case["q_heads"], case["kv_heads"], case["d"]
    dt = DT[case["dtype"]]
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "plan":   # other inputs: the same lengths in another order
        order = rs.permutation(n)
        ctx, new = ctx[order], new[order]
    end = ctx + new
    full_before, full_after = ctx // B, end // B
    held = int(full_before[0]) + 0 if case["shared"] else int(full_before.sum())
    taken = int((full_after - full_before).sum())
    n_slots = n + 3
    max_blocks = int(full_after.max()) + 2
    spare = 5
    n_pages = held + taken + spare
    pages = rs.permutation(n_pages).astype(np.int32)
    slots = rs.permutation(n_slots)[:n].astype(np.int32)
    buf = rs.randint(0, 2, n).astype(np.int32)
    state = np.zeros((n_slots, 2), dtype=np.int32)
    state[slots, 0], state[slots, 1] = ctx, buf
    table = np.full((n_slots, max_blocks), -1, dtype=np.int32)
    at = 0
    for i in range(n):
        m = int(full_before[i])
        table[slots[i], :m] = pages[:m] if case["shared"] else pages[at:at + m]
        at += 0 if case["shared"] else m
    free = np.zeros(n_pages, dtype=np.int32)
    n_free = n_pages - held
    free[:n_free] = pages[held:]
    total = int(new.sum())
    n_units = int(np.where(new > 0, (end + B - 1) // B - full_before, 0).sum())
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)   # noqa: E731
    refs = torch.zeros(n_pages + 1, dtype=torch.int32, device=DEV)
    refs[to(pages[:held]).long()] = n if case["shared"] else 1
    units_cap = min(total, total // B + 2 * n)
    st = {"case": case, "op": case["op"], "n": n, "total": total, "n_units": n_units, "max_new": int(new.max()),
          "max_len": int(end.max()), "new_dev": to(new.astype(np.int32)), "slots": to(slots), "state": to(state),
          "table": to(table), "free": to(free), "n_free": to(np.array([n_free], dtype=np.int32)),
          "refs_full": refs, "n_pages": n_pages, "n_slots": n_slots, "max_blocks": max_blocks,
          "scale": 1.0 / math.sqrt(d), "shape": (hq, hkv, d),
          # the plan's own buffers, as a program keeps them from step to step
          "rows": torch.zeros(n + 1, dtype=torch.int32, device=DEV),
          "units": torch.zeros((units_cap, 8), dtype=torch.int32, device=DEV),
          "counts": torch.zeros(2, dtype=torch.int32, device=DEV),
          "state_out": torch.zeros((n_slots, 2), dtype=torch.int32, device=DEV),
          "n_free_out": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if case["op"] == "plan":
        # nothing else of the cache is touched
        st.update(k=torch.zeros((n_pages + 1, 1, 1, 1), dtype=torch.int8, device=DEV))
        return st
    st.update(_plan_plain(st))   # append and attend are given a plan
    shape = (n_pages + 1, hkv, B, d)   # one page more than the cache has: see _append_plain

    def values(*size):   # activations, with heads of unequal size
        x = torch.randn(size, generator=gen, device=DEV)
        return x * (0.5 + torch.rand((size[-2], 1), generator=gen, device=DEV))

    if case["op"] == "append":
        st["k"] = torch.zeros(shape, dtype=torch.int8, device=DEV)
        st["v"] = torch.zeros(shape, dtype=torch.int8, device=DEV)
        st["k_scale"] = torch.zeros(shape[:2], device=DEV)
        st["v_scale"] = torch.zeros(shape[:2], device=DEV)
    else:
        # a block's largest of 64 d normal values is near 4: 8-bit steps of about 4 / 127
        st["k"] = (torch.randn(shape, generator=gen, device=DEV) * 32).round_().clamp_(-127, 127).to(torch.int8)
        st["v"] = (torch.randn(shape, generator=gen, device=DEV) * 32).round_().clamp_(-127, 127).to(torch.int8)
        st["k_scale"] = (0.02 + 0.03 * torch.rand(shape[:2], generator=gen, device=DEV))
        st["v_scale"] = (0.02 + 0.03 * torch.rand(shape[:2], generator=gen, device=DEV))
        # queries of heads that look at few keys and of heads that look at many
        temp = 0.5 + 2.5 * torch.rand((hq, 1), generator=gen, device=DEV)
        st["q"] = (torch.randn((total, hq, d), generator=gen, device=DEV) * temp).to(dt)
        st["out"] = torch.zeros((total, hq, d), dtype=dt, device=DEV)
    st["k_new"] = values(total, hkv, d).to(dt)
    st["v_new"] = values(total, hkv, d).to(dt)
    # the open blocks as they came: [slot][buffer][key / value][head][offset][d], one slot more than the cache has
    st["tail"] = torch.randn((n_slots + 1, 2, 2, hkv, B, d), generator=gen, device=DEV).to(dt)
    return st


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------

def _plan_plain(st):
    """Units of 64 absolute positions: [slot, block, page or -1, first offset, count, first row, tail read, tail written]."""
    dev = st["slots"].device
    slots, new = st["slots"].long(), st["new_dev"].long()
    ctx, buf = st["state"][slots, 0].long(), st["state"][slots, 1].long()
    rows = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), new.cumsum(0)])
    end = ctx + new
    first_block = ctx // B
    n_blocks = torch.where(new > 0, (end + B - 1) // B - first_block, torch.zeros_like(new))
    before = n_blocks.cumsum(0) - n_blocks
    U = st["n_units"]
    req = torch.repeat_interleave(torch.arange(st["n"], device=dev), n_blocks, output_size=U)
    block = first_block[req] + torch.arange(U, device=dev) - before[req]
    start = torch.maximum(ctx[req], block * B)
    stop = torch.minimum(end[req], block * B + B)
    closes = stop == block * B + B
    order = closes.long().cumsum(0) - 1
    page = st["free"].long()[(st["n_free"].long() - 1 - order).clamp_(0, st["n_pages"] - 1)]
    new_buf = torch.where(end // B != first_block, 1 - buf, buf)
    slot = slots[req]
    minus = torch.full_like(page, -1)
    units = torch.stack([slot, block, torch.where(closes, page, minus), start - block * B, stop - start,
                         rows[req] + start - ctx[req], buf[req], torch.where(closes, minus, new_buf[req])], 1)
    old = st["table"][slot, block.clamp(max=st["max_blocks"] - 1)]
    st["table"][slot, block.clamp(max=st["max_blocks"] - 1)] = torch.where(closes, page.int(), old)
    st["refs_full"][torch.where(closes, page, torch.full_like(page, st["n_pages"]))] = 1
    st["state_out"][slots] = torch.stack([end, new_buf], 1).int()
    st["n_free_out"].copy_(st["n_free"] - closes.sum())
    st["rows"].copy_(rows)
    st["units"][:U] = units.int()
    st["counts"][:1] = U
    return {}


def _append_plain(st):
    """Blocks that close: absmax / 127 per block and head, rounded to nearest even. The last block into the tail."""
    U, (_, hkv, d) = st["n_units"], st["shape"]
    u = st["units"][:U].long()
    slot, page, first, count, row, src, dst = u[:, 0], u[:, 2], u[:, 3], u[:, 4], u[:, 5], u[:, 6], u[:, 7]
    off = torch.arange(B, device=u.device)
    fresh = (off >= first[:, None]) & (off < (first + count)[:, None])
    at = (row[:, None] + off - first[:, None]).clamp_(0, st["total"] - 1)
    closes = page >= 0
    to_page = torch.where(closes, page, torch.full_like(page, st["n_pages"]))      # open blocks: to the page that
    to_slot = torch.where(closes, torch.full_like(slot, st["n_slots"]), slot)      # no one reads, closed: the slot
    out_buf = dst.clamp(min=0)
    limit = torch.full((), 127.0, device=u.device)
    m = fresh[:, None, :, None]
    new_k, new_v = st["k_new"][at].transpose(1, 2), st["v_new"][at].transpose(1, 2)    # [U][head][64][d]
    x = torch.where(m, new_k, st["tail"][slot, src, 0]).float()
    scale = x.abs().amax((2, 3)) / limit
    y = torch.where(scale[..., None, None] > 0, x / scale[..., None, None], torch.zeros_like(x)).round()
    st["k"][to_page] = y.to(torch.int8)
    st["k_scale"][to_page] = scale
    x = torch.where(m, new_v, st["tail"][slot, src, 1]).float()
    scale = x.abs().amax((2, 3)) / limit
    y = torch.where(scale[..., None, None] > 0, x / scale[..., None, None], torch.zeros_like(x)).round()
    st["v"][to_page] = y.to(torch.int8)
    st["v_scale"][to_page] = scale
    st["tail"][to_slot, out_buf, 0] = torch.where(m, new_k, st["tail"][to_slot, out_buf, 0])
    st["tail"][to_slot, out_buf, 1] = torch.where(m, new_v, st["tail"][to_slot, out_buf, 1])


def _attend_plain(st):
    """softmax(scale q k^T) v over [complete blocks before the query's own, from 8 bits; its own block as it came]."""
    hq, hkv, d = st["shape"]
    g, n, dev = hq // hkv, st["n"], st["q"].device
    slots, new = st["slots"].long(), st["new_dev"].long()
    ctx, buf = st["state"][slots, 0].long(), st["state"][slots, 1].long()
    rows, T = st["rows"].long(), st["max_new"]
    t = torch.arange(T, device=dev)
    at = (rows[:-1, None] + t).clamp_(max=st["total"] - 1)                              # [n][T]
    q = st["q"][at].float().view(n, T, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, T * g, d) * st["scale"]
    qpos = ctx[:, None] + t
    qblk = qpos // B
    # complete blocks, from 8 bits
    nb = max(1, (st["max_len"] - 1) // B)
    pages = st["table"][slots, :nb].long().clamp_(min=0)                                # [n][nb]
    k = (st["k"][pages].float() * st["k_scale"][pages][..., None, None]).transpose(1, 2).reshape(n, hkv, nb * B, d)
    v = (st["v"][pages].float() * st["v_scale"][pages][..., None, None]).transpose(1, 2).reshape(n, hkv, nb * B, d)
    see = torch.arange(nb * B, device=dev) // B < qblk[..., None]                       # [n][T][nb 64]
    # the blocks that the new tokens lie in, as they came
    base = ctx // B * B
    R = min(T + B - 1, -(-st["max_len"] // B) * B)
    r = torch.arange(R, device=dev)
    kpos = base[:, None] + r                                                            # [n][R]
    in_tail = (kpos < ctx[:, None])[..., None, None]
    fresh = (rows[:-1, None] + kpos - ctx[:, None]).clamp_(0, st["total"] - 1)
    tail = st["tail"][slots, buf].permute(1, 0, 3, 2, 4)[:, :, r.clamp(max=B - 1)]      # [2][n][R][hkv][d]
    kr = torch.where(in_tail, tail[0], st["k_new"][fresh]).float().transpose(1, 2)      # [n][hkv][R][d]
    vr = torch.where(in_tail, tail[1], st["v_new"][fresh]).float().transpose(1, 2)
    see_r = (kpos[:, None, :] // B == qblk[..., None]) & (kpos[:, None, :] <= qpos[..., None])
    s = torch.cat([q @ k.transpose(2, 3), q @ kr.transpose(2, 3)], 3)
    mask = torch.cat([see, see_r], 2)[:, None, :, None, :].expand(n, 1, T, g, nb * B + R).reshape(n, 1, T * g, -1)
    s.masked_fill_(~mask, float("-inf"))
    s -= s.amax(3, keepdim=True).clamp_(min=-1e30)
    s.exp_()
    total = s.sum(3, keepdim=True)
    o = (s[..., :nb * B] @ v + s[..., nb * B:] @ vr) / total.clamp_(min=1e-30)
    o = o.view(n, hkv, T, g, d).permute(0, 2, 1, 3, 4).reshape(n * T, hq, d)
    req = torch.repeat_interleave(torch.arange(n, device=dev), new, output_size=st["total"])
    st["out"].copy_(o[req * T + torch.arange(st["total"], device=dev) - rows[req]])


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def _handles(st):
    """The library's handles over the program's buffers, made once, as a program makes them."""
    if "handles" not in st:
        from chunked_gated_deltanet_gb300 import gdn
        hq, hkv, d = st["shape"]
        desc = gdn.make_attn_desc(hq, hkv, d, gdn.GDN_FP32 if st["case"]["dtype"] == "fp32" else gdn.GDN_BF16,
                                  st["scale"])
        P, S = st["n_pages"], st["n_slots"]
        if st["op"] == "plan":
            cache = gdn.KvCache(desc, P, S, st["max_blocks"], DEV, state=st["state"], table=st["table"],
                                free=st["free"], n_free=st["n_free"], refs=st["refs_full"][:P])
        else:
            cache = gdn.KvCache(desc, P, S, st["max_blocks"], DEV, k=st["k"][:P], v=st["v"][:P],
                                k_scale=st["k_scale"][:P], v_scale=st["v_scale"][:P], tail=st["tail"][:S],
                                state=st["state"], table=st["table"], free=st["free"], n_free=st["n_free"],
                                refs=st["refs_full"][:P])
        plan = gdn.KvPlan(st["rows"], st["units"], st["counts"])
        ws = gdn.kv_attention_workspace(desc, st["total"], st["n"], st["max_len"], DEV) if st["op"] == "attend" else None
        st["handles"] = (gdn, desc, cache, plan, ws)
    return st["handles"]


def run(st):
    if own:
        gdn, desc, cache, plan, ws = _handles(st)
        if st["op"] == "plan":
            gdn.gdn_kv_plan(desc, cache, st["slots"], st["new_dev"], plan, state_out=st["state_out"],
                            n_free_out=st["n_free_out"])
        elif st["op"] == "append":
            gdn.gdn_kv_append(desc, cache, plan, st["k_new"], st["v_new"])
        else:
            gdn.gdn_kv_attention(desc, cache, plan, st["q"], st["k_new"], st["v_new"], st["out"], ws,
                                 st["max_new"], st["max_len"])
    else:
        {"plan": _plan_plain, "append": _append_plain, "attend": _attend_plain}[st["op"]](st)
    if st["op"] == "plan":
        return {"rows": st["rows"], "units": st["units"][:st["n_units"]], "counts": st["counts"],
                "table": st["table"], "refs": st["refs_full"][:st["n_pages"]], "state": st["state_out"],
                "n_free": st["n_free_out"]}
    if st["op"] == "append":   # the 8-bit values are whole numbers, times the scale beside them
        P, S = st["n_pages"], st["n_slots"]
        return {"k": st["k"][:P], "v": st["v"][:P], "k_scale": st["k_scale"][:P], "v_scale": st["v_scale"][:P],
                "tail": st["tail"][:S]}
    return {"out": st["out"]}


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------

def work(case):
    ctx, new = _lens(case)
    end = ctx + new
    hq, hkv, d, n = case["q_heads"], case["kv_heads"], case["d"], case["n"]
    e = 4 if case["dtype"] == "fp32" else 2
    total = float(new.sum())
    closed = float((end // B - ctx // B).sum())
    n_units = float(np.where(new > 0, (end + B - 1) // B - ctx // B, 0).sum())
    if case["op"] == "plan":   # slots, counts, lengths, free pages in; rows, units, table entries, page counts out
        return {"bytes": n * (4 + 4 + 8) + closed * 4 + (n + 1) * 4 + n_units * 32 + closed * 8 + n * 8, "flops": 0}
    if case["op"] == "append":
        first, last = ctx % B, end % B
        cross = end // B != ctx // B
        old = float(np.where(cross & (new > 0), first, 0).sum())             # tail rows that a closing block takes in
        opened = float(np.where(cross, last, new).sum())                     # new rows that stay open
        return {"bytes": 2 * hkv * (d * (e * (total + old) + e * opened + closed * B) + 4 * closed) + 32 * n_units,
                "flops": 3 * 2 * hkv * d * closed * B}
    pos = lambda m: m * (m + 1) / 2.0   # noqa: E731  keys seen by the queries at positions 0 .. m - 1
    keys = float((pos(end) - pos(ctx)).sum())
    blocks = np.maximum(end - 1, 0) // B
    held = float(blocks.max()) if case["shared"] else float(blocks.sum())    # branches share their prefix's pages
    if case["shared"]:
        held += float((blocks - ctx // B).sum())
    old = float((ctx % B).sum())
    return {"bytes": 2 * hkv * (held * (B * d + 4) + old * d * e + total * d * e) + 2 * total * hq * d * e + 32 * n_units,
            "flops": 4.0 * d * hq * keys}


# ---------------------------------------------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":
        return None
    st = prepare(case, seed)
    ctx, new = _lens(case)
    hq, hkv, d = st["shape"]
    P, S = st["n_pages"], st["n_slots"]
    slots, bufs = st["slots"].tolist(), st["state"][st["slots"].long(), 1].tolist()
    starts = np.concatenate([[0], np.cumsum(new)])
    table = st["table"].cpu().numpy()

    def history(i, which, name):
        """Request i's rows from its first touched block on, as they came: [len][hkv][d]."""
        o = int(ctx[i]) % B
        old = st["tail"][slots[i], bufs[i], which, :, :o].transpose(0, 1)
        return torch.cat([old, st[name][starts[i]:starts[i + 1]]], 0).double()

    if case["op"] == "append":
        if 2.0 * hkv * d * float(new.sum()) > 6e8:
            return None
        out = {"k": None, "v": None, "k_scale": st["k_scale"][:P].double(), "v_scale": st["v_scale"][:P].double(),
               "tail": st["tail"][:S].double()}
        for i in range(case["n"]):
            b0, b1 = int(ctx[i]) // B, int(ctx[i] + new[i]) // B
            for which, name in ((0, "k"), (1, "v")):
                h = history(i, which, name + "_new")
                m = (b1 - b0) * B
                if m:
                    top = h[:m].abs().view(b1 - b0, B, hkv, d).amax((1, 3)) / 127
                    out[name + "_scale"][torch.from_numpy(table[slots[i], b0:b1].astype(np.int64)).to(top.device)] = top
                o = 0 if b1 > b0 else int(ctx[i]) % B
                dst = bufs[i] ^ int(b1 > b0)
                out["tail"][slots[i], dst, which, :, o:h.shape[0] - m] = h[m + o:].transpose(0, 1)
        return out
    T = new.astype(np.float64)
    if float((T * (ctx + new)).sum()) * hq * d * 4 > 1.5e12:
        return None
    out = torch.zeros((st["total"], hq, d), dtype=torch.float64, device=DEV)
    for i in range(case["n"]):
        c, m, b0 = int(ctx[i]), int(new[i]), int(ctx[i]) // B
        kr, vr = history(i, 0, "k_new"), history(i, 1, "v_new")
        nb = (c + m - 1) // B
        pg = torch.from_numpy(np.maximum(table[slots[i], :nb], 0).astype(np.int64)).to(DEV)
        for h in range(hkv):
            k8 = (st["k"][pg, h].double() * st["k_scale"][pg, h].double()[:, None, None]).reshape(-1, d)
            v8 = (st["v"][pg, h].double() * st["v_scale"][pg, h].double()[:, None, None]).reshape(-1, d)
            for b in range(b0, (c + m - 1) // B + 1):   # the queries of one block
                lo, hi = max(c, b * B), min(c + m, b * B + B)
                keys = torch.cat([k8[:b * B], kr[(b - b0) * B:hi - b0 * B, h]])
                vals = torch.cat([v8[:b * B], vr[(b - b0) * B:hi - b0 * B, h]])
                r = slice(int(starts[i]) + lo - c, int(starts[i]) + hi - c)
                qs = st["q"][r].double().view(hi - lo, hkv, hq // hkv, d)[:, h]
                logit = torch.einsum("tgd,kd->tgk", qs, keys) * st["scale"]
                late = torch.arange(hi, device=DEV)[None, :] > torch.arange(lo, hi, device=DEV)[:, None]
                p = torch.softmax(logit.masked_fill(late[:, None, :], float("-inf")), -1)
                out[r].view(hi - lo, hkv, hq // hkv, d)[:, h] = torch.einsum("tgk,kd->tgd", p, vals)
    return {"out": out}
