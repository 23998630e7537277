"""The paged 8-bit key/value cache and its attention from their definition, on the CPU: a plain model of the slots in
numpy (float32 for the quantiser, which is defined by IEEE operations, float64 for the attention), and the bounds that
the kernels' roundings give.

Bounds of an output element, with p the softmax weights and v the values it sums:
  bf16: each weight enters the second product rounded to bf16 (half a unit in the last place, 2^-9 of its size) and the
        result is rounded once more: 2^-9 (sum p |v| + |out|);
  both: a score is a sum of d fp32 products, off by at most d 2^-24 scale sum |q k| (and as much again for the
        scalings, the exponential and the sums), which changes every weight by that share: 2 share sum p |v|.
"""
from __future__ import annotations

import numpy as np
import torch

from chunked_gated_deltanet_gb300 import gdn

B = 64
TORCH = {gdn.GDN_BF16: torch.bfloat16, gdn.GDN_FP32: torch.float32}


def quantise(x: np.ndarray):
    """x: fp32 [64][d] of one head -> (int8 values, fp32 scale)."""
    scale = np.float32(np.abs(x).max()) / np.float32(127)
    if scale == 0:
        return np.zeros(x.shape, np.int8), scale
    return np.rint(x / scale).astype(np.int8), scale


class Slot:
    def __init__(self):
        self.k, self.v = [], []      # fp32 [Hkv][d] per token, as they came

    def copy(self):
        s = Slot()
        s.k, s.v = list(self.k), list(self.v)
        return s


class Model:
    """A cache on the GPU beside its plain model; step() runs plan, append and attention and checks all of them."""

    def __init__(self, heads, d, dtype, n_pages=64, n_slots=5, max_blocks=32, seed=0, device="cuda", scale=None):
        self.hq, self.hkv = heads
        self.d, self.dtype = d, dtype
        self.desc = gdn.make_attn_desc(self.hq, self.hkv, d, dtype, scale)
        self.cache = gdn.KvCache(self.desc, n_pages, n_slots, max_blocks, device)
        self.slots = [Slot() for _ in range(n_slots)]
        self.gen = torch.Generator().manual_seed(seed)
        self.dev = device
        self.ws_bytes = None

    def draw(self, n, heads, size=1.0):
        return (torch.randn((n, heads, self.d), generator=self.gen) * size).to(TORCH[self.dtype])

    def i32(self, a):
        return torch.tensor(a, dtype=torch.int32, device=self.dev)

    def step(self, slots, new, q_size=1.0, check=True, data=None, max_new=None, max_len=None):
        n = sum(new)
        q, k, v = data or (self.draw(n, self.hq, q_size), self.draw(n, self.hkv), self.draw(n, self.hkv))
        plan = gdn.KvPlan.new(max(n, 1), len(slots), self.dev)
        gdn.gdn_kv_plan(self.desc, self.cache, self.i32(slots), self.i32(new), plan)
        assert gdn.gdn_kv_status(plan) == gdn.GDN_OK
        qd, kd, vd = (t.to(self.dev) for t in (q, k, v))
        out = torch.full((n, self.hq, self.d), float("nan"), dtype=TORCH[self.dtype], device=self.dev)
        gdn.gdn_kv_append(self.desc, self.cache, plan, kd, vd)
        ends = [len(self.slots[s].k) + m for s, m in zip(slots, new)]
        max_new, max_len = max_new or max(max(new), 1), max_len or max(max(ends), 1)
        ws = gdn.kv_attention_workspace(self.desc, max(n, 1), len(slots), max_len, self.dev)
        if self.ws_bytes:
            ws = ws[:self.ws_bytes]
        gdn.gdn_kv_attention(self.desc, self.cache, plan, qd, kd, vd, out, ws, max_new, max_len)
        assert gdn.gdn_device_status() == gdn.GDN_OK
        k32, v32 = k.float().numpy(), v.float().numpy()
        row, before = 0, {}
        for s, m in zip(slots, new):
            before[s] = len(self.slots[s].k)
            self.slots[s].k += list(k32[row:row + m])
            self.slots[s].v += list(v32[row:row + m])
            row += m
        if check:
            row, got = 0, out.double().cpu().numpy()
            for s, m in zip(slots, new):
                if m:
                    ref, bound = self.attention(s, before[s], q[row:row + m].double().numpy())
                    err = np.abs(got[row:row + m] - ref)
                    assert (err <= bound).all(), (s, m, float((err / bound).max()))
                row += m
        return out

    def held(self, s):
        """8-bit view of a slot: dequantised float64 K and V of its complete blocks."""
        sl, nb = self.slots[s], len(self.slots[s].k) // B
        out = []
        for rows in (sl.k, sl.v):
            x = np.zeros((nb * B, self.hkv, self.d))
            for b in range(nb):
                for h in range(self.hkv):
                    qv, sc = quantise(np.stack([rows[b * B + j][h] for j in range(B)]))
                    x[b * B:(b + 1) * B, h] = qv.astype(np.float64) * np.float64(sc)
            out.append(x)
        return out

    def attention(self, s, start, q):
        """Outputs of the queries at positions start .. of slot s and their error bounds."""
        k8, v8 = self.held(s)
        kr, vr = np.stack(self.slots[s].k).astype(np.float64), np.stack(self.slots[s].v).astype(np.float64)
        G, scale = self.hq // self.hkv, self.desc.scale
        out, bound = np.zeros_like(q), np.zeros_like(q)
        for t in range(q.shape[0]):
            p = start + t
            b = p // B * B
            for h in range(self.hkv):
                K = np.concatenate([k8[:b, h], kr[b:p + 1, h]])
                V = np.concatenate([v8[:b, h], vr[b:p + 1, h]])
                qq = q[t, h * G:(h + 1) * G]
                x = scale * qq @ K.T
                w = np.exp(x - x.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                o, size = w @ V, w @ np.abs(V)
                share = (self.d * 2.0 ** -24 * scale * np.abs(qq) @ np.abs(K).T).max(1, keepdims=True) + 2.0 ** -19
                e = 2 * share * size
                if self.dtype == gdn.GDN_BF16:
                    e += 2.0 ** -9 * (size * (1 + share) + np.abs(o) + e)
                out[t, h * G:(h + 1) * G], bound[t, h * G:(h + 1) * G] = o, e
        return out, bound

    def check_contents(self):
        """Lengths, block tables, pages, scales, open blocks and the free stack against the plain model."""
        c = self.cache
        state, table = c.state.cpu().numpy(), c.table.cpu().numpy()
        refs, n_free = c.refs.cpu().numpy(), int(c.n_free.item())
        pk, pv, ks, vs = (t.cpu().numpy() for t in (c.k, c.v, c.k_scale, c.v_scale))
        tail = c.tail.float().cpu().numpy()
        used = {}
        for s, sl in enumerate(self.slots):
            n = len(sl.k)
            assert state[s, 0] == n
            for b in range(n // B):
                page = int(table[s, b])
                used[page] = used.get(page, 0) + 1
                for h in range(self.hkv):
                    for pool, scales, rows in ((pk, ks, sl.k), (pv, vs, sl.v)):
                        qv, sc = quantise(np.stack([rows[b * B + j][h] for j in range(B)]))
                        assert scales[page, h] == sc
                        assert np.array_equal(pool[page, h], qv)
            o = n % B
            for which, rows in ((0, sl.k), (1, sl.v)):
                if o:
                    assert np.array_equal(tail[s, state[s, 1], which, :, :o], np.stack(rows[n - o:]).transpose(1, 0, 2))
        assert n_free == c.n_pages - len(used)
        free = set(c.free[:n_free].tolist())
        assert len(free) == n_free and not free & set(used)
        for page, m in used.items():
            assert refs[page] == m
