"""The model of kv_ref.py with bounds taken from what the bf16 attention states about its roundings, key by key.

With p the softmax weights of a row, v the values they sum, N their number:
  scores        sums of d fp32 products, scalings and exponentials: kv_ref.py's share of every weight, 2 share sum p |v|;
  complete      weights in fp16, half a unit in the last place 2^-11 of their size, and where they are small 2^-25 of a unit
  blocks        that is 2^-4 of the row's largest weight or less (few rows: 2^-15). These roundings are independent, and of N
                they add up to about 2 sqrt(N) of one, an eighth of N from some 300 keys on: 2^-32 each; blocks whose value
                scales differ by up to 2^8 share the unit, so that a small one's weights lose as much:
                sum of 2^-11 p |v| + 2^-32 min(spread, 2^8) max(p) |v|;
  own block     weights in two bf16 numbers of 8 bits: 2^-16 sum p |v|;
  sums          fp32, a rounding per 8 products: N / 8 2^-24 sum p |v|;
  result        bf16, 8 bits: 2^-8 (|out| + all of these).
"""
from __future__ import annotations

import numpy as np

from chunked_gated_deltanet_gb300 import gdn
from kv_ref import B, Model


class Bounded(Model):
    def attention(self, s, start, q):
        out, bound = super().attention(s, start, q)
        if self.dtype != gdn.GDN_BF16:
            return out, bound
        k8, v8 = self.held(s)
        kr, vr = (np.stack(x).astype(np.float64) for x in (self.slots[s].k, self.slots[s].v))
        G, scale = self.hq // self.hkv, self.desc.scale
        for t in range(q.shape[0]):
            p = start + t
            b = p // B * B
            for h in range(self.hkv):
                K, V = np.concatenate([k8[:b, h], kr[b:p + 1, h]]), np.abs(np.concatenate([v8[:b, h], vr[b:p + 1, h]]))
                qq = q[t, h * G:(h + 1) * G]
                x = scale * qq @ K.T
                w = np.exp(x - x.max(1, keepdims=True))
                total = w.sum(1, keepdims=True)
                w /= total
                share = (self.d * 2.0 ** -24 * scale * np.abs(qq) @ np.abs(K).T).max(1, keepdims=True) + 2.0 ** -19
                size = w @ V
                tops = [x for x in V[:b].reshape(-1, B * self.d).max(1) if x > 0] if b else []
                spread = min(max(tops) / min(tops), 256.0) if tops else 1.0
                e = 2 * share * size + 2.0 ** -11 * w[:, :b] @ V[:b] + 2.0 ** -32 * spread / total * V[:b].sum(0) \
                    + 2.0 ** -16 * w[:, b:] @ V[b:] + (p + 1) / 8 * 2.0 ** -24 * size
                rows = slice(h * G, (h + 1) * G)
                bound[t, rows] = e + 2.0 ** -8 * (np.abs(out[t, rows]) + e)
        return out, bound
