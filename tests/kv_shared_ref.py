"""Steps of a batch whose requests share their first blocks, beside the plain model of kv_ref.py. The bounds are those of
kv_bounds.py: the shared blocks' pieces are segments like others, and a join of up to 300 of them adds at most as many fp32
roundings of 2^-24 of sum p |v|, which the model's 2^-18 of it covers."""
from __future__ import annotations

import numpy as np
import torch

from chunked_gated_deltanet_gb300 import gdn
from kv_bounds import Bounded
from kv_ref import B, TORCH


def expected_groups(table, slots, new, before, bounds):
    """groups and, per request, its shared blocks, from the block tables after the plan."""
    rows = np.concatenate([[0], np.cumsum(new)])
    recs, start = [], np.zeros(len(slots), np.int64)
    for a, b in zip(bounds, bounds[1:]):
        live = [i for i in range(a, b) if new[i]]
        if not live:
            recs.append([rows[a], 0, 0, 0])
            continue
        shared = min(before[i] // B for i in live)
        for i in live[1:]:
            same = table[slots[i], :shared] == table[slots[live[0]], :shared]
            shared = shared if same.all() else int(np.argmin(same))
        recs.append([rows[a], rows[b] - rows[a], slots[live[0]], shared])
        start[live] = shared
    return np.array(recs), start


class Shared(Bounded):
    def fork(self, src, *dst):
        for t in dst:
            gdn.gdn_kv_fork(self.desc, self.cache, src, t)
            self.slots[t] = self.slots[src].copy()

    def shared_step(self, slots, new, bounds, q_size=1.0, data=None, max_new=None, max_len=None, max_suffix=None, check=True,
                    max_groups=None, stream=None, fill=float("nan"), rows_check=None):
        n = sum(new)
        q, k, v = data or (self.draw(n, self.hq, q_size), self.draw(n, self.hkv), self.draw(n, self.hkv))
        plan = gdn.KvPlan.new(max(n, 1), len(slots), self.dev)
        groups = gdn.KvGroups.new(plan, max_groups or len(bounds) - 1)
        groups.groups.fill_(-7)
        groups.starts.fill_(-7)
        before = [len(self.slots[s].k) for s in slots]
        ends = [b + m for b, m in zip(before, new)]
        qd, kd, vd = (t.to(self.dev) for t in (q, k, v))
        out = torch.full((n, self.hq, self.d), fill, dtype=TORCH[self.dtype], device=self.dev)
        args = [self.i32(a) for a in (slots, new, bounds)]
        max_new, max_len = max_new or max(max(new), 1), max_len or max(max(ends), 1)
        max_suffix = max_suffix or max_len
        ws = gdn.kv_shared_workspace(self.desc, max(n, 1), max_len, max_suffix, self.dev)
        ws.fill_(255)                  # NaN, whatever is read before it is written
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            gdn.gdn_kv_plan(self.desc, self.cache, args[0], args[1], plan)
            gdn.gdn_kv_append(self.desc, self.cache, plan, kd, vd)
            gdn.gdn_kv_group(self.desc, self.cache, plan, args[2], groups)
            gdn.gdn_kv_attention_shared(self.desc, self.cache, plan, groups, qd, kd, vd, out, ws, max_new, max_len, max_suffix)
        if stream is not None:
            stream.synchronize()
        assert gdn.gdn_kv_status(plan) == gdn.GDN_OK
        k32, v32 = k.float().numpy(), v.float().numpy()
        row = 0
        for s, m in zip(slots, new):
            self.slots[s].k += list(k32[row:row + m])
            self.slots[s].v += list(v32[row:row + m])
            row += m
        self.last = plan, groups
        if not check:
            return out
        assert gdn.gdn_device_status() == gdn.GDN_OK
        recs, start = expected_groups(self.cache.table.cpu().numpy(), slots, new, before, bounds)
        got_groups = groups.groups.cpu().numpy()
        assert np.array_equal(got_groups[:len(recs)], recs), (got_groups, recs)
        assert not got_groups[len(recs):].any()
        units = plan.units[:int(plan.counts[0])].cpu().numpy()
        of = {s: start[i] for i, s in enumerate(slots)}
        assert np.array_equal(groups.starts[:len(units)].cpu().numpy(), [of[u[0]] for u in units])
        row, got = 0, out.double().cpu().numpy()
        for i, (s, m) in enumerate(zip(slots, new)):
            if m and (rows_check is None or i in rows_check):
                ref, bound = self.attention(s, before[i], q[row:row + m].double().numpy())
                err = np.abs(got[row:row + m] - ref)
                assert (err <= bound).all(), (s, m, float(np.nanmax(err / bound)), bool(np.isnan(err).any()))
            row += m
        return out
