"""Group bounds that name requests which the plan does not have, in a map that has room for them (and may hold an earlier plan's
prefix sums there): no group shares anything, the call is reported, the rows are right (bounds: kv_shared_ref.py)."""
import numpy as np
import pytest
import torch

from chunked_gated_deltanet_gb300 import gdn
from kv_shared_ref import Shared

pytestmark = pytest.mark.gpu

BF, F32 = gdn.GDN_BF16, gdn.GDN_FP32


@pytest.mark.parametrize("bounds", [[0, 3], [0, 2, 3], [0, 1, 4], [0, 6], [3, 4], [0, 2, 2, 5]], ids=str)
@pytest.mark.parametrize("earlier", [[1, 1, 1, 1], [100, 1, 200, 3, 40, 2]], ids=["few rows", "many rows"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_bounds_past_the_plans_requests(cuda_device, dtype, earlier, bounds):
    m = Shared((4, 2), 64, dtype, n_slots=6, max_blocks=16, seed=3)
    plan = gdn.KvPlan.new(400, 6, m.dev)
    gdn.gdn_kv_plan(m.desc, m.cache, m.i32(range(len(earlier))), m.i32(earlier), plan)   # its prefix sums stay in the map
    for s in range(6):
        gdn.gdn_kv_release(m.desc, m.cache, s)
    m.step([0], [200], check=False)
    m.fork(0, 1)
    new = [70, 65]
    n = sum(new)
    q, k, v = m.draw(n, 4), m.draw(n, 2), m.draw(n, 2)
    qd, kd, vd = (t.to(m.dev) for t in (q, k, v))
    groups = gdn.KvGroups.new(plan, 4)
    gdn.gdn_kv_plan(m.desc, m.cache, m.i32([0, 1]), m.i32(new), plan)
    gdn.gdn_kv_append(m.desc, m.cache, plan, kd, vd)
    gdn.gdn_kv_group(m.desc, m.cache, plan, m.i32(bounds), groups)
    out = torch.full_like(qd, float("nan"))
    ws = gdn.kv_shared_workspace(m.desc, n, 300, 300, m.dev)
    ws.fill_(255)
    gdn.gdn_kv_attention_shared(m.desc, m.cache, plan, groups, qd, kd, vd, out, ws, 70, 300, 300)
    status = gdn.gdn_device_status()
    for i, r in enumerate((slice(0, 70), slice(70, n))):
        m.slots[i].k += list(k[r].float().numpy())
        m.slots[i].v += list(v[r].float().numpy())
        ref, bound = m.attention(i, 200, q[r].double().numpy())
        assert (np.abs(out[r].double().cpu().numpy() - ref) <= bound).all()
    assert status == gdn.GDN_ERR_INVALID_ARG
    assert not groups.groups[:, 3].any() and not groups.starts[:int(plan.counts[0])].any()


def test_the_plans_own_requests_are_in_range(cuda_device):
    """The last request's end is a bound, whatever the map held behind it."""
    m = Shared((4, 2), 64, BF, n_slots=6, seed=3)
    plan = gdn.KvPlan.new(400, 6, m.dev)
    gdn.gdn_kv_plan(m.desc, m.cache, m.i32(range(6)), m.i32([1] * 6), plan)
    for s in range(6):
        gdn.gdn_kv_release(m.desc, m.cache, s)
    m.step([0], [200], check=False)
    m.fork(0, 1, 2)
    groups = gdn.KvGroups.new(plan, 1)
    for new in ([1, 1, 1], [0, 2, 0]):
        gdn.gdn_kv_plan(m.desc, m.cache, m.i32([0, 1, 2]), m.i32(new), plan)
        gdn.gdn_kv_group(m.desc, m.cache, plan, m.i32([0, 3]), groups)
        assert gdn.gdn_device_status() == gdn.GDN_OK
        assert groups.groups[0, 1] == sum(new) and groups.groups[0, 3] == 3
