"""Single tokens (and pairs) of batches so wide that a CTA works through several segments of a request's own keys, one after
another: long own parts past shared blocks that end at every remainder of the segments' length (bounds: kv_shared_ref.py)."""
import numpy as np
import pytest
import torch

from chunked_gated_deltanet_gb300 import gdn
from kv_shared_ref import B, Shared

pytestmark = pytest.mark.gpu

BF = gdn.GDN_BF16
OWN = [12, 13, 14, 15, 16, 17, 18, 19, 20, 21, 22, 25, 27, 28, 29, 30]      # own blocks of the long requests
OPEN = [1, 63, 5, 62, 17, 0, 33, 2, 48, 61, 9, 0, 60, 31, 63, 7]            # and tokens of their open blocks
PREFIX = [4, 1, 6, 3, 0, 5, 2, 7]                # shared blocks of a family


@pytest.mark.parametrize("families", [4, 40], ids=lambda n: f"{n} families")     # large ones, and small ones in one launch
# requests of 8 kv heads: 160 have two CTAs for each of them along the segments, so own parts of 3 make chains; 320 have one
@pytest.mark.parametrize("heads,d,new,requests", [((16, 8), 64, 1, 160), ((16, 8), 128, 1, 160), ((16, 8), 256, 1, 160),
                                                  ((64, 8), 128, 2, 160), ((16, 8), 64, 1, 320)],
                         ids=lambda x: f"{x[0]}q{x[1]}kv" if isinstance(x, tuple) else str(x))
def test_chained_own_segments(cuda_device, heads, d, new, requests, families):
    m = Shared(heads, d, BF, n_pages=900, n_slots=requests, max_blocks=48, seed=d + new)
    size = requests // families
    first = list(range(0, requests, size))
    prefix = [B * PREFIX[f % 8] + 20 + f for f in range(families)]
    m.step(first, prefix, check=False)
    for s in first:
        m.fork(s, *range(s + 1, s + size))
    # the long requests, spread over the families: as many from each
    long = [first[i % families] + 1 + i // families for i in range(16)]
    here = [prefix[i % families] for i in range(16)]
    m.step(long, [B * (PREFIX[i % families % 8] + OWN[i]) + OPEN[i] - here[i] for i in range(16)], check=False)
    bounds = first + [requests]
    ends = [len(s.k) + new for s in m.slots]
    suffix = max(e - B * PREFIX[s // size % 8] for s, e in enumerate(ends))
    n = requests * new
    data = m.draw(n, m.hq, 3.0), m.draw(n, m.hkv), m.draw(n, m.hkv)
    out = m.shared_step(list(range(requests)), [new] * requests, bounds, data=data, max_suffix=suffix,
                        rows_check=set(long) | set(first) | {requests - 1})
    # all of them through the unshared call. Two results, each off by 2^-8 of itself and, with v up to top and scores whose
    # sums are off by a share of the weights, (2 share + 2^-11 + 2^-16 + N 2^-24) top (kv_shared_ref.py); together 2 (..)
    plan, _ = m.last
    q, k, v = (t.to(m.dev) for t in data)
    whole = torch.full_like(out, float("nan"))
    ws = gdn.kv_attention_workspace(m.desc, n, requests, max(ends), m.dev)
    gdn.gdn_kv_attention(m.desc, m.cache, plan, q, k, v, whole, ws, new, max(ends))
    assert gdn.gdn_device_status() == gdn.GDN_OK
    top = max(float(np.abs(np.stack(m.slots[s].v)).max()) for s in [*first, *long])
    key = max(float(np.abs(np.stack(m.slots[s].k)).max()) for s in [*first, *long])
    share = d * 2.0 ** -24 * m.desc.scale * float(q.float().abs().sum(2).max()) * key + 2.0 ** -19
    tol = 2 * (2.0 ** -8 * whole.float().abs() + (2 * share + 2.0 ** -10 + max(ends) * 2.0 ** -24) * max(top, float(v.abs().max())))
    assert bool(((out.float() - whole.float()).abs() <= tol).all())
