"""Batched forks and releases, and compaction, of the paged cache: every book entry and page equal to the plain model's."""
import numpy as np
import pytest
import torch

from chunked_gated_deltanet_gb300 import gdn
from kv_ref import B, Model, Slot

pytestmark = pytest.mark.gpu

BF, F32 = gdn.GDN_BF16, gdn.GDN_FP32


def books(c):
    return [t.cpu().numpy().copy() for t in (c.state, c.table, c.refs, c.free, c.n_free)]


def plain_fork(c, src, dst):
    """The books after a batch of forks, from those before it."""
    state, table, refs, free, n_free = books(c)
    was, old_table, old_refs = state.copy(), table.copy(), refs.copy()
    for s, t in zip(src, dst):
        if s >= 0:
            np.add.at(refs, old_table[s, :was[s, 0] // B], 1)
    for s, t in zip(src, dst):
        np.subtract.at(refs, old_table[t, :was[t, 0] // B], 1)
        if s >= 0:
            nb = was[s, 0] // B
            table[t, :nb] = old_table[s, :nb]
        state[t] = was[s] if s >= 0 else (0, was[t, 1])
    freed = np.flatnonzero((refs == 0) & (old_refs > 0))
    free[n_free[0]:n_free[0] + len(freed)] = freed
    return state, table, refs, free, n_free + len(freed)


def same_books(c, want):
    state, table, refs, free, n_free = books(c)
    w_state, w_table, w_refs, w_free, w_n = want
    assert np.array_equal(state, w_state) and np.array_equal(refs, w_refs) and np.array_equal(n_free, w_n)
    assert np.array_equal(table, w_table)
    assert np.array_equal(free[:n_free[0]], w_free[:w_n[0]])


def fork_batch(m, src, dst):
    want = plain_fork(m.cache, src, dst)
    gdn.gdn_kv_fork_batch(m.desc, m.cache, m.i32(src), m.i32(dst))
    same_books(m.cache, want)
    slots = [m.slots[s].copy() if s >= 0 else Slot() for s in src]
    for t, s in zip(dst, slots):
        m.slots[t] = s


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("heads,d", [((2, 1), 64), ((6, 3), 128), ((2, 2), 256)])
def test_forks_and_releases(cuda_device, heads, d, dtype):
    """Forks of one and of several slots over empty, full and sharing ones; releases; forks of an empty slot."""
    m = Model(heads, d, dtype, n_pages=64, n_slots=9, max_blocks=8, seed=d)
    m.step([0, 3], [200, 64], check=False)
    fork_batch(m, [0, 0, 3], [1, 2, 4])
    m.step([1, 2, 4, 0], [100, 3, 64, 1])                 # forks go apart
    m.check_contents()
    fork_batch(m, [1, 3, -1, 1, 8], [0, 2, 4, 5, 6])      # over what was held; 8 and so 6 are empty
    m.check_contents()
    fork_batch(m, [5], [1])                               # the pages of slot 1 keep their names through 0 and 5
    fork_batch(m, [-1, -1, -1, -1], [0, 1, 5, 7])
    m.step([2, 3, 0], [70, 1, 5])
    m.check_contents()
    fork_batch(m, [-1] * 9, list(range(9)))
    assert int(m.cache.n_free) == 64 and not m.cache.refs.any()


def test_the_call_equals_forks_one_by_one(cuda_device):
    m, one = (Model((4, 2), 128, BF, n_pages=40, n_slots=6, max_blocks=8, seed=3) for _ in range(2))
    for x in (m, one):
        x.step([0, 4], [333, 70], check=False)
    gdn.gdn_kv_fork_batch(m.desc, m.cache, m.i32([0, 4, 0]), m.i32([1, 2, 5]))
    for s, t in ((0, 1), (4, 2), (0, 5)):
        gdn.gdn_kv_fork(one.desc, one.cache, s, t)
    got, want = books(m.cache), books(one.cache)
    valid = np.arange(8) < got[0][:, :1] // B                # the other entries of a table were never written
    got[1], want[1] = got[1][valid], want[1][valid]
    for a, b in zip(got, want):
        assert np.array_equal(a, b)


def test_many_slots(cuda_device):
    """4,096 pairs of 8,200 slots, several sources, over slots that held pages of their own."""
    n_slots = 8200
    m = Model((1, 1), 64, BF, n_pages=20000, n_slots=n_slots, max_blocks=6, seed=1)
    rs = np.random.RandomState(0)
    order = rs.permutation(n_slots).tolist()
    src, dst = order[:5], order[5:4101]
    # books alone: lengths and tables without contents
    state = np.zeros((n_slots, 2), np.int32)
    table = np.full((n_slots, 6), -1, np.int32)
    state[src, 0], state[dst[:3000], 0] = [0, 63, 64, 200, 384], rs.randint(0, 385, 3000)
    state[:, 1] = rs.randint(0, 2, n_slots)
    pages = rs.permutation(20000)
    refs, at = np.zeros(20000, np.int32), 0
    for s in src + dst:
        nb = state[s, 0] // B
        table[s, :nb] = pages[at:at + nb]
        refs[pages[at:at + nb]] = 1
        at += nb
    free = np.zeros(20000, np.int32)
    free[:20000 - at] = pages[at:]
    for t, x in ((m.cache.state, state), (m.cache.table, table), (m.cache.refs, refs), (m.cache.free, free)):
        t.copy_(torch.from_numpy(x))
    m.cache.n_free.fill_(20000 - at)
    m.cache.tail.normal_()
    tail = m.cache.tail.clone()
    pick = [src[i] if i < 5 else -1 for i in rs.randint(0, 6, 4096)]
    want = plain_fork(m.cache, pick, dst)
    gdn.gdn_kv_fork_batch(m.desc, m.cache, m.i32(pick), m.i32(dst))
    same_books(m.cache, want)
    for s, t in zip(pick, dst):
        if s >= 0:
            o, b = state[s, 0] % B, state[s, 1]
            tail[t, b, :, :, :o] = tail[s, b, :, :, :o]
    assert torch.equal(tail, m.cache.tail)


def test_unsound_batches_change_nothing(cuda_device):
    m = Model((2, 1), 64, BF, n_slots=5, seed=3)
    m.step([0, 1], [130, 70], check=False)
    before = books(m.cache)
    for src, dst in (([0, 1], [2, 2]), ([0, 2], [2, 3]), ([0], [0]), ([5], [1]), ([-2], [1]), ([0], [5]), ([0], [-1])):
        gdn.gdn_kv_fork_batch(m.desc, m.cache, m.i32(src), m.i32(dst))
        assert gdn.gdn_device_status() == gdn.GDN_ERR_INVALID_ARG, (src, dst)
        for a, b in zip(books(m.cache), before):
            assert np.array_equal(a, b)
    gdn.gdn_kv_fork_batch(m.desc, m.cache, m.i32([]), m.i32([]))
    assert gdn.gdn_device_status() == gdn.GDN_OK
    m.check_contents()


# ---- compaction ----

def plain_compact(c, n_out):
    state, table, refs, free, n_free = books(c)
    used = np.flatnonzero(refs > 0)
    count = len(used)
    holes, movers = [p for p in range(count) if refs[p] == 0], [p for p in used if p >= count]
    now = dict(zip(movers, holes))
    for s in range(len(table)):
        for b in range(state[s, 0] // B):
            table[s, b] = now.get(table[s, b], table[s, b])
    out = np.zeros(n_out, np.int32)
    out[:count] = refs[:count]
    for a, b in now.items():
        out[b] = refs[a]
    return table, out, np.arange(n_out - 1, count - 1, -1), count, len(movers)


def scattered(m, seed):
    """Sessions of random lengths, some forked, some released, so that pages in use lie anywhere."""
    rs = np.random.RandomState(seed)
    n = len(m.slots)
    for _ in range(3):
        for s in range(n):
            if rs.uniform() < 0.5:
                m.step([s], [int(rs.randint(1, 150))], check=False)
        for s in range(n):
            if rs.uniform() < 0.3:
                fork_batch(m, [-1], [s])
        a, b = rs.choice(n, 2, replace=False).tolist()
        fork_batch(m, [a], [b])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("heads,d", [((2, 1), 64), ((6, 3), 128), ((2, 2), 256)])
def test_compaction_in_place(cuda_device, heads, d, dtype):
    m = Model(heads, d, dtype, n_pages=70, n_slots=6, max_blocks=16, seed=d)
    ws, counts = gdn.kv_compact_workspace(70, m.dev), torch.zeros(3, dtype=torch.int32, device=m.dev)
    for seed in range(3):
        scattered(m, seed)
        table, refs, free, used, moved = plain_compact(m.cache, 70)
        state = m.cache.state.clone()
        gdn.gdn_kv_compact(m.desc, m.cache, ws, counts)
        assert counts.tolist() == [used, 0, moved]
        assert np.array_equal(m.cache.table.cpu().numpy(), table) and np.array_equal(m.cache.refs.cpu().numpy(), refs)
        assert int(m.cache.n_free) == 70 - used and np.array_equal(m.cache.free[:70 - used].cpu().numpy(), free)
        assert torch.equal(state, m.cache.state)
        m.check_contents()
        m.step([0, 1, 2], [1, 65, 3])
        gdn.gdn_kv_compact(m.desc, m.cache, ws, counts)
        gdn.gdn_kv_compact(m.desc, m.cache, ws, counts)      # nothing left to move
        assert counts[2] == 0
        m.check_contents()


def test_a_pool_is_cut_and_grown(cuda_device):
    """Books elsewhere for a pool of as many pages as are in use, of fewer (refused), and of more."""
    m = Model((4, 2), 128, BF, n_pages=60, n_slots=6, max_blocks=16, seed=4)
    scattered(m, 7)
    used = int((m.cache.refs > 0).sum())
    c, i32 = m.cache, lambda *s: torch.full(s, -1, dtype=torch.int32, device=m.dev)   # noqa: E731
    ws, counts = gdn.kv_compact_workspace(60, m.dev), i32(3)
    before = books(c)
    pages = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    outs = i32(6, 16), i32(used - 1), i32(used - 1), i32(1)
    gdn.gdn_kv_compact(m.desc, c, ws, counts, *outs)
    assert counts.tolist() == [used, 1, 0] and all((t == -1).all() for t in outs)
    for a, b in zip(books(c), before):
        assert np.array_equal(a, b)
    assert all(torch.equal(a, b) for a, b in zip(pages, (c.k, c.v, c.k_scale, c.v_scale)))

    table, refs, free, _, moved = plain_compact(c, used)
    outs = i32(6, 16), i32(used), i32(used), i32(1)
    gdn.gdn_kv_compact(m.desc, c, ws, counts, *outs)
    assert counts.tolist() == [used, 0, moved]
    valid = np.arange(16) < (before[0][:, :1] // B)
    assert np.array_equal(outs[0].cpu().numpy()[valid], table[valid]) and (outs[0].cpu().numpy()[~valid] == -1).all()
    assert np.array_equal(outs[1].cpu().numpy(), refs) and int(outs[3]) == 0
    for a, b in zip(books(c), before):
        assert np.array_equal(a, b)                              # the old books are as they were

    # a pool of those pages alone
    cut = gdn.KvCache(m.desc, used, 6, 16, m.dev, k=c.k[:used].clone(), v=c.v[:used].clone(), k_scale=c.k_scale[:used].clone(),
                      v_scale=c.v_scale[:used].clone(), tail=c.tail, state=c.state, table=outs[0], refs=outs[1], free=outs[2],
                      n_free=outs[3])
    m.cache = cut
    m.check_contents()
    # grown again: room in the buffers, then the books
    grow = lambda t, n: torch.cat([t, torch.zeros((n - len(t), *t.shape[1:]), dtype=t.dtype, device=m.dev)])   # noqa: E731
    big = [grow(t, used + 20) for t in (cut.k, cut.v, cut.k_scale, cut.v_scale)]
    view = gdn.KvCache(m.desc, used, 6, 16, m.dev, k=big[0][:used], v=big[1][:used], k_scale=big[2][:used], v_scale=big[3][:used],
                       tail=cut.tail, state=cut.state, table=cut.table, refs=cut.refs, free=cut.free, n_free=cut.n_free)
    refs, free = i32(used + 20), i32(used + 20)
    gdn.gdn_kv_compact(m.desc, view, ws, counts, refs_out=refs, free_out=free)
    assert counts.tolist() == [used, 0, 0] and int(cut.n_free) == 20
    m.cache = gdn.KvCache(m.desc, used + 20, 6, 16, m.dev, k=big[0], v=big[1], k_scale=big[2], v_scale=big[3], tail=cut.tail,
                          state=cut.state, table=cut.table, refs=refs, free=free, n_free=cut.n_free)
    m.check_contents()
    m.step([0, 1], [100, 64])
    m.check_contents()


@pytest.mark.parametrize("pages,share", [(1, 1.0), (1, 0.0), (5000, 0.0), (5000, 1.0), (9001, 0.5), (40000, 0.3)])
def test_pools_of_every_size(cuda_device, pages, share):
    """Random counts, down to none and up to all pages in use; a slot per page."""
    rs = np.random.RandomState(pages)
    used = rs.permutation(pages)[:int(share * pages)]
    m = Model((1, 1), 64, BF, n_pages=pages, n_slots=max(len(used), 1), max_blocks=1, seed=1)
    c = m.cache
    refs = np.zeros(pages, np.int32)
    refs[used] = 1
    free = np.zeros(pages, np.int32)
    free[:pages - len(used)] = np.flatnonzero(refs == 0)
    c.refs.copy_(torch.from_numpy(refs))
    c.free.copy_(torch.from_numpy(free))
    c.n_free.fill_(pages - len(used))
    if len(used):
        c.state[:, 0] = 64
        c.table[:, 0] = torch.from_numpy(used.astype(np.int32)).to(m.dev)
    for t in (c.k, c.v):
        t.copy_(torch.randint(-127, 128, t.shape, device=m.dev, dtype=torch.int8))
    for t in (c.k_scale, c.v_scale):
        t.uniform_()
    held = lambda: [t[c.table[:len(used), 0].long()].clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]   # noqa: E731
    before = held()
    table, want, stack, count, moved = plain_compact(c, pages)
    counts = torch.zeros(3, dtype=torch.int32, device=m.dev)
    graph = torch.cuda.CUDAGraph()
    ws = gdn.kv_compact_workspace(pages, m.dev)
    with torch.cuda.graph(graph):
        gdn.gdn_kv_compact(m.desc, c, ws, counts)
    graph.replay()
    assert counts.tolist() == [count, 0, moved]
    assert np.array_equal(c.refs.cpu().numpy(), want) and np.array_equal(c.free[:pages - count].cpu().numpy(), stack)
    assert np.array_equal(c.table.cpu().numpy()[:len(used)], table[:len(used)])
    assert all(torch.equal(a, b) for a, b in zip(before, held()))


def test_pages_past_four_gigabytes(cuda_device):
    """Byte offsets beyond 32 bits: the last pages of a pool of 5 GB move to its first."""
    pages = 40000                                             # 4 heads of 256: 64 KB of keys a page
    m = Model((4, 4), 256, BF, n_pages=pages, n_slots=2, max_blocks=2, seed=1)
    c = m.cache
    a, b = pages - 1, pages - 5
    c.refs[[a, b]] = 1
    c.state[0, 0], c.state[1, 0] = 64, 64
    c.table[0, 0], c.table[1, 0] = a, b
    for t in (c.k, c.v):
        for p in (a, b):
            t[p].copy_(torch.randint(-127, 128, t.shape[1:], device=m.dev, dtype=torch.int8))
    want = [(c.k[p].clone(), c.v[p].clone()) for p in (b, a)]
    counts = torch.zeros(3, dtype=torch.int32, device=m.dev)
    gdn.gdn_kv_compact(m.desc, c, gdn.kv_compact_workspace(pages, m.dev), counts)
    assert counts.tolist() == [2, 0, 2] and c.table[:, 0].tolist() == [1, 0]
    for p, (k, v) in enumerate(want):
        assert torch.equal(c.k[p], k) and torch.equal(c.v[p], v)
