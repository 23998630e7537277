"""A hybrid block (one Gated-DeltaNet layer, one full-attention layer) that serves a conversation: two turns of prompt, a
fork into branches, and single tokens for all branches from one CUDA graph.

Per session the GDN layer keeps its state (S, conv) and the attention layer its keys and values, in 8-bit pages of 64
tokens that branches share: they are forked in one call, and their tokens attend to the shared pages together. Queries
and keys are normalised and rotated in half of each head on their way out of the q/k/v product. Weights and inputs are
random: the layers' outputs stand in for token embeddings.

    python examples/hybrid_session.py [--turn 2048] [--branches 8] [--steps 64]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from chunked_gated_deltanet_gb300 import gdn   # noqa: E402

HIDDEN, GRID = 1024, 64
BF = torch.bfloat16


class HybridBlock:
    """x + gdn(norm(x)), then x + attention(norm(x)), for the sessions of one cache."""

    def __init__(self, n_sessions: int, max_tokens: int, max_len: int, device="cuda", seed=0):
        self.dev, self.max_len = torch.device(device), max_len
        self.gd = gdn.make_desc(4, 8, 128, 128, GRID, gdn.GDN_BF16, gdn.GDN_BF16)
        self.ad = gdn.make_attn_desc(8, 2, 128, gdn.GDN_BF16)
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *s, scale: (torch.randn(s, generator=gen) * scale).to(self.dev)   # noqa: E731
        c, hv = gdn.channels(self.gd), self.gd.n_v_heads
        self.w_conv_in = rand(HIDDEN, c, scale=HIDDEN ** -0.5).to(BF)
        self.w_gate_in = rand(HIDDEN, 2 * hv, scale=HIDDEN ** -0.5).to(BF)
        self.conv_w = rand(c, 4, scale=0.5).to(BF)
        self.A_log, self.dt_bias = rand(hv, scale=0.2), rand(hv, scale=0.2)
        self.w_gdn_out = rand(hv * 128, HIDDEN, scale=HIDDEN ** -0.5).to(BF)
        self.w_qkv = rand(HIDDEN, (8 + 2 * 2) * 128, scale=HIDDEN ** -0.5).to(BF)
        self.q_norm, self.k_norm = (1 + rand(128, scale=0.1)).to(BF), (1 + rand(128, scale=0.1)).to(BF)
        self.rope = gdn.make_rope_desc(64, gdn.GDN_ROPE_HALF, 1e6)
        self.rope_table = gdn.rope_table(self.rope, self.dev)
        self.w_attn_out = rand(8 * 128, HIDDEN, scale=HIDDEN ** -0.5).to(BF)
        # what the sessions hold, and the scratch of a call
        self.states = [gdn.Session(self.gd, self.dev) for _ in range(n_sessions)]
        blocks = -(-max_len // gdn.GDN_KV_BLOCK)
        self.cache = gdn.KvCache(self.ad, n_sessions * blocks, n_sessions, blocks, self.dev)
        self.plan = gdn.KvPlan.new(max_tokens, n_sessions, self.dev)
        self.gdn_ws = gdn.workspace(self.gd, max_tokens, 1, self.dev)
        self.attn_ws = gdn.kv_attention_workspace(self.ad, max_tokens, n_sessions, max_len, self.dev)
        self.groups = gdn.KvGroups.new(self.plan, 1)
        self.shared_ws = gdn.kv_shared_workspace(self.ad, n_sessions, max_len, max_len, self.dev)

    def _gdn_inputs(self, x):
        n, hk, hv = x.shape[0], self.gd.n_qk_heads * 128, self.gd.n_v_heads
        x = torch.nn.functional.rms_norm(x, (HIDDEN,))
        q, k, v = (t.contiguous() for t in (x @ self.w_conv_in).split([hk, hk, hv * 128], 1))
        a, b = (t.contiguous() for t in (x @ self.w_gate_in).float().split([hv, hv], 1))
        gdn.gdn_gates(self.gd, a, b, self.A_log, self.dt_bias, a, b)
        return q, k, v, a, b, torch.empty((n, hv, 128), dtype=BF, device=self.dev)

    def _attention(self, x, slots, counts, max_new, family=None):
        """slots, counts: int32 on the GPU; x in their order. family: [0, n] on the GPU where all requests are forks of one
        session. One plan, with its positions and groups, serves every attention layer of a model."""
        n = x.shape[0]
        gdn.gdn_kv_plan(self.ad, self.cache, slots, counts, self.plan)
        pos = torch.empty(n, dtype=torch.int32, device=self.dev)
        gdn.gdn_kv_positions(self.plan, pos)
        qkv = (torch.nn.functional.rms_norm(x, (HIDDEN,)) @ self.w_qkv).view(n, 12, 128).split([8, 2, 2], 1)
        q, k, v = (torch.empty((n, h, 128), dtype=BF, device=self.dev) for h in (8, 2, 2))
        gdn.gdn_rope(self.ad, self.rope, self.rope_table, pos, qkv[0], qkv[1], q, k, qkv[2], v, self.q_norm, self.k_norm)
        gdn.gdn_kv_append(self.ad, self.cache, self.plan, k, v)
        out = torch.empty_like(q)
        if family is None:
            gdn.gdn_kv_attention(self.ad, self.cache, self.plan, q, k, v, out, self.attn_ws, max_new, self.max_len)
        else:
            gdn.gdn_kv_group(self.ad, self.cache, self.plan, family, self.groups)
            gdn.gdn_kv_attention_shared(self.ad, self.cache, self.plan, self.groups, q, k, v, out, self.shared_ws, max_new,
                                        self.max_len, self.max_len)
        return x + out.reshape(n, -1) @ self.w_attn_out

    def prompt(self, session: int, x):
        """One session's next tokens, a multiple of the GDN layer's chunk grid."""
        q, k, v, g, beta, out = self._gdn_inputs(x)
        if gdn.gdn_prefill_chunks(self.gd, self.states[session], q, k, v, g, beta, self.conv_w, out, self.gdn_ws) != len(x):
            raise ValueError("a turn here is a multiple of the chunk grid")
        x = x + out.reshape(len(x), -1) @ self.w_gdn_out
        i32 = lambda v: torch.tensor([v], dtype=torch.int32, device=self.dev)   # noqa: E731
        return self._attention(x, i32(session), i32(len(x)), len(x))

    def fork(self, src: int, dst):
        """The sessions dst continue where src is: copies of the GDN state, and src's complete blocks by reference."""
        for s in dst:
            gdn.gdn_state_restore(self.gd, self.states[s], self.states[src])
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=self.dev)   # noqa: E731
        gdn.gdn_kv_fork_batch(self.ad, self.cache, i32([src] * len(dst)), i32(list(dst)))

    def token(self, sessions, slots, ones, x, family):
        """The next token of every session, all of them forks of one; captures in a CUDA graph."""
        q, k, v, g, beta, out = self._gdn_inputs(x)
        gdn.gdn_decode_step(self.gd, [self.states[s] for s in sessions], q, k, v, g, beta, self.conv_w, out)
        x = x + out.reshape(len(x), -1) @ self.w_gdn_out
        return self._attention(x, slots, ones, 1, family)


def run(turn=2048, branches=8, steps=64, device="cuda"):
    """Two identical families of branches, one advanced token by token and one by graph replays; returns the largest
    difference of their outputs and the microseconds per replay."""
    dev = torch.device(device)
    n = 2 * branches
    m = HybridBlock(n, max(turn, n), 2 * turn + steps + 8, dev)
    gen = torch.Generator().manual_seed(1)
    draw = lambda k: torch.randn((k, HIDDEN), generator=gen).to(BF).to(dev)   # noqa: E731
    for x in (draw(turn), draw(turn)):
        m.prompt(0, x)
    m.fork(0, range(1, n))
    if gdn.gdn_kv_status(m.plan) != gdn.GDN_OK:
        raise RuntimeError("the cache is too small")
    families = [list(range(branches)), list(range(branches, n))]
    slots = [torch.tensor(f, dtype=torch.int32, device=dev) for f in families]
    ones = torch.ones(branches, dtype=torch.int32, device=dev)
    family = torch.tensor([0, branches], dtype=torch.int32, device=dev)
    x0 = draw(branches)
    want, x = [], x0
    for _ in range(steps):
        x = m.token(families[0], slots[0], ones, x, family)
        want.append(x)
    buf = x0.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        buf.copy_(m.token(families[1], slots[1], ones, buf, family))
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    got = torch.empty((steps, *buf.shape), dtype=BF, device=dev)
    start.record()
    for i in range(steps):
        graph.replay()
        got[i].copy_(buf)
    end.record()
    torch.cuda.synchronize()
    if gdn.gdn_device_status() != gdn.GDN_OK:
        raise RuntimeError("a kernel reported an error")
    return float((torch.stack(want).float() - got.float()).abs().max()), start.elapsed_time(end) / steps * 1e3


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--turn", type=int, default=2048)
    p.add_argument("--branches", type=int, default=8)
    p.add_argument("--steps", type=int, default=64)
    args = p.parse_args()
    diff, us = run(args.turn, args.branches, args.steps)
    print(f"{args.branches} branches of a session of {2 * args.turn} tokens: {us:.1f} us per step of all branches; "
          f"replayed and eager steps differ by {diff:g}")
