"""A small hybrid's decode: GatedDeltaNet layers and softmax-attention layers in one transaction.

    python examples/hybrid_decode.py [--requests 4] [--prompt 300] [--steps 12] [--layers 3] [--attention 2]

Requests share a system prompt: its rows are turned to their positions, attended to in chunks and committed once, and
the other requests fork its pages.
Every step is one transaction of K-draft verification: the planner grants drafts, the GatedDeltaNet layers verify
into checkpoints, the attention layers read the paged 8-bit cache and the transaction's own rows, the drafts are
accepted greedily, and the commit moves both kinds of state by the accepted rows.  Halfway one request leaves and
the pool is compacted.  Projections are random draws (there is no trained model here): what is shown is the order of
the calls and what each of them owns.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gdnsynth as sy  # noqa: E402
from speculative_decoding_hybrid_gb300 import binding as gs  # noqa: E402
from speculative_decoding_hybrid_gb300.kvcache import PagedKv  # noqa: E402
from speculative_decoding_hybrid_gb300.prefill import Rope, attend_prompts  # noqa: E402
from speculative_decoding_hybrid_gb300.step import DecodeLoop, LayerRows, VerifyStep  # noqa: E402

VOCAB = 512


class HybridDecode:
    """GatedDeltaNet states, checkpoints and slots (VerifyStep, DecodeLoop) beside the attention layers' paged cache,
    for a fixed set of requests."""

    def __init__(self, requests, gdn_layers, attention_layers, max_tokens, h_q=8, h_kv=2, d=128, page_tokens=32,
                 k_max=3, device="cuda", seed=0):
        self.B, self.k_max, self.dev = requests, k_max, torch.device(device)
        self.gen = torch.Generator(device=self.dev).manual_seed(seed)
        self.gdn = gs.dims(2, 4, 64, 64)
        cap = requests * (k_max + 1)
        self.vs = VerifyStep(self.gdn, gdn_layers, requests, cap, requests, VOCAB, self.dev)
        slots = gs.Pool(requests)
        self.loop = DecodeLoop(self.vs, [slots.alloc() for _ in range(requests)], slots, k_max=k_max)
        pages = requests * (-(-max_tokens // page_tokens) + 1)
        # one status word for both kinds of layer: a timed-out wait in either stops the commits of both
        self.kv = PagedKv(attention_layers, pages, requests, max_tokens, h_q, h_kv, d, page_tokens, device=self.dev,
                          status=self.vs.status)
        self.rope = Rope(d, d // 2, base=1e6, device=self.dev)
        self.drafted = self.accepted = 0

    def normal(self, *shape, scale=1.0):
        return (torch.randn(shape, generator=self.gen, device=self.dev) * scale).to(torch.bfloat16)

    def attention_rows(self, n):
        """One fused projection (queries, keys, values side by side), split into views."""
        kv = self.kv
        qkv = self.normal(n, (kv.h_q + 2 * kv.h_kv) * kv.d)
        q, k, v = qkv.split([kv.h_q * kv.d, kv.h_kv * kv.d, kv.h_kv * kv.d], 1)
        return q.unflatten(1, (kv.h_q, kv.d)), k.unflatten(1, (kv.h_kv, kv.d)), v.unflatten(1, (kv.h_kv, kv.d))

    def rotate(self, q, k, cu, length):
        """Queries and keys turned to their positions, in place in the projection's rows."""
        return self.rope.rotate(q, k, cu, length, self.kv.status, in_place=True)

    def prefill(self, request, tokens, chunk=256):
        """A prompt through every attention layer, `chunk` rows a transaction: the first ones attend to their own rows,
        later ones to the cache and their own.  -> per chunk a list of the layers' (q, k, v, o)."""
        kv, seen = self.kv, []
        for at in range(0, tokens, chunk):
            n, held = min(chunk, tokens - at), int(self.kv.length[request])
            kv.reserve([request], [n])
            table, length = kv.upload([request])
            cu = torch.tensor([0, n], dtype=torch.int32, device=self.dev)
            rows = []
            for layer in range(kv.kv.shape[1]):
                q, k, v = self.attention_rows(n)
                self.rotate(q, k, cu, length)
                if held == 0:
                    o, _ = attend_prompts(q, k, v, cu, n, kv.status)
                else:
                    o, _ = kv.attend_chunk(layer, table, length, cu, q, k, v, max_len=held, max_rows=n, total_len=held)
                kv.append(layer, table, length, cu, k, v, max_rows=n)
                rows.append((q, k, v, o))
            kv.advance([request], [n])
            seen.append(rows)
        return seen

    def prompt(self, request, tokens, chunk=256):
        """prefill; -> per attention layer the keys and values that were committed."""
        seen = self.prefill(request, tokens, chunk)
        return [tuple(torch.cat([rows[layer][i] for rows in seen]) for i in (1, 2))
                for layer in range(self.kv.kv.shape[1])]

    def step(self, drafts):
        """One transaction; -> per attention layer (q, k, v, o), and the accept lengths."""
        loop, vs, kv, live = self.loop, self.vs, self.kv, list(range(self.B))
        plan = loop.plan_step(drafts)
        cu = plan.dec_cu
        n = [cu[i + 1] - cu[i] for i in live]
        kv.reserve(live, n)                             # room for every draft; shared pages are copied
        loop.upload_tables()
        table, length = kv.upload(live)
        vs.txn = (vs.txn + 1) & 0xFFFFFFFF
        rows = cu[-1]
        for layer in range(vs.L):
            x = sy.rows(self.gen, rows, sy.Dims(2, 4, 64, 64), device=self.dev)
            vs.verify_layer(layer, self.B, loop.cu_rows, loop.src_slot, LayerRows(x.q, x.k, x.v, x.g, x.beta))
        seen = []
        for layer in range(kv.kv.shape[1]):
            q, k, v = self.attention_rows(rows)
            self.rotate(q, k, loop.cu_rows, length)
            o, _ = kv.attend(layer, table, length, loop.cu_rows, q, k, v, max_len=kv.max_len, max_rows=max(n))
            seen.append((q, k, v, o))
        logits = self.normal(vs.cap, VOCAB, scale=2.0)
        tokens = logits.argmax(1).to(torch.int32).roll(1)  # drafts the target agrees with ...
        miss = torch.rand(vs.cap, generator=self.gen, device=self.dev) > 0.85
        tokens = torch.where(miss, (tokens + 1) % VOCAB, tokens)   # ... 85 times in 100
        vs.accept(self.B, loop.cu_rows, logits, tokens)
        vs.commit(self.B, loop.cu_rows, loop.dst_slot)
        for layer, (_, k, v, _) in enumerate(seen):
            kv.append(layer, table, length, loop.cu_rows, k, v, accept_len=vs.accept_len, max_rows=max(n))
        accept, _, _ = loop.readback()                  # the transaction's one wait
        if int(vs.status.item()):
            raise RuntimeError("device status %d" % int(vs.status.item()))
        loop.finish(accept)
        kv.advance(live, [int(accept[i]) + 1 for i in live])
        self.drafted += sum(n) - self.B
        self.accepted += int(accept[:self.B].sum())
        return seen, accept[:self.B].clone()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--layers", type=int, default=3)
    ap.add_argument("--attention", type=int, default=2)
    a = ap.parse_args(argv)
    h = HybridDecode(a.requests, a.layers, a.attention, a.prompt + 4 * a.steps + 64)
    h.prompt(0, a.prompt)
    for r in range(1, a.requests):
        h.kv.fork(0, r)                                 # whole pages shared, the unfinished last one copied
    shared = h.kv.pool.c.num_slots - h.kv.pool.c.free_count
    for step in range(a.steps):
        h.step([h.k_max] * a.requests)
        if step == a.steps // 2 and a.requests > 1:
            last = a.requests - 1
            keep = int(h.kv.length[last])
            h.kv.free(last)                             # a request leaves, another forks in: holes in the pool
            h.kv.fork(0, last, min(keep, int(h.kv.length[0])))
            print("step %d: %d pages moved by compaction" % (step, h.kv.compact()))
    used = h.kv.pool.c.num_slots - h.kv.pool.c.free_count
    print("%d requests, prompt of %d tokens in %d pages; after %d transactions %s tokens in %d pages; %d of %d drafts "
          "accepted" % (a.requests, a.prompt, shared, a.steps, h.kv.length.tolist(), used, h.accepted, h.drafted))
    return h


if __name__ == "__main__":
    main()
