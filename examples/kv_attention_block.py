"""The attention block of a generator on coded weights and a 4-bit cache.

q, k, v and o are 4-bit entropy-coded matrices decoded inside their products;
the tokens' keys and values go to a 4-bit paged cache as they are made, and
attention reads them there.  Several sequences of different prompt lengths are
fed, then each generates tokens, one a step: the step's four calls (the grouped
q, k, v product, the cache write, attention, the o product) are captured once
and replayed.

    python examples/kv_attention_block.py [--steps 16] [--prompts 37 5 120 200]

Prints the error of the last step against a plain computation in 64 bits on the
cached values, the cache's bytes against bf16, and the time of a step.
"""
import argparse
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from decode_gemv_gb300 import inputs, lw  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, PAGE = 1024, 8, 2, 128, 64


class Block:
    """Coded projections, a cache with room for `room` tokens a sequence, and the buffers of a
    step of `batch` sequences."""

    def __init__(self, batch, room, device="cuda", seed=7):
        import torch
        self.torch, self.device, self.batch = torch, device, batch
        rows = {"q": Q_HEADS * DIM, "k": KV_HEADS * DIM, "v": KV_HEADS * DIM, "o": HIDDEN}
        self.weights, self.db = {}, {}
        for i, (name, n) in enumerate(rows.items()):
            k = Q_HEADS * DIM if name == "o" else HIDDEN
            m = inputs.small_q4(seed + i, n, k)
            self.weights[name] = m
            hb = lw.lw_encode_bundle(lw.LW_FMT_Q4_PAIR, m["codes"], m["scales"], m["mins"])
            self.db[name] = lw.DeviceBundle.upload(hb, device)
        pages = -(-room // PAGE)
        self.cache = lw.KvCache.empty(batch * pages, KV_HEADS, DIM, PAGE, device)
        # pages as a pool hands them out: in any order
        order = torch.randperm(batch * pages, generator=torch.Generator().manual_seed(seed))
        self.table = order.to(torch.int32).view(batch, pages).to(device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        qkv = [self.db[n] for n in "qkv"]
        self.group_ws = torch.zeros(lw.lw_workspace_bytes_group(qkv), dtype=torch.uint8, device=device)
        self.o_ws = torch.zeros(max(lw.lw_workspace_bytes(self.db["o"], b) for b in (batch, 256)),
                                dtype=torch.uint8, device=device)
        self.start = torch.arange(batch + 1, dtype=torch.int32, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.x = torch.zeros(batch, HIDDEN, **f32)
        self.q = torch.empty(batch, Q_HEADS, DIM, **f32)
        self.k = torch.empty(batch, KV_HEADS, DIM, **f32)
        self.v = torch.empty(batch, KV_HEADS, DIM, **f32)
        self.att = torch.empty_like(self.q)
        self.y = torch.empty(batch, HIDDEN, **f32)
        self.slots = torch.zeros(batch, dtype=torch.int64, device=device)
        need = lw.lw_kv_workspace_bytes(self.cache, Q_HEADS, max(batch, 256), batch)
        self.att_ws = torch.zeros(need, dtype=torch.uint8, device=device)

    def slots_of(self, b, positions):
        """Cache slots of a sequence's positions."""
        page = self.table[b][(positions // PAGE).long()].long()
        return page * PAGE + positions % PAGE

    def prompt(self, b, x):
        """Feed x [tokens, HIDDEN] to sequence b (256 tokens at a time); the block's outputs."""
        torch = self.torch
        outs = []
        for part in x.split(256):
            t = part.shape[0]
            part = part.contiguous()
            made = {}
            for name in "qkv":
                db = self.db[name]
                y = torch.empty(t, db.rows, dtype=torch.float32, device=self.device)
                ws = torch.zeros(lw.lw_workspace_bytes(db, t), dtype=torch.uint8, device=self.device)
                lw.lw_decode_gemm(db, part, t, y, ws, self.status)
                made[name] = y.view(t, -1, DIM)
            n = int(self.lens[b])
            slots = self.slots_of(b, torch.arange(n, n + t, device=self.device))
            lw.lw_kv_write(self.cache, made["k"], made["v"], slots, self.status)
            self.lens[b] += t
            att = torch.empty_like(made["q"])
            lw.lw_kv_attention(self.cache, made["q"], torch.tensor([0, t], dtype=torch.int32, device=self.device),
                               self.lens[b:b + 1], self.table[b:b + 1], att, self.att_ws, self.status, max_q=t)
            y = torch.empty(t, HIDDEN, dtype=torch.float32, device=self.device)
            lw.lw_decode_gemm(self.db["o"], att.view(t, -1), t, y, self.o_ws, self.status)
            outs.append(y)
        return torch.cat(outs)

    def step_calls(self):
        """One token of every sequence: x -> y through the cache (slots and lens hold the token's
        own place)."""
        qkv = [self.db[n] for n in "qkv"]
        lw.lw_decode_gemm_group(qkv, [self.x] * 3, self.batch, [self.q, self.k, self.v], self.group_ws,
                                self.status)
        lw.lw_kv_write(self.cache, self.k, self.v, self.slots, self.status)
        lw.lw_kv_attention(self.cache, self.q, self.start, self.lens, self.table, self.att, self.att_ws,
                           self.status, max_q=1)
        lw.lw_decode_gemm(self.db["o"], self.att.view(self.batch, -1), self.batch, self.y, self.o_ws, self.status)

    def capture(self):
        self.graph = lw.StepGraph(self.torch.cuda.Stream())
        with self.graph.capture():
            self.step_calls()

    def step(self, x):
        torch = self.torch
        self.x.copy_(x)
        for b in range(self.batch):
            self.slots[b] = self.slots_of(b, self.lens[b])
        self.lens += 1
        side = self.graph.stream
        side.wait_stream(torch.cuda.current_stream())
        self.graph.launch()
        torch.cuda.current_stream().wait_stream(side)
        return self.y


def weight(m):
    """A 4-bit matrix in 64 bits."""
    s = np.repeat(m["scales"].view(np.float16).astype(np.float64), 256, axis=1)
    z = np.repeat(m["mins"].view(np.float16).astype(np.float64), 256, axis=1)
    return s * m["codes"] + z


def check(block):
    """The last step's output against a plain computation on the cached values: the largest
    difference over the largest output."""
    torch = block.torch
    w = {n: weight(block.weights[n]) for n in "qo"}
    worst, top = 0.0, 0.0
    for b in range(block.batch):
        n = int(block.lens[b])
        slots = block.slots_of(b, torch.arange(n, device=block.device))
        k = torch.empty(n, KV_HEADS, DIM, device=block.device)
        v = torch.empty_like(k)
        lw.lw_kv_read(block.cache, slots, k, v, block.status)
        k, v = k.double().cpu().numpy(), v.double().cpu().numpy()
        q = (w["q"] @ block.x[b].double().cpu().numpy()).reshape(Q_HEADS, DIM)
        att = np.empty((Q_HEADS, DIM))
        for h in range(Q_HEADS):
            s = k[:, h // (Q_HEADS // KV_HEADS)] @ q[h] / np.sqrt(DIM)
            p = np.exp(s - s.max())
            att[h] = p @ v[:, h // (Q_HEADS // KV_HEADS)] / p.sum()
        want = w["o"] @ att.reshape(-1)
        got = block.y[b].double().cpu().numpy()
        worst, top = max(worst, np.abs(got - want).max()), max(top, np.abs(want).max())
    return worst / top


def main(prompts=(37, 5, 120, 200), steps=16, seed=7):
    import torch
    batch = len(prompts)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    block = Block(batch, max(prompts) + steps + 1)

    def norm(h):
        return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6)

    h = torch.empty(batch, HIDDEN, device="cuda")
    for b, t in enumerate(prompts):
        x = torch.randn(t, HIDDEN, device="cuda", generator=gen)
        h[b] = x[-1] + block.prompt(b, norm(x))[-1]
    block.capture()
    for i in range(steps):
        h = h + block.step(norm(h))
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    with torch.cuda.stream(block.graph.stream):   # the last step again: it writes what it wrote
        begin.record()
        for i in range(20):
            block.graph.launch()
        end.record()
    torch.cuda.synchronize()
    assert int(block.status) == 0, f"device status {int(block.status)}"
    err = check(block)
    tokens = int(block.lens.sum())
    kept = tokens * lw.lw_kv_tile_bytes(DIM) // lw.LW_KV_TILE * KV_HEADS
    return dict(error=err, tokens=tokens, cache_bytes=kept, bf16_bytes=tokens * KV_HEADS * DIM * 4,
                step_us=begin.elapsed_time(end) / 20 * 1e3)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--prompts", type=int, nargs="+", default=[37, 5, 120, 200])
    a = ap.parse_args()
    r = main(a.prompts, a.steps)
    print(f"{len(a.prompts)} sequences, {r['tokens']} cached tokens in {r['cache_bytes']} bytes "
          f"(bf16: {r['bf16_bytes']}), a step {r['step_us']:.1f} us, error {r['error']:.2e} of the largest output")
