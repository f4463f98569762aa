"""Run one library call on a full-size workload matrix, or on a cache, a few
times, for profiler captures of a single kernel (e.g. ``ncu -k regex:q_lut -s 2 -c 1``):

    python -m decode_gemv_gb300.kernel_targets <target> [--reps N]

Targets (matrices from the seeded workload generators, encoded on the host,
uploaded once; every call on the same device buffers):

  gate_q4            lw_decode_gemv, Mistral-7B-shaped gate 14336x4096, 4-bit coded
  gate_q4_twin       lw_twin_gemv on the same matrix's fixed-width twin
  gate_q4_b16        lw_decode_gemm, batch 16 (tensor-core route)
  gate_q4_b32        lw_decode_gemm, batch 32
  gate_q4_decode     lw_decode (decode only) of the 4-bit gate
  llama_gate_bf16    lw_decode_gemv, Llama-3.1-8B MLP gate, BF16 exponent coding
  llama_gate_bf16_b16      lw_decode_gemm of the same, batch 16 (tensor cores)
  llama_gate_bf16_b64      lw_decode_gemm of the same, batch 64 (tensor cores)
  llama_gate_bf16_decode   lw_decode of the same
  kv_write           lw_kv_write, 65536 tokens of 8 heads of 128, bf16
  kv_decode          lw_kv_attention, 8 sequences of 16384 keys, 32 query heads on 8 of 128, bf16
  kv_chunk           lw_kv_attention, a chunk of 2048 tokens on 16384 keys, the same heads
  kv_window          lw_kv_attention, 5 prompts of 2048, fp16, 16 heads on 2 of 64, window 1024
  kv_rotary          lw_kv_write_rotary, 32768 tokens of 32 query and 8 key/value heads of 128, bf16
  kv_weigh           lw_kv_weigh, one token of 8 sequences of 16384 keys, the heads of kv_decode
  kv_weigh_chunk     lw_kv_weigh, a chunk of 1024 tokens on 8192 keys, the same heads
  kv_evict           lw_kv_evict, 8 sequences of 16384 keys cut to 4096, in place
  kv_blocks          lw_kv_summarise of 8 sequences of 16384 keys, lw_kv_attention_blocks, 32 pages of 64

Exits nonzero if a call reports a device status."""
import argparse
import sys

import torch

from decode_gemv_gb300 import inputs, lw

TARGETS = ("gate_q4", "gate_q4_twin", "gate_q4_b16", "gate_q4_b32", "gate_q4_decode",
           "llama_gate_bf16", "llama_gate_bf16_b16", "llama_gate_bf16_b64", "llama_gate_bf16_decode",
           "kv_write", "kv_decode", "kv_chunk", "kv_window", "kv_rotary", "kv_weigh", "kv_weigh_chunk",
           "kv_evict", "kv_blocks")
# query tokens, keys, sequences, query heads, key/value heads, head_dim, page, type, window
KV_CALLS = {"kv_decode": (1, 16384, 8, 32, 8, 128, 64, torch.bfloat16, 0),
            "kv_chunk": (2048, 16384, 1, 32, 8, 128, 64, torch.bfloat16, 0),
            "kv_window": (2048, 2048, 5, 16, 2, 64, 32, torch.float16, 1024),
            "kv_weigh": (1, 16384, 8, 32, 8, 128, 64, torch.bfloat16, 0),
            "kv_weigh_chunk": (1024, 8192, 1, 32, 8, 128, 64, torch.bfloat16, 0),
            "kv_evict": (1, 16384, 8, 32, 8, 128, 64, torch.bfloat16, 0),
            "kv_blocks": (1, 16384, 8, 32, 8, 128, 64, torch.bfloat16, 0)}


def kv_target(t, reps, dev, st):
    gen = torch.Generator(device=dev).manual_seed(1)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, device=dev, generator=gen).to(dtype)

    if t == "kv_write":
        cache = lw.KvCache.empty(1024, 8, 128, 64, dev)
        k, v, slots = randn(65536, 8, 128), randn(65536, 8, 128), torch.arange(65536, device=dev)
        for _ in range(reps):
            lw.lw_kv_write(cache, k, v, slots, st)
        return
    if t == "kv_rotary":
        cache = lw.KvCache.empty(512, 8, 128, 64, dev)
        q, k, v, slots = randn(32768, 32, 128), randn(32768, 8, 128), randn(32768, 8, 128), torch.arange(32768, device=dev)
        table = torch.empty(32768, 128, device=dev)
        lw.lw_rotary_table(table)
        for _ in range(reps):
            lw.lw_kv_write_rotary(cache, k, v, slots, slots, table, st, q=q, q_out=q)
        return
    T, n, batch, hq, hk, dim, page, dtype, window = KV_CALLS[t]
    width = -(-n // page)
    cache = lw.KvCache.empty(batch * width, hk, dim, page, dev)
    table = torch.randperm(batch * width, device=dev, generator=gen).to(torch.int32).view(batch, width)
    for p in range(0, batch * width * page, 4096):
        slots = torch.arange(p, min(p + 4096, batch * width * page), device=dev)
        lw.lw_kv_write(cache, randn(len(slots), hk, dim), randn(len(slots), hk, dim), slots, st)
    q = randn(batch * T, hq, dim, dtype=dtype)
    out = torch.empty_like(q)
    start = torch.arange(batch + 1, device=dev, dtype=torch.int32) * T
    lens = torch.full((batch,), n, dtype=torch.int32, device=dev)
    if t.startswith("kv_weigh"):
        lse, w = torch.full((batch * T, hq), 10.0, device=dev), torch.zeros(batch, hk, n, device=dev)
        ws = torch.empty(max(lw.lw_kv_weigh_workspace_bytes(cache, hq, batch * T), 1), dtype=torch.uint8, device=dev)
        for _ in range(reps):
            lw.lw_kv_weigh(cache, q, lse, start, lens, table, w, ws, st, max_q=T, add_to=w)
        return
    if t == "kv_evict":
        w, kept = torch.rand(batch, hk, n, device=dev, generator=gen) ** 8, torch.empty(batch, hk, 4096, dtype=torch.int32, device=dev)
        for _ in range(reps):
            lw.lw_kv_evict(cache, w, lens, table, table, torch.empty_like(lens), None, kept, st, keep=4096, first=4, recent=512)
        return
    if t == "kv_blocks":
        summary = torch.empty(lw.lw_kv_summary_bytes(cache), dtype=torch.uint8, device=dev)
        ws = torch.zeros(lw.lw_kv_blocks_workspace_bytes(cache, hq, batch, width, 32), dtype=torch.uint8, device=dev)
        for _ in range(reps):
            lw.lw_kv_summarise(cache, summary, torch.zeros_like(lens), lens, table, st)
            lw.lw_kv_attention_blocks(cache, summary, q, start, lens, table, out, ws, st, blocks=32, first=1, recent=2)
        return
    ws = torch.zeros(lw.lw_kv_workspace_bytes(cache, hq, batch * T, batch), dtype=torch.uint8, device=dev)
    for _ in range(reps):
        lw.lw_kv_attention(cache, q, start, lens, table, out, ws, st, max_q=T, window=window)


def main(argv=None) -> int:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("target", choices=TARGETS)
    p.add_argument("--reps", type=int, default=3)
    args = p.parse_args(argv)
    lw.load()
    dev = "cuda"
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    t = args.target
    if t.startswith("kv_"):
        kv_target(t, args.reps, dev, st)
        return finish(t, args.reps, st)
    if t.startswith("gate_q4"):
        spec = inputs.workload_specs(inputs.MISTRAL_LAYER)[4]
        batch = 16 if t.endswith("b16") else 32 if t.endswith("b32") else 1
        m = inputs.make_matrix(inputs.MISTRAL_LAYER, spec, 0, 4, batch=batch)
        hb = lw.lw_encode_bundle(lw.LW_FMT_Q4_PAIR, m["codes"], m["scales"], m["mins"],
                                 twin=t.endswith("twin"))
        X = torch.from_numpy(m["x"]).to(dev)
    else:
        spec = inputs.workload_specs(inputs.LLAMA_MLP_BF16)[0]
        batch = 16 if t.endswith("b16") else 64 if t.endswith("b64") else 1
        m = inputs.make_matrix(inputs.LLAMA_MLP_BF16, spec, 0, 0, batch=batch)
        hb = lw.lw_encode_bundle(lw.LW_FMT_BF16_EXP, m["bits"], None, None)
        X = torch.from_numpy(m["x"].view("int16")).to(dev).reshape(batch, -1)
    db = lw.DeviceBundle.upload(hb, dev)
    if t.endswith("decode"):
        if db.fmt == lw.LW_FMT_Q4_PAIR:
            out = torch.zeros(spec.rows * spec.cols // 2, dtype=torch.uint8, device=dev)
        else:
            out = torch.zeros(spec.rows * spec.cols, dtype=torch.int16, device=dev)
        for _ in range(args.reps):
            lw.lw_decode(db, out, st)
    else:
        Y = torch.empty((batch, spec.rows), dtype=torch.float32, device=dev)
        ws = torch.zeros(lw.lw_workspace_bytes(db, batch) // 4 + 64, dtype=torch.float32, device=dev)
        for _ in range(args.reps):
            if t.endswith("twin"):
                lw.lw_twin_gemv(db, X[0], Y[0], ws, st)
            elif batch == 1:
                lw.lw_decode_gemv(db, X[0], Y[0], ws, st)
            else:
                lw.lw_decode_gemm(db, X, batch, Y, ws, st)
    return finish(t, args.reps, st)


def finish(t, reps, st) -> int:
    torch.cuda.synchronize()
    code = int(st.item())
    print(f"{t}: {reps} calls, device status {code}")
    return 1 if code else 0


if __name__ == "__main__":
    sys.exit(main())
