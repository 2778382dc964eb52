"""Run one attention layer kind a few times on synthetic inputs (for profilers).

    python -m long_context_anchor_gb300.runcase KIND [--batch B] [--kv-len N]
        [--heads HQ HKV] [--head-dim D] [--topk K] [--reps R] [--pooled]
        [--block-size T] [--prefix P]

KIND: dense_decode, anchor_decode, anchor_decode_fused, reuse_decode, topk,
dense_prefill, anchor_prefill, reuse_prefill, or over a paged 4-bit cache of
the same shape qcache_dense, qcache_anchor, qcache_reuse, qcache_append and
qcache_read (rows of a sequence batch * kv_len long), qcache_plan (that many
new tokens), qcache_append_rope (as qcache_append, with queries, all rows turned),
qcache_prefix (the first P of each sequence's kv_len tokens are shared); or
qk_rope (queries and keys of a prompt, normalised and turned). Defaults are the Llama-3.1-8B attention shape
with batch 2 (decode: about 0.5 GB of K/V per layer, larger than L2), so a
profiler capture of one launch stays small. Inputs are drawn once; every
repetition runs the same launch sequence. --pooled uses one index set per KV
head (anchor and reuse kinds).
"""
import argparse

import torch

from . import kascade as K


def cache_case(a, dev):
    """A step's call over a paged 4-bit cache that the planner laid out, as a function."""
    g = torch.Generator(device=dev).manual_seed(7)
    B, N, (Hq, Hkv), d, bs = a.batch, a.kv_len, a.heads, a.head_dim, a.block_size
    blocks = (N + bs - 1) // bs
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    shared = a.prefix // bs if a.kind == "qcache_prefix" else 0    # blocks, the order's last ones
    P = shared * bs
    lens, new = i32(*[P] * B), i32(*[N - P] * B)
    order = torch.randperm(shared + B * (blocks - shared), generator=g, device=dev).to(torch.int32)
    count = i32(B * (blocks - shared))
    front = order[B * (blocks - shared):]
    table = torch.zeros(B, blocks, dtype=torch.int32, device=dev)
    table[:, :shared] = front
    ws = K.Workspace(dev)
    plan = lambda: K.qcache_plan(lens, new, table, order.clone(), count, bs, B * (N - P), ws=ws)
    if a.kind == "qcache_plan":
        return plan, ws
    slots, _, lens, _ = plan()
    at = torch.arange(bs, dtype=torch.int32, device=dev)
    slots = torch.cat([(front[:, None] * bs + at).reshape(-1), slots])
    pages = K.qcache_alloc(order.numel(), Hkv, d, bs, dev)
    q = torch.randn(B, Hq, d, generator=g, device=dev).to(torch.bfloat16)
    k, v = (torch.randn(len(slots), Hkv, d, generator=g, device=dev).to(torch.bfloat16)
            for _ in range(2))
    append = lambda: K.qcache_append(k, v, slots, pages, ws=ws)
    append()
    common = dict(kv_len=N, ws=ws)
    k_top = a.topk or max(1, N // 8)
    calls = {
        "qcache_append": append,
        "qcache_read": lambda: K.qcache_read(pages, slots, k=k, v=v, ws=ws),
        "qcache_prefix": lambda: K.qcache_prefix_decode(q, pages, table, lens, P, **common),
        "qcache_dense": lambda: K.qcache_dense_decode(q, pages, table, lens, **common),
        "qcache_anchor": lambda: K.qcache_anchor_decode(q, pages, table, lens, k_top,
                                                        pooled=a.pooled, **common),
    }
    if a.kind == "qcache_append_rope":
        rope = rotation(N, d, dev)
        qs = torch.randn(len(slots), Hq, d, generator=g, device=dev).to(torch.bfloat16)
        positions = torch.arange(N, dtype=torch.int32, device=dev).repeat(B)
        return lambda: K.qcache_append_rope(k, v, slots, pages, rope, positions, q=qs, ws=ws), ws
    if a.kind == "qcache_reuse":
        idx = K.qcache_anchor_decode(q, pages, table, lens, k_top, pooled=a.pooled, **common)[1]
        return lambda: K.qcache_reuse_decode(q, pages, table, lens, idx, pooled=a.pooled,
                                             **common), ws
    if a.kind not in calls:
        raise SystemExit("unknown kind " + a.kind)
    return calls[a.kind], ws


def rotation(n, d, dev):
    return K.rope_table(1e4 ** (-torch.arange(d // 2, dtype=torch.float64) * 2 / d), n, device=dev)


def rotation_case(a, dev):
    """A prompt's queries and keys, [B,H,N,d], as a function that normalises and turns them."""
    g = torch.Generator(device=dev).manual_seed(7)
    B, N, (Hq, Hkv), d = a.batch, a.kv_len, a.heads, a.head_dim
    q, k = (torch.randn(B, h, N, d, generator=g, device=dev).to(torch.bfloat16) for h in (Hq, Hkv))
    w = torch.ones(d, dtype=torch.bfloat16, device=dev)
    positions = torch.arange(N, dtype=torch.int32, device=dev).repeat(B, 1)
    rope, ws = rotation(N, d, dev), K.Workspace(dev)
    return lambda: K.qk_norm_rope(q, k, positions, rope, w, w, ws=ws), ws


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("kind")
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--kv-len", type=int, default=32768)
    ap.add_argument("--heads", type=int, nargs=2, default=(32, 8))
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--topk", type=int, default=0, help="default kv_len // 8")
    ap.add_argument("--reps", type=int, default=3)
    ap.add_argument("--pooled", action="store_true", help="one index set per KV head")
    ap.add_argument("--block-size", type=int, default=64, help="tokens per block of a paged cache")
    ap.add_argument("--prefix", type=int, default=0, help="tokens that the sequences share")
    a = ap.parse_args()
    dev = torch.device("cuda", 0)
    if a.kind.startswith("qcache_") or a.kind == "qk_rope":
        call, ws = (rotation_case if a.kind == "qk_rope" else cache_case)(a, dev)
        torch.cuda.synchronize()
        for _ in range(a.reps):
            call()
        finish(a, ws)
        return
    g = torch.Generator(device=dev).manual_seed(7)
    B, N, (Hq, Hkv), d = a.batch, a.kv_len, a.heads, a.head_dim
    k_top = a.topk or max(1, N // 8)
    bf = torch.bfloat16
    if "decode" in a.kind or a.kind == "topk":
        q = torch.randn(B, Hq, d, generator=g, device=dev).to(bf)
    else:
        q = torch.randn(B, Hq, N, d, generator=g, device=dev).to(bf)
    k = torch.randn(B, Hkv, N, d, generator=g, device=dev).to(bf)
    v = torch.randn(B, Hkv, N, d, generator=g, device=dev).to(bf)
    ws = K.Workspace(dev)
    idx = None
    pl = a.pooled
    if a.kind == "reuse_decode":
        _, idx = K.anchor_decode(q, k, v, k_top, ws=ws, pooled=pl)
    if a.kind == "reuse_prefill":
        _, idx = K.anchor_prefill(q, k, v, k_top, ws=ws, pooled=pl)
    scores = None
    if a.kind == "topk":
        scores = torch.randn(B * Hq, N, generator=g, device=dev)
    torch.cuda.synchronize()
    for _ in range(a.reps):
        if a.kind == "dense_decode":
            K.dense_decode(q, k, v, ws=ws)
        elif a.kind == "anchor_decode":
            K.anchor_decode(q, k, v, k_top, ws=ws, pooled=pl)
        elif a.kind == "anchor_decode_fused":
            K.anchor_decode(q, k, v, k_top, ws=ws, fused=True)
        elif a.kind == "reuse_decode":
            K.reuse_decode(q, k, v, idx, ws=ws, pooled=pl)
        elif a.kind == "topk":
            K.topk(scores, k_top, ws=ws)
        elif a.kind == "dense_prefill":
            K.dense_prefill(q, k, v, ws=ws)
        elif a.kind == "anchor_prefill":
            K.anchor_prefill(q, k, v, k_top, ws=ws, pooled=pl)
        elif a.kind == "reuse_prefill":
            K.reuse_prefill(q, k, v, idx, ws=ws, pooled=pl)
        else:
            raise SystemExit("unknown kind " + a.kind)
    finish(a, ws)


def finish(a, ws):
    torch.cuda.synchronize()
    err = ws.device_error()
    if err != K.OK:
        raise SystemExit("device error: " + K.status_string(err))
    print("ok", a.kind)


if __name__ == "__main__":
    main()
