"""Single-kernel cases for profiler captures: one warm-up launch, then `--reps` launches of
one hot-path kernel at a workload's shape, inputs larger than L2 and a few GB at most.

    python -m bit_compressed_throughput_gb300.profile_cases gemm-fc1-opt67b
    python -m bit_compressed_throughput_gb300.profile_cases decode-attn-opt67b
    python -m bit_compressed_throughput_gb300.profile_cases decode-attn-kv
    python -m bit_compressed_throughput_gb300.profile_cases prefill-attn-opt67b
    python -m bit_compressed_throughput_gb300.profile_cases gemm-prefill-opt175b --reps 0
    python -m bit_compressed_throughput_gb300.profile_cases layer-prefill-opt175b --reps 0

Inputs are seeded random device tensors (no parity check here; the tests do that).
"""
from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def gemm_case(M, K, N, epi, reps):
    import torch
    from bit_compressed_throughput_gb300 import fg
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    X = torch.randn((M, K), generator=g, device="cuda").half()
    W = fg.Q4Weight.from_fp16((torch.randn((K, N), generator=g, device="cuda") * 0.02).half())
    bias = torch.zeros(N, dtype=torch.float16, device="cuda")
    Y = torch.empty((M, N), dtype=torch.float16, device="cuda")
    wsb = fg.fg_gemm_workspace_bytes(M, K, N)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda") if wsb else None
    for _ in range(1 + reps):
        fg.fg_dequant_gemm_q4(X, W, bias, epi, None, Y, ws)
    fg.fg_check_device_error()


def gemm_shapes(shapes, reps):
    """Several GEMM shapes one after the other, each with its own tensors (freed before the
    next shape is allocated)."""
    import torch
    for M, K, N, epi in shapes:
        gemm_case(M, K, N, epi, reps)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()


def attn_case(B, H, d, length, reps, topk=0):
    import torch
    import fg_synth
    from bit_compressed_throughput_gb300 import fg
    cap = (length + 15) // 16 * 16
    kc, vc, ka, va = fg_synth.random_q4_cache_torch(B, H, cap, d, seed=3)
    cache = fg.KVCacheQ4.__new__(fg.KVCacheQ4)
    cache.B, cache.cap, cache.h, cache.H, cache.d = B, cap, H * d, H, d
    cache.k_codes, cache.v_codes, cache.k_ab, cache.v_ab = kc, vc, ka, va
    q = torch.randn((B, H * d), device="cuda").half()
    out = torch.empty_like(q)
    wsb = fg.fg_decode_attn_workspace_bytes(cache, length)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda") if wsb else None
    tws = torch.empty(fg.fg_decode_attn_topk_workspace_bytes(cache, length), dtype=torch.uint8,
                      device="cuda") if topk else None
    for _ in range(1 + reps):
        if topk:
            fg.fg_decode_attn_q4kv_topk(q, H * d, cache, length, topk, 1.0 / math.sqrt(d), out,
                                        tws)
        else:
            fg.fg_decode_attn_q4kv(q, H * d, cache, length, 1.0 / math.sqrt(d), out, ws)
    torch.cuda.synchronize()


def prefill_case(nseq, s, H, d, reps):
    import torch
    from bit_compressed_throughput_gb300 import fg
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    qkv = torch.randn((nseq * s, 3 * H * d), generator=g, device="cuda").half()
    out = torch.empty((nseq * s, H * d), dtype=torch.float16, device="cuda")
    for _ in range(1 + reps):
        fg.fg_prefill_attn(qkv, nseq, s, H, d, 1.0 / math.sqrt(d), out)
    fg.fg_check_device_error()


def window_case(op, B, Hq, H, d, lens, window, reps):
    """One ragged cache call or windowed attention over B sequences of lengths between lens[0] and
    lens[1], a window (0: none) and 4 first positions."""
    import torch
    from bit_compressed_throughput_gb300 import fg
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    n = [lens[0] + (lens[1] - lens[0]) * i // max(1, B - 1) for i in range(B)]
    off = torch.tensor([0] + n, device="cuda").cumsum(0).int()
    pos, ln = torch.zeros(B, dtype=torch.int32, device="cuda"), off[1:] - off[:-1]
    rows, h, scale = sum(n), H * d, 1.0 / math.sqrt(d)
    kv = torch.randn((rows, 2 * h), generator=g, device="cuda").half()
    k, v = kv[:, :h], kv[:, h:]
    cache = fg.KVCacheQ4(B, lens[1], h, H)
    fg.fg_kv_append_q4_ragged(k, v, off, pos, cache)
    q = torch.randn((B if op == "decode" else rows, Hq * d), generator=g, device="cuda").half()
    out = torch.empty_like(q)
    back = torch.empty_like(kv)
    ws = torch.empty(fg.fg_decode_attn_window_workspace_bytes(cache, Hq), dtype=torch.uint8,
                     device="cuda")
    for _ in range(1 + reps):
        if op == "append":
            fg.fg_kv_append_q4_ragged(k, v, off, pos, cache)
        elif op == "read":
            fg.fg_kv_read_q4_ragged(cache, off, pos, back[:, :h], back[:, h:])
        elif op == "decode":
            fg.fg_decode_attn_q4kv_window(q, Hq, cache, ln, scale, out, ws, window=window, sinks=4)
        else:
            fg.fg_prefill_attn_window(q, off, k, v, off, Hq, H, scale, out, window=window, sinks=4)
    fg.fg_check_device_error()


def paged_case(op, Hq, H, d, page, lens, new, reps, window=0, keep=0):
    """Rotary positions, append, attention, received weights or eviction over pages: sequences of the
    given lengths, with their newest `new` positions as query (and appended) rows."""
    import torch
    from bit_compressed_throughput_gb300 import fg
    g = torch.Generator(device="cuda")
    g.manual_seed(19)
    B, G = len(lens), Hq // H
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    offs = lambda x: i32([0] + [sum(x[:i + 1]) for i in range(B)])
    need = [(n + page - 1) // page for n in lens]
    kept_pages = (keep + page - 1) // page
    order = torch.randperm(sum(need) + B * kept_pages, generator=g, device="cuda").int()
    table = torch.zeros((B, max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    pages = fg.KVPagesQ4(sum(need) + B * kept_pages, page, H * d, H)
    x = torch.randn((sum(lens), 2 * H * d), generator=g, device="cuda").half()
    fg.fg_kv_append_q4_paged(x[:, :H * d], x[:, H * d:], offs(lens), i32([0] * B), pages, table)
    angles = torch.empty((max(lens), d // 2, 2), device="cuda")
    fg.fg_rope_table(angles, 1e4)
    rows, pos = sum(new), i32([n - m for n, m in zip(lens, new)])
    q = torch.randn((rows, Hq * d), generator=g, device="cuda").half()
    out, lse = torch.empty_like(q), torch.empty((rows, Hq), device="cuda")
    acc = torch.rand((B, H, max(lens)), generator=g, device="cuda")
    ws = torch.empty(fg.fg_attn_paged_workspace_bytes(pages, Hq, max(new)), dtype=torch.uint8,
                     device="cuda")
    args = (q, offs(new), Hq, pages, table, i32(lens), 1.0 / math.sqrt(d))
    attend = lambda: fg.fg_attn_q4kv_paged(*args, out, ws, max_q=max(new), window=window, lse=lse)
    if op == "rope":
        call = lambda: fg.fg_rope(q, d, offs(new), pos, angles, out)
    elif op == "append":
        call = lambda: fg.fg_kv_append_q4_paged(x[:rows, :H * d], x[:rows, H * d:], offs(new), pos,
                                                pages, table, angles=angles)
    elif op == "attend":
        call = attend
    elif op == "weights":
        attend()
        call = lambda: fg.fg_attn_weights_q4_paged(*args, lse, acc, acc, max_q=max(new),
                                                   window=window)
    else:
        dst = order[at:].view(B, kept_pages)
        kept = torch.empty((B, H, keep), dtype=torch.int32, device="cuda")
        acc_out, left = torch.empty((B, H, keep), device="cuda"), i32([0] * B)
        call = lambda: fg.fg_kv_evict_q4_paged(pages, table, i32(lens), acc, 256, dst, kept, acc_out,
                                               left)
    for _ in range(1 + reps):
        call()
    fg.fg_check_device_error()


def between(lo, hi, n):
    """n lengths spread evenly over lo .. hi."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def layer_prefill_case(h, H, f, g, s, reps):
    """One decoder layer's prefill over one GPU batch (g sequences of s tokens): the layer
    restores its weights to fp16 once, then runs LN, the four projections (the CTA-pair GEMM
    in its fp16-weight mode), the K/V append and prefill attention."""
    import torch
    from bit_compressed_throughput_gb300 import fg
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    params = {}
    for name, (K, N) in {"wqkv": (h, 3 * h), "wo": (h, h), "w1": (h, f), "w2": (f, h)}.items():
        params[name] = (torch.randn((K, N), generator=gen, device="cuda") * 0.02).half()
    params.update({"bqkv": torch.zeros(3 * h), "bo": torch.zeros(h), "ln1_g": torch.ones(h),
                   "ln1_b": torch.zeros(h), "ln2_g": torch.ones(h), "ln2_b": torch.zeros(h),
                   "b1": torch.zeros(f), "b2": torch.zeros(h)})
    layer = fg.LayerQ4.from_fp16(params, H)
    del params
    torch.cuda.empty_cache()
    eng = fg.StackEngine([layer], g, 1, s, s)
    x = torch.randn((g, s, h), generator=gen, device="cuda").half()
    y = torch.empty_like(x)
    for _ in range(1 + reps):
        eng.prefill(x, y, s)
    fg.fg_check_device_error()


CASES = {
    # 6.7B prefill FC1 of one GPU batch: M = 16*512, K = 4096, N = 16384, ReLU
    "gemm-fc1-opt67b": lambda r: gemm_case(8192, 4096, 16384, 1, r),
    # 6.7B prefill QKV: N = 3*4096
    "gemm-qkv-opt67b": lambda r: gemm_case(8192, 4096, 12288, 0, r),
    # OPT-175B prefill projections of one GPU batch (36 sequences x 512 = 18432 tokens):
    # QKV, O, FC1 (ReLU), FC2 in layer order, at most 2.6 GB on the device at a time
    "gemm-prefill-opt175b": lambda r: gemm_shapes(((18432, 12288, 36864, 0),
                                                   (18432, 12288, 12288, 0),
                                                   (18432, 12288, 49152, 1),
                                                   (18432, 49152, 12288, 0)), r),
    # one OPT-175B layer's prefill over one GPU batch (36 x 512 tokens): ~9 GB on the device
    "layer-prefill-opt175b": lambda r: layer_prefill_case(12288, 96, 49152, 36, 512, r),
    # one opt-6.7b layer's prefill over one GPU batch (16 x 512 tokens): ~2 GB on the device,
    # for multi-pass captures of the fp16-weight GEMM (launches QKV, O, FC1, FC2 in order)
    "layer-prefill-opt67b": lambda r: layer_prefill_case(4096, 32, 16384, 16, 512, r),
    # 6.7B decode FC1 (M = B = 64, split K)
    "gemm-fc1-decode-opt67b": lambda r: gemm_case(64, 4096, 16384, 1, r),
    # 6.7B decode attention at the last step: 64 sequences x 32 heads x 543 positions
    "decode-attn-opt67b": lambda r: attn_case(64, 32, 128, 543, r),
    # KV-dominated workload: 512 sequences x 56 heads x 1056 positions (4.3 GB of cache)
    "decode-attn-kv": lambda r: attn_case(512, 56, 128, 1056, r),
    # a quarter of it (128 sequences, 1.1 GB of cache): the same per-warp work, capture-sized
    "decode-attn-kv-quarter": lambda r: attn_case(128, 56, 128, 1056, r),
    # top-K sparse attention on the quarter KV workload: the top 10% (106 of 1056 positions)
    "decode-attn-topk-kv-quarter": lambda r: attn_case(128, 56, 128, 1056, r, topk=106),
    # 6.7B prefill attention of one GPU batch: 16 sequences x 32 heads x 512 (201 MB of QKV)
    "prefill-attn-opt67b": lambda r: prefill_case(16, 512, 32, 128, r),
    # KV-workload prefill attention, a quarter of one GPU batch: 32 x 56 heads x 1024 (1.3 GB)
    "prefill-attn-kv-quarter": lambda r: prefill_case(32, 1024, 56, 128, r),
    # ragged cache calls over 36 prompts of 400 .. 512 tokens, 96 heads (0.8 GB of fp16 K/V)
    "kv-append-ragged": lambda r: window_case("append", 36, 96, 96, 128, (400, 512), 0, r),
    "kv-read-ragged": lambda r: window_case("read", 36, 96, 96, 128, (400, 512), 0, r),
    # windowed decode attention: 128 sequences x 56 heads of 512 .. 1055 positions, all visible
    # (0.8 GB of cache), and 4 query heads per K/V head over long contexts
    "decode-window-full": lambda r: window_case("decode", 128, 56, 56, 128, (512, 1055), 0, r),
    "decode-window-grouped": lambda r: window_case("decode", 16, 32, 8, 128, (9000, 32760), 16384,
                                                   r),
    # windowed prefill attention: long documents with grouped heads, and prompts
    "prefill-window-long": lambda r: window_case("prefill", 2, 32, 8, 128, (7001, 8191), 1024, r),
    "prefill-window-prompts": lambda r: window_case("prefill", 16, 32, 32, 128, (300, 512), 0, r),
    "rope-prompts": lambda r: paged_case("rope", 64, 8, 128, 16, between(300, 512, 16),
                                         between(300, 512, 16), r),
    "append-paged": lambda r: paged_case("append", 32, 32, 128, 64, between(300, 512, 16),
                                         between(300, 512, 16), r),
    "attend-paged-step": lambda r: paged_case("attend", 32, 8, 128, 16, between(9000, 32760, 16),
                                              [1] * 16, r),
    "attend-paged-pieces": lambda r: paged_case("attend", 32, 32, 128, 32, between(400, 2000, 8),
                                                between(100, 256, 8), r),
    "attend-paged-long": lambda r: paged_case("attend", 32, 8, 128, 64, [12001, 16384], [1501, 2048],
                                              r, window=8192),
    "attn-weights-step": lambda r: paged_case("weights", 32, 8, 128, 16, between(2000, 4096, 32),
                                              [1] * 32, r),
    "attn-weights-recent": lambda r: paged_case("weights", 32, 8, 128, 64, between(8001, 16001, 8),
                                                [64] * 8, r),
    "evict-long": lambda r: paged_case("evict", 8, 8, 128, 64, between(20001, 32001, 4), [1] * 4, r,
                                       keep=8192),
    # top-K on the full KV workload (launch lists only: 4.3 GB of cache)
    "decode-attn-topk-kv": lambda r: attn_case(512, 56, 128, 1056, r, topk=106),
}


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("case", choices=sorted(CASES))
    ap.add_argument("--reps", type=int, default=2)
    a = ap.parse_args()
    import torch
    import __graft_entry__
    __graft_entry__.build()
    CASES[a.case](a.reps)
    torch.cuda.synchronize()
    print(f"{a.case}: ok")


if __name__ == "__main__":
    main()
