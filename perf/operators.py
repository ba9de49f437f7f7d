"""What is measured of the ragged, windowed K/V-cache operators: the cases, their inputs, a plain
form in torch and the calls a user makes.

Operators (names of the package's binding):

- ``fg_kv_append_q4_ragged``: new K/V rows of sequences of different lengths are quantised to 4
  bits (groups of 64) and written at each sequence's own position of the cache;
- ``fg_kv_read_q4_ragged``: ranges of cached positions are restored to fp16 rows;
- ``fg_decode_attn_q4kv_window``: one query per sequence over its own length of the 4-bit cache,
  with a sliding window, first positions that stay visible, and query heads that share K/V heads;
- ``fg_prefill_attn_window``: many queries per sequence over fp16 K/V rows, with the same mask.

Query position i sees key position t when t <= i and (window == 0 or t > i - window or t < sinks).
"""
import math

import torch

own = False

GROUP = 64


# ------------------------------------------------------------------------------------ cases
#
# op "append": append, then the written rows read back (what the cache holds in 4 bits is returned
#              as the values it stands for); op "read": ranges of a filled cache read back;
#              op "decode": one token per sequence; op "prefill": many queries per sequence.
# lo, hi: the range of the sequences' lengths (drawn from the seed, odd ones among them).


def listed():
    return [
        # ---- one generation step over the 4-bit cache
        # one user, short context: latency counts
        dict(name="decode_one", op="decode", B=1, Hq=32, Hkv=32, d=128, lo=513, hi=513,
             window=256, sinks=4),
        # a block of 64 sequences of a 32-head model, each with its own length, sliding window
        dict(name="decode_window", op="decode", B=64, Hq=32, Hkv=32, d=128, lo=200, hi=2048,
             window=1024, sinks=4),
        # a block whose K/V cache is what a step costs: 56 heads, everything visible
        dict(name="decode_full", op="decode", B=128, Hq=56, Hkv=56, d=128, lo=512, hi=1055,
             window=0, sinks=0),
        # long contexts, four query heads per K/V head, a long window
        dict(name="decode_grouped_long", op="decode", B=16, Hq=32, Hkv=8, d=128, lo=9000,
             hi=32760, window=16384, sinks=64),
        # ---- prompts, and pieces of prompts
        # a few short prompts of a small model
        dict(name="prefill_short", op="prefill", nseq=3, Hq=12, Hkv=12, d=64, qlo=1, qhi=130,
             past=0, window=64, sinks=4),
        # a GPU batch of 16 prompts of up to 512 tokens, all of each prompt visible
        dict(name="prefill_prompts", op="prefill", nseq=16, Hq=32, Hkv=32, d=128, qlo=300,
             qhi=512, past=0, window=0, sinks=0),
        # long documents under a sliding window, grouped heads
        dict(name="prefill_long_window", op="prefill", nseq=2, Hq=32, Hkv=8, d=128, qlo=7001,
             qhi=8191, past=0, window=1024, sinks=4),
        # a piece of 256 tokens of each of 8 prompts against what is cached of it
        dict(name="prefill_piece", op="prefill", nseq=8, Hq=32, Hkv=32, d=128, qlo=200, qhi=256,
             past=2000, window=1024, sinks=16),
        # ---- writing the cache and reading it back
        # one new token of each of 64 sequences
        dict(name="append_step", op="append", B=64, Hkv=32, d=128, lo=1, hi=1, past=700),
        # the prompts of a GPU batch
        dict(name="append_prompts", op="append", B=16, Hkv=32, d=128, lo=300, hi=512, past=0),
        # the prompts of a GPU batch of a 96-head model
        dict(name="append_wide", op="append", B=36, Hkv=96, d=128, lo=400, hi=512, past=0),
        # the recent part of long contexts, for a piece of prompt that attends to it in fp16
        dict(name="read_recent", op="read", B=16, Hkv=8, d=128, lo=2000, hi=4096, past=5000),
    ]


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads = [(4, 4), (12, 12), (32, 32), (56, 56), (96, 96), (32, 8), (28, 4), (40, 8), (8, 1)]
    cap = {op: max(_cost(c) for c in listed() if c["op"] == op)
           for op in ("decode", "prefill", "append", "read")}
    while True:
        op = rng.choice(["decode", "decode", "prefill", "prefill", "append", "read"])
        Hq, Hkv = rng.choice(heads)
        d = rng.choice([64, 128])
        window = rng.choice([0, _log_int(rng, 1, 8192), _log_int(rng, 64, 4096)])
        sinks = rng.choice([0, 4, rng.randint(1, 100)]) if window else 0
        if op == "decode":
            hi = _log_int(rng, 1, 32768)
            c = dict(op=op, B=_log_int(rng, 1, 160), Hq=Hq, Hkv=Hkv, d=d,
                     lo=max(1, int(hi * rng.uniform(0.2, 1.0))), hi=hi, window=window, sinks=sinks)
        elif op == "prefill":
            hi = _log_int(rng, 1, 8192)
            c = dict(op=op, nseq=_log_int(rng, 1, 24), Hq=Hq, Hkv=Hkv, d=d,
                     qlo=max(1, int(hi * rng.uniform(0.2, 1.0))), qhi=hi,
                     past=rng.choice([0, _log_int(rng, 1, 4096)]), window=window, sinks=sinks)
        else:
            hi = _log_int(rng, 1, 4096)
            c = dict(op=op, B=_log_int(rng, 1, 128), Hkv=Hkv, d=d,
                     lo=max(1, int(hi * rng.uniform(0.2, 1.0))), hi=hi,
                     past=rng.choice([0, _log_int(rng, 1, 4096)]))
        if _cost(c) > cap[op]:
            continue
        # the plain form holds the cache (or the rows) in 32 bits: bounded like the listed cases
        if op != "prefill" and c["B"] * c["Hkv"] * d * (c["hi"] + c.get("past", 0)) > 1.2e9:
            continue
        return c


def _mean(lo, hi):
    return (lo + hi) / 2.0


def _visible(nq, nk, window, sinks):
    """Visible (query, key) pairs of nq queries at the end of nk keys."""
    n = 0
    for i in range(nk - nq, nk):
        a = i + 1
        if window:
            a = min(a, window + min(sinks, max(0, i + 1 - window)))
        n += a
    return n


def work(case):
    op, d = case["op"], case["d"]
    if op in ("append", "read"):
        n = case["B"] * _mean(case["lo"], case["hi"]) * case["Hkv"] * d
        q4 = 2 * n * (0.5 + 4.0 / GROUP)
        if op == "read":
            return {"bytes": q4 + 4 * n, "flops": 4.0 * n}
        return {"bytes": 4 * n + q4 + 4 * n, "flops": 12.0 * n}
    if op == "decode":
        vis = sum(_visible(1, L, case["window"], case["sinks"])
                  for L in _spread(case["lo"], case["hi"], case["B"]))
        kv = 2 * vis * case["Hkv"] * d * (0.5 + 4.0 / GROUP)
        return {"bytes": kv + 4.0 * case["B"] * case["Hq"] * d,
                "flops": 4.0 * vis * case["Hq"] * d}
    qs = _spread(case["qlo"], case["qhi"], case["nseq"])
    vis = sum(_visible(q, q + case["past"], case["window"], case["sinks"]) for q in qs)
    rows_k = 0
    for q in qs:
        nk = q + case["past"]
        seen = nk
        if case["window"]:
            first = max(0, nk - q - case["window"] + 1)      # oldest key in any query's window
            seen = nk - first + min(case["sinks"], first)
        rows_k += seen
    return {"bytes": 4.0 * sum(qs) * case["Hq"] * d + 4.0 * rows_k * case["Hkv"] * d,
            "flops": 4.0 * vis * case["Hq"] * d}


def _spread(lo, hi, n):
    return [int(round(lo + (hi - lo) * i / (n - 1))) for i in range(n)] if n > 1 else [hi]


# ------------------------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lengths(lo, hi, n, seed):
    """n lengths spread over [lo, hi], in an order of the seed's own (their sum is the case's)."""
    g = torch.Generator()
    g.manual_seed(seed * 7919 + n)
    return torch.tensor(_spread(lo, hi, n))[torch.randperm(n, generator=g)].tolist()


def _offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def _kv_like(shape, gen):
    """Keys or values as a projection gives them: normal, some channels several times larger."""
    x = torch.randn(shape, device="cuda", generator=gen, dtype=torch.float32)
    ch = 0.5 + torch.rand(shape[-1], device="cuda", generator=gen)
    ch[torch.randint(0, shape[-1], (max(1, shape[-1] // 64),), device="cuda", generator=gen)] *= 4
    return (x * ch).half()


def _cap16(n):
    return (n + 15) // 16 * 16


def prepare(case, seed):
    gen = _gen(seed)
    op, d = case["op"], case["d"]
    st = {"case": dict(case), "scale": 1.0 / math.sqrt(d)}
    if op == "prefill":
        nq = _lengths(case["qlo"], case["qhi"], case["nseq"], seed)
        nk = [q + case["past"] for q in nq]
        Hq, Hkv = case["Hq"], case["Hkv"]
        st["nq"], st["nk"] = nq, nk
        st["q_off"], st["kv_off"] = _offsets(nq), _offsets(nk)
        if case["past"] == 0:
            # Q, K and V as the projection leaves them, side by side in one buffer
            w = (Hq + 2 * Hkv) * d
            buf = torch.empty((sum(nq), w), dtype=torch.float16, device="cuda")
            buf[:, :Hq * d] = torch.randn((sum(nq), Hq * d), device="cuda", generator=gen).half()
            buf[:, Hq * d:] = _kv_like((sum(nq), 2 * Hkv * d), gen)
            st["q"], st["k"] = buf[:, :Hq * d], buf[:, Hq * d:(Hq + Hkv) * d]
            st["v"] = buf[:, (Hq + Hkv) * d:]
        else:
            # the piece's queries, and K/V rows read back from the cache
            st["q"] = torch.randn((sum(nq), Hq * d), device="cuda", generator=gen).half()
            st["k"], st["v"] = _kv_like((sum(nk), Hkv * d), gen), _kv_like((sum(nk), Hkv * d), gen)
        st["out"] = torch.empty((sum(nq), Hq * d), dtype=torch.float16, device="cuda")
        return st

    B, H = case["B"], case["Hkv"]
    lens = _lengths(case["lo"], case["hi"], B, seed)
    past = case.get("past", 0)
    pos = _lengths(max(0, past - past // 4), past, B, seed + 1)
    cap = _cap16(max(p + n for p, n in zip(pos, lens)))
    if op != "append":
        # a cache filled by earlier steps, in the library's layout
        kc, ka, vc, va = [], [], [], []
        for _ in range(B):                       # one sequence at a time: bounded scratch
            for codes, ab in ((kc, ka), (vc, va)):
                x = _kv_like((cap, H * d), gen).view(cap, H, d).transpose(0, 1)
                q, a, b = _plain_quantize(x)
                c, w = _pack(q, a, b)
                codes.append(c)
                ab.append(w)
        st["k_codes"], st["k_ab"] = torch.stack(kc), torch.stack(ka)
        st["v_codes"], st["v_ab"] = torch.stack(vc), torch.stack(va)
    else:
        st["k_codes"] = torch.zeros((B, H, cap, d // 2), dtype=torch.uint8, device="cuda")
        st["k_ab"] = torch.zeros((B, H, cap, d // GROUP), dtype=torch.int32, device="cuda")
        st["v_codes"], st["v_ab"] = torch.zeros_like(st["k_codes"]), torch.zeros_like(st["k_ab"])
    st["lens_list"], st["pos_list"] = lens, pos
    if op == "decode":
        Hq = case["Hq"]
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["q"] = torch.randn((B, Hq * d), device="cuda", generator=gen).half()
        st["out"] = torch.empty((B, Hq * d), dtype=torch.float16, device="cuda")
    else:
        rows = sum(lens)
        st["row_off"] = _offsets(lens)
        st["pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
        if op == "append":
            # K and V as the projection leaves them, side by side in one buffer
            buf = _kv_like((rows, 2 * H * d), gen)
            st["k_new"], st["v_new"] = buf[:, :H * d], buf[:, H * d:]
        st["k_out"] = torch.empty((rows, H * d), dtype=torch.float16, device="cuda")
        st["v_out"] = torch.empty_like(st["k_out"])
    if own:
        from bit_compressed_throughput_gb300 import fg
        cache = fg.KVCacheQ4(B, 16, H * d, H)
        cache.cap = cap
        cache.k_codes, cache.k_ab = st["k_codes"], st["k_ab"]
        cache.v_codes, cache.v_ab = st["v_codes"], st["v_ab"]
        st["cache"] = cache
        if op == "decode":
            n = fg.fg_decode_attn_window_workspace_bytes(cache, case["Hq"])
            st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------------------------ one pass


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from bit_compressed_throughput_gb300 import fg
    c = st["case"]
    if c["op"] == "prefill":
        fg.fg_prefill_attn_window(st["q"], st["q_off"], st["k"], st["v"], st["kv_off"], c["Hq"],
                                  c["Hkv"], st["scale"], st["out"], window=c["window"],
                                  sinks=c["sinks"])
        return st["out"]
    if c["op"] == "decode":
        fg.fg_decode_attn_q4kv_window(st["q"], c["Hq"], st["cache"], st["lens"], st["scale"],
                                      st["out"], st["ws"], window=c["window"], sinks=c["sinks"])
        return st["out"]
    if c["op"] == "append":
        fg.fg_kv_append_q4_ragged(st["k_new"], st["v_new"], st["row_off"], st["pos"], st["cache"])
    fg.fg_kv_read_q4_ragged(st["cache"], st["row_off"], st["pos"], st["k_out"], st["v_out"])
    return st["k_out"], st["v_out"]


# The plain form: elementary torch operations in 32 bits, rounded to fp16 once at the end.


def _plain_quantize(x):
    """Codes (32-bit, 0..15) and fp16 (a, b) of fp16 x [..., d] in groups of 64."""
    g = x.float().unflatten(-1, (-1, GROUP))
    a, b = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    r = b - a
    q = torch.round((g - a) * 15.0 / torch.where(r == 0, torch.ones_like(r), r))
    q = torch.where(r == 0, torch.zeros_like(q), q.clamp(0, 15))
    return q.flatten(-2), a.squeeze(-1).half(), b.squeeze(-1).half()


def _pack(q, a, b):
    q = q.to(torch.uint8)
    codes = q[..., 0::2] | (q[..., 1::2] << 4)
    ab = torch.stack((a, b), -1).contiguous().view(torch.int32).squeeze(-1)
    return codes.contiguous(), ab.contiguous()


def _plain_restore(codes, ab):
    """fp16 values [..., d] of packed codes [..., d/2] and statistics words [..., d/64]."""
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    s = ab.contiguous().view(torch.float16).unflatten(-1, (-1, 2)).float()
    a, b = s[..., 0:1], s[..., 1:2]
    return (a + q.unflatten(-1, (-1, GROUP)) * ((b - a) / 15.0)).flatten(-2).half()


def _plain_mask(i, t, window, sinks):
    ok = t <= i
    if window:
        ok = ok & ((t > i - window) | (t < sinks))
    return ok


def _plain_attend(s, ok, v):
    """softmax of s [..., nq, nk] over the visible keys, times v [..., nk, d]; 0 where none is."""
    s = s.masked_fill(~ok, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(l == 0, torch.ones_like(l), l)


def _run_plain(st):
    c, d = st["case"], st["case"]["d"]
    if c["op"] == "prefill":
        Hq, Hkv = c["Hq"], c["Hkv"]
        out, q0, k0 = [], 0, 0
        for nq, nk in zip(st["nq"], st["nk"]):
            q = st["q"][q0:q0 + nq].float().view(nq, Hkv, Hq // Hkv, d).permute(1, 2, 0, 3)
            k = st["k"][k0:k0 + nk].float().view(nk, Hkv, 1, d).permute(1, 2, 0, 3)
            v = st["v"][k0:k0 + nk].float().view(nk, Hkv, 1, d).permute(1, 2, 0, 3)
            t = torch.arange(nk, device="cuda")
            step = max(1, (1 << 28) // (Hq * nk))               # bounded scratch
            for r in range(0, nq, step):
                i = torch.arange(r, min(nq, r + step), device="cuda")[:, None] + (nk - nq)
                s = torch.matmul(q[:, :, r:r + step], k.transpose(-1, -2)) * st["scale"]
                o = _plain_attend(s, _plain_mask(i, t, c["window"], c["sinks"]), v)
                out.append(o.permute(2, 0, 1, 3).reshape(-1, Hq * d).half())
            q0, k0 = q0 + nq, k0 + nk
        return torch.cat(out)
    if c["op"] == "decode":
        B, Hq, Hkv = c["B"], c["Hq"], c["Hkv"]
        n = max(st["lens_list"])
        k = _plain_restore(st["k_codes"][:, :, :n], st["k_ab"][:, :, :n]).float()
        v = _plain_restore(st["v_codes"][:, :, :n], st["v_ab"][:, :, :n]).float()
        q = st["q"].float().view(B, Hkv, Hq // Hkv, d)
        i = (st["lens"] - 1)[:, None, None, None]
        ok = _plain_mask(i, torch.arange(n, device="cuda"), c["window"], c["sinks"])
        s = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
        return _plain_attend(s, ok, v).reshape(B, Hq * d).half()
    B, H = c["B"], c["Hkv"]
    lens = torch.tensor(st["lens_list"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), lens,
                                  output_size=st["k_out"].shape[0])
    t = torch.arange(len(seq), device="cuda") - st["row_off"][seq] + st["pos"][seq]
    if c["op"] == "append":
        for new, codes, ab in ((st["k_new"], st["k_codes"], st["k_ab"]),
                               (st["v_new"], st["v_codes"], st["v_ab"])):
            codes[seq, :, t], ab[seq, :, t] = _pack(*_plain_quantize(new.unflatten(1, (H, d))))
    return tuple(_plain_restore(codes[seq, :, t], ab[seq, :, t]).flatten(1)
                 for codes, ab in ((st["k_codes"], st["k_ab"]), (st["v_codes"], st["v_ab"])))


# ------------------------------------------------------------------------------------ exact
#
# From the definitions, in 64 bits.  Codes and restored values are defined with one binary32
# rounding per operation (and restored values with a last one to fp16): these roundings are made,
# everything else is 64-bit.


def _f32(x):
    return x.float().double()


def _exact_codes(x):
    """x: 64-bit values of fp16 numbers [rows][groups][64] -> 64-bit (codes, a, b)."""
    a = x.min(dim=2).values[:, :, None]
    b = x.max(dim=2).values[:, :, None]
    width = _f32(b - a)
    num = _f32(_f32(x - a) * 15)
    code = _f32(num / width.masked_fill(width == 0, 1)).round()
    return code.clamp(min=0, max=15).masked_fill(width == 0, 0), a, b


def _exact_values(code, a, b):
    step = _f32(_f32(b - a) / 15)
    return _f32(a + _f32(code * step)).half().double()


def _exact_cache(codes, ab):
    """64-bit values [n][d] of n cached positions (of one or more heads)."""
    n = codes.shape[0]
    byte = codes.long()
    code = torch.empty((n, 2 * codes.shape[1]), dtype=torch.float64, device=codes.device)
    code[:, 0::2] = (byte % 16).double()
    code[:, 1::2] = (byte // 16).double()
    word = ab.long() & 0xFFFFFFFF
    a = (word & 0xFFFF).to(torch.int32).to(torch.int16).view(torch.float16).double()
    b = (word >> 16).to(torch.int32).to(torch.int16).view(torch.float16).double()
    return _exact_values(code.view(n, -1, GROUP), a[:, :, None], b[:, :, None]).view(n, -1)


def _exact_rows(q, k, v, first, window, sinks, scale):
    """Outputs of queries q [..][n][d] at positions first, first + 1, .. over keys [..][nk][d]."""
    n, nk = q.shape[-2], k.shape[-2]
    i = torch.arange(first, first + n, device=q.device).view(n, 1)
    t = torch.arange(nk, device=q.device).view(1, nk)
    hidden = t > i
    if window > 0:
        hidden = hidden | ((t <= i - window) & (t >= sinks))
    e = (q @ k.mT) * scale
    e[..., hidden] = -math.inf
    return torch.softmax(e, dim=-1) @ v


def exact(case, seed):
    st = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "prefill":
        Hq, Hkv = case["Hq"], case["Hkv"]
        dense = sum(4.0 * nq * nk * Hq * d for nq, nk in zip(st["nq"], st["nk"]))
        if dense > 6e12:
            return None
        res = torch.empty((sum(st["nq"]), Hq * d), dtype=torch.float64, device="cuda")
        q0 = k0 = 0
        for nq, nk in zip(st["nq"], st["nk"]):
            for h in range(Hq):
                cq, ck = slice(h * d, h * d + d), slice(h // (Hq // Hkv) * d,
                                                        h // (Hq // Hkv) * d + d)
                k, v = st["k"][k0:k0 + nk, ck].double(), st["v"][k0:k0 + nk, ck].double()
                for r in range(0, nq, 2048):
                    rr = slice(q0 + r, q0 + min(nq, r + 2048))
                    res[rr, cq] = _exact_rows(st["q"][rr, cq].double(), k, v, nk - nq + r,
                                              case["window"], case["sinks"], st["scale"])
            q0, k0 = q0 + nq, k0 + nk
        return res
    if op == "decode":
        Hq, Hkv = case["Hq"], case["Hkv"]
        res = torch.empty((case["B"], Hq * d), dtype=torch.float64, device="cuda")
        for b, n in enumerate(st["lens_list"]):
            k, v = (_exact_cache(st[x + "_codes"][b, :, :n].flatten(0, 1),
                                 st[x + "_ab"][b, :, :n].flatten(0, 1)).view(Hkv, n, d)
                    for x in "kv")
            res[b] = _exact_rows(st["q"][b].double().view(Hkv, Hq // Hkv, 1, d), k[:, None],
                                 v[:, None], n - 1, case["window"], case["sinks"],
                                 st["scale"]).flatten()
        return res
    if op == "append":
        outs = []
        for new in (st["k_new"], st["v_new"]):
            rows, parts = new.shape[0], []
            for r in range(0, rows, 2048):
                x = new[r:r + 2048].double()
                parts.append(_exact_values(*_exact_codes(x.view(x.shape[0], -1, GROUP)))
                             .view(x.shape[0], -1))
            outs.append(torch.cat(parts))
        return tuple(outs)
    outs = []
    for codes, ab in ((st["k_codes"], st["k_ab"]), (st["v_codes"], st["v_ab"])):
        parts = []
        for b, (p, n) in enumerate(zip(st["pos_list"], st["lens_list"])):
            parts.append(torch.cat([_exact_cache(codes[b, h, p:p + n], ab[b, h, p:p + n])
                                    for h in range(case["Hkv"])], dim=1))
        outs.append(torch.cat(parts))
    return tuple(outs)
