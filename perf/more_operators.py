"""What is measured of the paged 4-bit K/V cache and its rotary positions: the cases, their inputs, a
plain form in torch and the calls a user makes.

Operators (names of the package's binding):

- ``fg_rope``: rotary positions of packed rows, pairs in halves or interleaved, all or part of a
  head, each sequence at its own first position, angles from a table;
- ``fg_kv_append_q4_paged`` and ``fg_kv_read_q4_paged``: new K/V rows (K rotated on the way, if a
  table is given) quantised to 4 bits into the pages of their sequences, and restored from them;
- ``fg_attn_q4kv_paged``: the newest tokens of every sequence, one or many, over its pages, with a
  sliding window, first positions that stay visible, and query heads that share K/V heads;
- ``fg_attn_weights_q4_paged``: the softmax weights that cached positions receive from given
  queries, added to what they received before;
- ``fg_kv_evict_q4_paged``: every K/V head keeps its newest positions and the heaviest of the others,
  moved into pages of their own.

A block of pages [pages][H][bytes] holds, per page of P positions and K/V head, K codes [P][d/2], K
statistics [P][d/64], V codes, V statistics.  Query position i sees key position t when t <= i and
(window == 0 or t > i - window or t < sinks).
"""
import math

import torch

own = False

GROUP = 64


# ------------------------------------------------------------------------------------ cases
#
# lo, hi: the range of the sequences' rows (rope, append) or cached positions (the others), drawn
# from the seed, odd ones among them; qlo, qhi: the range of their query rows, of which the first
# `ones` sequences have one.


def listed():
    return [
        # ---- rotary positions
        # the queries of one generation step of 64 sequences, far into their contexts
        dict(name="rope_step", op="rope", B=64, heads=32, d=128, rot=128, interleaved=False,
             lo=1, hi=1, past=20000),
        # Q and K of a GPU batch of prompts, half of each head rotated, neighbouring pairs
        dict(name="rope_prompts", op="rope", B=16, heads=64, d=128, rot=64, interleaved=True,
             lo=300, hi=512, past=0),
        # ---- writing pages and reading them back
        # one new token of each of 64 sequences, K rotated, eight K/V heads
        dict(name="append_step", op="append", B=64, Hkv=8, d=128, page=16, rot=128,
             interleaved=False, lo=1, hi=1, past=700),
        # the prompts of a GPU batch, K rotated
        dict(name="append_prompts", op="append", B=16, Hkv=32, d=128, page=64, rot=128,
             interleaved=False, lo=300, hi=512, past=0),
        # ---- attention over pages
        # one user, one token, short context: latency counts
        dict(name="attend_one", op="attend", B=1, Hq=32, Hkv=8, d=128, page=16, ones=1, qlo=1, qhi=1,
             lo=513, hi=513, window=0, sinks=0),
        # a step of 16 long contexts, four query heads per K/V head
        dict(name="attend_step_long", op="attend", B=16, Hq=32, Hkv=8, d=128, page=16, ones=16,
             qlo=1, qhi=1, lo=9000, hi=32760, window=0, sinks=0),
        # continuous batching: 40 sequences generate while 8 take in a piece of their prompt
        dict(name="attend_mixed", op="attend", B=48, Hq=32, Hkv=32, d=128, page=32, ones=40,
             qlo=100, qhi=256, lo=400, hi=2000, window=0, sinks=0),
        # long pieces of two documents behind what is cached of them, under a sliding window
        dict(name="attend_pieces_long", op="attend", B=2, Hq=32, Hkv=8, d=128, page=64, ones=0,
             qlo=1501, qhi=2048, lo=12001, hi=16384, window=8192, sinks=4),
        # ---- what each cached position received
        # one token of each of 32 sequences
        dict(name="weights_step", op="weights", B=32, Hq=32, Hkv=8, d=128, page=16, ones=32,
             qlo=1, qhi=1, lo=2000, hi=4096, window=0, sinks=0),
        # the last 64 tokens of 8 long prompts, before their caches are made smaller
        dict(name="weights_recent", op="weights", B=8, Hq=32, Hkv=8, d=128, page=64, ones=0,
             qlo=64, qhi=64, lo=8001, hi=16001, window=0, sinks=0),
        # ---- smaller caches
        # prompts of a GPU batch cut to a quarter
        dict(name="evict_prompts", op="evict", B=16, Hkv=8, d=128, page=16, lo=2000, hi=4096,
             keep=1024, recent=256),
        # long contexts cut to 8192 positions
        dict(name="evict_long", op="evict", B=4, Hkv=8, d=128, page=64, lo=20001, hi=32001,
             keep=8192, recent=1024),
    ]


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads = [(4, 4), (12, 12), (32, 32), (56, 56), (32, 8), (28, 4), (40, 8), (8, 1)]
    ops = ("rope", "append", "attend", "weights", "evict")
    cap = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ops}
    while True:
        op = rng.choice(ops + ("attend", "attend"))
        Hq, Hkv = rng.choice(heads)
        d = rng.choice([64, 128])
        page = rng.choice([16, 32, 64, 128, 256])
        if op == "rope" or op == "append":
            hi = _log_int(rng, 1, 4096)
            c = dict(op=op, B=_log_int(rng, 1, 128), d=d, rot=rng.choice([d, d // 2, d // 4]),
                     interleaved=rng.choice([True, False]),
                     lo=max(1, int(hi * rng.uniform(0.2, 1.0))), hi=hi,
                     past=rng.choice([0, _log_int(rng, 1, 32768 if op == "rope" else 4096)]))
            if op == "rope":
                c["heads"] = rng.choice([Hq, Hq + Hkv])
            else:
                c["Hkv"], c["page"] = Hkv, page
                c["rot"] = rng.choice([0, c["rot"]])
            cells = 0 if op == "rope" else c["B"] * Hkv * d * (hi + c["past"])
        elif op == "evict":
            hi = _log_int(rng, 1, 32768)
            keep = _log_int(rng, 1, 8192)
            c = dict(op=op, B=_log_int(rng, 1, 64), Hkv=Hkv, d=d, page=page,
                     lo=max(1, int(hi * rng.uniform(0.2, 1.0))), hi=hi, keep=keep,
                     recent=rng.randint(0, keep))
            cells = c["B"] * Hkv * d * (hi + keep)
        else:
            B = _log_int(rng, 1, 64)
            window = rng.choice([0, _log_int(rng, 1, 8192), _log_int(rng, 64, 4096)])
            qhi = rng.choice([1, _log_int(rng, 1, 2048)])
            past = rng.choice([0, _log_int(rng, 1, 32768)])
            c = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, ones=rng.choice([0, B // 2, B]),
                     qlo=max(1, int(qhi * rng.uniform(0.2, 1.0))), qhi=qhi,
                     lo=qhi + int(past * rng.uniform(0.2, 1.0)), hi=qhi + past, window=window,
                     sinks=rng.choice([0, 4, rng.randint(1, 100)]) if window else 0)
            cells = B * Hkv * d * c["hi"]
        # the plain form holds the cache in 32 bits: bounded like the listed cases
        if _cost(c) <= cap[op] and cells <= 6e8:
            return c


def _spread(lo, hi, n):
    return [int(round(lo + (hi - lo) * i / (n - 1))) for i in range(n)] if n > 1 else [hi] * n


def _seen(nq, n, window, sinks):
    """Visible (query, key) pairs of nq queries at the end of n keys, and keys that one sees."""
    pairs = 0
    for i in range(n - nq, n):
        a = i + 1
        if window:
            a = min(a, window + min(sinks, max(0, i + 1 - window)))
        pairs += a
    first = max(0, n - nq - window + 1) if window else 0     # the oldest key of a window
    return pairs, n - first + min(sinks, first)


def _query_rows(case):
    """Query rows of the sequences, in the order of their lengths."""
    k = case["ones"]
    return [1] * k + _spread(case["qlo"], case["qhi"], case["B"] - k)


def work(case):
    op, d = case["op"], case["d"]
    if op == "rope":
        rows = sum(_spread(case["lo"], case["hi"], case["B"]))
        return {"bytes": 4.0 * rows * case["heads"] * d + 4.0 * rows * case["rot"],
                "flops": 3.0 * rows * case["heads"] * case["rot"]}
    q4 = 2 * case["Hkv"] * d * (0.5 + 4.0 / GROUP)           # K and V of one position
    fp16 = 4.0 * case["Hkv"] * d
    if op == "append":
        rows = sum(_spread(case["lo"], case["hi"], case["B"]))
        return {"bytes": rows * (fp16 + q4 + fp16 + 4.0 * case["rot"]),
                "flops": rows * case["Hkv"] * d * 12.0}
    if op == "evict":
        n = sum(_spread(case["lo"], case["hi"], case["B"]))
        kept = sum(min(x, case["keep"]) for x in _spread(case["lo"], case["hi"], case["B"]))
        return {"bytes": 4.0 * n * case["Hkv"] + kept * (2 * q4 + 8.0 * case["Hkv"] + fp16),
                "flops": 4.0 * n * case["Hkv"] + 4.0 * kept * case["Hkv"] * d}
    lens = _spread(case["lo"], case["hi"], case["B"])
    pairs = keys = rows = 0
    for nq, n in zip(_query_rows(case), lens):
        p, k = _seen(min(nq, n), n, case["window"], case["sinks"])
        pairs, keys, rows = pairs + p, keys + k, rows + nq
    wide = rows * case["Hq"] * d
    if op == "attend":
        return {"bytes": 4.0 * wide + keys * q4, "flops": 4.0 * pairs * case["Hq"] * d}
    return {"bytes": 2.0 * wide + 4.0 * rows * case["Hq"] + keys * q4 / 2
            + 8.0 * sum(lens) * case["Hkv"],
            "flops": 2.0 * pairs * case["Hq"] * d}


# ------------------------------------------------------------------------------------ inputs


def _order(n, seed):
    g = torch.Generator()
    g.manual_seed(seed * 7919 + n)
    return torch.randperm(n, generator=g).tolist()


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return _ints(off)


def _channels(n, gen):
    """Scales of channels, some several times larger."""
    ch = 0.5 + torch.rand(n, device="cuda", generator=gen)
    ch[torch.randint(0, n, (max(1, n // 64),), device="cuda", generator=gen)] *= 4
    return ch


def _normal(shape, gen):
    return torch.randn(shape, device="cuda", generator=gen, dtype=torch.float32)


def _angles(positions, rot, scaled):
    """cos and sin [positions][rot/2][2] in 64 bits, rounded once; the low frequencies of a long
    context stretched four times."""
    w = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if scaled:
        w = torch.where(w * 8192 / (2 * math.pi) < 1.0, w / 4, w)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * w
    return torch.stack((a.cos(), a.sin()), -1).float()


def _pool(case, positions, seed, fill, gen, spare=0):
    """Pages for sequences of so many positions, in an order of the seed's own, filled with cached
    K/V or zero, and the sequences' page tables (and second ones of `spare` positions each)."""
    H, d, P = case["Hkv"], case["d"], case["page"]
    need = [(n + P - 1) // P for n in positions]
    more = (spare + P - 1) // P
    pages = sum(need) + more * len(need) + 3
    order = iter(_order(pages, seed))
    tables = []
    for counts in (need, [more] * len(need)):
        t = torch.zeros((len(need), max(1, max(counts))), dtype=torch.int32)
        for b, n in enumerate(counts):
            t[b, :n] = torch.tensor([next(order) for _ in range(n)], dtype=torch.int32)
        tables.append(t.cuda())
    blocks = torch.zeros((pages, H, P * 9 * d // 8), dtype=torch.uint8, device="cuda")
    if fill:
        step = max(1, (1 << 26) // (H * P * d))              # bounded scratch
        for part in _parts(blocks, d):
            ch = _channels(H * d, gen).view(H, 1, d)
            for p in range(0, pages, step):
                n = min(step, pages - p)
                x = (_normal((n, H, P, d), gen) * ch).half()
                codes, ab = _pack(*_plain_quantize(x))
                part[0][p:p + n], part[1][p:p + n] = codes, ab
    return blocks, tables


def _parts(blocks, d):
    """Views of the blocks: ((K codes, K statistics), (V codes, V statistics)), the statistics as
    fp16 [pages][H][P][d/64][2]."""
    P = blocks.shape[-1] * 8 // (9 * d)
    nc, na = P * d // 2, P * d // GROUP * 4
    out = []
    for at in (0, nc + na):
        codes = blocks[..., at:at + nc].unflatten(-1, (P, d // 2))
        ab = blocks[..., at + nc:at + nc + na].view(torch.float16)
        out.append((codes, ab.unflatten(-1, (P, d // GROUP, 2))))
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, d, B = case["op"], case["d"], case["B"]
    st = {"case": dict(case), "scale": 1.0 / math.sqrt(d)}
    lens = _spread(case["lo"], case["hi"], B)
    if op in ("rope", "append"):
        order = _order(B, seed)
        lens = [lens[i] for i in order]
        past = _spread(max(0, case["past"] - case["past"] // 4), case["past"], B)
        past = [past[i] for i in _order(B, seed + 1)]
        rows = sum(lens)
        st["lens_list"], st["past_list"] = lens, past
        st["row_off"], st["pos"] = _offsets(lens), _ints(past)
        st["interleaved"] = case["interleaved"]
        most = max(p + n for p, n in zip(past, lens))
        if case["rot"]:
            st["angles"] = _angles(most, case["rot"], case["past"] > 8192)
        if op == "rope":
            wide = case["heads"] * d
            st["x"] = (_normal((rows, wide), gen) * _channels(wide, gen)).half()
            st["y"] = torch.empty_like(st["x"])
            return st
        wide = case["Hkv"] * d
        # K and V as the projection leaves them, side by side in one buffer
        buf = (_normal((rows, 2 * wide), gen) * _channels(2 * wide, gen)).half()
        st["k_new"], st["v_new"] = buf[:, :wide], buf[:, wide:]
        st["blocks"], (st["table"], _) = _pool(case, [p + n for p, n in zip(past, lens)], seed,
                                               False, gen)
        st["k_out"] = torch.empty((rows, wide), dtype=torch.float16, device="cuda")
        st["v_out"] = torch.empty_like(st["k_out"])
    elif op == "evict":
        lens = [lens[i] for i in _order(B, seed)]
        H, keep = case["Hkv"], case["keep"]
        st["lens_list"], st["lens"] = lens, _ints(lens)
        st["blocks"], (st["table"], st["dst"]) = _pool(case, lens, seed, True, gen, spare=keep)
        # weights received: few heavy positions, many light ones, some never seen
        acc = torch.exp(2.0 * _normal((B, H, max(lens)), gen))
        acc[torch.rand(acc.shape, device="cuda", generator=gen) < 0.05] = 0.0
        st["acc"] = acc
        st["kept"] = torch.empty((B, H, keep), dtype=torch.int32, device="cuda")
        st["acc_out"] = torch.zeros((B, H, keep), device="cuda")
        st["dst_lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
        left = [min(n, keep) for n in lens]
        st["row_off"], st["zero"] = _offsets(left), torch.zeros_like(st["lens"])
        st["k_out"] = torch.empty((sum(left), H * d), dtype=torch.float16, device="cuda")
        st["v_out"] = torch.empty_like(st["k_out"])
    else:
        nq = _query_rows(case)
        order = _order(B, seed)
        lens, nq = [lens[i] for i in order], [min(nq[i], lens[i]) for i in order]
        Hq, Hkv = case["Hq"], case["Hkv"]
        st["lens_list"], st["nq"] = lens, nq
        st["lens"], st["q_off"] = _ints(lens), _offsets(nq)
        st["blocks"], (st["table"], _) = _pool(case, lens, seed, True, gen)
        st["q"] = _normal((sum(nq), Hq * d), gen).half()
        st["groups"] = _groups(case, nq, lens, st["table"])
        if op == "attend":
            st["out"] = torch.empty_like(st["q"])
        else:
            # what attention says of these queries, and what the positions received before
            st["lse"] = torch.empty((sum(nq), Hq), device="cuda")
            for group in st["groups"]:
                s, ok = _plain_scores(st, group)
                z = torch.logsumexp(s.masked_fill(~ok, -math.inf), -1).permute(0, 3, 1, 2)
                st["lse"][group[1]] = z.flatten(0, 1).flatten(1)[group[2]]
            st["acc"] = torch.rand((B, Hkv, max(lens)), device="cuda", generator=gen)
            st["acc_out"] = torch.zeros_like(st["acc"])
    if own:
        from bit_compressed_throughput_gb300 import fg
        st["pages"] = fg.KVPagesQ4.of(st["blocks"], d)
        if op == "attend":
            n = fg.fg_attn_paged_workspace_bytes(st["pages"], case["Hq"], max(st["nq"]))
            st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------------------------ one pass


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from bit_compressed_throughput_gb300 import fg
    c = st["case"]
    op = c["op"]
    if op == "rope":
        fg.fg_rope(st["x"], c["d"], st["row_off"], st["pos"], st["angles"], st["y"],
                   interleaved=st["interleaved"])
        return st["y"]
    if op == "append":
        fg.fg_kv_append_q4_paged(st["k_new"], st["v_new"], st["row_off"], st["pos"], st["pages"],
                                 st["table"], angles=st.get("angles"),
                                 interleaved=st["interleaved"])
        fg.fg_kv_read_q4_paged(st["pages"], st["table"], st["row_off"], st["pos"], st["k_out"],
                               st["v_out"])
        return st["k_out"], st["v_out"]
    if op == "attend":
        fg.fg_attn_q4kv_paged(st["q"], st["q_off"], c["Hq"], st["pages"], st["table"], st["lens"],
                              st["scale"], st["out"], st["ws"], max_q=max(st["nq"]),
                              window=c["window"], sinks=c["sinks"])
        return st["out"]
    if op == "weights":
        fg.fg_attn_weights_q4_paged(st["q"], st["q_off"], c["Hq"], st["pages"], st["table"],
                                    st["lens"], st["scale"], st["lse"], st["acc"], st["acc_out"],
                                    max_q=max(st["nq"]), window=c["window"], sinks=c["sinks"])
        return st["acc_out"]
    fg.fg_kv_evict_q4_paged(st["pages"], st["table"], st["lens"], st["acc"], c["recent"], st["dst"],
                            st["kept"], st["acc_out"], st["dst_lens"])
    fg.fg_kv_read_q4_paged(st["pages"], st["dst"], st["row_off"], st["zero"], st["k_out"],
                           st["v_out"])
    return st["kept"], st["acc_out"], st["dst_lens"], st["k_out"], st["v_out"]


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
    return q[..., 0::2] | (q[..., 1::2] << 4), torch.stack((a, b), -1)


def _plain_restore(codes, ab):
    """fp16 values [..., d] of codes [..., d/2] and statistics [..., d/64][2]."""
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    a, b = ab[..., 0:1].float(), ab[..., 1:2].float()
    return (a + q.unflatten(-1, (-1, GROUP)) * ((b - a) / 15.0)).flatten(-2).half()


def _plain_rotate(x, d, angles, at, interleaved):
    """fp16 rows [n][heads*d], rotated by the table's rows `at`."""
    rot = 2 * angles.shape[1]
    x = x.unflatten(1, (-1, d))
    c, s = (angles[at][:, None, :, i] for i in (0, 1))
    head = x[..., :rot].float()
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        y = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((y.half(), x[..., rot:]), -1).flatten(1)


def _plain_rows(st):
    """Sequence and position of every packed row."""
    lens = torch.tensor(st["lens_list"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), lens,
                                  output_size=sum(st["lens_list"]))
    t = torch.arange(len(seq), device="cuda") - st["row_off"][seq] + st["pos"][seq]
    return seq, t.long()


def _plain_cells(st, table, seq, t):
    P = st["case"]["page"]
    return table[seq, t // P].long(), t % P


def _plain_read(st, cells):
    p, r = cells
    return tuple(_plain_restore(codes[p, :, r], ab[p, :, r]).flatten(1)
                 for codes, ab in _parts(st["blocks"], st["case"]["d"]))


def _groups(case, nq, lens, table):
    """Sequences with about as many query rows, to be padded to the most query rows and the longest
    context among them: which they are, their rows of q, the places of those rows in the padded
    [n][rows], query rows of each, pages, and the padded extents."""
    off = [0]
    for n in nq:
        off.append(off[-1] + n)
    todo = sorted(range(len(nq)), key=lambda b: (nq[b], lens[b]))
    out = []
    while todo:
        group = []
        while todo:                                          # bounded scratch
            b = todo[-1]
            rows = max(nq[x] for x in group + [b])
            keys = max(lens[x] for x in group + [b])
            if group and ((len(group) + 1) * case["Hq"] * rows * keys > 1 << 29
                          or 2 * nq[b] < rows):
                break
            group.append(todo.pop())
        rows, keys = max(nq[b] for b in group), max(lens[b] for b in group)
        at = [off[b] + i for b in group for i in range(nq[b])]
        place = [g * rows + i for g, b in enumerate(group) for i in range(nq[b])]
        which = torch.tensor(group, device="cuda")
        out.append((which, torch.tensor(at, device="cuda"), torch.tensor(place, device="cuda"),
                    torch.tensor([nq[b] for b in group], device="cuda"),
                    table[which, :(keys + case["page"] - 1) // case["page"]].long(), rows, keys))
    return out


def _plain_padded(x, group):
    """Packed rows [rows][w] in their places of a padded [n][rows][w], zeros elsewhere."""
    which, at, place, _, _, rows, _ = group
    y = torch.zeros((len(which) * rows, x.shape[1]), dtype=torch.float32, device="cuda")
    y[place] = x[at].float()
    return y.unflatten(0, (-1, rows))


def _plain_cached(st, group, which):
    """fp32 K (0) or V (1) [n][Hkv][keys][d] of a group."""
    codes, ab = _parts(st["blocks"], st["case"]["d"])[which]
    x = _plain_restore(codes[group[4]], ab[group[4]])        # [n][pages][Hkv][P][d]
    return x.transpose(1, 2).flatten(2, 3)[:, :, :group[6]].float()


def _plain_scores(st, group):
    """Scores [n][Hkv][G][rows][keys] of a group, and what its rows see of them."""
    c = st["case"]
    which, _, _, nq, _, rows, keys = group
    q = _plain_padded(st["q"], group).unflatten(2, (c["Hkv"], -1, c["d"])).permute(0, 2, 3, 1, 4)
    s = torch.matmul(q.flatten(2, 3), _plain_cached(st, group, 0).transpose(-1, -2))
    i = (torch.arange(rows, device="cuda") + (st["lens"][which] - nq)[:, None])[..., None]
    t = torch.arange(keys, device="cuda")
    ok = t <= i
    if c["window"]:
        ok = ok & ((t > i - c["window"]) | (t < c["sinks"]))
    return s.unflatten(2, (-1, rows)) * st["scale"], ok[:, None, None]


def _plain_attend(st):
    out = torch.empty_like(st["q"])
    for group in st["groups"]:
        s, ok = _plain_scores(st, group)
        s = s.masked_fill(~ok, -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
        l = p.sum(-1, keepdim=True)
        p = p / torch.where(l == 0, torch.ones_like(l), l)
        o = torch.matmul(p.flatten(2, 3), _plain_cached(st, group, 1)).unflatten(2, p.shape[2:4])
        o = o.permute(0, 3, 1, 2, 4).flatten(0, 1).flatten(1)     # [n * rows][Hq*d]
        out[group[1]] = o[group[2]].half()
    return out


def _plain_weights(st):
    c = st["case"]
    out = torch.zeros_like(st["acc"])
    for group in st["groups"]:
        which, _, place, _, _, rows, keys = group
        s, ok = _plain_scores(st, group)
        lse = _plain_padded(st["lse"], group).unflatten(2, (c["Hkv"], -1)).permute(0, 2, 3, 1)
        real = torch.zeros(len(which) * rows, dtype=torch.bool, device="cuda")
        real[place] = True
        p = torch.exp(s - lse[..., None])
        p = p.masked_fill(~(ok & real.view(-1, 1, 1, rows, 1)), 0.0)
        inside = torch.arange(keys, device="cuda") < st["lens"][which][:, None]
        new = st["acc"][which, :, :keys] + p.sum((2, 3))
        out[which, :, :keys] = torch.where(inside[:, None], new, torch.zeros_like(new))
    return out


def _plain_evict(st):
    c, (B, H, n) = st["case"], st["acc"].shape
    keep, P = c["keep"], c["page"]
    lens = st["lens"][:, None, None].long()
    t = torch.arange(n, device="cuda").expand(B, H, n)
    # the newest before everything, the heaviest next, ties to the lower position
    newest = (t >= lens - c["recent"]) | (lens <= keep)
    rank = torch.where(newest, torch.full_like(st["acc"], math.inf), st["acc"])
    rank = torch.where(t < lens, rank, torch.full_like(rank, -math.inf))
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    left = torch.clamp(lens, max=keep)
    slot = torch.arange(best.shape[-1], device="cuda")
    best = torch.sort(torch.where(slot < left, best, torch.full_like(best, n)), dim=-1).values
    kept = torch.full((B, H, keep), -1, dtype=torch.int32, device="cuda")
    kept[..., :best.shape[-1]] = torch.where(slot < left, best, torch.full_like(best, -1))
    at = kept.long().clamp(min=0)
    acc = torch.where(kept >= 0, torch.gather(st["acc"], 2, at), torch.zeros((), device="cuda"))
    # (slots past what is left hold position 0)
    b, h, dst = (torch.arange(x, device="cuda").view(v) for x, v in
                 ((B, (B, 1, 1)), (H, (1, H, 1)), (keep, (1, 1, keep))))
    p0, p1 = st["table"][b, at // P].long(), st["dst"][b, dst // P].long()
    for codes, ab in _parts(st["blocks"], c["d"]):
        codes[p1, h, dst % P] = codes[p0, h, at % P]
        ab[p1, h, dst % P] = ab[p0, h, at % P]
    dst_lens = left.flatten().int()
    row_b = torch.repeat_interleave(torch.arange(B, device="cuda"), dst_lens,
                                    output_size=st["k_out"].shape[0])
    row_t = torch.arange(len(row_b), device="cuda") - st["row_off"][row_b]
    k, v = _plain_read(st, _plain_cells(st, st["dst"], row_b, row_t.long()))
    return kept, acc, dst_lens, k, v


def _run_plain(st):
    c = st["case"]
    op, d = c["op"], c["d"]
    if op == "rope":
        return _plain_rotate(st["x"], d, st["angles"], _plain_rows(st)[1], st["interleaved"])
    if op == "append":
        seq, t = _plain_rows(st)
        k = st["k_new"]
        if c["rot"]:
            k = _plain_rotate(k, d, st["angles"], t, st["interleaved"])
        cells = _plain_cells(st, st["table"], seq, t)
        for new, (codes, ab) in zip((k, st["v_new"]), _parts(st["blocks"], d)):
            codes[cells[0], :, cells[1]], ab[cells[0], :, cells[1]] = _pack(
                *_plain_quantize(new.unflatten(1, (-1, d))))
        return _plain_read(st, cells)
    return {"attend": _plain_attend, "weights": _plain_weights, "evict": _plain_evict}[op](st)


# ------------------------------------------------------------------------------------ exact
#
# From the definitions, in 64 bits.  Codes, restored values and the rotated keys that are quantised
# are defined with one binary32 rounding per operation (and a last one to fp16): these roundings are
# made, everything else is 64-bit.


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


def _exact_turn(x, angles, at, heads, interleaved, rnd):
    """x [rows][heads][d] in 64 bits, turned pair by pair; rnd rounds every operation's result."""
    y = x.clone()
    half = angles.shape[1]
    for j in range(half):
        lo, hi = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        c = angles[at, j, 0].double()[:, None]
        s = angles[at, j, 1].double()[:, None]
        u, v = x[:, :, lo], x[:, :, hi]
        y[:, :, lo] = rnd(rnd(u * c) - rnd(v * s))
        y[:, :, hi] = rnd(rnd(u * s) + rnd(v * c))
    return y


def _exact_positions(st):
    return torch.cat([torch.arange(p, p + n) for p, n in zip(st["past_list"],
                                                            st["lens_list"])]).cuda()


def _exact_pages(st, b, n, which, table="table"):
    """64-bit values [Hkv][n][d] of sequence b's first n positions, K (0) or V (1)."""
    c = st["case"]
    P, d = c["page"], c["d"]
    raw = st["blocks"][st[table][b, :(n + P - 1) // P].long()]           # [pages][H][bytes]
    half = raw.shape[2] // 2
    raw = raw[:, :, which * half:which * half + half]
    byte = raw[:, :, :P * d // 2].long().reshape(raw.shape[0], raw.shape[1], P, d // 2)
    code = torch.empty(byte.shape[:3] + (d,), dtype=torch.float64, device=raw.device)
    code[..., 0::2] = (byte % 16).double()
    code[..., 1::2] = (byte // 16).double()
    word = raw[:, :, P * d // 2:].contiguous().view(torch.float16).double()
    word = word.reshape(raw.shape[0], raw.shape[1], P, d // GROUP, 2)
    x = _exact_values(code.unflatten(3, (-1, GROUP)), word[..., 0:1], word[..., 1:2]).flatten(3)
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_hidden(first, count, n, window, sinks):
    i = torch.arange(first, first + count, device="cuda").view(count, 1)
    t = torch.arange(n, device="cuda").view(1, n)
    hidden = t > i
    if window > 0:
        hidden = hidden | ((t <= i - window) & (t >= sinks))
    return hidden


def exact(case, seed):
    st = prepare(case, seed)
    op, d, B = case["op"], case["d"], case["B"]
    if op == "rope":
        at = _exact_positions(st)
        heads = case["heads"]
        return torch.cat([
            _exact_turn(st["x"][r:r + 1024].double().view(-1, heads, d), st["angles"],
                        at[r:r + 1024], heads, case["interleaved"], lambda v: v).flatten(1)
            for r in range(0, len(at), 1024)])
    if op == "append":
        at = _exact_positions(st)
        heads, outs = case["Hkv"], []
        for new, turned in ((st["k_new"], case["rot"]), (st["v_new"], 0)):
            parts = []
            for r in range(0, len(at), 1024):
                x = new[r:r + 1024].double().view(-1, heads, d)
                if turned:
                    x = _exact_turn(x, st["angles"], at[r:r + 1024], heads, case["interleaved"],
                                    _f32).half().double()
                parts.append(_exact_values(*_exact_codes(x.reshape(x.shape[0], -1, GROUP)))
                             .reshape(x.shape[0], -1))
            outs.append(torch.cat(parts))
        return tuple(outs)
    if op == "evict":
        H, keep = case["Hkv"], case["keep"]
        acc = torch.zeros((B, H, keep), dtype=torch.float64, device="cuda")
        outs = [[], []]
        for b, n in enumerate(st["lens_list"]):
            a = st["acc"][b, :, :n]
            old = n - min(n, case["recent"])
            order = torch.argsort(a[:, :old].double(), dim=1, descending=True, stable=True)
            at = order[:, :max(0, min(n, keep) - (n - old))]
            at = torch.cat((at, torch.arange(old, n, device="cuda").expand(H, n - old)), 1)
            at = at[:, -min(n, keep):].sort(dim=1).values
            acc[b, :, :at.shape[1]] = a.double().gather(1, at)
            for x, out in enumerate(outs):
                v = _exact_pages(st, b, n, x)
                out.append(v.gather(1, at[:, :, None].expand(-1, -1, d)).transpose(0, 1).flatten(1))
        return None, acc, None, torch.cat(outs[0]), torch.cat(outs[1])
    Hq, Hkv = case["Hq"], case["Hkv"]
    G = Hq // Hkv
    if sum(4.0 * nq * n * Hq * d for nq, n in zip(st["nq"], st["lens_list"])) > 6e12:
        return None
    if op == "attend":
        res = torch.empty((sum(st["nq"]), Hq * d), dtype=torch.float64, device="cuda")
    else:
        res = torch.zeros(st["acc"].shape, dtype=torch.float64, device="cuda")
    q0 = 0
    for b, (nq, n) in enumerate(zip(st["nq"], st["lens_list"])):
        k = _exact_pages(st, b, n, 0)
        v = _exact_pages(st, b, n, 1) if op == "attend" else None
        if op == "weights":
            res[b, :, :n] = st["acc"][b, :, :n].double()
        step = max(1, (1 << 27) // (Hq * n))
        for r in range(0, nq, step):
            rr = slice(q0 + r, q0 + min(nq, r + step))
            q = st["q"][rr].double().view(-1, Hkv, G, d).permute(1, 2, 0, 3)
            e = (q.flatten(1, 2) @ k.mT).unflatten(1, (G, -1)) * st["scale"]
            e.masked_fill_(_exact_hidden(n - nq + r, q.shape[2], n, case["window"],
                                         case["sinks"]), -math.inf)
            if op == "attend":
                o = torch.softmax(e, dim=-1).flatten(1, 2) @ v
                res[rr] = o.unflatten(1, (G, -1)).permute(2, 0, 1, 3).flatten(1)
            else:
                z = st["lse"][rr].double().view(-1, Hkv, G).permute(1, 2, 0)
                res[b, :, :n] += torch.exp(e - z[..., None]).sum((1, 2))
        q0 += nq
    return res
