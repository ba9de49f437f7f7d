"""The paged operators as a program runs them: on streams, in captured graphs, beside one another, over
batches of single tokens and pieces, and in pools past 32-bit offsets."""
import math

import numpy as np
import pytest
import torch

import fg_synth
from paged_util import fill, i32, need, offsets, tables
from parity_util import dev, host, lib
from test_gpu_paged import check_attend, paged_case, run_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg():
    return lib()


class Program:
    """Rotary positions, append, attention, weights and eviction over static buffers."""

    def __init__(self, fg, seed, B=3, d=64, H=2, G=2, P=16, cap=640, rows=300, keep=64):
        self.fg, self.B, self.d, self.H, self.Hq = fg, B, d, H, H * G
        self.h, self.cap, self.rows, self.keep = H * d, cap, rows, keep
        rng = np.random.default_rng(seed)
        width = cap // P
        pages = B * (width + keep // P)
        self.pool = fg.KVPagesQ4(pages, P, self.h, H)
        self.pool.blocks.zero_()
        order = rng.permutation(pages).astype(np.int32)
        self.table = dev(order[:B * width].reshape(B, width).copy())
        self.after = dev(order[B * width:].reshape(B, keep // P).copy())
        self.qkv = dev(fg_synth.random_fp16((rows, (self.Hq + 2 * H) * d), seed=seed))
        self.src = self.qkv.clone()
        self.off, self.pos, self.lens = i32([0] * (B + 1)), i32([0] * B), i32([0] * B)
        self.angles = torch.empty((cap, d // 2, 2), device="cuda")
        fg.fg_rope_table(self.angles, 1e4)
        self.out = torch.zeros((rows, self.Hq * d), dtype=torch.float16, device="cuda")
        self.lse = torch.zeros((rows, self.Hq), device="cuda")
        self.ws = torch.full((fg.fg_attn_paged_workspace_bytes(self.pool, self.Hq, rows),), 255,
                             dtype=torch.uint8, device="cuda")
        self.acc = torch.zeros((B, H, cap), device="cuda")
        self.kept = torch.zeros((B, H, keep), dtype=torch.int32, device="cuda")
        self.acc_out = torch.zeros((B, H, keep), device="cuda")
        self.dst_lens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def extents(self, nq, pos):
        self.off.copy_(i32(offsets(nq)))
        self.pos.copy_(i32(pos))
        self.lens.copy_(i32([n + p for n, p in zip(nq, pos)]))

    def run(self):
        fg, h, q = self.fg, self.h, self.qkv[:, :self.Hq * self.d]
        k, v = self.qkv[:, self.Hq * self.d:][:, :h], self.qkv[:, self.Hq * self.d + h:]
        self.qkv.copy_(self.src)
        fg.fg_rope(q, self.d, self.off, self.pos, self.angles, q)
        fg.fg_kv_append_q4_paged(k, v, self.off, self.pos, self.pool, self.table, angles=self.angles)
        fg.fg_attn_q4kv_paged(q, self.off, self.Hq, self.pool, self.table, self.lens, 0.125, self.out,
                              self.ws, lse=self.lse)
        fg.fg_attn_weights_q4_paged(q, self.off, self.Hq, self.pool, self.table, self.lens, 0.125,
                                    self.lse, self.acc, self.acc)
        fg.fg_kv_evict_q4_paged(self.pool, self.table, self.lens, self.acc, 8, self.after, self.kept,
                                self.acc_out, self.dst_lens)

    def results(self):
        # (what the calls leave undefined, behind a sequence's kept entries, is left out)
        n = host(self.dst_lens)
        kept, acc = host(self.kept), host(self.acc_out)
        return [host(self.out), host(self.lse), host(self.acc), n] + \
            [x[b, :, :n[b]] for b in range(self.B) for x in (kept, acc)] + \
            [host(self.pool.blocks)]


STEPS = [([130, 1, 40], [0, 0, 0]), ([1, 1, 1], [130, 1, 40]), ([70, 0, 200], [131, 2, 41]),
         ([1, 3, 1], [201, 2, 241])]


def all_equal(a, b):
    for i, (x, y) in enumerate(zip(a, b)):
        assert np.array_equal(x, y, equal_nan=x.dtype.kind == "f"), i


def test_another_stream_and_graph_replays(fg):
    """The same bits from eager calls on the default stream, on another one, and from one captured
    graph replayed with other extents in the same buffers."""
    ways = [Program(fg, 5) for _ in range(3)]
    side = torch.cuda.Stream()
    ways[2].extents(*STEPS[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ways[2].run()
    for nq, pos in STEPS:
        for p in ways:
            p.extents(nq, pos)
        torch.cuda.synchronize()
        ways[0].run()
        with torch.cuda.stream(side):
            ways[1].run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        fg.fg_check_device_error()
        want = ways[0].results()
        for p in ways[1:]:
            all_equal(want, p.results())


def test_two_programs_at_once(fg):
    """Two programs on two streams, each with buffers and scratch of its own, do not meet."""
    alone = [Program(fg, s, rows=340, cap=1280) for s in (7, 8)]
    both = [Program(fg, s, rows=340, cap=1280) for s in (7, 8)]
    steps = ([200, 1, 130], [800, 500, 30])
    for p in alone + both:
        p.extents(*steps)
    torch.cuda.synchronize()
    for p in alone:
        for _ in range(5):
            p.run()
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(5):
        for s, p in zip(streams, both):
            with torch.cuda.stream(s):
                p.run()
    torch.cuda.synchronize()
    fg.fg_check_device_error()
    for a, b in zip(alone, both):
        all_equal(a.results(), b.results())


@pytest.mark.parametrize("d,H,G", [(128, 2, 1), (64, 2, 4), (128, 1, 5), (64, 1, 6), (128, 1, 8),
                                   (64, 1, 9)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_single_tokens_beside_pieces(fg, d, H, G, window, sinks):
    """Steps and pieces in one batch give what each gives in a batch of its own kind, and the
    definition's values; the log-sum-exp is every row's."""
    lens, nq, P = [300, 1, 77, 1500, 129, 0, 40, 2], [1, 1, 20, 1, 129, 0, 1, 2], 32
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, lens, nq, 17 + G, G)
    scale, width = 1.0 / math.sqrt(d), H * G * d
    t, kw = dev(q)[:, :width], dict(window=window, sinks=sinks)
    out, z = run_attend(fg, t, q_off, H * G, pool, table, lens, scale, max_q=max(nq), **kw)
    fg.fg_check_device_error()
    check_attend(out, z, q, q_off, H * G, k, v, table, lens, scale, window, sinks)
    one = [b for b in range(len(nq)) if nq[b] == 1]
    rows = [q_off[b] for b in one]
    alone, za = run_attend(fg, t[rows], offsets([1] * len(one)), H * G, pool,
                           np.ascontiguousarray(table[one]), [lens[b] for b in one], scale, max_q=1,
                           **kw)
    fg.fg_check_device_error()
    check_attend(alone, za, q[rows], offsets([1] * len(one)), H * G, k, v, table[one],
                 [lens[b] for b in one], scale, window, sinks)
    outside = np.r_[0:q_off[0], q_off[-1]:len(q)]
    assert np.all(host(out)[outside] == 7.0) and np.all(host(z)[outside] == 7.0)


@pytest.mark.parametrize("nq", [1, 2])
def test_many_sequences(fg, nq):
    """More sequences than a block has threads, of 0 to 40 positions."""
    rng = np.random.default_rng(9)
    B, d, H, G, P = 1500, 64, 1, 2, 16
    lens = rng.integers(0, 41, B).tolist()
    rows = [min(nq, n) for n in lens]
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, lens, rows, 23, G)
    out, z = run_attend(fg, dev(q)[:, :G * d], q_off, G, pool, table, lens, 0.125, max_q=nq)
    fg.fg_check_device_error()
    check_attend(out, z, q, q_off, G, k, v, table, lens, 0.125)
    acc = torch.zeros((B, H, 48), device="cuda")
    fg.fg_attn_weights_q4_paged(dev(q)[:, :G * d], i32(q_off), G, pool, dev(table), i32(lens), 0.125, z,
                                acc, acc, max_q=nq)
    fg.fg_check_device_error()
    # every query head hands out a weight of 1 in all.  Its log-sum-exp and its weights come from the
    got = host(acc).sum(-1)[:, 0]
    assert np.all(np.abs(got - G * np.asarray(rows)) <= 0.1 * G * np.asarray(rows))


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5)])
def test_many_blocks(fg, window, sinks):
    """So many key tiles that every multiprocessor has several blocks, whole ones and cut ones."""
    d, H, G, P = 64, 32, 1, 64
    lens, nq = [1300, 900, 1177, 640, 1290, 1, 1024, 799], [200, 300, 129, 128, 257, 1, 64, 255]
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, lens, nq, 61, G)
    out, z = run_attend(fg, dev(q)[:, :H * G * d], q_off, H * G, pool, table, lens, 0.125,
                        max_q=max(nq), window=window, sinks=sinks)
    fg.fg_check_device_error()
    check_attend(out, z, q, q_off, H * G, k, v, table, lens, 0.125, window, sinks)


def test_pool_past_32_bits(fg):
    """Pages whose offsets pass 2^32 bytes hold what pages at the start hold, bit for bit."""
    d, H, G, P, lens, nq = 128, 2, 2, 64, [200, 333], [70, 1]
    pages = 5 * 2 ** 30 // (H * P * 9 * d // 8)
    used = sum(need(lens, P))
    low = np.full((2, 6), -1, np.int32)
    for b, n in enumerate(need(lens, P)):
        low[b, :n] = b * 6 + np.arange(n)
    high = np.where(low < 0, low, pages - 1 - low)
    keep = 128
    to = [np.array([[20, 21], [22, 23]], np.int32), np.array([[pages - 30, pages - 31],
                                                               [pages - 32, pages - 33]], np.int32)]
    pool = fg.KVPagesQ4(pages, P, H * d, H)
    assert (pages - 40) * H * P * 9 * d // 8 > 2 ** 32 and used < 20
    new = dev(fg_synth.random_fp16((sum(lens), 2 * H * d), seed=1))
    q = dev(fg_synth.random_fp16((sum(nq), H * G * d), seed=2))
    got = []
    for table, dst in zip((low, high), to):
        fg.fg_kv_append_q4_paged(new[:, :H * d], new[:, H * d:], i32(offsets(lens)), i32([0, 0]), pool,
                                 dev(table))
        back = torch.zeros_like(new)
        fg.fg_kv_read_q4_paged(pool, dev(table), i32(offsets(lens)), i32([0, 0]), back[:, :H * d],
                               back[:, H * d:])
        acc = torch.zeros((2, H, 333), device="cuda")
        res = [back]
        for most, qq, off in ((70, q, offsets(nq)), (1, q[69:], offsets([1, 1]))):
            out, z = run_attend(fg, qq, off, H * G, pool, table, lens, 0.1, max_q=most)
            fg.fg_attn_weights_q4_paged(qq, i32(off), H * G, pool, dev(table), i32(lens), 0.1, z, acc,
                                        acc, max_q=most)
            res += [out, z, acc.clone()]
        kept = torch.zeros((2, H, keep), dtype=torch.int32, device="cuda")
        acc_out = torch.zeros((2, H, keep), device="cuda")
        n = torch.zeros(2, dtype=torch.int32, device="cuda")
        fg.fg_kv_evict_q4_paged(pool, dev(table), i32(lens), acc, 16, dev(dst), kept, acc_out, n)
        fg.fg_kv_read_q4_paged(pool, dev(dst), i32([0, 128, 256]), i32([0, 0]), back[:256, :H * d],
                               back[:256, H * d:])
        fg.fg_check_device_error()
        got.append([host(x) for x in res + [kept, acc_out, n, back]])
    all_equal(*got)


def test_sequences_that_share_pages(fg):
    """A common beginning in the same pages: each sequence gets what it gets with pages of its own."""
    d, H, G, P = 64, 2, 2, 32
    lens, nq = [200, 170, 129], [40, 1, 3]
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, lens, nq, 41, G)
    t, Hq = dev(q)[:, :H * G * d], H * G
    blocks = pool.blocks.view(pool.pages, -1)
    for b in (1, 2):                                         # copies of sequence 0's first 128
        blocks[table[b, :4].tolist()] = blocks[table[0, :4].tolist()]
    shared = table.copy()
    shared[1:, :4] = table[0, :4]
    got = []
    for tab in (table, shared):
        out, z = run_attend(fg, t, q_off, Hq, pool, tab, lens, 0.125, max_q=max(nq))
        acc = torch.zeros((3, H, 200), device="cuda")
        fg.fg_attn_weights_q4_paged(t, i32(q_off), Hq, pool, dev(tab), i32(lens), 0.125, z, acc, acc,
                                    max_q=max(nq))
        fg.fg_check_device_error()
        got.append([host(out), host(z), host(acc)])
    all_equal(*got)
