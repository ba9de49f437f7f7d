"""Outputs of the paged operators that lie over their inputs or over one another are refused (no GPU
needed: validation fails before any address is used)."""
import ctypes as C

import pytest

Q, OUT, LSE, ACC, FAR = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000


@pytest.fixture(scope="module")
def fg():
    import __graft_entry__ as g
    g.build()
    from bit_compressed_throughput_gb300 import fg as mod
    return mod


def test_attention(fg):
    kv = fg.fg_kvpages(0x1000000, 8, 32, 256, 2)

    def call(out=OUT, lse=LSE, qs=512, os=512):              # 8 rows of 4 heads of 128; ws too small
        return fg.lib.fg_attn_q4kv_paged(Q, qs, 8, FAR, 4, 4, C.byref(kv), FAR, 4, FAR, 2, 0, 0, 0.1,
                                         out, os, lse, None, 0, None)

    assert call() == call(lse=None) == call(out=Q) == fg.FG_ERR_WORKSPACE
    assert call(lse=OUT + 8 * 1024) == call(lse=Q - 128) == fg.FG_ERR_WORKSPACE      # side by side
    for lse in (OUT, OUT + 8 * 1024 - 4, OUT - 124, Q, Q + 4096):
        assert call(lse=lse) == fg.FG_ERR_ARG, hex(lse)
    # between the rows of a wider buffer
    assert call(lse=OUT + 1024, os=1024) == fg.FG_ERR_WORKSPACE
    assert call(lse=OUT + 1024 + 1000, os=1024) == fg.FG_ERR_ARG


def test_weights(fg):
    kv = fg.fg_kvpages(0x1000000, 8, 32, 256, 2)

    def call(acc=ACC, out=OUT, lse=LSE, stride=64):          # acc: 2 x 2 x 64 sums, 1 KB
        return fg.lib.fg_attn_weights_q4_paged(Q, 512, 8, FAR, 4, 4, C.byref(kv), FAR, 4, FAR, 2, 0, 0,
                                               0.1, lse, acc, out, stride, None)

    # (a call that passes would be made where there is a GPU: none passes here)
    for kw in (dict(out=Q), dict(out=Q + 8 * 1024 - 4), dict(out=Q - 1020), dict(out=LSE),
               dict(out=LSE + 124), dict(out=LSE - 1020), dict(out=ACC + 64), dict(out=ACC - 1020),
               dict(acc=None, out=LSE), dict(acc=OUT, out=OUT, lse=OUT + 1020)):
        assert call(**kw) == fg.FG_ERR_ARG, kw


def test_evict(fg):
    kv = fg.fg_kvpages(0x1000000, 8, 32, 256, 2)
    kept, out, lens = 0x60000, 0x70000, 0x80000              # 2 x 2 x 32 words, 512 bytes; 8 bytes

    def call(table=0xA0000, dst=0xB0000, n=0xC0000, acc=ACC, kept=kept, acc_out=out, dl=lens):
        return fg.lib.fg_kv_evict_q4_paged(C.byref(kv), table, 4, 2, n, acc, 64, 32, 8, dst, 4, kept,
                                           acc_out, dl, None)

    for kw in (dict(kept=out), dict(kept=out + 508), dict(acc_out=kept - 508), dict(dl=kept + 508),
               dict(dl=out - 4), dict(kept=ACC), dict(kept=ACC + 1020), dict(acc_out=ACC - 508),
               dict(dl=ACC + 4), dict(dl=0xC0004), dict(kept=0xC0000), dict(acc_out=0xC0004),
               dict(kept=0xA0000), dict(acc_out=0xB0000 + 28), dict(dl=0xB0000 + 28),
               dict(dl=0xA0000 - 4)):
        assert call(**kw) == fg.FG_ERR_ARG, kw


def test_extents_past_64_bits(fg):
    """Strides whose product with the sequences and heads passes 64 bits still cover what lies in them."""
    kv = fg.fg_kvpages(0x1000000, 8, 32, 256, 2)
    for stride in (1 << 46, 1 << 47, (1 << 60) - 1):

        def weights(acc, lse):
            return fg.lib.fg_attn_weights_q4_paged(Q, 512, 8, FAR, 4, 4, C.byref(kv), FAR, 4, FAR, 65535, 0,
                                                   0, 0.1, lse, acc, OUT, stride, None)

        assert weights(None, 0x7000000000) == fg.FG_ERR_ARG, hex(stride)
        assert weights(0x7000000000, LSE) == fg.FG_ERR_ARG, hex(stride)

        def evict(kept):
            return fg.lib.fg_kv_evict_q4_paged(C.byref(kv), 0x9000, 4, 2, 0xB000, OUT, stride, 32, 8,
                                               0xA000, 4, kept, 0x8000, 0x6000, None)

        assert evict(0x7000000000) == fg.FG_ERR_ARG, hex(stride)
    # rows that no address space holds
    assert fg.lib.fg_attn_weights_q4_paged(Q, 512, 8, FAR, 4, 4, C.byref(kv), FAR, 4, FAR, 2, 0, 0, 0.1, LSE,
                                           ACC, OUT, 1 << 61, None) == fg.FG_ERR_SHAPE
    assert fg.lib.fg_kv_evict_q4_paged(C.byref(kv), 0x9000, 4, 2, 0xB000, OUT, 1 << 61, 32, 8, 0xA000, 4,
                                       0x7000, 0x8000, 0x6000, None) == fg.FG_ERR_SHAPE
