"""The binding's own checks, and what it does without a GPU or without torch."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def fg():
    import __graft_entry__ as g
    g.build()
    from bit_compressed_throughput_gb300 import fg as mod
    return mod


def test_import_needs_no_torch(fg):
    """The binding loads, and the library's host-side calls work, where torch cannot be imported;
    importing it imports no torch."""
    code = (
        "import sys\n"
        "{}\n"
        "from bit_compressed_throughput_gb300 import fg\n"
        "assert fg.fg_gemm_workspace_bytes(16, 256, 256) >= 0\n"
        "assert fg.lib.fg_status_string(0) == b'ok'\n"
        "assert sys.modules.get('torch') is None\n")
    for first in ("sys.modules['torch'] = None", ""):
        subprocess.run([sys.executable, "-c", code.format(first)], cwd=ROOT, check=True)


def calls_on(fg, cache):
    """The calls that take this cache, with arguments that fit its B, h and H."""
    rows = torch.zeros((4, cache.h), dtype=torch.float16)
    q = torch.zeros((cache.B, cache.h), dtype=torch.float16)
    off = torch.zeros(cache.B + 1, dtype=torch.int32)
    pos = torch.zeros(cache.B, dtype=torch.int32)
    return [lambda: fg.fg_kv_append_q4_ragged(rows, rows, off, pos, cache),
            lambda: fg.fg_kv_read_q4_ragged(cache, off, pos, rows, None),
            lambda: fg.fg_decode_attn_q4kv_window(q, cache.H, cache, pos, 0.1, q)]


@pytest.mark.parametrize("change", [
    dict(cap=32), dict(B=3), dict(h=256, H=2), dict(d=64), dict(H=0),
    dict(k_codes=torch.zeros((2, 1, 15, 64), dtype=torch.uint8)),
    dict(v_codes=torch.zeros((2, 1, 16, 64), dtype=torch.int8)),
    dict(k_ab=torch.zeros((2, 1, 16, 1), dtype=torch.int32)),
    dict(v_ab=torch.zeros((2, 1, 16, 4), dtype=torch.int32)[..., ::2]),
    dict(v_ab=torch.zeros((2, 1, 16, 2), dtype=torch.int32, device="meta")),
])
def test_cache_tensors_that_do_not_fit(fg, change):
    """A cache whose tensors do not have the sizes that it says is refused by the calls that would
    read and write it by those sizes, also when it was in order before."""
    cache = fg.KVCacheQ4(2, 16, 128, 1, device="cpu")
    cache.check()
    for name, value in change.items():
        setattr(cache, name, value)
    with pytest.raises(ValueError, match="cache"):
        cache.check()
    if change.get("H", 1):
        for call in calls_on(fg, cache):
            with pytest.raises(ValueError):
                call()


def test_cache_tensors_set_anew(fg):
    """A cache whose capacity and tensors were replaced by ones that fit is in order."""
    cache = fg.KVCacheQ4(2, 16, 128, 1, device="cpu")
    cache.cap = 48
    cache.k_codes = torch.zeros((2, 1, 48, 64), dtype=torch.uint8)
    cache.v_codes = torch.zeros_like(cache.k_codes)
    with pytest.raises(ValueError, match="cache.k_ab"):
        cache.check()
    cache.k_ab = torch.zeros((2, 1, 48, 2), dtype=torch.int32)
    cache.v_ab = torch.zeros_like(cache.k_ab)
    cache.check()


@pytest.mark.parametrize("name", ["window", "sinks"])
@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 5, 1 << 62, -(1 << 32)])
def test_window_of_more_than_32_bits(fg, name, value):
    """2^32 + 5 is not a window of 5, and 2^32 not none at all."""
    cache = fg.KVCacheQ4(2, 16, 128, 1, device="cpu")
    q = torch.zeros((2, 128), dtype=torch.float16)
    off, lens = torch.tensor([0, 1, 2], dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="32-bit"):
        fg.fg_decode_attn_q4kv_window(q, 1, cache, lens, 0.1, q, **{name: value})
    with pytest.raises(ValueError, match="32-bit"):
        fg.fg_prefill_attn_window(q, off, q, q, off, 1, 1, 0.1, q.clone(), **{name: value})
