"""The binding's own checks, and what it does without a GPU or without torch."""
import os
import subprocess
import sys

import pytest

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
