"""The refusals and sizes of the gated delta rule's and the block norms' calls with a C ABI layer that is
instrumented for the host (as the other layers' are)."""
import os

import pytest


def test_block_refusals_under_asan_ubsan(tmp_path):
    san = pytest.importorskip("tests.test_host_sanitizers")
    lib, runtime = san._sanitized_abi(tmp_path)
    files = [os.path.join(san.ROOT, "tests", n) for n in ("test_blocks_host.py", "test_delta_host.py")]
    code = f"""
import sys
sys.path.insert(0, {san.ROOT!r})
from linear_recurrent_sequence_mamba_amd import binding as m3
m3.LIB_PATH = {lib!r}
import pytest
sys.exit(pytest.main([*{files!r}, "-q", "-s", "-p", "no:cacheprovider", "-k", "refus or workspace or exports"]))
"""
    r = san._run(code, runtime)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-3000:])
    assert " passed" in r.stdout and int(r.stdout.split(" passed")[0].split()[-1]) >= 8, r.stdout[-500:]
