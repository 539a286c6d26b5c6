"""Evictions that are the first of their process: whether a call is taken does not hang on what was called
before it.  A kernel that uses more than 48 KB of shared memory, its own declarations counted in, has to be opted in;
these tables and counts lie around that border (a table's slots, and two bytes for each that stays, beside some
18 KB that the kernel for wide tables declares)."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# (slots of the table, keep): 31136 bytes, 31152 (48 KB are passed), 32768, and 32784
SIZES = {64: [(30208, 464), (30208, 465), (16384, 8192), (16384, 8193)],
         128: [(24576, 4096), (30208, 464)],
         256: [(28672, 2048), (24576, 3281)]}


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_first_evictions_of_a_process(dim):
    from quantised_decode_mat_gb300 import build as qbuild
    qbuild.build()
    run = "from tests.test_gpu_kv4 import evict_case\n"
    for slots, keep in SIZES[dim]:  # (the table is a page wider than its longest sequence needs)
        run += f"s, _ = evict_case([{slots - 70}, 300], {keep}, 4, 100, 1, {dim}, 64, seed={keep})\n"
        run += f"assert s.table.shape[1] * 64 == {slots}\n"
    got = subprocess.run([sys.executable, "-c", run], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stderr[-2000:]
