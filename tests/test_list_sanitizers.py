"""The host paths of the tensor-list and balance-loss entry points under AddressSanitizer and UBSan (CPU)."""
import os
import subprocess

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
EXE = os.path.join(HERE, "c", "list_checks")


@pytest.mark.skipif(torch.cuda.device_count() != 0, reason="made-up device addresses: CPU-only test")
def test_refusals_and_overlap_search_under_the_sanitizers():
    if not os.path.exists(EXE):
        pytest.skip("list_checks not built (no sanitizer runtime in the toolchain)")
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="halt_on_error=1")
    out = subprocess.run([EXE], env=env, capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip().endswith("ok"), out.stdout[-2000:] + out.stderr[-2000:]
