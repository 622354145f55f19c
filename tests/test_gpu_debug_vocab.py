"""The debug build (-DTXL_DEBUG) on the token embedding and the log probabilities: in a child
process that loads it, their tests pass with every device-side index check active (places of
sorted positions)."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


def test_vocab_tests_pass_with_index_checks():
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/test_gpu_embed.py", "tests/test_gpu_logprob.py"],
                       cwd=ROOT, env=dict(os.environ, TXL_DEBUG_LIB="1"), capture_output=True, text=True,
                       timeout=1800)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
