"""The 16-bit and page tests through the bounds-checking debug library: the
same answers, and no index past its buffer (KVQ_DEVERR_BOUNDS stays clear, as
the tests ask of every error word)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_debug_library_over_16_bit_pages_and_page_calls():
    lib = os.path.join(os.path.dirname(HERE), "sub_byte_quantized_write_gb300", "libkvq_debug.so")
    if not os.path.exists(lib):
        pytest.fail("libkvq_debug.so is not built (build() makes it)")
    files = [os.path.join(HERE, f) for f in ("test_gpu_decode16.py", "test_gpu_pages.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", *files],
                       env=dict(os.environ, KVQ_BOUNDS_CHECK="1"), capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
