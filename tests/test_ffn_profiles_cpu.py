"""The committed trace and counters of the 16-bit feed-forward operators name the sources
they were taken on: the digest of the code, without comments, of every csrc/ffn* file."""
import glob
import hashlib
import os

import pytest

import bench


@pytest.mark.parametrize("name", ["ffn_kernel_trace.txt", "ffn_counters.txt"])
def test_taken_on_the_sources_as_they_are(name):
    csrc = os.path.join(bench.ROOT, "bit_quantized_matmul_col_amd", "csrc")
    h = hashlib.sha256()
    for p in sorted(glob.glob(os.path.join(csrc, "ffn*"))):
        with open(p, encoding="utf-8") as f:
            h.update(bench._code_only(f.read()).encode())
    with open(os.path.join(bench.PROFILES, name), encoding="utf-8") as f:
        digests = [line.split(":", 1)[1].strip() for line in f
                   if line.startswith("kernel_source_digest:")]
    assert digests == [h.hexdigest()[:16]]
