"""Orders between threads that no run can show to be missing, looked up in the
kernels' source."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_latent_kv_15_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def code(path):
    """The source without its comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(p) for p in SOURCES])
def test_plain_writes_for_the_other_cta_are_released_to_the_cluster(path):
    # A thread that fences its own shared-memory writes for the tensor cores and then
    # signals a barrier of the other CTA: the plain remote arrival is ordered in its
    # own CTA alone.
    for m in re.finditer(r"fence_proxy_async_smem\(\);", code(path)):
        behind = code(path)[m.end():m.end() + 600].split("fence_proxy_async_smem")[0]
        signals = re.findall(r"\b(mbar_arrive\w*|st_async\w*|tma_store\w*|named_bar\w*|mma_ts)\s*\(", behind)
        assert not signals or signals[0] != "mbar_arrive_remote", behind
