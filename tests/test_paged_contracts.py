"""What the whole-layer calls promise around their mathematics, as far as the host and the sources show it: barriers that
are made before they are used, first calls from several threads, calls without tokens."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_paged_kv_page_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu"))))
def test_barriers_are_made_before_any_warp_uses_them(name):
    """Between the making of a kernel's mbarriers and the first arming of one stands a barrier of the block, or one of
    the warp where each warp makes its own."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for made in re.finditer(r"mbar_init_fence\(\)", src):
        begin = src.rfind("mbar_init(", 0, made.start())
        first = re.search(r"__syncthreads\(\)|__syncwarp\(\)|mbar_arrive\w*\(|tma_load_\w+\(|cp_bulk\w*\(", src[made.end():])
        assert first, "the barriers are never used"
        met = first.group()
        assert met.startswith("__sync"), f"{met} before the threads have met"
        if met == "__syncwarp()":
            assert "[warp]" in src[begin:made.start()], "a warp met, but the barriers are not its own"
