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


FIRST_CALLS = r"""
#include <chrono>
#include <cstdio>
#include <thread>

#include "tma_map.h"

// A lookup that takes its time, in place of the runtime's.
extern "C" cudaError_t CUDARTAPI cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned int, unsigned long long,
                                                                  cudaDriverEntryPointQueryResult* q) {
  std::this_thread::sleep_for(std::chrono::milliseconds(300));
  *p = reinterpret_cast<void*>(0x1000);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

int main() {
  sa::EncodeFn seen[2];
  std::thread first([&] { seen[0] = sa::encode_fn(); });
  std::this_thread::sleep_for(std::chrono::milliseconds(100));
  std::thread second([&] { seen[1] = sa::encode_fn(); });
  first.join();
  second.join();
  std::printf("%d%d\n", seen[0] != nullptr, seen[1] != nullptr);
}
"""


def test_first_calls_from_two_threads_both_find_the_tensor_map_encoder(tmp_path):
    import subprocess
    from sparse_paged_kv_page_gb300 import build as B
    src, exe = tmp_path / "first_calls.cpp", tmp_path / "first_calls"
    src.write_text(FIRST_CALLS)
    subprocess.run([B._nvcc(), "-std=c++17", "-cudart", "none", "-I", B.CSRC, "-I", B.INCLUDE, str(src), "-o", str(exe),
                    "-lpthread"], check=True)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout.strip() == "11"


def test_calls_without_tokens_need_no_rows():
    """An empty tensor has no address: where a call has no token, its rows may be null (nothing is launched)."""
    import ctypes
    from sparse_paged_kv_page_gb300 import _lib, build as B
    B.build()
    lib, P = _lib.load(), ctypes.c_void_p
    c = _lib.SaCache(k=P(0x100000), v=P(0x200000), meta=P(0x300000), dtype=0, num_blocks=4, num_kv_heads=2, page_size=16,
                     head_dim=128, kstd=None)
    b = _lib.SaBatch(block_table=P(0x20000), seq_lens=P(0x10000), batch=1, bt_stride=4)
    cu, ref = P(0x800000), ctypes.byref

    def rope(axes=1):
        sec = (_lib.c_i32 * 4)(*([64, 0] if axes == 1 else [32, 32]), 0, 0)
        return _lib.SaRope(table=P(0x400000), positions=None, q_weight=None, k_weight=None, max_pos=64, rot_dim=128,
                           interleaved=0, num_axes=axes, sections=sec, eps=1e-6)

    def append(T, most, r=rope()):
        return lib.sa_append_kv_rope(ref(c), ref(b), ref(r), None, 512, 4, None, 256, None, 256, cu, T, most, 0, None, None,
                                     None, None, 0, None, None)

    def prefill(T):
        return lib.sa_paged_prefill(ref(c), ref(b), None, 4, cu, T, 0, 0, 0.0, None, None, P(0xa00000), 1 << 30, None, None)

    assert append(0, 0) == 0 and append(0, 4) == 0 and append(0, 0, rope(2)) == 0
    assert append(3, 3) == 1 and append(3, 3, rope(2)) == 1
    assert prefill(0) == 0 and prefill(3) == 1
    plain = lambda most: lib.sa_append_kv(ref(c), ref(b), None, None, cu, most, None, None, None, 0, None, None)  # noqa: E731
    assert plain(0) == 0 and plain(3) == 1
