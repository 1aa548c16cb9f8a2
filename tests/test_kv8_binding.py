"""Which cache objects the binding takes (no GPU)."""
import pytest
import torch

from kv8_util import E4M3


def test_the_binding_takes_caches_of_derived_classes():
    import sparse_paged_kv_page_gb300 as S

    class Mine(S.SaCache):
        pass

    class Mine8(S.SaCache8):
        pass

    pool = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16)
    c = Mine()
    c._keep = (pool, pool)
    c8 = Mine8()
    c8._keep, c8._dtype = (pool.to(E4M3), pool.to(E4M3)), torch.bfloat16
    rows, long = torch.zeros((1, 4, 128), dtype=torch.bfloat16), torch.zeros((1, 5, 128), dtype=torch.bfloat16)
    # past the kind of cache, the first thing that is wrong is the number of heads
    for call, cache in ((S.sa_paged_decode, c), (S.sa_paged_decode8, c8)):
        with pytest.raises(ValueError, match="q must be"):
            call(cache, S.SaBatch(), long, 4, 0.0, rows)
    for call, cache in ((S.sa_paged_prefill, c), (S.sa_paged_prefill8, c8)):
        with pytest.raises(ValueError, match="q must be"):
            call(cache, S.SaBatch(), long, 4, None, 0.0, rows)
    for call, cache in ((S.sa_paged_decode, c8), (S.sa_paged_decode8, c)):
        with pytest.raises(ValueError, match="cache must be"):
            call(cache, S.SaBatch(), rows, 4, 0.0, rows)
    with pytest.raises(ValueError, match="k_new"):
        S.sa_append_kv_rope(c, S.SaBatch(), None, None, rows, rows, None, 1, None)
