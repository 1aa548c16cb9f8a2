"""Refusals of the whole-layer calls, checked on the host before any launch (no GPU needed: the addresses given
are never used)."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from sparse_paged_kv_page_gb300 import build as B
    B.build()
    from sparse_paged_kv_page_gb300 import _lib
    return _lib.load()


def _args(**change):
    from sparse_paged_kv_page_gb300 import _lib
    c = dict(k=P(0x100000), v=P(0x200000), meta=P(0x300000), dtype=0, num_blocks=4, num_kv_heads=2, page_size=16,
             head_dim=128, kstd=None)
    b = dict(block_table=P(0x20000), seq_lens=P(0x10000), batch=1, bt_stride=4)
    r = dict(table=P(0x400000), positions=None, q_weight=None, k_weight=None, max_pos=64, rot_dim=128, interleaved=0,
             num_axes=1, sections=(_lib.c_i32 * 4)(64, 0, 0, 0), eps=1e-6)
    for d in (c, b, r):
        d.update({k: v for k, v in change.items() if k in d})
    return _lib.SaCache(**c), _lib.SaBatch(**b), _lib.SaRope(**r)


def _append(lib, q=P(0x500000), qs=512, hq=4, k=P(0x600000), ks=256, v=P(0x700000), vs=256, cu=P(0x800000), T=4, most=4,
            out=P(0x900000), hh=None, pos=None, cnt=None, cap=0, **change):
    c, b, r = _args(**change)
    return lib.sa_append_kv_rope(ctypes.byref(c), ctypes.byref(b), ctypes.byref(r), q, qs, hq, k, ks, v, vs, cu, T, most, 0,
                                 out, hh, pos, cnt, cap, None, None)


@pytest.mark.parametrize("change", [
    dict(k=None), dict(v=None), dict(cu=None), dict(out=None), dict(q=None), dict(hq=0), dict(T=-1), dict(most=-1),
    dict(qs=508), dict(ks=128), dict(vs=260), dict(q=P(0x500008)), dict(out=P(0x900004)), dict(table=P(0x400008)),
    dict(table=None), dict(max_pos=0), dict(rot_dim=130), dict(rot_dim=132), dict(rot_dim=-4), dict(rot_dim=20),
    dict(num_axes=0), dict(num_axes=5), dict(num_axes=2), dict(pos=P(0x1000)), dict(pos=P(0x1000), cnt=P(0x2000)),
    dict(eps=-1.0), dict(eps=float("nan")), dict(dtype=2), dict(batch=0), dict(q_weight=P(0x1004)),
    dict(meta=None, kstd=P(0x1000))])
def test_append_refuses_bad_arguments(lib, change):
    assert _append(lib, **change) == 1


def test_append_refuses_sections_that_do_not_fill_the_pairs(lib):
    from sparse_paged_kv_page_gb300 import _lib
    for sec in ((30, 30, 0, 0), (60, 8, 0, 0), (-4, 68, 0, 0)):
        assert _append(lib, positions=P(0x1000), num_axes=2, sections=(_lib.c_i32 * 4)(*sec)) == 1


def test_append_refuses_what_it_does_not_implement_and_takes_nothing(lib):
    assert _append(lib, head_dim=96) == 2 and _append(lib, page_size=24) == 2 and _append(lib, page_size=256) == 2
    assert _append(lib, T=0) == 0 and _append(lib, most=0) == 0      # no token: nothing is launched


def _decode(lib, q=P(0x500000), hq=4, window=0, sink=0, out=P(0x900000), ws=P(0xa00000), wbytes=1 << 30, **change):
    c, b, _ = _args(**change)
    return lib.sa_paged_decode(ctypes.byref(c), ctypes.byref(b), q, hq, window, sink, 0.0, out, None, ws, wbytes, None, None)


def _prefill(lib, q=P(0x500000), hq=4, cu=P(0x800000), T=4, window=0, sink=0, out=P(0x900000), ws=P(0xa00000),
             wbytes=1 << 30, **change):
    c, b, _ = _args(**change)
    return lib.sa_paged_prefill(ctypes.byref(c), ctypes.byref(b), q, hq, cu, T, window, sink, 0.0, out, None, ws, wbytes,
                                None, None)


@pytest.mark.parametrize("call", [_decode, _prefill])
def test_attention_refuses_bad_arguments(lib, call):
    for change in (dict(q=None), dict(out=None), dict(hq=0), dict(hq=3), dict(window=-1), dict(sink=-1), dict(q=P(0x500008)),
                   dict(out=P(0x900008)), dict(batch=0), dict(bt_stride=0), dict(dtype=7), dict(block_table=None)):
        assert call(lib, **change) == 1, change
    for change in (dict(hq=34), dict(head_dim=32), dict(page_size=48)):
        assert call(lib, **change) == 2, change
    for change in (dict(ws=None), dict(wbytes=255), dict(ws=P(0xa00008))):
        assert call(lib, **change) == 3, change


def test_attention_limits(lib):
    assert _decode(lib, batch=1025) == 2
    assert _decode(lib, bt_stride=1 << 28) == 2                      # more tokens than a position counts
    assert _prefill(lib, cu=None) == 1 and _prefill(lib, T=-1) == 1
    assert _prefill(lib, T=0) == 0


def test_workspace_sizes(lib):
    assert lib.sa_paged_decode_workspace_size(0, 2, 4, 128) == 0
    assert lib.sa_paged_decode_workspace_size(2, 2, 5, 128) == 0
    assert lib.sa_paged_decode_workspace_size(2, 2, 4, 128) > 4 * 4
    assert lib.sa_paged_prefill_workspace_size(1, 2, 4, 128, -1) == 0
    # a workspace made for many rows serves fewer
    assert lib.sa_paged_prefill_workspace_size(1, 2, 4, 128, 100_000) >= lib.sa_paged_prefill_workspace_size(1, 2, 4, 128, 1)


def test_binding_refuses_what_the_library_cannot_see(lib):
    import torch
    import sparse_paged_kv_page_gb300 as S
    with pytest.raises(ValueError):
        S.make_rope(torch.zeros(4, 64))                              # not on a GPU
    with pytest.raises(ValueError):
        S.make_rope(None, positions=torch.zeros(2, 3, dtype=torch.int32), sections=[32])


def test_rope_struct_layout_matches_the_binding(lib):
    import sparse_paged_kv_page_gb300 as S
    from sparse_paged_kv_page_gb300 import _lib
    assert S.sa_struct_size(2) == ctypes.sizeof(_lib.SaRope)


def test_rope_table_is_the_float64_angle_rounded_once():
    import torch
    import sparse_paged_kv_page_gb300 as S
    t = S.rope_table(1000, 8, 100.0, device="cpu").double()
    a = 997.0 * 100.0 ** (-2.0 * 3 / 8)
    assert abs(t[997, 3] - torch.tensor(a, dtype=torch.float64).cos()) < 2.0 ** -24
    assert abs(t[997, 7] - torch.tensor(a, dtype=torch.float64).sin()) < 2.0 ** -24
