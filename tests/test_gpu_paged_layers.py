"""The whole-layer operators on the GPU against their plain float64 forms: the append with norm and rotation
(sa_append_kv_rope), one token over the whole cache (sa_paged_decode), and prompts over it (sa_paged_prefill)."""
import math

import pytest
import torch

from paged_util import Problem, attention64, check_attention, half_step, rotate64

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ append
def _append(lens, new, *, rot=None, interleaved=False, sections=None, norm=True, advanced=False, dtype="bf16", D=128,
            ps=16, Hkv=2, Hq=8, pad=0, std=False, meta=True, seed=0, eps=1e-5, theta=10000.0):
    """One call and its checks; returns the problem."""
    p = Problem(lens, Hkv=Hkv, G=1, D=D, ps=ps, dtype=dtype, meta=meta, std=std, seed=seed,
                extra_pages=-(-max(new) // ps) + 1)
    S, B, T = p.S, p.B, sum(new) + pad
    rot = D if rot is None else rot
    sections = sections or [rot // 2]
    qkv = p.rand(T, Hq + 2 * Hkv, D, scale=1.5)
    q, kn, vn = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cu = torch.tensor([0] + [sum(new[: i + 1]) for i in range(B)], dtype=torch.int32).cuda()
    table = S.rope_table(max(l + n for l, n in zip(lens, new)) + 300, rot, theta) if rot else None
    place = torch.cat([torch.arange(l, l + n) for l, n in zip(lens, new)] + [torch.zeros(pad, dtype=torch.int64)]).cuda()
    places = torch.stack([place if a == 0 else (place * (7 + a)) % 251 for a in range(len(sections))])
    positions = places.to(torch.int32) if len(sections) > 1 else None
    qw, kw = (1 + 0.2 * p.rand(D)).to(p.dt) if norm else None, (1 + 0.2 * p.rand(D)).to(p.dt) if norm else None
    rope = S.make_rope(table, interleaved=interleaved, sections=sections, positions=positions, q_weight=qw, k_weight=kw,
                       eps=eps)
    if advanced:
        p.seq_lens += (cu[1:] - cu[:-1])
    q_out = torch.full((T, Hq, D), 3.0, dtype=p.dt, device="cuda")
    before_k, before_v = p.k.clone(), p.v.clone()
    S.sa_append_kv_rope(p.cache, p.batch, rope, q, kn, vn, cu, max(new), q_out, advanced=advanced, dev_status=p.status)
    torch.cuda.synchronize()
    assert int(p.status) == 0
    assert p.seq_lens.tolist() == [l + n for l, n in zip(lens, new)]
    n_all = sum(new)
    want_q, tol_q = rotate64(q[:n_all], qw, eps, places[:, :n_all], theta, rot, interleaved, sections)
    want_k, tol_k = rotate64(kn[:n_all], kw, eps, places[:, :n_all], theta, rot, interleaved, sections)
    assert bool(((q_out[:n_all].double() - want_q).abs() <= tol_q).all())
    assert bool((q_out[n_all:] == 3.0).all())                         # padding rows are left alone
    written = torch.zeros_like(p.k, dtype=torch.bool)
    for b in range(B):
        L, n, r0 = lens[b], new[b], int(cu[b])
        k, v = p.rows(b, L + n), p.rows(b, L + n, p.v)
        assert bool(((k[L:].double() - want_k[r0:r0 + n]).abs() <= tol_k[r0:r0 + n]).all())
        assert torch.equal(v[L:], vn[r0:r0 + n])
        for j in range(L, L + n):
            written[int(p.table[b, j // ps]), :, j % ps] = True
        if meta:                                                     # exact, from the keys that were written
            for pg in range(L // ps, -(-(L + n) // ps)):
                blk, rows = int(p.table[b, pg]), k[pg * ps:(pg + 1) * ps].double()
                assert torch.equal(p.meta[blk, :, 0].double(), rows.amin(0))
                assert torch.equal(p.meta[blk, :, 1].double(), rows.amax(0))
                assert torch.equal(p.meta[blk, :, 2], rows.mean(0).to(p.dt)) or \
                    bool(((p.meta[blk, :, 2].double() - rows.mean(0)).abs() <= half_step(p.dt) * rows.mean(0).abs() + 2.0 ** -25).all())
                if std:
                    s = rows.var(0, unbiased=False).sqrt()
                    assert bool(((p.std[blk].double() - s).abs() <= half_step(p.dt) * s + 2.0 ** -25).all())
    for now, then in ((p.k, before_k), (p.v, before_v)):             # nothing else was touched
        assert torch.equal(now[~written].view(torch.int16), then[~written].view(torch.int16))
    return p


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 64), (128, 64), (64, 16), (128, 96), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_rotation_forms(dtype, D, rot, interleaved):
    _append([5, 0, 31], [18, 7, 1], dtype=dtype, D=D, rot=rot, interleaved=interleaved, norm=rot != 64, pad=3)


@pytest.mark.parametrize("ps", [1, 2, 8, 16, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_append_page_sizes(ps, D):
    _append([0, 3, 150, 127], [1, 33, 130, 2], ps=ps, D=D, advanced=ps % 3 == 1)


@pytest.mark.parametrize("Hkv,Hq", [(1, 1), (8, 32), (3, 21), (5, 5), (4, 6)])
def test_append_heads(Hkv, Hq):
    _append([9, 1024], [1, 1], Hkv=Hkv, Hq=Hq, advanced=True)
    _append([0, 17], [40, 3], Hkv=Hkv, Hq=Hq, dtype="fp16")


@pytest.mark.parametrize("sections", [[16, 24, 24], [1, 62, 1], [10, 20, 30, 4], [0, 64]])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_axes(sections, interleaved):
    _append([4, 40], [50, 9], sections=sections, interleaved=interleaved)


def test_append_many_requests_and_a_long_prompt():
    lens = [(37 * i) % 91 for i in range(70)]
    _append(lens, [1 + (i % 5) for i in range(70)], Hkv=1, Hq=2, D=64)
    _append([3], [1500], Hkv=2, Hq=16, norm=True)
    _append([100], [300], std=True, Hkv=2, Hq=4)
    _append([100, 5], [1, 40], std=True, ps=32, D=64, dtype="fp16")


def test_append_far_positions_keep_their_angles():
    # the table is made in float64: an angle of 10^5 radians is off by its float32 rounding alone
    _append([131000], [20], ps=128, Hkv=1, Hq=2, theta=500000.0)


def test_append_without_queries_and_in_place():
    p = Problem([10], Hkv=2, G=2, meta=True, extra_pages=3)
    S = p.S
    rope = S.make_rope(S.rope_table(64, 128))
    kn, vn, q = p.rand(5, 2, 128), p.rand(5, 2, 128), p.rand(5, 4, 128)
    cu = torch.tensor([0, 5], dtype=torch.int32).cuda()
    want, tol = rotate64(q, None, 0.0, torch.arange(10, 15)[None].cuda(), 10000.0, 128, False, [64])
    S.sa_append_kv_rope(p.cache, p.batch, rope, None, kn, vn, cu, 5, None, dev_status=p.status)
    assert p.seq_lens.tolist() == [15]
    S.sa_append_kv_rope(p.cache, p.batch, rope, q, kn, vn, cu, 5, q, advanced=True, dev_status=p.status)
    assert p.seq_lens.tolist() == [15] and int(p.status) == 0
    assert bool(((q.double() - want).abs() <= tol).all())


def test_append_token_level_lists_and_scores():
    p = Problem([6, 2], Hkv=2, G=2, ps=1, extra_pages=12)
    S, cap = p.S, 16
    hh = torch.full((p.k.shape[0], 2), 5.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((2, 2, cap), dtype=torch.int32, device="cuda")
    cnt = torch.tensor([[6, 3], [2, 2]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 4, 5], dtype=torch.int32).cuda()
    kn, vn = p.rand(5, 2, 128), p.rand(5, 2, 128)
    S.sa_append_kv_rope(p.cache, p.batch, S.make_rope(S.rope_table(64, 128)), None, kn, vn, cu, 4, None, hh=hh,
                        ret_pos=pos, ret_cnt=cnt, ret_cap=cap, dev_status=p.status)
    assert cnt.tolist() == [[10, 7], [3, 3]] and p.seq_lens.tolist() == [10, 3] and int(p.status) == 0
    assert pos[0, 1, 3:7].tolist() == [6, 7, 8, 9] and pos[1, 0, 2].item() == 2
    wrote = torch.zeros_like(hh, dtype=torch.bool)
    wrote[p.table[0, 6:10].long()] = True
    wrote[p.table[1, 2:3].long()] = True
    assert bool((hh[wrote] == 0).all()) and bool((hh[~wrote] == 5).all())


def test_append_bad_data_is_flagged_and_skipped():
    S = __import__("sparse_paged_kv_page_gb300")
    rope = S.make_rope(S.rope_table(40, 128))

    def call(lens, new, change, max_new=None, advanced=False, positions=None):
        p = Problem(lens, Hkv=1, G=1, meta=True, extra_pages=1)
        T = sum(new)
        kn, vn = p.rand(T, 1, 128), p.rand(T, 1, 128)
        q = p.rand(T, 1, 128)
        cu = torch.tensor([0] + [sum(new[: i + 1]) for i in range(len(new))], dtype=torch.int32).cuda()
        change(p, cu)
        out = torch.full_like(q, 3.0)
        r = rope if positions is None else S.make_rope(S.rope_table(40, 128), positions=positions)
        S.sa_append_kv_rope(p.cache, p.batch, r, q, kn, vn, cu, max_new or max(new), out, advanced=advanced,
                            dev_status=p.status)
        return p, out, int(p.status)

    nothing = lambda p, cu: None  # noqa: E731
    p, out, st = call([30], [5], nothing, max_new=3)                       # more tokens than announced
    assert st == 2 and p.seq_lens.tolist() == [33] and bool((out[3:] == 3).all())
    p, out, st = call([20], [30], nothing)                                 # 48 slots: two are dropped
    assert st & 2 and p.seq_lens.tolist() == [48] and bool((out[28:] == 3).all())
    p, out, st = call([20, 20], [2, 2], lambda p, cu: p.table[0].fill_(10_000))
    assert st == 1 and bool(torch.isfinite(p.rows(1, 22).float()).all())
    p, out, st = call([20, 20], [2, 2], lambda p, cu: cu[2].fill_(9))      # rows behind the call's
    assert st == 4 and p.seq_lens.tolist() == [22, 20] and bool((out[2:] == 3).all())
    p, out, st = call([20, 20], [2, 2], lambda p, cu: p.seq_lens[1:].fill_(1), advanced=True)
    assert st == 4 and bool((out[2:] == 3).all())
    p, out, st = call([20], [2], nothing, positions=torch.tensor([-1, 40], dtype=torch.int32).cuda())
    assert st == 16 and bool(torch.isfinite(p.rows(0, 22).float()).all())


# ------------------------------------------------------------------------------------------------ decode
def _decode(p, window=0, n_sink=0, scale=0.0, ws=None, q=None):
    S = p.S
    q = p.rand(p.B, p.Hq, p.D, scale=2.0) if q is None else q
    out = torch.full_like(q, float("nan"))
    lse = torch.full((p.B, p.Hq), float("nan"), device="cuda")
    ws = S.alloc_paged_decode_workspace(p.B, p.H, p.Hq, p.D) if ws is None else ws
    S.sa_paged_decode(p.cache, p.batch, q, p.Hq, scale, out, window=window, n_sink=n_sink, lse=lse, workspace=ws,
                      dev_status=p.status)
    torch.cuda.synchronize()
    assert int(p.status) == 0
    sc = scale or p.D ** -0.5
    for b, L in enumerate(p.lens):
        want = attention64(q[b:b + 1], *p.seqs[b], torch.tensor([L - 1], device="cuda"), sc, window, n_sink)
        check_attention(out[b:b + 1], lse[b:b + 1], want)
    assert not bool(ws[: 4 * p.B * p.H].any())                        # the counters are zero again
    return q, out, lse, ws


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [1, 2, 4, 8, 16, 32, 128])
def test_decode_page_sizes(dtype, D, ps):
    p = Problem([0, 1, 15, 16, 17, 333, 2100], D=D, ps=ps, dtype=dtype)
    _decode(p)
    _decode(p, window=100, n_sink=5)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 9, 16])
def test_decode_groups(G):
    _decode(Problem([700, 63, 1], G=G, Hkv=3))


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (16, 4), (17, 16), (64, 1), (65, 100), (1000, 4), (5000, 8),
                                           (33, 0), (256, 640)])
def test_decode_windows(window, n_sink):
    p = Problem([1, 40, 64, 900, 1003], Hkv=2, G=4)
    # tokens that the query does not see hold NaN and infinity: freed pages are reused
    for b, L in enumerate(p.lens):
        for j in range(L):
            if j < L - window and j >= n_sink:
                blk, s = int(p.table[b, j // p.ps]), j % p.ps
                p.k[blk, :, s], p.v[blk, :, s] = float("nan"), math.inf if j % 2 else float("nan")
    _decode(p, window=window, n_sink=n_sink)
    p1 = Problem([900], Hkv=2, G=4, ps=2)
    _decode(p1, window=window, n_sink=n_sink)


def test_decode_many_requests_and_long_ones():
    _decode(Problem([(53 * i) % 400 for i in range(130)], Hkv=1, G=2, D=64))
    _decode(Problem([40_000, 9], Hkv=1, G=4, D=64))
    _decode(Problem([20_000], Hkv=8, G=4, D=128), window=0)


def test_decode_scores_far_apart_and_equal():
    p = Problem([500, 500], Hkv=1, G=2)
    q = p.rand(2, 2, 128, scale=30.0)
    _decode(p, q=q)
    p.k.zero_()
    p.seqs = [[k * 0, v] for k, v in p.seqs]
    _decode(p, q=q, scale=0.3)


def test_decode_repeats_bit_for_bit_in_a_shared_workspace_and_on_a_stream():
    p = Problem([5000, 17, 3000], Hkv=2, G=4)
    q, out, lse, ws = _decode(p)
    for _ in range(3):
        again = _decode(p, q=q, ws=ws)
        assert torch.equal(again[1], out) and torch.equal(again[2], lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = _decode(p, q=q, ws=ws)
    s.synchronize()
    assert torch.equal(again[1], out)


def test_decode_bad_data_is_flagged():
    p = Problem([100, 50, 20], Hkv=1, G=2)
    q = p.rand(3, 2, 128)
    ws = p.S.alloc_paged_decode_workspace(3, 1, 2, 128)
    out = torch.empty_like(q)
    p.table[0, 1] = -5
    p.seq_lens[1] = 100_000
    p.seq_lens[2] = -3
    p.S.sa_paged_decode(p.cache, p.batch, q, 2, 0.0, out, workspace=ws, dev_status=p.status)
    assert int(p.status) & 7 == 7
    keep = [j for j in range(100) if not 16 <= j < 32]
    k, v = (x[keep] for x in p.seqs[0])
    want = attention64(q[:1], k, v, torch.tensor([len(keep) - 1], device="cuda"), 128 ** -0.5, 0, 0)
    check_attention(out[:1], None, want)
    assert bool((out[2] == 0).all())


# ----------------------------------------------------------------------------------------------- prefill
def _prefill(p, new, window=0, n_sink=0, pad=0, ws=None, q=None, scale=0.0):
    S, T = p.S, sum(new) + pad
    q = p.rand(T, p.Hq, p.D, scale=2.0) if q is None else q
    out = torch.full_like(q, 3.0)
    lse = torch.full((T, p.Hq), 3.0, device="cuda")
    cu = torch.tensor([0] + [sum(new[: i + 1]) for i in range(p.B)], dtype=torch.int32).cuda()
    ws = S.alloc_paged_prefill_workspace(p.B, p.H, p.Hq, p.D, T) if ws is None else ws
    S.sa_paged_prefill(p.cache, p.batch, q, p.Hq, cu, scale, out, window=window, n_sink=n_sink, lse=lse, workspace=ws,
                       dev_status=p.status)
    torch.cuda.synchronize()
    assert int(p.status) == 0
    for b, (L, n) in enumerate(zip(p.lens, new)):
        r = slice(int(cu[b]), int(cu[b]) + n)
        want = attention64(q[r], *p.seqs[b], torch.arange(L - n, L, device="cuda"), scale or p.D ** -0.5, window, n_sink)
        check_attention(out[r], lse[r], want)
    n = sum(new)
    assert bool((out[n:] == 3.0).all()) and bool((lse[n:] == 3.0).all())
    return q, out, lse, ws


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [1, 2, 4, 8, 16, 32, 128])
def test_prefill_page_sizes(dtype, D, ps):
    p = Problem([0, 1, 130, 300, 129], D=D, ps=ps, dtype=dtype)
    _prefill(p, [0, 1, 130, 40, 2], pad=2)
    _prefill(p, [0, 1, 130, 40, 2], window=50, n_sink=3)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 9, 12, 16])
def test_prefill_groups(G):
    p = Problem([150, 77, 600], G=G, Hkv=2)
    _prefill(p, [150, 1, 33])


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (16, 4), (17, 16), (64, 1), (129, 200), (1000, 4), (128, 0),
                                           (256, 128)])
def test_prefill_windows(window, n_sink):
    p = Problem([700, 900, 5], Hkv=2, G=4)
    _prefill(p, [700, 130, 5], window=window, n_sink=n_sink)
    p1 = Problem([800], Hkv=1, G=2, ps=4, D=64, dtype="fp16")
    _prefill(p1, [300], window=window, n_sink=n_sink)


def test_prefill_window_never_uses_freed_pages():
    p = Problem([900], Hkv=2, G=4)
    window, n_sink, n = 100, 4, 40
    for j in range(n_sink, 900 - n - window + 1):
        blk, s = int(p.table[0, j // p.ps]), j % p.ps
        p.k[blk, :, s], p.v[blk, :, s] = float("nan"), math.inf if j % 2 else float("nan")
    _prefill(p, [n], window=window, n_sink=n_sink)


def test_prefill_few_tokens_over_long_caches():
    p = Problem([6000, 2500, 9], Hkv=2, G=4)
    q, out, lse, ws = _prefill(p, [3, 8, 1])
    for _ in range(2):
        again = _prefill(p, [3, 8, 1], q=q, ws=ws)
        assert torch.equal(again[1], out) and torch.equal(again[2], lse)
    _prefill(Problem([30_000], Hkv=1, G=8), [2])


def test_prefill_many_requests_and_a_long_prompt():
    lens = [(53 * i) % 200 + 1 for i in range(70)]
    _prefill(Problem(lens, Hkv=1, G=4, D=64), [1 + (i * 7) % n for i, n in enumerate(lens)])
    _prefill(Problem([2500], Hkv=1, G=4), [2500])
    _prefill(Problem([2000], Hkv=2, G=8, D=64, dtype="fp16"), [2000], window=300, n_sink=4)


def test_prefill_scores_far_apart_and_equal():
    p = Problem([500], Hkv=1, G=2)
    q = p.rand(300, 2, 128, scale=30.0)
    _prefill(p, [300], q=q)
    # the running maximum rises through the sequence
    ramp = torch.linspace(0, 3, 500, device="cuda")[:, None, None]
    p.seqs[0][0] = (ramp * torch.ones_like(p.seqs[0][0])).to(p.dt)
    for j in range(500):
        p.k[int(p.table[0, j // 16]), :, j % 16] = p.seqs[0][0][j]
    _prefill(p, [300], q=q.abs())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [700, 3])
def test_prefill_scores_that_rise_along_the_cache(dtype, D, new):
    # the reference of the softmax has to follow every few steps, in whole items and in parts
    p = Problem([1500, 1301], Hkv=1, G=4, D=D, dtype=dtype)
    for b, n in enumerate(p.lens):
        ramp = torch.linspace(0, 3, n, device="cuda")[:, None, None]
        p.seqs[b][0] = (ramp * torch.ones_like(p.seqs[b][0])).to(p.dt)
        for j in range(n):
            p.k[int(p.table[b, j // 16]), :, j % 16] = p.seqs[b][0][j]
    q = p.rand(2 * new, 4, D, scale=2.0).abs()
    _prefill(p, [new, new], q=q)
    _prefill(p, [new, new], q=q, window=400, n_sink=3)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 4200])
def test_prefill_items_behind_the_last_full_round(D, window):
    # 8 heads x 16 queries: 168 (328 at head dim 64) items, the last of them, of the last head, in parts
    p = Problem([5000], Hkv=8, G=16, D=D)
    q, out, lse, ws = _prefill(p, [320], window=window, n_sink=window and 5)
    again = _prefill(p, [320], window=window, n_sink=window and 5, q=q, ws=ws)
    assert torch.equal(again[1], out) and torch.equal(again[2], lse)
    _prefill(Problem([700, 4500, 40], Hkv=8, G=16, D=D), [40, 290, 1], window=window, ws=ws)


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_of_few_rows_in_halves_and_whole(D):
    # 1 - 3 halves of rows over few keys (items of one half) and over many (items of two)
    for L in (900, 40_000):
        p = Problem([L, 700], Hkv=8, G=8, D=D)
        for new in ([15, 1], [30, 40], [16, 33]):
            q, out, lse, ws = _prefill(p, new)
            _prefill(p, new, window=600, n_sink=4, q=q, ws=ws)
            again = _prefill(p, new, q=q, ws=ws)
            assert torch.equal(again[1], out) and torch.equal(again[2], lse)


def test_prefill_of_more_items_than_run_at_once():
    _prefill(Problem([3000, 33, 0, 1200], Hkv=8, G=7, D=64, ps=32), [2999, 30, 0, 5])
    _prefill(Problem([1900, 700], Hkv=8, G=5, D=64, ps=4), [1500, 700], window=333, n_sink=2)


def test_prefill_bad_data_is_flagged():
    p = Problem([100, 50, 40], Hkv=1, G=2)
    q = p.rand(12, 2, 128)
    out = torch.full_like(q, 3.0)
    lse = torch.zeros((12, 2), device="cuda")
    ws = p.S.alloc_paged_prefill_workspace(3, 1, 2, 128, 12)
    cu = torch.tensor([0, 4, 8, 20], dtype=torch.int32).cuda()           # the last request leaves the rows
    p.table[0, 1] = 12345
    p.seq_lens[1] = 2                                                     # fewer than its new tokens
    p.S.sa_paged_prefill(p.cache, p.batch, q, 2, cu, 0.0, out, lse=lse, workspace=ws, dev_status=p.status)
    assert int(p.status) & 5 == 5
    keep = [j for j in range(100) if not 16 <= j < 32]
    k, v = (x[keep] for x in p.seqs[0])
    want = attention64(q[:4], k, v, torch.arange(len(keep) - 4, len(keep), device="cuda"), 128 ** -0.5, 0, 0)
    check_attention(out[:4], None, want)
    assert bool((out[4:6] == 0).all()) and bool(torch.isneginf(lse[4:6]).all())
    want = attention64(q[6:8], *(x[:2] for x in p.seqs[1]), torch.arange(2, device="cuda"), 128 ** -0.5, 0, 0)
    check_attention(out[6:8], None, want)
    assert bool((out[8:] == 3.0).all())
    # overlapping requests: nothing is written, and the workspace serves the next call
    p = Problem([400, 300, 200], Hkv=1, G=2)
    ws = p.S.alloc_paged_prefill_workspace(3, 1, 2, 128, 12)
    q = p.rand(12, 2, 128)
    out = torch.full_like(q, 3.0)
    p.S.sa_paged_prefill(p.cache, p.batch, q, 2, torch.tensor([0, 12, 0, 12], dtype=torch.int32).cuda(), 0.0, out,
                         workspace=ws, dev_status=p.status)
    assert int(p.status) == 4 and bool((out == 3.0).all())
    p.status.zero_()
    _prefill(p, [4, 4, 4], ws=ws, q=q)
