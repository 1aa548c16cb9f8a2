"""Whole layers as they run: prompts in chunks, then single tokens, through SparseDecoder and through the calls
themselves; captured graphs, streams, layers that share one batch."""
import pytest
import torch

from paged_util import Problem, attention64, check_attention, rotate64

pytestmark = pytest.mark.gpu

THETA = 10000.0


def _rows(dec, b, n, pool):
    pages = dec.block_table[b, : -(-n // dec.ps)].long()
    return pool[pages].transpose(1, 2).reshape(-1, dec.H_kv, dec.D)[:n]


def _decoder(B, *, ps=16, D=128, Hkv=2, Hq=8, capacity=512, dtype=torch.bfloat16, weights=True, **kw):
    import sparse_paged_kv_page_gb300 as S
    from sparse_paged_kv_page_gb300.step import SparseDecoder
    g = torch.Generator().manual_seed(5)
    w = [(1 + 0.1 * torch.randn(D, generator=g)).to(dtype).cuda() if weights else None for _ in range(2)]
    rope = S.make_rope(S.rope_table(capacity + 8, D, THETA), q_weight=w[0], k_weight=w[1], eps=1e-6)
    stride = capacity // ps
    dec = SparseDecoder(batch=B, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=ps, num_blocks=B * stride + 3,
                        bt_stride=stride, dtype=dtype, rope=rope, **kw)
    dec.cache.k.fill_(float("nan"))
    dec.cache.v.fill_(float("nan"))
    dec.set_block_table(torch.randperm(B * stride + 3, generator=g)[: B * stride].view(B, stride))
    return dec, w, lambda *s: (1.5 * torch.randn(s, generator=g)).to(dtype).cuda()


def _turned(x, w, first):
    place = torch.cat([torch.arange(f, f + n) for f, n in first])[None].cuda()
    return rotate64(x, w, 1e-6, place, THETA, x.shape[-1], False, [x.shape[-1] // 2])


def _check_cache(dec, w, keys, values):
    """The pools hold the turned keys and the values given so far, per request."""
    for b in range(dec.B):
        k, v = torch.cat(keys[b]), torch.cat(values[b])
        want, tol = _turned(k, w[1], [(0, k.shape[0])])
        assert bool(((_rows(dec, b, k.shape[0], dec.cache.k).double() - want).abs() <= tol).all())
        assert torch.equal(_rows(dec, b, k.shape[0], dec.cache.v), v)


def _check_out(dec, b, out, q, w, n, L, lse=None):
    """Attention of the last n tokens, from the cache's own keys; the query's rounding is the kernel's own."""
    want_q, tol_q = _turned(q, w[0], [(L - n, n)])
    rounded = want_q.to(dec.dtype)
    k, v = _rows(dec, b, L, dec.cache.k), _rows(dec, b, L, dec.cache.v)
    o, l, tol, tol_l = attention64(rounded, k, v, torch.arange(L - n, L, device="cuda"), dec.D ** -0.5, dec.window,
                                   dec.n_sink if dec.window else 0)
    # A query element whose float64 value lies within the kernel's float32 error of a rounding border may round the
    # other way, a whole step of eps 2^e (2^e <= |x| < 2^(e+1)); its logit then moves by scale step_d |k_d|.
    eps = torch.finfo(dec.dtype).eps
    step = eps * torch.exp2(torch.floor(torch.log2(want_q.abs().clamp(min=2.0 ** -14))))
    error32 = tol_q - eps / 2 * want_q.abs()
    flip = ((rounded.double() - want_q).abs() >= step / 2 - error32).double() * step
    move = torch.stack([(flip[:, h] @ k[:, h // (dec.H_q // dec.H_kv)].double().abs().t()).amax(1)
                        for h in range(dec.H_q)], 1) * dec.D ** -0.5
    big = v.double().abs().amax()
    check_attention(out, lse, (o, l, tol + (2 * move * big)[..., None], tol_l + move))


@pytest.mark.parametrize("kw", [dict(dense=True), dict(dense=True, window=40, n_sink=3), dict(dense=True, ps=1, D=64, Hq=6),
                                dict(topk=64)])
def test_prompt_in_chunks_then_tokens(kw):
    dec, w, rand = _decoder(3, **kw)
    keys, values, L = [[] for _ in range(3)], [[] for _ in range(3)], [0, 0, 0]
    for lens in ([70, 5, 33], [1, 40, 17], [130, 0, 2]):
        T = sum(lens)
        q, k, v = rand(T, dec.H_q, dec.D), rand(T, dec.H_kv, dec.D), rand(T, dec.H_kv, dec.D)
        lse = torch.zeros((T, dec.H_q), device="cuda")
        out = dec.prefill_attend(q, k, v, lens, lse=lse)
        at = 0
        for b, n in enumerate(lens):
            keys[b].append(k[at:at + n])
            values[b].append(v[at:at + n])
            L[b] += n
            if n:
                _check_out(dec, b, out[at:at + n], q[at:at + n], w, n, L[b], lse[at:at + n])
            at += n
    assert dec.seq_lens.tolist() == L
    for t in range(6):
        if t == 3:
            dec.capture()                               # the last three tokens replay a captured step
        q, k, v = rand(3, dec.H_q, dec.D), rand(3, dec.H_kv, dec.D), rand(3, dec.H_kv, dec.D)
        if t < 3:
            out = dec.step(q, k, v)
        else:
            for buf, x in ((dec.q_buf, q), (dec.k_buf, k), (dec.v_buf, v)):
                buf.copy_(x)
            out = dec.replay()
        for b in range(3):
            keys[b].append(k[b:b + 1])
            values[b].append(v[b:b + 1])
            L[b] += 1
            if dec.dense or -(-L[b] // dec.ps) <= dec.topk:
                _check_out(dec, b, out[b:b + 1], q[b:b + 1], w, 1, L[b], dec.lse[b:b + 1])
    assert dec.seq_lens.tolist() == L and int(dec.dev_status.item()) == 0
    _check_cache(dec, w, keys, values)


@pytest.mark.parametrize("ps", [16, 64, 128])
def test_rotated_sparse_steps_equal_steps_on_turned_inputs(ps):
    """The sparse chain with a rotation is the chain without one on the turned queries and keys, bit for bit."""
    from sparse_paged_kv_page_gb300.step import SparseDecoder
    dec, w, rand = _decoder(2, topk=4, ps=ps)
    plain = SparseDecoder(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=ps,
                          num_blocks=dec.cache.k.shape[0], bt_stride=dec.bt_stride, topk=4)
    plain.set_block_table(dec.block_table)
    lens = [200, 77]
    k, v = rand(277, 2, 128), rand(277, 2, 128)
    dec.prefill(k, v, lens)
    turned = torch.cat([_rows(dec, b, n, dec.cache.k) for b, n in enumerate(lens)])
    plain.prefill(turned, v, lens)
    for t in range(4):
        q, kn, vn = rand(2, 8, 128), rand(2, 2, 128), rand(2, 2, 128)
        out = dec.step(q, kn, vn)
        new = torch.stack([_rows(dec, b, lens[b] + t + 1, dec.cache.k)[-1] for b in range(2)])
        want = plain.step(dec.q_rot, new, vn)
        assert torch.equal(out, want) and torch.equal(dec.sel_idx, plain.sel_idx) and torch.equal(dec.lse, plain.lse)
    for b in range(2):
        n = -(-(lens[b] + 4) // ps)
        blk = dec.block_table[b, :n].long()
        assert torch.equal(dec.cache.meta[blk], plain.cache.meta[blk])


def test_layers_share_one_batch():
    """Lengths are advanced once; every layer writes its own tokens (advanced) and attends."""
    lens, new = [50, 0, 7], [3, 20, 1]
    total = [a + b for a, b in zip(lens, new)]
    layers = [Problem(lens, Hkv=2, G=4, seed=s, extra_pages=2, meta=True) for s in range(2)]
    S, T = layers[0].S, sum(new)
    table = layers[0].table
    seq_lens = torch.tensor(total, dtype=torch.int32).cuda()
    cu = torch.tensor([0, 3, 23, 24], dtype=torch.int32).cuda()
    ws = S.alloc_paged_prefill_workspace(3, 2, 8, 128, T)
    rope = S.make_rope(S.rope_table(128, 128))
    place = [(l, n) for l, n in zip(lens, new)]
    for p in layers:
        # each layer has its pages where the shared table says
        for b, n in enumerate(lens):
            for j in range(n):
                blk = int(table[b, j // 16])
                p.k[blk, :, j % 16], p.v[blk, :, j % 16] = p.seqs[b][0][j], p.seqs[b][1][j]
        p.table, p.seq_lens = table, seq_lens
        p.bind()
        q, k, v = p.rand(T, 8, 128), p.rand(T, 2, 128), p.rand(T, 2, 128)
        out = torch.empty_like(q)
        S.sa_append_kv_rope(p.cache, p.batch, rope, q, k, v, cu, 20, q, advanced=True, dev_status=p.status)
        S.sa_paged_prefill(p.cache, p.batch, q, 8, cu, 0.0, out, workspace=ws, dev_status=p.status)
        torch.cuda.synchronize()
        assert int(p.status) == 0 and seq_lens.tolist() == total
        want, tol = _turned(k, None, place)
        for b in range(3):
            r = slice(int(cu[b]), int(cu[b + 1]))
            kb, vb = p.rows(b, total[b]), p.rows(b, total[b], p.v)
            assert bool(((kb[lens[b]:].double() - want[r]).abs() <= tol[r]).all()) and torch.equal(vb[lens[b]:], v[r])
            check_attention(out[r], None, attention64(q[r], kb, vb, torch.arange(lens[b], total[b], device="cuda"),
                                                      128 ** -0.5, 0, 0))


def test_calls_on_two_streams_with_workspaces_of_their_own():
    p = Problem([3000, 40, 1500], Hkv=2, G=4)
    S = p.S
    cu = torch.tensor([0, 5, 6, 9], dtype=torch.int32).cuda()
    qd, qp = p.rand(3, 8, 128), p.rand(9, 8, 128)
    wanted = []
    for again in range(2):
        outs = []
        torch.cuda.synchronize()
        for s in (torch.cuda.Stream(), torch.cuda.Stream()):
            with torch.cuda.stream(s):
                ws = S.alloc_paged_decode_workspace(3, 2, 8, 128), S.alloc_paged_prefill_workspace(3, 2, 8, 128, 9)
                o = torch.empty_like(qd), torch.empty_like(qp)
                for _ in range(5):
                    S.sa_paged_decode(p.cache, p.batch, qd, 8, 0.0, o[0], workspace=ws[0])
                    S.sa_paged_prefill(p.cache, p.batch, qp, 8, cu, 0.0, o[1], workspace=ws[1])
                outs.append((o, ws))
        torch.cuda.synchronize()
        wanted.append([x for o, _ in outs for x in o])
    for a, b in zip(wanted[0], wanted[1]):
        assert torch.equal(a, b)
    assert torch.equal(wanted[0][0], wanted[0][2]) and torch.equal(wanted[0][1], wanted[0][3])


def test_two_graphs_share_a_workspace_in_order():
    p = Problem([900, 64], Hkv=2, G=4)
    S = p.S
    q1, q2 = p.rand(2, 8, 128), p.rand(2, 8, 128)
    o = [torch.empty_like(q1) for _ in range(4)]
    ws = S.alloc_paged_decode_workspace(2, 2, 8, 128)
    call = lambda q, out: S.sa_paged_decode(p.cache, p.batch, q, 8, 0.0, out, workspace=ws)  # noqa: E731
    call(q1, o[0])
    call(q2, o[1])
    graphs = []
    for q, out in ((q1, o[2]), (q2, o[3])):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(q, out)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o[0], o[2]) and torch.equal(o[1], o[3])


def test_outputs_over_the_queries_and_first_calls_captured():
    p = Problem([700, 64, 3], Hkv=1, G=4, D=64, ps=8, dtype="fp16")
    S = p.S
    cu = torch.tensor([0, 300, 301, 304], dtype=torch.int32).cuda()
    qd, qp = p.rand(3, 4, 64), p.rand(304, 4, 64)
    od, op = torch.empty_like(qd), torch.empty_like(qp)
    wd, wp = S.alloc_paged_decode_workspace(3, 1, 4, 64), S.alloc_paged_prefill_workspace(3, 1, 4, 64, 304)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.sa_paged_decode(p.cache, p.batch, qd, 4, 0.0, od, workspace=wd)
        S.sa_paged_prefill(p.cache, p.batch, qp, 4, cu, 0.0, op, workspace=wp)
    g.replay()
    S.sa_paged_decode(p.cache, p.batch, qd, 4, 0.0, qd, workspace=wd)
    S.sa_paged_prefill(p.cache, p.batch, qp, 4, cu, 0.0, qp, workspace=wp)
    torch.cuda.synchronize()
    assert torch.equal(od, qd) and torch.equal(op, qp)


def test_windows_as_long_as_the_cache_hide_nothing():
    p = Problem([500, 1], Hkv=2, G=2)
    S = p.S
    q = p.rand(2, 4, 128)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    ws = S.alloc_paged_decode_workspace(2, 2, 4, 128), S.alloc_paged_prefill_workspace(2, 2, 4, 128, 2)
    for window in (500, 2 ** 31 - 1):
        o = [torch.empty_like(q) for _ in range(4)]
        for i, w in ((0, 0), (1, window)):
            S.sa_paged_decode(p.cache, p.batch, q, 4, 0.0, o[i], window=w, n_sink=i, workspace=ws[0])
            S.sa_paged_prefill(p.cache, p.batch, q, 4, cu, 0.0, o[2 + i], window=w, n_sink=i, workspace=ws[1])
        torch.cuda.synchronize()
        assert torch.equal(o[0], o[1]) and torch.equal(o[2], o[3])


def test_a_thousand_requests():
    lens = [(17 * i) % 61 for i in range(1000)]
    new = [1 + i % 3 for i in range(1000)]
    p = Problem([a + b for a, b in zip(lens, new)], Hkv=1, G=2, D=64)
    S, T = p.S, sum(new)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    q, out = p.rand(T, 2, 64), torch.empty((T, 2, 64), dtype=p.dt, device="cuda")
    lse = torch.empty((T, 2), device="cuda")
    S.sa_paged_prefill(p.cache, p.batch, q, 2, cu, 0.0, out, lse=lse, dev_status=p.status,
                       workspace=S.alloc_paged_prefill_workspace(1000, 1, 2, 64, T))
    last = q[cu[1:].long() - 1].contiguous()
    od, ld = torch.empty_like(last), torch.empty((1000, 2), device="cuda")
    S.sa_paged_decode(p.cache, p.batch, last, 2, 0.0, od, lse=ld, dev_status=p.status,
                      workspace=S.alloc_paged_decode_workspace(1000, 1, 2, 64))
    torch.cuda.synchronize()
    assert int(p.status) == 0
    for b in list(range(0, 1000, 37)) + [999]:
        L, n, r = p.lens[b], new[b], slice(int(cu[b]), int(cu[b + 1]))
        want = attention64(q[r], *p.seqs[b], torch.arange(L - n, L, device="cuda"), 0.125, 0, 0)
        check_attention(out[r], lse[r], want)
        check_attention(od[b:b + 1], ld[b:b + 1], [x[-1:] for x in want])


def test_binding_refuses_other_shapes_and_types():
    p = Problem([20], Hkv=2, G=2, meta=True)
    S = p.S
    rope = S.make_rope(S.rope_table(64, 128))
    q, k, v = p.rand(3, 4, 128), p.rand(3, 2, 128), p.rand(3, 2, 128)
    cu = torch.tensor([0, 3], dtype=torch.int32).cuda()
    ws = S.alloc_paged_prefill_workspace(1, 2, 4, 128, 3)
    bad = [
        lambda: S.sa_append_kv_rope(p.cache, p.batch, rope, q.half(), k, v, cu, 3, q),
        lambda: S.sa_append_kv_rope(p.cache, p.batch, rope, q, k[:, :1], v, cu, 3, q),
        lambda: S.sa_append_kv_rope(p.cache, p.batch, rope, q, k, v[:2], cu, 3, q),
        lambda: S.sa_append_kv_rope(p.cache, p.batch, rope, q, k, v, cu, 3, q[:2]),
        lambda: S.sa_append_kv_rope(p.cache, p.batch, rope, q.transpose(0, 1), k, v, cu, 3, q),
        lambda: S.sa_append_kv_rope(p.cache, p.batch, rope, q, k, v, cu[:1], 3, q),
        lambda: S.sa_append_kv_rope(p.cache, p.batch, S.make_rope(S.rope_table(64, 128), positions=cu), q, k, v, cu, 3, q),
        lambda: S.sa_append_kv_rope(p.cache, p.batch, S.make_rope(S.rope_table(64, 128), q_weight=q[0, 0].half()), q, k, v,
                                    cu, 3, q),
        lambda: S.sa_paged_prefill(p.cache, p.batch, q, 2, cu, 0.0, q, workspace=ws),
        lambda: S.sa_paged_prefill(p.cache, p.batch, q, 4, cu.long(), 0.0, q, workspace=ws),
        lambda: S.sa_paged_prefill(p.cache, p.batch, q, 4, cu, 0.0, q[:2], workspace=ws),
        lambda: S.sa_paged_decode(p.cache, p.batch, q, 4, 0.0, q, workspace=ws),
        lambda: S.sa_paged_decode(p.cache, p.batch, q[:1].float(), 4, 0.0, q[:1], workspace=ws),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: S.sa_paged_decode(p.cache, p.batch, q[:1], 4, 0.0, torch.empty_like(q[:1])),
              lambda: S.sa_paged_prefill(p.cache, p.batch, q, 4, cu, 0.0, torch.empty_like(q), workspace=ws[:64])):
        with pytest.raises(S.SaError) as e:
            f()
        assert e.value.status == 3
    with pytest.raises(S.SaError):                                   # rot_dim 40
        S.sa_append_kv_rope(p.cache, p.batch, S.make_rope(S.rope_table(64, 40)), q, k, v, cu, 3, q)
    assert p.seq_lens.tolist() == [20]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [4, 16])
def test_nan_in_a_query_or_a_visible_key_shows(D, ps):
    # never a silent 0: the rows that see it are NaN, the others as without it
    import sparse_paged_kv_page_gb300 as S
    lens, new = [3000, 50, 700], [40, 20, 3]
    p = Problem(lens, Hkv=1, G=4, D=D, ps=ps)
    qd, qp = p.rand(3, 4, D), p.rand(63, 4, D)
    cu = torch.tensor([0, 40, 60, 63], dtype=torch.int32).cuda()

    def run():
        od, op = torch.empty_like(qd), torch.empty_like(qp)
        ld, lp = (torch.empty(x.shape[:2], device="cuda") for x in (qd, qp))
        S.sa_paged_decode(p.cache, p.batch, qd, 4, 0.0, od, lse=ld, workspace=S.alloc_paged_decode_workspace(3, 1, 4, D))
        S.sa_paged_prefill(p.cache, p.batch, qp, 4, cu, 0.0, op, lse=lp,
                           workspace=S.alloc_paged_prefill_workspace(3, 1, 4, D, 63))
        torch.cuda.synchronize()
        return od, ld, op, lp

    want = run()
    qd[1, 2, 5] = qp[7, 1, 3] = float("nan")
    od, ld, op, lp = run()
    for out, lse, at, o, l in ((od, ld, (1, 2), want[0], want[1]), (op, lp, (7, 1), want[2], want[3])):
        assert bool(out[at].isnan().all()) and bool(lse[at].isnan())
        rest = torch.ones(lse.shape, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert torch.equal(out[rest], o[rest]) and torch.equal(lse[rest], l[rest])
    qd[1, 2, 5] = qp[7, 1, 3] = 0.0
    want = run()
    j = 2980                                               # of request 0: its new tokens 20 .. 39 see it
    p.k[int(p.table[0, j // ps]), 0, j % ps, 0] = float("nan")
    od, ld, op, lp = run()
    assert bool(od[0].isnan().all()) and torch.equal(od[1:], want[0][1:])
    assert bool(op[20:40].isnan().all()) and bool(lp[20:40].isnan().all())
    assert torch.equal(op[:20], want[2][:20]) and torch.equal(op[40:], want[2][40:])
