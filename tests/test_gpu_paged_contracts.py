"""What the whole-layer calls promise around their mathematics, on the GPU: first copies of cold kernels, workspaces that
calls of other sizes have used, calls without tokens, retained lists behind a prompt, means of pages rounded once."""
import pytest
import torch

from paged_util import Problem, attention64, check_attention

pytestmark = pytest.mark.gpu


def _decode_once(p, q, ws, n_heads=None):
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    p.S.sa_paged_decode(p.cache, p.batch, q, n_heads or p.Hq, 0.0, out, lse=lse, workspace=ws, dev_status=p.status)
    return out, lse


@pytest.mark.parametrize("D", [64, 128])
def test_decode_after_other_kernels_has_its_first_copies(D):
    # each launch begins with its code and its constants out of the SMs' caches, one warp ahead of the others
    p = Problem([700, 64, 3, 2500], Hkv=2, G=4, D=D)
    q = p.rand(4, 8, D)
    ws = p.S.alloc_paged_decode_workspace(4, 2, 8, D)
    other = torch.randn(2048, 2048, device="cuda")
    flush = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")
    want = None
    for i in range(60):
        flush.fill_(i)
        other = torch.tanh(other @ other.t() * 1e-3) + torch.sort(other, 1)[0]
        got = _decode_once(p, q, ws)
        torch.cuda.synchronize()
        if want is None:
            want = got
            for b, L in enumerate(p.lens):
                check_attention(got[0][b:b + 1], got[1][b:b + 1],
                                attention64(q[b:b + 1], *p.seqs[b], torch.tensor([L - 1], device="cuda"), D ** -0.5, 0, 0))
        assert int(p.status) == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def _prefill_once(p, q, new, ws, **kw):
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    cu = torch.tensor([0] + list(new), dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    p.S.sa_paged_prefill(p.cache, p.batch, q, p.Hq, cu, 0.0, out, lse=lse, workspace=ws, dev_status=p.status, **kw)
    return out, lse


def test_one_workspace_serves_calls_of_all_sizes():
    """Allocated once for the largest, as a server does: small batches, large ones, other heads, both operators in turn,
    each against float64 and the same bits again in a workspace of its own."""
    import sparse_paged_kv_page_gb300 as S
    kinds = [dict(lens=[3000], Hkv=8, G=4), dict(lens=[1500 + 40 * i for i in range(16)], Hkv=8, G=4),
             dict(lens=[9000, 70, 800], Hkv=3, G=7, D=64), dict(lens=[50] * 63 + [4000], Hkv=8, G=8),
             dict(lens=[2000, 1], Hkv=1, G=16, dtype="fp16", ps=4), dict(lens=[5000], Hkv=8, G=16, D=64)]
    calls = []
    for seed, kw in enumerate(kinds):
        p = Problem(kw.pop("lens"), seed=seed, **kw)
        few = [min(n, 1 + b % 3) for b, n in enumerate(p.lens)]
        qd, qp = p.rand(p.B, p.Hq, p.D), p.rand(sum(few), p.Hq, p.D)
        calls += [(p, lambda ws, p=p, q=qd: _decode_once(p, q, ws), qd, [1] * p.B),
                  (p, lambda ws, p=p, q=qp, n=few: _prefill_once(p, q, n, ws), qp, few)]
    # whole items and, behind the last full round of CTAs, items in parts
    for seed, D in ((20, 128), (21, 64)):
        p = Problem([5000], Hkv=8, G=16, D=D, seed=seed)
        q = p.rand(320, p.Hq, D)
        calls.append((p, lambda ws, p=p, q=q: _prefill_once(p, q, [320], ws), q, [320]))
    size = max(max(S.sa_paged_decode_workspace_size(p.B, p.H, p.Hq, p.D),
                   S.sa_paged_prefill_workspace_size(p.B, p.H, p.Hq, p.D, q.shape[0])) for p, _, q, _ in calls)
    shared = torch.zeros(size, dtype=torch.uint8, device="cuda")
    order = list(range(len(calls))) + [len(calls) - 1 - i for i in range(len(calls))] + [2, 0, 6, 2, 7, 1, 12, 3, 13, 0, 6, 11, 2]
    wanted = {}
    for i in order:
        p, call, q, new = calls[i]
        out, lse = call(shared)
        torch.cuda.synchronize()
        assert int(p.status) == 0
        if i not in wanted:
            wanted[i] = out, lse
            at = 0
            for b, (L, n) in enumerate(zip(p.lens, new)):
                r = slice(at, at + n)
                check_attention(out[r], lse[r], attention64(q[r], *p.seqs[b], torch.arange(L - n, L, device="cuda"),
                                                            p.D ** -0.5, 0, 0))
                at += n
            alone = call(torch.zeros(size, dtype=torch.uint8, device="cuda"))
            assert torch.equal(alone[0], out) and torch.equal(alone[1], lse)
        assert torch.equal(out, wanted[i][0]) and torch.equal(lse, wanted[i][1]), f"call {i} changed"


@pytest.mark.parametrize("rotated", [False, True])
def test_calls_without_tokens(rotated):
    import sparse_paged_kv_page_gb300 as S
    from sparse_paged_kv_page_gb300.step import SparseDecoder
    rope = S.make_rope(S.rope_table(64, 128)) if rotated else None
    dec = SparseDecoder(batch=2, num_q_heads=4, num_kv_heads=2, head_dim=128, page_size=16, num_blocks=8, bt_stride=4,
                        dense=True, rope=rope)
    dec.set_block_table(torch.arange(8).view(2, 4))
    g = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    dec.prefill(rand(9, 2, 128), rand(9, 2, 128), [5, 4])
    k, v = dec.cache.k.clone(), dec.cache.v.clone()
    none = lambda h: torch.empty((0, h, 128), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    out = dec.prefill_attend(none(4), none(2), none(2), [0, 0])
    dec.prefill(none(2), none(2), [0, 0])
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    three = S.make_rope(S.rope_table(64, 128), sections=[32, 32], positions=torch.empty((2, 0), dtype=torch.int32, device="cuda"))
    S.sa_append_kv_rope(dec.cache.struct, dec.batch, three, none(4), none(2), none(2), cu, 0, none(4))
    torch.cuda.synchronize()
    assert out.shape == (0, 4, 128) and dec.seq_lens.tolist() == [5, 4] and int(dec.dev_status) == 0
    assert torch.equal(dec.cache.k.view(torch.int16), k.view(torch.int16))
    assert torch.equal(dec.cache.v.view(torch.int16), v.view(torch.int16))


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("proxy", [False, True])
def test_attended_prompts_leave_the_lists_that_prompts_leave(proxy, rotated):
    """Token-level decoders: prefill_attend retains, scores and evicts as prefill does, and the steps behind it agree."""
    import sparse_paged_kv_page_gb300 as S
    from sparse_paged_kv_page_gb300.step import SparseDecoder
    B, Hkv, Hq, D, stride = 2, 2, 8, 64, 256
    rope = S.make_rope(S.rope_table(stride, D)) if rotated else None
    g = torch.Generator().manual_seed(11)
    rand = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    decs = []
    for _ in range(2):
        dec = SparseDecoder(batch=B, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=1, num_blocks=B * stride,
                            bt_stride=stride, budget=40, n_sink=4, grace=6, decay=0.95, ret_cap=48 if proxy else 200,
                            proxy_prefill=proxy, rope=rope)
        dec.set_block_table(torch.arange(B * stride).view(B, stride))
        decs.append(dec)
    seen, done = [[] for _ in range(B)], [0] * B
    for lens in ([90, 30], [25, 60]):                     # the prompt is longer than the lists of the trimmed one
        T = sum(lens)
        q, k, v = rand(T, Hq, D), rand(T, Hkv, D), rand(T, Hkv, D)
        decs[0].prefill(k, v, lens)
        out = decs[1].prefill_attend(q, k, v, lens)
        at = 0
        for b, n in enumerate(lens):
            done[b] += n
            if not rotated:                               # every cached token is attended, whatever is retained
                seen[b].append((k[at:at + n], v[at:at + n]))
                kb, vb = (torch.cat(x) for x in zip(*seen[b]))
                check_attention(out[at:at + n], None,
                                attention64(q[at:at + n], kb, vb, torch.arange(done[b] - n, done[b], device="cuda"),
                                            D ** -0.5, 0, 0))
            at += n
        torch.cuda.synchronize()
        for name in ("seq_lens", "ret_cnt", "dev_status"):
            assert torch.equal(getattr(decs[0], name), getattr(decs[1], name)), name
        assert int(decs[1].dev_status) == 0
        assert decs[1].ret_cnt.tolist() == [[40] * Hkv if proxy and n > 40 else [n] * Hkv for n in done]
        for b in range(B):
            for h in range(Hkv):
                pos = [d.ret_pos[b, h, : int(d.ret_cnt[b, h])] for d in decs]
                assert torch.equal(*pos)
                hh = [d.cache.hh[d.block_table[b, x.long()].long(), h] for d, x in zip(decs, pos)]
                assert torch.equal(*hh)
    for _ in range(3):
        q, k, v = rand(B, Hq, D), rand(B, Hkv, D), rand(B, Hkv, D)
        assert torch.equal(*[d.step(q, k, v) for d in decs])


# ---------------------------------------------------------------------------------------------- page means
def _round_once(x, dtype):
    """float64 rounded once to the type, to nearest even (a cast by way of float32 would round twice)."""
    bits, least = (8, -133) if dtype is torch.bfloat16 else (11, -24)     # significant bits; exponent of the smallest step
    _, e = torch.frexp(x)
    step = torch.exp2((e.double() - bits).clamp(min=least))
    return (torch.round(x / step) * step).to(dtype)


def _columns(n, heads, D, dtype, g):
    """Keys [n, heads, D] whose columns are, in turn: random; of mixed magnitude; cancelling; equal but for one step; on a
    rounding border, or off it by a power of two. Their sums are exact in float64 in any order (44 bits)."""
    k = torch.randn((n, heads, D), generator=g, dtype=torch.float64)
    ulp = 2.0 ** -7 if dtype is torch.bfloat16 else 2.0 ** -10
    low = -33 if dtype is torch.bfloat16 else -24
    k[..., 1::8] *= torch.exp2(torch.randint(-9, 10, k[..., 1::8].shape, generator=g).double())
    if n > 1:
        k[n // 2: 2 * (n // 2), :, 2::8] = -k[: n // 2, :, 2::8].to(dtype).double()
    k[..., 3::8] = 1.0
    k[n // 3, :, 3::8] = 1.0 + ulp
    if n >= 4 and n % 2 == 0:                             # the sum of all rows but the last is n (1 + ulp / 2)
        for at in (4, 5, 6, 7):
            k[..., at::8] = 1.0
            k[0, :, at::8] = 2.0
            k[1, :, at::8] = 1.0 + n / 2 * ulp
            m = k[n - 1, :, at::8]
            m[:] = torch.exp2(torch.randint(low, -8, m.shape, generator=g).double()) * (-1.0 if at & 1 else 1.0)
            if at == 4:
                m[:] = 0.0
    return k.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [1, 2, 4, 8, 16, 32, 64, 128])
def test_page_means_are_rounded_once(dtype, D, ps):
    """min, max and mean of every page, exactly: whole pages, partly filled ones, pages completed by a second call; few
    pages (a page's rows shared by warps) and many."""
    import sparse_paged_kv_page_gb300 as S
    H, g = 8, torch.Generator().manual_seed(ps + D)
    rope = S.make_rope(None)                              # no rotation, no norm: the keys are stored as they come
    for first, second in ((3 * ps + (ps + 1) // 2, 5 * ps), (0, 1500 * min(ps, 16) + 1)):
        n = first + second
        pages = -(-n // ps)
        keys = torch.cat([_columns(min(ps, n - p * ps), H, D, dtype, g) for p in range(min(pages, 12))])
        if pages > 12:                                    # the same twelve pages again and again
            keys = torch.cat([keys.repeat(-(-pages // 12), 1, 1)[: n]])
        keys = keys.cuda()
        k = torch.full((pages, H, ps, D), float("nan"), dtype=dtype, device="cuda")
        meta = torch.full((pages, H, 3, D), 7.0, dtype=dtype, device="cuda")
        cache = S.make_cache(k, k.clone(), meta)
        lens = torch.zeros(1, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        table = torch.randperm(pages, generator=g).to(torch.int32).cuda()[None]
        batch = S.make_batch(table, lens)
        for part in (keys[:first], keys[first:]):
            if part.shape[0]:
                cu = torch.tensor([0, part.shape[0]], dtype=torch.int32, device="cuda")
                S.sa_append_kv_rope(cache, batch, rope, None, part, part, cu, part.shape[0], None, dev_status=status)
        torch.cuda.synchronize()
        assert int(status) == 0 and lens.tolist() == [n]
        got = meta[table[0].long()]                       # [pages, H, 3, D]
        whole = n // ps
        groups = [(got[:whole], keys[: whole * ps].view(whole, ps, H, D).transpose(1, 2))]
        if n % ps:
            groups.append((got[whole:], keys[whole * ps:].transpose(0, 1)[None]))
        for m, rows in groups:
            assert torch.equal(m[:, :, 0], rows.amin(2)) and torch.equal(m[:, :, 1], rows.amax(2))
            want = _round_once(rows.double().sum(2) / rows.shape[2], dtype)
            off = m[:, :, 2] != want
            assert not bool(off.any()), f"{int(off.sum())} means, first at {off.nonzero()[0].tolist()}"


@pytest.mark.parametrize("ps", [4, 16, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_page_statistics_of_wide_ranges_are_those_of_the_plain_append(D, ps):
    """bf16 columns over all its exponents, with infinities and NaN: the same bits from both appends."""
    import sparse_paged_kv_page_gb300 as S
    H, n, g = 4, 5 * ps + ps // 2, torch.Generator().manual_seed(ps)
    keys = torch.randn((n, H, D), generator=g, dtype=torch.float64)
    keys *= torch.exp2(torch.randint(-130, 127, (n, 1, D), generator=g).double())
    keys[:, 0] = torch.exp2(torch.randint(-133, 127, (1, D), generator=g).double()) * torch.randint(-3, 4, (n, D), generator=g)
    keys[1, 1, 5::16], keys[2, 1, 6::16], keys[3, 2, 7::16] = float("inf"), -float("inf"), float("nan")
    keys[4, 1, 5::32] = -float("inf")
    keys = keys.to(torch.bfloat16).cuda()
    pages, metas = -(-n // ps), []
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for rotated in (False, True):
        k = torch.zeros((pages, H, ps, D), dtype=torch.bfloat16, device="cuda")
        meta = torch.full((pages, H, 3, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lens = torch.zeros(1, dtype=torch.int32, device="cuda")
        cache, batch = S.make_cache(k, k.clone(), meta), S.make_batch(table, lens)
        if rotated:
            S.sa_append_kv_rope(cache, batch, S.make_rope(None), None, keys, keys, cu, n, None)
        else:
            S.sa_append_kv(cache, batch, keys, keys, cu, n)
        metas.append(meta)
    torch.cuda.synchronize()
    a, b = metas
    assert torch.equal(a.isnan(), b.isnan())
    assert torch.equal(torch.where(a.isnan(), 0, a).view(torch.int16), torch.where(b.isnan(), 0, b).view(torch.int16))
