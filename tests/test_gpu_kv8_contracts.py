"""The calls over a cache held in 8 bits at what their documentation says beside the results: which rows a NaN reaches,
which scale bytes a cache may hold, what weights the rows of a call get, what is flagged, counters that are zero again."""
import pytest
import torch

from kv8_util import E4M3, Problem8, attention8, held64, quantise64
from paged_util import check_attention

pytestmark = pytest.mark.gpu


def _offsets(new):
    return torch.tensor([0] + [sum(new[: i + 1]) for i in range(len(new))], dtype=torch.int32).cuda()


def _prefill(p, q, new, ws=None, **kw):
    T = q.shape[0]
    ws = p.S.alloc_paged_prefill8_workspace(p.B, p.H, p.Hq, p.D, T) if ws is None else ws
    out, lse = torch.full_like(q, 3.0), torch.full((T, p.Hq), 3.0, device="cuda")
    p.S.sa_paged_prefill8(p.cache, p.batch, q, p.Hq, _offsets(new), kw.pop("scale", 0.0), out, lse=lse, workspace=ws,
                          dev_status=p.status, **kw)
    return out, lse


@pytest.mark.parametrize("parts,D", [(1, 128), (2, 64), (9, 128), (9, 64), (17, 128), (57, 128), (57, 64)])
def test_drafts_a_nan_key_or_value_in_any_part(parts, D):
    """Four drafted tokens of one request whose tiles are cut into that many parts of 128 tokens for each of 8 KV heads: a
    key that is NaN makes out and lse of the rows that see it NaN, a value their out, and nothing else, wherever it lies."""
    L, head = 128 * parts, 3
    p = Problem8([L], Hkv=8, G=4, D=D)
    q = p.rand(4, 32, D)
    rows = slice(4 * head, 4 * head + 4)
    for token in sorted({0, 60, L // 2, L - 130, L - 100, L - 3, L - 1} & set(range(L))):
        blk, slot = int(p.table[0, token // 16]), token % 16
        for x in range(2):
            if x == 1 and token >= L - 4:                             # (a value that some row does not see is to be finite)
                continue
            old = int(p.scale[blk, head, x, slot])
            p.scale[blk, head, x, slot] = 255
            out, lse = _prefill(p, q, [4])
            p.scale[blk, head, x, slot] = old
            nan = torch.zeros((4, 32), dtype=torch.bool)
            nan[[t for t in range(4) if L - 4 + t >= token], rows] = True
            assert torch.equal(out.isnan().all(-1).cpu(), nan) and torch.equal(out.isnan().any(-1).cpu(), nan), (token, x)
            assert torch.equal(lse.isnan().cpu(), nan & (x == 0)), (token, x)
            assert bool(out[~nan.cuda()].isfinite().all())
    assert int(p.status) == 0


@pytest.mark.parametrize("T,D", [(40, 64), (40, 128), (700, 64), (700, 128), (2900, 64), (2900, 128)])
def test_prompts_a_nan_key_reaches_the_rows_that_see_it(T, D):
    """From codes, whole and in parts, and on pages in the workspace: as drafts, at the ends of the cache and of the chunk."""
    L = 3000
    p = Problem8([L], Hkv=2, G=16, D=D)
    q = p.rand(T, 32, D)
    for token in (0, L - T, L - T // 2, L - 2):
        blk, slot = int(p.table[0, token // 16]), token % 16
        old = int(p.scale[blk, 1, 0, slot])
        p.scale[blk, 1, 0, slot] = 255
        out, lse = _prefill(p, q, [T])
        p.scale[blk, 1, 0, slot] = old
        nan = torch.zeros((T, 32), dtype=torch.bool, device="cuda")
        nan[max(0, token - (L - T)):, 16:] = True
        assert torch.equal(out.isnan().all(-1), nan) and torch.equal(out.isnan().any(-1), nan) and torch.equal(lse.isnan(), nan), token
    assert int(p.status) == 0


ENDS = {torch.bfloat16: (63, 190), torch.float16: (112, 134)}


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("end", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
def test_every_call_agrees_at_the_ends_of_the_scale_bytes(dtype, end, D):
    """Keys and values whose scale bytes are the least or the largest that a cache of the type may hold: decode, lists of
    pages, drafts, prompts from codes and on pages, and reading back all take the row as c 2^(byte - 127)."""
    L, G = 3000, 16
    p = Problem8([L], Hkv=1, G=G, D=D, dtype=dtype)
    byte = ENDS[p.dt][end]
    e = byte - 127
    held, unit = [], []
    for x in range(2):
        code = quantise64(p.rand(L, 1, D).double(), p.dt)[0].float().to(E4M3)
        p.put(0, 0, L, x, code, torch.full((L, 1), byte, dtype=torch.uint8, device="cuda"))
        unit.append(code.double())
        held.append(held64(code, torch.full((L, 1), byte, dtype=torch.uint8, device="cuda")))
    scale = 2.0 ** -e / 2048

    def check(out, lse, q, n, half_weights):
        # the values in units of 2^e, so that the tolerance's absolute terms are those of numbers near 1
        o, l, tol, tol_l = attention8(q, held[0], unit[1], torch.zeros_like(p.exps[0]), torch.arange(L - n, L, device="cuda"), scale,
                                      0, 0, half_weights)
        if p.dt == torch.float16:
            tol = tol + 2.0 ** (-25 - e)                              # half a step of subnormal outputs
        check_attention(out.double() * 2.0 ** -e, lse, (o, l, tol, tol_l))

    S = p.S
    q = p.rand(1, G, D)
    out, lse = torch.empty_like(q), torch.empty((1, G), device="cuda")
    ws = S.alloc_paged_decode8_workspace(1, 1, G, D)
    S.sa_paged_decode8(p.cache, p.batch, q, G, scale, out, lse=lse, workspace=ws, dev_status=p.status)
    check(out, lse, q, 1, True)
    n = -(-L // 16)
    sel = torch.arange(n, dtype=torch.int32, device="cuda").view(1, 1, n)
    S.sa_sparse_decode8(p.cache, p.batch, q, G, sel, torch.full((1, 1), n, dtype=torch.int32, device="cuda"), n, scale, out, lse=lse,
                        workspace=ws, dev_status=p.status)
    check(out, lse, q, 1, True)
    for T, few in ((1, True), (40, False), (2900, False)):            # by warps, from codes, on pages
        q = p.rand(T, G, D)
        check(*_prefill(p, q, [T], scale=scale), q, T, few)
    rows = [torch.empty((L, 1, D), dtype=p.dt, device="cuda") for _ in range(2)]
    S.sa_read_kv8(p.cache, p.batch, _offsets([L]), None, *rows, dev_status=p.status)
    for x in range(2):
        assert torch.equal(rows[x].double(), held[x])
    assert int(p.status) == 0


@pytest.mark.parametrize("lens,new,kw", [
    ([6000, 2500, 9], [3, 8, 1], dict(Hkv=2, G=4, D=64)), ([30_000], [2], dict(Hkv=1, G=8)),
    ([5000, 700, 40, 1, 0, 33, 260, 9], [1, 15, 1, 1, 0, 1, 2, 0], dict(Hkv=3, G=4)),
    ([5000, 700, 40, 1, 0, 33, 260, 9], [1, 7, 1, 1, 0, 1, 2, 0], dict(Hkv=3, G=8, D=64)),
    ([2600] + [40 + 9 * i for i in range(63)], [70] + [1] * 63, dict(Hkv=2, G=4)),
    ([2600] + [40 + 9 * i for i in range(63)], [190] + [1] * 63, dict(Hkv=2, G=8, D=64, ps=4))])
def test_requests_of_few_rows_on_the_mean_get_16_bit_weights_of_11_bits(lens, new, kw):
    """Calls of bfloat16 whose requests have few rows on the mean, and all of their requests, long ones too: weights are
    rounded as in sa_paged_decode8 (2^-11), not to the element type."""
    p = Problem8(lens, **kw)
    assert sum(new) * p.G <= (32 if p.D == 64 or p.B * p.H >= 16 else 16) * p.B
    for window, n_sink in ((0, 0), (300, 4)):
        q = p.rand(sum(new), p.Hq, p.D, scale=2.0)
        out, lse = _prefill(p, q, new, window=window, n_sink=n_sink)
        cu = _offsets(new).tolist()
        for b, L in enumerate(p.lens):
            r = slice(cu[b], cu[b + 1])
            want = attention8(q[r], *p.seqs[b], p.exps[b], torch.arange(L - new[b], L, device="cuda"), p.D ** -0.5, window, n_sink, True)
            check_attention(out[r], lse[r], want)
    assert int(p.status) == 0


@pytest.mark.parametrize("D", [64, 128])
def test_all_counters_of_a_workspace_are_zero_after_every_call(D):
    """The counters are four for each SM of the device, whatever the call's size."""
    counters = 4 * 4 * torch.cuda.get_device_properties(0).multi_processor_count
    p = Problem8([40_000, 9, 2500, 0], Hkv=4, G=4, D=D)
    S = p.S
    for T, new in ((4, [1, 1, 1, 1]), (14, [5, 0, 9, 0]), (700, [300, 9, 391, 0]), (2500, [0, 0, 2500, 0])):
        q = p.rand(T, p.Hq, D)
        ws = S.alloc_paged_prefill8_workspace(p.B, p.H, p.Hq, D, T)
        first, _ = _prefill(p, q, new if T > 4 else [1, 1, 1, 0], ws=ws)
        assert not bool(ws[:counters].any())
        again, _ = _prefill(p, q, new if T > 4 else [1, 1, 1, 0], ws=ws)
        assert torch.equal(first, again) and not bool(ws[:counters].any())
    ws = S.alloc_paged_decode8_workspace(p.B, p.H, p.Hq, D)
    q = p.rand(p.B, p.Hq, D)
    out = torch.empty_like(q)
    S.sa_paged_decode8(p.cache, p.batch, q, p.Hq, 0.0, out, workspace=ws, dev_status=p.status)
    assert not bool(ws[:counters].any())
    n = 2500
    sel = torch.arange(n, dtype=torch.int32, device="cuda").expand(p.B, p.H, n).contiguous()
    cnt = torch.tensor([n, 1, 157, 0], dtype=torch.int32, device="cuda")[:, None].expand(p.B, p.H).contiguous()
    S.sa_sparse_decode8(p.cache, p.batch, q, p.Hq, sel, cnt, n, 0.0, out, workspace=ws, dev_status=p.status)
    assert not bool(ws[:counters].any()) and int(p.status) == 0


def test_every_kind_of_bad_data_of_a_decode_is_flagged():
    p = Problem8([100, 50, 20], Hkv=1, G=2)
    q = p.rand(3, 2, 128)
    ws, out = p.S.alloc_paged_decode8_workspace(3, 1, 2, 128), torch.empty_like(q)
    for change, bit in ((lambda: None, 0), (lambda: p.table[0, 1].fill_(-5), 1), (lambda: p.seq_lens[1].fill_(100_000), 2),
                        (lambda: p.seq_lens[2].fill_(-3), 4)):
        change()
        p.status.zero_()
        p.S.sa_paged_decode8(p.cache, p.batch, q, 2, 0.0, out, workspace=ws, dev_status=p.status)
        assert int(p.status) & 7 & ~(2 * bit - 1 if bit else 0) == 0 and (int(p.status) & bit) == bit
    assert int(p.status) == 7


@pytest.mark.parametrize("G,rows", [(4, 8), (4, 600)])
def test_offsets_that_decrease_leave_their_request_without_rows(G, rows):
    """By warps and by the tensor cores: a request whose offsets decrease has no rows, and the others theirs."""
    p = Problem8([900, 900, 900], Hkv=1, G=G)
    q = p.rand(rows, G, 128)
    out, ws = torch.full_like(q, 3.0), p.S.alloc_paged_prefill8_workspace(3, 1, G, 128, rows)
    n = rows - 4
    cu = torch.tensor([0, n, n - 2, rows - 2], dtype=torch.int32).cuda()
    p.S.sa_paged_prefill8(p.cache, p.batch, q, G, cu, 0.0, out, workspace=ws, dev_status=p.status)
    assert int(p.status) == 0
    want = attention8(q[:n - 2], *p.seqs[0], p.exps[0], torch.arange(900 - n, 898, device="cuda"), 128 ** -0.5, 0, 0, rows == 8)
    check_attention(out[:n - 2], None, want)
    want = attention8(q[n:n + 2], *p.seqs[2], p.exps[2], torch.arange(898, 900, device="cuda"), 128 ** -0.5, 0, 0, rows == 8)
    check_attention(out[n:n + 2], None, want)
    assert bool((out[n + 2:] == 3.0).all())


@pytest.mark.parametrize("T,D", [(3000, 64), (6000, 128)])
def test_a_workspace_for_more_requests_serves_fewer(T, D):
    """The size for 64 requests has no room for 16-bit pages, which one request of as many tokens would like: it runs without."""
    G = 16
    p = Problem8([T], Hkv=1, G=G, D=D)
    most, one = (p.S.sa_paged_prefill8_workspace_size(b, 1, G, D, T) for b in (64, 1))
    assert most < one
    ws = p.S.alloc_paged_prefill8_workspace(64, 1, G, D, T)
    q = p.rand(T, G, D)
    out, lse = _prefill(p, q, [T], ws=ws)
    for r in (slice(0, 300), slice(T - 300, T)):
        want = attention8(q[r], *p.seqs[0], p.exps[0], torch.arange(r.start, r.stop, device="cuda"), D ** -0.5, 0, 0, False)
        check_attention(out[r], lse[r], want)
    for T, new in ((2, [2]), (100, [100]), (1000, [1000])):
        q = p.rand(T, G, D)
        out, lse = _prefill(p, q, new, ws=ws)
        want = attention8(q, *p.seqs[0], p.exps[0], torch.arange(p.lens[0] - T, p.lens[0], device="cuda"), D ** -0.5, 0, 0, T == 2)
        check_attention(out, lse, want)
    assert int(p.status) == 0


@pytest.mark.parametrize("kw,new", [
    (dict(lens=[6000, 300, 9], Hkv=2, G=4), [5, 3, 1]), (dict(lens=[6000, 300, 9, 0], Hkv=4, G=7), [8, 3, 1, 0]),
    (dict(lens=[3000], Hkv=2, G=16, D=64), [40]), (dict(lens=[9000, 2500], Hkv=8, G=4), [400, 300]),
    (dict(lens=[6000], Hkv=1, G=16), [6000])])
def test_prompts_and_drafts_into_their_queries(kw, new):
    """out may be q itself: by warps, from codes, in parts and on pages the same bits as into rows of their own."""
    lens = kw.pop("lens")
    p = Problem8(lens, **kw)
    q = p.rand(sum(new), p.Hq, p.D, scale=2.0)
    out, lse = _prefill(p, q, new)
    ws, lse2 = p.S.alloc_paged_prefill8_workspace(p.B, p.H, p.Hq, p.D, sum(new)), torch.empty_like(lse)
    for _ in range(3):
        x = q.clone()
        p.S.sa_paged_prefill8(p.cache, p.batch, x, p.Hq, _offsets(new), 0.0, x, lse=lse2, workspace=ws, dev_status=p.status)
        assert torch.equal(x, out) and torch.equal(lse, lse2)
    assert int(p.status) == 0
