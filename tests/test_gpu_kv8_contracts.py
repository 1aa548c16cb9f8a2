"""The calls over a cache held in 8 bits at what their documentation says beside the results: which rows a NaN reaches."""
import pytest
import torch

from kv8_util import Problem8

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
