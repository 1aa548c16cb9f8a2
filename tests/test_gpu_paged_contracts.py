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
