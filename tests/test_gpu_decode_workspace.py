"""sa_sparse_decode with more splits than a cluster holds (its splits then meet by counters in the workspace): one buffer
for calls of other sizes, against the plain float64 form."""
import pytest
import torch

from paged_util import Problem, attention64, check_attention

pytestmark = pytest.mark.gpu


def test_one_workspace_serves_batches_of_other_sizes():
    import sparse_paged_kv_page_gb300 as S
    stride = 36_000                                       # entries of a selection: 9 splits of at most 4096
    calls = []
    for seed, lens in enumerate(([2000], [40 + 9 * i for i in range(11)], [700, 1, 90])):
        p = Problem(lens, Hkv=8, G=2, ps=1, D=64, seed=seed)
        sel = torch.zeros((p.B, 8, stride), dtype=torch.int32, device="cuda")
        sel[:, :, : max(lens)] = torch.arange(max(lens), dtype=torch.int32, device="cuda")
        cnt = p.seq_lens[:, None].expand(p.B, 8).contiguous()     # every cached token is selected
        calls.append((p, p.rand(p.B, 16, 64, scale=2.0), sel, cnt))
    shared = torch.zeros(max(S.sa_decode_workspace_size(p.B, 8, 16, 64, 1, stride) for p, *_ in calls), dtype=torch.uint8,
                         device="cuda")
    for i in (0, 1, 2, 1, 0, 1):
        p, q, sel, cnt = calls[i]
        out = torch.full_like(q, float("nan"))
        lse = torch.full((p.B, 16), float("nan"), device="cuda")
        S.sa_sparse_decode(p.cache, p.batch, q, 16, sel, cnt, stride, 0.0, out, lse=lse, workspace=shared,
                           dev_status=p.status)
        torch.cuda.synchronize()
        assert int(p.status) == 0
        for b, L in enumerate(p.lens):
            check_attention(out[b:b + 1], lse[b:b + 1],
                            attention64(q[b:b + 1], *p.seqs[b], torch.tensor([L - 1], device="cuda"), 64 ** -0.5, 0, 0))
