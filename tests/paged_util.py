"""Plain float64 forms of the whole-layer operators (rotated append, attention over the whole paged cache) and
small problems for them. Independent of the oracle's sparse step and of the package's kernels."""
import math

import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dtype):
    """Largest relative error of one rounding to the type."""
    return torch.finfo(dtype).eps / 2


class Problem:
    """A paged cache with shuffled pages whose unwritten slots and unreferenced blocks hold NaN."""

    def __init__(self, lens, *, Hkv=2, G=4, D=128, ps=16, dtype="bf16", seed=0, extra_pages=1, meta=False, std=False):
        import sparse_paged_kv_page_gb300 as S
        self.S, self.lens, self.H, self.G, self.D, self.ps = S, list(lens), Hkv, G, D, ps
        self.dt, self.B, self.Hq = DT[dtype], len(lens), Hkv * G
        g = self.gen = torch.Generator().manual_seed(1000 + seed)
        self.stride = max(-(-n // ps) for n in self.lens) + extra_pages
        blocks = self.B * self.stride + 2
        perm = torch.randperm(blocks, generator=g)[: self.B * self.stride].to(torch.int32)
        self.table = perm.view(self.B, self.stride).cuda()
        pool = lambda: torch.full((blocks, Hkv, ps, D), float("nan"), dtype=self.dt).cuda()  # noqa: E731
        self.k, self.v = pool(), pool()
        self.meta = torch.full((blocks, Hkv, 3, D), 7.0, dtype=self.dt).cuda() if meta else None
        self.std = torch.full((blocks, Hkv, D), 7.0, dtype=self.dt).cuda() if std else None
        self.seqs = []
        for b, n in enumerate(self.lens):
            kv = [self.rand(n, Hkv, D), self.rand(n, Hkv, D)]
            self.seqs.append(kv)
            for j0 in range(0, n, ps):
                blk, m = int(self.table[b, j0 // ps]), min(ps, n - j0)
                self.k[blk, :, :m] = kv[0][j0:j0 + m].transpose(0, 1)
                self.v[blk, :, :m] = kv[1][j0:j0 + m].transpose(0, 1)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.status = torch.zeros(1, dtype=torch.int32).cuda()
        self.bind()

    def rand(self, *shape, scale=1.0):
        return (scale * torch.randn(shape, generator=self.gen)).to(self.dt).cuda()

    def bind(self):
        self.cache = self.S.make_cache(self.k, self.v, self.meta, self.std)
        self.batch = self.S.make_batch(self.table, self.seq_lens)

    def rows(self, b, n, pool=None):
        """The first n token rows of request b in a pool, [n, H, D]."""
        pool = self.k if pool is None else pool
        pages = self.table[b, : -(-n // self.ps)].long()
        return pool[pages].transpose(1, 2).reshape(-1, self.H, self.D)[:n]


def visible(i, j, window, n_sink):
    see = j <= i
    return see & ((j > i - window) | (j < n_sink)) if window else see


def attention64(q, k, v, pos, scale, window, n_sink):
    """q [n, Hq, D] at positions pos [n], k and v [L, H, D]: out, lse, and the tolerances of a kernel that keeps
    sums in 32 bits, rounds the weights p once to the element type and the output once.

    With u the half step: |o - o*| <= u sum p|v| (weights) + 2 d sum p|v| (logits off by d, in numerator and
    denominator) + u |o*| (output), d = (D + 4) 2^-24 scale max_j sum_d |q_d k_jd| + 2^-20 (dot product, exponential,
    sums of up to 64 terms in a row a lane). Weights below fp16's normal range are off by 2^-25 absolutely."""
    n, Hq, D = q.shape
    L, H = k.shape[0], k.shape[1]
    out = torch.zeros((n, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    if L == 0:
        return out, lse, tol, tol_lse
    u = half_step(q.dtype)
    j = torch.arange(L, device=q.device)[None]
    see = visible(pos[:, None], j, window, n_sink)
    for h in range(Hq):
        kh, vh, qh = k[:, h // (Hq // H)].double(), v[:, h // (Hq // H)].double(), q[:, h].double()
        z = torch.where(see, qh @ kh.t() * scale, torch.tensor(-math.inf, dtype=torch.float64, device=q.device))
        m = z.amax(1, keepdim=True)
        p = torch.where(see, (z - m.clamp(min=-1e300)).exp(), torch.zeros_like(z))
        l = p.sum(1, keepdim=True)
        some = l > 0
        w = torch.where(some, p / l.clamp(min=1e-300), torch.zeros_like(p))
        out[:, h] = w @ vh
        lse[:, h] = torch.where(some, m + l.log(), m)[:, 0]
        size = torch.where(see, qh.abs() @ kh.abs().t() * scale, torch.zeros_like(z)).amax(1, keepdim=True)
        d = (D + 4) * 2.0 ** -24 * size + 2.0 ** -20 + L / 16 * 2.0 ** -24
        av = w @ vh.abs()
        tol[:, h] = (u + 2 * d) * av + u * out[:, h].abs() + 1e-7
        if q.dtype == torch.float16:
            tol[:, h] += 2.0 ** -25 * (see.double() @ vh.abs()) / l.clamp(min=1.0) + 2.0 ** -25
        tol_lse[:, h] = (d + 2.0 ** -22 * (1 + lse[:, h].abs().nan_to_num(posinf=0, neginf=0))[:, None])[:, 0]
    return out, lse, tol, tol_lse


def check_attention(out, lse, want):
    o, l, tol, tol_l = want
    err = (out.double() - o).abs()
    assert bool((err <= tol).all()), f"output off by {float((err / tol.clamp(min=1e-300)).max()):.3g} tolerances"
    if lse is not None:
        fin = torch.isfinite(l)
        assert bool((torch.isneginf(lse.double()) == ~fin).all())
        assert bool(((lse.double() - l).abs()[fin] <= tol_l[fin]).all()), float((lse.double() - l).abs()[fin].max())


def rotate64(x, w, eps, place, theta, rot, interleaved, sections):
    """Norm (if w) and rotation of x [T, H, D]; place [axes, T]. Also the tolerance of one rounding of a float32 result:
    u |y| + the float32 errors, (D + 8) 2^-24 of the pair's larger part, and the table's own rounding."""
    y = x.double()
    D = x.shape[-1]
    if w is not None:
        y = y / ((y * y).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    r = rot // 2
    freq = theta ** (-2.0 * torch.arange(r, dtype=torch.float64, device=x.device) / max(rot, 1))
    axis = torch.repeat_interleave(torch.arange(len(sections), device=x.device), torch.tensor(sections, device=x.device))
    a = place.double()[axis].t() * freq                      # [T, r]
    c, s = a.cos()[:, None], a.sin()[:, None]
    out, big = y.clone(), y.abs().clone()
    i0, i1 = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, r), slice(r, rot))
    u, v = y[..., i0], y[..., i1]
    out[..., i0], out[..., i1] = u * c - v * s, u * s + v * c
    big[..., i0] = big[..., i1] = u.abs() + v.abs()
    tol = half_step(x.dtype) * out.abs() + (D + 8) * 2.0 ** -24 * big
    if x.dtype == torch.float16:
        tol += 2.0 ** -25
    return out, tol
