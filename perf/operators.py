"""Cases of the operators that serve whole attention layers over the paged KV cache:

  append   ``sa_append_kv_rope``: per-head RMS norm and rotation of queries and keys, the rotated keys and the
           values written into their pages, the written pages' key statistics recomputed;
  decode   ``sa_paged_decode``: one new token per request over its whole cache, or a sliding window of it and the
           first few tokens;
  prefill  ``sa_paged_prefill``: the prompt's (or a chunk's) tokens over the cache, causal, with the same window.

``run`` makes the framework's call where ``own`` is true; elsewhere it computes the plain form in torch. Ragged
lengths are spread over [lo, hi] by the golden ratio, so that a case's work does not depend on the seed.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------------------------------- cases
def listed():
    append = dict(op="append", D=128, ps=16, rot=128, interleaved=False, axes=1, norm=False, window=0, sink=0)
    attend = dict(D=128, ps=16, window=0, sink=0)
    return [
        # one token of one request: launch and latency
        dict(append, name="append_one", B=1, Hq=32, Hkv=8, dtype="fp16", lo=1024, hi=1024, nlo=1, nhi=1),
        # one token of each request of a ragged batch, with query and key norms
        dict(append, name="append_batch", B=16, Hq=32, Hkv=8, dtype="bf16", norm=True, lo=2048, hi=8192, nlo=1, nhi=1),
        # a ragged batch of prompts with image tokens: positions of three axes, half of each head rotated in pairs
        dict(append, name="append_axes", B=5, Hq=28, Hkv=4, dtype="bf16", rot=64, interleaved=True, axes=3, lo=0,
             hi=777, nlo=17, nhi=2501),
        # long prompts of four requests
        dict(append, name="append_prompt", B=4, Hq=64, Hkv=8, dtype="bf16", norm=True, lo=0, hi=0, nlo=8192, nhi=8192),
        # one request of 1024 tokens
        dict(attend, name="decode_one", op="decode", B=1, Hq=32, Hkv=8, dtype="fp16", lo=1024, hi=1024),
        # a ragged batch
        dict(attend, name="decode_batch", op="decode", B=16, Hq=32, Hkv=8, dtype="bf16", lo=2048, hi=32768),
        # a token-level cache (pages of one token) behind a sliding window and four first tokens
        dict(attend, name="decode_window", op="decode", B=32, Hq=32, Hkv=8, ps=1, dtype="bf16", lo=100, hi=16384,
             window=4096, sink=4),
        # four requests of 128 k tokens
        dict(attend, name="decode_long", op="decode", B=4, Hq=64, Hkv=8, dtype="bf16", lo=131072, hi=131072),
        # a few tokens of each request (a draft to verify) over long caches
        dict(attend, name="prefill_few", op="prefill", B=4, Hq=32, Hkv=8, dtype="bf16", lo=8000, hi=30001, nlo=3, nhi=8),
        # ragged prompts with a sliding window, small heads
        dict(attend, name="prefill_window", op="prefill", B=4, Hq=16, Hkv=2, D=64, dtype="fp16", lo=0, hi=1000, nlo=33,
             nhi=8191, window=1024, sink=4),
        # one long prompt
        dict(attend, name="prefill_prompt", op="prefill", B=1, Hq=32, Hkv=8, dtype="bf16", lo=0, hi=0, nlo=16384, nhi=16384),
        # a chunk of a prompt far into a long context
        dict(attend, name="prefill_chunk", op="prefill", B=1, Hq=64, Hkv=8, dtype="bf16", lo=64000, hi=64000, nlo=2048,
             nhi=2048),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    c = dict(op=rng.choice(["append", "decode", "prefill"]), D=rng.choice([64, 128, 128]), ps=rng.choice([1, 2, 8, 16, 16, 32, 64, 128]),
             dtype=rng.choice(["bf16", "fp16"]), Hkv=rng.choice([1, 2, 4, 8]), window=0, sink=0)
    c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if c["op"] == "append":
        c.update(B=_log(rng, 1, 32), axes=rng.choice([1, 1, 3, 4]), norm=rng.random() < 0.5, interleaved=rng.random() < 0.4,
                 rot=rng.choice([c["D"], c["D"], c["D"] // 2]))
        c["hi"] = _log(rng, 1, 4096) - 1
        c["nhi"] = 1 if rng.random() < 0.3 else _log(rng, 1, max(1, min(8192, 150_000_000 // (c["B"] * c["Hq"] * c["D"]))))
    elif c["op"] == "decode":
        c["B"] = _log(rng, 1, 64)
        c["hi"] = _log(rng, 1, min(131072, 268_435_456 // (c["B"] * c["Hkv"] * c["D"])))
        c["lo"] = rng.randint(0, c["hi"])
    else:
        c["B"] = _log(rng, 1, 8)
        c["hi"] = _log(rng, 1, 32768) - 1
        c["nhi"] = _log(rng, 1, min(8192, max(8, 4_000_000_000 // (c["B"] * c["Hq"] * (c["hi"] + 8192)))))
    if c["op"] != "decode":
        c["lo"], c["nlo"] = rng.randint(0, c["hi"]), rng.randint(1, c["nhi"])
    if c["op"] != "append" and rng.random() < 0.4:
        c["window"], c["sink"] = _log(rng, 1, 4096), rng.randint(0, 16)
    return c


def _spread(lo, hi, n, turn):
    """n whole numbers in [lo, hi], the last of them hi."""
    v = [lo + int((hi - lo + 1) * ((i + 1) * turn % 1.0)) for i in range(n)]
    return v[:-1] + [hi]


def _lengths(c):
    """(tokens cached before, new tokens) of each request."""
    old = _spread(c["lo"], c["hi"], c["B"], 0.6180339887)
    return old, _spread(c["nlo"], c["nhi"], c["B"], 0.7548776662) if c["op"] != "decode" else [0] * c["B"]


def _sections(c):
    """Pairs of dimensions that each axis of the positions turns."""
    half, n = c["rot"] // 2, c["axes"]
    rest = half * 3 // (4 * (n - 1)) if n > 1 else 0
    return [half - rest * (n - 1)] + [rest] * (n - 1)


def _visible(c):
    """Pairs of (new token, visible token), and the tokens of the cache that some new one sees, over all requests."""
    pairs = seen = 0
    for o, n in zip(*_lengths(c)):
        o, n = (o - 1, 1) if c["op"] == "decode" else (o, n)
        w, s = c["window"] or o + n, c["sink"]
        i = range(o, o + n)
        pairs += sum(min(p + 1, w) + max(0, min(s, p + 1 - w)) for p in i if p >= 0)
        seen += min(o + n, w + n - 1) + max(0, min(s, o + n - (w + n - 1)))
    return pairs, seen


def work(c):
    e, D = 2, c["D"]
    if c["op"] == "append":
        old, new = _lengths(c)
        T, ps = sum(new), c["ps"]
        pages = sum((o + n - 1) // ps - o // ps + 1 for o, n in zip(old, new))
        before = sum(o % ps for o in old)
        rows = T * (2 * c["Hq"] + 4 * c["Hkv"]) + (before + 3 * pages) * c["Hkv"]
        return {"bytes": rows * D * e + T * c["rot"] * 4, "flops": T * (c["Hq"] + c["Hkv"]) * D * (7 if c["norm"] else 3)}
    pairs, seen = _visible(c)
    T = c["B"] if c["op"] == "decode" else sum(_lengths(c)[1])
    return {"bytes": (2 * seen * c["Hkv"] + 2 * T * c["Hq"]) * D * e + 4 * T * c["Hq"], "flops": 4 * pairs * c["Hq"] * D}


# -------------------------------------------------------------------------------------------------- inputs
def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, B, Hq, Hkv, D, ps = DT[c["dtype"]], c["B"], c["Hq"], c["Hkv"], c["D"], c["ps"]
    normal = lambda *shape: torch.randn(shape, dtype=torch.float32, device="cuda", generator=gen)  # noqa: E731
    old, new = _lengths(c)
    total = [o + n for o, n in zip(old, new)]
    stride = max(1, max(-(-t // ps) for t in total))
    blocks = B * stride + 3
    # pages anywhere in the pool; keys with a direction that a head's tokens share, as projections give them
    table = torch.randperm(blocks, device="cuda", generator=gen)[: B * stride].to(torch.int32).view(B, stride)
    kv = [torch.randn((blocks, Hkv, ps, D), dtype=dt, device="cuda", generator=gen) for _ in range(2)]
    kv[0] += (0.5 * normal(1, Hkv, 1, D)).to(dt)
    kv[1] += (0.25 * normal(1, Hkv, 1, D)).to(dt)
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + [sum(new[: i + 1]) for i in range(B)], dtype=torch.int32, device="cuda")
    T = sum(new) if c["op"] != "decode" else B
    s = dict(case=c, k=kv[0], v=kv[1], table=table, lens=lens, cu=cu, most_new=max(new), longest=max(total))
    if c["op"] == "append":
        qkv = (normal(T, Hq + 2 * Hkv, D) * 1.5).to(dt)  # one projection's output, split without a copy
        s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["weights"] = [(1 + 0.1 * normal(D)).to(dt) for _ in range(2)] if c["norm"] else [None, None]
        most = s["longest"] + 64
        freq = 500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        angle = torch.arange(most, dtype=torch.float64, device="cuda")[:, None] * freq
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["axis"] = torch.repeat_interleave(torch.arange(c["axes"], device="cuda"), torch.tensor(_sections(c), device="cuda"))
        # text tokens have their place on every axis; with several axes, runs of image tokens lie on a grid 32 wide
        first = torch.tensor([o - a for o, a in zip(old, [sum(new[:i]) for i in range(B)])], device="cuda")
        place = torch.arange(T, device="cuda") + first.repeat_interleave(torch.tensor(new, device="cuda"))
        grid = [place, place // 32, place % 32, place // 64][: c["axes"]]
        s["positions"] = torch.stack([torch.where(place % 256 < 128, g, place) for g in grid]).to(torch.int32)
        s["meta"] = torch.zeros((blocks, Hkv, 3, D), dtype=dt, device="cuda")
        s["q_out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
    else:
        s["q"] = (1.5 * normal(T, Hq, D)).to(dt)
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((T, Hq), dtype=torch.float32, device="cuda")
    if own:  # the handles on these buffers that a program keeps for a layer, and its workspace
        import sparse_paged_kv_page_gb300 as S
        s["cache"], s["batch"] = S.make_cache(s["k"], s["v"], s.get("meta")), S.make_batch(table, lens)
        if c["op"] == "append":
            s["rotation"] = S.make_rope(s["rope"], interleaved=c["interleaved"], sections=_sections(c), eps=1e-6,
                                        positions=s["positions"] if c["axes"] > 1 else None,
                                        q_weight=s["weights"][0], k_weight=s["weights"][1])
        elif c["op"] == "decode":
            s["workspace"] = S.alloc_paged_decode_workspace(B, Hkv, Hq, D)
        else:
            s["workspace"] = S.alloc_paged_prefill_workspace(B, Hkv, Hq, D, T)
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _rotate(x, weight, angles, c):
    """Norm over each head (if it has weights), then the rotation of its first `rot` dimensions, in 32 bits."""
    y, rot, dt = x.float(), c["rot"], x.dtype
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    cos, sin = angles[:, None, : rot // 2], angles[:, None, rot // 2:]
    turn = y[..., :rot]
    a, b = (turn[..., 0::2], turn[..., 1::2]) if c["interleaved"] else (turn[..., : rot // 2], turn[..., rot // 2:])
    parts = a * cos - b * sin, a * sin + b * cos
    turn = torch.stack(parts, -1).flatten(-2) if c["interleaved"] else torch.cat(parts, -1)
    return torch.cat([turn, y[..., rot:]], -1).to(dt)


def _append_plain(s):
    c, ps = s["case"], s["case"]["ps"]
    # angles of each token: the table's row of its position on each pair's axis
    at = s["positions"].long()[s["axis"]].t()                                   # [T, rot / 2]
    pair = torch.arange(at.shape[1], device=at.device)
    angles = torch.cat([s["rope"][at, pair], s["rope"][at, pair + at.shape[1]]], 1)
    q, k = _rotate(s["q"], s["weights"][0], angles, c), _rotate(s["k_new"], s["weights"][1], angles, c)
    # where each new token goes
    count = (s["cu"][1:] - s["cu"][:-1]).long()
    first = s["lens"].long() - count
    token = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(s["cu"][1:].long(), token, right=True)
    place = first[b] + token - s["cu"].long()[b]
    block, slot = s["table"][b, place // ps].long(), place % ps
    s["k"][block, :, slot] = k
    s["v"][block, :, slot] = s["v_new"]
    # statistics of the pages written: the first and every token that opens a page stands for its page
    head = (slot == 0) | (token == s["cu"].long()[b])
    page, pb, blk = place[head] // ps, b[head], block[head]
    fill = (s["lens"].long()[pb] - page * ps).clamp(max=ps)
    keys = s["k"][blk].float()                                                  # [pages, Hkv, ps, D]
    there = (torch.arange(ps, device=q.device) < fill[:, None])[:, None, :, None]
    s["meta"][blk, :, 0] = keys.masked_fill(~there, math.inf).amin(2).to(k.dtype)
    s["meta"][blk, :, 1] = keys.masked_fill(~there, -math.inf).amax(2).to(k.dtype)
    total = keys.double().masked_fill(~there, 0).sum(2)                         # the mean lies next to rounding borders
    s["meta"][blk, :, 2] = (total / fill[:, None, None]).to(k.dtype)
    return [q, s["k"], s["v"], s["meta"]]


def _attend_plain(s):
    c = s["case"]
    B, Hkv, G, D, ps, dt = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"], c["ps"], s["q"].dtype
    n, L = max(1, s["most_new"]), s["longest"]
    # requests side by side, padded to the longest
    if c["op"] == "decode":
        q, rows = s["q"][:, None], None
        place = s["lens"].long()[:, None] - 1
    else:
        step = torch.arange(n, device="cuda")
        rows = s["cu"][:-1].long()[:, None] + step
        rows = torch.where(rows < s["cu"][1:].long()[:, None], rows, -1)
        q = s["q"][rows.clamp(min=0)]
        place = s["lens"].long()[:, None] - (s["cu"][1:] - s["cu"][:-1]).long()[:, None] + step
    q = q.float().view(B, -1, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    pages = s["table"].long()
    k, v = (x[pages].transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L].float() for x in (s["k"], s["v"]))
    z = torch.matmul(q, k.transpose(-1, -2)).mul_(D ** -0.5).view(B, Hkv, G, -1, L)
    j, i = torch.arange(L, device="cuda"), place[..., None]
    seen = (j <= i) & (i < s["lens"].long()[:, None, None])
    if c["window"]:
        seen &= (j > i - c["window"]) | (j < c["sink"])
    z.masked_fill_(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-1e30)
    z.sub_(top).exp_()
    norm = z.sum(-1, keepdim=True)
    lse = (top + norm.log()).squeeze(-1)                                        # [B, Hkv, G, n]
    out = torch.matmul(z.view(B, Hkv, -1, L), v).view(B, Hkv, G, -1, D) / norm.clamp(min=1e-30)
    out, lse = out.permute(0, 3, 1, 2, 4).flatten(2, 3), lse.permute(0, 3, 1, 2).flatten(2, 3)
    if rows is None:
        return [out[:, 0].to(dt), lse[:, 0].contiguous()]
    return [out[rows >= 0].to(dt), lse[rows >= 0]]


def run(s):
    c = s["case"]
    if not own:
        return _append_plain(s) if c["op"] == "append" else _attend_plain(s)
    import sparse_paged_kv_page_gb300 as S
    if c["op"] == "append":
        # the batch's lengths were advanced once for all layers; this layer writes its tokens
        S.sa_append_kv_rope(s["cache"], s["batch"], s["rotation"], s["q"], s["k_new"], s["v_new"], s["cu"], s["most_new"],
                            s["q_out"], advanced=True)
        return [s["q_out"], s["k"], s["v"], s["meta"]]
    if c["op"] == "decode":
        S.sa_paged_decode(s["cache"], s["batch"], s["q"], c["Hq"], 0.0, s["out"], window=c["window"], n_sink=c["sink"],
                          lse=s["lse"], workspace=s["workspace"])
    else:
        S.sa_paged_prefill(s["cache"], s["batch"], s["q"], c["Hq"], s["cu"], 0.0, s["out"], window=c["window"],
                           n_sink=c["sink"], lse=s["lse"], workspace=s["workspace"])
    return [s["out"], s["lse"]]


# ------------------------------------------------------------------------------------- the definition, 64 bits
def _turned(x, weight, place, c):
    """Norm and rotation of one token's heads [H, D], as complex numbers times e^(i position frequency)."""
    x, rot = x.double(), c["rot"]
    if weight is not None:
        x = x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * weight.double()
    freq = torch.exp(torch.arange(rot // 2, dtype=torch.float64, device=x.device) * (-2 * math.log(500000.0) / rot))
    spin = torch.polar(torch.ones_like(freq).expand(place.shape), place.double() * freq)[:, None]
    y = x.clone()
    if c["interleaved"]:
        z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * spin
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., : rot // 2], x[..., rot // 2: rot]) * spin
        y[..., : rot // 2], y[..., rot // 2: rot] = z.real, z.imag
    return y


def exact(c, seed):
    s = prepare(c, seed)
    old, new = _lengths(c)
    ps, D, Hkv, G = c["ps"], c["D"], c["Hkv"], c["Hq"] // c["Hkv"]
    table = s["table"].cpu().tolist()
    if c["op"] == "append":
        place = torch.cat([s["positions"][a:a + 1].t().expand(-1, w) for a, w in enumerate(_sections(c))], 1)
        q, k = _turned(s["q"], s["weights"][0], place, c), _turned(s["k_new"], s["weights"][1], place, c)
        pool_k, pool_v, meta = s["k"].double(), s["v"].double(), s["meta"].double()
        row = 0
        for b in range(c["B"]):
            p0, p1 = old[b] // ps, (old[b] + new[b] - 1) // ps
            blocks = torch.tensor(table[b][p0:p1 + 1], device="cuda")
            flat = lambda pool: pool[blocks].transpose(1, 2).reshape(-1, Hkv, D)  # noqa: E731
            keys, values = flat(pool_k), flat(pool_v)
            at = old[b] - p0 * ps
            keys[at:at + new[b]], values[at:at + new[b]] = k[row:row + new[b]], s["v_new"][row:row + new[b]].double()
            row += new[b]
            paged = keys.view(-1, ps, Hkv, D).transpose(1, 2)
            pool_k[blocks], pool_v[blocks] = paged, values.view(-1, ps, Hkv, D).transpose(1, 2)
            end = at + new[b]
            whole = end // ps
            if whole:
                meta[blocks[:whole]] = torch.stack([paged[:whole].amin(2), paged[:whole].amax(2), paged[:whole].mean(2)], 2)
            if end % ps:
                part = paged[-1][:, : end % ps]
                meta[blocks[-1]] = torch.stack([part.amin(1), part.amax(1), part.mean(1)], 1)
        return [q, pool_k, pool_v, meta]
    if work(c)["flops"] > 6e12:
        return None
    outs, lses, row = [], [], 0
    for b in range(c["B"]):
        n = 1 if c["op"] == "decode" else new[b]
        L = old[b] if c["op"] == "decode" else old[b] + new[b]
        q = s["q"][row:row + n].double()
        row += n
        blocks = torch.tensor(table[b][: -(-L // ps)], device="cuda", dtype=torch.int64)
        k, v = (x[blocks].transpose(0, 1).reshape(Hkv, -1, D)[:, :L].double() for x in (s["k"], s["v"]))
        outs.append(torch.zeros((n, c["Hq"], D), dtype=torch.float64, device="cuda"))
        lses.append(torch.full((n, c["Hq"]), -math.inf, dtype=torch.float64, device="cuda"))
        for t in range(0, n if L else 0, 256):
            i = torch.arange(L - n + t, L - n + min(n, t + 256), device="cuda")[:, None]
            far = int(i[-1]) + 1
            j = torch.arange(far, device="cuda")
            hidden = j > i
            if c["window"]:
                hidden = hidden | ((i - j >= c["window"]) & (j >= c["sink"]))
            for h in range(c["Hq"]):
                z = (q[t:t + 256, h] @ k[h // G, :far].t() / math.sqrt(D)).masked_fill(hidden, -math.inf)
                lses[-1][t:t + 256, h] = torch.logsumexp(z, -1)
                outs[-1][t:t + 256, h] = torch.softmax(z, -1) @ v[h // G, :far]
    return [torch.cat(outs), torch.cat(lses)]
