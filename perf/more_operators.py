"""Cases of the operators over the 8-bit paged KV cache (e4m3 codes, one power-of-two scale per token and KV head):

  append   ``sa_append_kv8``: per-head RMS norm and rotation of queries and keys, the rotated keys and the values
           quantised into their pages, the written pages' key statistics recomputed;
  decode   ``sa_paged_decode8``: one new token per request over its whole cache, or a sliding window of it and the
           first few tokens;
  sparse   ``sa_sparse_decode8``: one new token per request over the pages selected for each KV head;
  prefill  ``sa_paged_prefill8``: the prompt's (or a chunk's) tokens over the cache, causal, with the same window;
  read     ``sa_read_kv8``: ranges of each request's cached tokens back as rows of 16 bits.

``run`` makes the framework's call where ``own`` is true; elsewhere it computes the plain form in torch. Ragged
lengths are spread over [lo, hi] by the golden ratio, so that a case's work does not depend on the seed.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# --------------------------------------------------------------------------------------------------- cases
def listed():
    append = dict(op="append", D=128, ps=16, rot=128, interleaved=False, axes=1, norm=False)
    attend = dict(D=128, ps=16, window=0, sink=0)
    return [
        # one token of each request of a ragged batch, with query and key norms: launch and latency
        dict(append, name="append_batch", B=16, Hq=32, Hkv=8, dtype="bf16", norm=True, lo=2048, hi=8192, nlo=1, nhi=1),
        # a ragged batch of prompts with image tokens: positions of three axes, half of each head rotated in pairs
        dict(append, name="append_axes", B=5, Hq=28, Hkv=4, dtype="fp16", rot=64, interleaved=True, axes=3, lo=0,
             hi=777, nlo=17, nhi=2501),
        # long prompts of four requests
        dict(append, name="append_prompt", B=4, Hq=64, Hkv=8, dtype="bf16", norm=True, lo=0, hi=0, nlo=8192, nhi=8192),
        # one request of 1024 tokens: latency
        dict(attend, name="decode_one", op="decode", B=1, Hq=32, Hkv=8, dtype="fp16", lo=1024, hi=1024),
        # a ragged batch
        dict(attend, name="decode_batch", op="decode", B=16, Hq=32, Hkv=8, dtype="bf16", lo=2048, hi=32768),
        # four requests of 128 k tokens
        dict(attend, name="decode_long", op="decode", B=4, Hq=64, Hkv=8, dtype="bf16", lo=131072, hi=131072),
        # the selected pages of a ragged batch
        dict(attend, name="sparse_batch", op="sparse", B=16, Hq=32, Hkv=8, dtype="bf16", lo=2048, hi=32768, topk=64),
        # the selected pages of four requests of 128 k tokens
        dict(attend, name="sparse_long", op="sparse", B=4, Hq=64, Hkv=8, dtype="bf16", lo=131072, hi=131072, topk=256),
        # a few tokens of each request (a draft to verify) over long caches
        dict(attend, name="prefill_few", op="prefill", B=4, Hq=32, Hkv=8, dtype="bf16", lo=8000, hi=30001, nlo=3, nhi=8),
        # one long prompt
        dict(attend, name="prefill_prompt", op="prefill", B=1, Hq=32, Hkv=8, dtype="bf16", lo=0, hi=0, nlo=16384, nhi=16384),
        # a window of a few requests' tokens, in a token-level cache (pages of one token)
        dict(attend, name="read_window", op="read", B=7, Hkv=2, ps=1, dtype="fp16", lo=1, hi=1000, nlo=1, nhi=333),
        # four prefixes of 8192 tokens for a computation in 16 bits
        dict(attend, name="read_prefix", op="read", B=4, Hkv=8, dtype="bf16", lo=0, hi=0, nlo=8192, nhi=8192),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    c = dict(op=rng.choice(["append", "decode", "sparse", "prefill", "read"]), D=rng.choice([64, 128, 128]),
             ps=rng.choice([1, 2, 8, 16, 16, 32, 64, 128]), dtype=rng.choice(["bf16", "fp16"]), Hkv=rng.choice([1, 2, 4, 8]))
    if c["op"] != "read":
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if c["op"] == "append":
        c.update(B=_log(rng, 1, 32), axes=rng.choice([1, 1, 3, 4]), norm=rng.random() < 0.5, interleaved=rng.random() < 0.4,
                 rot=rng.choice([c["D"], c["D"], c["D"] // 2]))
        c["hi"] = _log(rng, 1, 4096) - 1
        c["nhi"] = 1 if rng.random() < 0.3 else _log(rng, 1, max(1, min(8192, 150_000_000 // (c["B"] * c["Hq"] * c["D"]))))
    elif c["op"] in ("decode", "sparse"):
        c["B"] = _log(rng, 1, 64)
        c["hi"] = _log(rng, 1, min(131072, 268_435_456 // (c["B"] * c["Hkv"] * c["D"])))
        c["lo"] = rng.randint(0, c["hi"])
        if c["op"] == "sparse":
            c["topk"] = _log(rng, 1, max(1, min(4096, c["hi"]) // c["ps"]))
    elif c["op"] == "prefill":
        c["B"] = _log(rng, 1, 8)
        c["hi"] = _log(rng, 1, 32768) - 1
        c["nhi"] = _log(rng, 1, min(8192, max(8, 2_000_000_000 // (c["B"] * c["Hq"] * (c["hi"] + 8192)))))
    else:
        c["B"] = _log(rng, 1, 32)
        c["hi"] = _log(rng, 1, 8192) - 1
        c["nhi"] = _log(rng, 1, max(1, min(8192, 33_554_432 // (c["B"] * c["Hkv"] * c["D"]))))
    if c["op"] not in ("decode", "sparse"):
        c["lo"], c["nlo"] = rng.randint(0, c["hi"]), rng.randint(1, c["nhi"])
    if c["op"] not in ("append", "read"):
        c["window"] = c["sink"] = 0
    if c["op"] in ("decode", "prefill") and rng.random() < 0.4:
        c["window"], c["sink"] = _log(rng, 1, 4096), rng.randint(0, 16)
    return c


def _spread(lo, hi, n, turn):
    """n whole numbers in [lo, hi], the last of them hi."""
    v = [lo + int((hi - lo + 1) * ((i + 1) * turn % 1.0)) for i in range(n)]
    return v[:-1] + [hi]


def _lengths(c):
    """(tokens cached before, new tokens) of each request; for a read, the first position and the tokens read."""
    old = _spread(c["lo"], c["hi"], c["B"], 0.6180339887)
    return old, [0] * c["B"] if c["op"] in ("decode", "sparse") else _spread(c["nlo"], c["nhi"], c["B"], 0.7548776662)


def _sections(c):
    """Pairs of dimensions that each axis of the positions turns."""
    half, n = c["rot"] // 2, c["axes"]
    rest = half * 3 // (4 * (n - 1)) if n > 1 else 0
    return [half - rest * (n - 1)] + [rest] * (n - 1)


def _visible(c):
    """Pairs of (new token, visible token), and the tokens of the cache that some new one sees, over all requests."""
    pairs = seen = 0
    for o, n in zip(*_lengths(c)):
        if c["op"] == "sparse":  # the tail page and full ones
            here = min(o, (min(c["topk"], -(-o // c["ps"])) - 1) * c["ps"] + (o - 1) % c["ps"] + 1)
            pairs, seen = pairs + here, seen + here
            continue
        o, n = (o - 1, 1) if c["op"] == "decode" else (o, n)
        w, s = c["window"] or o + n, c["sink"]
        i = range(o, o + n)
        pairs += sum(min(p + 1, w) + max(0, min(s, p + 1 - w)) for p in i if p >= 0)
        seen += min(o + n, w + n - 1) + max(0, min(s, o + n - (w + n - 1)))
    return pairs, seen


def work(c):
    D = c["D"]
    old, new = _lengths(c)
    T, ps = sum(new), c["ps"]
    if c["op"] == "append":
        pages = sum((o + n - 1) // ps - o // ps + 1 for o, n in zip(old, new))
        before = sum(o % ps for o in old)
        rows16 = T * (2 * c["Hq"] + 2 * c["Hkv"]) + 3 * pages * c["Hkv"]
        rows8 = (2 * T + before) * c["Hkv"]
        return {"bytes": rows16 * D * 2 + rows8 * (D + 1) + T * c["rot"] * 4, "flops": T * (c["Hq"] + c["Hkv"]) * D * (7 if c["norm"] else 3)}
    if c["op"] == "read":
        return {"bytes": 2 * T * c["Hkv"] * (D + 1 + 2 * D), "flops": 2 * T * c["Hkv"] * D}
    pairs, seen = _visible(c)
    T = c["B"] if c["op"] != "prefill" else T
    return {"bytes": 2 * seen * c["Hkv"] * (D + 1) + 4 * T * c["Hq"] * (D + 1), "flops": 4 * pairs * c["Hq"] * D}


# -------------------------------------------------------------------------------------------- the 8-bit rows
def _power(k):
    """2 ** k in float32, k whole numbers of a normal exponent."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """Rows of float32 as e4m3 codes (bytes) and their scale 2 ** (byte - 127): the least power of two that brings the
    row's largest finite magnitude to 448 at most, its exponent kept in [-64, 63]; what is not finite becomes NaN."""
    finite = x.isfinite()
    part, e = torch.frexp(x.abs().masked_fill(~finite, 0).amax(-1))
    k = torch.where(part > 0, e - 9 + (part > 0.875), -64).clamp(-64, 63)
    code = (x * _power(-k)[..., None]).clamp(-448, 448).masked_fill(~finite, math.nan).to(E4M3)
    return code.view(torch.uint8), (k + 127).to(torch.uint8)


def _values(code, scale):
    """What codes and scales (bytes) stand for, in float32."""
    return code.view(E4M3).float() * _power(scale.to(torch.int32) - 127)[..., None]


# -------------------------------------------------------------------------------------------------- inputs
def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, B, Hkv, D, ps = DT[c["dtype"]], c["B"], c["Hkv"], c["D"], c["ps"]
    Hq = c.get("Hq", 0)
    normal = lambda *shape: torch.randn(shape, dtype=torch.float32, device="cuda", generator=gen)  # noqa: E731
    old, new = _lengths(c)
    total = [o + n for o, n in zip(old, new)]
    stride = max(1, max(-(-t // ps) for t in total))
    blocks = B * stride + 3
    # pages anywhere in the pool; keys with a direction that a head's tokens share, as projections give them
    table = torch.randperm(blocks, device="cuda", generator=gen)[: B * stride].to(torch.int32).view(B, stride)
    code = [torch.empty((blocks, Hkv, ps, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = torch.empty((blocks, Hkv, 2, ps), dtype=torch.uint8, device="cuda")
    shared = 0.5 * normal(1, Hkv, 1, D), 0.25 * normal(1, Hkv, 1, D)
    some = max(1, (1 << 26) // (Hkv * ps * D))
    for b in range(0, blocks, some):
        for x in range(2):
            rows = normal(*code[x][b:b + some].shape) + shared[x]
            code[x][b:b + some], scale[b:b + some, :, x] = _quantise(rows)
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + [sum(new[: i + 1]) for i in range(B)], dtype=torch.int32, device="cuda")
    T = sum(new) if c["op"] not in ("decode", "sparse") else B
    s = dict(case=c, k=code[0].view(E4M3), v=code[1].view(E4M3), scale=scale, table=table, lens=lens, cu=cu,
             most_new=max(new), longest=max(total))
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
    elif c["op"] == "read":
        s["first"] = torch.tensor(old, dtype=torch.int32, device="cuda")
        s["out"] = [torch.empty((T, Hkv, D), dtype=dt, device="cuda") for _ in range(2)]
    else:
        s["q"] = (1.5 * normal(T, Hq, D)).to(dt)
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((T, Hq), dtype=torch.float32, device="cuda")
    if c["op"] == "sparse":
        # the tail page and the best of the others by a random score, ascending
        n = torch.tensor([-(-t // ps) for t in total], device="cuda")[:, None, None]
        page = torch.arange(stride, device="cuda")
        score = normal(B, Hkv, stride).masked_fill(page == n - 1, math.inf).masked_fill(page >= n, -math.inf)
        rank = score.sort(-1, descending=True).indices[..., : c["topk"]]
        count = n.clamp(max=c["topk"]).expand(B, Hkv, 1)
        place = torch.arange(rank.shape[-1], device="cuda")
        rank = rank.masked_fill(place >= count, 1 << 30).sort(-1).values
        s["sel"] = torch.zeros((B, Hkv, c["topk"]), dtype=torch.int32, device="cuda")
        s["sel"][..., : rank.shape[-1]] = rank.masked_fill(place >= count, 0).to(torch.int32)
        s["cnt"] = count[..., 0].to(torch.int32).contiguous()
    if own:  # the handles on these buffers that a program keeps for a layer, and its workspace
        import sparse_paged_kv_page_gb300 as S
        s["cache"], s["batch"] = S.make_cache8(s["k"], s["v"], scale, s.get("meta"), dtype=dt), S.make_batch(table, lens)
        if c["op"] == "append":
            s["rotation"] = S.make_rope(s["rope"], interleaved=c["interleaved"], sections=_sections(c), eps=1e-6,
                                        positions=s["positions"] if c["axes"] > 1 else None,
                                        q_weight=s["weights"][0], k_weight=s["weights"][1])
        elif c["op"] == "prefill":
            s["workspace"] = S.alloc_paged_prefill8_workspace(B, Hkv, Hq, D, T)
        elif c["op"] != "read":
            s["workspace"] = S.alloc_paged_decode8_workspace(B, Hkv, Hq, D)
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _rotate(x, weight, angles, c):
    """Norm over each head (if it has weights), then the rotation of its first `rot` dimensions, in 32 bits."""
    y, rot = x.float(), c["rot"]
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    cos, sin = angles[:, None, : rot // 2], angles[:, None, rot // 2:]
    turn = y[..., :rot]
    a, b = (turn[..., 0::2], turn[..., 1::2]) if c["interleaved"] else (turn[..., : rot // 2], turn[..., rot // 2:])
    parts = a * cos - b * sin, a * sin + b * cos
    turn = torch.stack(parts, -1).flatten(-2) if c["interleaved"] else torch.cat(parts, -1)
    return torch.cat([turn, y[..., rot:]], -1)


def _append_plain(s):
    c, ps = s["case"], s["case"]["ps"]
    dt = s["q"].dtype
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
    k8, v8 = s["k"].view(torch.uint8), s["v"].view(torch.uint8)
    k8[block, :, slot], s["scale"][block, :, 0, slot] = _quantise(k)
    v8[block, :, slot], s["scale"][block, :, 1, slot] = _quantise(s["v_new"].float())
    # statistics of the pages written: the first and every token that opens a page stands for its page
    head = (slot == 0) | (token == s["cu"].long()[b])
    page, pb, blk = place[head] // ps, b[head], block[head]
    fill = (s["lens"].long()[pb] - page * ps).clamp(max=ps)
    keys = _values(k8[blk], s["scale"][blk, :, 0]).to(dt).float()               # [pages, Hkv, ps, D], as they are read
    there = (torch.arange(ps, device=q.device) < fill[:, None])[:, None, :, None]
    s["meta"][blk, :, 0] = keys.masked_fill(~there, math.inf).amin(2).to(dt)
    s["meta"][blk, :, 1] = keys.masked_fill(~there, -math.inf).amax(2).to(dt)
    total = keys.double().masked_fill(~there, 0).sum(2)                         # the mean lies next to rounding borders
    s["meta"][blk, :, 2] = (total / fill[:, None, None]).to(dt)
    return [q.to(dt), s["k"], s["v"], s["scale"].view(E8M0), s["meta"]]


def _weighted(z, hidden, v):
    """Softmax over the last axis of z where it is not hidden, times v [.., L, D]: the sums and their log-sum-exp."""
    z.masked_fill_(hidden, -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-1e30)
    z.sub_(top).exp_()
    norm = z.sum(-1, keepdim=True)
    lse = (top + norm.log()).squeeze(-1)
    return torch.matmul(z.flatten(2, -2), v).view(*z.shape[:-1], v.shape[-1]) / norm.clamp(min=1e-30), lse


def _attend_plain(s):
    c = s["case"]
    B, Hkv, G, D, dt = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"], s["q"].dtype
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
    k, v = (_values(x.view(torch.uint8)[pages], s["scale"][pages, :, i]).transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L]
            for i, x in enumerate((s["k"], s["v"])))
    z = torch.matmul(q, k.transpose(-1, -2)).mul_(D ** -0.5).view(B, Hkv, G, -1, L)
    j, i = torch.arange(L, device="cuda"), place[..., None]
    seen = (j <= i) & (i < s["lens"].long()[:, None, None])
    if c["window"]:
        seen &= (j > i - c["window"]) | (j < c["sink"])
    out, lse = _weighted(z, ~seen[:, None, None], v)
    out, lse = out.permute(0, 3, 1, 2, 4).flatten(2, 3), lse.permute(0, 3, 1, 2).flatten(2, 3)
    if rows is None:
        return [out[:, 0].to(dt), lse[:, 0].contiguous()]
    return [out[rows >= 0].to(dt), lse[rows >= 0]]


def _sparse_plain(s):
    c = s["case"]
    B, Hkv, G, D, ps = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"], c["ps"]
    sel = s["sel"].long()
    block = s["table"].long()[torch.arange(B, device="cuda")[:, None, None], sel]               # [B, Hkv, topk]
    head = torch.arange(Hkv, device="cuda")[:, None]
    k, v = (_values(x.view(torch.uint8)[block, head], s["scale"][block, head, i]).flatten(2, 3) for i, x in enumerate((s["k"], s["v"])))
    place = sel[..., None] * ps + torch.arange(ps, device="cuda")
    seen = (place < s["lens"].long()[:, None, None, None]) & (torch.arange(c["topk"], device="cuda") < s["cnt"][..., None])[..., None]
    z = torch.matmul(s["q"].float().view(B, Hkv, G, D), k.transpose(-1, -2)).mul_(D ** -0.5)
    out, lse = _weighted(z, ~seen.flatten(2)[:, :, None], v)
    return [out.flatten(1, 2).to(s["q"].dtype), lse.flatten(1, 2)]


def _read_plain(s):
    c, ps = s["case"], s["case"]["ps"]
    token = torch.arange(s["out"][0].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), token, right=True)
    place = s["first"].long()[b] + token - s["cu"].long()[b]
    block, slot = s["table"][b, place // ps].long(), place % ps
    return [_values(x.view(torch.uint8)[block, :, slot], s["scale"][block, :, i, slot]).to(DT[c["dtype"]]) for i, x in enumerate((s["k"], s["v"]))]


def run(s):
    c = s["case"]
    if not own:
        return {"append": _append_plain, "sparse": _sparse_plain, "read": _read_plain}.get(c["op"], _attend_plain)(s)
    import sparse_paged_kv_page_gb300 as S
    if c["op"] == "append":
        # the batch's lengths were advanced once for all layers; this layer writes its tokens
        S.sa_append_kv8(s["cache"], s["batch"], s["rotation"], s["q"], s["k_new"], s["v_new"], s["cu"], s["most_new"],
                        s["q_out"], advanced=True)
        return [s["q_out"], s["k"], s["v"], s["scale"].view(E8M0), s["meta"]]
    if c["op"] == "read":
        S.sa_read_kv8(s["cache"], s["batch"], s["cu"], s["first"], s["out"][0], s["out"][1])
        return s["out"]
    if c["op"] == "decode":
        S.sa_paged_decode8(s["cache"], s["batch"], s["q"], c["Hq"], 0.0, s["out"], window=c["window"], n_sink=c["sink"],
                           lse=s["lse"], workspace=s["workspace"])
    elif c["op"] == "sparse":
        S.sa_sparse_decode8(s["cache"], s["batch"], s["q"], c["Hq"], s["sel"], s["cnt"], c["topk"], 0.0, s["out"],
                            lse=s["lse"], workspace=s["workspace"])
    else:
        S.sa_paged_prefill8(s["cache"], s["batch"], s["q"], c["Hq"], s["cu"], 0.0, s["out"], window=c["window"],
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


def _rounded8(x):
    """Rows of float64: the values of their e4m3 codes, on the format's grid, and their scales."""
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -60) / 448.0)).clamp(-64, 63))
    scale = torch.where(top <= 224 * scale, (scale / 2).clamp(min=2.0 ** -64), scale)           # a logarithm just above a whole number
    y = x / scale
    quantum = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)             # 3 stored bits; fixed below 2 ** -6
    return (torch.round(y / quantum) * quantum).clamp(-448, 448), scale[..., 0]


def _held(code, scale):
    return code.double() * torch.exp2(scale.double() - 127)[..., None]


def exact(c, seed):
    s = prepare(c, seed)
    old, new = _lengths(c)
    ps, D, Hkv = c["ps"], c["D"], c["Hkv"]
    table = s["table"].cpu().tolist()
    if c["op"] == "append":
        place = torch.cat([s["positions"][a:a + 1].t().expand(-1, w) for a, w in enumerate(_sections(c))], 1)
        q, k = _turned(s["q"], s["weights"][0], place, c), _turned(s["k_new"], s["weights"][1], place, c)
        new_rows = [_rounded8(k), _rounded8(s["v_new"].double())]
        pools, meta = [s["k"].double(), s["v"].double()], s["meta"].double()
        scales = torch.exp2(s["scale"].double() - 127)
        row = 0
        for b in range(c["B"]):
            p0, p1 = old[b] // ps, (old[b] + new[b] - 1) // ps
            blocks = torch.tensor(table[b][p0:p1 + 1], device="cuda")
            at, end = old[b] - p0 * ps, old[b] - p0 * ps + new[b]
            for x, (code, scale) in enumerate(new_rows):
                rows = pools[x][blocks].transpose(1, 2).reshape(-1, Hkv, D)
                rows[at:end] = code[row:row + new[b]]
                pools[x][blocks] = rows.view(-1, ps, Hkv, D).transpose(1, 2)
                flat = scales[blocks][:, :, x].transpose(1, 2).reshape(-1, Hkv)
                flat[at:end] = scale[row:row + new[b]]
                scales[blocks, :, x] = flat.view(-1, ps, Hkv).transpose(1, 2)
            row += new[b]
            paged = pools[0][blocks] * scales[blocks][:, :, 0, :, None]
            whole = end // ps
            if whole:
                meta[blocks[:whole]] = torch.stack([paged[:whole].amin(2), paged[:whole].amax(2), paged[:whole].mean(2)], 2)
            if end % ps:
                part = paged[-1][:, : end % ps]
                meta[blocks[-1]] = torch.stack([part.amin(1), part.amax(1), part.mean(1)], 1)
        return [q, *pools, scales, meta]
    if c["op"] == "read":
        outs = [[], []]
        for b in range(c["B"]):
            p0, p1 = old[b] // ps, (old[b] + new[b] - 1) // ps
            blocks = torch.tensor(table[b][p0:p1 + 1], device="cuda")
            for x, pool in enumerate((s["k"], s["v"])):
                rows = _held(pool.view(torch.uint8)[blocks].view(E4M3), s["scale"][blocks][:, :, x]).transpose(1, 2).reshape(-1, Hkv, D)
                outs[x].append(rows[old[b] - p0 * ps:][: new[b]])
        return [torch.cat(x) for x in outs]
    G = c["Hq"] // Hkv
    if work(c)["flops"] > 6e12:
        return None
    outs, lses, row = [], [], 0
    for b in range(c["B"]):
        n = new[b] if c["op"] == "prefill" else 1
        L = old[b] + new[b]
        q = s["q"][row:row + n].double()
        row += n
        outs.append(torch.zeros((n, c["Hq"], D), dtype=torch.float64, device="cuda"))
        lses.append(torch.full((n, c["Hq"]), -math.inf, dtype=torch.float64, device="cuda"))
        blocks = torch.tensor(table[b][: -(-L // ps)], device="cuda", dtype=torch.int64)
        for h in range(Hkv if L else 0):
            k, v = (_held(x.view(torch.uint8)[blocks, h].view(E4M3), s["scale"][blocks, h, i]).flatten(0, 1)[:L] for i, x in enumerate((s["k"], s["v"])))
            if c["op"] == "sparse":
                pages = s["sel"][b, h, : int(s["cnt"][b, h])].long()
                at = (pages[:, None] * ps + torch.arange(ps, device="cuda")).flatten()
                at = at[at < L]
                z = q[0, h * G:(h + 1) * G] @ k[at].t() / math.sqrt(D)
                lses[-1][0, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                outs[-1][0, h * G:(h + 1) * G] = torch.softmax(z, -1) @ v[at]
                continue
            for t in range(0, n, 256):
                i = torch.arange(L - n + t, L - n + min(n, t + 256), device="cuda")[:, None]
                far = int(i[-1]) + 1
                j = torch.arange(far, device="cuda")
                hidden = j > i
                if c["window"]:
                    hidden = hidden | ((i - j >= c["window"]) & (j >= c["sink"]))
                for g in range(h * G, (h + 1) * G):
                    z = (q[t:t + 256, g] @ k[:far].t() / math.sqrt(D)).masked_fill(hidden, -math.inf)
                    lses[-1][t:t + 256, g] = torch.logsumexp(z, -1)
                    outs[-1][t:t + 256, g] = torch.softmax(z, -1) @ v[:far]
    return [torch.cat(outs), torch.cat(lses)]
