"""Cases of further decoder-layer operators: rotary positions, the append that
rotates on the way into the paged cache, a cache held in 4 bits with the
attention that reads it, and the norms before and after a block in one pass.

`own` picks the side: False computes each operator from elementary torch
operations in 32 bits, True calls the package.  Shapes follow the 70B-shaped
layer of synthetic/workloads.py (width 8192; a fused QKV row of 10240 values
holds 64 query, 8 key and 8 value heads of 128) and its token counts (decode
batches of 1 to 64, prompts of 2048); the other sizes are generic.

Formats.  A rotation's table is float32 [positions, rot / 2, 2], cosine and
sine.  A cache is [pages, key/value heads, page, dim] in bf16, in e4m3 with one
power-of-two scale per row, or in e2m1 (two values a byte, the even dim low)
with one power-of-two scale per 32 dims of a row.  A group's scale is the
smallest 2^e with max|x| <= 448 * 2^e (e4m3) or 6 * 2^e (e2m1), e kept within
-120..120 (-120 for a group of zeros).  A 4-bit cache is returned as the rows
read back from it.
"""

import math
import random

import torch

own = False

EPS = 1e-5
GROUP = 32             # dims of a row that share a scale in 4 bits
SPREAD = 1.36          # std of a projection of N(0,1) by 8192 weights N(0, 0.015)
MOST_PAIRS = 2.2e9     # query/key/head products of the largest listed case
MOST_TURNED = 1 << 24  # values that a drawn rotation takes


def _case(name, op, **more):
    return dict(name=name, op=op, **more)


def listed():
    layer = dict(heads=64, kv_heads=8, dim=128)
    return [
        # the queries of one decoding request, where latency counts
        _case("rotate_token", "rotate", tokens=1, heads=64, dim=128, rot=128, interleaved=False,
              length=8192, factor=1.0),
        # a long prompt's keys, half of each head turned, positions past 100000
        _case("rotate_prompt_partial", "rotate", tokens=16001, heads=8, dim=128, rot=64,
              interleaved=True, length=131072, factor=8.0),
        # the largest decode batch: queries turned, keys and values into a 4-bit cache
        _case("append_tokens_4bit", "append", tokens=64, page=64, pages=128, bits=4, rot=128,
              interleaved=False, length=16384, factor=1.0, **layer),
        # a prompt's, into an 8-bit cache
        _case("append_prompt_8bit", "append", tokens=2048, page=16, pages=160, bits=8, rot=128,
              interleaved=True, length=8192, factor=1.0, **layer),
        # a request's keys and values moved in without a rotation (another process's, already
        # turned) and read back, an odd number
        _case("cache_rows_4bit", "cache", tokens=333, page=32, pages=16, bits=4, **layer),
        # a long cached prefix
        _case("cache_prefix_4bit", "cache", tokens=16001, page=64, pages=300, bits=4, **layer),
        # one request decoding at 4097 tokens of context
        _case("attend_token_4bit", "attend", seqs=1, new_lo=1, new_hi=1, past_lo=4096,
              past_hi=4096, lens=1, window=0, page=16, bits=4, **layer),
        # the largest decode batch, contexts of very different lengths
        _case("attend_batch_4bit", "attend", seqs=64, new_lo=1, new_hi=1, past_lo=1000,
              past_hi=16000, lens=2, window=0, page=64, bits=4, **layer),
        # a chunk of a long prompt over what is cached of it
        _case("attend_chunk_4bit", "attend", seqs=1, new_lo=509, new_hi=509, past_lo=16384,
              past_hi=16384, lens=5, window=0, page=64, bits=4, **layer),
        # chunks and single tokens in one call, heads of 64, a sliding window
        _case("attend_mixed_window_4bit", "attend", seqs=24, new_lo=1, new_hi=200, past_lo=0,
              past_hi=3000, lens=6, window=1000, page=16, bits=4, heads=32, kv_heads=8, dim=64),
        # one request between two blocks: the first's norm, the residual, the next one's norm
        _case("block_norm_token", "block", rows=1, cols=8192, post=True, gate="none", scale=1.0),
        # a prompt, a gate for each token and value
        _case("block_norm_prompt", "block", rows=2048, cols=8192, post=True, gate="rows",
              scale=0.5),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 2))) - 1)))


def draw(rng):
    op = rng.choice(["rotate", "append", "append", "cache", "attend", "attend", "attend", "block"])
    if op == "block":
        cols = rng.choice([8192, 4096, _log(rng, 64, 16384)])
        return dict(op=op, rows=_log(rng, 1, max(1, (1 << 24) // cols)), cols=cols,
                    post=rng.random() < 0.8, gate=rng.choice(["none", "cols", "rows"]),
                    scale=rng.choice([1.0, 0.25, 0.9]))
    turn = dict(interleaved=rng.random() < 0.5, length=_log(rng, 256, 131072),
                factor=rng.choice([1.0, 4.0, 8.0]))
    if op == "rotate":
        heads = rng.choice([1, 8, 28, 64])
        dim = rng.choice([64, 80, 96, 128, 128, 256, 2 * rng.randint(8, 128)])
        rot = rng.choice([dim, dim, dim // 4 * 2, 2 * rng.randint(1, dim // 2)])
        return dict(op=op, tokens=_log(rng, 1, max(1, MOST_TURNED // (heads * dim))), heads=heads,
                    dim=dim, rot=rot, **turn)
    kv_heads = rng.choice([1, 2, 4, 8, 8])
    dim = rng.choice([64, 128, 128])
    base = dict(heads=kv_heads * rng.choice([1, 2, 4, 7, 8, 8]), kv_heads=kv_heads, dim=dim,
                page=rng.choice([16, 32, 64, 128]), bits=4)
    if op in ("append", "cache"):
        tokens = _log(rng, 1, 2048 if op == "append" else 16000)
        c = dict(op=op, tokens=tokens, pages=tokens * 5 // (4 * base["page"]) + 2, **base)
        if op == "append":
            c.update(turn, bits=rng.choice([4, 4, 8, 16]),
                     rot=rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)]))
        return c
    while True:
        seqs = _log(rng, 1, 64)
        new_hi = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 2, 2048)])
        past_hi = _log(rng, 1, 16000)
        c = dict(op=op, seqs=seqs, new_lo=rng.choice([1, new_hi]), new_hi=new_hi,
                 past_lo=rng.choice([0, past_hi // 16, past_hi]), past_hi=past_hi,
                 lens=rng.randrange(1 << 20), window=rng.choice([0, 0, _log(rng, 1, 4096)]), **base)
        new, kv = _lengths(c)
        # what the plain form spends and holds for the padded batch
        if (seqs * max(new) * max(kv) * c["heads"] <= MOST_PAIRS / 2 and
                seqs * max(kv) * kv_heads * c["dim"] <= 1.0e9):
            return c


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """(new tokens, keys) of each sequence, by the case alone."""
    rng = random.Random(case["lens"])
    new = [_log(rng, case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    past = [_log(rng, case["past_lo"], case["past_hi"]) for _ in range(case["seqs"])]
    return new, [n + p for n, p in zip(new, past)]


def _pages_of(case):
    _, kv = _lengths(case)
    return [-(-n // case["page"]) for n in kv]


def _scale_of(amax, bits):
    """The power-of-two scale of groups whose largest magnitude is amax (float32)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8) if bits == 8 else torch.where(m <= 0.75, e - 3, e - 2)
    e = torch.where(amax > 0, e.clamp(-120, 120), torch.full_like(e, -120))
    return ((e + 127) << 23).view(torch.float32)


def _to_8bit(x):
    """e4m3 values of float32 groups along the last dimension, and their scales."""
    s = _scale_of(x.abs().amax(-1), 8)
    top = 240.0 * 2.0 ** 120
    return (x.clamp(-top, top) / s.unsqueeze(-1)).to(torch.float8_e4m3fn), s


def _to_4bit(x):
    """e2m1 codes of float32 groups along the last dimension, and their scales."""
    s = _scale_of(x.abs().amax(-1), 4)
    t = x.abs() / s.unsqueeze(-1)
    # borders between 0, 0.5, 1, 1.5, 2, 3, 4, 6; a tie goes to the even code
    code = ((t > 0.25).to(torch.uint8) + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) +
            (t >= 3.5) + (t > 5))
    return code | (torch.signbit(x).to(torch.uint8) << 3), s


def _scale_bytes(s):
    return (s.view(torch.int32) >> 23).to(torch.uint8).view(torch.float8_e8m0fnu)


def _pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).view(torch.float4_e2m1fn_x2)


def _rows(g, n, dev):
    return torch.randn(n, generator=g, device=dev).mul_(SPREAD).to(torch.bfloat16)


def _cache(case, g, pages, dev, filled):
    rows = (pages, case["kv_heads"], case["page"])
    out = {}
    for name in ("k", "v"):
        x = torch.randn(rows + (case["dim"],), generator=g, device=dev).mul_(SPREAD) if filled \
            else torch.zeros(rows + (case["dim"],), device=dev)
        if case["bits"] == 16:
            out[name], out[name + "_scale"] = x.to(torch.bfloat16), None
            continue
        x = x.to(torch.bfloat16).float()
        if case["bits"] == 8:
            q, s = _to_8bit(x)
        else:
            q, s = _to_4bit(x.unflatten(3, (-1, GROUP)))
            q = _pack(q.flatten(3))
        out[name], out[name + "_scale"] = q, _scale_bytes(s)
    return out


def _table(case, dev):
    """Cosines and sines of position / factor * 10000^(-2 i / rot)."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=dev)
    p = torch.arange(case["length"], dtype=torch.float64, device=dev) / case["factor"]
    angle = p.unsqueeze(1) * torch.pow(10000.0, i * (-2.0 / case["rot"]))
    return torch.stack([angle.cos().float(), angle.sin().float()], 2)


def _positions(case, g, dev):
    """A prompt's run of positions, or each request's own where the tokens are few."""
    n, most = case["tokens"], case["length"]
    if 64 < n <= most:
        first = int(torch.randint(0, most - n + 1, (1,), generator=g, device=dev))
        return torch.arange(first, first + n, dtype=torch.int32, device=dev)
    return torch.randint(0, most, (n,), generator=g, device=dev).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "block":
        rows, cols = case["rows"], case["cols"]
        s["x"] = torch.randn((rows, cols), generator=g, device=dev).mul_(SPREAD).bfloat16()
        s["residual"] = torch.randn((rows, cols), generator=g, device=dev).mul_(3.0).bfloat16()
        for name, there in (("post", case["post"]), ("weight", True)):
            w = torch.randn(cols, generator=g, device=dev).mul_(0.1).add_(1.0).bfloat16()
            s[name] = w if there else None
        shape = {"none": None, "cols": (cols,), "rows": (rows, cols)}[case["gate"]]
        s["gate"] = torch.rand(shape, generator=g, device=dev).bfloat16() if shape else None
        return s
    if case["op"] == "rotate":
        s["x"] = _rows(g, case["tokens"] * case["heads"] * case["dim"], dev) \
            .view(case["tokens"], case["heads"], case["dim"])
        s["table"], s["positions"] = _table(case, dev), _positions(case, g, dev)
        return s
    width = (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
    if case["op"] in ("append", "cache"):
        slots = case["pages"] * case["page"]
        s.update(_cache(case, g, case["pages"], dev, False))
        s["slots"] = torch.randperm(slots, generator=g, device=dev)[:case["tokens"]].to(torch.int32)
        s["qkv"] = _rows(g, case["tokens"] * width, dev).view(case["tokens"], width)
        if case["op"] == "append":
            s["table"], s["positions"] = _table(case, dev), _positions(case, g, dev)
        return s
    new, kv = _lengths(case)
    need = _pages_of(case)
    s.update(_cache(case, g, sum(need) + 1, dev, True))
    order = torch.randperm(sum(need) + 1, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(len(need), max(need), dtype=torch.int32, device=dev)
    at = torch.tensor([sum(need[:i]) for i in range(len(need))], device=dev).unsqueeze(1)
    col = torch.arange(max(need), device=dev).unsqueeze(0)
    live = col < torch.tensor(need, device=dev).unsqueeze(1)
    s["table"] = torch.where(live, order[(at + col).clamp(max=sum(need))], table)
    s["cu_q"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32,
                             device=dev)
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    s["max_q"], s["max_kv"] = max(new), max(kv)
    s["qkv"] = _rows(g, sum(new) * width, dev).view(sum(new), width)
    return s


def _split(s):
    """The query, key and value heads of the fused projection's rows, as views."""
    c, x = s["case"], s["qkv"]
    q, k, v = x.split([c["heads"] * c["dim"], c["kv_heads"] * c["dim"], c["kv_heads"] * c["dim"]],
                      1)
    return (q.unflatten(1, (c["heads"], c["dim"])), k.unflatten(1, (c["kv_heads"], c["dim"])),
            v.unflatten(1, (c["kv_heads"], c["dim"])))


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import tenant_linear_layers_amd as T
    c = s["case"]
    if c["op"] == "block":
        y, h = T.rms_norm_block(s["x"], s["residual"], s["post"], s["weight"], EPS, s["gate"],
                                c["scale"])
        return {"y": y, "h": h}
    if c["op"] == "rotate":
        return T.rotary(s["x"], s["positions"], s["table"], c["interleaved"])
    q, k, v = _split(s)
    if c["op"] == "attend":
        return T.paged_attention(q, s["k"], s["v"], s["table"], s["cu_q"], s["kv_len"],
                                 s["max_q"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                 window=c["window"])
    cache = [s[n] for n in ("k", "v", "k_scale", "v_scale")]
    out = {}
    if c["op"] == "append":
        out["q"] = T.kv_append(q, k, v, s["positions"], s["table"], s["slots"], *cache,
                               interleaved=c["interleaved"])
    else:
        T.kv_write(k, v, s["slots"], *cache)
    if c["bits"] == 4:
        out["k"], out["v"] = T.kv_read(s["slots"], *cache)
    else:
        out.update(zip(("k", "v", "k_scale", "v_scale"), cache))
    return out


def _run_plain(s):
    c = s["case"]
    return {"block": _block, "rotate": _rotate, "append": _append, "cache": _append,
            "attend": _attend}[c["op"]](s, c)


def _unit(x):
    """Rows over their root mean square."""
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)


def _block(s, c):
    u = s["x"].float()
    if c["post"]:
        u = _unit(u) * s["post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    h = s["residual"].float() + u * c["scale"]
    return {"y": (_unit(h) * s["weight"].float()).bfloat16(), "h": h.bfloat16()}


def _turn(x, s, c):
    """Rows [tokens, heads, dim] turned by their tokens' angles, in float32."""
    x, rot = x.float(), c["rot"]
    cos, sin = s["table"][s["positions"].long()].unsqueeze(1).unbind(3)
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
    return torch.cat([turned, x[..., rot:]], 2)


def _rotate(s, c):
    return _turn(s["x"], s, c).bfloat16()


def _append(s, c):
    q, k, v = _split(s)
    out = {}
    if c["op"] == "append":
        out["q"] = _turn(q, s, c).bfloat16()
        k = _turn(k, s, c)
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]

    def put(name, x):
        if c["bits"] == 16:
            s[name][page, :, at] = x.bfloat16()
            return
        if c["bits"] == 8:
            q8, scale = _to_8bit(x)
        else:
            q8, scale = _to_4bit(x.unflatten(2, (-1, GROUP)))
            q8 = _pack(q8.flatten(2))
        s[name].view(torch.uint8)[page, :, at] = q8.view(torch.uint8)
        s[name + "_scale"].view(torch.uint8)[page, :, at] = _scale_bytes(scale).view(torch.uint8)

    put("k", k.float())
    put("v", v.float())
    if c["bits"] == 4:
        rows = slice(None)
        out.update({n: _rows_4bit(s, n, page, rows, at).bfloat16() for n in ("k", "v")})
    else:
        out.update({n: s[n] for n in ("k", "v", "k_scale", "v_scale")})
    return out


def _rows_4bit(s, name, *index):
    """Cached rows at an index, as the float32 values that they stand for."""
    b = s[name].view(torch.uint8)[index]
    code = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=b.device)
    x = torch.cat([grid, -grid])[code.to(torch.int32)].unflatten(-1, (-1, GROUP))
    e = s[name + "_scale"].view(torch.uint8)[index].to(torch.int32)
    return (x * (e << 23).view(torch.float32).unsqueeze(-1)).flatten(-2)


def _attend(s, c):
    """Every sequence padded to the longest: scores, a masked softmax, the product with v."""
    q, _, _ = _split(s)
    dev = q.device
    b, h, d, g = c["seqs"], c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    n_q = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    i = torch.arange(s["max_q"], device=dev)
    row = s["cu_q"][:-1].long().unsqueeze(1) + i                       # [b, max_q]
    mine = i < n_q.unsqueeze(1)
    qp = q.float()[row.clamp(max=q.shape[0] - 1)]                      # [b, max_q, heads, d]
    qp = qp.unflatten(2, (h, g)).permute(0, 2, 1, 3, 4).reshape(b, h, s["max_q"] * g, d)

    def keys(name):
        x = _rows_4bit(s, name, s["table"].long())                     # [b, p, h, page, d]
        return x.transpose(1, 2).reshape(b, h, -1, d)[:, :, :s["max_kv"]]

    j = torch.arange(s["max_kv"], device=dev)
    at = s["kv_len"].long().unsqueeze(1) - n_q.unsqueeze(1) + i        # a query's position
    sees = (j <= at.unsqueeze(2)) & mine.unsqueeze(2)                  # [b, max_q, max_kv]
    if c["window"]:
        sees &= j > at.unsqueeze(2) - c["window"]
    sees = sees.unsqueeze(1).repeat_interleave(g, 2)                   # a group's queries together
    w = torch.matmul(qp, keys("k").transpose(2, 3).contiguous()).mul_(1.0 / math.sqrt(d))
    w.masked_fill_(~sees, -math.inf)
    w.sub_(w.amax(3, keepdim=True).clamp(min=-1e30)).exp_()
    total = w.sum(3, keepdim=True)
    out = torch.matmul(w, keys("v").contiguous()) / total.clamp(min=1e-30)
    out = out.view(b, h, s["max_q"], g, d).permute(0, 2, 1, 3, 4).reshape(b, s["max_q"], h * g, d)
    # each row of the result takes its place in the padded batch
    r = torch.arange(q.shape[0], device=dev)
    seq = torch.searchsorted(s["cu_q"][1:].long(), r, right=True)
    return out[seq, r - s["cu_q"].long()[seq]].to(torch.bfloat16)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "block":
        n, cols = case["rows"] * case["cols"], case["cols"]
        gate = {"none": 0, "cols": 2 * cols, "rows": 2 * n}[case["gate"]]
        return {"bytes": 8 * n + gate + 2 * cols * (1 + case["post"]), "flops": 10 * n}
    if case["op"] == "rotate":
        n = case["tokens"] * case["heads"]
        # a position that two tokens share is counted for both
        return {"bytes": 4 * n * case["dim"] + case["tokens"] * (4 + 4 * case["rot"]),
                "flops": 3 * n * case["rot"]}
    d = case["dim"]
    row = {16: 2 * d, 8: d + 1, 4: d // 2 + d // GROUP}[case["bits"]]
    if case["op"] in ("append", "cache"):
        n = 2 * case["tokens"] * case["kv_heads"]
        moved = n * (row + 2 * d) + 4 * case["tokens"]
        flops = n * d * (1 if case["bits"] == 16 else 3)
        if case["bits"] == 4:             # and read back
            moved, flops = moved + n * (row + 2 * d) + 4 * case["tokens"], flops + n * d
        if case["op"] == "append":
            turned = case["tokens"] * (case["heads"] + case["kv_heads"])
            moved += 4 * case["tokens"] * (case["heads"] * d + 1 + case["rot"])
            flops += 3 * turned * case["rot"]
        return {"bytes": moved, "flops": flops}
    keys, pairs, new_all = 0, 0, 0
    for n, kv in zip(*_lengths(case)):
        first = max(0, kv - n - case["window"] + 1) if case["window"] else 0
        new_all += n
        keys += kv - first
        if case["window"]:
            pairs += sum(min(p + 1, case["window"]) for p in range(kv - n, kv))
        else:
            pairs += n * (kv - n) + n * (n + 1) // 2
    moved = 2 * keys * case["kv_heads"] * row + 4 * new_all * case["heads"] * d
    return {"bytes": moved + 4 * sum(_pages_of(case)), "flops": 4 * pairs * case["heads"] * d}


# ------------------------------------------------------------------ the definitions in 64 bits
def _two_to(e):
    """2^e in float64 for whole e, by its bits (pow may be a last place off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _grid(x, top, lowest, places):
    """The nearest value of a small floating type (largest `top`, smallest normal 2^lowest,
    `places` bits behind the point) to float64 groups over their scales, by arithmetic alone:
    (values over the scale, exponent of the scale)."""
    a = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(a > 0, a, torch.ones_like(a)) / top))
    e = torch.where(a > top * _two_to(e), e + 1, e)                # log2 rounded down
    e = torch.where((a > 0) & (a <= top / 2 * _two_to(e)), e - 1, e)   # or up
    e = torch.where(a > 0, e, torch.full_like(e, -120)).clamp(-120, 120)
    t = x / _two_to(e)
    # frexp's mantissa is in [1/2, 1): its exponent is one more
    step = _two_to(torch.frexp(t.abs().clamp(min=2.0 ** lowest))[1] - 1 - places)
    return torch.round(t / step) * step, e.squeeze(-1)


def _turn64(x, s, case):
    """The rotation as a product of complex numbers."""
    rot, x = case["rot"], x.double()
    spin = torch.view_as_complex(s["table"].double())[s["positions"].long()].unsqueeze(1)
    out = x.clone()
    first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
    second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
    z = torch.complex(x[..., first], x[..., second]) * spin
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_rows(s, case):
    """What append and cache return."""
    d, hk, page, bits = case["dim"], case["kv_heads"], case["page"], case["bits"]
    n, slots = case["tokens"], s["slots"].long()
    parts = [s["qkv"][:, a * d:b * d].reshape(n, -1, d).double()
             for a, b in ((0, case["heads"]), (case["heads"], case["heads"] + hk),
                          (case["heads"] + hk, case["heads"] + 2 * hk))]
    out = {}
    if case["op"] == "append":
        out["q"] = _turn64(parts[0], s, case)
        parts[1] = _turn64(parts[1], s, case)
    for name, x in zip(("k", "v"), parts[1:]):
        if bits == 4:
            x, e = _grid(x.view(n, hk, -1, GROUP), 6.0, 0, 1)
            out[name] = (x * _two_to(e).unsqueeze(-1)).flatten(2)
            continue
        old = torch.zeros(case["pages"] * page, hk, d, dtype=torch.float64, device=x.device)
        out[name + "_scale"] = None
        if bits == 8:
            x, e = _grid(x, 448.0, -6, 3)
            # a row that was never written keeps the scale that its zeros have
            sc = torch.full((case["pages"] * page, hk), 2.0 ** -120, dtype=torch.float64,
                            device=x.device)
            sc[slots] = _two_to(e)
            out[name + "_scale"] = sc.view(-1, page, hk).permute(0, 2, 1)
        old[slots] = x
        out[name] = old.view(-1, page, hk, d).permute(0, 2, 1, 3)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "block":
        def unit(x, w):
            return x / torch.sqrt((x * x).sum(1, keepdim=True) / case["cols"] + EPS) * w.double()
        u = unit(s["x"].double(), s["post"]) if case["post"] else s["x"].double()
        h = case["scale"] * u * (1.0 if s["gate"] is None else s["gate"].double()) + \
            s["residual"].double()
        return {"y": unit(h, s["weight"]), "h": h}
    if case["op"] == "rotate":
        return _turn64(s["x"], s, case)
    if case["op"] in ("append", "cache"):
        return _exact_rows(s, case)
    d, hk, page = case["dim"], case["kv_heads"], case["page"]
    g = case["heads"] // hk
    parts = []
    start = 0
    table = s["table"].long()
    for b, (n, m) in enumerate(zip(*_lengths(case))):
        slot = torch.arange(m, device=table.device)
        pages, at = table[b][slot // page], slot % page

        def mine(name):
            """A sequence's rows in float64: sign, exponent and half of each code."""
            byte = s[name].view(torch.uint8)[pages, :, at].long()
            code = torch.stack([byte & 15, byte >> 4], 3).flatten(2)
            e, half = code >> 1 & 3, (code & 1).double()
            mag = torch.where(e > 0, (1.0 + half / 2) * _two_to(e - 1), half / 2)
            x = torch.where(code > 7, -mag, mag)
            sc = _two_to(s[name + "_scale"].view(torch.uint8)[pages, :, at].long() - 127)
            return x * sc.repeat_interleave(GROUP, 2)

        k, v = mine("k"), mine("v")
        p = torch.arange(m - n, m, device=table.device).unsqueeze(1)
        hidden = slot > p
        if case["window"]:
            hidden |= slot <= p - case["window"]
        out = torch.empty(n, case["heads"], d, dtype=torch.float64, device=table.device)
        for head in range(case["heads"]):
            qh = s["qkv"][start:start + n, head * d:(head + 1) * d].double()
            z = (qh @ k[:, head // g].t().contiguous()) / math.sqrt(d)
            z = torch.where(hidden, torch.full_like(z, -math.inf), z)
            z = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
            out[:, head] = z @ v[:, head // g].contiguous()
        parts.append(out)
        start += n
    return torch.cat(parts)
