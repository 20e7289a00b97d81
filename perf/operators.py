"""Cases of the paged 4-bit cache operators: what they compute in plain torch, and the calls that
a serving program makes of the library.

The cache is a pool of pages.  A page holds `page` tokens of every key/value head; inside a
(page, head) the tokens lie in groups of 16, keys before values, each half being 16 rows of
packed 4-bit codes (E2M1, two channels a byte, the even one low) and then 16 rows of scales
(E4M3, one for 16 channels).  A value is code * scale.
"""
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the page plan of one decode step: eight requests, a token each
        dict(name="plan_decode_8", op="plan", B=8, page=16, T=8192, n=1),
        # a scheduler's step over a full server: thousands of requests, prompts among them
        dict(name="plan_mixed_4096", op="plan", B=4096, page=32, T=4096, n=48),
        # positions of one decode step, grouped heads
        dict(name="rope_decode_8", op="rope", dtype="bf16", n=8, Hq=32, Hkv=8, D=128, rot=128, axes=1,
             adjacent=False, inverse=False),
        # a video prompt: time, height and width positions
        dict(name="rope_video_32k", op="rope", dtype="bf16", n=32768, Hq=32, Hkv=8, D=128, rot=128, axes=3,
             adjacent=False, inverse=False),
        # one decode step's keys and values into the cache, and those tokens read back
        dict(name="append_decode_8", op="append", dtype="bf16", n=8, Hkv=8, D=128, page=16),
        # a long prompt, every query head with a key/value head of its own
        dict(name="append_prompt_32k", op="append", dtype="fp16", n=32768, Hkv=32, D=128, page=64),
        # a short conversation, one request: latency counts
        dict(name="decode_1x1000", op="attention", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, page=16, T=1000, nq=1, window=0),
        # a ragged batch of ordinary contexts, one query head per key/value head
        dict(name="decode_8x8k", op="attention", dtype="fp16", B=8, Hq=32, Hkv=32, D=128, page=16, T=8192, nq=1, window=0),
        # four long contexts, grouped heads: what a token costs at 128 K
        dict(name="decode_4x128k", op="attention", dtype="bf16", B=4, Hq=32, Hkv=8, D=128, page=64, T=131072, nq=1, window=0),
        # a draft of four tokens checked for each of eight requests
        dict(name="verify_8x8k", op="attention", dtype="bf16", B=8, Hq=32, Hkv=8, D=128, page=32, T=8192, nq=4, window=0),
        # ragged prompts' first chunks, odd sizes
        dict(name="chunk_3x777", op="attention", dtype="fp16", B=3, Hq=32, Hkv=8, D=128, page=16, T=777, nq=333, window=0),
        # a chunk of a long prompt against what is cached of it
        dict(name="chunk_2048_of_32k", op="attention", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, page=64, T=32768, nq=2048, window=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["plan", "rope", "append", "attention", "attention", "attention"])
    if op == "plan":
        return dict(op=op, B=_log(rng, 1, 4096), page=rng.choice([16, 32, 64, 128]), T=_log(rng, 1, 8192), n=_log(rng, 1, 48))
    if op == "rope":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 8, 32])
        return dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), n=_log(rng, 1, 12000), Hq=Hkv * rng.choice([1, 4] if Hkv < 32 else [1]),
                    Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2]), axes=rng.choice([1, 2, 3]), adjacent=rng.random() < 0.4, inverse=rng.random() < 0.4)
    if op == "append":
        return dict(op=op, dtype=rng.choice(["bf16", "fp16"]), n=_log(rng, 1, 32000), Hkv=rng.choice([1, 3, 8, 32]), D=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128]))
    form = rng.choice(["decode", "verify", "chunk"])
    Hkv, G = rng.choice([(1, 8), (2, 7), (4, 3), (8, 4), (8, 1), (32, 1), (1, 16)])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), B=_log(rng, 1, 32), Hq=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128]),
             page=rng.choice([16, 32, 64, 128]), T=_log(rng, 1, 65536), nq=1, window=rng.choice([0, 0, 0, 1000]))
    while c["B"] * c["T"] * Hkv > 1 << 21:
        c["T"] = max(1, c["T"] // 2 - rng.randrange(3))
    if form == "verify":
        c["nq"] = rng.randrange(2, 17)
    if form == "chunk":
        c["nq"] = min(c["T"], _log(rng, 17, 2048))
        while c["B"] * c["nq"] * c["T"] * c["Hq"] > 1 << 30:
            c["B"], c["nq"] = max(1, c["B"] // 2), max(1, c["nq"] // 2 + 1)
            c["T"] = max(c["nq"], c["T"] // 2 + 1)
    return c


def _lens(c):
    """Cached tokens (the new ones among them) and new tokens of each request: ragged, the first the longest."""
    lens = [max(1, c["T"] - (b * 2654435761 % (c["T"] // 2 + 1) if b else 0)) for b in range(c["B"])]
    new = [max(1, min(lens[b], c["nq"] - (b * 40503 % (c["nq"] // 2 + 1) if b else 0))) for b in range(c["B"])]
    return lens, new


def _plan_counts(c):
    r = random.Random(c["B"] * 7919 + c["T"])
    lens = [r.randrange(c["T"] + 1) for _ in range(c["B"])]
    new = [1 if r.random() < 0.5 else r.randrange(2 * c["n"]) for _ in range(c["B"])] if c["n"] > 1 else [1] * c["B"]
    return lens, new


def work(c):
    if c["op"] == "plan":
        lens, new = _plan_counts(c)
        pages = sum(-(-(a + n) // c["page"]) - -(-a // c["page"]) for a, n in zip(lens, new))
        return {"bytes": 4 * (4 * c["B"] + 2 * sum(new) + 2 * pages + 3), "flops": 0}
    if c["op"] == "rope":
        size = 4 if c["dtype"] == "fp32" else 2
        values = c["n"] * (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": 2 * size * values + 4 * c["n"] * c["axes"] + 4 * c["rot"], "flops": 3 * values}
    if c["op"] == "append":
        values = 2 * c["n"] * c["Hkv"] * c["D"]
        return {"bytes": values * (2 + 9 / 16 + 9 / 16 + 2) + 4 * c["n"], "flops": 4 * values}
    lens, new = _lens(c)
    seen = rows = 0
    for a, n in zip(lens, new):
        w = c["window"] or a
        first = max(0, a - n + 1 - w)
        rows += a - first
        seen += sum(min(w, a - n + 1 + i) for i in range(n))
    q = sum(new) * c["Hq"]
    return {"bytes": rows * c["Hkv"] * 2 * c["D"] * 9 / 16 + q * (4 * c["D"] + 4) + 8 * c["B"], "flops": 4.0 * c["D"] * c["Hq"] * seen}


# ------------------------------------------------------------------------------------ the pool
def _encode(x):
    """Codes (uint8, one for each value) and scale bytes of x [..., D], groups of 16 channels."""
    x = x.float().unflatten(-1, (-1, 16))
    scale = (x.abs().amax(-1, keepdim=True) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    s = scale.float()
    y = torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0).abs()
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)).to(torch.uint8)
    return (code + 8 * (x < 0).to(torch.uint8)).flatten(-2), scale.view(torch.uint8).squeeze(-1)


def _parts(pool, D):
    """Views of the codes [pages, Hkv, P/16, 2, 16, D/2] and scales [pages, Hkv, P/16, 2, 16, D/16] of a pool."""
    return pool[..., :8 * D].unflatten(-1, (16, D // 2)), pool[..., 8 * D:].unflatten(-1, (16, D // 16))


def _decode(codes, scales):
    """Values (float32) of packed codes [..., D/2] and their scale bytes [..., D/16]."""
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return (table[c.long()].unflatten(-1, (-1, 16)) * scales.contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _new_pool(pages, Hkv, page, D):
    return torch.zeros((pages, Hkv, page // 16, 2, 9 * D), dtype=torch.uint8, device=DEV)


def _kv(g, shape, dtype):
    """Keys and values as layers give them: keys with a few strong channels, values with a mean."""
    k = torch.randn(shape, generator=g, device=DEV)
    k[..., ::21] *= 5.0
    v = torch.randn(shape, generator=g, device=DEV) + torch.randn(shape[-2:], generator=g, device=DEV) * 0.5
    return k.to(dtype), v.to(dtype)


def _handle(c, pool, num_pages, max_pages):
    import long_context_decode_nuq_b200 as K
    cfg = K.make_paged_cfg(c.get("Hq", c["Hkv"]), c["Hkv"], c["D"], c["page"], num_pages, max_pages, TYPES[c["dtype"]])
    return K.PagedCache(cfg, pool=pool)


def prepare(c, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=DEV)
    s = {"c": c, "op": c["op"]}
    if c["op"] == "plan":
        lens, new = _plan_counts(c)
        want = [-(-(a + n) // c["page"]) for a, n in zip(lens, new)]
        have = torch.tensor([-(-a // c["page"]) for a in lens], device=DEV)
        B, width, total = c["B"], max(max(want), 1), sum(new)
        perm = torch.randperm(sum(want) + 7, generator=g, device=DEV).int()
        taken = int(have.sum())
        table = torch.full((B, width), -1, **i32)
        table[torch.arange(width, device=DEV) < have[:, None]] = perm[:taken]
        free = perm[taken:].contiguous()
        s |= dict(lens=torch.tensor(lens, **i32), new=torch.tensor(new, **i32), table=table, free=free,
                  n_free=torch.tensor([free.numel()], **i32), total=total, page=c["page"],
                  cu=torch.empty(B + 1, **i32), len_out=torch.empty(B, **i32), n_free_out=torch.empty(1, **i32),
                  slots=torch.empty(total, **i32), pos=torch.empty(total, **i32))
        if own:
            import long_context_decode_nuq_b200 as K
            s["cache"] = K.PagedCache(K.make_paged_cfg(1, 1, 64, c["page"], int(perm.numel()), width, torch.bfloat16))
        return s
    if c["op"] == "rope":
        dt, n, half = TYPES[c["dtype"]], c["n"], c["rot"] // 2
        q = torch.randn((n, c["Hq"], c["D"]), generator=g, device=DEV).to(dt)
        k = torch.randn((n, c["Hkv"], c["D"]), generator=g, device=DEV).to(dt)
        pos = torch.randint(0, 1 << 20, (c["axes"], n), generator=g, device=DEV).int()
        axis = [i * c["axes"] // half for i in range(half)]
        freqs = 1e4 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        s |= dict(q=q, k=k, pos=pos, axis=torch.tensor(axis, device=DEV), freqs=freqs, q_out=torch.empty_like(q), k_out=torch.empty_like(k))
        if own:
            import long_context_decode_nuq_b200 as K
            s["cfg"] = K.make_rope_cfg(c["Hq"], c["Hkv"], c["D"], c["rot"], axis, dt, adjacent=c["adjacent"])
        return s
    if c["op"] == "append":
        pages = -(-c["n"] // c["page"]) + 3
        k, v = _kv(g, (c["n"], c["Hkv"], c["D"]), TYPES[c["dtype"]])
        # consecutive tokens of one request, its pages anywhere in the pool, the first page begun already
        at = torch.arange(c["n"], device=DEV) + int(seed) % c["page"]
        slots = torch.randperm(pages, generator=g, device=DEV)[at // c["page"]] * c["page"] + at % c["page"]
        s |= dict(k=k, v=v, slots=slots.int(), pool=_new_pool(pages, c["Hkv"], c["page"], c["D"]), khat=torch.empty_like(k), vhat=torch.empty_like(v))
        if own:
            s["cache"] = _handle(c, s["pool"], pages, pages)
        return s
    lens, new = _lens(c)
    P, D, Hkv, B = c["page"], c["D"], c["Hkv"], c["B"]
    width = -(-c["T"] // P)
    need = [-(-a // P) for a in lens]
    pages = sum(need) + 2
    pool = _new_pool(pages, Hkv, P, D)
    codes, scales = _parts(pool, D)
    step = max(1, (1 << 26) // (Hkv * P * D))
    for lo in range(0, pages, step):
        m = min(step, pages - lo)
        kv = torch.stack(_kv(g, (m, P // 16, 16, Hkv, D), TYPES[c["dtype"]]))  # [2, m, P/16, 16, Hkv, D]
        cd, sc = _encode(kv.permute(1, 4, 2, 0, 3, 5))
        codes[lo:lo + m] = cd[..., 0::2] | cd[..., 1::2] << 4
        scales[lo:lo + m] = sc
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.zeros((B, width), **i32)
    table[torch.arange(width, device=DEV) < torch.tensor(need, device=DEV)[:, None]] = perm[:sum(need)]
    total = sum(new)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn((total, c["Hq"], D), generator=g, device=DEV).to(TYPES[c["dtype"]])
    s |= dict(q=q, pool=pool, table=table, lens=torch.tensor(lens, **i32), cu=torch.tensor(cu, **i32), max_q=max(new),
              scale=D ** -0.5, out=torch.empty_like(q), lse=torch.empty((total, c["Hq"]), device=DEV))
    if own:
        import long_context_decode_nuq_b200 as K
        s["cache"] = _handle(c, pool, pages, width)
        s["ws"] = torch.empty(K.kvq_paged_attention_workspace(s["cache"].cfg, B, total, s["max_q"], c["T"]), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"plan": _plan, "rope": _rope, "append": _append, "attention": _attention}[s["op"]](s)


def _run_own(s):
    import long_context_decode_nuq_b200 as K
    c = s["c"]
    if s["op"] == "plan":
        K.kvq_page_plan(s["cache"], s["lens"], s["new"], s["table"], s["free"], s["n_free"], s["cu"], s["len_out"], s["n_free_out"],
                        s["slots"], s["pos"])
        return s["table"], s["len_out"], s["cu"], s["slots"], s["pos"], s["n_free_out"]
    if s["op"] == "rope":
        K.kvq_rope(s["cfg"], s["q"], s["k"], s["pos"], s["freqs"], s["q_out"], s["k_out"], inverse=c["inverse"])
        return s["q_out"], s["k_out"]
    if s["op"] == "append":
        K.kvq_paged_append(s["cache"], s["k"], s["v"], s["slots"])
        K.kvq_paged_dequantize(s["cache"], s["slots"], s["khat"], s["vhat"])
        return s["khat"], s["vhat"]
    K.kvq_paged_attention(s["cache"], s["q"], s["cu"], s["lens"], s["table"], s["max_q"], c["T"], s["scale"], s["out"], s["ws"],
                          window=c["window"], lse=s["lse"])
    return s["out"], s["lse"]


def _plan(s):
    P, lens, new, table, width = s["page"], s["lens"], s["new"], s["table"], s["table"].shape[1]
    have, want = (lens + P - 1) // P, (lens + new + P - 1) // P
    need = torch.where(want > width, 0, want - have)
    upto = need.cumsum(0)
    ok = (want <= width) & ((need == 0) | (upto <= s["n_free"]))
    j = torch.arange(width, device=DEV) - have[:, None]
    at = (s["n_free"] - 1 - (upto - need)[:, None] - j).clamp(0, s["free"].numel() - 1)
    table = torch.where((j >= 0) & (j < need[:, None]) & ok[:, None], s["free"][at], table)
    cu = torch.cat((torch.zeros_like(new[:1]), new.cumsum(0).int()))
    i = torch.arange(s["total"], device=DEV)
    b = torch.searchsorted(cu, i.int(), right=True) - 1
    pos = lens[b] + i.int() - cu[b]
    slots = torch.where(ok[b], table[b, (pos // P).clamp(max=width - 1)] * P + pos % P, -1)
    return table, torch.where(ok, lens + new, lens), cu, slots.int(), pos, (s["n_free"] - (need * ok).sum()).int()


def _rope(s):
    c = s["c"]
    angle = s["pos"][s["axis"]].double().T * s["freqs"]  # far positions: 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c["inverse"]:
        sin = -sin

    def turn(x):
        a, rest = x[..., :c["rot"]].float(), x[..., c["rot"]:]
        u, v = (a[..., 0::2], a[..., 1::2]) if c["adjacent"] else a.chunk(2, -1)
        u, v = u * cos - v * sin, v * cos + u * sin
        y = torch.stack((u, v), -1).flatten(-2) if c["adjacent"] else torch.cat((u, v), -1)
        return torch.cat((y.to(x.dtype), rest), -1)

    return turn(s["q"]), turn(s["k"])


def _append(s):
    c = s["c"]
    codes, scales = _parts(s["pool"], c["D"])
    cd, sc = _encode(torch.stack((s["k"], s["v"]), 1))  # [n, 2, Hkv, ...]
    slot = s["slots"].long()[:, None, None]
    at = (slot // c["page"], torch.arange(c["Hkv"], device=DEV), slot % c["page"] // 16, torch.arange(2, device=DEV)[:, None], slot % 16)
    codes[at] = cd[..., 0::2] | cd[..., 1::2] << 4
    scales[at] = sc
    back = _decode(codes[at], scales[at]).to(s["k"].dtype)
    return back[:, 0], back[:, 1]


def _attention(s):
    c = s["c"]
    B, Hkv, D, G = c["B"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    codes, scales = _parts(s["pool"][s["table"].long()], D)  # [B, width, Hkv, P/16, 2, 16, ...]
    kv = _decode(codes, scales).permute(4, 0, 2, 1, 3, 5, 6).reshape(2, B, Hkv, -1, D)
    n = s["cu"].diff()
    i = torch.arange(s["max_q"], device=DEV)
    row = (s["cu"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()  # [B, max_q]
    q = s["q"][row].float().reshape(B, -1, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D) * s["scale"]
    last = (s["lens"] - n)[:, None] + i  # each query's own position
    t = torch.arange(kv.shape[3], device=DEV)
    seen = t <= last[..., None]
    if c["window"]:
        seen &= t > last[..., None] - c["window"]
    x = (q @ kv[0].transpose(-1, -2)).unflatten(2, (-1, G))
    x = x.masked_fill(~seen[:, None, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = (x - top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ kv[1]).unflatten(2, (-1, G)) / total
    lse = (top + total.log()).squeeze(-1)
    use = i < n[:, None]
    return o.permute(0, 2, 1, 3, 4)[use].reshape(-1, c["Hq"], D).to(s["q"].dtype), lse.permute(0, 2, 1, 3)[use].reshape(-1, c["Hq"])


# ------------------------------------------------------------------------------------ in 64 bits
def _value64(codes, scales):
    """What the bytes stand for, from the formats' bit fields: E2M1 (bias 1) times E4M3 (bias 7)."""
    e, m = codes >> 1 & 3, (codes & 1).double()
    mag = torch.where(e == 0, m / 2, torch.exp2(e.double() - 1) * (1 + m / 2))
    se, sm = scales >> 3 & 15, (scales & 7).double()
    s = torch.where(se == 0, sm * 2.0 ** -9, torch.exp2(se.double() - 7) * (1 + sm / 8))
    return torch.where(codes >= 8, -mag, mag) * s.repeat_interleave(16, -1)


def exact(c, seed):
    if c["op"] == "plan":
        return None  # whole numbers throughout
    s = prepare(c, seed)
    if c["op"] == "rope":
        angle = torch.stack([s["pos"][a] * f for a, f in zip(s["axis"].tolist(), s["freqs"])], -1).unsqueeze(1)
        turn = torch.polar(torch.ones_like(angle), -angle if c["inverse"] else angle)
        both = []
        for x in (s["q"], s["k"]):
            x, h = x.double(), c["rot"] // 2
            first, second = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["adjacent"] else (slice(0, h), slice(h, c["rot"]))
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            both.append(x)
        return tuple(both)
    if c["op"] == "append":
        levels = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)
        steps = torch.arange(127, device=DEV)
        sizes = torch.where(steps < 8, steps * 2.0 ** -9, (8 + steps % 8) * 2.0 ** (steps // 8 - 10.0)).double()

        def nearest(x, grid):  # ties to the even index
            up = torch.searchsorted(grid, x).clamp(1, grid.numel() - 1)
            lo, hi = x - grid[up - 1], grid[up] - x
            return torch.where((lo < hi) | ((lo == hi) & (up % 2 == 1)), up - 1, up)

        both = []
        for x in (s["k"], s["v"]):
            x = x.double().unflatten(-1, (-1, 16))
            size = sizes[nearest(x.abs().amax(-1, keepdim=True) / 6, sizes)]
            y = levels[nearest(x.abs() / torch.where(size == 0, 1.0, size), levels)] * size
            both.append((y * x.sign()).flatten(-2))
        return tuple(both)
    lens, new = _lens(c)
    if 4.0 * c["D"] * sum(new) * c["Hq"] * c["T"] > 4e12:
        return None
    P, D, G = c["page"], c["D"], c["Hq"] // c["Hkv"]
    out, lse = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV), torch.empty(s["lse"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (a, n) in enumerate(zip(lens, new)):
        pages = s["pool"][s["table"][b, :-(-a // P)].long()]
        for h in range(c["Hkv"]):
            raw = pages[:, h].reshape(-1, 2, 9 * D)
            byte = raw[..., :8 * D].reshape(-1, 2, 16, D // 2)
            nib = torch.empty((*byte.shape[:-1], D), dtype=torch.uint8, device=DEV)
            nib[..., 0::2], nib[..., 1::2] = byte % 16, byte // 16
            kv = _value64(nib, raw[..., 8 * D:].reshape(-1, 2, 16, D // 16)).transpose(0, 1).reshape(2, -1, D)[:, :a]
            where = torch.arange(a - n, a, device=DEV)[:, None]
            t = torch.arange(a, device=DEV)
            hide = (t > where) if not c["window"] else (t > where) | (t <= where - c["window"])
            for hq in range(h * G, h * G + G):
                x = s["q"][at:at + n, hq].double() @ kv[0].T * s["scale"]
                x[hide] = -torch.inf
                lse[at:at + n, hq] = x.logsumexp(-1)
                out[at:at + n, hq] = (x - lse[at:at + n, hq, None]).exp() @ kv[1]
        at += n
    return out, lse
