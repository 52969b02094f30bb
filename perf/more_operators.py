"""The operators of a prompt's path beside a paged KV cache, as cases to be timed and checked.

Three operators that a serving loop calls before its decode steps (and the second one in every step):

  prompt  causal attention over whole prompts, grouped heads, packed sequences of different lengths; also new tokens
          behind a context that was there before (their keys and values lie packed together)
  write   RMS norms of queries and keys for each head, the position rotation and the write of keys and values into
          the paged cache (as bf16, E4M3 or NVFP4) in one pass
  read    cached keys and values read back from the pages into packed bf16 rows

`run` computes a case in plain torch operations, or, where `own` is true, through the framework's calls. What an NVFP4
cache was written with is returned as the values that the cache gives back, so that case's pass is a write and a read.
"""
import math
import random

import torch

own = False

P = 16        # tokens per page
EPS = 1e-6    # of the RMS norms


# ---- the cases -------------------------------------------------------------------------------------------------

def listed():
    return [
        # the smallest call: two short chats; latency
        dict(name="prompt_small", op="prompt", B=2, Hq=4, Hkv=2, D=64, dist="uniform", n_lo=37, n_hi=100, ctx_lo=0,
             ctx_hi=0, fused=False, shape=1),
        # a batch of chats of mixed lengths, q, k and v as the projection left them: views of one buffer
        dict(name="prompt_ragged", op="prompt", B=32, Hq=32, Hkv=8, D=128, dist="lognormal", n_lo=1, n_hi=2048, ctx_lo=0,
             ctx_hi=0, fused=True, shape=2),
        # the next 512 tokens of four long documents, six query heads to a kv head
        dict(name="prompt_chunk", op="prompt", B=4, Hq=12, Hkv=2, D=128, dist="uniform", n_lo=512, n_hi=512, ctx_lo=6000,
             ctx_hi=32000, fused=False, shape=3),
        # the largest: one long document, seven query heads to a kv head
        dict(name="prompt_long", op="prompt", B=1, Hq=28, Hkv=4, D=128, dist="uniform", n_lo=16384, n_hi=16384, ctx_lo=0,
             ctx_hi=0, fused=False, shape=4),
        # one decode step's new tokens, padded to the batch size of a captured graph; latency
        dict(name="write_step", op="write", B=61, pad=3, Hq=32, Hkv=8, D=128, dtype="bf16", layout="NHD", style="neox",
             weight="bf16", k_out=False, n_lo=1, n_hi=1, ctx_lo=1, ctx_hi=4000, shape=5),
        # prompts' cache fill, with the keys kept for the prompts' own attention
        dict(name="write_fill", op="write", B=32, pad=0, Hq=32, Hkv=8, D=128, dtype="bf16", layout="NHD", style="neox",
             weight="bf16", k_out=True, n_lo=300, n_hi=2000, ctx_lo=0, ctx_hi=0, shape=6),
        # chunks of prompts into an FP8 cache with a static scale per kv head
        dict(name="write_fp8", op="write", B=16, pad=5, Hq=12, Hkv=2, D=128, dtype="fp8", layout="HND",
             style="interleaved", weight="f32", k_out=True, n_lo=900, n_hi=2048, ctx_lo=0, ctx_hi=8000, shape=7),
        # prompts into an NVFP4 cache, read back as a later request with the same prefix finds them
        dict(name="write_fp4", op="write", B=16, pad=0, Hq=28, Hkv=4, D=128, dtype="nvfp4", layout="HND", style="neox",
             weight="bf16", k_out=True, n_lo=500, n_hi=1500, ctx_lo=0, ctx_hi=100, shape=8),
        # a short prefix of one request; latency
        dict(name="read_small", op="read", B=1, Hkv=2, D=64, dtype="bf16", layout="HND", len_lo=90, len_hi=90, first_hi=0,
             shape=9),
        # a batch of prefixes that a prompt cache holds
        dict(name="read_batch", op="read", B=32, Hkv=8, D=128, dtype="bf16", layout="NHD", len_lo=1, len_hi=8192,
             first_hi=0, shape=10),
        # the same from FP8
        dict(name="read_fp8", op="read", B=32, Hkv=8, D=128, dtype="fp8", layout="HND", len_lo=1, len_hi=8192,
             first_hi=100, shape=11),
        # two long documents in NVFP4
        dict(name="read_fp4", op="read", B=2, Hkv=4, D=128, dtype="nvfp4", layout="HND", len_lo=32000, len_hi=32768,
             first_hi=0, shape=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt"] * 3 + ["write"] * 2 + ["read"])
    shape = rng.randrange(1 << 20)
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128, 128])
    G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    while Hkv * G > 48:
        G = max(1, G // 2)
    if op == "prompt":
        # products of scores within those of the largest listed case
        most = 28 * 16384 * 16384 // 6
        n_hi = _log_int(rng, 1, 8192)
        ctx_hi = rng.choice([0, 0, _log_int(rng, 1, 16384)])
        while Hkv * G * n_hi * (n_hi + ctx_hi) > most:
            n_hi = max(1, n_hi // 2)
        B = _log_int(rng, 1, max(1, min(100, most // (Hkv * G * n_hi * (n_hi + ctx_hi)))))
        return dict(op="prompt", B=B, Hq=Hkv * G, Hkv=Hkv, D=D, dist=rng.choice(["uniform", "lognormal"]),
                    n_lo=rng.randrange(B == 1, n_hi + 1), n_hi=n_hi, ctx_lo=rng.randrange(0, ctx_hi + 1), ctx_hi=ctx_hi,
                    fused=rng.choice([False, True]) and ctx_hi == 0, shape=shape)
    common = dict(Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "fp8", "nvfp4"]), layout=rng.choice(["HND", "NHD"]), shape=shape)
    if op == "write":
        n_hi = rng.choice([1, _log_int(rng, 2, 2048)])
        B = _log_int(rng, 1, max(1, min(256, 36000 // n_hi)))
        return dict(op="write", B=B, pad=rng.choice([0, rng.randrange(1, 9)]), Hq=Hkv * G, style=rng.choice(["neox", "interleaved"]),
                    weight=rng.choice(["bf16", "f32"]), k_out=rng.choice([False, True]), n_lo=rng.randrange(B == 1, n_hi + 1),
                    n_hi=n_hi, ctx_lo=0, ctx_hi=_log_int(rng, 1, 4000), **common)
    len_hi = _log_int(rng, 1, 32768)
    B = _log_int(rng, 1, max(1, min(64, 130000 // len_hi)))
    return dict(op="read", B=B, len_lo=rng.randrange(B == 1, len_hi + 1), len_hi=len_hi,
                first_hi=rng.choice([0, _log_int(rng, 1, 1000)]), **common)


def _lens(c):
    """Per sequence: (rows of this call, positions before them)."""
    r = random.Random(c["shape"])
    if c["op"] == "read":
        return [r.randint(c["len_lo"], c["len_hi"]) for _ in range(c["B"])], [r.randint(0, c["first_hi"]) for _ in range(c["B"])]
    n = []
    for _ in range(c["B"]):
        if c.get("dist") == "lognormal":
            n.append(min(max(int(round(min(1024, c["n_hi"] / 4) * math.exp(r.gauss(0, 1)))), c["n_lo"]), c["n_hi"]))
        else:
            n.append(r.randint(c["n_lo"], c["n_hi"]))
    return n, [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["B"])]


# ---- inputs ------------------------------------------------------------------------------------------------------

def _pages(n):
    return -(-n // P)


def _starts(n, dev):
    return torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device=dev)


def _tables(counts, pool, g, dev):
    """Block tables from a shuffled pool: row b takes the next counts[b] pages of a permutation; -1 elsewhere."""
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    cnt = torch.tensor(counts, device=dev)
    col = torch.arange(max(1, max(counts)), device=dev)
    at = (torch.cumsum(cnt, 0) - cnt)[:, None] + col
    held = col < cnt[:, None]
    return torch.where(held, perm[torch.where(held, at, 0)], -1).to(torch.int32)


def _cache_shape(c, pool, width):
    return (pool, c["Hkv"], P, width) if c["layout"] == "HND" else (pool, P, c["Hkv"], width)


def _cos_sin(n, D, dev):
    f = 10000.0 ** (-torch.arange(0, D, 2, device=dev, dtype=torch.float64) / D)
    a = torch.arange(n, device=dev, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).to(torch.float32)


def prepare(case, seed):
    s = _prepare(case, seed)
    if own:
        # a serving program keeps its buffers, and binds them once
        import paged_kv_gqa_04_gb300 as pkv
        if s["c"]["op"] == "prompt":
            sms = torch.cuda.get_device_properties(s["q"].device).multi_processor_count
            s["workspace"] = torch.empty(pkv.prompt_attention_workspace(s["c"]["D"], sms), dtype=torch.uint8,
                                         device=s["q"].device)
        s["bound"] = {k: pkv.bind(x) for k, x in s.items() if x is None or isinstance(x, torch.Tensor)}
    return s


def _prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"c": c, "err": torch.zeros(1, dtype=torch.int32, device=dev)}
    n, ctx = _lens(c)
    T = sum(n)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)

    if c["op"] == "prompt":
        Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
        L = [a + b for a, b in zip(n, ctx)]
        if c["fused"]:
            s["q"], s["k"], s["v"] = randn(T, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], 1)
        else:
            s["q"], s["k"], s["v"] = randn(T, Hq, D), randn(sum(L), Hkv, D), randn(sum(L), Hkv, D)
        s["q_start"] = _starts(n, dev)
        s["k_start"] = _starts(L, dev) if c["ctx_hi"] else None
        s["scale"] = D ** -0.5
        s["out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros((T, Hq), dtype=torch.float32, device=dev)
        s["n_max"], s["L_max"] = max(n), max(L)
        return s

    # a pool with the pages of all sequences
    Hkv, D = c["Hkv"], c["D"]
    counts = [_pages(a + b) for a, b in zip(n, ctx)]
    pool = max(1, sum(counts))
    s["tables"] = _tables(counts, pool, g, dev)
    s["start"] = _starts(n, dev)
    s["first"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    fp4 = c["dtype"] == "nvfp4"
    width = D // 2 if fp4 else D
    s["k_cache"] = torch.zeros(_cache_shape(c, pool, width), device=dev,
                               dtype={"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "nvfp4": torch.uint8}[c["dtype"]])
    s["v_cache"] = torch.zeros_like(s["k_cache"])
    for x in ("k", "v"):
        s[x + "_bs"] = torch.zeros(_cache_shape(c, pool, D // 16), dtype=torch.float8_e4m3fn, device=dev) if fp4 else None
        # static scales that put a normal value's largest magnitudes near the top of the format
        top = {"bf16": 0.0, "fp8": 5.0 / 448, "nvfp4": 5.0 / (6 * 448)}[c["dtype"]]
        s[x + "_scale"] = None if c["dtype"] == "bf16" else top * (0.5 + torch.rand(Hkv, generator=g, device=dev))
    if c["op"] == "read" or fp4:
        s["k_rows"] = torch.zeros((T, Hkv, D), dtype=torch.bfloat16, device=dev)
        s["v_rows"] = torch.zeros_like(s["k_rows"])
    # where each row of the call lies: what a program's scheduler keeps on the host too
    seq = torch.repeat_interleave(torch.arange(len(n), device=dev), torch.tensor(n, device=dev), output_size=T)
    pos = torch.arange(T, device=dev) - s["start"].long()[seq] + s["first"].long()[seq]
    page = s["tables"].long()[seq, pos // P]
    s["slots"] = (page * P + pos % P).to(torch.int32)
    if c["op"] == "read":
        for x in ("k", "v"):
            if fp4:
                s[x + "_cache"].copy_(torch.randint(0, 256, s[x + "_cache"].shape, generator=g, device=dev, dtype=torch.uint8))
                s[x + "_bs"].copy_(torch.rand(s[x + "_bs"].shape, generator=g, device=dev) * 300 + 20)
            else:
                y = torch.randn(s[x + "_cache"].shape, generator=g, device=dev, dtype=torch.bfloat16)
                s[x + "_cache"].copy_(y if c["dtype"] == "bf16" else (y.float() * 100).clamp(-448, 448))
        return s
    Hq, pad = c["Hq"], c["pad"]
    s["q"], s["k"], s["v"] = randn(T + pad, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], 1)
    # a model's norms: weights around one
    for x in ("q", "k"):
        w = 1 + 0.3 * torch.randn(D, generator=g, device=dev)
        s[x + "_weight"] = w.to(torch.bfloat16) if c["weight"] == "bf16" else w
    s["positions"] = torch.cat([pos, torch.zeros(pad, device=dev)]).to(torch.int32)
    s["slots"] = torch.cat([s["slots"], torch.full((pad,), -1, dtype=torch.int32, device=dev)])
    s["cos_sin"] = _cos_sin(max(a + b for a, b in zip(n, ctx)) + 1, D, dev)
    s["k_out"] = torch.zeros((T + pad, Hkv, D), dtype=torch.bfloat16, device=dev) if c["k_out"] else None
    return s


# ---- one pass ----------------------------------------------------------------------------------------------------

def run(s):
    c = s["c"]
    op = c["op"]
    if own:
        import paged_kv_gqa_04_gb300 as pkv
        t = s["bound"]
        if op == "prompt":
            pkv.prompt_attention(t["q"], t["k"], t["v"], t["q_start"], t["k_start"], s["scale"], t["out"], t["lse"],
                                 t["workspace"], err_flag=t["err"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "write":
            pkv.qk_norm_rope_kv_write(t["q"], t["k"], t["v"], t["q_weight"], t["k_weight"], EPS, t["positions"],
                                      t["cos_sin"], t["k_cache"], t["v_cache"], t["slots"], t["k_scale"], t["v_scale"],
                                      k_block_scale=t["k_bs"], v_block_scale=t["v_bs"], k_out=t["k_out"],
                                      layout=c["layout"], rope_style=c["style"], err_flag=t["err"])
        if op == "read" or c["dtype"] == "nvfp4":
            pkv.gather_kv(t["k_cache"], t["v_cache"], t["tables"], t["start"], t["first"], t["k_rows"], t["v_rows"],
                          t["k_scale"], t["v_scale"], k_block_scale=t["k_bs"], v_block_scale=t["v_bs"],
                          layout=c["layout"], err_flag=t["err"])
        return _outputs(s)
    if op == "prompt":
        return _plain_prompt(s)
    if op == "write":
        _plain_write(s)
    if op == "read" or c["dtype"] == "nvfp4":
        _plain_read(s)
    return _outputs(s)


def _outputs(s):
    if s["c"]["op"] == "read":
        return {"k": s["k_rows"], "v": s["v_rows"]}
    out = {"q": s["q"]}
    if s["k_out"] is not None:
        out["k_out"] = s["k_out"]
    if s["c"]["dtype"] == "nvfp4":
        return {**out, "k": s["k_rows"], "v": s["v_rows"]}
    return {**out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ---- plain forms ---------------------------------------------------------------------------------------------------

def _plain_prompt(s):
    c = s["c"]
    B, Hq, Hkv, D, N, M = c["B"], c["Hq"], c["Hkv"], c["D"], s["n_max"], s["L_max"]
    G, dev = Hq // Hkv, s["q"].device
    qs = s["q_start"].long()
    ks = qs if s["k_start"] is None else s["k_start"].long()
    n, L = qs[1:] - qs[:-1], ks[1:] - ks[:-1]
    out, lse = torch.zeros_like(s["out"]), torch.zeros_like(s["lse"])
    i, j = torch.arange(N, device=dev), torch.arange(M, device=dev)
    row = (qs[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    col = (ks[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    live = i < n[:, None]
    q = s["q"][row].to(torch.float32).reshape(B, N, Hkv, G, D).permute(0, 2, 3, 1, 4)
    k = s["k"][col].to(torch.float32).permute(0, 2, 3, 1)[:, :, None]
    v = s["v"][col].to(torch.float32).permute(0, 2, 1, 3)[:, :, None]
    score = torch.matmul(q, k)
    score.mul_(s["scale"])
    seen = j <= (i[:, None] + (L - n)[:, None, None])
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    m = score.amax(4, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    w = score.sub_(m).exp_()
    z = w.sum(4, keepdim=True)
    o = torch.matmul(w, v) / torch.where(z > 0, z, torch.ones_like(z))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)
    e = (m + torch.log(z))[..., 0].permute(0, 3, 1, 2).reshape(B, N, Hq)
    out[row[live]] = o[live].to(torch.bfloat16)
    lse[row[live]] = e[live]
    return {"out": out, "lse": lse}


def _rotated(x, cs, style):
    D = x.shape[-1]
    c, sn = cs[:, None, :D // 2], cs[:, None, D // 2:]
    if style == "neox":
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * c - b * sn, b * c + a * sn], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)


def _e2m1(z):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 to each magnitude (ties to the even code), with z's sign."""
    a = z.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
    return torch.copysign(torch.round(a / step) * step, z)


def _nvfp4(y, g):
    """Codes and block scales of rows y [..., D] under the static scale g [..., 1, 1]."""
    b = y.reshape(y.shape[:-1] + (-1, 16))
    sc = (b.abs().amax(-1, keepdim=True) / (6 * g)).clamp(max=448.0).to(torch.float32).to(torch.float8_e4m3fn)
    d = g * sc.to(y.dtype)
    e = torch.where(d > 0, _e2m1(b / torch.where(d > 0, d, torch.ones_like(d))), torch.zeros_like(b))
    return e, sc


def _pack(e):
    """E2M1 values [..., D] as bytes of two codes, the even-indexed value in the low half."""
    a = e.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + 8 * torch.signbit(e).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2]


def _plain_write(s):
    c = s["c"]
    live = s["slots"] >= 0
    page, off = (s["slots"].long() // P)[live], (s["slots"].long() % P)[live]
    cs = s["cos_sin"][s["positions"].long()]

    def normed(x, w):
        x = x.to(torch.float32)
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.to(torch.float32)
        return _rotated(x, cs, c["style"])

    k = normed(s["k"], s["k_weight"])
    s["q"].copy_(torch.where(live[:, None, None], normed(s["q"], s["q_weight"]).to(torch.bfloat16), s["q"]))
    if s["k_out"] is not None:
        s["k_out"].copy_(torch.where(live[:, None, None], k.to(torch.bfloat16), s["k_out"]))

    def put(cache, y):
        if c["layout"] == "HND":
            cache[page, :, off] = y
        else:
            cache[page, off] = y

    for name, y in (("k", k[live]), ("v", s["v"][live].to(torch.float32))):
        cache, g = s[name + "_cache"], s[name + "_scale"]
        if c["dtype"] == "bf16":
            put(cache, y.to(torch.bfloat16))
        elif c["dtype"] == "fp8":
            put(cache.view(torch.uint8), (y / g[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            e, sc = _nvfp4(y, g[:, None, None])
            put(cache, _pack(e.flatten(-2)))
            put(s[name + "_bs"].view(torch.uint8), sc[..., 0].view(torch.uint8))


def _plain_read(s):
    c = s["c"]
    slots = s["slots"].long()
    slots = slots[:s["k_rows"].shape[0]]
    page, off = slots // P, slots % P
    for name in ("k", "v"):
        g = s[name + "_scale"]

        def rows(cache):
            x = cache.view(torch.uint8) if cache.element_size() == 1 else cache
            return (x[page, :, off] if c["layout"] == "HND" else x[page, off]).view(cache.dtype)

        y = rows(s[name + "_cache"])
        if c["dtype"] == "fp8":
            y = y.to(torch.float32) * g[:, None]
        elif c["dtype"] == "nvfp4":
            values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=y.device)
            code = torch.stack([y & 15, y >> 4], -1).flatten(-2).long()
            e = values[code & 7] * (1 - 2 * (code >> 3)).to(torch.float32)
            sc = rows(s[name + "_bs"]).to(torch.float32) * g[:, None]
            y = (e.reshape(e.shape[:-1] + (-1, 16)) * sc[..., None]).flatten(-2)
        s[name + "_rows"].copy_(y)


# ---- what a pass cannot do without -----------------------------------------------------------------------------------

def work(c):
    n, ctx = _lens(c)
    T = sum(n)
    if c["op"] == "prompt":
        keys = sum(a + b for a, b in zip(n, ctx) if a)
        pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(n, ctx))
        nbytes = T * c["Hq"] * (4 * c["D"] + 4) + keys * c["Hkv"] * 4 * c["D"] + 8 * c["B"]
        return {"bytes": nbytes + 1, "flops": 4 * pairs * c["Hq"] * c["D"]}
    Hkv, D = c["Hkv"], c["D"]
    row = {"bf16": 2 * D, "fp8": D, "nvfp4": D // 2 + D // 16}[c["dtype"]]
    pages = sum(_pages(a + b) - b // P for a, b in zip(n, ctx) if a)
    read = T * 2 * Hkv * (row + 2 * D) + 4 * pages + 8 * c["B"]
    if c["op"] == "read":
        return {"bytes": read + 1, "flops": 0}
    turns = len({p for a, b in zip(n, ctx) for p in range(b, a + b)})
    nbytes = T * (c["Hq"] * 4 * D + 2 * Hkv * (2 * D + row) + (2 * D * Hkv if c["k_out"] else 0) + 8) + turns * 4 * D
    nbytes += read if c["dtype"] == "nvfp4" else 0
    return {"bytes": nbytes + 1, "flops": 0}


# ---- from the definition, in 64 bits ---------------------------------------------------------------------------------

def exact(case, seed):
    s = _prepare(case, seed)
    return {"prompt": _exact_prompt, "write": _exact_write, "read": _exact_read}[case["op"]](s)


def _exact_prompt(s):
    c = s["c"]
    n, ctx = _lens(c)
    if sum(a * (a + b) for a, b in zip(n, ctx)) * c["Hq"] * c["D"] * 4 > 1e13:
        return None
    G = c["Hq"] // c["Hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=s["q"].device)
    a = e = 0
    for b in range(c["B"]):
        N, L = n[b], n[b] + ctx[b]
        hidden = torch.arange(L, device=out.device) > torch.arange(ctx[b], L, device=out.device)[:, None]
        for h in range(c["Hq"]):
            x = s["q"][a:a + N, h].double() @ s["k"][e:e + L, h // G].double().T * s["scale"]
            x.masked_fill_(hidden, float("-inf"))
            lse[a:a + N, h] = torch.logsumexp(x, 1)
            out[a:a + N, h] = torch.softmax(x, 1) @ s["v"][e:e + L, h // G].double()
        a, e = a + N, e + L
    return {"out": out, "lse": lse}


def _exact_values(y, g, dtype):
    """What a cache that was written with y [T, Hkv, D] stands for (bf16 and E4M3: the value that it holds)."""
    if dtype == "bf16":
        return y
    if dtype == "fp8":
        return (y / g.double()[:, None]).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
    b = y.reshape(y.shape[0], y.shape[1], -1, 16)
    gg = g.double()[:, None, None]
    sc = (b.abs().amax(-1, keepdim=True) / (6 * gg)).clamp(max=448.0).float().to(torch.float8_e4m3fn).double()
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=y.device, dtype=torch.float64)
    z = (b / (gg * sc).clamp(min=1e-300)).clamp(-6, 6)
    lo = torch.bucketize(z.abs(), levels, right=True) - 1
    hi = (lo + 1).clamp(max=7)
    down, up = z.abs() - levels[lo], levels[hi] - z.abs()
    e = levels[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)] * torch.sign(z)
    return (e * (gg * sc)).flatten(-2)


def _exact_write(s):
    c = s["c"]
    n, _ = _lens(c)
    T, D = sum(n), c["D"]
    ang = s["cos_sin"][s["positions"].long()].double()
    turn = torch.complex(ang[:, :D // 2], ang[:, D // 2:])[:, None]

    def head(x, w):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
        x = x.unflatten(-1, (2, D // 2)).transpose(-1, -2) if c["style"] == "neox" else x.unflatten(-1, (D // 2, 2))
        x = torch.view_as_real(torch.view_as_complex(x.contiguous()) * turn)
        return (x.transpose(-1, -2) if c["style"] == "neox" else x).flatten(-2)

    q, k = head(s["q"], s["q_weight"]), head(s["k"], s["k_weight"])
    got = {"q": torch.cat([q[:T], s["q"][T:].double()])}
    if c["k_out"]:
        got["k_out"] = torch.cat([k[:T], torch.zeros_like(k[T:])])
    for name, y in (("k", k[:T]), ("v", s["v"][:T].double())):
        y = _exact_values(y, s[name + "_scale"], c["dtype"])
        if c["dtype"] == "nvfp4":
            got[name] = y
            continue
        cache = torch.zeros(s[name + "_cache"].shape, dtype=torch.float64, device=y.device)
        flat = cache.transpose(1, 2) if c["layout"] == "HND" else cache
        slots = s["slots"][:T].long()
        flat[slots // P, slots % P] = y
        got[name + "_cache"] = cache
    return got


def _exact_read(s):
    c = s["c"]
    n, first = _lens(c)
    got = {}
    for name in ("k", "v"):
        cache = s[name + "_cache"]
        parts = []
        for b in range(c["B"]):
            pages = s["tables"][b, :_pages(first[b] + n[b])].long()
            x = (cache.view(torch.uint8) if cache.element_size() == 1 else cache)[pages].view(cache.dtype)
            if c["dtype"] == "nvfp4":
                x = torch.stack([x % 16, x // 16], -1).flatten(-2)
                mag = torch.where(x % 8 < 4, (x % 8) * 0.5, torch.where(x % 8 < 6, x % 8 - 2.0, (x % 8) * 2.0 - 8)).double()
                x = torch.where(x >= 8, -mag, mag)
                sc = s[name + "_bs"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
                x = x * sc.repeat_interleave(16, -1)
            x = x.double()
            if c["layout"] == "HND":
                x = x.transpose(1, 2)
            x = x.flatten(0, 1)[first[b]:first[b] + n[b]]
            parts.append(x if c["dtype"] == "bf16" else x * s[name + "_scale"].double()[:, None])
        got[name] = torch.cat(parts)
    return got
