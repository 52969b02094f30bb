"""The speculative-decoding operators over a paged KV cache, as cases to be timed and checked.

Four operators that a serving loop calls around the decode step:

  tree    attention of the drafted tokens of every sequence over its paged cache: the context in full, the
          drafted tokens under a tree mask (or as a chain)
  accept  the accepted drafted tokens' cache rows moved together behind the context, in every layer's cache
  fork    sequences forked from others: full pages shared, the partial last page copied in every layer's cache
  resize  block tables grown and trimmed: pages taken from and returned to the pool's reference counts

`run` computes a case in plain torch operations, or, where `own` is true, through the framework's calls.
"""
import math
import random

import torch

own = False

P = 16  # tokens per page


# ---- the cases -------------------------------------------------------------------------------------------------

def listed():
    return [
        # the smallest call: two short chats, a few drafted tokens each; latency
        dict(name="tree_small", op="tree", B=2, Hq=4, Hkv=2, D=64, dtype="bf16", layout="HND", dist="uniform",
             ctx_lo=37, ctx_hi=100, n_lo=5, n_hi=8, mask="tree", shape=1),
        # a batch of medium contexts whose draft model proposes one chain per sequence (no mask tensor)
        dict(name="tree_chain", op="tree", B=32, Hq=12, Hkv=2, D=128, dtype="bf16", layout="HND", dist="uniform",
             ctx_lo=512, ctx_hi=4096, n_lo=4, n_hi=9, mask="chain", shape=2),
        # two long documents, seven query heads to a kv head, a tree of 17 tokens
        dict(name="tree_longctx", op="tree", B=2, Hq=28, Hkv=4, D=128, dtype="bf16", layout="HND", dist="uniform",
             ctx_lo=32700, ctx_hi=32768, n_lo=17, n_hi=17, mask="tree", shape=3),
        # a mixed batch with draft counts that the scheduler sets per sequence, some with a single token
        dict(name="tree_ragged", op="tree", B=64, Hq=32, Hkv=8, D=128, dtype="bf16", layout="NHD", dist="lognormal",
             ctx_lo=1, ctx_hi=8192, n_lo=1, n_hi=31, mask="tree", shape=4),
        # an FP8 cache with a static scale per kv head
        dict(name="tree_fp8", op="tree", B=16, Hq=12, Hkv=2, D=128, dtype="fp8", layout="HND", dist="uniform",
             ctx_lo=2048, ctx_hi=16384, n_lo=24, n_hi=24, mask="tree", shape=5),
        # the largest: wide trees over long contexts, as much arithmetic as memory traffic
        dict(name="tree_wide", op="tree", B=16, Hq=32, Hkv=8, D=128, dtype="bf16", layout="HND", dist="uniform",
             ctx_lo=7001, ctx_hi=8192, n_lo=64, n_hi=64, mask="tree", shape=6),
        # one sequence's acceptance in a 28-layer model: latency
        dict(name="accept_one", op="accept", B=1, layers=28, Hkv=2, D=128, dtype="bf16", layout="HND", ctx_lo=70,
             ctx_hi=90, n_lo=8, n_hi=8, shape=7),
        # a batch's acceptance in a 32-layer model
        dict(name="accept_batch", op="accept", B=64, layers=32, Hkv=8, D=128, dtype="bf16", layout="NHD", ctx_lo=1,
             ctx_hi=150, n_lo=1, n_hi=31, shape=8),
        # sixteen samples from one long prompt in a 28-layer model
        dict(name="fork_samples", op="fork", parents=1, children=16, layers=28, Hkv=2, D=128, dtype="bf16",
             layout="HND", len_lo=5003, len_hi=5003, shape=9),
        # a beam step of a batch: every sequence forked three times, FP8 cache
        dict(name="fork_beams", op="fork", parents=32, children=96, layers=32, Hkv=8, D=128, dtype="fp8",
             layout="NHD", len_lo=1, len_hi=400, shape=10),
        # a batch trimmed to what was accepted and grown again for the next drafts
        dict(name="resize_batch", op="resize", B=256, pages=16384, len_lo=1, len_hi=800, step=33, shape=11),
        # thousands of short sequences in a pool of half a million pages, where half of them come and go
        dict(name="resize_pool", op="resize", B=4096, pages=524288, len_lo=1, len_hi=1600, step=1600, shape=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree"] * 5 + ["accept", "fork", "resize"])
    shape = rng.randrange(1 << 20)
    if op == "tree":
        Hkv = rng.choice([1, 2, 4, 8])
        D = rng.choice([64, 128, 128])
        n_hi = _log_int(rng, 1, 70)
        G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        while n_hi * G > 512:
            G = max(1, G // 2)
        hi = _log_int(rng, 20, 33000)
        # cache values and score products within those of the largest listed case
        room = min(16 * 8192 * 8 * 128 / (hi * Hkv * D), 16 * 8192 * 8 * 256 * 128 / (hi * Hkv * D * n_hi * G), 100)
        B = _log_int(rng, 1, max(1, int(room)))
        return dict(op="tree", B=B, Hq=Hkv * G, Hkv=Hkv, D=D,
                    dtype=rng.choice(["bf16", "bf16", "fp8"]), layout=rng.choice(["HND", "NHD"]),
                    dist=rng.choice(["uniform", "lognormal"]), ctx_lo=rng.randrange(0, hi), ctx_hi=hi,
                    n_lo=rng.randrange(B == 1, n_hi + 1), n_hi=n_hi, mask=rng.choice(["tree", "tree", "chain"]), shape=shape)
    layers = _log_int(rng, 1, 32)
    Hkv = rng.choice([1, 2, 4, 8])
    common = dict(layers=layers, Hkv=Hkv, D=rng.choice([64, 128]), dtype=rng.choice(["bf16", "fp8"]),
                  layout=rng.choice(["HND", "NHD"]), shape=shape)
    if op == "accept":
        n_hi = _log_int(rng, 4, 31)
        return dict(op="accept", B=_log_int(rng, 1, 64), ctx_lo=0, ctx_hi=rng.randrange(1, 150),
                    n_lo=rng.randrange(1, n_hi + 1), n_hi=n_hi, **common)
    if op == "fork":
        parents = _log_int(rng, 1, 32)
        hi = _log_int(rng, 1, 400 if parents > 1 else 5000)
        return dict(op="fork", parents=parents, children=_log_int(rng, 1, 96), len_lo=rng.randrange(0, hi), len_hi=hi,
                    **common)
    B = _log_int(rng, 1, 4096)
    hi = _log_int(rng, 2, 1600)
    step = _log_int(rng, 1, hi)
    need = B * -(-(hi + step) // P)
    return dict(op="resize", B=B, pages=min(524288, max(need + 1, _log_int(rng, 64, 524288))), len_lo=0, len_hi=hi,
                step=step, shape=shape)


def _lens(c):
    """The case's lengths: (context, drafted) of each sequence for tree and accept, lengths otherwise."""
    r = random.Random(c["shape"])
    if c["op"] in ("tree", "accept"):
        ctx = []
        for _ in range(c["B"]):
            if c.get("dist") == "lognormal":
                x = int(round(min(1024, c["ctx_hi"] / 4) * math.exp(r.gauss(0, 1))))
                ctx.append(min(max(x, c["ctx_lo"]), c["ctx_hi"]))
            else:
                ctx.append(r.randint(c["ctx_lo"], c["ctx_hi"]))
        return ctx, [r.randint(c["n_lo"], c["n_hi"]) for _ in range(c["B"])]
    if c["op"] == "fork":
        return [r.randint(c["len_lo"], c["len_hi"]) for _ in range(c["parents"])], \
               [r.randrange(c["parents"]) for _ in range(c["children"])]
    return [r.randint(c["len_lo"], c["len_hi"]) for _ in range(c["B"])], [r.randint(0, c["step"]) for _ in range(c["B"])]


def _accepted(c):
    """Accepted path of each sequence: strictly increasing draft indices."""
    r = random.Random(c["shape"] + 1)
    _, n = _lens(c)
    return [sorted(r.sample(range(k), r.randint(0, min(k, 7)))) for k in n]


# ---- inputs ------------------------------------------------------------------------------------------------------

def _pages(n):
    return -(-n // P)


def _tables(counts, width, pool, g, dev):
    """Block tables from a shuffled pool: row b takes the next counts[b] pages of a permutation; -1 elsewhere."""
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    cnt = torch.tensor(counts, device=dev)
    col = torch.arange(width, device=dev)
    at = (torch.cumsum(cnt, 0) - cnt)[:, None] + col
    held = col < cnt[:, None]
    return torch.where(held, perm[torch.where(held, at, 0)], -1).to(torch.int32)


def _pool(c, n, g, dev):
    """n x [pages, ...] caches of random values in one tensor (bf16 bits or E4M3 bytes as random finite numbers)."""
    shape = (n, c["_pool"], c["Hkv"], P, c["D"]) if c["layout"] == "HND" else (n, c["_pool"], P, c["Hkv"], c["D"])
    if c["dtype"] == "fp8":
        return torch.randint(0, 0x7F, shape, generator=g, device=dev, dtype=torch.uint8)
    return torch.randint(0, 0x7F00, shape, generator=g, device=dev, dtype=torch.int16).view(torch.bfloat16)


def prepare(case, seed):
    s = _prepare(case, seed)
    if own:
        # a serving program keeps its buffers, and binds them once
        import paged_kv_gqa_04_gb300 as pkv
        if s["c"]["op"] == "tree":
            sms = torch.cuda.get_device_properties(s["q"].device).multi_processor_count
            size = pkv.tree_decode_workspace(s["q"].shape[0], s["c"]["Hq"], s["c"]["D"], sms)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["q"].device)
        s["bound"] = {k: pkv.bind(x) for k, x in s.items()
                      if k != "pool" and (x is None or isinstance(x, (torch.Tensor, list)))}
    return s


def _prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"c": c, "err": torch.zeros(1, dtype=torch.int32, device=dev)}
    if c["op"] == "tree":
        return _prepare_tree(c, seed, s, g, dev)
    if c["op"] == "accept":
        ctx, n = _lens(c)
        lens = [a + b for a, b in zip(ctx, n)]
        counts = [_pages(x) for x in lens]
        c["_pool"] = max(1, sum(counts))
        acc = _accepted(c)
        s["pool"] = _pool(c, 2 * c["layers"], g, dev)
        s["caches"] = list(s["pool"].unbind(0))
        s["tables"] = _tables(counts, max(1, max(counts)), c["_pool"], g, dev)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q_start"] = torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device=dev)
        s["accepted"] = torch.tensor([a + [-1] * (8 - len(a)) for a in acc], dtype=torch.int32, device=dev)
        s["n_accepted"] = torch.tensor([len(a) for a in acc], dtype=torch.int32, device=dev)
        s["seq_lens_out"] = torch.zeros_like(s["seq_lens"])
        return s
    if c["op"] == "fork":
        # the state after a first fork: children hold shared pages and a tail page of their own
        lens, of = _lens(c)
        counts = [_pages(x) for x in lens]
        width = max(1, max(counts))
        c["_pool"] = max(1, sum(counts) + len(of) + 8)
        table = _tables(counts, width, c["_pool"], g, dev)
        s["pool"] = _pool(c, 2 * c["layers"], g, dev)
        s["caches"] = list(s["pool"].unbind(0))
        kids = len(of)
        s["tables"] = torch.cat([table, torch.full((kids, width), -1, dtype=torch.int32, device=dev)])
        s["counts"] = torch.tensor(counts + [0] * kids, dtype=torch.int32, device=dev)
        s["seq_lens"] = torch.tensor(lens + [0] * kids, dtype=torch.int32, device=dev)
        s["refs"] = torch.zeros(c["_pool"], dtype=torch.int32, device=dev)
        s["refs"][table[table >= 0].long()] = 1
        s["drop"] = torch.tensor([-1] * len(lens) + [0] * kids, dtype=torch.int32, device=dev)
        s["forks"] = torch.tensor([[p, len(lens) + i] for i, p in enumerate(of)], dtype=torch.int32, device=dev)
        s["copies"] = torch.full((kids, 2), -1, dtype=torch.int32, device=dev)
        _plain_fork(s)
        return s
    # resize: the state grown
    lens, step = _lens(c)
    hi = [a + b for a, b in zip(lens, step)]
    counts = [_pages(x) for x in hi]
    s["tables"] = _tables(counts, max(1, max(counts)), c["pages"], g, dev)
    s["counts"] = torch.tensor(counts, dtype=torch.int32, device=dev)
    s["refs"] = torch.zeros(c["pages"], dtype=torch.int32, device=dev)
    s["refs"][s["tables"][s["tables"] >= 0].long()] = 1
    s["lo"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["hi"] = torch.tensor(hi, dtype=torch.int32, device=dev)
    return s


def _prepare_tree(c, seed, s, g, dev):
    ctx, n = _lens(c)
    lens = [a + b for a, b in zip(ctx, n)]
    counts = [_pages(x) for x in lens]
    pool = max(1, sum(counts))
    shape = (pool, c["Hkv"], P, c["D"]) if c["layout"] == "HND" else (pool, P, c["Hkv"], c["D"])
    for name in ("k", "v"):
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
        if c["dtype"] == "fp8":
            x = (x.float() * 40.0).clamp(-448, 448).to(torch.float8_e4m3fn)
            s[name + "_scale"] = torch.rand(c["Hkv"], generator=g, device=dev) * 0.02 + 0.01
        else:
            s[name + "_scale"] = None
        s[name] = x
    T = sum(n)
    s["tables"] = _tables(counts, max(1, max(counts)), pool, g, dev)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["q_start"] = torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device=dev)
    s["q"] = torch.randn((T, c["Hq"], c["D"]), generator=g, device=dev, dtype=torch.bfloat16)
    s["scale"] = c["D"] ** -0.5
    s["mask"] = None
    if c["mask"] == "tree":
        # each drafted token hangs below an earlier one or below the context; it sees its ancestors and itself
        words = max(1, -(-max(n) // 32))
        r = random.Random(seed * 7919 + c["shape"])
        rows = []
        for k in n:
            anc = []
            for i in range(k):
                parent = r.randrange(-1, i)
                anc.append((anc[parent] if parent >= 0 else 0) | 1 << i)
            rows += [[x >> 32 * w & 0xFFFFFFFF for w in range(words)] for x in anc]
        s["mask"] = torch.tensor(rows, dtype=torch.int64, device=dev).reshape(T, words).to(torch.int32)
    s["n_max"], s["L_max"] = max(n), max(lens)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros((T, c["Hq"]), dtype=torch.float32, device=dev)
    return s


# ---- one pass ----------------------------------------------------------------------------------------------------

def run(s):
    op = s["c"]["op"]
    if own:
        import paged_kv_gqa_04_gb300 as pkv
        lay, t = s["c"].get("layout"), s["bound"]
        if op == "tree":
            pkv.paged_tree_decode(t["q"], t["k"], t["v"], t["tables"], t["seq_lens"], t["q_start"], t["mask"],
                                  s["scale"], t["out"], t["lse"], t["workspace"], t["k_scale"], t["v_scale"],
                                  layout=lay, err_flag=t["err"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "accept":
            pkv.accept_drafts(t["caches"], t["tables"], t["seq_lens"], t["q_start"], t["accepted"], t["n_accepted"],
                              t["seq_lens_out"], layout=lay, err_flag=t["err"])
            return _accept_outputs(s)
        if op == "fork":
            pkv.resize_sequences(t["tables"], t["counts"], t["drop"], t["refs"], P, err_flag=t["err"])
            pkv.fork_sequences(t["caches"], t["tables"], t["counts"], t["seq_lens"], t["forks"], t["refs"],
                               t["copies"], layout=lay, err_flag=t["err"])
            return _fork_outputs(s)
        pkv.resize_sequences(t["tables"], t["counts"], t["lo"], t["refs"], P, err_flag=t["err"])
        pkv.resize_sequences(t["tables"], t["counts"], t["hi"], t["refs"], P, err_flag=t["err"])
        return _resize_outputs(s)
    if op == "tree":
        return _plain_tree(s)
    if op == "accept":
        _plain_accept(s)
        return _accept_outputs(s)
    if op == "fork":
        _plain_resize(s, s["drop"])
        _plain_fork(s)
        return _fork_outputs(s)
    _plain_resize(s, s["lo"])
    _plain_resize(s, s["hi"])
    return _resize_outputs(s)


def _bits(x):
    return x if x.dtype == torch.uint8 else x.view(torch.int16)


def _accept_outputs(s):
    return {"caches": _bits(s["pool"]), "seq_lens": s["seq_lens_out"]}


def _fork_outputs(s):
    return {"caches": _bits(s["pool"]), "tables": s["tables"], "counts": s["counts"], "seq_lens": s["seq_lens"],
            "refs": s["refs"], "copies": s["copies"]}


def _resize_outputs(s):
    return {"tables": s["tables"], "counts": s["counts"], "refs": s["refs"]}


# ---- plain forms ---------------------------------------------------------------------------------------------------

def _plain_tree(s):
    c = s["c"]
    B, Hkv, D, G, N = c["B"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"], s["n_max"]
    out, lse = torch.zeros_like(s["out"]), torch.zeros_like(s["lse"])
    if s["q"].shape[0] == 0:
        return {"out": out, "lse": lse}
    dev = s["q"].device
    ids = s["tables"].long().clamp(min=0)

    def gathered(name):
        x = s[name][ids].to(torch.float32)  # [B, pages, Hkv, P, D] or [B, pages, P, Hkv, D]
        x = x.permute(0, 2, 1, 3, 4) if c["layout"] == "HND" else x.permute(0, 3, 1, 2, 4)
        x = x.reshape(B, Hkv, -1, D)
        return x if s[name + "_scale"] is None else x * s[name + "_scale"][:, None, None]

    start, L = s["q_start"].long(), s["seq_lens"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(N, device=dev)
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    live = i < n[:, None]
    q = s["q"][row].to(torch.float32).reshape(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    k = gathered("k")
    score = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    pos = torch.arange(score.shape[3], device=dev)
    j = pos - (L - n)[:, None]                       # drafted token's index at each position, negative in the context
    if s["mask"] is None:
        seen = j[:, None, :] <= i[None, :, None]
    else:
        jj = j.clamp(0, 32 * s["mask"].shape[1] - 1)[:, None, :].expand(B, N, -1)
        word = torch.gather(s["mask"][row].long(), 2, jj >> 5)
        seen = (j[:, None, :] < 0) | ((word >> (jj & 31)) & 1).bool()
    seen = seen & (pos < L[:, None])[:, None, :]
    seen = seen[:, None, :, None, :].expand(B, Hkv, N, G, -1).reshape(B, Hkv, N * G, -1)
    score = score.masked_fill(~seen, float("-inf"))
    m = score.amax(3, keepdim=True)
    m0 = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    w = torch.exp(score - m0)
    del score, seen
    z = w.sum(3, keepdim=True)
    o = torch.matmul(w, gathered("v")) / torch.where(z > 0, z, torch.ones_like(z))
    o = o.reshape(B, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, c["Hq"], D)
    e = (m0 + torch.log(z)).reshape(B, Hkv, N, G).permute(0, 2, 1, 3).reshape(B, N, c["Hq"])
    out[row[live]] = o[live].to(torch.bfloat16)
    lse[row[live]] = e[live]
    return {"out": out, "lse": lse}


def _plain_accept(s):
    hnd = s["c"]["layout"] == "HND"
    start, L = s["q_start"].long(), s["seq_lens"].long()
    base = L - (start[1:] - start[:-1])
    A = s["accepted"].shape[1]
    j = torch.arange(A, device=L.device)
    src = base[:, None] + s["accepted"].long()
    dst = base[:, None] + j
    move = (j < s["n_accepted"].long()[:, None]) & (src != dst)
    b = torch.arange(L.shape[0], device=L.device)[:, None].expand(-1, A)[move]
    src, dst = src[move], dst[move]
    table = s["tables"].long()
    ps, pd = table[b, src // P], table[b, dst // P]
    x = s["pool"]
    if hnd:
        x = x.transpose(2, 3)
    x[:, pd, dst % P] = x[:, ps, src % P]
    s["seq_lens_out"].copy_(base + s["n_accepted"])


def _plain_resize(s, lens):
    table, counts, refs = s["tables"], s["counts"], s["refs"]
    want = torch.where(lens < 0, counts, (lens + P - 1) // P)
    col = torch.arange(table.shape[1], device=table.device)
    drop = (col >= want[:, None]) & (col < counts[:, None])
    pages = table[drop].long()
    refs.index_add_(0, pages, torch.full_like(pages, -1, dtype=torch.int32))
    table[drop] = -1
    grow = (col < want[:, None]) & (col >= counts[:, None])
    free = torch.nonzero(refs == 0)[:, 0][: int(grow.sum())]
    table[grow] = free.to(torch.int32)
    refs[free] = 1
    counts.copy_(want)


def _plain_fork(s):
    table, counts, refs = s["tables"], s["counts"], s["refs"]
    p, k = s["forks"][:, 0].long(), s["forks"][:, 1].long()
    L = s["seq_lens"][p].long()
    full, part = L // P, L % P > 0
    col = torch.arange(table.shape[1], device=table.device)
    rows = torch.where(col < full[:, None], table[p], -1)
    shared = rows[rows >= 0].long()
    free = torch.nonzero(refs == 0)[:, 0][: int(part.sum())]
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    refs[free] = 1
    tail = table[p[part], full[part]]
    rows[part, full[part]] = free.to(torch.int32)
    table[k] = rows
    counts[k] = (full + part).to(torch.int32)
    s["seq_lens"][k] = L.to(torch.int32)
    s["copies"].fill_(-1)
    s["copies"][part] = torch.stack([tail, free.to(torch.int32)], 1)
    s["pool"][:, free] = s["pool"][:, tail.long()]


# ---- what a pass cannot do without -----------------------------------------------------------------------------------

def work(c):
    if c["op"] == "tree":
        ctx, n = _lens(c)
        e = 1 if c["dtype"] == "fp8" else 2
        T = sum(n)
        live = sum(a + b for a, b in zip(ctx, n) if b)
        pages = sum(_pages(a + b) for a, b in zip(ctx, n) if b)
        nbytes = 2 * live * c["Hkv"] * c["D"] * e + 4 * pages + T * c["Hq"] * (4 * c["D"] + 4) + 8 * c["B"]
        flops = sum(4 * (a + b) * b * c["Hq"] * c["D"] for a, b in zip(ctx, n))
        return {"bytes": nbytes + 1, "flops": flops}
    e = 1 if c.get("dtype") == "fp8" else 2
    if c["op"] == "accept":
        # rows that are in place already are not moved
        acc = _accepted(c)
        moved = sum(a != i for path in acc for i, a in enumerate(path))
        row = c["Hkv"] * c["D"] * e
        return {"bytes": 2 * moved * row * 2 * c["layers"] + 4 * sum(map(len, acc)) + 20 * len(acc), "flops": 0}
    if c["op"] == "fork":
        lens, of = _lens(c)
        page = c["Hkv"] * P * c["D"] * e
        copied = sum(1 for p in of if lens[p] % P)
        entries = sum(_pages(lens[p]) for p in of)
        # released and forked again: entries read and written, a count read and written for each, both ways
        return {"bytes": 2 * copied * page * 2 * c["layers"] + 2 * 16 * entries + 24 * len(of), "flops": 0}
    lens, step = _lens(c)
    moved = sum(_pages(a + b) - _pages(a) for a, b in zip(lens, step))
    # entries and counts of the pages that come and go, and the counts that are searched for free pages
    return {"bytes": 2 * 16 * moved + 4 * c["pages"] + 2 * 16 * c["B"], "flops": 0}


# ---- from the definition, in 64 bits ---------------------------------------------------------------------------------

def exact(case, seed):
    """The tree attention sequence by sequence in float64; the other operators only move whole numbers."""
    if case["op"] != "tree":
        return None
    s = prepare(case, seed)
    c = s["c"]
    ctx, n = _lens(c)
    G = c["Hq"] // c["Hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=s["q"].device)
    at = 0
    for b in range(c["B"]):
        if n[b] == 0:
            continue
        t = torch.arange(ctx[b] + n[b], device=out.device)
        page, off = s["tables"][b].long()[t // P], t % P

        def tokens(name):
            x = s[name][page, :, off] if c["layout"] == "HND" else s[name][page, off]
            x = x.double()
            return x if s[name + "_scale"] is None else x * s[name + "_scale"].double()[:, None]

        k, v = tokens("k"), tokens("v")
        q = s["q"][at:at + n[b]].double().reshape(n[b], c["Hkv"], G, c["D"])
        x = torch.einsum("nhgd,thd->nhgt", q, k) * s["scale"]
        if s["mask"] is None:
            vis = torch.ones(n[b], n[b], device=out.device).tril() > 0
        else:
            m = s["mask"][at:at + n[b]].long()
            vis = torch.stack([(m[:, j // 32] >> (j % 32)) & 1 for j in range(n[b])], 1) > 0
        x[..., ctx[b]:].masked_fill_(~vis[:, None, None, :], float("-inf"))
        lse[at:at + n[b]] = torch.logsumexp(x, 3).reshape(n[b], c["Hq"])
        out[at:at + n[b]] = torch.einsum("nhgt,thd->nhgd", torch.softmax(x, 3), v).reshape(n[b], c["Hq"], c["D"])
        at += n[b]
    return {"out": out, "lse": lse}
