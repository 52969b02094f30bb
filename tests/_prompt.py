"""Plain statements of the prompt operators, in float64, straight from their definitions in include/pkv.h."""
import torch

import paged_kv_gqa_04_gb300 as pkv


def make_prompt(n, ctx, Hq, Hkv, D, seed=0, fused=False, spare=0, q_mult=1.0, scale=None, k_gap=0):
    """Device inputs of one prompt attention: n[b] tokens behind ctx[b] keys each; `spare` rows behind the last
    sequence and `k_gap` rows of k and v before every sequence belong to nobody (they hold NaN)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, L = sum(n), [a + b for a, b in zip(n, ctx)]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    def starts(x, gap=0):
        at, s = 0, []
        for y in x:
            s.append(at + gap)
            at += gap + y
        return s, at
    s = {"D": D, "scale": D ** -0.5 if scale is None else scale, "n": list(n), "L": L}
    qs, _ = starts(n)
    if fused:
        s["q"], s["k"], s["v"] = randn(T + spare, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], 1)
        s["k_start"], ks = None, qs
    else:
        ks, Tk = starts(L, k_gap)
        s["q"], s["k"], s["v"] = randn(T + spare, Hq, D), randn(max(1, Tk + spare), Hkv, D), randn(max(1, Tk + spare), Hkv, D)
        # (a range ends where the next one starts, so gaps are rows of a sequence without tokens)
        flat = sum([[k - k_gap, k] if k_gap else [k] for k in ks], []) + [Tk]
        s["k_start"] = torch.tensor(flat, dtype=torch.int32, device="cuda")
        if k_gap:
            qs = sum([[q, q] for q in qs], [])
    s["ks"] = ks
    s["q_start"] = torch.tensor(qs + [T], dtype=torch.int32, device="cuda")
    s["q"].mul_(q_mult)
    own = torch.zeros(s["k"].shape[0], dtype=torch.bool, device="cuda")
    for a, b in zip(ks, L):
        own[a:a + b] = True
    for x in ("k", "v"):
        s[x][~own] = float("nan")
    s["q"][T:] = float("nan")
    s["out"] = torch.full((T + spare, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.full((T + spare, Hq), 7.0, device="cuda")
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def workspace(D):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return torch.randint(0, 255, (pkv.prompt_attention_workspace(D, sms),), dtype=torch.uint8, device="cuda")


def run_prompt(s, **over):
    a = dict(s, **over)
    ws = a["ws"] if "ws" in a else workspace(a["D"])
    pkv.prompt_attention(a["q"], a["k"], a["v"], a["q_start"], a["k_start"], a["scale"], a["out"], a["lse"], ws,
                         err_flag=a["err"], stream=a.get("stream"))


def prompt_reference(s, b, rows=None):
    """(out, lse, tol_out, tol_lse) [rows, Hq, ..] in float64 of sequence b (of its rows `rows`).

    Tolerances count the roundings of the operator. Score: D products exact in fp32, at most D + 8 additions and
    products of relative error 2^-24 over sum |q k|. Weight: the score's error, 2^-20 for the exponential and its
    reference, 2^-8 for its rounding to bf16 (half a step); it meets |v|. Sums over L keys: 2^-24 each. Output: 2^-8 of
    itself for the final rounding."""
    n, L, a, e = s["n"][b], s["L"][b], sum(s["n"][:b]), s["ks"][b]
    Hq, D, Hkv = s["q"].shape[1], s["D"], s["k"].shape[1]
    G = Hq // Hkv
    i = torch.arange(n, device="cuda") if rows is None else torch.tensor(rows, device="cuda")
    vis = torch.arange(L, device="cuda") <= (L - n + i)[:, None]
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    outs = []
    for h in range(Hq):
        q, k, v = s["q"][a + i, h].double(), s["k"][e:e + L, h // G].double(), s["v"][e:e + L, h // G].double()
        x = torch.where(vis, q @ k.T * s["scale"], zero - float("inf"))
        mag = torch.where(vis, q.abs() @ k.abs().T * abs(s["scale"]), zero).nan_to_num(0.0)
        empty = ~vis.any(1)
        ds = (mag.amax(1) if L else torch.zeros(len(i), device="cuda").double()) * (D + 8) * 2.0 ** -24
        m = torch.where(empty, zero, x.amax(1) if L else zero)
        w = torch.exp(x - m[:, None])
        z = torch.where(empty, zero + 1, w.sum(1))
        # (0 times a value that is not finite is nothing where the key is not seen, and NaN where it is)
        odd = ~torch.isfinite(v).all(1)
        o = w @ torch.where(odd[:, None], zero, v)
        av = w @ torch.where(odd[:, None], zero, v).abs()
        for j in odd.nonzero()[:, 0].tolist():
            o[vis[:, j]] += w[vis[:, j], j, None] * v[j]
        o, av = o / z[:, None], av / z[:, None]
        more = (2 * ds + 2.0 ** -20 + (L + 8) * 2.0 ** -24)[:, None]
        lse = torch.where(empty, zero - float("inf"), m + torch.log(z))
        outs.append((o, lse, 2.0 ** -8 * o.abs() + (2.0 ** -8 + more) * (1 + 2.0 ** -8) * av,
                     ds + 2.0 ** -20 + (L + 8) * 2.0 ** -24 + 2.0 ** -22 * lse.nan_to_num(0, 0, 0).abs()))
    return [torch.stack(x, 1) for x in zip(*outs)]


def check_prompt(s, flags=0, rows=None):
    torch.cuda.synchronize()
    assert int(s["err"].item()) == flags
    T = sum(s["n"])
    assert bool((s["out"][T:] == 7.0).all()) and bool((s["lse"][T:] == 7.0).all())
    for b, n in enumerate(s["n"]):
        if n == 0:
            continue
        a = sum(s["n"][:b])
        out, lse, tol, tol_l = prompt_reference(s, b, rows)
        at = torch.arange(a, a + n, device="cuda") if rows is None else a + torch.tensor(rows, device="cuda")
        got, gl = s["out"][at].double(), s["lse"][at].double()
        assert torch.equal(torch.isnan(got), torch.isnan(out)), f"sequence {b}: NaN where there is none, or none"
        inf = torch.isinf(out)
        assert torch.equal(got[inf], out[inf])
        fine = torch.isfinite(out)
        err = (got - out).abs()[fine]
        assert bool((err <= tol[fine] + 1e-30).all()), f"sequence {b}: out {float((err - tol[fine]).max())} over its bound"
        assert torch.equal(gl == -float("inf"), lse == -float("inf")) and torch.equal(torch.isnan(gl), torch.isnan(lse))
        fl = torch.isfinite(lse)
        assert bool(((gl - lse).abs()[fl] <= tol_l[fl]).all()), f"sequence {b}: lse {float((gl - lse).abs()[fl].max())}"


# ---- normed and rotated writes, and rows read back -------------------------------------------------------------------

WIDTH = {"bf16": 1.0, "fp8": 1.0, "nvfp4": 0.5}


def make_write(T, Hq, Hkv, D, dtype="bf16", layout="HND", style="neox", weight="f32", k_out=True, P=16, seed=0, packed=True,
               skip=(), signs=False, pages=None, eps=1e-6):
    """Device inputs of one normed write: T tokens at random positions and slots; `skip`: tokens without a slot."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        x = torch.randn(shape, generator=g, device="cuda")
        return (torch.where(x < 0, -1.0, 1.0) if signs else x).bfloat16()
    s = dict(D=D, Hq=Hq, Hkv=Hkv, dtype=dtype, layout=layout, style=style, P=P, eps=0.0 if signs else eps)
    if packed:
        s["q"], s["k"], s["v"] = randn(T, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], 1)
    else:
        s["q"], s["k"], s["v"] = randn(T, Hq, D), randn(T, Hkv, D), randn(T, Hkv, D)
    s["v"].mul_(1.5 + torch.randn(T, 1, 1, generator=g, device="cuda").bfloat16())
    for x in ("q", "k"):
        w = 1 + 0.4 * torch.randn(D, generator=g, device="cuda")
        s[x + "_weight"] = w.bfloat16() if weight == "bf16" or signs else w
        if signs and weight == "f32":
            s[x + "_weight"] = s[x + "_weight"].float()
    pool = pages or -(-T // P) + 3
    slots = torch.randperm(pool * P, generator=g, device="cuda")[:T].to(torch.int32)
    for t in skip:
        slots[t] = -1
    s["slots"], s["pool"] = slots, pool
    s["positions"] = torch.randint(0, 3000, (T,), generator=g, device="cuda", dtype=torch.int32)
    f = 10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    ang = torch.arange(3000, device="cuda", dtype=torch.float64)[:, None] * f
    s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()

    def cache(width, dt, fill):
        shape = (pool, Hkv, P, width) if layout == "HND" else (pool, P, Hkv, width)
        return torch.full(shape, fill, dtype=dt, device="cuda")
    for x in ("k", "v"):
        if dtype == "bf16":
            s[x + "_cache"] = cache(D, torch.bfloat16, 7.0)
        else:
            s[x + "_cache"] = cache(D if dtype == "fp8" else D // 2, torch.uint8, 0x55)
        s[x + "_bs"] = cache(D // 16, torch.uint8, 0x55) if dtype == "nvfp4" else None
        top = 5.0 / 448 if dtype == "fp8" else 5.0 / (6 * 448)
        s[x + "_scale"] = None if dtype == "bf16" else top * (0.5 + torch.rand(Hkv, generator=g, device="cuda"))
    s["k_out"] = torch.full((T, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") if k_out else None
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def run_write(s, **over):
    a = dict(s, **over)
    pkv.qk_norm_rope_kv_write(a["q"], a["k"], a["v"], a["q_weight"], a["k_weight"], a["eps"], a["positions"], a["cos_sin"],
                              a["k_cache"], a["v_cache"], a["slots"], a["k_scale"], a["v_scale"], k_block_scale=a["k_bs"],
                              v_block_scale=a["v_bs"], k_out=a["k_out"], layout=a["layout"], rope_style=a["style"],
                              err_flag=a["err"], stream=a.get("stream"))


def normed(s, x, w):
    """(rotated rows, bound of their float32 errors) in float64.

    The sum of squares is off by at most D / 2 + 8 additions' and products' 2^-24 of itself, which halves under the
    root; the reciprocal root adds four (two units in the last place), two products one each. A rotated value is a
    difference of two products of such values, each rounded once more, and the sum."""
    x, w, D = x.double(), w.double(), s["D"]
    y = x / (x.pow(2).mean(-1, keepdim=True) + s["eps"]).sqrt() * w
    cs = s["cos_sin"].double()[s["positions"].long().clamp(0, s["cos_sin"].shape[0] - 1)][:, None]
    c, sn = cs[..., :D // 2], cs[..., D // 2:]
    a, b = (y[..., :D // 2], y[..., D // 2:]) if s["style"] == "neox" else (y[..., 0::2], y[..., 1::2])
    u, v = a * c - b * sn, b * c + a * sn
    eu, ev = (a * c).abs() + (b * sn).abs(), (b * c).abs() + (a * sn).abs()
    out, err = (torch.cat(z, -1) if s["style"] == "neox" else torch.stack(z, -1).flatten(-2) for z in ((u, v), (eu, ev)))
    return out, err * (D / 4 + 16) * 2.0 ** -24


def rows_of(s, cache, slots):
    """[n, Hkv, width] of a cache at the given slots."""
    page, off = slots.long() // s["P"], slots.long() % s["P"]
    return cache[page, :, off] if s["layout"] == "HND" else cache[page, off]


E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def fp4_values(b):
    code = torch.stack([b & 15, b >> 4], -1).flatten(-2).long()
    return E2M1.to(b.device)[code & 7] * (1 - 2 * (code >> 3)).float()


def check_write(s, before, flags=0):
    """before: q, k and v as they were."""
    torch.cuda.synchronize()
    assert int(s["err"].item()) == flags
    n_slots = s["pool"] * s["P"]
    live = (s["slots"] >= 0) & (s["slots"] < n_slots) & (s["positions"] >= 0) & (s["positions"] < s["cos_sin"].shape[0])
    q, eq = normed(s, before["q"], s["q_weight"])
    k, ek = normed(s, before["k"], s["k_weight"])
    outs = [(s["q"], q, eq, before["q"])]
    if s["k_out"] is not None:
        outs.append((s["k_out"], k, ek, torch.full_like(s["k_out"], 7.0)))
    for got, want, e, old in outs:
        assert torch.equal(got[~live], old[~live])
        d = (got.double() - want).abs()[live]
        assert bool((d <= (2.0 ** -8 * want.abs() + e * (1 + 2.0 ** -8) + 2.0 ** -133)[live]).all())
    assert torch.equal(s["v"], before["v"])
    slots = s["slots"][live]
    used = torch.zeros(n_slots, dtype=torch.bool, device="cuda")
    used[slots.long()] = True
    idle = torch.arange(n_slots, device="cuda")[~used]
    for x, y, e in (("k", k[live], ek[live]), ("v", before["v"].double()[live], torch.zeros_like(ek[live]))):
        cache, sc = s[x + "_cache"], s[x + "_scale"]
        fill = 7.0 if s["dtype"] == "bf16" else 0x55
        assert bool((rows_of(s, cache, idle) == fill).all())
        got = rows_of(s, cache, slots)
        if s["dtype"] == "bf16":
            assert bool(((got.double() - y).abs() <= 2.0 ** -8 * y.abs() + e * (1 + 2.0 ** -8) + 2.0 ** -133).all())
            if x == "v":
                assert torch.equal(got, before["v"][live])
            continue
        g = sc.double()[:, None]
        if s["dtype"] == "fp8":
            z, ez = (y / g), e / g + 2.0 ** -23 * (y / g).abs()
            c = got.view(torch.float8_e4m3fn).double()
            assert bool(((c - z.clamp(-448, 448)).abs() <= 2.0 ** -4 * z.abs() + 2.0 ** -10 + ez * 1.07).all())
            continue
        bs = rows_of(s, s[x + "_bs"], slots)
        assert bool((rows_of(s, s[x + "_bs"], idle) == 0x55).all())
        b, eb = y.unflatten(-1, (-1, 16)), e.unflatten(-1, (-1, 16))
        want_s = (b.abs().amax(-1) / (6 * g)).clamp(max=448.0)
        got_s = bs.view(torch.float8_e4m3fn).double()
        assert bool(((got_s - want_s).abs() <= 2.0 ** -4 * want_s + 2.0 ** -10 + 2 * eb.amax(-1) / (6 * g)).all())
        den = (g * got_s)[..., None]
        z = torch.where(den > 0, b / den.clamp(min=1e-300), torch.zeros_like(b))
        step = torch.where(z.abs() < 2, 0.5, torch.where(z.abs() < 4, 1.0, 2.0))
        ez = torch.where(den > 0, eb / den.clamp(min=1e-300), torch.zeros_like(b)) + 2.0 ** -22 * z.abs()
        c = fp4_values(got).double().unflatten(-1, (-1, 16))
        assert bool(((c - z.clamp(-6, 6)).abs() <= step / 2 + ez * 1.01 + 1e-12).all())


def make_read(n, first, Hkv, D, dtype="bf16", layout="HND", P=16, seed=0, spare=0, strided=False):
    """Device inputs of one reading back: rows n[b] from position first[b] on of sequences in shuffled pages."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    need = [-(-(a + b) // P) for a, b in zip(n, first)]
    pool = sum(need) + 2
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((len(n), max(1, max(need, default=1))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(need):
        bt[b, :c] = perm[at:at + c]
        at += c
    s = dict(D=D, Hkv=Hkv, dtype=dtype, layout=layout, P=P, bt=bt, n=list(n), first_list=list(first))

    def cache(width, dt):
        shape = (pool, Hkv, P, width) if layout == "HND" else (pool, P, Hkv, width)
        if strided:
            shape = (pool, 2) + shape[1:]
        if dt == torch.bfloat16:
            x = torch.randn(shape, generator=g, device="cuda").bfloat16()
        else:
            x = torch.randint(0, 0x7F, shape, generator=g, device="cuda", dtype=torch.uint8)
            x |= torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) * 0x80
        return x[:, 1] if strided else x
    for x in ("k", "v"):
        s[x + "_cache"] = cache(D // 2 if dtype == "nvfp4" else D, torch.bfloat16 if dtype == "bf16" else torch.uint8)
        s[x + "_bs"] = cache(D // 16, torch.uint8) & 0x7F if dtype == "nvfp4" else None
        s[x + "_scale"] = None if dtype == "bf16" else torch.rand(Hkv, generator=g, device="cuda") * 0.02 + 0.01
        s[x + "_out"] = torch.full((sum(n) + spare, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    starts = [sum(n[:i]) for i in range(len(n) + 1)]
    s["start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["first"] = torch.tensor(list(first), dtype=torch.int32, device="cuda") if any(first) else None
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def run_read(s, **over):
    a = dict(s, **over)
    pkv.gather_kv(a["k_cache"], a["v_cache"], a["bt"], a["start"], a["first"], a["k_out"], a["v_out"], a["k_scale"],
                  a["v_scale"], k_block_scale=a["k_bs"], v_block_scale=a["v_bs"], layout=a["layout"], err_flag=a["err"],
                  stream=a.get("stream"))


def read_reference(s, x):
    """Rows of one cache, bit for bit: bf16( f32( scale * value ) )."""
    seq = torch.cat([torch.full((c,), b, dtype=torch.long) for b, c in enumerate(s["n"])] or [torch.zeros(0).long()]).cuda()
    pos = torch.cat([torch.arange(f, f + c) for f, c in zip(s["first_list"], s["n"])] or [torch.zeros(0).long()]).cuda()
    entry = pos // s["P"]
    inside = (pos >= 0) & (entry < s["bt"].shape[1])
    page = torch.where(inside, s["bt"][seq, entry.clamp(0, s["bt"].shape[1] - 1)].long(), -1)
    ok = (page >= 0) & (page < s[x + "_cache"].shape[0])
    slot = page.clamp(0, s[x + "_cache"].shape[0] - 1) * s["P"] + pos % s["P"]
    y = rows_of(s, s[x + "_cache"], slot)
    if s["dtype"] != "bf16":
        g = s[x + "_scale"][:, None]
        if s["dtype"] == "fp8":
            y = y.view(torch.float8_e4m3fn).float() * g
        else:
            sc = rows_of(s, s[x + "_bs"], slot).view(torch.float8_e4m3fn).float()
            y = (fp4_values(y).unflatten(-1, (-1, 16)) * sc[..., None]).flatten(-2) * g
        y = y.bfloat16()
    return torch.where(ok[:, None, None], y, torch.zeros_like(y))


def check_read(s, flags=0):
    torch.cuda.synchronize()
    assert int(s["err"].item()) == flags
    T = sum(s["n"])
    for x in ("k", "v"):
        want, got = read_reference(s, x), s[x + "_out"]
        assert torch.equal(got[:T].view(torch.int16), want.view(torch.int16)) or \
            torch.equal(torch.nan_to_num(got[:T].float(), 1e30), torch.nan_to_num(want.float(), 1e30))
        assert bool((got[T:] == 7.0).all())
