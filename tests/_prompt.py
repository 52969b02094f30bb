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
