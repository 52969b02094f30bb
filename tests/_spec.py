"""Plain statements of the drafted-token and page operators, on the host.

Test infrastructure: the attention in float64 sequence by sequence, the page
operators entry by entry, straight from their definitions in include/pkv.h."""
import numpy as np
import torch

P = 16


def make_tree(lens, drafts, Hq, Hkv, D, dtype="bf16", layout="HND", seed=0, mask="tree", spare_rows=0, spare_pages=3,
              num_pages=None, pool_strides=False, k_mult=1.0):
    """Device inputs of one tree decode: random cache, shuffled pages, random trees (or "chain" / "random" bits)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = np.random.RandomState(seed)
    need = [-(-L // P) for L in lens]
    pool = num_pages or max(1, sum(need) + spare_pages)
    shape = (pool, Hkv, P, D) if layout == "HND" else (pool, P, Hkv, D)
    s = {"layout": layout, "dtype": dtype, "D": D, "scale": D ** -0.5}
    if pool_strides:  # K and V as views of one tensor of both
        both = torch.randn((pool, 2) + shape[1:], generator=g, device="cuda", dtype=torch.bfloat16)
        kv = {"k": both[:, 0], "v": both[:, 1]}
    else:
        kv = {n: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) for n in ("k", "v")}
    kv["k"].mul_(k_mult)
    for n in ("k", "v"):
        s[n] = kv[n] if dtype == "bf16" else (kv[n].float() * 40).clamp(-448, 448).to(torch.float8_e4m3fn)
        s[n + "_scale"] = None if dtype == "bf16" else torch.rand(Hkv, generator=g, device="cuda") * 0.02 + 0.01
    perm = r.permutation(pool)
    bt = np.full((len(lens), max(1, max(need, default=1))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[at:at + n] if num_pages is None else perm[::-1][at:at + n]
        at += n
    T = sum(drafts) + spare_rows
    start = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
    s["q"] = torch.randn((T, Hq, D), generator=g, device="cuda", dtype=torch.bfloat16)
    W = max(1, -(-max(drafts, default=1) // 32))
    vis = np.zeros((T, 32 * W), bool)
    for b, n in enumerate(drafts):
        for i in range(n):
            if mask == "random":
                vis[start[b] + i, :n] = r.rand(n) < 0.5
            else:
                p = r.randint(-1, i) if i else -1
                if p >= 0:
                    vis[start[b] + i] = vis[start[b] + p]
                vis[start[b] + i, i] = True
    words = np.packbits(vis.reshape(T, W, 32), axis=2, bitorder="little").view(np.uint32).reshape(T, W)
    s["mask"] = None if mask == "chain" else torch.from_numpy(words.view(np.int32).copy()).cuda()
    s["bt"], s["q_start"] = torch.from_numpy(bt).cuda(), torch.from_numpy(start).cuda()
    s["seq_lens"] = torch.tensor(list(lens), dtype=torch.int32, device="cuda")
    s["out"] = torch.full_like(s["q"], 7.0)
    s["lse"] = torch.full((T, Hq), 7.0, device="cuda")
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def run_tree(s, **over):
    import paged_kv_gqa_04_gb300 as pkv
    a = dict(s, **over)
    if "ws" not in a:
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        n = pkv.tree_decode_workspace(a["q"].shape[0], a["q"].shape[1], a["D"], sms)
        a["ws"] = torch.randint(0, 255, (n,), dtype=torch.uint8, device="cuda")
    pkv.paged_tree_decode(a["q"], a["k"], a["v"], a["bt"], a["seq_lens"], a["q_start"], a["mask"], a["scale"], a["out"],
                          a["lse"], a["ws"], a["k_scale"], a["v_scale"], layout=a["layout"], err_flag=a["err"],
                          stream=a.get("stream"))


def tree_reference(s):
    """(out, lse, tol_out, tol_lse) in float64; rows of no sequence are NaN.

    Tolerances count the roundings of the operator. Score: D products exact in
    fp32, at most D + 8 additions and products of relative error 2^-24 over
    sum |q k| (with room for the order of the sum). Weight: the score's error,
    2^-20 for the exponential, 2^-8 for its rounding to bf16 (half a step); it
    meets |v|. Output: 2^-8 of itself for the final rounding."""
    q, D = s["q"].double(), s["D"]
    T, Hq = q.shape[:2]
    start, lens, bt = s["q_start"].tolist(), s["seq_lens"].tolist(), s["bt"].long()
    pool = s["k"].shape[0]
    Hkv = s["k"].shape[1] if s["layout"] == "HND" else s["k"].shape[2]
    G = Hq // Hkv
    out, tol = torch.full((T, Hq, D), float("nan")).double(), torch.zeros(T, Hq, D).double()
    lse, tol_l = torch.full((T, Hq), float("nan")).double(), torch.zeros(T, Hq).double()
    for b in range(len(lens)):
        a, e = min(max(start[b], 0), T), min(max(start[b + 1], max(start[b], 0)), T)
        n = e - a
        if n == 0:
            continue
        L = min(max(lens[b], 0), bt.shape[1] * P)
        t = torch.arange(L, device=q.device)
        page = bt[b][t // P]
        ok = (page >= 0) & (page < pool)
        t, page = t[ok], page[ok]

        def tokens(name):
            x = s[name][page, :, t % P] if s["layout"] == "HND" else s[name][page, t % P]
            x = x.float().double()
            return x if s[name + "_scale"] is None else x * s[name + "_scale"].double()[:, None]
        k, v = tokens("k"), tokens("v")
        j = t - (L - n)
        i = torch.arange(n, device=q.device)
        if s["mask"] is None:
            vis = j[None] <= i[:, None]
        else:
            W = s["mask"].shape[1]
            jj = j.clamp(0, 32 * W - 1)
            vis = (s["mask"][a:e].long()[:, jj >> 5] >> (jj & 31) & 1).bool() & (j < 32 * W) | (j < 0)
        qq = q[a:e].reshape(n, Hkv, G, D)
        seen = vis[:, None, None, :].expand(n, Hkv, G, -1)
        zero = torch.zeros((), dtype=torch.float64, device=q.device)
        x = torch.einsum("nhgd,thd->nhgt", qq, k) * s["scale"]
        mag = torch.einsum("nhgd,thd->nhgt", qq.abs(), k.abs()) * abs(s["scale"])
        ds = torch.where(seen, mag, zero).nan_to_num(0.0).amax(3) * (D + 8) * 2.0 ** -24 if t.numel() else torch.zeros(n, Hkv, G).double().to(q.device)
        x = torch.where(seen, x, zero - float("inf"))
        empty = ~seen.any(3)
        m = torch.where(empty, zero, x.amax(3) if t.numel() else zero.expand(n, Hkv, G))
        w = torch.exp(x - m[..., None])
        z = w.sum(3)
        o = torch.zeros(n, Hkv, G, D, dtype=torch.float64, device=q.device)
        av = torch.zeros_like(o)
        for r0 in range(n):  # only visible tokens: a masked NaN stays out
            c = vis[r0]
            o[r0] = torch.einsum("hgt,thd->hgd", w[r0][..., c], v[c])
            av[r0] = torch.einsum("hgt,thd->hgd", w[r0][..., c], v[c].abs())
        zz = torch.where(empty, zero + 1, z)[..., None]
        o, av = o / zz, av / zz
        out[a:e] = o.reshape(n, Hq, D).cpu()
        tol[a:e] = (2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * ds + 2.0 ** -20)[..., None] * av).reshape(n, Hq, D).cpu()
        lse[a:e] = torch.where(empty, zero - float("inf"), m + torch.log(z)).reshape(n, Hq).cpu()
        tol_l[a:e] = (ds + 2.0 ** -20 + 2.0 ** -22 * lse[a:e].reshape(n, Hkv, G).to(q.device).nan_to_num(0, 0, 0).abs()).reshape(n, Hq).cpu()
    return out, lse, tol, tol_l


def check_tree(s, rows=None, flags=0):
    torch.cuda.synchronize()
    assert int(s["err"].item()) == flags
    out, lse, tol, tol_l = tree_reference(s)
    got, gl = s["out"].double().cpu(), s["lse"].double().cpu()
    covered = torch.zeros(out.shape[0], dtype=torch.bool)
    start = s["q_start"].tolist()
    for a, e in zip(start, start[1:]):
        covered[max(a, 0):max(e, 0)] = True
    assert bool((got[~covered] == 7.0).all()) and bool((gl[~covered] == 7.0).all())
    out, lse, tol, tol_l, got, gl = (x[covered] for x in (out, lse, tol, tol_l, got, gl))
    assert torch.equal(torch.isnan(got), torch.isnan(out))
    fine = torch.isfinite(out)
    err = (got - out).abs()[fine]
    assert bool((err <= tol[fine] + 1e-30).all()), f"out: worst {float((err - tol[fine]).max())} over its bound"
    assert torch.equal(gl == -float("inf"), lse == -float("inf")) and torch.equal(torch.isnan(gl), torch.isnan(lse))
    fl = torch.isfinite(lse)
    assert bool(((gl - lse).abs()[fl] <= tol_l[fl]).all()), f"lse: {float((gl - lse).abs()[fl].max())}"


# ---- pages ---------------------------------------------------------------------------------------------------------

DRAFT_RANGE, POOL_EMPTY, PAGE_STATE, SEQ_LEN_RANGE, PAGE_RANGE = 0x80, 0x100, 0x200, 0x08, 0x04


def resize_reference(bt, counts, new_lens, refs, page_size):
    """The four arrays after the call, and its flags (arrays are copied)."""
    bt, counts, refs = bt.copy(), counts.copy(), refs.copy()
    flags = 0
    B, width = bt.shape
    grow = []
    for b in range(B):
        want = counts[b]
        if not 0 <= counts[b] <= width:
            flags |= PAGE_STATE
        elif new_lens[b] >= 0:
            need = -(-int(new_lens[b]) // page_size)
            if need > width:
                flags |= SEQ_LEN_RANGE
            else:
                want = need
        for j in range(want, counts[b]):
            page = bt[b, j]
            bt[b, j] = -1
            if not 0 <= page < len(refs):
                flags |= PAGE_RANGE
            elif refs[page] <= 0:
                flags |= PAGE_STATE
            else:
                refs[page] -= 1
        grow.append(want)
    free = [int(p) for p in np.flatnonzero(refs == 0)]
    used = 0
    for b in range(B):
        if grow[b] > counts[b]:
            used += grow[b] - counts[b]
            if used > len(free):
                flags |= POOL_EMPTY
                continue
            for j in range(counts[b], grow[b]):
                bt[b, j] = free[used - grow[b] + j]
                refs[bt[b, j]] = 1
        counts[b] = grow[b]
    return bt, counts, refs, flags


def fork_reference(pools, bt, counts, lens, forks, refs, P_):
    """pools: list of [pages, P-bytes...] arrays (page first). Returns the
    arrays after the call, the copies and the flags."""
    pools = [p.copy() for p in pools]
    bt0, c0, l0 = bt, counts, lens
    bt, counts, lens, refs = bt.copy(), counts.copy(), lens.copy(), refs.copy()
    flags, copies, taken = 0, [], set()
    free = [int(p) for p in np.flatnonzero(refs == 0)]
    used = 0
    for p, c in forks:
        copies.append((-2, -2))
        if p < 0:
            continue
        if p >= len(bt) or not 0 <= c < len(bt) or c0[c] > 0:
            flags |= PAGE_STATE
            continue
        L = int(l0[p])
        full, part = L // P_, L % P_ > 0
        if L < 0 or full + part > min(max(c0[p], 0), bt.shape[1]):
            flags |= SEQ_LEN_RANGE
            continue
        if part and not 0 <= bt0[p, full] < len(refs):
            flags |= PAGE_RANGE
            continue
        if c in taken:
            flags |= PAGE_STATE
            continue
        taken.add(c)
        if part:
            used += 1
            if used > len(free):
                flags |= POOL_EMPTY
                continue
        for j in range(full):
            bt[c, j] = bt0[p, j]
            if 0 <= bt0[p, j] < len(refs):
                refs[bt0[p, j]] += 1
            else:
                flags |= PAGE_RANGE
        copies[-1] = (-1, -1)
        if part:
            dst = free[used - 1]
            bt[c, full] = dst
            refs[dst] = 1
            copies[-1] = (int(bt0[p, full]), dst)
            for x in pools:
                x[dst] = x[bt0[p, full]]
        counts[c] = full + part
        lens[c] = L
    return pools, bt, counts, lens, refs, np.array(copies, np.int32).reshape(-1, 2), flags


def accept_reference(pools, bt, lens, start, accepted, n_acc, P_):
    """pools: list of [pages, P, bytes] arrays. Returns (pools, lens_out, flags)."""
    pools = [p.copy() for p in pools]
    out = lens.copy()
    flags = 0
    for b in range(len(lens)):
        L, N, n = int(lens[b]), int(start[b + 1] - start[b]), int(n_acc[b])
        if not 0 <= L <= bt.shape[1] * P_:
            flags |= SEQ_LEN_RANGE
            continue
        acc = [int(x) for x in accepted[b, :max(n, 0)]]
        if not 0 <= N <= L or not 0 <= n <= min(N, accepted.shape[1]) or any(
                not 0 <= x < N for x in acc) or any(y <= x for x, y in zip(acc, acc[1:])):
            flags |= DRAFT_RANGE
            continue
        base = L - N
        out[b] = base + n
        for j, a in enumerate(acc):
            if a == j:
                continue
            s, d = base + a, base + j
            ps, pd = bt[b, s // P_], bt[b, d // P_]
            if not (0 <= ps < pools[0].shape[0] and 0 <= pd < pools[0].shape[0]):
                flags |= PAGE_RANGE
                continue
            for x in pools:
                x[pd, d % P_] = x[ps, s % P_]
    return pools, out, flags
