"""GPU tests of how exactly the drafted-token attention (pkv_paged_tree_decode)
carries its weights, with tolerances that count each rounding of its own, and
of single rows of V at every place of a long context."""
import pytest
import torch

import paged_kv_gqa_04_gb300 as pkv
from tests._spec import check_tree, make_tree, run_tree

pytestmark = pytest.mark.gpu


def _reference(s):
    """(out, sum of weights x |v|, worst score error) per row and head in float64, from the tables."""
    q, D = s["q"].double(), s["D"]
    T, Hq = q.shape[:2]
    hnd = s["layout"] == "HND"
    Hkv = s["k"].shape[1 if hnd else 2]
    start, lens = s["q_start"].tolist(), s["seq_lens"].tolist()
    out, av, ds = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(T, Hq, dtype=torch.float64, device=q.device)
    for b, L in enumerate(lens):
        a, e = start[b], start[b + 1]
        n = e - a
        if n == 0:
            continue
        t = torch.arange(L, device=q.device)
        page = s["bt"][b].long()[t // 16]

        def tokens(name):
            x = (s[name][page, :, t % 16] if hnd else s[name][page, t % 16]).float().double()
            return x if s[name + "_scale"] is None else x * s[name + "_scale"].double()[:, None]
        k, v = tokens("k"), tokens("v")
        j, i = t - (L - n), torch.arange(n, device=q.device)
        if s["mask"] is None:
            vis = j[None] <= i[:, None]
        else:
            jj = j.clamp(min=0)
            vis = (s["mask"][a:e].long()[:, jj >> 5] >> (jj & 31) & 1).bool() | (j < 0)
        qq = q[a:e].reshape(n, Hkv, -1, D)
        x = torch.einsum("nhgd,thd->nhgt", qq, k) * s["scale"]
        mag = torch.einsum("nhgd,thd->nhgt", qq.abs(), k.abs()) * abs(s["scale"])
        w = torch.softmax(x.masked_fill(~vis[:, None, None], -float("inf")), 3)
        out[a:e] = torch.einsum("nhgt,thd->nhgd", w, v).reshape(n, Hq, D)
        av[a:e] = torch.einsum("nhgt,thd->nhgd", w, v.abs()).reshape(n, Hq, D)
        # D products exact in fp32, at most D + 8 additions and products, the argument of the exponential
        ds[a:e] = ((D + 8) * 2.0 ** -24 * mag.amax(3) + 2.0 ** -22 * x.abs().amax(3)).reshape(n, Hq)
    return out, av, ds


def _check_weights(s, weight):
    """`weight`: the relative rounding of a weight.

    Beside it, of sum(w |v|): the scores' errors twice (weights and their sum), 2^-20 for the exponential,
    and 2^-22 for each of the K-steps (16 positions of one term) that the accumulator takes; and half a
    step of bf16 of the output."""
    torch.cuda.synchronize()
    assert int(s["err"].item()) == 0
    out, av, ds = _reference(s)
    steps = 2 * (max(s["seq_lens"].tolist()) // 16 + 8)
    tol = 2.0 ** -8 * out.abs() + (weight + 2 * ds + 2.0 ** -20 + steps * 2.0 ** -22)[..., None] * av
    worst = float(((s["out"].double() - out).abs() / tol).max())
    assert worst <= 1, f"{worst:.2f} times the bound"


SHAPES = {
    "one_row_tile": ([150, 40, 290], [9, 16, 1], 8, 2, 128, {}),
    "two_row_tiles": ([200, 90], [64, 33], 32, 8, 128, {}),
    "d64": ([150, 290], [31, 100], 8, 2, 64, dict(mask="random")),
    "chain": ([250, 129], [60, 9], 12, 2, 128, dict(mask="chain", layout="NHD")),
}


@pytest.mark.parametrize("name", SHAPES)
def test_bf16_weights_keep_sixteen_bits(name):
    """As in the decode step: a rounded term (2^-8) and the rounded rest (2^-8 of that). Scores near one
    another, so that what the weights lose is not hidden by the scores' own roundings."""
    lens, drafts, Hq, Hkv, D, more = SHAPES[name]
    s = make_tree(lens, drafts, Hq, Hkv, D, seed=31, k_mult=0.1, **more)
    run_tree(s)
    _check_weights(s, 2.0 ** -16)


@pytest.mark.parametrize("name", SHAPES)
def test_fp8_weights_keep_eleven_bits(name):
    """f16: half a step of 2^-11."""
    lens, drafts, Hq, Hkv, D, more = SHAPES[name]
    s = make_tree(lens, drafts, Hq, Hkv, D, dtype="fp8", seed=35, k_mult=0.1, **more)
    run_tree(s)
    _check_weights(s, 2.0 ** -11)


@pytest.mark.parametrize("L", [3000, 131072, 1 << 20])
@pytest.mark.parametrize("at", ["first", "middle"])
def test_fp8_weights_beside_a_dominant_position(L, at):
    """One position takes nearly all the weight and the others, together, the rest: a weight each of 2^-7.9 to
    2^-26 of it. f16 holds 2^7 of a weight: 2^-11 of it, or half of f16's smallest step, 2^-32 of the reference.
    160 sequences of the same pages, so that no CTA has less than a whole one."""
    N, G, D, B = 3, 8, 64, 160
    ratio = torch.tensor([7.9, 10, 15, 18, 21, 24, 24.9, 26], dtype=torch.float64)
    s = make_tree([L], [N], G, 1, D, dtype="fp8", seed=32, mask="chain")
    pos = 0 if at == "first" else L // 2
    s["scale"] = 2.0 ** -4
    s["k_scale"].fill_(0.5)
    s["v_scale"].fill_(1.0)
    q = torch.zeros(N, G, D, device="cuda", dtype=torch.float64)
    q[..., 0] = (ratio / (2.0 ** -4 * 0.5 * 64 * 1.4426950408889634)).cuda()
    s["q"] = q.to(torch.bfloat16).repeat(B, 1, 1)
    s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros(B * N, G, device="cuda")
    flat = s["bt"][0].long()[torch.arange(L, device="cuda") // 16] * 16 + torch.arange(L, device="cuda") % 16
    k, v = torch.zeros(L, D, device="cuda"), torch.randint(1, 4, (L, D), device="cuda").float() / 2
    k[pos, 0] = 64
    v[pos, ::2] = 0
    for name, x in (("k", k), ("v", v)):
        rows = torch.zeros(s[name].shape[0] * 16, D, device="cuda").to(torch.float8_e4m3fn)
        rows.view(torch.uint8)[flat] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        s[name] = rows.view(s[name].shape)
    s["bt"], s["seq_lens"] = s["bt"].repeat(B, 1), s["seq_lens"].repeat(B)
    s["q_start"] = torch.arange(B + 1, dtype=torch.int32, device="cuda") * N
    run_tree(s)
    torch.cuda.synchronize()
    assert int(s["err"].item()) == 0
    score = s["q"][:N, :, 0].double() * 64 * 0.5 * 2.0 ** -4                  # [N, G]; 0 for the others
    w = torch.exp(-score)
    v = v.double()
    seen = L - N + 1 + torch.arange(N, device="cuda")
    total = torch.stack([v[:int(n)].sum(0) for n in seen]) - v[pos]         # [N, D]
    z = 1 + w * (seen - 1)[:, None]
    out = (v[pos] + w[..., None] * total[:, None]) / z[..., None]           # (av = out: no negative values)
    ds = 4 * 2.0 ** -24 * score * 1.4426950408889634
    steps = L // 16 + 8
    tol = (2.0 ** -8 + 2.0 ** -11 + 2 * ds + 2.0 ** -20 + steps * 2.0 ** -22)[..., None] * out
    tol = tol + 2.0 ** -32 * total[:, None] / z[..., None]
    worst = ((s["out"].double().reshape(B, N, G, D) - out).abs() / tol).amax((0, 1, 3))
    assert float(worst.max()) <= 1, worst.tolist()
    # The sum of the weights is fp32: a row adds up to 36 times within a tile, once per tile of its group (every
    # second one: L / 256), and twice at the end, each time rounding by at most 2^-24 of a sum that is no more than z.
    # d ln(z) = dz / z: with the dominant weight first these roundings are alike and add up (2^20: 1.8e-4 of the
    # 2.5e-4 that this allows).
    lse, adds = score + torch.log(z), L // 256 + 40
    assert bool(((s["lse"].double().reshape(B, N, G) - lse).abs() <= ds + 2.0 ** -20 + 2.0 ** -22 * lse + adds * 2.0 ** -24).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("drafts,Hq,Hkv,D,mask", [(9, 8, 2, 128, "tree"), (40, 32, 4, 128, "chain"), (20, 4, 1, 64, "tree")])
def test_every_row_of_v_has_its_weight(dtype, drafts, Hq, Hkv, D, mask):
    """Equal scores, and in each column of each head one row of V that is not zero: every position of a context that
    many CTAs share (page, tile and stretch ends among them) is seen in turn by the rows that see it."""
    L = 20003
    s = make_tree([L], [drafts], Hq, Hkv, D, dtype=dtype, seed=33, mask=mask)
    s["q"].zero_()
    t, col = torch.arange(L, device="cuda"), torch.arange(D, device="cuda")
    page, off = s["bt"][0].long()[t // 16], t % 16
    j = t - (L - drafts)
    i = torch.arange(drafts, device="cuda")
    if mask == "chain":
        vis = j[None] <= i[:, None]
    else:
        jj = j.clamp(min=0)
        vis = (s["mask"].long()[:, jj >> 5] >> (jj & 31) & 1).bool() | (j < 0)
    seen = vis.sum(1).double()
    big, G = 256.0, Hq // Hkv
    vs = 1.0 if dtype == "bf16" else s["v_scale"].double()
    flat = s["v"].view(torch.uint8) if dtype == "fp8" else s["v"]
    one = 0x78 if dtype == "fp8" else big                                   # E4M3 0x78 = 256
    for base in range(0, L, Hkv * D):
        flat.zero_()
        at = base + torch.arange(Hkv, device="cuda")[:, None] * D + col     # [Hkv, D]: the position of that column
        head, c = torch.nonzero(at < L, as_tuple=True)
        p = at[head, c]
        flat[page[p], head, off[p], c] = one
        run_tree(s, ws=s.setdefault("ws", torch.empty(pkv.tree_decode_workspace(
            drafts, Hq, D, torch.cuda.get_device_properties(0).multi_processor_count), dtype=torch.uint8, device="cuda")))
        want = torch.zeros(drafts, Hkv, D, dtype=torch.float64, device="cuda")
        want[:, head, c] = vis[:, p].double() * big / seen[:, None]
        want = (want * (vs if dtype == "bf16" else vs[None, :, None]))[:, :, None].expand(-1, -1, G, -1)
        got = s["out"].double().reshape(drafts, Hkv, G, D)
        # exact weights: half a step of the output, and the roundings of 1 / sum, the scale and the joining
        assert bool(((got - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want).all()), base
    assert int(s["err"].item()) == 0


@pytest.mark.parametrize("per_head", [True, False])
@pytest.mark.parametrize("bad", [float("nan"), -0.03])
def test_k_scales_that_are_no_number_or_negative(bad, per_head):
    """As in the decode step the scale multiplies the scores, whatever it is; rows that see nothing have none."""
    s = make_tree([6, 700, 90], [6, 9, 40], 8, 2, 128, dtype="fp8", seed=34)
    s["mask"][:6] = 0
    x = s["v"].view(torch.uint8)
    t = 700 - 9 + 3                                                         # a drafted token whose V is not finite
    x[s["bt"][1, t // 16].long(), 1, t % 16, 5] = 0x7F
    if per_head:
        s["k_scale"][0] = bad
    else:
        s["k_scale"], s["v_scale"] = torch.tensor([bad], device="cuda"), s["v_scale"][:1].clone()
    run_tree(s)
    check_tree(s)
