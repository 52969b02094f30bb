"""GPU tests of how exactly the drafted-token attention (pkv_paged_tree_decode)
carries its weights, with tolerances that count each rounding of its own, and
of single rows of V at every place of a long context."""
import pytest
import torch

import paged_kv_gqa_04_gb300 as pkv
from tests._spec import make_tree, run_tree

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
