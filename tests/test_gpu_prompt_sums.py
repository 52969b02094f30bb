"""The prompts' attention's sums over more keys than the tensor cores add up in
one go (runs of 2^16): their size where all terms are of one sign, and what is
carried from one run of keys to the next."""
import pytest
import torch

from tests._prompt import make_prompt, run_prompt

pytestmark = pytest.mark.gpu

RUN = 2 ** 16  # keys
ROWS = [0, 1, 7, 8, 15, 16, 1000, 1777, 2446, 2447]


def check(s, rows, weights=2.0 ** -8):
    """Against float64, for one sequence and one kv head.

    A run adds up to 2^16 products, each cut off or rounded by at most 2^-23 of the sum so far, which is half of the
    run's in the mean (2^-8 of it), and rounds once for every 16 (2^-12). Runs are joined by one multiply-add each.
    Weights: `weights` each for their rounding (nothing where they are whole), 2^-20 for the exponential and its
    reference, and the scores' D + 8 roundings. Output: 2^-8 of itself. What fp32 and bf16 hold no normal number for may
    be zero: 2^-126 (with a step of 40 the answers are about 2^-165)."""
    torch.cuda.synchronize()
    assert int(s["err"].item()) == 0
    D, L, n, G = s["D"], s["L"][0], s["n"][0], s["q"].shape[1]
    k, v = s["k"][:L, 0].double(), s["v"][:L, 0].double()
    odd = ~torch.isfinite(v).all(1)
    for r in rows:
        vis = L - n + r + 1
        q = s["q"][r].double()
        x = q @ k[:vis].T * s["scale"]
        mag = (q.abs() @ k[:vis].abs().T * abs(s["scale"])).nan_to_num(0.0, 0.0, 0.0).amax(1)[:, None]
        w = torch.softmax(x, 1)
        o, av = w @ torch.where(odd[:, None], 0.0, v)[:vis], w @ torch.where(odd[:, None], 0.0, v.abs())[:vis]
        for j in odd[:vis].nonzero()[:, 0].tolist():
            o += w[:, j, None] * v[j]
        ds = mag * (D + 8) * 2.0 ** -24
        tol = 2.0 ** -8 * o.abs() + (weights + 2 * ds + 2.0 ** -20 + 2.0 ** -8 + 2.0 ** -12 + (L // RUN + 8) * 2.0 ** -24) * 1.01 * av
        tol = tol + 2.0 ** -126
        got = s["out"][r].double()
        assert torch.equal(torch.isnan(got), torch.isnan(o)) and torch.equal(got[torch.isinf(o)], o[torch.isinf(o)])
        fine = torch.isfinite(o)
        err = (got - o).abs()
        assert bool((err <= tol)[fine].all()), f"row {r}: {float((err / av)[fine].max())} of the sum of magnitudes"
        lse = torch.logsumexp(x, 1)
        # (a sum of L weights of one sign, rounded to nearest 64 at a time)
        tol_l = ds[:, 0] + 2.0 ** -20 + (L // 64 + 64) * 2.0 ** -24 + 2.0 ** -22 * lse.abs()
        assert bool(((s["lse"][r].double() - lse).abs() <= tol_l).all())


@pytest.mark.parametrize("D", [64, 128])
def test_a_sum_of_one_sign_over_many_keys(D):
    # 4 Mi keys with the same weight, values of about one: cut off product by product, their sum is 2.3% short
    s = make_prompt([153 * 16], [2 ** 22], 16, 1, D, seed=41)
    s["k"].zero_()
    s["v"].copy_((1 + 0.1 * s["v"].float()).bfloat16())
    run_prompt(s)
    check(s, ROWS[::3], weights=0.0)


@pytest.mark.parametrize("D,pairs,step", [(64, 153, 0.0), (128, 153, 0.0), (128, 330, 5.0), (64, 330, 5.0), (128, 330, -5.0),
                                          (128, 153, 20.0), (64, 153, 40.0)])
def test_what_runs_of_keys_add_up_to(D, pairs, step):
    """The runs' scores differ by `step`, and their values the other way by as much: all count the same."""
    ctx = 3 * RUN + 777
    s = make_prompt([pairs * 16], [ctx], 16, 1, D, seed=42 + pairs)
    at = torch.arange(s["k"].shape[0], device="cuda") // RUN
    s["scale"] = 1.0
    s["q"].mul_(0.1)
    s["q"][..., 0] = 1.0
    s["k"][:, 0, 0] = (step * at).bfloat16()
    by = torch.tensor([1.0, 3.0, -2.0, 5.0], device="cuda") * (2.0 ** round(-1.44 * step)) ** torch.arange(4, device="cuda")
    s["v"].copy_((by[at][:, None, None] * (1 + 0.2 * s["v"].float())).bfloat16())
    run_prompt(s)
    check(s, [r for r in ROWS if r < s["n"][0]])


@pytest.mark.parametrize("D", [64, 128])
def test_a_first_run_without_weight_and_values_that_are_not_finite(D):
    s = make_prompt([153 * 16], [2 * RUN + 300], 16, 1, D, seed=43)
    s["scale"] = 1.0
    s["q"].mul_(0.1)
    s["q"][..., 0], s["k"][..., 0] = 1.0, 0.0
    s["k"][:RUN + 200, :, 0] = -float("inf")
    run_prompt(s)
    check(s, ROWS[::2])
    s["k"][..., 0] = 0.0
    s["v"][300, 0, 3], s["v"][RUN + 3, 0, 5], s["v"][2 * RUN + 9, 0, 7] = float("nan"), float("inf"), -float("inf")
    s["v"][400, 0, 9], s["v"][RUN + 400, 0, 9] = float("inf"), -float("inf")
    run_prompt(s)
    check(s, ROWS[::2])
