"""GPU tests of the prompts' attention that a single wrong tile of keys does not
pass, however long the row: errors against what independent roundings give
(tests/_prompt_rounding.py), and values that say which tile they are of."""
import pytest
import torch

from tests._prompt import make_prompt, run_prompt
from tests._prompt_rounding import excess, squares, weights

pytestmark = pytest.mark.gpu

CASES = {
    # name: tokens, keys before them, Hq, Hkv, D, rows (None: all)
    "short": ([37, 100, 2, 1], [0, 0, 0, 5], 4, 2, 64, None),
    "tile_ends": ([127, 128, 129, 255, 256, 257, 15, 16, 17], [0] * 9, 8, 2, 128, None),
    "group_1": ([700, 260], [0, 0], 3, 3, 128, None),
    "group_3": ([400, 31], [0, 9], 6, 2, 64, None),
    "group_7": ([500, 90], [0, 0], 28, 4, 128, None),
    "group_16": ([200], [77], 32, 2, 128, None),
    "cut_items": ([3000], [0], 4, 1, 128, range(0, 3000, 7)),
    "cut_long_context": ([9, 70], [20000, 3000], 4, 2, 128, None),
    "mixed": ([1, 1800, 3, 64, 900, 700, 17, 16], [0] * 8, 8, 2, 128, None),
    "long": ([20000], [0], 4, 2, 128, [1, 127, 128, 5000, 9999, 10000, 15001, 19998, 19999]),
    "long_d64": ([20000], [0], 4, 2, 64, [1, 127, 128, 5000, 9999, 10000, 15001, 19998, 19999]),
    "runs_of_keys": ([330 * 16], [140_000], 16, 1, 128, [0, 9, 16, 2500, 2600, 5279]),
    "many_tiles_of_a_cta": ([420_000], [0], 8, 8, 64, [1, 128, 65_537, 131_071, 262_145, 300_001, 419_871, 419_999]),
}


def each_head(s, rows):
    """(sequence, head, rows of q and out, weights, values) of every sequence and head."""
    Hq, Hkv = s["q"].shape[1], s["k"].shape[1]
    for b, (n, L, e) in enumerate(zip(s["n"], s["L"], s["ks"])):
        i = torch.arange(n, device="cuda") if rows is None else torch.tensor([r for r in rows if r < n], device="cuda")
        at = sum(s["n"][:b]) + i
        for h in range(Hq):
            g = h // (Hq // Hkv)
            yield b, h, at, weights(s["q"][at, h], s["k"][e:e + L, g], s["scale"], L - n + 1 + i), s["v"][e:e + L, g].double()


@pytest.mark.parametrize("name", CASES)
def test_errors_are_those_of_independent_roundings(name):
    n, ctx, Hq, Hkv, D, rows = CASES[name]
    s = make_prompt(n, ctx, Hq, Hkv, D, seed=50 + len(name))
    run_prompt(s)
    torch.cuda.synchronize()
    assert int(s["err"].item()) == 0
    for b, h, at, w, v in each_head(s, rows):
        x = excess(s["out"][at, h].double(), w, v, w @ v)
        assert x <= 1, f"sequence {b}, head {h}: {x}"


@pytest.mark.parametrize("name", ["mixed", "cut_long_context", "long", "long_d64", "runs_of_keys", "many_tiles_of_a_cta"])
def test_every_tile_of_values_meets_its_own_weights(name):
    """Values are one in the column of their tile's number (mod D) and zero elsewhere: an output is the weight of every
    D-th tile. Weights are off by 2^-8 each and of one sign, as is the output; sums of runs of up to 2^16 keys by 2^-8."""
    n, ctx, Hq, Hkv, D, rows = CASES[name]
    s = make_prompt(n, ctx, Hq, Hkv, D, seed=70 + len(name))
    for e, L in zip(s["ks"], s["L"]):
        j = torch.arange(L, device="cuda")
        s["v"][e:e + L] = 0.0
        s["v"][e + j, :, j // 128 % D] = 1.0
    run_prompt(s)
    torch.cuda.synchronize()
    assert int(s["err"].item()) == 0
    for b, h, at, w, v in each_head(s, rows):
        o = w @ v
        e, g = s["ks"][b], h // (Hq // Hkv)
        mag = (s["q"][at, h].double().norm(dim=1) * s["k"][e:e + w.shape[1], g].double().norm(dim=1).max())[:, None] * s["scale"]
        # (a score: D + 8 roundings of sum |q k|, which is at most |q| |k|)
        tol = (2 * 2.0 ** -8 * 1.01 + min(w.shape[1], 2 ** 16) * 2.0 ** -24 + 2 * mag * (D + 8) * 2.0 ** -24 + 2.0 ** -19) * o
        tol = tol + 2.0 ** -126
        assert bool(((s["out"][at, h].double() - o).abs() <= tol).all()), f"sequence {b}, head {h}"


@pytest.mark.parametrize("D", [64, 128])
def test_a_row_that_sees_one_key_gives_its_value(D):
    # Its weight is one, to within the exponential's 2^-22, and so is their sum: bf16 holds their quotient, v, as it is.
    s = make_prompt([1, 5, 40, 700, 1], [0] * 5, 8, 2, D, seed=90)
    run_prompt(s)
    torch.cuda.synchronize()
    for at in (0, 1, 6, 46, 746):
        assert torch.equal(s["out"][at], s["v"][at].repeat_interleave(4, 0))


@pytest.mark.parametrize("q_mult", [1.0, 8.0])
@pytest.mark.parametrize("D", [64, 128])
def test_the_largest_weight_of_a_short_row_is_exact(D, q_mult):
    """Rows of up to a tile of keys: as errors of independent roundings, without one of the largest weight."""
    s = make_prompt([1, 2, 3, 17, 60, 127, 128], [0, 5, 0, 100, 0, 1, 0], 8, 2, D, seed=91, q_mult=q_mult)
    run_prompt(s)
    torch.cuda.synchronize()
    for b, h, at, w, v in each_head(s, None):
        o = w @ v
        others = w.scatter(1, w.argmax(1, keepdim=True), 0.0)
        # (fp32: the exponentials' 2^-20 and the scores' roundings, far below 2^-16 of w |v| each)
        small = 2.0 ** -32 * (w ** 2) @ (v ** 2).sum(1)
        err = ((s["out"][at, h].double() - o) ** 2).sum(1)
        assert bool((err <= 4 * (squares(others, v, o) + small)).all()), f"sequence {b}, head {h}"
