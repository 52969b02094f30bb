"""GPU tests of forms of the prompt calls that a serving loop meets beside the
usual ones: rows before the first sequence, other strides, single tokens, many
empty sequences, the outputs as halves of one buffer."""
import pytest
import torch

from tests._prompt import check_prompt, check_read, make_prompt, make_read, run_prompt, run_read

pytestmark = pytest.mark.gpu


def test_lse_of_the_heads_outermost():
    s = make_prompt([300, 77, 2500], [0, 50, 0], 8, 2, 128, seed=1)
    s["lse"] = torch.full((8, 2877), 7.0, device="cuda").T
    run_prompt(s)
    check_prompt(s)


def test_out_of_rows_that_are_not_32_byte_aligned():
    s = make_prompt([300, 77, 1900], [0, 50, 0], 8, 2, 64, seed=2)
    wide = torch.full((2277, 8 * 64 + 8), 7.0, device="cuda", dtype=torch.bfloat16)
    s["out"] = wide[:, 8:].unflatten(1, (8, 64))
    run_prompt(s)
    check_prompt(s)
    assert bool((wide[:, :8] == 7.0).all())


def test_sequences_that_start_behind_other_rows():
    s = make_prompt([200, 30], [100, 0], 8, 2, 128, seed=3)

    def behind(x, n, fill):
        return torch.cat([torch.full((n,) + x.shape[1:], fill, dtype=x.dtype, device="cuda"), x])
    whole = {k: behind(s[k], n, float("nan")) for k, n in (("q", 5), ("k", 9), ("v", 9))}
    out, lse = behind(s["out"], 5, 7.0), behind(s["lse"], 5, 7.0)
    run_prompt(s, **whole, q_start=s["q_start"] + 5, k_start=s["k_start"] + 9, out=out, lse=lse)
    torch.cuda.synchronize()
    assert bool((out[:5] == 7.0).all()) and bool((lse[:5] == 7.0).all())
    s["out"], s["lse"] = out[5:], lse[5:]
    check_prompt(s)


def test_keys_and_values_of_different_strides():
    s = make_prompt([333], [500], 6, 3, 64, seed=4)
    k, v = (torch.randn(833, *x, device="cuda").bfloat16() for x in ((3 * 64 + 24,), (2, 3, 64)))
    k[:, :192], v[:, 1] = s["k"].flatten(1), s["v"]
    s["k"], s["v"] = k[:, :192].unflatten(1, (3, 64)), v[:, 1]
    run_prompt(s)
    check_prompt(s)


@pytest.mark.parametrize("D,G", [(128, 4), (64, 1), (128, 7)])
def test_heads_outermost(D, G):
    s = make_prompt([300, 77, 2500], [0, 50, 0], 2 * G, 2, D, seed=8)
    for x in ("q", "k", "v", "out"):
        s[x] = s[x].transpose(0, 1).contiguous().transpose(0, 1)
    run_prompt(s)
    check_prompt(s)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx", [[100_000], [997 * i % 9000 for i in range(40)]], ids=["one", "forty"])
def test_single_tokens_behind_contexts(D, ctx):
    s = make_prompt([1] * len(ctx), ctx, 32, 4, D, seed=5)
    run_prompt(s)
    check_prompt(s)


def test_most_sequences_empty():
    # One token in every seventh sequence, which sees itself alone: its value, by the weight's and the output's rounding.
    n = [int(i % 7 == 0) for i in range(65_535)]
    s = make_prompt([0], [0], 2, 1, 64)
    g = torch.Generator(device="cuda").manual_seed(7)
    for x, h in (("q", 2), ("k", 1), ("v", 1)):
        s[x] = torch.randn(sum(n), h, 64, generator=g, device="cuda").bfloat16()
    s.update(q_start=torch.cumsum(torch.tensor([0] + n), 0).to(torch.int32).cuda(), k_start=None,
             out=torch.full_like(s["q"], 7.0), lse=torch.full((sum(n), 2), 7.0, device="cuda"))
    run_prompt(s)
    torch.cuda.synchronize()
    assert int(s["err"].item()) == 0
    v = s["v"].float()
    assert bool(((s["out"].float() - v).abs() <= 2.0 ** -7 * v.abs()).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "nvfp4"])
def test_rows_read_back_into_halves_of_one_buffer(dtype):
    s = make_read([100, 1, 0, 333], [0, 7, 3, 100], 4, 128, dtype, seed=6, spare=2)
    both = torch.full((s["k_out"].shape[0], 3, 4, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    s["k_out"], s["v_out"] = both[:, 0], both[:, 2]
    run_read(s)
    check_read(s)
    assert bool((both[:, 1] == 7.0).all())
