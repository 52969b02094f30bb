"""GPU tests of the prompts' attention (pkv_prompt_attention) against a float64
statement of it, with tolerances that count its roundings."""
import pytest
import torch

import paged_kv_gqa_04_gb300 as pkv
from paged_kv_gqa_04_gb300 import _abi
from tests._prompt import check_prompt, make_prompt, prompt_reference, run_prompt, workspace

pytestmark = pytest.mark.gpu

CASES = {
    # name: tokens, keys before them, Hq, Hkv, D, more
    "one_token": ([1], [0], 1, 1, 128, {}),
    "short": ([37, 100], [0, 0], 4, 2, 64, {}),
    "tile_ends": ([127, 128, 129, 255, 256, 257, 15, 16, 17], [0] * 9, 8, 2, 128, {}),
    "empty_between": ([0, 40, 0, 0, 300, 0], [0] * 6, 8, 4, 128, dict(spare=5)),
    "fused": ([60, 200, 1], [0] * 3, 8, 2, 128, dict(fused=True, spare=3)),
    "fused_d64": ([333, 65], [0] * 2, 6, 2, 64, dict(fused=True)),
    "group_1": ([700, 260], [0, 0], 3, 3, 128, {}),
    "group_1_d64": ([300, 513], [0, 0], 2, 2, 64, {}),
    "group_3": ([400, 31], [0, 9], 6, 2, 64, {}),
    "group_5": ([90, 311], [0, 0], 10, 2, 128, {}),
    "group_6": ([256, 77], [0, 1000], 12, 2, 128, {}),
    "group_7": ([500, 90], [0, 0], 28, 4, 128, {}),
    "group_12": ([140], [0], 12, 1, 128, {}),
    "group_16": ([200], [77], 32, 2, 128, {}),
    "group_16_d64": ([133, 65], [0, 7], 16, 1, 64, {}),
    "context": ([64, 1, 30, 129], [1000, 127, 128, 3], 8, 2, 128, dict(spare=7)),
    "context_gaps": ([64, 5, 30], [100, 0, 77], 8, 2, 128, dict(k_gap=9)),
    "cut_items": ([3000], [0], 4, 1, 128, {}),
    "cut_long_context": ([9, 70], [20000, 3000], 4, 2, 128, {}),
    "cut_d64": ([2500, 100], [0, 4000], 8, 4, 64, {}),
    "mixed": ([1, 1800, 3, 64, 900, 700, 17, 16], [0] * 8, 8, 2, 128, {}),
    "large_scores": ([900, 333], [0, 16], 8, 2, 128, dict(q_mult=30.0)),
    "negative_scale": ([300], [50], 4, 2, 128, dict(scale=-0.1)),
    "zero_scale": ([200], [0], 4, 2, 64, dict(scale=0.0)),
    "many": ([(37 * i) % 150 for i in range(150)], [(11 * i) % 90 for i in range(150)], 4, 2, 128, {}),
}


@pytest.mark.parametrize("name", CASES)
def test_against_float64(name):
    n, ctx, Hq, Hkv, D, more = CASES[name]
    s = make_prompt(n, ctx, Hq, Hkv, D, seed=len(name), **more)
    run_prompt(s)
    check_prompt(s)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("step", [0.2, 3.0, 300.0])
def test_scores_that_rise_along_the_keys(D, step):
    """Every tile's maximum is above the one before: the reference moves, by little and by more than 2^127."""
    s = make_prompt([700], [300], 4, 2, D, seed=3)
    up = torch.arange(1000, device="cuda").float() * step / 16
    s["k"][:1000] = (s["k"][:1000].float() * 0.05)
    s["q"][..., 0] = 16.0
    s["k"][:1000, :, 0] = up[:, None].bfloat16()
    s["scale"] = 1.0
    run_prompt(s)
    check_prompt(s)


@pytest.mark.parametrize("step", [-0.3, -40.0])
def test_scores_that_fall_along_the_keys(step):
    s = make_prompt([600], [0], 4, 2, 128, seed=4)
    s["q"][..., 0] = 1.0
    s["k"][..., 0] = (torch.arange(600, device="cuda").float() * step)[:, None].bfloat16()
    s["scale"] = 1.0
    run_prompt(s)
    check_prompt(s)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(D, value):
    s = make_prompt([200, 70, 300], [0, 3, 500], 8, 2, D, seed=6)
    for b, j in ((0, 100), (0, 131), (1, 71), (2, 700), (2, 799)):
        s["v"][s["ks"][b] + j, 1, j % D] = value
        s["v"][s["ks"][b] + j, 0, 5] = value
    run_prompt(s)
    check_prompt(s)
    assert not torch.isfinite(s["out"][150].float()).all() and torch.isfinite(s["out"][:100].float()).all()


def test_keys_that_are_not_finite_reach_only_rows_that_see_them():
    s = make_prompt([300, 40], [0, 0], 4, 2, 128, seed=7)
    s["k"][150, 0, 3] = float("nan")
    s["k"][320, 1, 3] = float("nan")
    run_prompt(s)
    torch.cuda.synchronize()
    got = torch.isfinite(s["out"].float()).all(2)
    want = torch.ones_like(got)
    want[150:300, :2] = False
    want[320:340, 2:] = False
    assert torch.equal(got, want)


@pytest.mark.parametrize("inf", [float("inf"), -float("inf")])
def test_infinite_scores(inf):
    """A score of -inf is a weight of zero, wherever it stands; one of +inf makes the row NaN, as its formula says."""
    s = make_prompt([300], [0], 2, 1, 128, seed=8)
    s["q"][..., 0], s["k"][..., 0] = 1.0, 0.0
    s["k"][0, 0, 0] = inf
    s["k"][200, 0, 0] = inf
    run_prompt(s)
    if inf < 0:
        # (row 0 sees nothing but a score of -inf: its weights are 0 / 0 by the formula, nothing here)
        s["out"][0], s["lse"][0] = 7.0, 7.0
        torch.cuda.synchronize()
        ref = prompt_reference(s, 0, list(range(1, 300)))
        assert bool(((s["out"][1:].double() - ref[0]).abs() <= ref[2]).all())
        assert bool(((s["lse"][1:].double() - ref[1]).abs() <= ref[3]).all())
    else:
        torch.cuda.synchronize()
        assert torch.isnan(s["out"]).all() and int(s["err"].item()) == 0


def test_the_same_bits_again_and_with_bound_buffers():
    s = make_prompt([2000, 300], [500, 0], 8, 2, 128, seed=5)
    run_prompt(s)
    first, lse = s["out"].clone(), s["lse"].clone()
    bound = {k: pkv.bind(v) for k, v in s.items() if v is None or isinstance(v, torch.Tensor)}
    pkv.prompt_attention(bound["q"], bound["k"], bound["v"], bound["q_start"], bound["k_start"], s["scale"], bound["out"],
                         bound["lse"], pkv.bind(workspace(128)), err_flag=bound["err"])
    torch.cuda.synchronize()
    assert torch.equal(first, s["out"]) and torch.equal(lse, s["lse"])


def test_without_lse_and_into_strided_rows():
    s = make_prompt([257, 12], [0, 40], 8, 2, 64, seed=9)
    run_prompt(s)
    wide = torch.full((s["out"].shape[0], 11, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    run_prompt(s, out=wide[:, 2:10], lse=None)
    torch.cuda.synchronize()
    assert torch.equal(wide[:, 2:10], s["out"]) and bool((wide[:, :2] == 7.0).all()) and bool((wide[:, 10:] == 7.0).all())


def test_captured_and_replayed_while_the_lengths_change():
    s = make_prompt([300, 100, 57], [0, 0, 0], 8, 2, 128, seed=10, fused=True, spare=2)
    ws = workspace(128)
    run_prompt(s, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            run_prompt(s, ws=ws)
    torch.cuda.synchronize()
    for n in ([300, 100, 57], [1, 400, 50], [0, 0, 457], [457, 0, 0]):
        s["n"], s["L"], s["ks"] = n, n, [0, n[0], n[0] + n[1]]
        s["q_start"].copy_(torch.tensor([0, n[0], n[0] + n[1], sum(n)], dtype=torch.int32))
        s["out"].fill_(7.0), s["lse"].fill_(7.0)
        graph.replay()
        check_prompt(s)


def test_ranges_that_contradict_the_rows_are_flagged():
    s = make_prompt([50, 60], [0, 0], 4, 2, 128, seed=11, fused=True)
    for start in ([0, 70, 30], [-5, 20, 110], [0, 50, 200], [2 ** 31 - 1, -2 ** 31, 5]):
        s["q_start"].copy_(torch.tensor(start))
        s["err"].zero_()
        run_prompt(s)
        torch.cuda.synchronize()
        assert int(s["err"].item()) == _abi.FLAG_ROW_RANGE
    # fewer keys than tokens: the first rows see nothing
    s = make_prompt([200, 30], [0, 0], 4, 2, 128, seed=12)
    s["k_start"].copy_(torch.tensor([0, 150, 160]))
    s["L"], s["ks"] = [150, 10], [0, 150]
    run_prompt(s)
    check_prompt(s, flags=_abi.FLAG_ROW_RANGE)
    assert bool((s["out"][:50] == 0).all()) and bool((s["lse"][:50] == -float("inf")).all())
    # no keys at all
    s["k_start"].zero_(), s["err"].zero_()
    s["L"], s["ks"] = [0, 0], [0, 0]
    run_prompt(s)
    check_prompt(s, flags=_abi.FLAG_ROW_RANGE)


def test_two_calls_at_once():
    """Two streams, each with its workspace."""
    a, b = make_prompt([1500], [0], 8, 2, 128, seed=13), make_prompt([700, 9], [2000, 0], 4, 1, 64, seed=14)
    run_prompt(a), run_prompt(b)
    torch.cuda.synchronize()
    want = [x[k].clone() for x in (a, b) for k in ("out", "lse")]
    streams, ws = [torch.cuda.Stream() for _ in range(2)], [workspace(128), workspace(64)]
    for x in (a, b):
        x["out"].fill_(7.0), x["lse"].fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(5):
        for x, st, w in zip((a, b), streams, ws):
            run_prompt(x, ws=w, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, [x[k] for x in (a, b) for k in ("out", "lse")]))
    assert int(a["err"].item()) == int(b["err"].item()) == 0


def test_long_prompt():
    s = make_prompt([20000], [0], 4, 2, 128, seed=15)
    run_prompt(s)
    check_prompt(s, rows=[0, 1, 127, 128, 5000, 9999, 10000, 15001, 19998, 19999])


def test_more_tiles_of_a_cta_than_sixteen_bits_count():
    # 21.6 million tiles: 134,726 a CTA on 160 of them
    n, H, D = 420_000, 8, 64
    s = make_prompt([n], [0], H, H, D, seed=31)
    run_prompt(s)
    check_prompt(s, rows=[0, 1, 127, 128, 65_537, 131_071, 262_145, 300_001, n - 129, n - 1])


def test_more_items_of_a_cta_than_sixteen_bits_count():
    # One token a sequence, which sees itself alone: its value is the answer. 12 million items.
    B, H, D = 60_000, 200, 64
    s = make_prompt([0], [0], H, H, D)
    g = torch.Generator(device="cuda").manual_seed(32)
    for x in ("q", "k", "v"):
        s[x] = torch.randn(B, H, D, generator=g, device="cuda", dtype=torch.bfloat16)
    s.update(q_start=torch.arange(B + 1, dtype=torch.int32, device="cuda"), k_start=None,
             out=torch.full_like(s["q"], 7.0), lse=torch.full((B, H), 7.0, device="cuda"))
    run_prompt(s)
    torch.cuda.synchronize()
    assert int(s["err"].item()) == 0
    # The weight w is one bf16, l its fp32: w v / l and the output's rounding are at most 2^-8 of v each.
    v = s["v"].float()
    assert bool(((s["out"].float() - v).abs() <= 2.0 ** -7 * v.abs()).all())
    x = (s["q"].float() * s["k"].float()).sum(-1) * s["scale"]
    mag = (s["q"].float() * s["k"].float()).abs().sum(-1) * s["scale"]
    assert bool(((s["lse"] - x).abs() <= (2 * D + 16) * 2.0 ** -24 * mag + 2.0 ** -20 + 2.0 ** -22 * x.abs()).all())


def test_workspace_refusals():
    s = make_prompt([5], [0], 2, 1, 64)
    need = workspace(64).numel()
    big = torch.zeros(need + 64, dtype=torch.uint8, device="cuda")
    for ws, status in ((None, _abi.PKV_ERR_INVALID_ARG), (big[:need - 1], _abi.PKV_ERR_INVALID_ARG),
                       (big[8:], _abi.PKV_ERR_UNSUPPORTED)):
        with pytest.raises(pkv.PkvError) as e:
            run_prompt(s, ws=ws)
        assert e.value.status == status
    assert bool((s["out"] == 7.0).all())


@pytest.mark.parametrize("D", [64, 128])
def test_more_tokens_than_keys_in_a_long_sequence(D):
    # flagged; the first 1600 rows see nothing, the others what they should, in items that are cut
    s = make_prompt([2500], [0], 4, 2, D, seed=33)
    s["k"], s["v"], s["L"] = s["k"][:900], s["v"][:900], [900]
    s["k_start"] = torch.tensor([0, 900], dtype=torch.int32, device="cuda")
    run_prompt(s)
    check_prompt(s, flags=pkv.FLAG_ROW_RANGE)
