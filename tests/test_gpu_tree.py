"""GPU tests of the drafted-token attention (pkv_paged_tree_decode) against a
float64 statement of it, with tolerances that count its roundings."""
import pytest
import torch

import paged_kv_gqa_04_gb300 as pkv
from paged_kv_gqa_04_gb300 import _abi
from tests._spec import check_tree, make_tree, run_tree

pytestmark = pytest.mark.gpu

CASES = {
    # name: lens, drafts, Hq, Hkv, D, more
    "one_token": ([1], [1], 1, 1, 128, {}),
    "short": ([37, 100], [5, 8], 4, 2, 64, {}),
    "no_context": ([8, 33, 1], [8, 33, 1], 8, 2, 128, {}),
    "page_ends": ([16, 17, 128, 129, 127, 256], [1, 2, 3, 16, 15, 1], 8, 4, 128, {}),
    "no_drafts_between": ([300, 40, 500], [0, 3, 0], 8, 4, 128, dict(spare_rows=5)),
    "group_1": ([700, 260], [9, 31], 3, 3, 128, {}),
    "group_3": ([700, 260], [9, 31], 6, 2, 64, {}),
    "group_7": ([1500, 90], [17, 20], 28, 4, 128, {}),
    "group_16": ([400], [9], 32, 2, 128, {}),
    "group_16_d64": ([333, 65], [40, 7], 16, 1, 64, {}),
    "two_tiles": ([2000, 777], [64, 33], 32, 8, 128, {}),
    "three_words": ([1000, 130], [70, 96], 4, 2, 128, dict(mask="random")),
    "five_tiles": ([900], [150], 8, 2, 128, {}),
    "chain": ([600, 5, 1024, 77], [4, 5, 1, 30], 12, 2, 128, dict(mask="chain")),
    "chain_chunk": ([1300, 450], [300, 450], 8, 4, 128, dict(mask="chain")),
    "chain_d64": ([1300, 450], [30, 200], 8, 8, 64, dict(mask="chain")),
    "random_bits": ([300, 60, 129], [20, 31, 1], 8, 2, 128, dict(mask="random")),
    "long": ([20000], [12], 28, 4, 128, {}),
    "mixed": ([1, 8000, 3, 64, 2500, 700, 17, 16], [1, 9, 3, 16, 32, 1, 2, 5], 32, 8, 128, dict(layout="NHD")),
    "large_scores": ([900, 333], [9, 16], 8, 2, 128, dict(k_mult=30.0)),
    "interleaved_pools": ([300, 260], [9, 16], 8, 4, 128, dict(pool_strides=True)),
    "fp8": ([3000, 129, 16], [24, 5, 16], 12, 2, 128, dict(dtype="fp8")),
    "fp8_nhd": ([700, 31], [30, 31], 32, 8, 128, dict(dtype="fp8", layout="NHD")),
    "fp8_d64": ([700, 2100], [64, 9], 16, 2, 64, dict(dtype="fp8", mask="random")),
    "fp8_chain": ([520], [200], 8, 2, 128, dict(dtype="fp8", mask="chain")),
    "many": ([(37 * i) % 400 + 33 for i in range(150)], [i % 9 for i in range(150)], 4, 2, 128, {}),
}


@pytest.mark.parametrize("name", CASES)
def test_against_float64(name):
    lens, drafts, Hq, Hkv, D, more = CASES[name]
    s = make_tree(lens, drafts, Hq, Hkv, D, seed=len(name), **more)
    run_tree(s)
    check_tree(s)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_same_bits_again_and_with_bound_buffers(dtype):
    s = make_tree([5000, 300], [20, 9], 16, 4, 128, dtype=dtype, seed=5)
    run_tree(s)
    first, lse = s["out"].clone(), s["lse"].clone()
    bound = {k: pkv.bind(v) for k, v in s.items() if v is None or isinstance(v, torch.Tensor)}
    run_tree(s, **{k: v for k, v in bound.items() if k != "q"})
    torch.cuda.synchronize()
    assert torch.equal(first, s["out"]) and torch.equal(lse, s["lse"])


def test_one_draft_agrees_with_the_decode_step():
    s = make_tree([300, 17, 2000], [1, 1, 1], 8, 2, 128, seed=3, mask="chain")
    run_tree(s)
    op, lp = torch.empty(3, 4, 8, 128, device="cuda"), torch.empty(3, 4, 8, device="cuda")
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    pkv.paged_gqa_decode(s["q"], s["k"], s["v"], s["bt"], s["seq_lens"], s["scale"], 4, op, lp)
    pkv.lse_merge(op, lp, out, lse)
    check_tree(s)
    check_tree(dict(s, out=out, lse=lse))


def test_lse_is_optional_and_rows_may_be_strided():
    s = make_tree([300, 90], [9, 16], 8, 2, 128, seed=4)
    qkv = torch.zeros((25, 12, 128), dtype=torch.bfloat16, device="cuda")
    qkv[:, 2:10] = s["q"]
    wide = torch.full((25, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    mask = torch.zeros((25, 3), dtype=torch.int32, device="cuda")
    mask[:, :1] = s["mask"]
    run_tree(s, q=qkv[:, 2:10], lse=None, out=wide[:, 4:12], mask=mask[:, :1])
    run_tree(s)
    check_tree(s)
    assert torch.equal(wide[:, 4:12], s["out"]) and bool((wide[:, :4] == 7).all()) and bool((wide[:, 12:] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("what", ["k", "v"])
def test_nan_in_places_that_no_row_sees(dtype, what):
    """Behind the sequence, in the last page, and in pages of no sequence."""
    s = make_tree([37, 129, 16], [5, 3, 2], 8, 2, 128, dtype=dtype, seed=6)
    x = s[what].view(torch.uint8) if dtype == "fp8" else s[what]
    bad = 0x7F if dtype == "fp8" else float("nan")
    used = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
    used[s["bt"][s["bt"] >= 0].long()] = True
    x[~used] = bad
    for b, L in enumerate([37, 129, 16]):
        if L % 16:
            x[s["bt"][b, L // 16].long(), :, L % 16:] = bad
    run_tree(s)
    check_tree(s)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("what", ["k", "v"])
def test_nan_and_infinity_in_masked_drafts(dtype, value, what):
    """A drafted token that is not finite reaches the rows that see it and no other."""
    if dtype == "fp8" and value == "inf":
        pytest.skip("E4M3 has no infinity")
    lens, drafts = [300, 40, 200], [9, 12, 40]
    s = make_tree(lens, drafts, 8, 2, 128, dtype=dtype, seed=7)
    x = s[what].view(torch.uint8) if dtype == "fp8" else s[what]
    for b, j in ((0, 4), (2, 0), (2, 33), (1, 11)):
        t = lens[b] - drafts[b] + j
        x[s["bt"][b, t // 16].long(), 1, t % 16, 17::50] = 0x7F if dtype == "fp8" else float(value)
    run_tree(s)
    check_tree(s)
    assert bool(torch.isfinite(s["out"][:, :4]).all())   # kv head 0 has none of it


def test_rows_that_see_nothing():
    s = make_tree([6, 300, 4], [6, 4, 4], 8, 2, 128, seed=8)
    s["mask"].zero_()
    run_tree(s)
    check_tree(s)
    assert bool((s["out"][:6] == 0).all()) and bool((s["lse"][10:] == -float("inf")).all())


def test_bad_values_are_flagged_and_left_out():
    s = make_tree([48, 70, 300], [3, 4, 5], 8, 2, 128, seed=9)
    s["bt"][0, 1] = s["k"].shape[0] + 1000
    s["bt"][2, 0] = -5
    run_tree(s)
    check_tree(s, flags=_abi.FLAG_PAGE_RANGE)
    s = make_tree([48, 70, 300], [3, 4, 5], 8, 2, 128, seed=9)
    s["seq_lens"][2] = 10 ** 6
    run_tree(s)
    check_tree(s, flags=_abi.FLAG_SEQ_LEN_RANGE)
    s["err"].zero_()
    s["seq_lens"][2] = -3         # clamped to 0: its five drafted tokens do not exist
    run_tree(s)
    check_tree(s, flags=_abi.FLAG_SEQ_LEN_RANGE | _abi.FLAG_DRAFT_RANGE)
    s = make_tree([48, 70, 3], [3, 4, 5], 8, 2, 128, seed=9)   # five drafted tokens, three in the cache
    run_tree(s)
    check_tree(s, flags=_abi.FLAG_DRAFT_RANGE)
    s = make_tree([48, 170], [3, 40], 8, 2, 128, seed=9)
    s["mask"] = s["mask"][:, :1].contiguous()                 # drafted tokens 32.. are behind the mask
    run_tree(s)
    check_tree(s, flags=_abi.FLAG_DRAFT_RANGE)


@pytest.mark.parametrize("start", [[0, 5, 99], [-4, 5, 12], [0, 12, 12]])
def test_row_ranges_are_clamped(start):
    s = make_tree([48, 70], [5, 7], 8, 2, 128, seed=10)
    s["q_start"].copy_(torch.tensor(start))
    run_tree(s)
    bad = any(not 0 <= x <= 12 for x in start)
    check_tree(s, flags=_abi.FLAG_DRAFT_RANGE if bad else 0)


def test_overlapping_ranges_past_the_work_that_is_counted():
    """32,768 sequences of 2^18 drafted tokens each, in the same rows of q: 3.2e9 tiles of work."""
    if torch.cuda.get_device_properties(0).total_memory < 40e9:
        pytest.skip("needs 1.5 GB")
    B, T = 65535, 1 << 18
    s = make_tree([300], [9], 16, 1, 64, seed=11)
    start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    start[1::2] = T
    s.update(q=torch.zeros((T, 16, 64), dtype=torch.bfloat16, device="cuda"), q_start=start, lse=None,
             seq_lens=torch.full((B,), 300, dtype=torch.int32, device="cuda"), bt=s["bt"].repeat(B, 1),
             mask=torch.zeros((T, 1), dtype=torch.int32, device="cuda"))
    s["out"] = torch.full_like(s["q"], 7.0)
    run_tree(s)
    torch.cuda.synchronize()
    assert int(s["err"].item()) == _abi.FLAG_DRAFT_RANGE and bool((s["out"] == 7).all())


def test_pool_past_32_bit_offsets():
    """Pages whose element and byte offsets pass 2^31 and 2^32."""
    if torch.cuda.get_device_properties(0).total_memory < 40e9:
        pytest.skip("needs a pool of 9 GB")
    s = make_tree([700, 200], [9, 16], 8, 8, 128, seed=11, num_pages=140000, layout="NHD")
    s["bt"][0, :44] = torch.arange(139000, 139044, dtype=torch.int32)
    run_tree(s)
    check_tree(s)


def test_captured_and_replayed_with_other_lengths():
    s = make_tree([700, 3000, 90], [9, 16, 4], 16, 4, 128, seed=12)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws = torch.empty(pkv.tree_decode_workspace(29, 16, 128, sms), dtype=torch.uint8, device="cuda")
    run_tree(s, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        run_tree(s, ws=ws)
    for lens in ([700, 3000, 90], [9, 16, 4], [500, 40, 89], [696, 2999, 4]):
        s["seq_lens"].copy_(torch.tensor(lens))
        g.replay()
        check_tree(s)


def test_two_streams_at_once():
    a, b = make_tree([3000, 800], [20, 9], 16, 4, 128, seed=13), make_tree([5000], [31], 8, 2, 64, seed=14)
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for x, stream in zip((a, b), st):
            run_tree(x, stream=stream, ws=x.setdefault("ws", torch.empty(pkv.tree_decode_workspace(
                x["q"].shape[0], x["q"].shape[1], x["D"], 152), dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    check_tree(a)
    check_tree(b)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("scale", [-0.11, 0.0])
def test_negative_and_zero_scales(dtype, scale):
    s = make_tree([700, 90], [9, 40], 8, 2, 128, dtype=dtype, seed=15)
    s["scale"] = scale
    run_tree(s)
    check_tree(s)
