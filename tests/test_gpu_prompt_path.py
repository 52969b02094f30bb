"""GPU tests of the normed cache write and of the rows read back (pkv_qk_norm_rope_kv_write,
pkv_gather_kv), and of a prompt's path through both and its attention."""
import pytest
import torch

import paged_kv_gqa_04_gb300 as pkv
from paged_kv_gqa_04_gb300 import _abi
from tests._prompt import (check_prompt, check_read, check_write, make_read, make_write, prompt_reference, read_reference,
                           run_prompt, run_read, run_write, workspace)

pytestmark = pytest.mark.gpu


def _before(s):
    return {x: s[x].clone() for x in ("q", "k", "v")}


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("style", ["neox", "interleaved"])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 6, 6), (128, 7, 1)])
def test_write_against_float64(dtype, layout, style, D, Hq, Hkv):
    s = make_write(57, Hq, Hkv, D, dtype, layout, style, weight="bf16" if Hkv == 2 else "f32", seed=D + Hq,
                   skip=(0, 13, 56), packed=Hkv != 6)
    b = _before(s)
    run_write(s)
    check_write(s, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("T", [1, 2, 5000, 9001])
def test_write_of_one_token_and_of_many(dtype, T):
    """Many: several heads a thread, with heads that do not divide."""
    s = make_write(T, 30 if T == 9001 else 32, 6 if T == 9001 else 8, 128, dtype, "NHD", seed=T, skip=(T // 2,) if T > 2 else ())
    b = _before(s)
    run_write(s)
    check_write(s, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("style", ["neox", "interleaved"])
@pytest.mark.parametrize("D,T", [(128, 33), (64, 33), (128, 9000)])
def test_write_is_the_plain_write_where_the_norm_is_exact(dtype, layout, style, D, T):
    """Rows of +-1 have a mean square of 1, so y = x w exactly, and w is a bf16 value: bit for bit what
    rope_kv_write makes of x w."""
    s = make_write(T, 16, 4, D, dtype, layout, style, seed=3, signs=True, weight="bf16" if D == 64 else "f32")
    q, k = (s[x] * s[x + "_weight"].bfloat16() for x in ("q", "k"))
    assert torch.equal(q.float(), s["q"].float() * s["q_weight"].float())
    want = {x: s[x].clone() for x in ("k_cache", "v_cache", "k_bs", "v_bs") if s[x] is not None}
    rest = (s["positions"], s["cos_sin"])
    if dtype == "nvfp4":
        pkv.rope_kv_write_nvfp4(q, k, s["v"], *rest, want["k_cache"], want["v_cache"], want["k_bs"], want["v_bs"], s["slots"],
                                s["k_scale"], s["v_scale"], layout=layout, rope_style=style)
    else:
        pkv.rope_kv_write(q, k, s["v"], *rest, want["k_cache"], want["v_cache"], s["slots"], s["k_scale"], s["v_scale"],
                          layout=layout, rope_style=style)
    plain = {x: torch.zeros((s["pool"], s["P"], 4, D), dtype=torch.bfloat16, device="cuda") for x in ("k", "v")}
    pkv.rope_kv_write(None, k, s["v"], *rest, plain["k"], plain["v"], s["slots"], layout="NHD", rope_style=style)
    run_write(s)
    torch.cuda.synchronize()
    assert torch.equal(s["q"], q) and all(torch.equal(s[x], y) for x, y in want.items())
    assert torch.equal(s["k_out"], plain["k"].flatten(0, 1)[s["slots"].long()])


@pytest.mark.parametrize("P", [1, 7, 64])
def test_write_into_pages_of_any_size(P):
    s = make_write(40, 4, 2, 64, "fp8", "HND", P=P, seed=P)
    b = _before(s)
    run_write(s)
    check_write(s, b)


def test_write_of_keys_in_place_and_without_q():
    s = make_write(50, 8, 2, 128, seed=4)
    b = _before(s)
    apart = {x: s[x].clone() for x in ("k_cache", "v_cache")}
    run_write(s)
    t = make_write(50, 8, 2, 128, seed=4)
    run_write(t, q=None, q_weight=None, k_out=t["k"])
    torch.cuda.synchronize()
    assert torch.equal(t["k"], s["k_out"]) and torch.equal(t["q"], b["q"]) and torch.equal(t["v"], b["v"])
    assert torch.equal(t["k_cache"], s["k_cache"]) and torch.equal(t["v_cache"], s["v_cache"])
    assert not torch.equal(apart["k_cache"], s["k_cache"])


def test_write_with_bad_slots_and_positions():
    s = make_write(20, 4, 2, 128, seed=5)
    s["slots"][3] = s["pool"] * 16
    s["positions"][7] = -1
    s["positions"][8] = 3000
    b = _before(s)
    run_write(s)
    check_write(s, b, flags=_abi.FLAG_SLOT_RANGE | _abi.FLAG_POSITION_RANGE)


def test_write_of_large_and_small_rows():
    """Rows of 2^60 and of 2^-60 have the same norm as others, but for eps; a row of zeros stays one."""
    s = make_write(9, 2, 2, 64, seed=6, packed=False)
    for x in ("q", "k"):
        s[x][0] *= 2.0 ** 60
        s[x][1] *= 2.0 ** -60
        s[x][2] = 0
    b = _before(s)
    run_write(s)
    check_write(s, b)
    assert bool((s["k_out"][2] == 0).all()) and float(s["q"][0].float().abs().max()) < 100


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("D,Hkv", [(128, 8), (64, 3), (128, 1), (64, 20)])
def test_read_bit_for_bit(dtype, layout, D, Hkv):
    s = make_read([37, 0, 1, 300, 16, 0], [0, 5, 31, 7, 16, 0], Hkv, D, dtype, layout, seed=D + Hkv, spare=3)
    run_read(s)
    check_read(s)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "nvfp4"])
def test_read_of_long_sequences_and_of_views(dtype):
    s = make_read([9000, 1, 4000], [0, 0, 0], 4, 128, dtype, "HND", seed=1, strided=True)
    wide = {x: torch.full((13001, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda") for x in ("k", "v")}
    s["k_out"], s["v_out"] = wide["k"][:, 1:5], wide["v"][:, 2:6]
    run_read(s)
    check_read(s)
    assert bool((wide["k"][:, 0] == 7.0).all()) and bool((wide["k"][:, 5] == 7.0).all()) and bool((wide["v"][:, :2] == 7.0).all())


@pytest.mark.parametrize("P", [1, 5, 128])
def test_read_from_pages_of_any_size(P):
    s = make_read([100, 30], [3, 0], 2, 64, "fp8", "NHD", P=P, seed=P)
    run_read(s)
    check_read(s)


def test_read_of_many_sequences():
    s = make_read([(7 * i) % 5 for i in range(3000)], [(3 * i) % 11 for i in range(3000)], 1, 64, seed=2)
    run_read(s)
    check_read(s)


def test_read_of_bad_pages_and_positions_gives_zeros():
    s = make_read([40, 50], [0, 10], 2, 128, seed=3)
    s["bt"][0, 1] = -1
    s["bt"][1, 2] = s["k_cache"].shape[0]
    run_read(s)
    check_read(s, flags=_abi.FLAG_PAGE_RANGE)
    s["err"].zero_()
    s["first"][1] = 30                      # past the table's four pages
    s["first_list"][1] = 30
    run_read(s)
    check_read(s, flags=_abi.FLAG_PAGE_RANGE | _abi.FLAG_SEQ_LEN_RANGE)
    s["err"].zero_()
    s["first"][0], s["first"][1] = -5, 2 ** 31 - 1
    s["first_list"] = [-5, 2 ** 31 - 1]
    run_read(s)
    check_read(s, flags=_abi.FLAG_PAGE_RANGE | _abi.FLAG_SEQ_LEN_RANGE)
    for bad in ([0, 60, 40], [-3, 20, 90], [0, 10, 200], [2 ** 31 - 1, -2 ** 31, 4]):
        s["err"].zero_()
        s["start"].copy_(torch.tensor(bad))
        run_read(s)
        torch.cuda.synchronize()
        assert int(s["err"].item()) & _abi.FLAG_ROW_RANGE


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "nvfp4"])
def test_what_is_written_is_read_back(dtype):
    """Slots in the order of a block table: the rows read back are the values written, to the cache's rounding."""
    s = make_write(70, 8, 2, 128, dtype, "HND", seed=7)
    s["slots"] = torch.arange(70, dtype=torch.int32, device="cuda") + 32
    b = _before(s)
    run_write(s)
    r = dict(s, bt=torch.arange(2, 7, dtype=torch.int32, device="cuda")[None], n=[70], first_list=[0], first=None,
             start=torch.tensor([0, 70], dtype=torch.int32, device="cuda"))
    for x in ("k", "v"):
        r[x + "_out"] = torch.full((70, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    run_read(r)
    check_read(r)
    check_write(s, b)
    if dtype == "bf16":
        assert torch.equal(r["k_out"], s["k_out"]) and torch.equal(r["v_out"], s["v"])


def _path(dtype, ctx, new, Hq=8, Hkv=2, D=128, seed=0):
    """Prompts written, attended to, read back and continued, and one decode step: as a serving loop calls them."""
    L = [a + b for a, b in zip(ctx, new)]
    T, pages = sum(L), [-(-(x + 1) // 16) for x in L]
    s = make_write(T, Hq, Hkv, D, dtype, "HND", weight="bf16", seed=seed, pages=sum(pages) + 3)
    g = torch.Generator(device="cuda").manual_seed(seed)
    perm = torch.randperm(s["pool"], generator=g, device="cuda").to(torch.int32)
    bt = torch.full((len(L), max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, p in enumerate(pages):
        bt[b, :p] = perm[at:at + p]
        at += p
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(L)]).cuda()
    pos = torch.cat([torch.arange(n) for n in L]).cuda()
    s["positions"] = pos.to(torch.int32)
    s["slots"] = (bt[seq, pos // 16].long() * 16 + pos % 16).to(torch.int32)
    run_write(s)
    starts = lambda n: torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
    p = dict(D=D, scale=D ** -0.5, q=s["q"], k=s["k_out"], v=s["v"], q_start=starts(L), k_start=None, n=L, L=L,
             ks=[sum(L[:i]) for i in range(len(L))], out=torch.zeros_like(s["q"]),
             lse=torch.zeros((T, Hq), device="cuda"), err=s["err"])
    run_prompt(p)
    # the last new[b] tokens of every sequence, over the cached context and themselves
    r = dict(s, bt=bt, n=L, first_list=[0] * len(L), first=None, start=starts(L))
    for x in ("k", "v"):
        r[x + "_out"] = torch.zeros((T, Hkv, D), dtype=torch.bfloat16, device="cuda")
    run_read(r)
    tail = torch.cat([torch.arange(sum(L[:b]) + ctx[b], sum(L[:b + 1])) for b in range(len(L))]).cuda()
    c = dict(D=D, scale=D ** -0.5, q=s["q"][tail].contiguous(), k=r["k_out"], v=r["v_out"], q_start=starts(new),
             k_start=starts(L), n=new, L=L, ks=p["ks"], out=torch.zeros((len(tail), Hq, D), dtype=torch.bfloat16, device="cuda"),
             lse=torch.zeros((len(tail), Hq), device="cuda"), err=s["err"])
    run_prompt(c)
    # and the prompts' last token through the decode over the same pages
    last = torch.tensor([sum(L[:b + 1]) - 1 for b in range(len(L))], device="cuda")
    sl = torch.tensor(L, dtype=torch.int32, device="cuda")
    op = torch.zeros((len(L), 2, Hq, D), device="cuda")
    lp = torch.zeros((len(L), 2, Hq), device="cuda")
    out, lse = torch.zeros((len(L), Hq, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((len(L), Hq), device="cuda")
    ql = s["q"][last].contiguous()
    if dtype == "nvfp4":
        pkv.paged_gqa_decode_nvfp4(ql, s["k_cache"], s["v_cache"], s["k_bs"], s["v_bs"], bt, sl, D ** -0.5, 2, op, lp,
                                   s["k_scale"], s["v_scale"], layout="HND", err_flag=s["err"])
    else:
        pkv.paged_gqa_decode(ql, s["k_cache"], s["v_cache"], bt, sl, D ** -0.5, 2, op, lp, s["k_scale"], s["v_scale"],
                             layout="HND", err_flag=s["err"])
    pkv.lse_merge(op, lp, out, lse)
    return s, p, c, tail, last, out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "nvfp4"])
def test_a_prompts_path(dtype):
    s, p, c, tail, last, out, lse = _path(dtype, [0, 100, 37, 400], [50, 1, 130, 64], seed=8)
    check_prompt(p)
    check_prompt(c)
    ends = [sum(c["n"][:b + 1]) - 1 for b in range(4)]
    # the decode reads the cache, as the continued prompt does (whose keys are rounded to bf16 again: 2^-8 of them)
    d = (out.double() - c["out"][ends].double()).abs()
    assert bool((d <= 2e-2 + 2e-2 * out.double().abs()).all()) and float((lse - c["lse"][ends]).abs().max()) < 3e-2
    if dtype == "bf16":
        # the same keys and values: the whole prompt's rows again, to the rounding of their weights and outputs
        for b in range(4):
            ref = prompt_reference(p, b)
            rows = torch.arange(sum(p["n"][:b]) + p["n"][b] - c["n"][b], sum(p["n"][:b + 1]), device="cuda")
            at = torch.arange(sum(c["n"][:b]), sum(c["n"][:b + 1]), device="cuda")
            e = (c["out"][at].double() - p["out"][rows].double()).abs()
            assert bool((e <= 2 * ref[2][-c["n"][b]:]).all())


def test_a_path_captured_and_replayed():
    """Write, attention and reading back in one graph, replayed over new inputs."""
    s = make_write(96, 8, 2, 128, "fp8", "HND", weight="bf16", seed=9)
    s["slots"] = torch.arange(96, dtype=torch.int32, device="cuda")
    p = dict(D=128, scale=0.1, q=s["q"], k=s["k_out"], v=s["v"], k_start=None,
             q_start=torch.tensor([0, 96], dtype=torch.int32, device="cuda"), out=torch.zeros_like(s["q"]),
             lse=torch.zeros((96, 8), device="cuda"), err=s["err"], ws=workspace(128))
    r = dict(s, bt=torch.arange(6, dtype=torch.int32, device="cuda")[None], first=None,
             start=torch.tensor([0, 96], dtype=torch.int32, device="cuda"), n=[96], first_list=[0])
    for x in ("k", "v"):
        r[x + "_out"] = torch.zeros((96, 2, 128), dtype=torch.bfloat16, device="cuda")

    def step():
        run_write(s)
        run_prompt(p)
        run_read(r)
    fresh = _before(s)
    step()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for k in range(3):
        for x in ("q", "k", "v"):
            s[x].copy_(fresh[x].roll(k, 0))
        graph.replay()
        torch.cuda.synchronize()
        got = [p["out"].clone(), p["lse"].clone(), r["k_out"].clone(), r["v_out"].clone()]
        for x in ("q", "k", "v"):
            s[x].copy_(fresh[x].roll(k, 0))
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, (p["out"], p["lse"], r["k_out"], r["v_out"])))
        assert torch.equal(r["k_out"], read_reference(r, "k"))
    assert int(s["err"].item()) == 0


def test_bound_buffers_and_another_stream():
    s, t = make_write(30, 8, 2, 128, "nvfp4", seed=10), make_write(30, 8, 2, 128, "nvfp4", seed=10)
    run_write(s)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    run_write({k: pkv.bind(v) if isinstance(v, torch.Tensor) else v for k, v in t.items()}, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(s[x], t[x]) for x in ("q", "k_out", "k_cache", "v_cache", "k_bs", "v_bs"))


@pytest.mark.parametrize("Hkv", [3, 8])
def test_read_flags_starts_wherever_they_are(Hkv):
    # (24 threads a row and 240 a CTA, or 256)
    for at in (1, 130, 239, 240, 247, 255, 256, 299):
        s = make_read([1] * 300, [0] * 300, Hkv, 64, seed=11)
        s["start"][at] = 301
        run_read(s)
        torch.cuda.synchronize()
        assert int(s["err"].item()) & pkv.FLAG_ROW_RANGE, at


@pytest.mark.parametrize("dtype", ["fp8", "nvfp4"])
def test_read_of_bad_pages_gives_zeros_whatever_the_scale(dtype):
    s = make_read([20], [0], 2, 64, dtype=dtype, seed=12)
    s["bt"][0, 1] = -1
    s["k_scale"][:] = float("nan")
    s["v_scale"][:] = float("inf")
    run_read(s)
    torch.cuda.synchronize()
    assert int(s["err"].item()) == pkv.FLAG_PAGE_RANGE
    assert bool((s["k_out"][16:] == 0).all()) and bool((s["v_out"][16:] == 0).all())
