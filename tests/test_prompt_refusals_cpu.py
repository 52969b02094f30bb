"""CPU tests of what the prompt calls (pkv_qk_norm_rope_kv_write, pkv_gather_kv,
pkv_prompt_attention) refuse, and of their empty calls. Pointers are made up:
every call returns before any GPU work."""
import pytest

import paged_kv_gqa_04_gb300 as pkv
from paged_kv_gqa_04_gb300 import _abi, _build
from tests.test_abi_cpu import _t

INVALID, UNSUPPORTED, OK = _abi.PKV_ERR_INVALID_ARG, _abi.PKV_ERR_UNSUPPORTED, _abi.PKV_OK
T, HQ, HKV, D, PAGES, P = 4, 8, 2, 128, 10, 16


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.lib()


def at(n):
    return 0x100000 * n  # tensors that do not overlap


# ---- pkv_prompt_attention --------------------------------------------------------------------------------------------

def prompt(lib, **over):
    a = dict(q=_t((T, HQ, D), "bf16", at(1)), k=_t((T, HKV, D), "bf16", at(2)), v=_t((T, HKV, D), "bf16", at(3)),
             qs=_t((3,), "i32", at(4)), ks=None, scale=0.1, out=_t((T, HQ, D), "bf16", at(5)),
             lse=_t((T, HQ), "f32", at(6)), ws=at(7), nbytes=1 << 40)
    a.update(over)
    return lib.pkv_prompt_attention(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["scale"], a["out"], a["lse"], a["ws"],
                                    a["nbytes"], None, None)


@pytest.mark.parametrize("name,over", {
    "no_q": dict(q=None),
    "q_f32": dict(q=_t((T, HQ, D), "f32", at(1))),
    "q_2d": dict(q=_t((T, HQ * D), "bf16", at(1))),
    "q_null": dict(q=_t((T, HQ, D), "bf16", 0)),
    "no_k": dict(k=None),
    "k_head_dim": dict(k=_t((T, HKV, 64), "bf16", at(2))),
    "k_null": dict(k=_t((T, HKV, D), "bf16", 0)),
    "v_fp8": dict(v=_t((T, HKV, D), "fp8", at(3))),
    "v_rows": dict(v=_t((T + 1, HKV, D), "bf16", at(3))),
    "v_heads": dict(v=_t((T, HKV + 1, D), "bf16", at(3))),
    "heads_that_do_not_divide": dict(k=_t((T, 3, D), "bf16", at(2)), v=_t((T, 3, D), "bf16", at(3))),
    "no_heads": dict(k=_t((T, 0, D), "bf16", at(2)), v=_t((T, 0, D), "bf16", at(3))),
    "no_q_start": dict(qs=None),
    "q_start_f32": dict(qs=_t((3,), "f32", at(4))),
    "q_start_2d": dict(qs=_t((3, 1), "i32", at(4))),
    "q_start_empty": dict(qs=_t((0,), "i32", at(4))),
    "q_start_null": dict(qs=_t((3,), "i32", 0)),
    "k_start_length": dict(ks=_t((4,), "i32", at(8))),
    "k_rows_without_k_start": dict(k=_t((T + 1, HKV, D), "bf16", at(2)), v=_t((T + 1, HKV, D), "bf16", at(3))),
    "no_out": dict(out=None),
    "out_f32": dict(out=_t((T, HQ, D), "f32", at(5))),
    "out_rows": dict(out=_t((T - 1, HQ, D), "bf16", at(5))),
    "out_null": dict(out=_t((T, HQ, D), "bf16", 0)),
    "lse_bf16": dict(lse=_t((T, HQ), "bf16", at(6))),
    "lse_heads": dict(lse=_t((T, HKV), "f32", at(6))),
    "scale_nan": dict(scale=float("nan")),
    "scale_inf": dict(scale=float("inf")),
    "out_is_q": dict(out=_t((T, HQ, D), "bf16", at(1))),
    "out_in_v": dict(out=_t((T, HQ, D), "bf16", at(3) - 64)),
    "lse_in_k": dict(lse=_t((T, HQ), "f32", at(2) + 16)),
}.items(), ids=lambda x: x if isinstance(x, str) else "")
def test_prompt_attention_invalid(lib, name, over):
    assert prompt(lib, **over) == INVALID


def heads(hq, hkv, d):
    return dict(q=_t((T, hq, d), "bf16", at(1)), k=_t((T, hkv, d), "bf16", at(2)), v=_t((T, hkv, d), "bf16", at(3)),
                out=_t((T, hq, d), "bf16", at(5)), lse=None)


@pytest.mark.parametrize("name,over", {
    "head_dim_96": heads(HQ, HKV, 96),
    "head_dim_256": heads(HQ, HKV, 256),
    "group_17": heads(34, 2, D),
    "sequences": dict(qs=_t((65537,), "i32", at(4))),
    "tokens": dict(q=_t((1 << 27, HQ, D), "bf16", 1 << 44), out=_t((1 << 27, HQ, D), "bf16", 1 << 45), lse=None,
                   ks=_t((3,), "i32", at(8))),
    "keys": dict(k=_t((1 << 27, HKV, D), "bf16", 1 << 44), v=_t((1 << 27, HKV, D), "bf16", 1 << 45), ks=_t((3,), "i32", at(8))),
    "no_keys": dict(k=_t((0, HKV, D), "bf16", at(2)), v=_t((0, HKV, D), "bf16", at(3)), ks=_t((3,), "i32", at(8))),
    "q_inner_stride": dict(q=_t((T, HQ, D), "bf16", at(1), (2 * HQ * D, 2 * D, 2))),
    "q_unaligned": dict(q=_t((T, HQ, D), "bf16", at(1) + 2)),
    "q_row_stride": dict(q=_t((T, HQ, D), "bf16", at(1), (HQ * D + 4, D, 1))),
    "k_head_stride": dict(k=_t((T, HKV, D), "bf16", at(2), (HKV * 132, 132, 1))),
    "v_unaligned": dict(v=_t((T, HKV, D), "bf16", at(3) + 8)),
    "out_unaligned": dict(out=_t((T, HQ, D), "bf16", at(5) + 8)),
}.items(), ids=lambda x: x if isinstance(x, str) else "")
def test_prompt_attention_unsupported(lib, name, over):
    assert prompt(lib, **over) == UNSUPPORTED


def test_prompt_attention_without_rows_or_sequences(lib):
    none = dict(q=_t((0, HQ, D), "bf16", 0), k=_t((0, HKV, D), "bf16", 0), v=_t((0, HKV, D), "bf16", 0),
                out=_t((0, HQ, D), "bf16", 0), lse=None, ws=None, nbytes=0)
    assert prompt(lib, **none) == OK
    assert prompt(lib, qs=_t((1,), "i32", at(4)), ws=None, nbytes=0) == OK


def test_prompt_attention_workspace_sizes():
    small, large = (pkv.prompt_attention_workspace(d, 152) for d in (64, 128))
    assert 0 < small < large and pkv.prompt_attention_workspace(128, 1) < large
    for bad in [(0, 152), (96, 152), (256, 152), (-64, 152), (128, 0), (128, -1)]:
        assert pkv.prompt_attention_workspace(*bad) == 0


# ---- pkv_qk_norm_rope_kv_write ---------------------------------------------------------------------------------------

def write(lib, layout=1, style=0, eps=1e-6, **over):
    a = dict(q=_t((T, HQ, D), "bf16", at(1)), k=_t((T, HKV, D), "bf16", at(2)), v=_t((T, HKV, D), "bf16", at(3)),
             qw=_t((D,), "f32", at(4)), kw=_t((D,), "f32", at(5)), pos=_t((T,), "i32", at(6)),
             cs=_t((100, D), "f32", at(7)), kc=_t((PAGES, HKV, P, D), "bf16", at(8)),
             vc=_t((PAGES, HKV, P, D), "bf16", at(10)), kbs=None, vbs=None, slot=_t((T,), "i32", at(12)), ks=None, vs=None,
             ko=_t((T, HKV, D), "bf16", at(13)))
    a.update(over)
    return lib.pkv_qk_norm_rope_kv_write(a["q"], a["k"], a["v"], a["qw"], a["kw"], eps, a["pos"], a["cs"], a["kc"], a["vc"],
                                         a["kbs"], a["vbs"], a["slot"], a["ks"], a["vs"], a["ko"], layout, style, None, None)


def fp4_caches(width=D // 2, bs=D // 16):
    return dict(kc=_t((PAGES, HKV, P, width), "fp4", at(8)), vc=_t((PAGES, HKV, P, width), "fp4", at(10)),
                kbs=_t((PAGES, HKV, P, bs), "fp8", at(14)), vbs=_t((PAGES, HKV, P, bs), "fp8", at(15)),
                ks=_t((HKV,), "f32", at(16)), vs=_t((HKV,), "f32", at(17)))


@pytest.mark.parametrize("name,over", {
    "layout": dict(layout=2),
    "style": dict(style=2),
    "eps_negative": dict(eps=-1e-6),
    "eps_nan": dict(eps=float("nan")),
    "eps_inf": dict(eps=float("inf")),
    "no_k": dict(k=None),
    "no_k_weight": dict(kw=None),
    "no_q_weight": dict(qw=None),
    "k_weight_length": dict(kw=_t((64,), "f32", at(5))),
    "k_weight_2d": dict(kw=_t((1, D), "f32", at(5))),
    "k_weight_fp8": dict(kw=_t((D,), "fp8", at(5))),
    "weights_of_two_types": dict(qw=_t((D,), "bf16", at(4))),
    "positions_length": dict(pos=_t((T + 1,), "i32", at(6))),
    "fp8_without_scales": dict(kc=_t((PAGES, HKV, P, D), "fp8", at(8)), vc=_t((PAGES, HKV, P, D), "fp8", at(10))),
    "k_out_f32": dict(ko=_t((T, HKV, D), "f32", at(13))),
    "k_out_rows": dict(ko=_t((T - 1, HKV, D), "bf16", at(13))),
    "k_out_heads": dict(ko=_t((T, HQ, D), "bf16", at(13))),
    "k_out_in_q": dict(ko=_t((T, HKV, D), "bf16", at(1))),
    "k_out_in_v": dict(ko=_t((T, HKV, D), "bf16", at(3) + 256)),
    "k_out_beside_k": dict(ko=_t((T, HKV, D), "bf16", at(2) + 256)),
    "k_out_in_a_cache": dict(ko=_t((T, HKV, D), "bf16", at(8) + 1024)),
    "k_out_in_block_scales": dict(fp4_caches(), ko=_t((T, HKV, D), "bf16", at(15))),
    "fp4_without_v_block_scales": dict(fp4_caches(), vbs=None),
    "fp4_block_scale_width": fp4_caches(bs=D // 8),
    "fp4_without_scales": dict(fp4_caches(), ks=None),
}.items(), ids=lambda x: x if isinstance(x, str) else "")
def test_write_invalid(lib, name, over):
    assert write(lib, **over) == INVALID


@pytest.mark.parametrize("name,over", {
    "k_weight_stride": dict(kw=_t((D,), "f32", at(5), (2,))),
    "weight_unaligned": dict(kw=_t((D,), "f32", at(5) + 4)),
    "k_out_unaligned": dict(ko=_t((T, HKV, D), "bf16", at(13) + 8)),
    "q_unaligned": dict(q=_t((T, HQ, D), "bf16", at(1) + 2)),
    "head_dim_96": dict(q=_t((T, HQ, 96), "bf16", at(1)), k=_t((T, HKV, 96), "bf16", at(2)), v=_t((T, HKV, 96), "bf16", at(3)),
                        qw=_t((96,), "f32", at(4)), kw=_t((96,), "f32", at(5)), cs=_t((100, 96), "f32", at(7)),
                        kc=_t((PAGES, HKV, P, 96), "bf16", at(8)), vc=_t((PAGES, HKV, P, 96), "bf16", at(10)), ko=None),
}.items(), ids=lambda x: x if isinstance(x, str) else "")
def test_write_unsupported(lib, name, over):
    assert write(lib, **over) == UNSUPPORTED


def test_write_of_no_tokens(lib):
    none = dict(q=_t((0, HQ, D), "bf16", 0), k=_t((0, HKV, D), "bf16", 0), v=_t((0, HKV, D), "bf16", 0),
                pos=_t((0,), "i32", 0), slot=_t((0,), "i32", 0), ko=None)
    assert write(lib, **none) == OK
    assert write(lib, **dict(none, eps=-1.0)) == INVALID


# ---- pkv_gather_kv ---------------------------------------------------------------------------------------------------

def gather(lib, layout=1, **over):
    a = dict(kc=_t((PAGES, HKV, P, D), "bf16", at(8)), vc=_t((PAGES, HKV, P, D), "bf16", at(10)), kbs=None, vbs=None,
             bt=_t((3, 5), "i32", at(1)), start=_t((4,), "i32", at(2)), first=_t((3,), "i32", at(3)),
             ko=_t((T, HKV, D), "bf16", at(4)), vo=_t((T, HKV, D), "bf16", at(5)), ks=None, vs=None)
    a.update(over)
    return lib.pkv_gather_kv(a["kc"], a["vc"], a["kbs"], a["vbs"], a["bt"], a["start"], a["first"], a["ko"], a["vo"], a["ks"],
                             a["vs"], layout, None, None)


@pytest.mark.parametrize("name,over", {
    "layout": dict(layout=-1),
    "no_k_cache": dict(kc=None),
    "caches_of_two_types": dict(vc=_t((PAGES, HKV, P, D), "fp8", at(10))),
    "caches_of_two_shapes": dict(vc=_t((PAGES, HKV, 2 * P, D), "bf16", at(10))),
    "cache_f32": dict(kc=_t((PAGES, HKV, P, D), "f32", at(8)), vc=_t((PAGES, HKV, P, D), "f32", at(10))),
    "fp8_without_scales": dict(kc=_t((PAGES, HKV, P, D), "fp8", at(8)), vc=_t((PAGES, HKV, P, D), "fp8", at(10))),
    "fp8_scale_length": dict(kc=_t((PAGES, HKV, P, D), "fp8", at(8)), vc=_t((PAGES, HKV, P, D), "fp8", at(10)),
                             ks=_t((3,), "f32", at(16)), vs=_t((3,), "f32", at(17))),
    "fp4_without_v_block_scales": dict(fp4_caches(), vbs=None),
    "no_tables": dict(bt=None),
    "tables_1d": dict(bt=_t((15,), "i32", at(1))),
    "tables_f32": dict(bt=_t((3, 5), "f32", at(1))),
    "no_start": dict(start=None),
    "start_length": dict(start=_t((3,), "i32", at(2))),
    "first_length": dict(first=_t((4,), "i32", at(3))),
    "no_k_out": dict(ko=None),
    "k_out_f32": dict(ko=_t((T, HKV, D), "f32", at(4))),
    "k_out_heads": dict(ko=_t((T, HKV + 1, D), "bf16", at(4))),
    "v_out_rows": dict(vo=_t((T + 1, HKV, D), "bf16", at(5))),
    "v_out_null": dict(vo=_t((T, HKV, D), "bf16", 0)),
    "k_out_in_v_cache": dict(ko=_t((T, HKV, D), "bf16", at(10) + 512)),
    "v_out_in_k_cache": dict(vo=_t((T, HKV, D), "bf16", at(8))),
    "v_out_in_block_scales": dict(fp4_caches(), vo=_t((T, HKV, D), "bf16", at(14))),
}.items(), ids=lambda x: x if isinstance(x, str) else "")
def test_gather_invalid(lib, name, over):
    assert gather(lib, **over) == INVALID


@pytest.mark.parametrize("name,over", {
    "head_dim_96": dict(kc=_t((PAGES, HKV, P, 96), "bf16", at(8)), vc=_t((PAGES, HKV, P, 96), "bf16", at(10)),
                        ko=_t((T, HKV, 96), "bf16", at(4)), vo=_t((T, HKV, 96), "bf16", at(5))),
    "k_out_unaligned": dict(ko=_t((T, HKV, D), "bf16", at(4) + 8)),
    "v_out_row_stride": dict(vo=_t((T, HKV, D), "bf16", at(5), (HKV * D + 4, D, 1))),
    "cache_unaligned": dict(kc=_t((PAGES, HKV, P, D), "bf16", at(8) + 2)),
}.items(), ids=lambda x: x if isinstance(x, str) else "")
def test_gather_unsupported(lib, name, over):
    assert gather(lib, **over) == UNSUPPORTED


def test_gather_of_no_rows_or_sequences(lib):
    assert gather(lib, ko=_t((0, HKV, D), "bf16", 0), vo=_t((0, HKV, D), "bf16", 0)) == OK
    assert gather(lib, bt=_t((0, 5), "i32", at(1)), start=_t((1,), "i32", at(2)), first=_t((0,), "i32", at(3))) == OK
