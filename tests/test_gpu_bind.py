"""GPU tests that calls take bound buffers (bind()) with the same results as tensors."""
import pytest
import torch

import paged_kv_gqa_04_gb300 as pkv

pytestmark = pytest.mark.gpu


def _nvfp4_state():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    B, Hq, Hkv, D, pages = 3, 8, 2, 128, 9
    n = dict(generator=g, device="cuda")
    s = dict(q=torch.randn((B, Hq, D), **n).bfloat16(), k=torch.randn((B, Hkv, D), **n).bfloat16(),
             v=torch.randn((B, Hkv, D), **n).bfloat16(), cs=torch.randn((64, D), **n))
    for name, w in (("kc", D // 2), ("vc", D // 2), ("kbs", D // 16), ("vbs", D // 16)):
        s[name] = torch.randint(0, 0x70, (pages, Hkv, 16, w), dtype=torch.uint8, **n)
    i32 = dict(dtype=torch.int32, device="cuda")
    s.update(pos=torch.tensor([30, 3, 47], **i32), slots=torch.tensor([30, 3 * 16 + 3, 8 * 16 + 15], **i32),
             bt=torch.tensor([[0, 1, -1], [3, -1, -1], [6, 7, 8]], **i32), sl=torch.tensor([31, 4, 48], **i32),
             sc=torch.full((1,), 0.5, device="cuda"), err=torch.zeros(1, **i32),
             op=torch.zeros((B, 2, Hq, D), device="cuda"), lp=torch.zeros((B, 2, Hq), device="cuda"),
             out=torch.zeros((B, Hq, D), dtype=torch.bfloat16, device="cuda"), lse=torch.zeros((B, Hq), device="cuda"))
    sp, _, work = pkv.plan_splits([31, 4, 48], Hkv, Hq, D, 3, "nvfp4", 152, 2)
    s.update(sp=torch.from_numpy(sp).cuda(), work=torch.from_numpy(work).cuda())
    return s


def _nvfp4_step(s, a):
    pkv.rope_kv_write_nvfp4(a["q"], a["k"], a["v"], a["pos"], a["cs"], a["kc"], a["vc"], a["kbs"], a["vbs"], a["slots"],
                            a["sc"], a["sc"], err_flag=a["err"])
    results = []
    pkv.paged_gqa_decode_nvfp4(a["q"], a["kc"], a["vc"], a["kbs"], a["vbs"], a["bt"], a["sl"], 0.1, 2, a["op"], a["lp"],
                               a["sc"], a["sc"], err_flag=a["err"])
    pkv.lse_merge(a["op"], a["lp"], a["out"], a["lse"])
    results += [s["out"].clone(), s["lse"].clone()]
    pkv.paged_gqa_decode_planned(a["q"], a["kc"], a["vc"], a["bt"], a["sl"], 0.1, a["sp"], a["work"], a["op"], a["lp"],
                                 a["sc"], a["sc"], err_flag=a["err"], k_block_scale=a["kbs"], v_block_scale=a["vbs"])
    pkv.lse_merge_planned(a["op"], a["lp"], a["sp"], a["out"], a["lse"])
    results += [s["out"].clone(), s["lse"].clone(), s["kc"], s["vc"], s["kbs"], s["vbs"], s["q"], s["err"]]
    torch.cuda.synchronize()
    return results


def test_nvfp4_calls_take_bound_buffers():
    x, y = _nvfp4_state(), _nvfp4_state()
    want, got = _nvfp4_step(x, x), _nvfp4_step(y, {k: pkv.bind(v) for k, v in y.items()})
    assert int(x["err"].item()) == 0 and bool(torch.isfinite(want[0].float()).all())
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_copy_and_measurement_calls_take_bound_buffers():
    src, dst = torch.arange(1000, device="cuda"), torch.zeros(1000, dtype=torch.int64, device="cuda")
    sink, src32 = torch.zeros(4, dtype=torch.int32, device="cuda"), src.to(torch.int32)
    b, d = pkv.bind(src32), torch.zeros(1000, dtype=torch.int32, device="cuda")
    pkv.copy(pkv.bind(d), b)
    pkv.stream_read(b, pkv.bind(sink))
    torch.cuda.synchronize()
    assert torch.equal(d, src32)
    pkv.copy(dst, src)
    torch.cuda.synchronize()
    assert torch.equal(dst, src)
