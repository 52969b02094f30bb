"""GPU tests of a key's norm in pkv_qk_norm_rope_kv_write to the last bit: the
cache bytes and the kept keys of random rows against the documented order of the
sum of squares, step by step in float32."""
import pytest
import torch

from tests._prompt import E2M1, make_write, rows_of, run_write

pytestmark = pytest.mark.gpu


def sum_in_order(x):
    """Squares of [.., D], each rounded: columns 32 apart in ascending order, then neighbours in pairs, pairs of pairs
    and so on."""
    s = (x * x).unflatten(-1, (-1, 32))
    t = s[..., 0, :]
    for i in range(1, s.shape[-2]):
        t = t + s[..., i, :]
    while t.shape[-1] > 1:
        t = t[..., 0::2] + t[..., 1::2]
    return t


def normed_and_rotated(s, k):
    x, D = k.float(), s["D"]
    r = torch.rsqrt(sum_in_order(x) * (1.0 / D) + s["eps"])
    y = (x * r) * s["k_weight"].float()
    cs = s["cos_sin"][s["positions"].long()][:, None]
    c, sn = cs[..., :D // 2], cs[..., D // 2:]
    a, b = (y[..., :D // 2], y[..., D // 2:]) if s["style"] == "neox" else (y[..., 0::2], y[..., 1::2])
    ac, bs, bc, as_ = a * c, b * sn, b * c, a * sn
    u, v = ac - bs, bc + as_
    return torch.cat((u, v), -1) if s["style"] == "neox" else torch.stack((u, v), -1).flatten(-2)


def e2m1_codes(z):
    """Nearest, ties to the even code, saturating; the sign of zero kept."""
    m, v = z.abs().clamp(max=6.0), E2M1.to(z.device)
    i = torch.bucketize(m, v, right=True) - 1
    lo, hi = v[i], v[(i + 1).clamp(max=7)]
    up = (m - lo > hi - m) | ((m - lo == hi - m) & (i % 2 == 1))
    return torch.where(up & (i < 7), i + 1, i) + 8 * torch.signbit(z).long()


@pytest.mark.parametrize("T", [1, 3, 40, 5000])
@pytest.mark.parametrize("dtype,style,weight", [("bf16", "neox", "f32"), ("fp8", "interleaved", "bf16"), ("nvfp4", "neox", "bf16"),
                                                ("nvfp4", "interleaved", "f32")])
@pytest.mark.parametrize("D", [64, 128])
def test_cached_keys_bit_for_bit(T, dtype, style, weight, D):
    s = make_write(T, 8, 4, D, dtype, style=style, weight=weight, seed=T + D)
    k = s["k"].clone()
    run_write(s)
    torch.cuda.synchronize()
    assert int(s["err"].item()) == 0
    y = normed_and_rotated(s, k)
    assert torch.equal(s["k_out"].view(torch.int16), y.bfloat16().view(torch.int16))
    got = rows_of(s, s["k_cache"], s["slots"])
    if dtype == "bf16":
        assert torch.equal(got.view(torch.int16), y.bfloat16().view(torch.int16))
        return
    g = s["k_scale"][:, None]
    if dtype == "fp8":
        want = (y / g).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(got, want)
        return
    b = y.unflatten(-1, (-1, 16))
    sc = (b.abs().amax(-1) / (6 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    assert torch.equal(rows_of(s, s["k_bs"], s["slots"]), sc.view(torch.uint8))
    den = (g * sc.float())[..., None]
    codes = torch.where(den > 0, e2m1_codes(b / den), 0).flatten(-2)
    assert torch.equal(got, (codes[..., 0::2] | codes[..., 1::2] << 4).to(torch.uint8))
