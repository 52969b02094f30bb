"""CPU tests of the drafted-token and page operators' host side: refusals of
inconsistent arguments before any CUDA work (fake, never dereferenced
pointers), the workspace size, and the statements of tests/_spec.py that the
GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import paged_kv_gqa_04_gb300 as pkv
from paged_kv_gqa_04_gb300 import _abi, _build
from tests._spec import accept_reference, fork_reference, resize_reference
from tests.test_abi_cpu import _t

BAD, NO = _abi.PKV_ERR_INVALID_ARG, _abi.PKV_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.lib()


def _caches(*ts):
    arr = (_abi.PkvTensor * max(len(ts), 1))()
    for i, t in enumerate(ts):
        arr[i] = t.contents
    return ctypes.cast(arr, ctypes.POINTER(_abi.PkvTensor)), len(ts), arr


def test_tree_decode_refusals(lib):
    T, Hq, Hkv, D, B = 9, 8, 2, 128, 3
    kc = _t((10, Hkv, 16, D), "bf16")
    base = dict(q=_t((T, Hq, D), "bf16"), kc=kc, vc=kc, bt=_t((B, 5), "i32"), sl=_t((B,), "i32"),
                qs=_t((B + 1,), "i32"), mask=_t((T, 1), "i32"), scale=0.1, out=_t((T, Hq, D), "bf16"),
                lse=_t((T, Hq), "f32"), ws=0x1000, n=1 << 40, ks=None, vs=None, layout=1)

    def call(**o):
        a = dict(base, **o)
        return lib.pkv_paged_tree_decode(a["q"], a["kc"], a["vc"], a["bt"], a["sl"], a["qs"], a["mask"], a["scale"],
                                         a["out"], a["lse"], a["ws"], a["n"], a["ks"], a["vs"], a["layout"], None, None)
    assert call(q=_t((T, Hq, D), "f32")) == BAD
    assert call(q=_t((T, 7, D), "bf16")) == BAD
    assert call(q=_t((T, Hq, 64), "bf16")) == BAD
    assert call(sl=_t((B + 1,), "i32")) == BAD
    assert call(qs=_t((B,), "i32")) == BAD
    assert call(qs=_t((B + 1,), "f32")) == BAD
    assert call(mask=_t((T + 1, 1), "i32")) == BAD
    assert call(mask=_t((T, 1), "f32")) == BAD
    assert call(out=_t((T, Hq, D), "f32")) == BAD
    assert call(out=_t((T + 1, Hq, D), "bf16")) == BAD
    assert call(lse=_t((T, Hq + 1), "f32")) == BAD
    assert call(scale=float("inf")) == BAD
    assert call(layout=3) == BAD
    assert call(vc=_t((11, Hkv, 16, D), "bf16")) == BAD
    fp8 = _t((10, Hkv, 16, D), "fp8")
    assert call(kc=fp8, vc=fp8) == BAD                                        # no scales
    assert call(kc=_t((10, Hkv, 8, D), "bf16"), vc=_t((10, Hkv, 8, D), "bf16")) == NO
    assert call(q=_t((T, 34, D), "bf16"), out=_t((T, 34, D), "bf16"), lse=_t((T, 34), "f32")) == NO   # groups of 17
    assert call(q=_t((T, Hq, D), "bf16", ptr=0x1008)) == NO
    assert call(out=_t((T, Hq, D), "bf16", strides=(Hq * D + 4, D, 1))) == NO
    assert call(mask=_t((T, 65), "i32")) == NO
    assert call(bt=_t((B, 5), "i32", strides=(1, B))) == NO
    assert call(q=_t((0, Hq, D), "bf16"), out=_t((0, Hq, D), "bf16"), lse=_t((0, Hq), "f32"),
                mask=None) == _abi.PKV_OK
    # NVFP4 caches are not taken
    fp4 = _t((10, Hkv, 16, D // 2), "fp4")
    assert call(kc=fp4, vc=fp4) == BAD


def test_bound_lists_are_not_taken_for_a_tensor():
    import torch
    x = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="list"):
        _abi._desc(_abi.Bound([x, x], None, 2))
    assert _abi._desc(_abi.Bound([x], 5, 1)) == 5


def test_workspace_sizes(lib):
    assert pkv.tree_decode_workspace(100, 32, 128, 152) > 0
    for bad in ((-1, 8, 128, 152), (5, 0, 128, 152), (5, 8, 96, 152), (5, 8, 128, 0)):
        assert pkv.tree_decode_workspace(*bad) == 0


def test_accept_refusals(lib):
    B, A = 3, 5
    base = dict(c=_caches(_t((10, 2, 16, 64), "bf16")), layout=1, bt=_t((B, 4), "i32"), sl=_t((B,), "i32"),
                qs=_t((B + 1,), "i32"), ac=_t((B, A), "i32"), na=_t((B,), "i32"), so=_t((B,), "i32", ptr=0x9000))

    def call(**o):
        a = dict(base, **o)
        return lib.pkv_accept_drafts(a["c"][0], a.get("n", a["c"][1]), a["layout"], a["bt"], a["sl"], a["qs"], a["ac"],
                                     a["na"], a["so"], None, None)
    assert call(layout=2) == BAD
    assert call(n=-1) == BAD
    assert call(n=5000) == NO
    assert call(so=_t((B,), "i32")) == BAD                                    # over seq_lens
    assert call(so=_t((B,), "i32", ptr=0x1008)) == BAD
    assert call(na=_t((B + 1,), "i32")) == BAD
    assert call(qs=_t((B,), "i32")) == BAD
    assert call(ac=_t((B + 1, A), "i32")) == BAD
    assert call(ac=_t((B, 1025), "i32")) == NO
    assert call(ac=_t((B, A), "i32", strides=(1, B))) == NO
    assert call(c=_caches(_t((10, 2, 16, 64), "bf16"), _t((11, 2, 16, 64), "bf16"))) == BAD
    assert call(c=_caches(_t((10, 2, 16, 64), "bf16"), _t((10, 2, 8, 64), "bf16"))) == BAD
    assert call(c=_caches(_t((10, 2), "bf16"))) == BAD
    assert call(c=_caches(_t((10, 2, 16, 64), "bf16", strides=(2048, 1024, 1, 16)))) == NO


def test_resize_refusals(lib):
    B = 3
    base = dict(bt=_t((B, 4), "i32"), pc=_t((B,), "i32"), nl=_t((B,), "i32"), pr=_t((50,), "i32"), P=16)

    def call(**o):
        a = dict(base, **o)
        return lib.pkv_resize_sequences(a["bt"], a["pc"], a["nl"], a["pr"], a["P"], None, None)
    assert call(P=0) == BAD
    assert call(P=65537) == NO
    assert call(pc=_t((B + 1,), "i32")) == BAD
    assert call(nl=_t((B,), "f32")) == BAD
    assert call(pr=_t((50, 1), "i32")) == BAD
    assert call(pr=_t((50,), "i32", strides=(2,))) == NO
    assert call(bt=_t((B, 4), "f32")) == BAD
    many = 16385
    assert call(bt=_t((many, 4), "i32"), pc=_t((many,), "i32"), nl=_t((many,), "i32")) == NO
    assert call(bt=_t((0, 4), "i32"), pc=_t((0,), "i32"), nl=_t((0,), "i32")) == _abi.PKV_OK


def test_fork_refusals(lib):
    R, n = 4, 2
    base = dict(c=_caches(_t((10, 2, 16, 64), "bf16")), layout=1, bt=_t((R, 4), "i32"), pc=_t((R,), "i32"),
                sl=_t((R,), "i32"), fk=_t((n, 2), "i32"), pr=_t((10,), "i32"), cp=_t((n, 2), "i32", ptr=0x9000))

    def call(**o):
        a = dict(base, **o)
        return lib.pkv_fork_sequences(a["c"][0], a["c"][1], a["layout"], a["bt"], a["pc"], a["sl"], a["fk"], a["pr"],
                                      a["cp"], None, None)
    assert call(c=_caches()) == BAD
    assert call(pr=_t((11,), "i32")) == BAD
    assert call(fk=_t((n, 3), "i32")) == BAD
    assert call(cp=_t((n + 1, 2), "i32", ptr=0x9000)) == BAD
    assert call(cp=_t((n, 2), "i32")) == BAD                                  # over forks
    assert call(fk=_t((n, 2), "i32", strides=(3, 1))) == NO
    assert call(fk=_t((16385, 2), "i32"), cp=_t((16385, 2), "i32", ptr=0x900000)) == NO
    assert call(fk=_t((0, 2), "i32"), cp=_t((0, 2), "i32")) == _abi.PKV_OK


def test_resize_statement():
    bt = np.full((3, 4), -1, np.int32)
    counts, refs = np.zeros(3, np.int32), np.array([0, 1, 0, 0, 0, 0], np.int32)
    bt, counts, refs, f = resize_reference(bt, counts, np.array([17, -1, 33]), refs, 16)
    assert f == 0 and bt.tolist() == [[0, 2, -1, -1], [-1] * 4, [3, 4, 5, -1]] and counts.tolist() == [2, 0, 3]
    bt, counts, refs, f = resize_reference(bt, counts, np.array([1, 48, 16]), refs, 16)
    assert f == 0 and bt.tolist() == [[0, -1, -1, -1], [2, 4, 5, -1], [3, -1, -1, -1]]
    bt, counts, refs, f = resize_reference(bt, counts, np.array([17, 64, 65]), refs, 16)
    assert f == pkv.FLAG_POOL_EMPTY | pkv.FLAG_SEQ_LEN_RANGE and counts.tolist() == [1, 3, 1]


def test_accept_and_fork_statements():
    pool = np.arange(4 * 2 * 1).reshape(4, 2, 1)
    bt = np.array([[3, 1, 0]], np.int32)               # positions 0..5 hold 6 7 2 3 0 1
    p, out, f = accept_reference([pool], bt, np.array([6], np.int32), [0, 5], np.array([[1, 2, 4]]), [3], 2)
    assert f == 0 and out.tolist() == [4]
    assert [int(p[0][bt[0, t // 2], t % 2, 0]) for t in range(4)] == [6, 2, 3, 1]
    bt2 = np.array([[3, 1, 0], [-1, -1, -1]], np.int32)
    pools, b, c, n, refs, copies, f = fork_reference([pool], bt2, np.array([3, 0], np.int32), np.array([5, 0], np.int32),
                                                     [(0, 1)], np.array([1, 1, 0, 1], np.int32), 2)
    assert f == 0 and b[1].tolist() == [3, 1, 2] and copies.tolist() == [[0, 2]] and refs.tolist() == [1, 2, 1, 2]
    assert np.array_equal(pools[0][2], pool[0]) and c.tolist() == [3, 3] and n.tolist() == [5, 5]
