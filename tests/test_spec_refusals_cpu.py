"""CPU tests of further refusals of the drafted-token and page calls, before any
CUDA work (fake, never dereferenced pointers)."""
import ctypes

import pytest
import torch

import paged_kv_gqa_04_gb300 as pkv
from paged_kv_gqa_04_gb300 import _abi, _build
from tests.test_abi_cpu import _t
from tests.test_spec_cpu import _caches

BAD, NO = _abi.PKV_ERR_INVALID_ARG, _abi.PKV_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.lib()


@pytest.mark.parametrize("name", ["bt", "sl", "qs", "ac", "na"])
@pytest.mark.parametrize("offset", [0, 4, -8])
def test_accepted_lengths_go_over_no_input(lib, name, offset):
    """Several CTAs read a sequence's inputs while one of them writes its new length."""
    B, A = 3, 5
    base = dict(bt=_t((B, 4), "i32", ptr=0x1000), sl=_t((B,), "i32", ptr=0x2000), qs=_t((B + 1,), "i32", ptr=0x3000),
                ac=_t((B, A), "i32", ptr=0x4000, strides=(A + 3, 1)), na=_t((B,), "i32", ptr=0x5000))
    caches = _caches(_t((10, 2, 16, 64), "bf16", ptr=0x100000))

    def call(ptr):
        return lib.pkv_accept_drafts(caches[0], caches[1], 1, base["bt"], base["sl"], base["qs"], base["ac"], base["na"],
                                     _t((B,), "i32", ptr=ptr), None, None)
    assert call(base[name].contents.ptr + offset) == BAD
    last = {"bt": (B * 4 - 1) * 4, "sl": 8, "qs": 12, "ac": ((B - 1) * (A + 3) + A - 1) * 4, "na": 8}[name]
    assert call(base[name].contents.ptr + last) == BAD


def test_pages_past_what_one_grid_copies_are_refused(lib):
    """A page in one piece is copied by CTAs of 16 KB, of which a grid has 65,535: a larger one would have been
    found out only behind the call's first half."""
    def call(nbytes):
        page = _t((10, 16, nbytes // 16), "fp8", strides=(nbytes, nbytes // 16, 1))
        c = _caches(page)
        return lib.pkv_fork_sequences(c[0], c[1], 1, _t((4, 4), "i32"), _t((4,), "i32"), _t((4,), "i32"),
                                      _t((0, 2), "i32"), _t((10,), "i32"), _t((0, 2), "i32"), None, None)
    assert call(65535 * 16384) == _abi.PKV_OK
    assert call(65535 * 16384 + 16) == NO
    assert call((1 << 30) - 16) == NO


def test_bound_nvfp4_values_have_their_descriptor():
    """bind() cannot know that uint8 values are pairs of E2M1; the NVFP4 calls say so."""
    x = torch.zeros((2, 3, 16, 32), dtype=torch.uint8)
    desc = _t(tuple(x.shape), "fp8", ptr=0x4000)
    b = _abi.Bound([x], desc, 1)
    d = _abi._fp4(b).contents
    assert d.dtype == _abi.PKV_FP4_E2M1X2 and d.ptr == 0x4000 and list(d.shape) == [2, 3, 16, 32]
    assert list(d.stride) == list(desc.contents.stride) and desc.contents.dtype == 1
    assert ctypes.addressof(_abi._fp4(b).contents) == ctypes.addressof(d)   # made once
    with pytest.raises(TypeError, match="uint8"):
        _abi._fp4(_abi.Bound([x.float()], desc, 1))
    with pytest.raises(TypeError, match="list"):
        _abi._fp4(_abi.Bound([x, x], desc, 2))


@pytest.mark.parametrize("bound", [False, True])
def test_a_workspace_is_as_large_as_its_memory(bound):
    """An expanded tensor has more elements than bytes behind them, and a strided one does not own all of its span."""
    make = (lambda x: _abi.Bound([x], None, 1)) if bound else (lambda x: x)
    x = torch.zeros(64, dtype=torch.uint8)
    assert _abi._workspace(make(x)) == (x.data_ptr(), 64)
    assert _abi._workspace(None) == (None, 0)
    for bad in (torch.zeros(1).expand(1 << 20), torch.zeros(8, 8)[:, ::2]):
        with pytest.raises(ValueError, match="contiguous"):
            _abi._workspace(make(bad))


def test_no_caches_may_be_none(lib, monkeypatch):
    """accept_drafts(None, ...) is accept_drafts([], ...), as a null pointer is in C."""
    seen = []
    monkeypatch.setattr(_abi, "_on_current_device", lambda *a: None)
    monkeypatch.setattr(_abi, "_stream", lambda s: None)
    monkeypatch.setattr(_abi, "lib", lambda: type("L", (), {"pkv_accept_drafts": lambda *a: seen.append(a[1:3]) or 0}))
    for caches in (None, []):
        _abi.accept_drafts(caches, None, None, None, None, None, None)
    assert seen == [(0, 1), (0, 1)]
