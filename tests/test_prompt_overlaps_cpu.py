"""CPU tests: what pkv_prompt_attention writes, its workspace among it, must not
lie over what it reads, nor over another of its outputs. Pointers are made up:
every call returns before any GPU work."""
import pytest

from tests.test_abi_cpu import _t
from tests.test_prompt_refusals_cpu import D, HQ, INVALID, T, at, lib, prompt  # noqa: F401

WS = 1 << 20  # bytes; at(30) .. at(31)


@pytest.mark.parametrize("name,over", {
    "lse_in_out": dict(lse=_t((T, HQ), "f32", at(5) + 64)),
    "out_over_q_start": dict(out=_t((T, HQ, D), "bf16", at(4))),
    "lse_over_k_start": dict(ks=_t((3,), "i32", at(8)), lse=_t((T, HQ), "f32", at(8))),
    "workspace_over_q": dict(ws=at(1) + 16),
    "workspace_over_k": dict(ws=at(2) - WS + 16),
    "workspace_over_v": dict(ws=at(3)),
    "workspace_over_out": dict(ws=at(5) + 32),
    "workspace_over_lse": dict(ws=at(6) - 64),
    "workspace_over_q_start": dict(ws=at(4)),
    "workspace_over_k_start": dict(ks=_t((3,), "i32", at(8)), ws=at(8)),
}.items(), ids=lambda x: x if isinstance(x, str) else "")
def test_prompt_attention_overlaps(lib, name, over):
    assert prompt(lib, **dict(dict(nbytes=WS, ws=at(30)), **over)) == INVALID
