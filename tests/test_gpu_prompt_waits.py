"""The prompts' attention's waits: none runs out while work goes on, however long
an item is. (That waits end where nothing comes is tested by the bounded waits'
self-test, which makes the forms used here run out.)"""
import math

import pytest
import torch

import paged_kv_gqa_04_gb300 as pkv

pytestmark = pytest.mark.gpu


def test_items_that_last_longer_than_the_limit_of_a_wait():
    # 153 pairs of row tiles of one kv head over 2^27 - 1 keys: an item and a piece of the next for every CTA, more
    # than a second each. Keys are zeros and values ones: all weights are one, and a thread's sum of them, 64 a tile, is
    # exact in fp32 (a whole number of 64s below 2^26), as are the values' in runs of 2^16 keys and the runs'.
    D, G, Tk = 64, 16, 2 ** 27 - 1
    T = 153 * 2 * (128 // G)
    if torch.cuda.mem_get_info()[0] < 60 * 2 ** 30:
        pytest.skip("needs 60 GB of device memory")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    q = torch.ones(T, G, D, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(Tk, 1, D, dtype=torch.bfloat16, device="cuda")
    v = torch.ones(Tk, 1, D, dtype=torch.bfloat16, device="cuda")
    starts = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (T, Tk)]
    out, lse = torch.zeros_like(q), torch.zeros(T, G, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(pkv.prompt_attention_workspace(D, sms), dtype=torch.uint8, device="cuda")
    first, last = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    first.record()
    pkv.prompt_attention(q, k, v, *starts, D ** -0.5, out, lse, ws, err_flag=err)
    last.record()
    torch.cuda.synchronize()
    assert first.elapsed_time(last) > 1000.0  # (or this tests nothing)
    assert int(err.item()) == 0
    assert bool((out == 1.0).all())
    # ln of 2^27 - T .. 2^27 - 1: log2 of an exact sum to 2^-22, times ln 2, and two roundings of a number below 32
    want = torch.log((Tk - T + 1 + torch.arange(T, device="cuda")).double())
    assert bool(((lse.double() - want[:, None]).abs() <= (2.0 ** -22 + 2.0 ** -19) * math.log(2) + 2.0 ** -19).all())
