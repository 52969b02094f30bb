"""CPU tests: pkv_gather_kv's two outputs must not lie over one another, nor over
what the call reads; views of one buffer that lie side by side are taken.
Pointers are made up: refused calls return before any GPU work, and those that
are taken are made only where there is no device to launch on."""
import random

import pytest
import torch

from tests.test_abi_cpu import _t
from tests.test_prompt_refusals_cpu import D, HKV, INVALID, T, at, gather, lib  # noqa: F401


@pytest.mark.parametrize("name,over", {
    "the_same": dict(vo=_t((T, HKV, D), "bf16", at(4))),
    "a_row_on": dict(vo=_t((T, HKV, D), "bf16", at(4) + 2 * HKV * D)),
    "a_head_on": dict(vo=_t((T, HKV, D), "bf16", at(4) + 2 * D)),
    "eight_values_on": dict(vo=_t((T, HKV, D), "bf16", at(4) + 16)),
    "a_row_back": dict(vo=_t((T, HKV, D), "bf16", at(4) - 2 * HKV * D)),
    "halves_that_meet": dict(ko=_t((T, HKV, D), "bf16", at(4), (2 * HKV * D, D, 1)),
                             vo=_t((T, HKV, D), "bf16", at(4) + 2 * (HKV - 1) * D, (2 * HKV * D, D, 1))),
    "other_strides": dict(ko=_t((T, HKV, D), "bf16", at(4), (2 * HKV * D, D, 1)), vo=_t((T, HKV, D), "bf16", at(4) + 256)),
    "k_out_over_start": dict(ko=_t((T, HKV, D), "bf16", at(2))),
    "v_out_over_first": dict(vo=_t((T, HKV, D), "bf16", at(3))),
    "v_out_over_tables": dict(vo=_t((T, HKV, D), "bf16", at(1))),
}.items(), ids=lambda x: x if isinstance(x, str) else "")
def test_gather_outputs_over_one_another(lib, name, over):
    assert gather(lib, **over) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers")
@pytest.mark.parametrize("name,over", {
    "halves_of_one_buffer": dict(ko=_t((T, HKV, D), "bf16", at(4), (2 * HKV * D, D, 1)),
                                 vo=_t((T, HKV, D), "bf16", at(4) + 2 * HKV * D, (2 * HKV * D, D, 1))),
    "the_halves_swapped": dict(vo=_t((T, HKV, D), "bf16", at(4), (2 * HKV * D, D, 1)),
                               ko=_t((T, HKV, D), "bf16", at(4) + 2 * HKV * D, (2 * HKV * D, D, 1))),
    "heads_in_turn": dict(ko=_t((T, HKV, D), "bf16", at(4), (2 * HKV * D, 2 * D, 1)),
                          vo=_t((T, HKV, D), "bf16", at(4) + 2 * D, (2 * HKV * D, 2 * D, 1))),
    "heads_outermost": dict(ko=_t((T, HKV, D), "bf16", at(4), (D, 2 * T * D, 1)),
                            vo=_t((T, HKV, D), "bf16", at(4) + 2 * T * D, (D, 2 * T * D, 1))),
    "one_behind_the_other": dict(vo=_t((T, HKV, D), "bf16", at(4) + 2 * T * HKV * D)),
}.items(), ids=lambda x: x if isinstance(x, str) else "")
def test_gather_outputs_side_by_side_are_taken(lib, name, over):
    # (as far as the launch, which wants a device)
    assert gather(lib, **over) != INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers")
def test_views_of_one_buffer_against_their_elements(lib):
    rng = random.Random(5)
    seen = set()
    for _ in range(400):
        n, heads = rng.randint(1, 5), rng.choice([HKV])
        row, head = rng.sample([64, 128, 136, 192, 256, 264, 384, 512, 640], 2)
        apart = 8 * rng.randint(-200, 200)

        def elements(first):
            return {first + i * row + j * head + d for i in range(n) for j in range(heads) for d in range(0, D, 8)}
        meet = bool(elements(0) & elements(apart))  # (all strides and distances are multiples of 8)
        a = dict(ko=_t((n, heads, D), "bf16", at(40), (row, head, 1)), vo=_t((n, heads, D), "bf16", at(40) + 2 * apart, (row, head, 1)))
        assert (gather(lib, **a) == INVALID) == meet, (n, row, head, apart)
        seen.add(meet)
    assert seen == {True, False}
