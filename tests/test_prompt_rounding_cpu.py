"""CPU tests of the bound that independent roundings give (tests/_prompt_rounding.py): what the operator computes stays
within it, and a tile that is lost, met twice or met by another tile's weights does not, however long the row."""
import pytest
import torch

from tests._prompt_rounding import excess, in_tiles, weights


def row_case(L, D, n=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(m, D, generator=g).bfloat16() for m in (n, L, L))
    w = weights(q, k, D ** -0.5, torch.tensor([L - n + 1 + i for i in range(n)]))
    return w, v, w @ v.double()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L", [3, 4, 5, 9, 33, 128, 129, 1000, 20_000])
def test_independent_roundings_stay_within(L, D):
    for seed in range(40 if L < 1000 else 3):
        w, v, o = row_case(L, D, seed=seed)
        assert excess(in_tiles(w, v), w, v.double(), o) <= 1


@pytest.mark.parametrize("L,D", [(700, 128), (20_000, 128), (20_000, 64), (420_000, 64)])
@pytest.mark.parametrize("fault", ["lost", "met_twice", "three_back", "next"])
def test_one_wrong_tile_does_not(L, D, fault):
    w, v, o = row_case(L, D, n=2, seed=L)
    assert excess(in_tiles(w, v), w, v.double(), o) <= 1
    last = -(-L // 128) - 1
    for at in sorted({3, last // 2, last - 1}):
        wrong = {"lost": lambda t: None if t == at else t,
                 "met_twice": lambda t: at if t == at + 1 else t,
                 "three_back": lambda t: t - 3 if t == at else t,
                 "next": lambda t: t + 1 if t == at else t}[fault]
        assert excess(in_tiles(w, v, wrong=wrong), w, v.double(), o) > 1, at
