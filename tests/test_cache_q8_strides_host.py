"""Which codes an 8-bit cache takes by their strides (no GPU)."""
import pytest
import torch

from learned_token_pruning_tg_b200 import tokengate as tg


def codes(*shape):
    return torch.zeros(*shape, dtype=torch.int8)


def test_strides_of_caches():
    assert tg._cache_strides(codes(2, 64, 3, 64), codes(2, 64, 3, 64)) == (192, 64 * 192)
    assert tg._cache_strides(codes(0, 64, 3, 64), codes(0, 64, 3, 64)) == (192, 64 * 192)
    assert tg._cache_strides(codes(2, 0, 3, 64), codes(2, 0, 3, 64)) == (192, 0)
    both = codes(2, 96, 2, 3, 64)                            # K and V of a token side by side, room behind a sequence
    assert tg._cache_strides(both[:, :64, 0], both[:, :64, 1]) == (384, 96 * 384)
    one = codes(1, 64, 1, 128).as_strided((1, 64, 1, 128), (0, 128, 0, 1))   # what strides of one entry say
    assert tg._cache_strides(one, one.clone()) == (128, 64 * 128)


@pytest.mark.parametrize("k", [
    codes(2, 1, 3, 64).expand(2, 64, 3, 64),                 # one token's codes for all
    codes(1, 64, 3, 64).expand(2, 64, 3, 64),                # one sequence's codes for both
    codes(2, 64, 1, 64).expand(2, 64, 3, 64),                # one head's codes for all
    codes(64 * 192).as_strided((2, 32, 3, 64), (192, 192, 64, 1)),   # sequences that begin inside one another
    codes(64 * 192).as_strided((2, 32, 3, 64), (6144, 128, 64, 1)),  # tokens that do
    codes(64, 2, 3, 64).transpose(0, 1),                     # the sequences' tokens in turn
    codes(2, 64, 64, 3).transpose(2, 3),
    codes(2, 64, 3, 65)[..., :64],
], ids=range(8))
def test_refused_strides(k):
    with pytest.raises(ValueError):
        tg._cache_strides(k, k)


def test_unequal_strides():
    with pytest.raises(ValueError):
        tg._cache_strides(codes(2, 64, 3, 64), codes(2, 96, 3, 64)[:, :64])
