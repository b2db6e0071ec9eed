"""The checks of ``fp8_sums`` see the mistakes they are there for: each is
planted in the oracle's product, at the largest number of columns."""
import numpy as np
import pytest

from oracle import fp8_oracle as F
from tests import fp8_sums as S


def _product(x, w, drop=None, scale=None, chain_round=None):
    """The oracle's product by blocks: block `drop` left out, block `scale`'s
    scale byte of w one too large, sums of 16 blocks through `chain_round`."""
    k = x.shape[1]
    xq, wq = F.roundtrip(x), F.roundtrip(w)
    parts = [xq[:, c:c + S.BLOCK] @ wq[:, c:c + S.BLOCK].T for c in range(0, k, S.BLOCK)]
    if drop is not None:
        parts[drop] = parts[drop] * 0
    if scale is not None:
        parts[scale] = parts[scale] * 2
    chains = [sum(parts[i:i + 16]) for i in range(0, len(parts), 16)]
    return sum(chain_round(c) if chain_round else c for c in chains)


def _bf16(v):
    m, e = np.frexp(v)
    return np.ldexp(np.rint(m * 256) / 256, e)


@pytest.mark.parametrize("k", [1111, 4096, 65536])
def test_whole_numbers_are_exact_and_see_mistakes(k):
    x, w = S.whole(np.random.default_rng(k), 5, k, 4)
    assert np.array_equal(F.roundtrip(x), x) and np.array_equal(F.roundtrip(w), w)
    want = x.astype(np.float64) @ w.astype(np.float64).T
    assert np.array_equal(_product(x, w), want) and 24 * k < 2 ** 24
    blocks = -(-k // S.BLOCK)
    for b in {0, 1, 15, 16, blocks // 2, blocks - 2, blocks - 1} & set(range(blocks)):
        assert not np.array_equal(_product(x, w, drop=b), want)
        assert not np.array_equal(_product(x, w, scale=b), want)
    if k > 4096:
        assert not np.array_equal(_product(x, w, chain_round=_bf16), want)


def test_one_block_sees_which():
    rng = np.random.default_rng(3)
    x, w = S.one_block(rng, 4, 1280, [7, 0, 9])
    want = _product(x, w)
    for t, b in enumerate([7, 0, 9]):
        lost = _product(x, w, drop=b)
        assert not np.array_equal(lost[t], want[t])
        assert all(np.array_equal(lost[s], want[s]) for s in range(3) if s != t)


@pytest.mark.parametrize("k", [9000, 65536])
def test_norm_sees_mistakes(k):
    rng = np.random.default_rng(k)
    x, w = rng.standard_normal((8, k)), rng.standard_normal((20, k))
    want = _product(x, w)
    assert S.relative_error(want.astype(np.float32), want) < 2.0 ** -24
    for bad in (dict(drop=3), dict(scale=3), dict(chain_round=_bf16)):
        assert S.relative_error(_product(x, w, **bad), want) > 20 * S.CHAIN_ERROR, bad
