"""No block is lost, doubled or misscaled, and sums keep their bits, at every
number of columns: exact on whole numbers, within the chains' truncation in the
2-norm on random ones (``fp8_sums``)."""
import numpy as np
import pytest

import sparse_quantized_rank_b200 as C
from tests import fp8_sums as S

pytestmark = pytest.mark.gpu

TYPES = ("float32", "float16", "bfloat16")


def _exact(x, w):
    return x.double() @ w.double().t()


def _sides(x, w, dev):
    import torch
    return torch.from_numpy(x).to(dev), torch.from_numpy(w).to(dev)


SIZES = [
    # n, k, tokens: one tile, odd numbers of blocks, ranges that start in a chunk, whole tiles and split ones
    (128, 65536, 1), (128, 65536, 4), (140, 65536, 16), (140, 65536, 30), (140, 65536, 70), (140, 65536, 300),
    (300, 11008, 2), (300, 11008, 12), (300, 11008, 32), (300, 11008, 40), (300, 11008, 200),
    (4096, 1111, 3), (20000, 1290, 2), (20000, 1290, 9), (20000, 1290, 31), (2000, 1290, 600),
    (640, 5000, 4), (640, 5000, 17), (9000, 2300, 96), (513, 129, 1), (513, 129, 100), (700, 2000, 33),
]


@pytest.mark.parametrize("n,k,tokens", SIZES)
def test_whole_numbers(n, k, tokens, cuda_dev):
    import torch
    x, w = _sides(*S.whole(np.random.default_rng(n + k + tokens), n, k, tokens), cuda_dev)
    want, layer = _exact(x, w), C.Fp8Linear(w)
    assert torch.equal(C.Fp8Matrix.quantize(x).dequantize(), x)
    for name in TYPES:
        t = getattr(torch, name)
        for src in (x.to(t), C.Fp8Matrix.quantize(x)):
            y = layer.forward(src, out_dtype=t)
            assert torch.equal(y, want.float().to(t)), (name, type(src).__name__)
    assert layer.device_status() == C.CQL_OK


GROUPED = [
    # experts, n, k, offsets
    (3, 200, 65536, [0, 2, 2, 5]), (3, 200, 65536, [0, 40, 41, 100]), (3, 200, 65536, [0, 200, 210, 500]),
    (40, 130, 1290, [min(3 * e, 90) for e in range(41)]), (5, 700, 2440, [0, 300, 300, 310, 311, 900]),
    (16, 520, 1111, [20 * e for e in range(17)]),
]


@pytest.mark.parametrize("e,n,k,off", GROUPED)
def test_whole_numbers_of_experts(e, n, k, off, cuda_dev):
    import torch
    x, w = _sides(*S.whole(np.random.default_rng(n + k), e * n, k, off[-1]), cuda_dev)
    layer = C.Fp8Experts(w.view(e, n, k))
    offsets = torch.tensor(off, dtype=torch.int32, device=cuda_dev)
    want = torch.cat([_exact(x[off[i]:off[i + 1]], w[i * n:(i + 1) * n]) for i in range(e)]).float()
    for src in (x, x.bfloat16(), C.Fp8Matrix.quantize(x)):
        assert torch.equal(layer.forward(src, offsets, out_dtype=torch.float32), want)
    assert layer.device_status() == C.CQL_OK


@pytest.mark.parametrize("n,k,tokens", [(130, 65536, 4), (130, 65536, 16), (130, 65536, 32), (130, 65536, 512), (600, 5000, 3),
                                        (600, 5000, 16), (600, 5000, 40), (300, 11008, 86), (20000, 1290, 2)])
def test_every_block_by_itself(n, k, tokens, cuda_dev):
    """Token t has values in one block alone; every block has its turn."""
    import torch
    blocks = -(-k // S.BLOCK)
    rng, layer, w = np.random.default_rng(n + k), None, None
    for first in range(0, blocks, tokens):
        mine = [(first + t) % blocks for t in range(tokens)]
        x, wn = S.one_block(rng, n if w is None else 1, k, mine)
        if w is None:
            w = torch.from_numpy(wn).to(cuda_dev)
            layer = C.Fp8Linear(w)
        x = torch.from_numpy(x).to(cuda_dev)
        want = _exact(x, w).float()
        for src in (x.bfloat16(), C.Fp8Matrix.quantize(x)):
            assert torch.equal(layer.forward(src, out_dtype=torch.float32), want), first
    assert layer.device_status() == C.CQL_OK


@pytest.mark.parametrize("n,k,tokens", [s for s in SIZES if s[1] > 1000])
@pytest.mark.parametrize("outliers", [False, True])
def test_error_in_the_norm(n, k, tokens, outliers, cuda_dev):
    import torch
    torch.manual_seed(n + k + tokens)
    w, x = torch.randn(n, k, device=cuda_dev), torch.randn(tokens, k, device=cuda_dev)
    if outliers:
        x = x * torch.where(torch.rand(k, device=cuda_dev) < 0.005, 30.0, 1.0)
    wq, xq = C.Fp8Matrix.quantize(w), C.Fp8Matrix.quantize(x)
    want = _exact(xq.dequantize(), wq.dequantize()).cpu().numpy()
    for src in (x, xq):
        y = C.Fp8Linear(wq).forward(src, out_dtype=torch.float32)
        err = S.relative_error(y.cpu().numpy(), want)
        print(f"{n}x{k} tokens {tokens}: relative error {err:.2e}")
        assert err < S.CHAIN_ERROR


def test_largest_sizes_in_whole_numbers(cuda_dev):
    """The most outputs, the most tokens: whole results."""
    import torch
    rng = np.random.default_rng(1)
    for n, k, tokens in [(1 << 20, 130, 3), (1 << 20, 130, 40), (136, 130, 1 << 20)]:
        x, w = _sides(*S.whole(rng, n, k, tokens), cuda_dev)
        y = C.Fp8Linear(w).forward(x)
        for a in range(0, n if n > tokens else tokens, 1 << 18):
            part = (slice(None), slice(a, a + (1 << 18))) if n > tokens else (slice(a, a + (1 << 18)), slice(None))
            want = _exact(x, w[part[1]]) if n > tokens else _exact(x[part[0]], w)
            assert torch.equal(y[part], want.float())
