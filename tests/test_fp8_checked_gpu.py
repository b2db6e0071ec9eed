"""Quantising, reading back and the forwards under the range-checked library, at
every remainder of rows, columns and alignment: the same bytes as the ordinary
library's, clean error words."""
import pytest

import sparse_quantized_rank_b200 as C

pytestmark = pytest.mark.gpu

SHAPES = [(r, c, gap, shift) for r, c in [(1, 1), (7, 3), (8, 128), (9, 129), (3, 511), (5, 512), (17, 513), (2, 1029), (33, 2047)]
          for gap, shift in ((0, 0), (8, 0), (3, 1))]


def _both(call):
    """The results of `call` under the two libraries."""
    out = []
    for checked in (False, True):
        C.use_library(checked)
        try:
            out.append(call())
        finally:
            C.use_library(False)
    return out


@pytest.fixture(scope="module", autouse=True)
def checked_lib():
    from sparse_quantized_rank_b200 import build as b
    b.build(checked=True)


@pytest.mark.parametrize("dt", ["float32", "float16", "bfloat16"])
def test_bytes_and_values(dt, cuda_dev):
    import torch
    torch.manual_seed(1)
    t = getattr(torch, dt)
    for rows, cols, gap, shift in SHAPES:
        flat = torch.randn(shift + rows * (cols + gap), device=cuda_dev).to(t)
        src = flat[shift:].view(rows, cols + gap)[:, :cols]
        a, b = _both(lambda: C.Fp8Matrix.quantize(src))
        assert torch.equal(a.buffer, b.buffer), (rows, cols, gap)

        def read():
            out = torch.full((shift + rows * (cols + gap),), 9.0, dtype=t, device=cuda_dev)
            a.dequantize(out=out[shift:].view(rows, cols + gap)[:, :cols])
            return out
        x, y = _both(read)
        assert torch.equal(x, y), (rows, cols, gap)


@pytest.mark.parametrize("tokens", [3, 5, 30, 77])
def test_forwards(tokens, cuda_dev):
    import torch
    torch.manual_seed(tokens)
    for n, k, gap, shift in [(1, 1, 0, 0), (130, 129, 3, 1), (257, 1111, 8, 0), (640, 2050, 0, 0)]:
        layer = C.Fp8Linear(torch.randn(n, k, device=cuda_dev))
        x = torch.randn(shift + tokens * (k + gap), device=cuda_dev).bfloat16()[shift:].view(tokens, k + gap)[:, :k]
        a, b = _both(lambda: (layer.forward(x, out_dtype=torch.float32), layer.device_status()))
        assert torch.equal(a[0], b[0]) and a[1] == b[1] == C.CQL_OK
