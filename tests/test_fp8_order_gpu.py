"""Weights and offsets written right before the forward that reads them, on the
paths that read before the kernels in front of them are complete."""
import numpy as np
import pytest

import sparse_quantized_rank_b200 as C

pytestmark = pytest.mark.gpu


def _random(rng, *shape):
    import torch
    return torch.from_numpy(rng.standard_normal(shape)).float().cuda()


@pytest.mark.parametrize("n,k,tokens", [(640, 2048, 3), (300, 5000, 12), (1024, 1111, 100), (4096, 1024, 300)])
def test_requantised_weight(n, k, tokens, cuda_dev):
    """The same buffer quantised anew before every forward: x quantised inside
    the product kernel, before it, and kept, few tokens and the pair kernel."""
    import torch
    rng = np.random.default_rng(n + tokens)
    ws, x = [_random(rng, n, k) for _ in range(3)], _random(rng, tokens, k).bfloat16()
    xq = C.Fp8Matrix.quantize(x)
    want = [[C.Fp8Linear(w).forward(v, out_dtype=torch.bfloat16) for v in (x, xq)] for w in ws]
    layer = C.Fp8Linear(ws[0])
    torch.cuda.synchronize()
    m, got = layer.weight, []
    for i in range(60):
        C.cql_fp8_quantize(ws[i % 3], C.CQL_DT_F32, n, k, k, m.buffer, m.nbytes)
        got.append(layer.forward((x, xq)[i % 2], out_dtype=torch.bfloat16))
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 3][i % 2]), i
    assert layer.device_status() == C.CQL_OK


@pytest.mark.parametrize("tokens", [6, 90, 600])
def test_requantised_experts_and_new_offsets(tokens, cuda_dev):
    """Offsets and the experts' weight rewritten before every forward."""
    import torch
    rng = np.random.default_rng(tokens)
    e, n, k = 3, 200, 1500
    ws, x = [_random(rng, e * n, k) for _ in range(2)], _random(rng, tokens, k).bfloat16()
    offs = [torch.tensor([0, tokens // a, tokens // 2, tokens], dtype=torch.int32, device=cuda_dev) for a in (6, 3, 2)]
    xq = C.Fp8Matrix.quantize(x)
    want = [[C.Fp8Experts(w.view(e, n, k)).forward(v, o, out_dtype=torch.float32) for o in offs for v in (x, xq)]
            for w in ws]
    layer, box = C.Fp8Experts(ws[0].view(e, n, k)), torch.zeros_like(offs[0])
    torch.cuda.synchronize()
    m, got = layer.weight, []
    for i in range(60):
        box.copy_(offs[i % 3])
        C.cql_fp8_quantize(ws[i % 2], C.CQL_DT_F32, e * n, k, k, m.buffer, m.nbytes)
        got.append(layer.forward((x, xq)[i // 3 % 2], box, out_dtype=torch.float32))
        box.copy_(offs[(i + 1) % 3])
        got.append(layer.forward(x, box, out_dtype=torch.float32))
    for i in range(60):
        assert torch.equal(got[2 * i], want[i % 2][2 * (i % 3) + i // 3 % 2]), i
        assert torch.equal(got[2 * i + 1], want[i % 2][2 * ((i + 1) % 3)]), i
    assert layer.device_status() == C.CQL_OK


def test_weight_copied_in_with_an_operation_between(cuda_dev):
    """A weight buffer written by a copy: anything that is not a forward in
    between makes the next forward safe."""
    import torch
    rng = np.random.default_rng(7)
    ms = [C.Fp8Matrix.quantize(_random(rng, 700, 1300)) for _ in range(3)]
    other, x = C.Fp8Linear(_random(rng, 512, 1300)), _random(rng, 2, 1300).bfloat16()
    want = [C.Fp8Linear(m).forward(x) for m in ms]
    layer, flag = C.Fp8Linear(C.Fp8Matrix(700, 1300, ms[0].buffer.clone())), torch.zeros(1, device=cuda_dev)
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        layer.weight.buffer.copy_(ms[i % 3].buffer)
        flag.add_(1)
        other.forward(x)
        got.append(layer.forward(x))
    assert all(torch.equal(y, want[i % 3]) for i, y in enumerate(got))
    assert layer.device_status() == C.CQL_OK
