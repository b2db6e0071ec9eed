"""Bounded waits of the FP8 product kernels that run out.

With CQL_FLAG_DEBUG_SKIP_X a forward withholds x, so that every role that waits
for it, or for what follows from it, gives up after about 10 ms: the call ends,
the error word says CQL_ERR_TIMEOUT with the detail of a role of that kernel, and
the next ordinary call on the same memory is right.  What was copied has landed
by then; the MMAs that were issued read memory of their own CTA."""
import pytest

import sparse_quantized_rank_b200 as C

pytestmark = pytest.mark.gpu

FEW, PAIR = range(40, 44), range(44, 48)

CASES = [
    # n, k, tokens, x's type, details
    (128, 256, 1, "bf16", FEW),                # one tile, two blocks: every copy is issued before the waits
    (256, 4096, 3, "f32", FEW),                # quantised on the way, columns split over a cluster
    (40000, 1000, 2, "f16", FEW),              # more tiles than CTAs
    (300, 6000, 16, "bf16", FEW),              # copied x, split
    (40000, 2500, 12, "bf16", FEW),            # copied x, whole tiles
    (512, 4096, 30, "bf16", FEW),              # 32 tokens a tile
    (300, 200, 70, "bf16", PAIR),              # one unit
    (4096, 4096, 200, "bf16", PAIR),           # units of two blocks
    (9000, 2300, 700, "f16", PAIR),            # units of one, more tiles than pairs
]


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("n,k,tokens,dt,details", CASES)
def test_withheld_x_is_reported(n, k, tokens, dt, details, kept, cuda_dev):
    import torch
    types = {"f32": (torch.float32, C.CQL_DT_F32), "f16": (torch.float16, C.CQL_DT_F16), "bf16": (torch.bfloat16, C.CQL_DT_BF16)}
    torch.manual_seed(n + tokens)
    layer = C.Fp8Linear(torch.randn(n, k, device=cuda_dev))
    x = torch.randn(tokens, k, device=cuda_dev).to(types[dt][0])
    src = C.Fp8Matrix.quantize(x) if kept else x
    want = layer.forward(src, out_dtype=torch.float32)
    assert layer.device_status() == C.CQL_OK
    y = torch.empty_like(want)
    x_dt, ldx, at = (C.CQL_DT_FP8_BLOCK, 0, src.buffer) if kept else (types[dt][1], k, x)
    size = C.cql_fp8_workspace_size(k, 1, tokens)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device=cuda_dev)
    call = lambda flag: C.cql_fp8_linear_forward(n, k, layer.weight.buffer, at, x_dt | flag, ldx, y, C.CQL_DT_F32, n, tokens,  # noqa: E731
                                                 ws, size, layer.status)
    for _ in range(2):
        call(C.CQL_FLAG_DEBUG_SKIP_X)
        torch.cuda.synchronize()
        assert int(layer.status[1]) in details
        assert layer.device_status() == C.CQL_ERR_TIMEOUT and layer.device_status() == C.CQL_OK
        y.fill_(7)
        call(0)
        assert torch.equal(y, want) and layer.device_status() == C.CQL_OK


@pytest.mark.parametrize("tokens,details", [(24, FEW), (150, FEW), (500, PAIR)])
def test_withheld_x_of_experts(tokens, details, cuda_dev):
    import torch
    torch.manual_seed(tokens)
    e, n, k = 7, 520, 1500
    layer = C.Fp8Experts(torch.randn(e, n, k, device=cuda_dev))
    x = torch.randn(tokens, k, device=cuda_dev).bfloat16()
    off = torch.tensor([0, 2, 2, 9, 11, 11, 20, tokens], dtype=torch.int32, device=cuda_dev)
    want = layer.forward(x, off, out_dtype=torch.float32)
    y = torch.empty_like(want)
    size = C.cql_fp8_workspace_size(k, e, tokens)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device=cuda_dev)
    call = lambda flag: C.cql_fp8_grouped_forward(n, k, e, layer.weight.buffer, x, C.CQL_DT_BF16 | flag, k, off, y,  # noqa: E731
                                                  C.CQL_DT_F32, n, tokens, ws, size, layer.status)
    call(C.CQL_FLAG_DEBUG_SKIP_X)
    torch.cuda.synchronize()
    assert int(layer.status[1]) in details and layer.device_status() == C.CQL_ERR_TIMEOUT
    call(0)
    assert torch.equal(y, want) and layer.device_status() == C.CQL_OK
