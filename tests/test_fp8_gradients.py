"""The FP8 layers have no backward pass: a forward whose gradient would be lost is
refused, one that asks for none is not."""
import pytest

import sparse_quantized_rank_b200 as C


class _Stub(C._Fp8Layer):
    """A layer's checks without a GPU: its launch only says that it was reached."""

    def __init__(self, device):
        import torch
        self.n_experts, self.n_out, self.k_in, self.device, self._index = 1, 3, 5, device, None
        self.weight = type("W", (), {"buffer": torch.zeros(1)})
        C._fp8_types()

    def _launch(self, *a):
        return "launched"


@pytest.fixture()
def stub(monkeypatch):
    import torch
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: None, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    from sparse_quantized_rank_b200 import build
    build.build()
    return _Stub(torch.device("cpu"))


def test_refusals(stub):
    import torch
    x, out = torch.zeros(2, 5), torch.zeros(2, 3)
    for t in (x.clone().requires_grad_(), x.clone().requires_grad_() * 2):
        with pytest.raises(ValueError, match="x requires grad"):
            stub._call(t, None, None, None, None)
        with torch.no_grad():
            assert stub._call(t, None, None, None, None) == "launched"
        with torch.inference_mode():
            assert stub._call(t, None, None, None, None) == "launched"
        assert stub._call(t.detach(), None, None, None, None) == "launched"
    with pytest.raises(ValueError, match="out requires grad"):
        stub._call(x, None, None, out.requires_grad_(), None)
    assert stub._call(x, None, None, out.detach(), None) == "launched"


@pytest.mark.gpu
def test_refusals_of_the_layers(cuda_dev):
    import torch
    lin = torch.nn.Linear(40, 24, bias=False, device=cuda_dev)
    layer, experts = C.Fp8Linear(lin.weight), C.Fp8Experts(torch.stack([lin.weight, lin.weight]))   # weights may be parameters
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=cuda_dev)
    x = torch.randn(4, 40, device=cuda_dev)
    want = layer.forward(x)
    history = x.clone().requires_grad_() * 1
    for call in (lambda t: layer.forward(t), lambda t: experts.forward(t, off)):
        with pytest.raises(ValueError, match="no backward pass"):
            call(history)
        with torch.no_grad():
            assert torch.equal(call(history), want)
        assert torch.equal(call(history.detach()), want) and not call(x).requires_grad
    assert torch.equal(layer.forward(C.Fp8Matrix.quantize(x)), want.bfloat16())
