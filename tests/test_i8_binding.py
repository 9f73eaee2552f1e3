"""What the binding of the per-token int8 operators needs of torch."""
import pytest
import torch

import block_quantized_int8_q8_amd as mmq


@pytest.fixture
def calls(monkeypatch):
    """What the binding looks up in a torch without two private names."""
    with monkeypatch.context() as m:
        for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
            m.delattr(torch._C, name, raising=False)
        c = mmq._Calls()
    monkeypatch.setattr(mmq, "_calls", c)
    return c


def test_binding_without_torchs_private_names(calls, monkeypatch):
    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(torch.cuda, "current_stream", lambda i: Stream)
    assert calls.current_device is torch.cuda.current_device and calls.raw_stream(0) == 77


@pytest.mark.gpu
def test_calls_without_torchs_private_names(calls):
    x = torch.randn((5, 64), generator=torch.Generator().manual_seed(1)).to("cuda:0")
    q, s = mmq.quantize_i8(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                      # the current stream and a named one
        a = mmq.gemm_i8(q, s, q, s)
        b = mmq.gemm_i8(q, s, q, s, stream=side)
    torch.cuda.synchronize()
    want = (q.cpu().double() @ q.cpu().double().T).float() * s.cpu()[:, None] * s.cpu()
    assert torch.equal(a.cpu(), want) and torch.equal(b.cpu(), want)
