"""4-bit tensors and products as programs call them: devices and streams that do not match, time-outs, extremes."""
import pytest
import torch

import latent_space_routed_b200 as lm
import lmoe_inputs as li

pytestmark = pytest.mark.gpu


def test_experts_of_another_device_are_refused(monkeypatch):
    w = li.custom("mx4", 4, 256, 64, 128, 16, 4, 128)
    W = {n: v.cuda() for n, v in li.weights(w).items()}
    Q = {n: lm.mx4_quantize(W[n]) for n in ("G", "U", "D")}
    with pytest.raises(ValueError, match="cuda:1"):
        Q["G"].check("G", torch.device("cuda", 1))
    assert Q["G"].check("G", torch.device("cuda", 0)) is Q["G"]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)       # the layer would be made there
    with pytest.raises(ValueError, match="G must be on cuda:1"):
        lm.LatentMoE(lm.config_for(w), {**W, **Q})


def test_streams_of_another_device_are_refused():
    """A kernel launched there would read this device's addresses."""
    s = torch.cuda.Stream()
    with pytest.raises(ValueError, match="stream"):
        lm._with(torch.device("cuda", 1), s)
    with lm._with(torch.device("cuda", 0), s):
        assert torch.cuda.current_stream() == s
    with lm._with(torch.device("cuda", 0), torch.cuda.ExternalStream(s.cuda_stream)):
        assert torch.cuda.current_stream().cuda_stream == s.cuda_stream


def operands(M=300, N=400, K=512):
    g = torch.Generator().manual_seed(3)
    return (lm.mx4_quantize(torch.randn(M, K, generator=g).cuda()), lm.mx4_quantize(torch.randn(N, K, generator=g).cuda()))


def test_a_wait_that_runs_out_is_reported():
    """Of calls without a workspace by mx4_gemm_check, whatever their stream; of one with it by its own word."""
    a, w = operands()
    want = lm.mx4_gemm(a, w)
    lm.mx4_gemm_check()
    s = torch.cuda.Stream()
    for stream in (None, s):
        lm.lmoe_debug_inject(lm.LMOE_INJECT_STALL_NEXT_MX4)
        lm.mx4_gemm(a, w, stream=stream)
        with pytest.raises(lm.LmoeError) as e:
            lm.mx4_gemm_check()
        assert e.value.status == lm.LMOE_ERR_DEVICE_TIMEOUT
        lm.mx4_gemm_check("cuda:0")                      # read and cleared
    ws = lm.mx4_gemm_workspace()
    lm.lmoe_debug_inject(lm.LMOE_INJECT_STALL_NEXT_MX4)
    lm.mx4_gemm(a, w, workspace=ws)
    lm.mx4_gemm_check()
    with pytest.raises(lm.LmoeError):
        lm.lmoe_mx4_gemm_check(ws)
    assert torch.equal(lm.mx4_gemm(a, w), want)          # the context is still usable
    lm.mx4_gemm_check()


def test_a_captured_wait_that_runs_out_is_reported():
    a, w = operands()
    want = lm.mx4_gemm(a, w)
    g, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    lm.lmoe_debug_inject(lm.LMOE_INJECT_STALL_NEXT_MX4)
    with torch.cuda.graph(g):
        lm.mx4_gemm(a, w, out=out)
    lm.mx4_gemm_check()
    g.replay()
    with pytest.raises(lm.LmoeError):
        lm.mx4_gemm_check()
    assert torch.equal(lm.mx4_gemm(a, w), want)


def test_the_layers_products_report_through_its_workspace():
    w = li.custom("mx4", 40, 256, 64, 128, 16, 4, 128)
    W = {n: v.cuda() for n, v in li.weights(w).items()}
    layer = lm.LatentMoE(lm.config_for(w), {**W, **{n: lm.mx4_quantize(W[n]) for n in ("G", "U", "D")}})
    x = li.tokens(w).cuda()
    want = layer(x)
    layer.check_device(40)
    lm.lmoe_debug_inject(lm.LMOE_INJECT_STALL_NEXT_MX4)
    layer(x)
    with pytest.raises(lm.LmoeError) as e:
        layer.check_device(40)
    assert e.value.status == lm.LMOE_ERR_DEVICE_TIMEOUT
    again = layer(x)
    layer.check_device(40)
    assert all(torch.equal(again[n], want[n]) for n in want)
