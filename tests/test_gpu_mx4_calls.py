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
