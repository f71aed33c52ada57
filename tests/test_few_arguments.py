"""What LatentMoE.forward_few_into refuses before the library sees an address.  No GPU: a layer without a handle."""
import pytest
import torch

import latent_space_routed_b200 as lm


def layer(device="cpu"):
    """Shapes and device of a layer; nothing behind them."""
    m = object.__new__(lm.LatentMoE)
    m.cfg, m.dtype, m.device, m.handle = lm.make_config(256, 64, 128, 16, 4, 128), torch.bfloat16, torch.device(device), None
    m._few_ws, m._captured_ws, m._ws = {}, [], None
    return m


X = torch.zeros(3, 256, dtype=torch.bfloat16)
WS = torch.zeros(1 << 20, dtype=torch.uint8)


def outputs(**kw):
    return {**layer().empty_outputs(3), **kw}


@pytest.mark.parametrize("name,bad", [
    ("output", torch.zeros(2, 256, dtype=torch.bfloat16)), ("output", torch.zeros(3, 256)),
    ("output", torch.zeros(256, 3, dtype=torch.bfloat16).t()), ("output", torch.zeros(3, 512, dtype=torch.bfloat16)[:, :256]),
    ("output", torch.zeros(3, 256, dtype=torch.bfloat16, device="meta")),
    ("selected_experts", torch.zeros(3, 4, dtype=torch.int64)), ("selected_experts", torch.zeros(3, 3, dtype=torch.int32)),
    ("mixture_weights", torch.zeros(3, 4)), ("mixture_weights", torch.zeros(11, dtype=torch.bfloat16)),
    ("latent_routed_aggregate", torch.zeros(3, 63, dtype=torch.bfloat16)),
    ("latent_routed_aggregate", torch.zeros(3, 64, dtype=torch.float16))])
def test_outputs_that_do_not_fit(name, bad):
    with pytest.raises(ValueError, match=name):
        layer().forward_few_into(X, outputs(**{name: bad}), WS)


def test_tensors_of_other_devices():
    """A host pointer, or another GPU's, would fault in the kernel."""
    for x, out, ws in ((X, outputs(), WS), (X.to("meta"), outputs(), WS)):
        with pytest.raises(ValueError, match="x must be"):
            layer("cuda:0").forward_few_into(x, out, ws)
    with pytest.raises(ValueError, match="workspace"):
        layer().forward_few_into(X, outputs(), WS.to("meta"))
    with pytest.raises(ValueError, match="workspace"):
        layer().forward_few_into(X, outputs(), WS[::2])


def test_larger_buffers_reach_the_library():
    """Outputs of eight tokens serve three (the library then refuses the missing handle)."""
    with pytest.raises(lm.LmoeError) as e:
        layer().forward_few_into(X, layer().empty_outputs(8), WS)
    assert e.value.status == lm.LMOE_ERR_INVALID_ARG and "handle" in str(e.value)
