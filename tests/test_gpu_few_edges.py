"""The few-token layer's router where values leave the ordinary range: NaN, infinities, zeros beside large values and
scores below fp32, against the router's formulas in 64 bits (biased scores that are NaN count as the lowest, as in
lmoe_forward).

Tolerance of the mixture weights: each is one quotient rounded to fp32, of scores rounded to fp32 (half a step each)
and their sum of k terms (half a step per addition), so (k + 2) 2^-24 of its value, and 2^-8 more in bf16."""
import pytest
import torch

import latent_space_routed_b200 as lm
import lmoe_inputs as li
from test_gpu_few import check, make

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
FLT_MAX = torch.finfo(torch.float32).max


def router64(x, W, k):
    """(scores, selected experts, mixture weights) in 64 bits."""
    r = 1.0 / (1.0 + torch.exp(-(x.double() @ W["W_r"].double().T)))
    key = torch.nan_to_num(r + W["b"].double(), nan=-INF, posinf=INF, neginf=-INF).clamp(min=-FLT_MAX)
    sel = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]
    p = r.gather(1, sel)
    return r, sel, p / p.sum(1, keepdim=True)


def check_router(out, x, W, k):
    _, sel, p = router64(x, W, k)
    assert torch.equal(out["selected_experts"].cpu().long(), sel)
    got = out["mixture_weights"]
    rel = (k + 2) * 2.0 ** -24 + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0)
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(p))
    ok = ~torch.isnan(p)
    assert ((got - p).abs() <= rel * p.abs())[ok].all()
    return sel


def layer_of(w, W):
    return lm.LatentMoE(lm.config_for(w), {n: v.cuda() for n, v in W.items()})


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [3, 13, 15, 16])
def test_biases_that_are_not_numbers_come_last(dtype, k):
    w, W, _ = make(3, 256, 64, 128, 16, k, dtype=dtype)
    W["b"] = W["b"].clone()
    W["b"][[2, 9]], W["b"][4], W["b"][11] = NAN, -INF, -NAN
    layer = layer_of(w, W)
    x = li.tokens(w)
    sel = check_router(layer.forward_few(x.cuda()), x, W, k)
    assert torch.equal(layer(x.cuda())["selected_experts"].cpu().long(), sel)       # lmoe_forward's rule
