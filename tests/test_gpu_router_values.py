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


def special(name, W, x):
    """W_r, x of a case (x [4, 448]: tokens 0 and 3 stay ordinary unless W_r is what changes)."""
    R, x = W["W_r"].clone(), x.clone()
    if name == "zero rows beside large tokens":       # scores of 1/2, told apart by biases 2^-40 apart
        R[::2], R[::4] = 0.0, -0.0
        x[1:3] *= 2.0 ** 100
    elif name == "zero tokens beside large rows":
        R *= 2.0 ** 120
        x[1:3] = 0.0
    elif name == "subnormal rows beside large tokens":
        R[::2] = 2.0 ** -140
        x[1] = 2.0 ** 110
    elif name == "nan rows":
        R[5, 17], R[38, 447] = NAN, -NAN
    elif name == "infinite rows":
        R[5, 17], R[6, 40], R[38, 0], R[7, 1], R[7, 2] = INF, -INF, INF, INF, -INF
    elif name == "infinite and zero":                 # infinity times zero
        R[5, 17], x[:, 17] = INF, 0.0
    elif name == "nan token":
        x[2, 17] = NAN
    elif name == "infinite tokens":
        x[1, 0], x[2, 447], R[9, 447] = INF, -INF, 0.0
    return {**W, "W_r": R}, x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["zero rows beside large tokens", "zero tokens beside large rows",
                                  "subnormal rows beside large tokens", "nan rows", "infinite rows",
                                  "infinite and zero", "nan token", "infinite tokens"])
@pytest.mark.parametrize("T", [1, 4, 8])
def test_router_of_special_values(name, dtype, T):
    """Selections and weights of tokens and router rows with zeros, subnormals, infinities and NaN."""
    w, W, _ = make(4, 448, 64, 128, 40, 6, dtype=dtype)
    W["b"] = torch.randperm(40, generator=torch.Generator().manual_seed(1)) * 2.0 ** -40
    W, x = special(name, W, li.tokens(w))
    x = torch.cat([x, x.flip(0)])[8 - T:] if T != 1 else x[1:2]
    layer = layer_of(w, W)
    out = layer.forward_few(x.cuda())
    lm.lmoe_check_device(layer.handle, T, layer.few_workspace(T))
    check_router(out, x, W, 6)
    again = layer.forward_few(x.cuda())
    assert all(torch.equal(again[n].view(torch.uint8), out[n].view(torch.uint8)) for n in out)


def test_nan_router_rows_are_left_out_as_in_lmoe_forward():
    w, W, _ = make(8, 256, 64, 128, 16, 4)
    W = {**W, "W_r": W["W_r"].clone()}
    W["W_r"][[3, 8], 20] = NAN
    layer = layer_of(w, W)
    x = li.tokens(w).cuda()
    few, many = layer.forward_few(x), layer(x)
    assert torch.equal(few["selected_experts"], many["selected_experts"])
    assert not ((few["selected_experts"] == 3) | (few["selected_experts"] == 8)).any()
    assert torch.isfinite(few["output"]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("low", [60, 80, 100, 110, 300, 700])
def test_weights_of_scores_below_fp32(low, dtype):
    """Logits -low, -low - 1/2, ...: scores that fp32 holds roughly or not at all have the weights of their ratios."""
    w, W, _ = make(3, 256, 64, 128, 16, 6, dtype=dtype)
    x = torch.ones_like(li.tokens(w))
    W["W_r"] = (-(low + torch.arange(16).flip(0) * 0.5) / 256)[:, None].repeat(1, 256)     # exact sums
    W["b"] = torch.zeros(16)
    layer = layer_of(w, W)
    out = layer.forward_few(x.cuda())
    check_router(out, x, W, 6)
    check(out, x, W, w)
