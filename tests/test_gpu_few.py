"""The few-token layer (lmoe_forward_few) against the fp64 oracle.

Selection and its order come from 64-bit scores and have to be the oracle's.  Floating outputs of a bf16 layer are off
by the last rounding, 2^-8 of the value, and by what the sums lose: activations enter as two bf16 terms (2^-16 of a
value) or, for 4-bit experts, two halves (2^-21), weights enter exactly.  One such error is at most 2^-16 sum |a w|,
and errors of random sign add up to about 2^-16 of the row's typical value a product, three products on a path; the
bound taken is 2^-9 of the row's largest value, the 2^7 over it being for single unlucky rows.  An fp32 layer has sums
of K <= 2688 fp32 terms: sqrt(K) 2^-24 = 3.1e-6 of the row's typical value a product, 1e-5 of its largest in all.
"""
import pytest
import torch

import latent_space_routed_b200 as lm
import lmoe_inputs as li
import mx4ref
import oracle

pytestmark = pytest.mark.gpu


def make(T, d, l, f, E, k, fs=128, dtype="bf16", standard=False, act=lm.LMOE_ACT_SWIGLU, mx4=False, seed=1, gemm=0):
    w = li.custom("few", T, d, l, f, E, k, fs, dtype=dtype, seed=seed, standard=standard)
    W = li.weights(w)
    cfg = lm.config_for(w, gemm=gemm, act=act)
    if not mx4:
        return w, W, lm.LatentMoE(cfg, {n: v.cuda() for n, v in W.items()})
    Q = {n: lm.mx4_quantize(W[n].cuda()) for n in ("G", "U", "D")}
    layer = lm.LatentMoE(cfg, {**{n: v.cuda() for n, v in W.items() if n not in Q}, **Q})
    # the oracle's experts: the 4-bit values, which bf16 holds exactly
    return w, {**W, **{n: mx4ref.values(*Q[n]).to(torch.bfloat16) for n in Q}}, layer


def check(out, x, W, w, act=lm.LMOE_ACT_SWIGLU, b=None):
    Wb = W if b is None else {**W, "b": b}
    ref = oracle.forward(x, Wb, w.k, act="situ" if act else "swiglu", use_norm=not w.standard)
    sel = torch.from_numpy(ref["selected_experts"].astype("int64"))
    assert torch.equal(out["selected_experts"].cpu().long(), sel)
    for n in ("output", "mixture_weights", "latent_routed_aggregate"):
        y, r = out[n].double().cpu(), torch.from_numpy(ref[n]).double()
        top = r.abs().amax(1, keepdim=True)
        tol = 1e-5 * top if w.dtype == "f32" else 2.0 ** -8 * r.abs() + 2.0 ** -9 * top
        err = (y - r).abs()
        assert (err <= tol).all(), f"{n}: worst error over tolerance {(err / tol).max().item():.3g}"


CASES = [
    dict(T=1, d=256, l=128, f=256, E=16, k=4), dict(T=2, d=256, l=64, f=128, E=8, k=1),
    dict(T=3, d=448, l=192, f=384, E=40, k=9), dict(T=4, d=128, l=64, f=128, E=7, k=7),
    dict(T=5, d=512, l=128, f=256, E=33, k=17), dict(T=6, d=320, l=320, f=128, E=130, k=33),
    dict(T=7, d=256, l=128, f=256, E=100, k=64), dict(T=8, d=640, l=128, f=256, E=1000, k=12, fs=256),
    dict(T=8, d=256, l=256, f=256, E=16, k=5, standard=True), dict(T=1, d=1024, l=1024, f=128, E=12, k=2, standard=True),
    dict(T=3, d=256, l=128, f=256, E=16, k=4, act=1),
    dict(T=8, d=7168, l=1792, f=128, E=8, k=3), dict(T=1, d=7168, l=64, f=128, E=8, k=3),       # segments, halved K
    dict(T=7, d=4096, l=4096, f=256, E=6, k=2, fs=2688),                                        # long rows everywhere
    dict(T=1, d=2048, l=512, f=1408, E=64, k=24, fs=1408),
    dict(T=8, d=7168, l=64, f=128, E=1024, k=64),                                               # the most of everything
    dict(T=8, d=256, l=128, f=8192, E=8, k=8, fs=8192),                                         # hidden rows in segments
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
@pytest.mark.parametrize("kind", ["bf16", "mx4", "f32"])
def test_against_the_oracle(c, kind):
    w, W, layer = make(**c, dtype="f32" if kind == "f32" else "bf16", mx4=kind == "mx4")
    x = li.tokens(w)
    out = layer.forward_few(x.cuda())
    lm.lmoe_check_device(layer.handle, w.T, layer.few_workspace(w.T))
    check(out, x, W, w, c.get("act", 0))
    again = layer.forward_few(x.cuda())
    assert all(torch.equal(again[n], out[n]) for n in out)


def test_cuda_core_handle():
    w, W, layer = make(5, 256, 128, 192, 16, 4, fs=192, gemm=1)
    x = li.tokens(w)
    check(layer.forward_few(x.cuda()), x, W, w)


@pytest.mark.parametrize("E,k", [(16, 5), (300, 20), (1024, 64)])
def test_exact_ties_go_to_the_lower_index(E, k):
    """W_r = 0: every score is 1/2, the bias alone decides, in groups of equal values."""
    w, W, layer = make(3, 256, 64, 128, E, k)
    W = {**W, "W_r": torch.zeros_like(W["W_r"])}
    layer = lm.LatentMoE(lm.config_for(w), {n: v.cuda() for n, v in W.items()})
    x = li.tokens(w)
    g = torch.Generator().manual_seed(E)
    for b in (torch.zeros(E), torch.randint(0, 4, (E,), generator=g) * 2.0 ** -6, torch.arange(E) * -2.0 ** -7):
        layer.set_bias(b.float().cuda())
        check(layer.forward_few(x.cuda()), x, W, w, b=b.float())


def test_close_scores_are_told_apart():
    """Biases 2^-30 apart over equal scores: beyond fp32 at 1/2, within 64 bits."""
    w, W, _ = make(2, 256, 64, 128, 64, 8)
    W = {**W, "W_r": torch.zeros_like(W["W_r"]), "b": (torch.randperm(64, generator=torch.Generator().manual_seed(3)) * 2.0 ** -30)}
    layer = lm.LatentMoE(lm.config_for(w), {n: v.cuda() for n, v in W.items()})
    x = li.tokens(w)
    check(layer.forward_few(x.cuda()), x, W, w)


def test_all_tokens_on_the_same_experts_and_all_apart():
    w, W, layer = make(8, 256, 128, 128, 64, 4)
    b = torch.zeros(64)
    b[[3, 17, 40, 63]] = 10.0
    layer.set_bias(b.cuda())
    x = li.tokens(w)
    check(layer.forward_few(x.cuda()), x, W, w, b=b)
    x = x[:1].repeat(8, 1)                       # the same token eight times
    out = layer.forward_few(x.cuda())
    check(out, x, W, w, b=b)
    assert (out["output"] == out["output"][0]).all()


def test_zero_and_large_tokens():
    for mx4 in (False, True):
        w, W, layer = make(4, 256, 128, 256, 16, 4, mx4=mx4)
        x = li.tokens(w)
        x[0], x[1], x[2] = 0.0, x[1] * 2.0 ** 40, x[2] * 2.0 ** -60
        out = layer.forward_few(x.cuda())
        ref = oracle.forward(x, W, w.k)
        for n in ("output", "latent_routed_aggregate"):
            y, r = out[n].double().cpu(), torch.from_numpy(ref[n])
            top = r.abs().amax(1, keepdim=True)
            assert ((y - r).abs() <= 2.0 ** -8 * r.abs() + 2.0 ** -9 * top + 1e-30).all(), n


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_token_that_is_not_finite_stays_alone(mx4, bad):
    w, W, layer = make(5, 256, 128, 256, 40, 6, mx4=mx4)
    x = li.tokens(w).cuda()
    x[2, 17] = bad
    out = layer.forward_few(x)
    lm.lmoe_check_device(layer.handle, 5, layer.few_workspace(5))
    sel = out["selected_experts"]
    assert ((sel >= 0) & (sel < 40)).all() and all(len(set(r)) == 6 for r in sel.tolist())
    rows = [0, 1, 3, 4]
    assert not torch.isfinite(out["output"][2]).any()
    for n in ("output", "mixture_weights", "latent_routed_aggregate"):
        assert torch.isfinite(out[n][rows]).all()
    ref = oracle.forward(x[rows].cpu(), W, w.k)
    assert torch.equal(sel[rows].cpu().long(), torch.from_numpy(ref["selected_experts"].astype("int64")))
    y, r = out["output"][rows].double().cpu(), torch.from_numpy(ref["output"])
    assert ((y - r).abs() <= 2.0 ** -8 * r.abs() + 2.0 ** -9 * r.abs().amax(1, keepdim=True)).all()


def test_streams_graphs_and_two_calls_at_once():
    w, W, layer = make(6, 512, 128, 256, 32, 6)
    xs = [li.tokens(w, seed=i).cuda() for i in range(4)]
    want = [layer.forward_few(x) for x in xs]
    n = lm.lmoe_few_workspace_size(layer.handle, 6)
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    torch.cuda.synchronize()
    for i in range(12):
        s = streams[i % 3]
        with torch.cuda.stream(s):
            out, ws = layer.empty_outputs(6), torch.empty(n, dtype=torch.uint8, device="cuda")
            got.append((i % 4, layer.forward_few_into(xs[i % 4], out, ws), ws))
    torch.cuda.synchronize()
    for i, out, _ in got:
        assert all(torch.equal(out[k], want[i][k]) for k in out)
    x, out, ws = xs[0].clone(), layer.empty_outputs(6), torch.empty(n, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    layer.forward_few_into(x, out, ws)
    with torch.cuda.graph(g):
        layer.forward_few_into(x, out, ws)
        layer.forward_few_into(x, out, ws)
    for i in (1, 2, 3):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[i][k]) for k in out)


def test_beside_another_kernel():
    """Blocks of another stream's work take SMs: not all of the layer's blocks are resident at once."""
    w, W, layer = make(3, 512, 128, 256, 32, 6)
    x = li.tokens(w).cuda()
    want = layer.forward_few(x)
    a = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s):
            for _ in range(4):
                a @ a
        out = layer.forward_few(x)
        assert all(torch.equal(out[k], want[k]) for k in out)
    torch.cuda.synchronize()


def test_few_then_many_share_a_layer():
    """Prompt through lmoe_forward, tokens through the few-token form, bias update between: both see the new bias."""
    w, W, layer = make(8, 256, 128, 256, 16, 4)
    big = li.tokens(w, T=100).cuda()
    x = li.tokens(w)
    first = layer(big)
    b = torch.linspace(-0.5, 0.5, 16)
    layer.set_bias(b.cuda())
    check(layer.forward_few(x.cuda()), x, W, w, b=b)
    second = layer(big)
    assert not torch.equal(first["selected_experts"], second["selected_experts"])
    layer.check_device(100)


def test_shapes_refusals_and_empty():
    w, W, layer = make(8, 256, 128, 256, 16, 4)
    x = li.tokens(w).cuda()
    out = layer.forward_few(x.reshape(2, 4, 256))
    flat = layer.forward_few(x)
    assert out["output"].shape == (2, 4, 256) and torch.equal(out["output"].reshape(8, 256), flat["output"])
    assert layer.forward_few(x[:0])["output"].shape == (0, 256)
    h, ws = layer.handle, layer.few_workspace(8)
    o = [flat[n] for n in ("output", "selected_experts", "mixture_weights", "latent_routed_aggregate")]
    with pytest.raises(lm.LmoeError) as e:
        layer.forward_few(torch.zeros(9, 256, device="cuda", dtype=torch.bfloat16))
    assert e.value.status == lm.LMOE_ERR_UNSUPPORTED
    for args, status in [((x, -1, *o, ws, ws.numel()), lm.LMOE_ERR_INVALID_ARG),
                         ((None, 8, *o, ws, ws.numel()), lm.LMOE_ERR_INVALID_ARG),
                         ((x, 8, None, *o[1:], ws, ws.numel()), lm.LMOE_ERR_INVALID_ARG),
                         ((x, 8, *o, ws, lm.lmoe_few_workspace_size(h, 8) - 1), lm.LMOE_ERR_WORKSPACE),
                         ((x, 8, *o, ws.data_ptr() + 128, ws.numel()), lm.LMOE_ERR_WORKSPACE),
                         ((x.data_ptr() + 2, 7, *o, ws, ws.numel()), lm.LMOE_ERR_UNSUPPORTED)]:
        with pytest.raises(lm.LmoeError) as e:
            lm.lmoe_forward_few(h, *args)
        assert e.value.status == status
    with pytest.raises(lm.LmoeError):
        lm.lmoe_few_workspace_size(h, 9)
    assert lm.lmoe_few_workspace_size(h, 0) == 0
    for bad in (x.float(), x.t().contiguous().t(), x[:, :128], x[0]):
        with pytest.raises(ValueError, match="contiguous"):
            layer.forward_few_into(bad, flat)
    with pytest.raises(TypeError, match="all be Mx4"):
        lm.LatentMoE(layer.cfg, {**{n: v.cuda() for n, v in W.items()}, "G": lm.mx4_quantize(W["G"].cuda())})


def test_a_wait_that_runs_out_is_reported():
    w, W, layer = make(2, 256, 128, 256, 16, 4)
    x = li.tokens(w).cuda()
    want = layer.forward_few(x)
    lm.lmoe_debug_inject(lm.LMOE_INJECT_STALL_NEXT_FEW)
    layer.forward_few(x)
    with pytest.raises(lm.LmoeError) as e:
        lm.lmoe_check_device(layer.handle, 2, layer.few_workspace(2))
    assert e.value.status == lm.LMOE_ERR_DEVICE_TIMEOUT
    again = layer.forward_few(x)
    lm.lmoe_check_device(layer.handle, 2, layer.few_workspace(2))
    assert all(torch.equal(again[n], want[n]) for n in want)
