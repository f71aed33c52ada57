"""Microscaled 4-bit tensors on the GPU: quantisation, its inverse, products, and the layer with 4-bit experts,
against the definition in 64 bits (mx4ref).

Tolerances: quantisation and its inverse are exact.  A product's fp32 sum of K terms is off by at most
K 2^-24 sum |a w| (each addition rounds by at most half a step of a partial sum, which is at most sum |a w|;
the products of two 4-bit values and two powers of two are exact); a bf16 result adds half a step, 2^-8 |c|."""
import pytest
import torch

import latent_space_routed_b200 as lm
import lmoe_inputs as li
import mx4ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rand(shape, seed, dtype=torch.float32, spread=2.0):
    """Rows of their own sizes."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    return (x * torch.exp2(spread * torch.randn((*shape[:-1], 1), generator=g))).to(dtype)


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (1001, 96), (7, 8192), (2, 5, 416), (300, 512)])
def test_quantize_is_the_definition(shape, dtype):
    x = rand(shape, 1, DT[dtype])
    q = lm.mx4_quantize(x.cuda())
    c, s = mx4ref.quantize(x)
    assert torch.equal(q.codes.cpu(), c) and torch.equal(q.scales.cpu(), s)
    for out in (torch.float32, torch.bfloat16):
        y = lm.mx4_dequantize(q, out)
        assert y.dtype == out and y.shape == x.shape
        assert torch.equal(y.double().cpu(), mx4ref.values(c, s))


def special_rows():
    x = torch.zeros(12, 32)
    x[1, :9] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.0])     # every tie
    x[2] = torch.linspace(-7.9, 7.9, 32)                                            # past 6
    x[3, 0] = 2.0 ** -126                                                           # scale below its range
    x[4, :2] = torch.tensor([1e-45, -1e-45])                                        # subnormal
    x[5, 0] = 3.0e38
    x[6, 5], x[7, 6], x[8, 7] = float("inf"), float("-inf"), float("nan")
    x[9] = -0.0
    x[10, 0], x[10, 1] = 1.0, 2.0 ** -40
    x[11] = 4.0
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_special_values(dtype):
    x = special_rows().to(DT[dtype])
    q = lm.mx4_quantize(x.cuda())
    c, s = mx4ref.quantize(x)
    assert torch.equal(q.codes.cpu(), c) and torch.equal(q.scales.cpu(), s)
    y = lm.mx4_dequantize(q, torch.float32).double().cpu()
    torch.testing.assert_close(y, mx4ref.values(c, s), rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dequantize_every_code_and_scale(dtype):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    y = lm.mx4_dequantize(lm.Mx4(codes.cuda(), scales.cuda()), DT[dtype]).double().cpu()
    ref = mx4ref.values(codes, scales)
    ref = ref.to(DT[dtype]).double()                 # magnitudes past the type's largest are infinite
    torch.testing.assert_close(y, ref, rtol=0, atol=0, equal_nan=True)


def test_quantize_strided_misaligned_and_empty():
    x = rand((40, 256), 3, torch.bfloat16).cuda()
    for v in (x[:, :96], x[::2, 64:128], x[:, 1:33], x.t()[:, :32], x[3:4, :64]):
        c, s = mx4ref.quantize(v)
        q = lm.mx4_quantize(v)
        assert torch.equal(q.codes.cpu(), c) and torch.equal(q.scales.cpu(), s)
    for shape in ((0, 64), (5, 0), (0, 0)):
        q = lm.mx4_quantize(torch.empty(shape, device="cuda"))
        assert q.shape == shape and lm.mx4_dequantize(q).shape == shape


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dequantize_into_rows_of_any_alignment(dtype):
    """Row strides and starts of 16 bytes, and of 32, through the C name."""
    q = lm.mx4_quantize(rand((37, 96), 6).cuda())
    want = mx4ref.values(*q)
    per16 = 4 if dtype == "f32" else 8
    for ld, at in ((96, 0), (96, per16), (96 + per16, 0), (96 + 2 * per16, 2 * per16), (96 + 2 * per16, per16)):
        y = torch.full((37 * ld + at + 64,), 5.0, dtype=DT[dtype], device="cuda")
        lm.lmoe_mx4_dequantize(q.codes, q.scales, 37, 96, lm.LMOE_F32 if dtype == "f32" else lm.LMOE_BF16,
                               y.data_ptr() + at * y.element_size(), ld)
        rows = y[at:at + 37 * ld].view(37, ld)
        assert torch.equal(rows[:, :96].double().cpu(), want)
        assert (rows[:, 96:] == 5.0).all() and (y[:at] == 5.0).all() and (y[at + 37 * ld:] == 5.0).all()


def test_quantize_on_another_stream_and_in_a_graph():
    x = rand((65, 128), 4, torch.bfloat16).cuda()
    want = lm.mx4_quantize(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q = lm.mx4_quantize(x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r = lm.mx4_quantize(x)
            y = lm.mx4_dequantize(r)
    s.synchronize()
    x.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q.codes, want.codes)
    assert torch.equal(r.codes, lm.mx4_quantize(x).codes) and torch.equal(y, lm.mx4_dequantize(r))


# ------------------------------------------------------------------ products
def operands(M, N, K, E, seed):
    """a, w as Mx4 (GPU) and their values in 64 bits (GPU)."""
    a = lm.mx4_quantize(rand((M, K), seed).cuda())
    w = lm.mx4_quantize(rand((E, N, K) if E else (N, K), seed + 1, spread=0.5).cuda())
    return a, w, mx4ref.values(*a).cuda(), mx4ref.values(*w).cuda()


def check_product(c, ref, size, K):
    tol = K * 2.0 ** -24 * size
    if c.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    err = (c.double() - ref).abs()
    assert (err <= tol).all(), f"worst error over tolerance {(err / tol.clamp(min=1e-300)).max().item():.3g}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 64), (1, 64, 128), (5, 33, 192), (128, 192, 256), (129, 193, 320),
                                   (300, 448, 1408), (1000, 200, 64), (257, 2048, 512)])
def test_dense_product(M, N, K, dtype):
    a, w, av, wv = operands(M, N, K, 0, M + N + K)
    c = lm.mx4_gemm(a, w, dtype=DT[dtype])
    check_product(c, av @ wv.T, av.abs() @ wv.abs().T, K)
    assert torch.equal(c, lm.mx4_gemm(a, w, dtype=DT[dtype]))


def grouped_reference(av, wv, offsets):
    ref, size = torch.zeros(av.shape[0], wv.shape[1]).double().cuda(), torch.zeros(av.shape[0], wv.shape[1]).double().cuda()
    for e, (i, j) in enumerate(zip(offsets[:-1], offsets[1:])):
        ref[i:j] = av[i:j] @ wv[e].T
        size[i:j] = av[i:j].abs() @ wv[e].abs().T
    return ref, size


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,counts", [(64, 64, [0, 1, 0, 2]), (320, 448, [128, 129, 0, 1, 127]), (200, 1024, [0, 0, 300]),
                                        (512, 192, [3] * 40), (96, 128, [1] * 1024), (448, 576, [700, 5, 256])])
def test_grouped_product(N, K, counts, dtype):
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    a, w, av, wv = operands(off[-1], N, K, len(counts), K)
    c = lm.mx4_gemm(a, w, offsets=torch.tensor(off, dtype=torch.int32).cuda(), dtype=DT[dtype])
    check_product(c, *grouped_reference(av, wv, off), K)


def test_rows_of_no_expert_are_left_alone():
    """Offsets that start late, end early, descend or leave [0, M]: only real rows are written, all inside out."""
    M, N, K = 400, 96, 128
    a, w, av, wv = operands(M, N, K, 3, 9)
    for off in ([37, 100, 100, 310], [0, 400, 400, 400], [5, 5, 5, 5], [50, 20, 90, 1000], [-7, 60, -3, 70]):
        out = torch.full((M + 2, N), 7.0, device="cuda")
        lm.mx4_gemm(a, w, offsets=torch.tensor(off, dtype=torch.int32).cuda(), out=out[1:-1])
        asc, top = [], 0
        for o in off:
            top = max(top, min(max(o, 0), M))
            asc.append(top)
        ref, size = grouped_reference(av, wv, asc)
        check_product(out[1:-1][asc[0]:asc[-1]], ref[asc[0]:asc[-1]], size[asc[0]:asc[-1]], K)
        untouched = torch.ones(M + 2, dtype=torch.bool)
        untouched[1 + asc[0]:1 + asc[-1]] = False
        assert (out.cpu()[untouched] == 7.0).all()


def test_product_into_strided_and_odd_places():
    a, w, av, wv = operands(150, 100, 192, 0, 5)
    ref, size = av @ wv.T, av.abs() @ wv.abs().T
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.zeros(150, 131, dtype=dtype, device="cuda")
        lm.mx4_gemm(a, w, out=buf[:, 7:107])
        check_product(buf[:, 7:107], ref, size, 192)
        assert (buf[:, :7] == 0).all() and (buf[:, 107:] == 0).all()
    # scales that begin at an odd address
    moved = torch.empty(a.scales.numel() + 1, dtype=torch.uint8, device="cuda")[1:].view_as(a.scales).copy_(a.scales)
    check_product(lm.mx4_gemm(lm.Mx4(a.codes, moved), w, dtype=torch.float32), ref, size, 192)


def test_product_of_extreme_scales():
    """Scales of 2^-127 and 2^60 and NaN blocks stay in their rows and columns."""
    a, w, _, _ = operands(140, 200, 256, 0, 6)
    a.scales[3], a.scales[4], w.scales[7] = 0, 187, 187
    a.scales[130, 2], w.scales[199, 0] = 255, 255
    av, wv = mx4ref.values(*a).cuda(), mx4ref.values(*w).cuda()
    c = lm.mx4_gemm(a, w, dtype=torch.float32)
    ref = av @ wv.T
    assert torch.equal(torch.isnan(c), torch.isnan(ref))
    ok = ~torch.isnan(ref)
    size = (av.abs().nan_to_num(0) @ wv.abs().nan_to_num(0).T)
    assert ((c.double() - ref).abs() <= 256 * 2.0 ** -24 * size)[ok].all()


def test_two_products_at_once_and_in_a_graph():
    a, w, av, wv = operands(260, 384, 512, 0, 8)
    want = lm.mx4_gemm(a, w, dtype=torch.float32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append([lm.mx4_gemm(a, w, dtype=torch.float32) for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for os in outs for o in os)
    ws, out = lm.mx4_gemm_workspace(), torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    lm.mx4_gemm(a, w, out=out, workspace=ws)
    with torch.cuda.graph(g):
        lm.mx4_gemm(a, w, out=out, workspace=ws)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    lm.lmoe_mx4_gemm_check(ws)


def test_python_refusals_on_the_device():
    a, w, _, _ = operands(4, 8, 64, 0, 1)
    with pytest.raises(ValueError, match="K differs"):
        lm.mx4_gemm(a, lm.mx4_quantize(torch.zeros(8, 128, device="cuda")))
    with pytest.raises(ValueError, match="offsets"):
        lm.mx4_gemm(a, lm.Mx4(w.codes[None], w.scales[None]), offsets=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="whole rows"):
        lm.mx4_gemm(a, w, out=torch.empty(8, 4, device="cuda").t())
    with pytest.raises(ValueError, match="multiple of 32"):
        lm.mx4_quantize(torch.zeros(4, 48, device="cuda"))
    x = lm.mx4_quantize(torch.zeros(4, 96, device="cuda"))
    with pytest.raises(lm.LmoeError):
        lm.mx4_gemm(x, x)


# ------------------------------------------------------------------ the layer with 4-bit experts
def mx4_layer(w, act=lm.LMOE_ACT_SWIGLU):
    W = li.weights(w)
    Q = {n: lm.mx4_quantize(W[n].cuda()) for n in ("G", "U", "D")}
    layer = lm.LatentMoE(lm.config_for(w, act=act), {k: Q.get(k, v if k in Q else v.cuda()) for k, v in W.items()})
    return layer, W, Q


def gate(act, g, u):
    if act == lm.LMOE_ACT_SITU:
        return 4.0 * torch.tanh(g / 4.0) * torch.sigmoid(g) * 25.0 * torch.tanh(u / 25.0)
    return g * torch.sigmoid(g) * u


@pytest.mark.parametrize("T,d,l,f,E,k,act,standard", [
    (1, 256, 128, 256, 16, 4, 0, False), (2, 256, 64, 128, 8, 3, 0, False), (9, 256, 192, 384, 24, 5, 1, False),
    (200, 512, 256, 256, 32, 6, 0, False), (700, 256, 256, 128, 16, 4, 0, True), (33, 448, 64, 128, 40, 7, 1, False)])
def test_layer_stages(T, d, l, f, E, k, act, standard):
    """lmoe_forward's 4-bit stages, each from the one before: slot rows quantised exactly; the hidden's codes those
    of the gate in 64 bits, but for values next to a rounding border; the weighted rows within bf16; and the sum."""
    w = li.custom("mx4", T, d, l, f, E, k, 128, seed=T, standard=standard)
    layer, W, Q = mx4_layer(w, act)
    out = layer(li.tokens(w).cuda())
    layer.check_device(T)
    S = T * k
    assert layer.launch_count(T) > 0
    Zp = layer.region(T, "Zp", torch.bfloat16, (S, l))
    c, s = mx4ref.quantize(Zp)
    zc, zs = layer.region(T, "Zp4", torch.uint8, (S, l // 2)), layer.region(T, "Zp4_scales", torch.uint8, (S, l // 32))
    assert torch.equal(zc.cpu(), c) and torch.equal(zs.cpu(), s)
    off = layer.region(T, "offsets", torch.int32, (E + 1,)).tolist()
    z = mx4ref.values(c, s).cuda()
    val = {n: mx4ref.values(*Q[n]).cuda() for n in Q}
    h, hg, hu = (torch.zeros(S, f).double().cuda() for _ in range(3))
    for e in range(E):
        i, j = off[e], off[e + 1]
        g, u = z[i:j] @ val["G"][e].T, z[i:j] @ val["U"][e].T
        h[i:j] = gate(act, g, u)
        # |dh| <= |d act/dg| dg + |d act/du| du with dg, du <= l 2^-24 sum |a w|, slopes at most 1.1 |u| + ... taken as
        # (1 + |u|) and (1 + |g|), and 2^-21 |h| for the gate's own fp32 functions
        dg, du = z[i:j].abs() @ val["G"][e].abs().T, z[i:j].abs() @ val["U"][e].abs().T
        hg[i:j] = l * 2.0 ** -24 * (dg * (1.2 + 1.2 * u.abs()) + du * (1.2 + 1.2 * g.abs())) + 2.0 ** -21 * h[i:j].abs()
    hc, hs = layer.region(T, "H4", torch.uint8, (S, f // 2)), layer.region(T, "H4_scales", torch.uint8, (S, f // 32))
    got = mx4ref.values(hc, hs).cuda()
    lo, hi = mx4ref.values(*mx4ref.quantize(h - hg)).cuda(), mx4ref.values(*mx4ref.quantize(h + hg)).cuda()
    mid = mx4ref.values(*mx4ref.quantize(h)).cuda()
    agree = got == mid
    # elsewhere the error bar crosses a border of the value or of its block's scale: one step either way
    step = torch.exp2(hs.double().cuda() - 127.0).repeat_interleave(32, 1) * 2.0
    assert agree.double().mean() > 0.99
    assert ((got - mid).abs() <= 2 * step + (hi - lo).abs())[~agree].all()
    p = layer.region(T, "p32", torch.float32, (T, k)).double()
    slot = layer.region(T, "slot_of", torch.int32, (T, k)).long()
    weight = torch.zeros(S).double().cuda()
    weight[slot.reshape(-1)] = p.reshape(-1)
    y, size = torch.zeros(S, l).double().cuda(), torch.zeros(S, l).double().cuda()
    for e in range(E):
        i, j = off[e], off[e + 1]
        y[i:j] = got[i:j] @ val["D"][e].T
        size[i:j] = got[i:j].abs() @ val["D"][e].abs().T
    y, size = y * weight[:, None], size * weight[:, None]
    Y = layer.region(T, "Y", torch.bfloat16, (S, l)).double()
    assert ((Y - y).abs() <= 2.0 ** -8 * y.abs() + (f + 2) * 2.0 ** -24 * size).all()
    u = Y[slot.reshape(-1)].reshape(T, k, l).sum(1)
    rows = Y[slot.reshape(-1)].reshape(T, k, l).abs().sum(1)
    assert ((out["latent_routed_aggregate"].double() - u).abs() <= 2.0 ** -8 * u.abs() + k * 2.0 ** -24 * rows).all()
    assert torch.isfinite(out["output"]).all()
    again = layer(li.tokens(w).cuda())
    assert all(torch.equal(again[n], out[n]) for n in out)


def test_nan_blocks_of_the_experts_reach_their_tokens_only():
    """A block of scale 255 stands for NaN whatever its codes: in the few-token form and in the other."""
    w = li.custom("mx4", 40, 256, 128, 256, 16, 4, 128, seed=3)
    W = li.weights(w)
    x = li.tokens(w).cuda()
    for name, at in (("G", (5, 17, 3)), ("U", (5, 0, 0)), ("D", (5, 127, 7))):
        Q = {n: lm.mx4_quantize(W[n].cuda()) for n in ("G", "U", "D")}
        Q[name].scales[at] = 255
        layer = lm.LatentMoE(lm.config_for(w), {**{n: v.cuda() for n, v in W.items() if n not in Q}, **Q})
        for out in (layer(x), layer.forward_few(x[:8]), layer.forward_few(x[3:4])):
            has = (out["selected_experts"] == 5).any(1)
            assert torch.equal(torch.isnan(out["latent_routed_aggregate"]).any(1), has)
            assert torch.equal(torch.isnan(out["output"]).any(1), has)


def test_layer_host_and_noalloc_forms():
    w = li.custom("mx4", 40, 256, 128, 256, 16, 4, 128, seed=2)
    layer, _, _ = mx4_layer(w)
    x = li.tokens(w)
    want = layer(x.cuda())
    host = layer.forward_host(x.pin_memory(), layer.empty_outputs(40, "cpu", pin=True))
    out = layer.empty_outputs(40)
    xc = x.cuda()
    lm.lmoe_forward_noalloc(layer.handle, xc, 40, *(out[n] for n in ("output", "selected_experts", "mixture_weights",
                                                                    "latent_routed_aggregate")))
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(host[n], want[n].cpu()) and torch.equal(out[n], want[n])


def test_layer_in_a_graph_and_launch_count():
    from torch.profiler import ProfilerActivity, profile
    w = li.custom("mx4", 48, 256, 128, 256, 16, 4, 128, seed=5)
    layer, _, _ = mx4_layer(w)
    xs = [li.tokens(w, seed=i).cuda() for i in range(2)]
    want = [layer(x) for x in xs]
    x, out = xs[0].clone(), layer.empty_outputs(48)
    layer.forward_into(x, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward_into(x, out)
    x.copy_(xs[1])
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], want[1][n]) for n in out)
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        layer.forward_into(x, out)
        torch.cuda.synchronize()
    kernels = [e for e in p.events() if "lmoe" in e.name and "cuda" not in e.name.lower()[:4]]
    assert len(kernels) == layer.launch_count(48)


def test_prompt_then_tokens():
    """A prompt through lmoe_forward and its first tokens again through the few-token form, on one 4-bit layer: the
    same experts, and results apart by the 4-bit rounding of z and H that only the former has.

    How far: in a block of 32 normal values scaled so that the largest lies in [4, 8), sigma is 1.8 to 3.6; the steps
    1/2, 1 and 2 below 2, 4 and 6 leave a variance of step^2 / 12 each, and what lies past 6 about 1.  With the
    shares of a normal variable that is 0.73/48 + 0.24/12 + 0.026/3 = 0.044 at sigma 1.8 and 0.42/48 + 0.31/12 +
    0.17/3 + 0.095 = 0.19 at 3.6: 0.12 of sigma at both ends.  g and u get 0.12 each from z; silu multiplies a
    relative error by 1 to 2, say 1.5, so their product has sqrt(0.18^2 + 0.12^2) = 0.22; H, with longer tails, adds
    about 0.14 of its own: 0.26 in the root mean square.  Rows of 256 values spread by some hundredths around that;
    half as much again is 0.4."""
    w = li.custom("mx4", 64, 512, 256, 512, 32, 6, 256, seed=11)
    layer, _, _ = mx4_layer(w)
    x = li.tokens(w).cuda()
    big, few = layer(x), layer.forward_few(x[:8])
    assert torch.equal(big["selected_experts"][:8].sort(1)[0], few["selected_experts"].sort(1)[0])
    a, b = big["latent_routed_aggregate"][:8].double(), few["latent_routed_aggregate"].double()
    assert ((a - b).norm(dim=1) <= 0.4 * b.norm(dim=1)).all()
    layer.check_device(64)
