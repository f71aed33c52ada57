"""Workloads of the few-token layer and of microscaled 4-bit tensors.

Three operators, each in a plain form (elementary torch operations) and, with
``own`` set, as the calls a user makes of this package:

``few``       the whole layer for 1 to 8 tokens (``LatentMoE.forward_few_into``): router, top-k, down-projection,
              routed experts, combine, RMSNorm, up-projection and shared experts, from weights in the token
              type or with the routed experts in 4 bits;
``quantize``  rows to microscaled 4-bit values (blocks of 32 along a row, each with a power-of-two scale) and
              back (``mx4_quantize``, ``mx4_dequantize``);
``product``   the product of two such matrices, dense or grouped by expert (``mx4_gemm``).

A 4-bit tensor is its codes [..., rows, cols / 2] (uint8, the even column in the low half) and its scales
[..., rows, cols / 32] (uint8, the biased exponent e of 2^(e - 127)).  A code is a sign bit over a magnitude out
of 0, 1/2, 1, 3/2, 2, 3, 4, 6.  A block's scale is 2^(floor(log2 of its largest magnitude) - 2), so that its
largest value falls in [4, 8); values round to the nearest magnitude, ties to the even code, those past 6 to 6.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _few(name, T, d, l, f, E, k, f_s, dtype="bf16", experts="same", act="swiglu", standard=False):
    c = dict(op="few", T=T, d=d, l=l, f=f, E=E, k=k, f_s=f_s, dtype=dtype, experts=experts, act=act, standard=standard)
    return dict(c, name=name) if name else c


def _quantize(name, rows, cols, dtype):
    c = dict(op="quantize", rows=rows, cols=cols, dtype=dtype)
    return dict(c, name=name) if name else c


def _product(name, M, N, K, E, dtype="bf16"):
    """E = 0: dense; otherwise M rows sorted by expert, E experts."""
    c = dict(op="product", M=M, N=N, K=K, E=E, dtype=dtype)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a handful of tokens through a toy layer in fp32: nothing but latency
        _few("few tiny fp32 T3", 3, 128, 64, 256, 16, 4, 256, dtype="f32"),
        # one token of a chat: the d = 2048 layer with many small experts
        _few("few d2048 T1", 1, 2048, 512, 1408, 256, 24, 1408),
        # the standard form of that layer (experts at the model width), SiTU gate, an odd batch of requests
        _few("few standard d2048 T5 situ", 5, 2048, 2048, 1408, 64, 6, 1408, act="situ", standard=True),
        # one token, and a batch of eight, of the widest layer: what decoding is bounded by
        _few("few d7168 T1", 1, 7168, 1792, 2048, 384, 32, 2048),
        _few("few d7168 T8", 8, 7168, 1792, 2048, 384, 32, 2048),
        # the same with the routed experts in 4 bits
        _few("few d7168 T1 mx4", 1, 7168, 1792, 2048, 384, 32, 2048, experts="mx4"),
        _few("few d7168 T6 mx4", 6, 7168, 1792, 2048, 384, 32, 2048, experts="mx4"),
        # the latent rows of a short, odd prompt; and a stack of expert weights from its fp32 master copy
        _quantize("quantize latents", 1001, 512, "bf16"),
        _quantize("quantize weights", 256 * 1408, 512, "f32"),
        # a whole projection at the model width; gate and up of a prompt's slot rows over 512 experts; and those
        # of 32 decoding requests, where each touched expert has a few rows
        _product("product dense", 4096, 2048, 2048, 0),
        _product("product prompt", 196608, 5376, 1024, 512),
        _product("product decode T32", 1024, 4096, 1792, 384, dtype="f32"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("few", "few", "quantize", "product", "product"))
    if op == "quantize":
        cols = _log(rng, 64, 8192, 32)
        rows = _log(rng, 1, max(1, min(400000, 150_000_000 // cols)))
        return _quantize(None, rows, cols, rng.choice(("bf16", "f32")))
    if op == "product":
        N, K = _log(rng, 64, 5376, 64), _log(rng, 128, 4096, 64)
        E = rng.choice((0, rng.randint(2, 300)))
        most = int(2e11 / (N * K)) if E else int(4e10 / (N * K))
        M = _log(rng, 1, max(2, min(60000, most)))
        return _product(None, M, N, K, E, rng.choice(("bf16", "bf16", "f32")))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    experts = rng.choice(("same", "mx4")) if dtype == "bf16" else "same"
    T = rng.randint(1, 8)
    E = _log(rng, 8, 256)
    k = rng.randint(1, min(32, E))
    d = _log(rng, 256, 4096, 64)
    standard = rng.random() < 0.25
    l = d if standard else max(64, min(2048, d // rng.choice((2, 4, 8)) // 64 * 64))
    f, f_s = _log(rng, 128, 2048, 128), _log(rng, 128, 2048, 128)
    if standard:
        E = min(E, 64)
        k = min(k, E)
    return _few(None, T, d, l, f, E, k, f_s, dtype, experts, rng.choice(("swiglu", "situ")), standard)


# ------------------------------------------------------------------ plain form: 4-bit values
def _magnitudes(device, dtype=torch.float32):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=dtype, device=device)


def _plain_quantize(x):
    """(codes, scales) of x [..., cols]."""
    b = x.float().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = b.abs().amax(-1)
    e = (torch.frexp(top)[1] - 3).clamp(min=-127)                  # floor(log2 top) - 2
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    v = torch.ldexp(b, -e.unsqueeze(-1).to(b.dtype))               # exact: a power of two
    a = v.abs()
    # nearest of the eight magnitudes; a tie goes to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(v)).to(torch.uint8).reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _plain_dequantize(codes, scales):
    """fp32 values [..., cols]."""
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(*scales.shape, 32)
    m = _magnitudes(codes.device)[(c & 7).long()]
    m = torch.where(c >= 8, -m, m)
    v = torch.ldexp(m, (scales.to(torch.int32) - 127).unsqueeze(-1).to(m.dtype))
    return v.reshape(*codes.shape[:-1], codes.shape[-1] * 2)


# ------------------------------------------------------------------ inputs
def _gen(seed, k=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1009 + k)
    return g


def _normal(shape, std, g, dtype):
    t = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    return t.mul_(std) if std != 1.0 else t


def _expert_stack(E, rows, cols, g, dtype, mx4):
    """[E, rows, cols] ~ N(0, 1 / cols): a tensor, or (codes, scales)."""
    if not mx4:
        return _normal((E, rows, cols), cols ** -0.5, g, dtype)
    codes = torch.empty((E, rows, cols // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, rows, cols // 32), dtype=torch.uint8, device="cuda")
    for e in range(0, E, 32):
        codes[e:e + 32], scales[e:e + 32] = _plain_quantize(
            _normal((min(32, E - e), rows, cols), cols ** -0.5, g, torch.float32))
    return codes, scales


def _counts(E, M, seed):
    """Rows of each expert: uneven, some possibly none."""
    r = np.random.RandomState(seed % (1 << 31))
    return r.multinomial(M, r.dirichlet(np.full(E, 8.0)))


def prepare(case, seed):
    op = case["op"]
    if op == "quantize":
        # activations and weights alike are near normal, each row of its own size
        g = _gen(seed)
        x = _normal((case["rows"], case["cols"]), 1.0, g, torch.float32)
        x.mul_(torch.exp2(_normal((case["rows"], 1), 2.0, g, torch.float32)))
        return {"case": case, "x": x.to(_DT[case["dtype"]])}
    if op == "product":
        g = _gen(seed)
        M, N, K, E = (case[n] for n in ("M", "N", "K", "E"))
        s = {"case": case, "a": _plain_quantize(_normal((M, K), 1.0, g, torch.float32))}
        w = _expert_stack(max(E, 1), N, K, g, None, True)
        s["w"] = w if E else tuple(t[0] for t in w)
        if E:
            counts = _counts(E, M, seed)
            s["most"] = int(counts.max())
            s["offsets"] = torch.tensor(np.concatenate(([0], np.cumsum(counts))), dtype=torch.int32, device="cuda")
        if own:
            import latent_space_routed_b200 as lm
            s["lm"] = lm
            s["a"], s["w"] = lm.Mx4(*s["a"]), lm.Mx4(*s["w"])
            s["out"] = torch.empty(M, N, dtype=_DT[case["dtype"]], device="cuda")
            s["workspace"] = lm.mx4_gemm_workspace()
        return s
    T, d, l, f, E, f_s = (case[n] for n in ("T", "d", "l", "f", "E", "f_s"))
    dt, mx4, g = _DT[case["dtype"]], case["experts"] == "mx4", _gen(seed)
    w = {"W_r": _normal((E, d), d ** -0.5, g, torch.float32),
         "b": torch.rand(E, generator=g, device="cuda") * 0.1 - 0.05,
         "G": _expert_stack(E, f, l, g, dt, mx4), "U": _expert_stack(E, f, l, g, dt, mx4),
         "D": _expert_stack(E, l, f, g, dt, mx4),
         "Gs": _normal((2, f_s, d), d ** -0.5, g, dt), "Us": _normal((2, f_s, d), d ** -0.5, g, dt),
         "Ds": _normal((2, d, f_s), f_s ** -0.5, g, dt)}
    if not case["standard"]:
        w["W_down"], w["W_up"] = _normal((l, d), d ** -0.5, g, dt), _normal((d, l), l ** -0.5, g, dt)
    s = {"case": case, "x": _normal((T, d), 1.0, g, dt), "w": w}
    if own:
        import latent_space_routed_b200 as lm
        if mx4:
            w = dict(w, **{n: lm.Mx4(*w[n]) for n in ("G", "U", "D")})
        cfg = lm.make_config(d, l, f, E, case["k"], f_s, dtype=lm.LMOE_F32 if case["dtype"] == "f32" else lm.LMOE_BF16,
                             act=lm.LMOE_ACT_SITU if case["act"] == "situ" else lm.LMOE_ACT_SWIGLU,
                             standard=int(case["standard"]))
        layer = lm.LatentMoE(cfg, w)
        s = {"case": case, "x": s["x"], "layer": layer, "out": layer.empty_outputs(T)}
    return s


# ------------------------------------------------------------------ one pass
def _gate(act, g, v):
    if act == "situ":
        return 4.0 * torch.tanh(g / 4.0) / (1 + torch.exp(-g)) * (25.0 * torch.tanh(v / 25.0))
    return g / (1 + torch.exp(-g)) * v


def _rows_of(w, i):
    """Experts i of a stack, in fp32."""
    return _plain_dequantize(w[0][i], w[1][i]) if isinstance(w, tuple) else w[i].float()


def _plain_few(case, x, w):
    T, d, k, dt, act = case["T"], case["d"], case["k"], _DT[case["dtype"]], case["act"]
    # the selection hangs on which scores are larger: in 64 bits
    r = 1 / (1 + torch.exp(-(x.double() @ w["W_r"].double().T)))
    sel = torch.sort(r + w["b"].double(), dim=1, descending=True, stable=True)[1][:, :k]
    p = r.gather(1, sel)
    p = (p / p.sum(1, keepdim=True)).float()
    xf = x.float()
    z = xf if case["standard"] else xf @ w["W_down"].float().T
    i = sel.reshape(-1)
    zs = z.repeat_interleave(k, 0).unsqueeze(2)                     # [T k, l, 1]
    h = _gate(act, _rows_of(w["G"], i) @ zs, _rows_of(w["U"], i) @ zs)
    e = (_rows_of(w["D"], i) @ h).reshape(T, k, -1)
    u = (e * p.unsqueeze(2)).sum(1)
    hs = _gate(act, xf @ w["Gs"].float().transpose(1, 2), xf @ w["Us"].float().transpose(1, 2))   # [2, T, f_s]
    y = (hs @ w["Ds"].float().transpose(1, 2)).sum(0)
    if case["standard"]:
        y = y + u
    else:
        y = y + (u * torch.rsqrt((u * u).mean(1, keepdim=True) + 1e-6)) @ w["W_up"].float().T
    return {"output": y.to(dt), "selected_experts": sel.to(torch.int32), "mixture_weights": p.to(dt),
            "latent_routed_aggregate": u.to(dt)}


def _plain_product(s):
    a, w, dt = _plain_dequantize(*s["a"]), _plain_dequantize(*s["w"]), _DT[s["case"]["dtype"]]
    if "offsets" not in s:
        return (a @ w.T).to(dt)
    # each expert's rows in a block of its own, as long as the longest
    off = s["offsets"].long()
    row = off[:-1, None] + torch.arange(s["most"], device=a.device)
    real = row < off[1:, None]
    c = a[row.clamp(max=a.shape[0] - 1)] @ w.transpose(1, 2)
    return c[real].to(dt)


def run(s):
    case = s["case"]
    if case["op"] == "few":
        if own:
            return s["layer"].forward_few_into(s["x"], s["out"])
        return _plain_few(case, s["x"], s["w"])
    if case["op"] == "quantize":
        if own:
            import latent_space_routed_b200 as lm
            return lm.mx4_dequantize(lm.mx4_quantize(s["x"]), s["x"].dtype)
        return _plain_dequantize(*_plain_quantize(s["x"])).to(s["x"].dtype)
    if own:
        return s["lm"].mx4_gemm(s["a"], s["w"], offsets=s.get("offsets"), out=s["out"], workspace=s["workspace"])
    return _plain_product(s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "quantize":
        # the values read, codes and scales written and read again, the values written
        n, b = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * b + 2 * (n // 2 + n // 32), "flops": 4 * n}
    if case["op"] == "product":
        M, N, K, E = (case[n] for n in ("M", "N", "K", "E"))
        # experts that get a row, were the rows dealt evenly
        touched = E * (1 - (1 - 1 / E) ** M) if E else 1
        return {"bytes": (M + touched * N) * (K // 2 + K // 32) + M * N * (2 if case["dtype"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    T, d, l, f, E, k, f_s = (case[n] for n in ("T", "d", "l", "f", "E", "k", "f_s"))
    b = 2 if case["dtype"] == "bf16" else 4
    touched = E * (1 - (1 - k / E) ** T)
    per = 3 * f * l * (17 / 32 if case["experts"] == "mx4" else b)
    proj = 0 if case["standard"] else 2 * d * l
    return {"bytes": touched * per + E * d * 4 + (proj + 6 * f_s * d) * b + T * (2 * d + l + k) * b + 4 * T * k,
            "flops": 2 * T * (E * d + proj + 3 * k * f * l + 6 * f_s * d)}


# ------------------------------------------------------------------ the definition, in 64 bits
def _values(codes, scales):
    """The values of a 4-bit tensor from its bits: one sign, two exponent bits, one mantissa bit."""
    lo_hi = torch.stack([codes % 16, codes // 16], dim=-1).flatten(-2).to(torch.int64)
    sign = 1.0 - 2.0 * (lo_hi // 8).double()
    ex, man = (lo_hi // 2) % 4, (lo_hi % 2).double()
    mag = torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man) * 2.0 ** (ex - 1).double())
    return sign * mag * (2.0 ** (scales.double() - 127.0)).repeat_interleave(32, dim=-1)


def _exact_quantize(x):
    v = x.double().unflatten(-1, (-1, 32))
    size = v.abs().max(dim=-1, keepdim=True).values
    top = 2.0 ** torch.round(torch.log2(size.clamp(min=2.0 ** -160)))
    top = torch.where(top > size, top / 2, top)                     # the largest power of two up to it
    step = torch.where(size > 0, (top / 4).clamp(min=2.0 ** -127), torch.ones_like(size))
    t = (v / step).clamp(-6.0, 6.0)
    # spacing of the values around t: 1/2 up to 2, 1 up to 4, then 2; rounding half to even within each
    gap = torch.where(t.abs() < 2, 0.5, torch.where(t.abs() < 4, 1.0, 2.0)).double()
    return (torch.round(t / gap) * gap * step).flatten(-2)


def _exact_gate(act, g, v):
    sg = torch.sigmoid(g)
    return 4.0 * torch.tanh(g / 4.0) * sg * 25.0 * torch.tanh(v / 25.0) if act == "situ" else g * sg * v


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "quantize":
        return torch.cat([_exact_quantize(c) for c in s["x"].split(1 << 15)])
    if case["op"] == "product":
        if "offsets" not in s:
            return _values(*s["a"]) @ _values(*s["w"]).T
        at = s["offsets"].tolist()
        return torch.cat([_values(s["a"][0][i:j], s["a"][1][i:j]) @ _values(s["w"][0][e], s["w"][1][e]).T
                          for e, (i, j) in enumerate(zip(at[:-1], at[1:]))])
    w, k, act = s["w"], case["k"], case["act"]
    one = (lambda t, e: _values(t[0][e], t[1][e])) if case["experts"] == "mx4" else (lambda t, e: t[e].double())
    Wr, b = w["W_r"].double(), w["b"].double()
    ys, sels, ps, us = [], [], [], []
    for x in s["x"].double():
        r = torch.sigmoid(Wr @ x)
        order = sorted(range(case["E"]), key=lambda e, q=(r + b).tolist(): (-q[e], e))[:k]
        p = r[order] / r[order].sum()
        z = x if case["standard"] else w["W_down"].double() @ x
        u = sum(p[j] * (one(w["D"], e) @ _exact_gate(act, one(w["G"], e) @ z, one(w["U"], e) @ z))
                for j, e in enumerate(order))
        y = sum(w["Ds"][i].double() @ _exact_gate(act, w["Gs"][i].double() @ x, w["Us"][i].double() @ x) for i in (0, 1))
        y = y + (u if case["standard"] else w["W_up"].double() @ (u / torch.sqrt((u * u).mean() + 1e-6)))
        ys.append(y), ps.append(p), us.append(u), sels.append(order)
    return {"output": torch.stack(ys), "selected_experts": torch.tensor(sels, dtype=torch.int32),
            "mixture_weights": torch.stack(ps), "latent_routed_aggregate": torch.stack(us)}
