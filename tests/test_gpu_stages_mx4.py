"""lmoe_forward with 4-bit experts: the requantised hidden value by value, and the stages behind the experts.

Every stage is compared with its formula in 64 bits on the inputs that it had (workspace regions).  Error bars, derived:
a sum of K fp32 terms is off by at most K 2^-24 sum |a w|; g and u are such sums, and act(g, u) moves by at most
(1.2 + 1.2 |u|) dg + (1.2 + 1.2 |g|) du (slopes of the gates: at most 1.1 |u| in g and |g| in u, the rest for dg du).  The
gate itself: SwiGLU in the product's epilogue has the hardware's exponential, off by at most 2 + 1.173 |g| units in the last
place (2^-23 of the value), its quotient two more, and four roundings; SiTU's tanhf and expf two units each.  Both stay
below (8 + 1.2 |g|) 2^-23 of the value.  A bf16 result adds 2^-8 of its value."""
import pytest
import torch

import latent_space_routed_b200 as lm
import lmoe_inputs as li
import mx4ref
from test_gpu_mx4 import gate

pytestmark = pytest.mark.gpu

CASES = [(1, 256, 128, 256, 16, 4, 0, False), (2, 256, 64, 128, 8, 3, 0, False), (9, 256, 192, 384, 24, 5, 1, False),
         (200, 512, 256, 256, 32, 6, 0, False), (700, 256, 256, 128, 16, 4, 0, True), (33, 448, 64, 128, 40, 7, 1, False),
         (5, 256, 256, 128, 16, 4, 1, True)]


def layer_of(T, d, l, f, E, k, act, standard, steeper=0):
    w = li.custom("mx4", T, d, l, f, E, k, 128, seed=T, standard=standard)
    W = li.weights(w)
    Q = {n: lm.mx4_quantize(W[n].cuda()) for n in ("G", "U", "D")}
    Q["G"].scales.add_(steeper)                        # gates larger by a power of two
    layer = lm.LatentMoE(lm.config_for(w, act=act), {n: Q.get(n, v if n in Q else v.cuda()) for n, v in W.items()})
    return w, {n: v.double().cuda() for n, v in W.items()}, Q, layer


def gate_bar(K, act, g, u, dg, du, h):
    return K * 2.0 ** -24 * (dg * (1.2 + 1.2 * u.abs()) + du * (1.2 + 1.2 * g.abs())) + (8 + 1.2 * g.abs()) * 2.0 ** -23 * h.abs()


def to_codes(x, scale):
    """x rounded to the 4-bit values of a given scale byte per 32 columns (monotone in x)."""
    s = torch.exp2(scale.double() - 127.0).repeat_interleave(32, 1)
    t = (x / s).clamp(-6.0, 6.0)
    gap = torch.where(t.abs() < 2, 0.5, torch.where(t.abs() < 4, 1.0, 2.0))
    return torch.round(t / gap) * gap * s              # (half to even: the even code)


@pytest.mark.parametrize("steeper", [0, 4])
@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(int(v)) for v in c))
def test_hidden_codes(c, steeper):
    """Each block's scale is that of a value within the bars, and each code lies between those of h - bar and h + bar."""
    T, d, l, f, E, k, act, standard = c
    w, W, Q, layer = layer_of(*c, steeper=steeper)
    layer(li.tokens(w).cuda())
    layer.check_device(T)
    S = T * k
    z = mx4ref.values(layer.region(T, "Zp4", torch.uint8, (S, l // 2)),
                      layer.region(T, "Zp4_scales", torch.uint8, (S, l // 32))).cuda()
    off = layer.region(T, "offsets", torch.int32, (E + 1,)).tolist()
    val = {n: mx4ref.values(*Q[n]).cuda() for n in ("G", "U")}
    h, bar = (torch.zeros(S, f, dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(E):
        i, j = off[e], off[e + 1]
        g, u = z[i:j] @ val["G"][e].T, z[i:j] @ val["U"][e].T
        h[i:j] = gate(act, g, u)
        bar[i:j] = gate_bar(l, act, g, u, z[i:j].abs() @ val["G"][e].abs().T, z[i:j].abs() @ val["U"][e].abs().T, h[i:j])
    hc, hs = layer.region(T, "H4", torch.uint8, (S, f // 2)), layer.region(T, "H4_scales", torch.uint8, (S, f // 32))
    got = mx4ref.values(hc, hs).cuda()

    def scale(top):                                    # of blocks with this largest magnitude
        return (torch.frexp(top.clamp(min=2.0 ** -140))[1] - 3).clamp(min=-127) + 127

    lowest = scale((h.abs() - bar).clamp(min=0).view(S, -1, 32).amax(2))
    highest = scale((h.abs() + bar).view(S, -1, 32).amax(2))
    assert ((hs >= lowest) & (hs <= highest)).all()
    assert (lowest == highest).double().mean() > 0.9   # (the bars are narrow: this says something)
    lo, hi = to_codes(h - bar, hs), to_codes(h + bar, hs)
    assert ((got >= lo) & (got <= hi)).all()
    assert (lo == hi).double().mean() > 0.9


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(int(v)) for v in c))
def test_output(c):
    """Shared experts, norm and the last product: from x and the experts' weighted rows to `output`."""
    T, d, l, f, E, k, act, standard = c
    w, W, Q, layer = layer_of(*c)
    x = li.tokens(w).cuda()
    out = layer(x)
    layer.check_device(T)
    x64, fs, cols = x.double(), w.f_s, 2 * w.f_s + (0 if standard else l)
    hs = layer.region(T, "HS", torch.bfloat16, (-1,))[:T * cols].view(T, cols).double()
    for i in range(2):
        g, u = x64 @ W["Gs"][i].T, x64 @ W["Us"][i].T
        h = gate(act, g, u)
        bar = gate_bar(d, act, g, u, x64.abs() @ W["Gs"][i].abs().T, x64.abs() @ W["Us"][i].abs().T, h)
        assert ((hs[:, i * fs:(i + 1) * fs] - h).abs() <= 2.0 ** -8 * h.abs() + 1.01 * bar).all()
    rows = layer.region(T, "Y", torch.bfloat16, (T * k, l)).double()[
        layer.region(T, "slot_of", torch.int32, (T, k)).long().reshape(-1)].view(T, k, l)
    u, size = rows.sum(1), rows.abs().sum(1)
    assert ((out["latent_routed_aggregate"].double() - u).abs() <= 2.0 ** -8 * u.abs() + k * 2.0 ** -24 * size).all()
    A, B = hs[:, :2 * fs], torch.cat([W["Ds"][0], W["Ds"][1]], 1)
    y = A @ B.T
    if standard:
        y = y + out["latent_routed_aggregate"].double()
    else:
        # the root of a mean of l squares: l terms' roundings at most, halved by the root, and four more
        n = u / torch.sqrt((u * u).mean(1, keepdim=True) + w.eps)
        of_sum = k * 2.0 ** -24 * size / torch.sqrt((u * u).mean(1, keepdim=True) + w.eps)
        of_norm = (l / 2 + 4) * 2.0 ** -24 * n.abs() + n.abs() * of_sum.amax(1, keepdim=True)
        assert ((hs[:, 2 * fs:] - n).abs() <= 2.0 ** -8 * n.abs() + 1.01 * (of_sum + of_norm)).all()
        A, B = hs, torch.cat([B, W["W_up"]], 1)
        y = A @ B.T
    bar = (A.shape[1] + 2) * 2.0 ** -24 * (A.abs() @ B.abs().T + y.abs())
    assert ((out["output"].double() - y).abs() <= 2.0 ** -8 * y.abs() + 1.01 * bar).all()
