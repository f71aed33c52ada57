"""Calls of the few-token layer as programs make them: several streams and threads, graphs, tensors that do not fit."""
import threading

import pytest
import torch

import latent_space_routed_b200 as lm
import lmoe_inputs as li
from test_gpu_few import check, make

pytestmark = pytest.mark.gpu


def same(a, b):
    return all(torch.equal(a[n], b[n]) for n in a)


def test_workspaces_of_streams_and_threads_differ():
    """A buffer of the layer's own serves calls that follow one another only: one stream, one thread."""
    w, W, layer = make(4, 256, 64, 128, 16, 4)
    s = torch.cuda.Stream()
    mine = layer.few_workspace(4)
    with torch.cuda.stream(s):
        other = layer.few_workspace(4)
    got = []
    t = threading.Thread(target=lambda: got.append(layer.few_workspace(4)))
    t.start(), t.join()
    assert len({v.data_ptr() for v in (mine, other, got[0], layer.few_workspace(5))}) == 4
    assert layer.few_workspace(4).data_ptr() == mine.data_ptr() == layer.few_workspace(4, torch.cuda.current_stream()).data_ptr()
    assert layer.few_workspace(4, s).data_ptr() == layer.few_workspace(4, s.cuda_stream).data_ptr() == other.data_ptr()


def test_two_streams_and_threads_without_workspaces():
    w, W, layer = make(6, 512, 128, 256, 32, 6)
    xs = [li.tokens(w, seed=i).cuda() for i in range(4)]
    want = [layer.forward_few(x) for x in xs]
    torch.cuda.synchronize()
    got = []

    def calls(streams, on_thread_stream):
        for i in range(40):
            s = streams[i % len(streams)]
            if on_thread_stream:                       # by the argument, or as the current stream
                got.append((i % 4, layer.forward_few(xs[i % 4], stream=s)))
            else:
                with torch.cuda.stream(s):
                    got.append((i % 4, layer.forward_few(xs[i % 4])))

    streams = [torch.cuda.Stream() for _ in range(3)]
    calls(streams[:2], False)
    calls(streams[1:], True)
    threads = [threading.Thread(target=calls, args=([streams[i % 2]], i > 1)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(got) == 240
    for i, out in got:
        assert same(out, want[i])


def test_graphs_without_workspaces_replay_at_once():
    w, W, layer = make(4, 512, 128, 256, 32, 6)
    xs = [li.tokens(w, seed=i).cuda() for i in range(2)]
    want = [layer.forward_few(x) for x in xs]
    graphs = []
    for x in xs:                                       # captured on one stream, one after the other
        g, out = torch.cuda.CUDAGraph(), layer.empty_outputs(4)
        with torch.cuda.graph(g):
            layer.forward_few_into(x, out)
            layer.forward_few_into(x, out)
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = layer.forward_few(xs[1])
    torch.cuda.synchronize()
    assert same(eager, want[1])
    for (_, out), r in zip(graphs, want):
        assert same(out, r)


def test_tokens_at_any_address():
    """x that is contiguous but not 16-byte aligned is copied, as mx4_quantize does."""
    for dtype in ("bf16", "f32"):
        w, W, layer = make(3, 256, 64, 128, 16, 4, dtype=dtype)
        x = li.tokens(w)
        want = layer.forward_few(x.cuda())
        flat = torch.empty(3 * 256 + 1, dtype=layer.dtype, device="cuda")
        odd = flat[1:].view(3, 256).copy_(x)
        assert odd.data_ptr() % 16
        assert same(layer.forward_few(odd), want)
        assert same(layer.forward_few_into(odd, layer.empty_outputs(3)), want)


def test_hidden_rows_of_2_to_the_26():
    """8 tokens' rows of the hidden are 2^31 bytes of activation terms: sizes beyond 32 bits come in segments too.
    Sums of 2^26 fp32 products in chains add errors of random sign, 2^13 2^-25 of a row's typical value; the rest as in
    test_gpu_few."""
    T, d, f = 8, 64, 2 ** 26
    w, W, _ = make(T, d, d, 128, 1, 1)
    g = torch.Generator(device="cuda").manual_seed(1)
    Q = {}
    for n, shape in (("G", (1, f, d)), ("U", (1, f, d)), ("D", (1, d, f))):
        codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device="cuda", dtype=torch.uint8)
        # values of 2^-5 in G and U, of 2^-13 in D
        scales = torch.full((*shape[:-1], shape[-1] // 32), 121 if n != "D" else 113, device="cuda", dtype=torch.uint8)
        Q[n] = lm.Mx4(codes, scales)
    cfg = lm.make_config(d, d, f, 1, 1, 128)
    layer = lm.LatentMoE(cfg, {**{n: v.cuda() for n, v in W.items()}, **Q})
    x = li.tokens(w).cuda()
    out = layer.forward_few(x)
    lm.lmoe_check_device(layer.handle, T, layer.few_workspace(T))
    z = x.double() @ W["W_down"].double().cuda().T
    u, n = torch.zeros(T, d, dtype=torch.float64, device="cuda"), 2 ** 21
    for i in range(0, f, n):
        G, U = (lm.mx4_dequantize(lm.Mx4(Q[k].codes[0, i:i + n], Q[k].scales[0, i:i + n]), torch.float32).double() for k in "GU")
        D = lm.mx4_dequantize(lm.Mx4(Q["D"].codes[0, :, i // 2:(i + n) // 2].contiguous(),
                                     Q["D"].scales[0, :, i // 32:(i + n) // 32].contiguous()), torch.float32).double()
        a = z @ G.T
        u += (a * torch.sigmoid(a) * (z @ U.T)) @ D.T
    got = out["latent_routed_aggregate"].double()
    assert ((got - u).abs() <= 2.0 ** -8 * u.abs() + 2.0 ** -9 * u.abs().amax(1, keepdim=True)).all()
    del layer, Q, out
    torch.cuda.empty_cache()


def test_misaligned_outputs_are_refused():
    """By the C name, whose addresses are anything: stores of the token type and of int32 would fault."""
    w, W, layer = make(3, 256, 64, 128, 16, 4)
    x, ws = li.tokens(w).cuda(), layer.few_workspace(3)
    room = torch.empty(4, 8192, dtype=torch.uint8, device="cuda")
    for which, by in ((0, 1), (1, 2), (2, 1), (3, 1)):
        o = [room[i].data_ptr() + (by if i == which else 0) for i in range(4)]
        with pytest.raises(lm.LmoeError, match="aligned") as e:
            lm.lmoe_forward_few(layer.handle, x, 3, *o, ws, ws.numel())
        assert e.value.status == lm.LMOE_ERR_UNSUPPORTED
