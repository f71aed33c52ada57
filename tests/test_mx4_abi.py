"""4-bit tensors and the few-token layer: what the entry points refuse, and the reference the GPU tests use.  No GPU."""
import ctypes

import numpy as np
import pytest
import torch

import latent_space_routed_b200 as lm
import mx4ref

A = 0x1000                 # an aligned address that is never dereferenced
BAD, UNS, WSP = lm.LMOE_ERR_INVALID_ARG, lm.LMOE_ERR_UNSUPPORTED, lm.LMOE_ERR_WORKSPACE


def test_reference_rounds_to_nearest_even_code():
    x = torch.zeros(1, 32, dtype=torch.float64)
    x[0, :12] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.1, 7.9, 0.26, -0.0])
    c, s = mx4ref.quantize(x)
    assert s.item() == 127
    v = mx4ref.values(c, s)[0, :12].tolist()
    assert v == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -6.0, 6.0, 0.5, 0.0]
    assert np.signbit(v[11])


def test_reference_scales():
    x = torch.zeros(4, 32, dtype=torch.float64)
    x[1, 3], x[2, 0], x[3, 0] = 8.0, 2.0 ** -140, float("nan")
    c, s = mx4ref.quantize(x)
    assert s[:, 0].tolist() == [0, 128, 0, 255]
    assert mx4ref.values(c, s)[1, 3] == 8.0 and torch.isnan(mx4ref.values(c, s)[3]).all()


@pytest.mark.parametrize("args,status", [
    ((None, 1, 4, 64, 64, A, A), BAD), ((A, 1, 4, 64, 64, None, A), BAD), ((A, 1, 4, 64, 64, A, None), BAD),
    ((A, 1, -1, 64, 64, A, A), BAD), ((A, 1, 4, -32, 64, A, A), BAD), ((A, 2, 4, 64, 64, A, A), BAD),
    ((A, 1, 4, 64, 63, A, A), BAD), ((A, 1, 4, 48, 64, A, A), UNS), ((A + 2, 1, 4, 64, 64, A, A), UNS),
    ((A, 1, 4, 64, 66, A, A), UNS), ((A, 0, 4, 64, 66, A, A), UNS), ((A, 1, 4, 64, 64, A + 2, A), UNS),
    ((A, 1, 1 << 46, 64, 64, A, A), UNS),
    ((None, 1, 0, 64, 64, None, None), lm.LMOE_OK), ((None, 0, 5, 0, 0, None, None), lm.LMOE_OK),
])
def test_quantize_refuses(args, status):
    x, dt, rows, cols, ld, codes, scales = args
    assert lm._lib.lmoe_mx4_quantize(x, dt, rows, cols, ld, codes, scales, None) == status
    assert lm._lib.lmoe_mx4_dequantize(codes, scales, rows, cols, dt, x, ld, None) == status
    assert (lm.lmoe_last_error() == "") == (status == lm.LMOE_OK)


def _gemm(**kw):
    a = dict(a=A, sa=A, M=5, w=A, sw=A, N=7, K=64, off=None, E=1, dt=1, out=A, ldo=7, ws=A, n=256)
    a.update(kw)
    return lm._lib.lmoe_mx4_gemm(a["a"], a["sa"], a["M"], a["w"], a["sw"], a["N"], a["K"], a["off"], a["E"], a["dt"],
                                 a["out"], a["ldo"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(a=None), BAD), (dict(sa=None), BAD), (dict(w=None), BAD), (dict(sw=None), BAD), (dict(out=None), BAD),
    (dict(M=-1), BAD), (dict(N=-1), BAD), (dict(K=-64), BAD), (dict(dt=3), BAD), (dict(ldo=6), BAD),
    (dict(off=A, E=0), BAD), (dict(off=A, E=1025), UNS), (dict(K=0), UNS), (dict(K=96), UNS), (dict(a=A + 8), UNS),
    (dict(w=A + 8), UNS), (dict(out=A + 1), UNS), (dict(out=A + 2, dt=0), UNS), (dict(M=1 << 31), UNS),
    (dict(N=1 << 31, ldo=1 << 31), UNS), (dict(off=A, E=1024, N=1 << 22, ldo=1 << 22), UNS),
    (dict(ws=None), WSP), (dict(n=255), WSP), (dict(ws=A + 128), WSP),
    (dict(M=0, a=None, out=None), lm.LMOE_OK), (dict(N=0, ldo=0, w=None), lm.LMOE_OK),
])
def test_gemm_refuses(kw, status):
    assert _gemm(**kw) == status, lm.lmoe_last_error()


def test_gemm_check_refuses_null():
    assert lm._lib.lmoe_mx4_gemm_check(None, None) == BAD


def test_few_refuses_without_a_handle():
    n = ctypes.c_size_t()
    assert lm._lib.lmoe_few_workspace_size(None, 1, ctypes.byref(n)) == BAD
    assert lm._lib.lmoe_forward_few(None, A, 1, A, A, A, A, A, 1 << 20, None) == BAD


@pytest.mark.parametrize("kw,experts,status", [
    (dict(), None, BAD), (dict(), (A, A, A, None, A, A), BAD), (dict(dtype=lm.LMOE_F32), (A,) * 6, UNS),
    (dict(gemm=1), (A,) * 6, UNS), (dict(), (A + 8, A, A, A, A, A), UNS), (dict(k=0), (A,) * 6, BAD),
])
def test_create_mx4_refuses(kw, experts, status):
    cfg = lm.make_config(**{**dict(d=256, l=128, f=256, E=16, k=4, f_shared=256), **kw})
    w = lm.lmoe_weights(A, A, A, A, None, None, None, A, A, A)
    x4 = ctypes.byref(lm.lmoe_mx4_experts(*experts)) if experts else None
    h = ctypes.c_void_p()
    assert lm._lib.lmoe_create_mx4(ctypes.byref(cfg), ctypes.byref(w), x4, None, ctypes.byref(h)) == status
    assert h.value is None


def test_python_refuses_before_the_library():
    q = lm.Mx4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    assert q.shape == (4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        q.check("q")
    with pytest.raises(TypeError, match="uint8"):
        lm.Mx4(torch.zeros(4, 32), q.scales).check("q")
    with pytest.raises(ValueError, match="match"):
        lm.Mx4(q.codes, torch.zeros(4, 3, dtype=torch.uint8)).check("q")
    with pytest.raises(TypeError):
        lm.mx4_quantize(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA"):
        lm.mx4_quantize(torch.zeros(4, 64))
    with pytest.raises(TypeError):
        lm.mx4_dequantize(q, torch.float64)
