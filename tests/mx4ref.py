"""Microscaled 4-bit values in 64 bits, from their definition (used by the 4-bit tests only).

A block of 32 values along a row has the scale 2^E, E = floor(log2 of its largest magnitude) - 2 and at least
-127; values go to the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6, ties to the even code, those past 6 to 6."""
import numpy as np
import torch

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x: torch.Tensor):
    """(codes [..., cols / 2], scales [..., cols / 32]) of x [..., cols] as uint8 CPU tensors."""
    v = x.detach().double().cpu().numpy()
    v = v.reshape(*v.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        top = np.abs(v).max(-1)
        bad = ~np.isfinite(v).all(-1)
        e = np.where(top > 0, np.frexp(np.where(np.isfinite(top), top, 1.0))[1] - 3, -127)
    e = np.clip(e, -127, None)
    t = np.where(bad[..., None], 0.0, np.abs(v)) * np.exp2(-e.astype(np.float64))[..., None]
    t = np.minimum(t, 6.0)
    d = np.abs(t[..., None] - MAGNITUDES)
    near = d == d.min(-1, keepdims=True)                       # one or, on a tie, two neighbours
    lo, hi = near.argmax(-1), 7 - near[..., ::-1].argmax(-1)
    code = np.where(lo % 2 == 0, lo, hi)
    code = np.where(bad[..., None], 0, code + 8 * np.signbit(v)).astype(np.uint8)
    code = code.reshape(*code.shape[:-2], -1, 2)
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    return torch.from_numpy(code[..., 0] | (code[..., 1] << 4)), torch.from_numpy(scale)


def values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """fp64 values [..., cols] (CPU)."""
    c, s = codes.cpu().numpy(), scales.cpu().numpy().astype(np.int64)
    c = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)
    f = np.where(s == 255, np.nan, np.exp2(s - 127.0))
    return torch.from_numpy(v * np.repeat(f, 32, -1))
