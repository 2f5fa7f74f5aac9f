"""References of the sub-layer's training operators, in 64 bits on the CPU, written from the definitions in include/mhc.h."""
import numpy as np

BLOCK = 32


def torch_dtype(f16):
    import torch
    return torch.float16 if f16 else torch.bfloat16


def to_16(a, f16):
    """float64 -> the nearest 16-bit values, as a torch CPU tensor."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch_dtype(f16))


def store(v, f16):
    """Codes (int8), scale bytes (uint8) of the float64 array v [..., D] of 16-bit values."""
    lead, D = v.shape[:-1], v.shape[-1]
    nb = -(-D // BLOCK)
    b = np.zeros((*lead, nb * BLOCK))
    b[..., :D] = v
    b = b.reshape(*lead, nb, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 6, -10000)
    e = np.maximum(e, -24 if f16 else -126)
    q = np.clip(np.rint(np.ldexp(b, -e[..., None])), -127, 127)      # rint: ties to even
    q = np.where(bad[..., None], 0, q)
    s = np.where(bad, 255, e + 127)
    return q.reshape(*lead, nb * BLOCK)[..., :D].astype(np.int8), s.astype(np.uint8)


def load(codes, scales):
    """The values a checkpoint stands for (float64, NaN where the block's scale is 255)."""
    s = scales.astype(np.int64)
    step = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return codes.astype(np.float64) * np.repeat(step, BLOCK, -1)[..., :codes.shape[-1]]


def half_step(ref, f16):
    """Half a step of the 16-bit format at ref: eps / 2 relative, half the least value near zero."""
    eps, least = (2.0 ** -11, 2.0 ** -25) if f16 else (2.0 ** -8, 2.0 ** -134)
    return np.maximum(eps * np.abs(ref), least)
