"""The 4-bit row format in numpy, in 64 bits, from its definition; the GPU
side's layout of a pool.  Test infrastructure only."""
import numpy as np

PARAM = 4                      # bytes of a row's (step, low)


def encode(x):
    """(codes uint8, step float16, low float16) of the rows of x [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    nan = np.isnan(x).any(-1)
    x = np.clip(np.where(nan[..., None], 0.0, x), -65504.0, 65504.0)
    low = x.min(-1).astype(np.float16)
    l64 = low.astype(np.float64)
    step = np.maximum((x.max(-1) - l64) / 15, 0.0).astype(np.float16)
    s64 = step.astype(np.float64)[..., None]
    code = np.rint(np.divide(x - l64[..., None], s64, out=np.zeros_like(x), where=s64 > 0))
    code = np.clip(code, 0, 15).astype(np.uint8)
    code[nan] = 0
    step[nan] = low[nan] = np.float16("nan")
    return code, step, low


def decode(code, step, low):
    """The rows' values in float64."""
    return low.astype(np.float64)[..., None] + step.astype(np.float64)[..., None] * code


def split(pool):
    """Views of a uint8 pool [NB, bs, Hkv, D/2 + 4]: codes [NB, Hkv, bs, D/2]
    and (step, low) float16 [NB, Hkv, bs, 2]."""
    NB, bs, Hkv, R = pool.shape
    flat = pool.reshape(NB, -1)
    n = Hkv * bs * (R - PARAM)
    codes = flat[:, :n].reshape(NB, Hkv, bs, R - PARAM)
    par = flat[:, n:].copy().view(np.float16).reshape(NB, Hkv, bs, 2)
    return codes, par


def rows(pool):
    """(codes [NB, bs, Hkv, D], step, low [NB, bs, Hkv]) of every row of a pool."""
    codes, par = split(pool)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:3] + (-1,))
    return (c.transpose(0, 2, 1, 3), par[..., 0].transpose(0, 2, 1).copy(), par[..., 1].transpose(0, 2, 1).copy())


def pack(code, step, low):
    """A pool of codes [NB, bs, Hkv, D] and parameters [NB, bs, Hkv]."""
    NB, bs, Hkv, D = code.shape
    c = code.transpose(0, 2, 1, 3)
    by = (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8).reshape(NB, -1)
    par = np.stack([step.transpose(0, 2, 1), low.transpose(0, 2, 1)], -1).astype(np.float16)
    par = np.ascontiguousarray(par).view(np.uint8).reshape(NB, -1)
    return np.concatenate([by, par], 1).reshape(NB, bs, Hkv, D // 2 + PARAM)
