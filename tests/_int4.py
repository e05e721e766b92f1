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


def values(pool):
    """The values of every row of a pool in float64, [NB, bs, Hkv, D], and the
    magnitude step * code + |low| that a rounded sum of the two terms may reach."""
    code, step, low = rows(pool)
    s, lo = step.astype(np.float64)[..., None], low.astype(np.float64)[..., None]
    return lo + s * code, np.abs(s) * code + np.abs(lo)


UNIT_OUT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def attention(q, pools, tables, lens, scale, q_start=None, q_dtype="f16"):
    """Attention over 4-bit pools in float64 and how far a kernel may be off.

    q [rows, Hq, D] float64.  The bound of an output element adds
      - half a step of the output type;
      - the probabilities' rounding to f16 (2^-11 each) on the values' terms;
      - the scores' error: D products of f32 rounding 2^-23 on their terms,
        which moves a probability by as much relative to it, twice (its
        numerator and the sum), and 2^-18 for exp2 and the sums of the tokens.
    """
    (kv, ka), (vv, va) = (values(p) for p in pools)
    NB, bs, Hkv, D = kv.shape
    kv, ka, vv, va = (x.reshape(-1, Hkv, D) for x in (kv, ka, vv, va))
    Hq = q.shape[1]
    G = Hq // Hkv
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for i, L in enumerate(lens):
        a, b = (i, i + 1) if q_start is None else (q_start[i], q_start[i + 1])
        pos = np.arange(L)
        slot = tables[i][pos // bs].astype(np.int64) * bs + pos % bs
        for r in range(a, b):
            n = L - (b - a) + (r - a) + 1                     # keys attended
            if n <= 0:
                continue
            sl = slot[:n]
            for h in range(Hq):
                g = h // G
                s = kv[sl, g] @ q[r, h] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[r, h] = p @ vv[sl, g]
                ds = (D + 2) * 2.0 ** -23 * (ka[sl, g] @ np.abs(q[r, h])) * abs(scale)
                tol[r, h] = (2.0 ** -11 + 2.0 ** -18 + 2 * ds.max()) * (p @ va[sl, g])
    return out, tol + UNIT_OUT[q_dtype] * np.abs(out) + 2.0 ** -25


def random_pools(rng, NB, bs, Hkv, D, k_mult=1.0, v_mult=1.0, offset=0.5):
    """K and V pools of N(0, 1) rows (keys with a mean per channel)."""
    out = []
    for mult, off in ((k_mult, offset), (v_mult, 0.0)):
        x = (rng.standard_normal((NB, bs, Hkv, D)) + off * rng.standard_normal((Hkv, D))) * mult
        out.append(pack(*encode(x.astype(np.float32))))
    return out


def poison(pool, used):
    """NaN parameters and full codes in every row that `used` [NB, bs] leaves out."""
    code, step, low = rows(pool)
    code, step, low = code.copy(), step.copy(), low.copy()
    code[~used], step[~used], low[~used] = 15, np.float16("nan"), np.float16("nan")
    return pack(code, step, low)


def tables_for(rng, lens, bs, spare=3, max_blocks=None):
    """Block tables over a random permutation of a pool, garbage behind each
    sequence's last block; (tables, number of blocks, used rows [NB, bs])."""
    n = [-(-L // bs) for L in lens]
    NB = sum(n) + spare
    MB = max_blocks or max(max(n), 1)
    order = rng.permutation(NB)
    t = np.empty((len(lens), MB), np.int32)
    t[:] = np.resize(np.array([-1, NB + 7], np.int32), MB)
    used = np.zeros((NB, bs), bool)
    k = 0
    for i, c in enumerate(n):
        t[i, :c] = order[k:k + c]
        for j in range(c):
            used[order[k + j], :min(bs, lens[i] - j * bs)] = True
        k += c
    return t, NB, used
