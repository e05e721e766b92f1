"""Attention of many query tokens from its definition, in 64 bits, with the
error that a kernel of 16-bit weights may make.  Test infrastructure only."""
import math

import torch

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}     # a rounding, relative


def attend(q, k, v, scale, last):
    """(out, tol) float64 [n, Hq, D] of query rows q [n, Hq, D] over keys and
    values [L, Hkv, D]; row j attends the keys t <= last[j].

    tol, with u the relative half step of the type: weights enter the second
    product with an error of u each and the output is rounded once, both against
    sum p|v|: 2 u.  A weight's exponent (in log2) errs by that of its score, a sum of
    D products and a subtraction in f32 and an exponential of 2^-22: under
    2^-20 (1 + c sum |q k|) for the largest of the row's scores, which p and l each
    may have.  Weights below 2^-31 of the largest may be lost: L 2^-31 max|v|.  An
    f16 output below 2^-14 has steps of 2^-24."""
    u = HALF[q.dtype]
    n, Hq, D = q.shape
    L, Hkv = k.shape[:2]
    out = torch.zeros(n, Hq, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    if L == 0 or n == 0:
        return out, tol
    pos = torch.arange(L, device=q.device)
    for h in range(Hq):
        g = h // (Hq // Hkv)
        qd, kd, vd = q[:, h].double(), k[:, g].double(), v[:, g].double()
        hide = pos[None, :] > last[:, None]
        x = (qd @ kd.T * scale).masked_fill(hide, -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m.masked_fill(m == -math.inf, 0.0))
        s = p.sum(-1, keepdim=True)
        vis = lambda w: torch.stack([torch.where(hide[j, :, None], 0.0, p[j, :, None] * w).sum(0)  # noqa: E731
                                     for j in range(n)]) if not torch.isfinite(w).all() else p @ w
        out[:, h] = torch.where(s > 0, vis(vd) / s, torch.where(s == 0, 0.0, math.nan))
        big = (qd.abs() @ kd.abs().T).masked_fill(hide, 0.0).nan_to_num(0.0, 0.0, 0.0).amax(-1, keepdim=True)
        fin = vd.abs().nan_to_num(0.0, 0.0, 0.0)
        mass = torch.where(s > 0, p.nan_to_num(0.0) @ fin / s, 0.0)
        tol[:, h] = (mass * (2 * u + 2 * 2.0 ** -20 * (1 + 1.4427 * abs(scale) * big)) * 1.01 +
                     L * 2.0 ** -31 * fin.amax() + 2.0 ** -25)
    return out, tol


def prompts(q, k, v, q_start, k_start, scale, fill):
    """(out, tol) of packed prompts; rows of no sequence hold `fill`, tol 0."""
    out = torch.full(q.shape, fill, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for i in range(len(q_start) - 1):
        a, b, c, d = q_start[i], q_start[i + 1], k_start[i], k_start[i + 1]
        last = torch.arange(d - c - (b - a), d - c, device=q.device)
        out[a:b], tol[a:b] = attend(q[a:b], k[c:d], v[c:d], scale, last)
    return out, tol


def check(got, out, tol, what=""):
    got = got.double()
    same = (got == out) | (got.isnan() & out.isnan())
    err = (got - out).abs()
    ok = same | (err <= tol)
    assert ok.all(), (f"{what}: {int((~ok).sum())} of {ok.numel()} outside; worst "
                      f"{float(torch.where(ok, 0.0, err - tol).nan_to_num(math.inf).max()):.3g} over its tolerance, first at "
                      f"{torch.nonzero(~ok)[0].tolist()}: {float(got[~ok][0]):.6g} for {float(out[~ok][0]):.6g}")


def starts(counts, first=0):
    s = [first]
    for c in counts:
        s.append(s[-1] + c)
    return s


def paged(k, v, k_start, bs, order, spare=2, fill=math.nan):
    """Pools and tables that hold contiguous rows; free places hold `fill`,
    table entries behind a sequence ids outside the pool."""
    lens = [b - a for a, b in zip(k_start, k_start[1:])]
    need = [-(-L // bs) for L in lens]
    NB = sum(need) + spare
    perm = torch.randperm(NB, generator=order).tolist()
    kc = torch.full((NB, bs) + tuple(k.shape[1:]), fill, dtype=k.dtype, device=k.device)
    vc = kc.clone()
    bt = torch.full((max(1, len(lens)), max(need + [0]) + 2), NB + 5, dtype=torch.int32)
    bt[:, 1::2] = -1
    at = 0
    for i, (n, L) in enumerate(zip(need, lens)):
        bt[i, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
        pos = torch.arange(L)
        blk, off = bt[i].long()[pos // bs].to(k.device), (pos % bs).to(k.device)
        kc[blk, off], vc[blk, off] = k[k_start[i]:k_start[i + 1]], v[k_start[i]:k_start[i + 1]]
    return kc, vc, bt.to(k.device), torch.tensor(lens, dtype=torch.int32, device=k.device)
