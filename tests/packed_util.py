"""Plain 64-bit attention and the error bounds of the packed and paged kernels.

Bounds, from the kernels' arithmetic (u = half a step of the 16-bit type, f = 2^-24):
  * a score is an fp32 sum of D products: off by at most e = (D + 2) f scale sum_d |q_d k_d|,
    and its exponent argument by a few roundings of |s| log2(e): 4 f |s|;
  * a weight is rounded to the 16-bit type (u relative), ex2 to 2^-22, the row sum over n
    weights to (64 + n / 128 + 8) f; numerator and denominator both carry the score error;
  * the output is rounded once (u relative).
So with A = sum_j p_j |v_j|:  |dO| <= u |O| + (1 + u) (u + 2 (e + 4 f |s|) + 2^-21 + 2 (72 + n / 128) f) A,
and |dLSE| <= e + (8 |s| + 72 + n / 128 + 2 |LSE|) f + 2^-21.  A merge of up to `pieces` partial
results adds (pieces + 8) f to both.
"""
import math

import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
F = 2.0 ** -24


def plain(q, k, v, see, scale, dtype, pieces=0):
    """q [T, D], k, v [n, D] of one head, see [T, n] bool: (O, LSE, bound of O, bound of LSE) in 64 bits."""
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    see = see.cpu()
    T, D = q.shape
    n = k.shape[0]
    if n == 0:
        z = torch.zeros(T, D, dtype=torch.float64)
        return z, torch.full((T,), -math.inf, dtype=torch.float64), z, z[:, 0]
    s = (q @ k.T) * scale
    mag = (q.abs() @ k.abs().T) * scale
    s = torch.where(see, s, -math.inf)
    m = s.amax(1, keepdim=True)
    none = m.squeeze(1) == -math.inf
    p = torch.exp(torch.where(see, s - torch.where(none[:, None], 0.0, m), -math.inf))
    total = p.sum(1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    # a key that is not seen contributes nothing, whatever its value is
    o = torch.zeros(T, D, dtype=torch.float64)
    a = torch.zeros(T, D, dtype=torch.float64)
    if torch.isfinite(v).all():
        o, a = p @ v, p @ v.abs()
    else:
        for t in range(T):
            w, x = p[t][see[t]], v[see[t]]
            o[t], a[t] = (w[:, None] * x).sum(0), (w[:, None] * x.abs()).sum(0)
    lse = (m + total.log()).squeeze(1)
    lse[none] = -math.inf
    big = torch.where(see, s.abs(), 0.0).nan_to_num(0, 0, 0).amax(1)
    e = (D + 2) * F * torch.where(see, mag, 0.0).nan_to_num(0, 0, 0).amax(1)
    u = torch.finfo(DT[dtype]).eps / 2
    add = (72 + n / 128 + pieces + 8) * F + 2.0 ** -21
    tol = u * o.abs() + (1 + u) * (u + 2 * (e + 4 * F * big) + 2 * add)[:, None] * a + 1e-30
    # a weight below the 16-bit type's smallest normal number is rounded to its fixed step
    if dtype == "f16":
        tol = tol + n * 2.0 ** -25 * v.abs().nan_to_num(0, 0, 0).amax() + 2.0 ** -25
    ltol = e + (8 * big + 2 * lse.abs().nan_to_num(0, 0, 0)) * F + add
    return o, lse, tol, ltol


def close(got, want, tol, what):
    got = got.double().cpu()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    off = (got - want).abs()
    ok = same | (off <= tol)
    if not bool(ok.all()):
        i = int((~ok).reshape(-1).nonzero()[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} values off; first at {i}: got "
                             f"{got.reshape(-1)[i]:.6g}, want {want.reshape(-1)[i]:.6g}, bound {tol.reshape(-1)[i]:.3g}")


def causal(Nq, Nk):
    return torch.ones(Nq, Nk, dtype=torch.bool).tril(Nk - Nq)


def offsets(lens, device="cuda"):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)) if lens else [0], dtype=torch.int32, device=device)
