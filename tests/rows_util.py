"""Bounds of the row operators' fp32 arithmetic against the fp64 oracle (test helper).

U = 2^-24 is half a step of fp32, E2 = 2^-22 the error of the hardware's base-2 exponential
(ex2.approx: relative 2^-22). A sum formed by d additions in sequence and in a tree carries at most
d U times the sum of its terms' sizes, where d is the number of additions on the longest way from a
term to the result. The output is rounded once: half a step of its type, relative eps / 2, or half
the smallest subnormal.
"""

import numpy as np
import torch

U, E2, LN2 = 2.0 ** -24, 2.0 ** -22, float(np.log(2.0))

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_SUBNORMAL = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}


def half_step(v, dtype):
    return np.abs(v) * torch.finfo(DTYPES[dtype]).eps / 2 + HALF_SUBNORMAL[dtype]


def rounded(v, err, dtype):
    """Bound of an output whose value before its one rounding is within err of v."""
    return err + half_step(np.abs(v) + err, dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def check(got, ref, tol, what):
    g = f64(got) if isinstance(got, torch.Tensor) else np.asarray(got, np.float64)
    assert g.shape == np.shape(ref), what
    same = (g == ref) | (np.isnan(g) & np.isnan(ref))  # infinities and NaN in their places
    with np.errstate(invalid="ignore"):
        err = np.where(same, 0.0, np.abs(g - ref))
    tol = np.broadcast_to(np.asarray(tol, np.float64), err.shape)
    with np.errstate(invalid="ignore", divide="ignore"):
        bad = ~((err <= tol) | same)
    worst = float(np.max(np.where(same, 0.0, err / np.maximum(tol, 1e-300)))) if err.size else 0.0
    print(f"  {what}: max|err| {float(np.max(err)) if err.size else 0:.3e} worst/tol {worst:.3f}")
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, worst/tol {worst:.3f}"


def norm_bounds(x, gamma, beta, y, mean, rstd, eps):
    """Errors of (y before rounding, mean, rstd). Longest way of a row's sum: one element of 32 per
    thread and 16 more additions across threads."""
    H = x.shape[1]
    d = -(-H // 32) + 16
    dm = (d + 2) * U * np.abs(x).mean(1)
    dev = x - mean[:, None]
    var = (dev * dev).mean(1)
    dvar = (d + 6) * U * var + 2 * dm * np.abs(dev).mean(1) + dm * dm
    rel = 0.5 * dvar / (var + eps) + 4 * U  # of rstd (first order; the second is far below U)
    xh = np.abs(dev) * rstd[:, None]
    g = np.ones(H) if gamma is None else np.abs(gamma)
    b = np.zeros(H) if beta is None else np.abs(beta)
    ey = g * (rstd[:, None] * (U * np.abs(dev) + dm[:, None]) * (1 + rel[:, None])
              + xh * (rel[:, None] + 3 * U)) + 2 * U * (np.abs(y) + b)
    return ey, dm, rstd * rel


def norm_bwd_bounds(d_y, x, gamma, mean, rstd, dtype="fp32"):
    """Errors of (d_x before rounding, d_gamma, d_beta). Token sums: fewer than T / 64 + 96
    additions in sequence where tokens are spread over 64 chains or more, and never above T.
    16-bit rows form (x - mean) f as x f + (c - mean f), f = r^2 c2 in size: the bracket and the sum
    are rounded at the size of mean f, U each."""
    T, H = x.shape
    d = -(-H // 32) + 16
    r = rstd[:, None]
    xh = np.abs(x - mean[:, None]) * r
    q = np.abs(d_y) * (1.0 if gamma is None else np.abs(gamma))
    c1, c2 = q.mean(1, keepdims=True), (q * xh).mean(1, keepdims=True)  # of sizes
    dc1, dc2 = (d + 4) * U * c1, (d + 8) * U * c2
    ex = r * (U * q + dc1 + xh * dc2 + 4 * U * xh * c2 + 4 * U * (q + c1 + xh * c2))
    if dtype != "fp32":
        ex = ex + 2 * U * r * (np.abs(mean)[:, None] * r) * c2
    n = min(T, -(-T // 64) + 96) + 4
    eg = (n + 4) * U * (np.abs(d_y) * xh).sum(0)
    eb = n * U * np.abs(d_y).sum(0)
    return ex, eg, eb


def row_sum_error(z, m, tau):
    """Relative error of s = sum exp((z - m) / tau), per row: E2 for each term and for each change
    of a thread's running maximum (at most one per round of windows, which are V / 4096 + 1 at most,
    and three joins; 2 U for its factor and product), the additions, and U |d| in each exponent d
    (twice: its scale and its rounding). Additions: a thread adds its elements two at a time. It has
    at most 8 windows of 8 elements up to V = 2048 (32 threads), 16 windows up to V = 16384 (128
    threads) and V / 256 + 8 elements beyond; then come one addition of the pair, five and seven over
    the threads and seven over the CTAs of a row."""
    z = np.asarray(z, np.float64)
    V = z.shape[1]
    tiles = -(-V // 4096) + 3
    adds = (64 if V <= 2048 else 128 if V <= 16384 else V / 256 + 8) / 2 + 20
    base = np.where(np.isfinite(m), m, 0.0)[:, None]
    with np.errstate(invalid="ignore", over="ignore"):
        d = (z - base) / tau / LN2
        e = np.exp2(d)
        mean_d = np.where(e > 0, e * np.abs(d), 0).sum(1) / np.maximum(e.sum(1), 1e-300)
    return (tiles + 2) * E2 + (2 * tiles + adds) * U + 2 * LN2 * U * (2 * mean_d + 1)


def logprob_bounds(r, z, tau):
    """Errors of (ln p at any index, entropy, s) for oracle.rows.token_logprobs's result r."""
    m, s, lp = r["m"], r["s"], r["lp"]
    rs = row_sum_error(z, m, tau)
    with np.errstate(invalid="ignore", divide="ignore"):
        ln_s = np.abs(np.where(s > 0, np.log(s), 0.0))
        fin = np.where(np.isfinite(lp), np.abs(lp), 0.0)
        e_lp = rs[:, None] + 4 * U * (fin + 2 * ln_s[:, None] + 1)
        ent = np.abs(r["entropy"])
        # u / s = sum p |d|: as a quotient of two sums, each within rs; u is ent + ln s in size
        e_ent = rs + (2 * rs + 6 * U) * (ent + ln_s) + 4 * U * (ln_s + ent + 1)
    return e_lp, e_ent, rs * np.abs(s)


def grad_bounds(lp, ent, tau, glp, gent, ds):
    """Error of the logits' gradient before rounding: p within E2, the roundings of its exponent and
    ds (relative error of the s given); the entropy term's bracket is a difference of sizes |ln p|,
    ln s (<= |ln p| + 1 in effect: s >= 1) and entropy, each rounded, and 1 / temperature."""
    with np.errstate(invalid="ignore"):
        p = np.where(np.isfinite(lp), np.exp(lp), 0.0)
        a = np.where(p > 0, np.abs(lp), 0.0)
    rel = E2 + (4 * a + 12) * U + ds
    big = np.log(lp.shape[1])  # ln s <= ln V
    g, h, e = np.abs(glp)[:, None], np.abs(gent)[:, None], ent[:, None]
    return (p * rel * (g + h * (a + e)) + p * h * 8 * U * (a + e + big + 1) + 4 * U * g
            * (p + 1e-30)) / tau
