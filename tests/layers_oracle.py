"""fp64 definitions of the convolution, the selective scan and masked window attention, written token by
token from the formulas, each with a bound on what a kernel in fp32 arithmetic may be off by.

The bounds are first-order error analyses, evaluated beside the results: U = 2^-24 is the half step of an fp32
rounding, ``half_step(dtype)`` that of the output's type.  CUDA documents expf's fast form with 2 + 1.173 |x| ulp
(an ulp is 2 U) and the fast quotient with 2 ulp; the approximate base-2 exponential has a relative error of 2^-22.
"""
import numpy as np
import torch

U = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _silu(x):
    return x / (1 + np.exp(-x))


def _silu_err(x):
    """relative error of x / (1 + exp(-x)): the exponential's, the sum's and the quotient's"""
    return (2 * (2 + 1.2 * np.abs(x)) + 1 + 4) * U


def conv(x, w, bias, state, lens, silu, out_dtype):
    """Returns (y, bound, state); rows of padding are NaN in y."""
    B, N, C = x.shape
    W = w.shape[1]
    x, w = f64(x), f64(w)
    bias = np.zeros(C) if bias is None else f64(bias)
    state = np.zeros((B, W - 1, C)) if state is None else f64(state)
    y, bound, last = np.full((B, N, C), np.nan), np.zeros((B, N, C)), np.empty((B, W - 1, C))
    for b in range(B):
        n = N if lens is None else int(lens[b])
        seq = np.concatenate([state[b], x[b, :n]])
        for t in range(n):
            terms = np.concatenate([bias[None], seq[t:t + W] * w.T])
            pre, mag = terms.sum(0), np.abs(terms).sum(0)
            err = (W + 2) * U * mag
            if silu:
                y[b, t] = _silu(pre)
                err = 1.1 * err + _silu_err(pre) * np.abs(y[b, t])  # |silu'| <= 1.1
            else:
                y[b, t] = pre
            bound[b, t] = err + half_step(out_dtype) * np.abs(y[b, t])
        last[b] = seq[n:]
    return y, bound, last


def ssm(u, delta, A, Bm, Cm, D, z, delta_bias, softplus, h, lens, out_dtype, segment=0):
    """Returns (y, y_bound, h, h_bound).  `segment`: tokens of a time segment where the scan is split, whose
    sum of steps has a rounding per token."""
    B, N, C = u.shape
    n, G = A.shape[1], Bm.shape[1]
    u, delta, A, Bm, Cm = (f64(t) for t in (u, delta, A, Bm, Cm))
    D = np.zeros(C) if D is None else f64(D)
    bias = np.zeros(C) if delta_bias is None else f64(delta_bias)
    zf = None if z is None else f64(z)
    h = np.zeros((B, C, n)) if h is None else f64(h).copy()
    e = np.zeros((B, C, n))
    y, bound = np.full((B, N, C), np.nan), np.zeros((B, N, C))
    group = np.arange(C) // (C // G)
    for b in range(B):
        for t in range(N if lens is None else int(lens[b])):
            raw = delta[b, t] + bias
            if softplus:
                dt = np.logaddexp(raw, 0)
                # the sum's rounding passes through with slope at most 1; then the exponential, the
                # quotient, the series' eight steps and the last sum
                e_dt = U * np.abs(raw) + dt * (2 * (2 + 1.2 * np.abs(raw)) + 24) * U
            else:
                dt = raw
                e_dt = U * np.abs(raw)
            Bt, Ct = Bm[b, group, t], Cm[b, group, t]  # [C, n]
            arg = dt[:, None] * A
            a = np.exp(arg)
            x = (dt * u[b, t])[:, None] * Bt
            e_a = 2.0 ** -22 + np.abs(arg) * (4 + segment) * U + e_dt[:, None] * np.abs(A)
            new = a * h[b] + x
            e[b] = a * e[b] + a * np.abs(h[b]) * (e_a + U) + e_dt[:, None] * np.abs(u[b, t][:, None] * Bt) + 3 * U * np.abs(x) + U * np.abs(new)
            h[b] = new
            terms = Ct * new
            pre = terms.sum(1) + D * u[b, t]
            err = (np.abs(Ct) * e[b]).sum(1) + (n + 4) * U * (np.abs(terms).sum(1) + np.abs(D * u[b, t]))
            if zf is not None:
                gate = _silu(zf[b, t])
                err = err * np.abs(gate) + np.abs(pre * gate) * (_silu_err(zf[b, t]) + U)
                pre = pre * gate
            y[b, t], bound[b, t] = pre, err + half_step(out_dtype) * np.abs(pre)
    return y, bound, h, e


def spans(Nq, Nk, B, window, key_lo, key_hi, q_pos0, lens):
    """[B, Nq] lists of (lo, hi): the keys each query sees; None for padding."""
    out = []
    for b in range(B):
        n = Nk if lens is None else int(lens[b])
        rows = []
        for i in range(Nq):
            p = q_pos0 + i
            if p >= n:
                rows.append(None)
                continue
            lo = max(0, int(key_lo[b, i]) if key_lo is not None else 0)
            hi = min(n, int(key_hi[b, i]) if key_hi is not None else p + 1)
            if window:
                lo = max(lo, p - window + 1)
            rows.append((lo, max(lo, hi)))
        out.append(rows)
    return out


def swa(q, k, v, scale, softcap, slopes, rows, q_pos0, out_dtype):
    """rows: spans().  Returns (o, bound); rows of padding are NaN."""
    in_dtype = q.dtype
    B, H, Nq, d = q.shape
    group = H // k.shape[1]
    q, k, v = f64(q), f64(k), f64(v)
    slopes = np.zeros(H) if slopes is None else f64(slopes)
    o, bound = np.full((B, H, Nq, d), np.nan), np.zeros((B, H, Nq, d))
    weight = half_step(in_dtype) if in_dtype == torch.bfloat16 else 0.0  # the weights' rounding for the product
    for b in range(B):
        for i in range(Nq):
            if rows[b][i] is None:
                continue
            lo, hi = rows[b][i]
            o[b, :, i] = 0
            if lo == hi:
                continue
            for h in range(H):
                kk, vv = k[b, h // group, lo:hi], v[b, h // group, lo:hi]
                terms = kk * q[b, h, i]
                s = scale * terms.sum(1)
                # sums on the tensor cores may cut off instead of rounding: 2 U a step
                es = (2 * d + 4) * U * abs(scale) * np.abs(terms).sum(1)
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                    # beyond half the cap: two quotients, an exponential and a sum, of values up to the cap, and the
                    # largest score is then above cap / 2.2; up to there a polynomial, off by 10 U of the score,
                    # and its six roundings
                    es = es + 16 * U * min(softcap, 2.2 * np.abs(s).max())
                dist = slopes[h] * np.abs(q_pos0 + i - np.arange(lo, hi))
                s = s - dist
                es = es + 2 * U * (dist + np.abs(s))
                m = s.max()
                w = np.exp(s - m)
                total = w.sum()
                # d(o)/d(s_j) = p_j (v_j - o); the exponential's own error beside the score's
                e_w = w * (es + es.max() + 2.0 ** -21 + 2 * U * np.abs(s - m))
                o[b, h, i] = w @ vv / total
                spread = np.abs(vv) + np.abs(o[b, h, i])
                err = (e_w[:, None] * spread).sum(0) / total
                err += (weight + (hi - lo + 4) * 2 * U) * (w @ np.abs(vv)) / total + weight * np.abs(o[b, h, i])
                bound[b, h, i] = err + half_step(out_dtype) * np.abs(o[b, h, i])
    return o, bound


def check(got, ref, bound, slack=1e-30):
    """got: tensor; every entry of ref that is not NaN is met within its bound."""
    got = got.detach().double().cpu().numpy()
    live = ~np.isnan(ref)
    off = np.abs(got - ref) - bound - slack
    assert np.all(np.isfinite(got[live])), "not finite"
    worst = np.max(np.where(live, off, -np.inf), initial=-np.inf)
    if worst > 0:
        at = np.unravel_index(np.argmax(np.where(live, off, -np.inf)), ref.shape)
        raise AssertionError(f"{got[at]} for {ref[at]} at {at}: off by {abs(got[at] - ref[at]):.3e}, bound {bound[at]:.3e}")
