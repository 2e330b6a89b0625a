"""fp64 definitions of the queries' and keys' norms with the position rotation, of the paged caches and of a step's
attention over them, each with a bound on what a kernel in fp32 arithmetic may be off by (first-order error analyses;
U = 2^-24 is the half step of an fp32 rounding)."""
import numpy as np
import torch

from tests.layers_oracle import U, check, f64, half_step  # noqa: F401

GROUP = 64


def tables(positions, rot, base=10000.0):
    """cos, sin fp32 [positions, rot / 2]."""
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    return torch.cos(angle).float(), torch.sin(angle).float()


def turn(x, cos, sin, interleaved):
    """x [..., d] with the pairs of its first elements turned, and |a c| + |b s| of each element; cos, sin [..., rot / 2]."""
    half = cos.shape[-1]
    y, mag = x.copy(), np.abs(x)
    first = np.arange(half) * 2 if interleaved else np.arange(half)
    second = first + (1 if interleaved else half)
    a, b = x[..., first], x[..., second]
    y[..., first], mag[..., first] = a * cos - b * sin, np.abs(a * cos) + np.abs(b * sin)
    y[..., second], mag[..., second] = b * cos + a * sin, np.abs(b * cos) + np.abs(a * sin)
    return y, mag


def norm_rope(x, weight, norm, eps, cos, sin, pos, interleaved, lens, out_dtype):
    """x [B, H, N, d]; pos [B, N] or None.  Returns (y, bound); rows of padding are NaN."""
    B, H, N, d = x.shape
    v = f64(x)
    if norm:
        ss = (v * v).sum(-1, keepdims=True)
        scale = 1 / np.sqrt((ss / d if norm == "rms" else ss) + eps)
        v = v * scale * (1.0 if weight is None else f64(weight))
    mag = np.abs(v)
    if cos is not None:
        c, s = f64(cos)[pos][:, None], f64(sin)[pos][:, None]
        v, mag = turn(v, c, s, interleaved)
    # the sum of squares is off by at most 8 + 5 steps of U of itself (eight terms a lane, five halvings), half of that
    # after the root; the share, eps and the root's 2 ulp; two products; the rotation's two roundings
    bound = (6.5 + 2 + 4 + 2 + 2) * U * mag + half_step(out_dtype) * np.abs(v)
    if lens is not None:
        for b, n in enumerate(lens):
            v[b, :, n:] = np.nan
    return v, bound


def quantise(x):
    """bf16-valued fp64 rows [..., d] -> (quotients [..., d], scales [..., d / 64], offsets): codes before their rounding, under
    the bf16 scale."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    lo, hi = g.min(-1), g.max(-1)
    scale = torch.from_numpy((hi - lo) / 15).float().to(torch.bfloat16).double().numpy()
    q = np.where(scale[..., None] > 0, (g - lo[..., None]) / np.where(scale > 0, scale, 1)[..., None], 0)
    return q.reshape(x.shape), scale, lo


def split(pages, d):
    """4-bit pages uint8 [P, H, page, 9 d / 16] -> (codes [P, H, page, d], scales, offsets [P, H, page, d / 64]), fp64, written
    from the layout in the header: page-wise codes, then bf16 pairs; word 2 e + g holds elements 64 g + 8 e + (0..7)."""
    raw = pages.cpu().contiguous().numpy()
    P, H, page, _ = raw.shape
    groups = d // GROUP
    raw = raw.reshape(P, H, -1)
    words = np.ascontiguousarray(raw[..., :page * d // 2]).view(np.uint32).reshape(P, H, page, d // 8)
    codes = np.zeros((P, H, page, d))
    for w in range(d // 8):
        g, e = w % groups, w // groups
        for j in range(8):
            codes[..., GROUP * g + 8 * e + j] = words[..., w] >> np.uint32(4 * j) & np.uint32(15)
    meta = np.ascontiguousarray(raw[..., page * d // 2:]).view(np.uint32).reshape(P, H, page, groups)
    scale = (meta << np.uint32(16)).view(np.float32).astype(np.float64)
    offset = (meta & np.uint32(0xffff0000)).view(np.float32).astype(np.float64)
    return codes, scale, offset


def values(pages, d):
    """Pages of any kind as fp64 elements [P, H, page, d] and the magnitudes their arithmetic meets."""
    if pages.dtype != torch.uint8:
        x = f64(pages)
        return x, np.abs(x)
    codes, scale, offset = split(pages, d)
    s, o = np.repeat(scale, GROUP, -1), np.repeat(offset, GROUP, -1)
    return o + s * codes, np.abs(o) + 32 * np.abs(s)


def gather(x, table, b, lo, hi):
    """Tokens lo .. hi - 1 of sequence b: [H, hi - lo, d]."""
    page = x.shape[2]
    p = np.arange(lo, hi)
    at = table[b].cpu().numpy()[p // page]
    return x[at, :, p % page].transpose(1, 0, 2)


def step(q, k_pages, v_pages, table, lens, window, scale, softcap, slopes, out_dtype):
    """q [S, H, d].  Returns (o, bound)."""
    S, H, d = q.shape
    (k, km), (v, vm) = values(k_pages, d), values(v_pages, d)
    group = H // k.shape[1]
    weight = 2.0 ** -16 if q.dtype == torch.bfloat16 else 0.0  # two bf16 parts: 2^-17 of a weight, and of its product with a scale
    q = f64(q)
    sl = np.zeros(H) if slopes is None else f64(slopes)
    o, bound = np.zeros((S, H, d)), np.zeros((S, H, d))
    for s in range(S):
        n = int(lens[s])
        lo = max(0, n - window) if window else 0
        if n == 0:
            continue
        kk, kkm, vv, vvm = (gather(x, table, s, lo, n) for x in (k, km, v, vm))
        for h in range(H):
            g = h // group
            x = scale * (kk[g] * q[s, h]).sum(1)
            # sums on the tensor cores may cut off instead of rounding: 2 U a step
            es = (2 * d + 8) * U * abs(scale) * (kkm[g] * np.abs(q[s, h])).sum(1)
            if softcap:
                x = softcap * np.tanh(x / softcap)
                es = es + 16 * U * min(softcap, 2.2 * np.abs(x).max())
            dist = sl[h] * (n - 1 - np.arange(lo, n))
            x = x - dist
            es = es + 5 * U * (dist + np.abs(x))
            m = x.max()
            w = np.exp(x - m)
            total = w.sum()
            # d(o)/d(x_j) = p_j (v_j - o); the exponential's own error beside the score's, the tile's maximum and the part's
            e_w = w * (es + es.max() + 3 * 2.0 ** -21 + 4 * U * np.abs(x - m))
            o[s, h] = w @ vv[g] / total
            err = (e_w[:, None] * (np.abs(vv[g]) + np.abs(o[s, h]))).sum(0) / total
            err += (weight + (n - lo + 8) * 2 * U) * (w @ vvm[g]) / total + (weight + 4 * U) * np.abs(o[s, h])
            bound[s, h] = err + half_step(out_dtype) * np.abs(o[s, h])
    return o, bound
