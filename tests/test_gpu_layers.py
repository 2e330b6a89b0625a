"""GPU parity of the short causal convolution, the selective state space scan and masked window attention over
prompts, and of their one-token steps, against fp64 definitions with per-entry error bounds."""
import numpy as np
import pytest
import torch

import linear_attention_recurrence_chunked_gb300 as la
from tests import layers_oracle as ref
from tests.helpers import cuda_device

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=FP, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def pad_rows(t, dev, fill=float("nan")):
    """The tensor on the device as rows of a wider buffer: row starts on 16 bytes, what lies between unreadable as numbers."""
    C = t.shape[-1]
    wide = torch.full((*t.shape[:-1], -(-C // 8) * 8 + 8), fill, dtype=t.dtype, device=dev)
    wide[..., :C] = t.to(dev)
    return wide[..., :C]


def on(dev, *ts):
    return [None if t is None else t.to(dev) for t in ts]


# ------------------------------------------------------------------------------------------ convolution
@pytest.mark.parametrize("B,N,C,W,dtype,w_dtype,out,silu,bias,state,lens", [
    (1, 1, 8, 4, BF, BF, BF, True, True, True, None),
    (2, 2, 1, 4, BF, FP, FP, True, False, True, None),
    (3, 77, 1001, 4, BF, BF, BF, True, True, False, [77, 0, 2]),
    (2, 33, 12, 3, FP, BF, FP, False, True, True, [1, 33]),
    (2, 40, 20, 2, FP, FP, BF, True, False, True, None),
    (1, 300, 264, 3, BF, BF, FP, False, False, True, [299]),
    (4, 9, 64, 4, FP, FP, FP, True, True, True, [0, 1, 3, 9]),
])
def test_conv_prefill(B, N, C, W, dtype, w_dtype, out, silu, bias, state, lens):
    dev = cuda_device()
    g = gen(N * 7 + C)
    x, w = randn(g, B, N, C, dtype=dtype), randn(g, C, W, dtype=w_dtype, scale=0.5)
    bs = randn(g, C, dtype=w_dtype) if bias else None
    st = randn(g, B, W - 1, C, dtype=dtype) if state else None
    y_ref, bound, last = ref.conv(x, w, bs, st, lens, silu, out)
    xd = pad_rows(x, dev)
    ln = None
    if lens is not None:
        ln = torch.tensor(lens, dtype=torch.int64, device=dev)
        for b, n in enumerate(lens):
            xd[b, n:] = float("nan")  # padding reaches nothing
    y = pad_rows(torch.full((B, N, C), 5.0, dtype=out), dev)
    wd, bd, sd = on(dev, w, bs, st)
    got, s_out = la.la_conv_prefill(xd, wd, bias=bd, state_in=sd, lens=ln, silu=silu, y=y)
    ref.check(got, y_ref, bound)
    assert torch.equal(s_out.double().cpu(), torch.from_numpy(last))
    for b, n in enumerate(lens or []):
        assert torch.all(got[b, n:] == 5.0)  # rows of padding stay
    if sd is not None:  # in place
        la.la_conv_prefill(xd, wd, bias=bd, state_in=sd, state_out=sd, lens=ln, silu=silu)
        assert torch.equal(sd, s_out)
    assert la.la_device_status() == la.LA_OK


@pytest.mark.parametrize("dtype,W,C", [(BF, 4, 72), (FP, 3, 13), (BF, 2, 9)])
def test_conv_steps_continue_a_prompt(dtype, W, C):
    dev = cuda_device()
    S, N, steps = 3, 21, 6
    g = gen(C)
    x, w, bias = randn(g, S, N + steps, C, dtype=dtype), randn(g, C, W, dtype=dtype, scale=0.5), randn(g, C, dtype=dtype)
    y_ref, bound, last = ref.conv(x, w, bias, None, None, True, dtype)
    xd, wd, bd = pad_rows(x, dev), w.to(dev), bias.to(dev)
    _, state = la.la_conv_prefill(xd[:, :N], wd, bias=bd)
    for t in range(steps):
        out = la.la_conv_decode_step(xd[:, N + t], wd, state, bias=bd)
        ref.check(out, y_ref[:, N + t], bound[:, N + t])
    assert torch.equal(state.double().cpu(), torch.from_numpy(last))


# ------------------------------------------------------------------------------------------ selective scan
def ssm_inputs(B, N, C, n, G, dtype, z, seed):
    g = gen(seed)
    A = -(0.05 + torch.rand((C, n), generator=g) * 4)
    t = {"u": randn(g, B, N, C, dtype=dtype), "delta": randn(g, B, N, C, dtype=dtype), "A": A,
         "Bm": randn(g, B, G, N, n, dtype=dtype), "Cm": randn(g, B, G, N, n, dtype=dtype), "D": randn(g, C),
         "z": randn(g, B, N, C, dtype=dtype) if z else None, "bias": randn(g, C) - 3, "h": randn(g, B, C, n)}
    return t


@pytest.mark.parametrize("B,N,C,n,G,dtype,out,z,softplus,state,lens", [
    (1, 1, 8, 16, 1, BF, BF, True, True, True, None),
    (2, 37, 40, 16, 2, BF, BF, True, True, True, [37, 0]),
    (2, 70, 33, 4, 1, FP, FP, False, True, True, None),
    (1, 65, 130, 8, 1, BF, FP, True, True, False, [33]),
    (3, 129, 24, 24, 3, FP, FP, True, True, True, [129, 128, 1]),
    (1, 100, 10, 64, 2, BF, BF, False, True, True, None),
    (1, 50, 16, 33, 1, FP, BF, True, True, True, None),
    (2, 31, 7, 1, 1, FP, FP, True, True, False, None),
    (1, 40, 21, 7, 3, BF, BF, True, False, True, None),
    (1, 2000, 48, 16, 1, BF, BF, True, True, True, None),      # time segments
    (2, 1500, 24, 8, 1, FP, FP, True, True, True, [700, 1499]),
])
def test_ssm_prefill(B, N, C, n, G, dtype, out, z, softplus, state, lens):
    dev = cuda_device()
    t = ssm_inputs(B, N, C, n, G, dtype, z, N + C)
    if not softplus:
        t["delta"] = t["delta"].abs() * 0.2
        t["bias"] = t["bias"].abs() * 0.1
    h0 = t["h"] if state else None
    y_ref, bound, h_ref, h_bound = ref.ssm(t["u"], t["delta"], t["A"], t["Bm"], t["Cm"], t["D"], t["z"], t["bias"],
                                           softplus, h0, lens, out, segment=N)
    ud, dd = pad_rows(t["u"], dev), pad_rows(t["delta"], dev)
    zd = pad_rows(t["z"], dev) if z else None
    # B and C as slices of one projection, at an odd offset
    proj = torch.full((B, N, 2 * G * n + 1), float("nan"), dtype=dtype, device=dev)
    proj[..., 1:] = torch.cat([t["Bm"].transpose(1, 2).reshape(B, N, G * n), t["Cm"].transpose(1, 2).reshape(B, N, G * n)], -1).to(dev)
    Bd = proj[..., 1:1 + G * n].unflatten(-1, (G, n)).transpose(1, 2)
    Cd = proj[..., 1 + G * n:].unflatten(-1, (G, n)).transpose(1, 2)
    ln = None
    if lens is not None:
        ln = torch.tensor(lens, dtype=torch.int64, device=dev)
        for b, m in enumerate(lens):
            for x in (ud, dd, zd, proj):
                if x is not None:
                    x[b, m:] = float("nan")
    y = pad_rows(torch.full((B, N, C), 5.0, dtype=out), dev)
    Ad, Dd, bd, hd = on(dev, t["A"], t["D"], t["bias"], h0)
    kw = dict(D=Dd, z=zd, delta_bias=bd, delta_softplus=softplus, lens=ln)
    got, h = la.la_ssm_prefill(ud, dd, Ad, Bd, Cd, h_in=hd, y=y, **kw)
    ref.check(h, h_ref, h_bound)
    ref.check(got, y_ref, bound)
    for b, m in enumerate(lens or []):
        assert torch.all(got[b, m:] == 5.0)
    if hd is not None:  # in place, the same bits
        _, h2 = la.la_ssm_prefill(ud, dd, Ad, Bd, Cd, h_in=hd, h_out=hd, **kw)
        assert torch.equal(h2, h)
    assert la.la_device_status() == la.LA_OK


def test_ssm_long_memory():
    """States that forget over thousands of tokens: the decays' errors must not add up to a bias."""
    dev = cuda_device()
    B, N, C, n = 1, 6000, 32, 16
    t = ssm_inputs(B, N, C, n, 1, BF, False, 5)
    t["A"] = t["A"] * 0 - torch.linspace(0.2, 1.5, n)
    t["bias"] = torch.full((C,), -7.5)  # steps near 5e-4
    y_ref, bound, h_ref, _ = ref.ssm(t["u"], t["delta"], t["A"], t["Bm"], t["Cm"], t["D"], None, t["bias"], True, None, None, FP,
                                     segment=256)
    u, delta, A, Bm, Cm, D, bias = on(dev, *(t[k] for k in ("u", "delta", "A", "Bm", "Cm", "D", "bias")))
    y, h = la.la_ssm_prefill(u, delta, A, Bm, Cm, D=D, delta_bias=bias, out_dtype=FP)
    err = np.linalg.norm(h.double().cpu().numpy() - h_ref) / np.linalg.norm(h_ref)
    # about 3000 tokens of memory; each rounding of 2^-24 enters at random: sqrt(3000) 2^-24 = 3.3e-6, three of them a step
    assert err < 1e-5
    ref.check(y, y_ref, bound)


@pytest.mark.parametrize("dtype,n,G,C", [(BF, 16, 1, 40), (FP, 24, 2, 18), (BF, 7, 1, 9), (BF, 64, 1, 12), (FP, 4, 1, 70), (BF, 8, 3, 33)])
def test_ssm_steps_continue_a_prompt(dtype, n, G, C):
    dev = cuda_device()
    S, N, steps = 5, 19, 5
    t = ssm_inputs(S, N + steps, C, n, G, dtype, True, C + n)
    y_ref, bound, h_ref, h_bound = ref.ssm(t["u"], t["delta"], t["A"], t["Bm"], t["Cm"], t["D"], t["z"], t["bias"], True, None, None, dtype)
    u, delta, z = (pad_rows(t[k], dev) for k in ("u", "delta", "z"))
    A, Bm, Cm, D, bias = on(dev, *(t[k] for k in ("A", "Bm", "Cm", "D", "bias")))
    kw = dict(D=D, delta_bias=bias)
    _, h = la.la_ssm_prefill(u[:, :N], delta[:, :N], A, Bm[:, :, :N], Cm[:, :, :N], z=z[:, :N], **kw)
    for i in range(N, N + steps):
        before = h.clone()
        other = torch.empty_like(h)
        out2 = la.la_ssm_decode_step(u[:, i], delta[:, i], A, Bm[:, :, i], Cm[:, :, i], h, z=z[:, i], state_out=other, **kw)
        assert torch.equal(h, before)
        out = la.la_ssm_decode_step(u[:, i], delta[:, i], A, Bm[:, :, i], Cm[:, :, i], h, z=z[:, i], **kw)
        assert torch.equal(h, other) and torch.equal(out, out2)
        ref.check(out, y_ref[:, i], bound[:, i])
    ref.check(h, h_ref, h_bound)


# ------------------------------------------------------------------------------------------ attention
def swa_case(B, H, Hkv, Nq, Nk, d, dtype, seed):
    g = gen(seed)
    return (randn(g, B, Nq, H, d, dtype=dtype, scale=1.5).transpose(1, 2), randn(g, B, Nk, Hkv, d, dtype=dtype, scale=1.5).transpose(1, 2),
            randn(g, B, Nk, Hkv, d, dtype=dtype).transpose(1, 2))


def slopes_of(H):
    return torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H)


def run_swa(q, k, v, out, window=0, softcap=0.0, slopes=None, key_lo=None, key_hi=None, q_pos0=None, lens=None, cache=False):
    dev = cuda_device()
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    pos0 = Nk - Nq if q_pos0 is None else q_pos0
    rows = ref.spans(Nq, Nk, B, window, key_lo, key_hi, pos0, lens)
    o_ref, bound = ref.swa(q, k, v, d ** -0.5, softcap, slopes, rows, pos0, out)
    qd, kd, vd, sl, lo, hi = on(dev, q, k, v, slopes, key_lo, key_hi)
    ln = None
    if lens is not None:
        ln = torch.tensor(lens, dtype=torch.int64, device=dev)
        for b, n in enumerate(lens):
            kd[b, :, n:] = float("nan")
            vd[b, :, n:] = float("nan")
            qd[b, :, max(0, n - pos0):] = float("nan")
    o = torch.full((B, Nq, H, d), 5.0, dtype=out, device=dev).transpose(1, 2)
    kc = torch.full((B, Hkv, window, d), 3.0, dtype=q.dtype, device=dev) if cache else None
    vc = torch.full((B, Hkv, window, d), 3.0, dtype=q.dtype, device=dev) if cache else None
    la.la_swa_prefill(qd, kd, vd, window=window, softcap=softcap, slopes=sl, key_lo=lo, key_hi=hi, q_pos0=q_pos0, lens=ln, o=o,
                      k_cache=kc, v_cache=vc)
    assert la.la_device_status() == la.LA_OK
    ref.check(o, o_ref, bound)
    for b in range(B):
        for i in range(Nq):
            if rows[b][i] is None:
                assert torch.all(o[b, :, i] == 5.0)
            elif rows[b][i][0] == rows[b][i][1]:
                assert torch.all(o[b, :, i] == 0.0)
    if cache:
        for b in range(B):
            n = Nk if lens is None else lens[b]
            want_k, want_v = torch.full((Hkv, window, d), 3.0, dtype=q.dtype), torch.full((Hkv, window, d), 3.0, dtype=q.dtype)
            for p in range(max(0, n - window), n):
                want_k[:, p % window], want_v[:, p % window] = k[b, :, p], v[b, :, p]
            assert torch.equal(kc[b].cpu(), want_k) and torch.equal(vc[b].cpu(), want_v)
    return o


@pytest.mark.parametrize("dtype,out", [(BF, BF), (FP, FP), (BF, FP), (FP, BF)])
@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,d,window,softcap,slopes,lens,cache", [
    (1, 2, 2, 1, 1, 64, 0, 0.0, False, None, False),
    (2, 4, 2, 77, 77, 64, 64, 0.0, False, None, True),
    (1, 3, 1, 300, 300, 128, 0, 0.0, False, None, False),
    (2, 4, 4, 130, 130, 40, 17, 0.0, True, [130, 64], True),
    (2, 6, 3, 133, 333, 96, 200, 20.0, True, None, True),
    (1, 8, 1, 129, 257, 8, 0, 30.0, False, None, False),
    (3, 2, 1, 256, 256, 72, 1, 0.0, False, [0, 1, 255], True),
    (1, 2, 2, 400, 400, 128, 130, 50.0, True, [399], True),
])
def test_swa_prefill(B, H, Hkv, Nq, Nk, d, window, softcap, slopes, lens, cache, dtype, out):
    q, k, v = swa_case(B, H, Hkv, Nq, Nk, d, dtype, Nq + d)
    run_swa(q, k, v, out, window, softcap, slopes_of(H) if slopes else None, lens=lens, cache=cache)


def intervals(B, N, docs, prefix, empty):
    """Packed documents of the given lengths, a bidirectional prefix in each, every `empty`-th row sees nothing."""
    lo, hi = torch.zeros((B, N), dtype=torch.int32), torch.zeros((B, N), dtype=torch.int32)
    for b in range(B):
        at, which = 0, b
        while at < N:
            end = min(N, at + docs[which % len(docs)])
            for i in range(at, end):
                lo[b, i], hi[b, i] = at, max(i + 1, min(end, at + prefix))
                if empty and i % empty == empty - 1:
                    hi[b, i] = lo[b, i]
            at, which = end, which + 1
    return lo, hi


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("N,docs,prefix,empty,window,d", [
    (300, [1, 70, 128, 5], 0, 0, 0, 64), (300, [90, 40], 33, 7, 0, 128), (515, [200, 3, 129], 20, 5, 50, 96),
    (140, [140], 140, 0, 0, 64), (260, [64], 64, 2, 0, 32)])
def test_swa_documents_and_prefixes(N, docs, prefix, empty, window, d, dtype):
    q, k, v = swa_case(2, 4, 2, N, N, d, dtype, N)
    lo, hi = intervals(2, N, docs, prefix, empty)
    run_swa(q, k, v, dtype, window=window, slopes=slopes_of(4), key_lo=lo, key_hi=hi)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_swa_out_of_range_intervals_are_clamped_and_no_row_sees_anything(dtype):
    q, k, v = swa_case(1, 2, 2, 150, 150, 64, dtype, 3)
    lo = torch.full((1, 150), -(1 << 31), dtype=torch.int32)
    hi = torch.full((1, 150), (1 << 31) - 1, dtype=torch.int32)
    run_swa(q, k, v, dtype, key_lo=lo, key_hi=hi)           # everything sees everything
    run_swa(q, k, v, dtype, window=9, key_lo=lo, key_hi=hi)  # and from 8 back to the end
    run_swa(q, k, v, dtype, key_lo=hi, key_hi=lo)            # nothing


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_swa_masked_keys_and_values_reach_nothing(bad, dtype):
    """One token's key and value are not finite: queries that do not see it keep their bits."""
    dev = cuda_device()
    N, at, window = 300, 141, 60
    q, k, v = (t.to(dev) for t in swa_case(1, 4, 2, N, N, 64, dtype, 9))
    clean = la.la_swa_prefill(q, k, v, window=window)
    k, v = k.clone(), v.clone()
    k[0, :, at] = bad
    v[0, :, at, 5] = bad
    o = la.la_swa_prefill(q, k, v, window=window)
    sees = torch.zeros(N, dtype=torch.bool, device=dev)
    sees[at:at + window] = True
    assert torch.isfinite(o[:, :, ~sees]).all()
    assert (o[:, :, ~sees].float() - clean[:, :, ~sees].float()).abs().max() < 2e-2  # another order of sums at most
    v2 = v.clone()
    k2, _ = swa_case(1, 4, 2, N, N, 64, dtype, 9)[1].to(dev), None
    o2 = la.la_swa_prefill(q, k2, v2, window=window)
    assert la.la_device_status() == la.LA_OK
    assert torch.isnan(o2[0, :, at:at + window, 5]).all() or torch.isinf(o2[0, :, at:at + window, 5]).all()
    assert torch.isfinite(o2[0, :, :, 6]).all()


@pytest.mark.parametrize("dtype,H,Hkv,d,window,softcap,slopes", [
    (BF, 4, 4, 64, 64, 0.0, False), (BF, 8, 2, 128, 256, 30.0, True), (FP, 6, 3, 40, 33, 20.0, True), (BF, 16, 1, 72, 100, 0.0, True),
    (FP, 3, 1, 128, 256, 0.0, False), (BF, 2, 2, 8, 1, 0.0, True), (BF, 12, 4, 96, 200, 50.0, False)])
def test_swa_steps_continue_a_prompt(dtype, H, Hkv, d, window, softcap, slopes):
    dev = cuda_device()
    S, N, steps = 3, 90, 6
    q, k, v = swa_case(S, H, Hkv, N + steps, N + steps, d, dtype, d + H)
    sl = slopes_of(H) if slopes else None
    lens = [N, 0, 17]
    rows = ref.spans(N + steps, N + steps, S, window, None, None, 0, None)
    o_ref, bound = ref.swa(q, k, v, d ** -0.5, softcap, sl, rows, 0, dtype)
    qd, kd, vd, sld = on(dev, q, k, v, sl)
    kc, vc = (torch.zeros((S, Hkv, window, d), dtype=dtype, device=dev) for _ in range(2))
    ln = torch.tensor(lens, dtype=torch.int64, device=dev)
    la.la_swa_prefill(qd[:, :, :N], kd[:, :, :N], vd[:, :, :N], window=window, softcap=softcap, slopes=sld, lens=ln, k_cache=kc, v_cache=vc)
    for t in range(steps):
        at = [n + t for n in lens]
        qt, kt, vt = (torch.stack([x[s, :, at[s]] for s in range(S)]) for x in (qd, kd, vd))
        out = la.la_swa_biased_decode_step(qt, kt, vt, kc, vc, ln + t, softcap=softcap, slopes=sld)
        want = np.stack([o_ref[s, :, at[s]] for s in range(S)])
        ref.check(out, want, np.stack([bound[s, :, at[s]] for s in range(S)]))
        for s in range(S):
            assert torch.equal(kc[s, :, at[s] % window], kt[s]) and torch.equal(vc[s, :, at[s] % window], vt[s])


def test_swa_biased_step_without_extras_meets_the_plain_step():
    dev = cuda_device()
    S, H, d, w = 7, 4, 64, 64
    g = gen(1)
    q, k, v = (randn(g, S, H, d, dtype=BF).to(dev) for _ in range(3))
    kc, vc = (randn(g, S, H, w, d, dtype=BF).to(dev) for _ in range(2))
    pos = torch.tensor([0, 1, 63, 64, 65, 1000, 1 << 40], dtype=torch.int64, device=dev)
    k1, v1, k2, v2 = kc.clone(), vc.clone(), kc.clone(), vc.clone()
    a = la.la_swa_decode_step(q, k, v, k1, v1, pos, out_dtype=FP)
    b = la.la_swa_biased_decode_step(q, k, v, k2, v2, pos, out_dtype=FP)
    assert torch.equal(k1, k2) and torch.equal(v1, v2)
    # the biased step rounds each weight to bf16 for its product with v: off by at most 2^-8 of the weighted mean
    # of |v|; beside that both sum up to 64 fp32 terms in their own order
    largest = torch.cat([v2, v.unsqueeze(2)], 2).float().abs().max()
    assert (a - b).abs().max() < (2 ** -8 + 64 * 2 ** -23) * largest


# ------------------------------------------------------------------------------------------ errors, streams, graphs
def test_lengths_and_positions_out_of_range_are_reported_and_skipped():
    dev = cuda_device()
    x, w = torch.randn((3, 10, 16), device=dev), torch.randn((16, 4), device=dev)
    lens = torch.tensor([11, 4, -1], dtype=torch.int64, device=dev)
    y = torch.full_like(x, 7.0)
    _, st = la.la_conv_prefill(x, w, lens=lens, y=y)
    assert la.la_device_status() == la.LA_ERR_INVALID_ARGUMENT and la.la_device_status() == la.LA_OK
    assert torch.all(y[0] == 7.0) and torch.all(y[2] == 7.0) and torch.all(y[1, 4:] == 7.0) and not torch.any(y[1, :4] == 7.0)
    assert torch.all(st[0] == 0) and torch.all(st[2] == 0)
    A, bc = -torch.rand((16, 16), device=dev), torch.randn((3, 1, 10, 16), device=dev)
    y = torch.full_like(x, 7.0)
    _, h = la.la_ssm_prefill(x, x, A, bc, bc, lens=lens, y=y)
    assert la.la_device_status() == la.LA_ERR_INVALID_ARGUMENT
    assert torch.all(y[0] == 7.0) and torch.all(y[2] == 7.0) and torch.all(h[0] == 0) and torch.isfinite(h).all()
    q = torch.randn((3, 2, 10, 64), device=dev, dtype=BF)
    o = torch.full_like(q, 7.0)
    kc, vc = torch.zeros((3, 2, 8, 64), device=dev, dtype=BF), torch.zeros((3, 2, 8, 64), device=dev, dtype=BF)
    la.la_swa_prefill(q, q, q, window=8, lens=lens, o=o, k_cache=kc, v_cache=vc)
    assert la.la_device_status() == la.LA_ERR_INVALID_ARGUMENT
    assert torch.all(o[0] == 7.0) and torch.all(o[2] == 7.0) and torch.all(kc[0] == 0) and torch.any(kc[1] != 0)
    out = torch.full((2, 2, 64), 7.0, device=dev, dtype=BF)
    qs = torch.randn((2, 2, 64), device=dev, dtype=BF)
    rings = [torch.zeros((2, 2, 8, 64), device=dev, dtype=BF) for _ in range(2)]
    la.la_swa_biased_decode_step(qs, qs, qs, *rings, torch.tensor([-1, 0], device=dev), out=out)
    assert la.la_device_status() == la.LA_ERR_INVALID_ARGUMENT
    assert torch.all(out[0] == 7.0) and torch.all(rings[0][0] == 0) and not torch.any(out[1] == 7.0)


def hybrid(dev, B, N, seed):
    """Inputs of one convolution, one scan and one attention layer of a small hybrid model."""
    g = gen(seed)
    C, n, H, Hkv, d = 64, 16, 4, 2, 32
    t = {"x": randn(g, B, N, C, dtype=BF), "w": randn(g, C, 4, dtype=BF, scale=0.5), "bias": randn(g, C, dtype=BF), "delta": randn(g, B, N, C, dtype=BF),
         "z": randn(g, B, N, C, dtype=BF), "A": -(0.2 + torch.rand((C, n), generator=g)), "D": randn(g, C), "dt_bias": randn(g, C) - 3,
         "Bm": randn(g, B, 1, N, n, dtype=BF), "Cm": randn(g, B, 1, N, n, dtype=BF), "k": randn(g, B, Hkv, N, d, dtype=BF), "v": randn(g, B, Hkv, N, d, dtype=BF)}
    return {name: x.to(dev) for name, x in t.items()}


def prompt_pass(t, N, window, lens=None, workspace=None):
    B = t["x"].shape[0]
    y, conv = la.la_conv_prefill(t["x"][:, :N], t["w"], bias=t["bias"], lens=lens)
    y, h = la.la_ssm_prefill(y, t["delta"][:, :N], t["A"], t["Bm"][:, :, :N], t["Cm"][:, :, :N], D=t["D"], z=t["z"][:, :N],
                             delta_bias=t["dt_bias"], lens=lens, workspace=workspace)
    kc, vc = (torch.zeros((B, 2, window, 32), dtype=BF, device=y.device) for _ in range(2))
    q = torch.cat([y, y], -1).unflatten(-1, (4, 32)).transpose(1, 2)
    o = la.la_swa_prefill(q, t["k"][:, :, :N], t["v"][:, :, :N], window=window, softcap=20.0, slopes=t["D"][:4].abs().contiguous(), lens=lens,
                          k_cache=kc, v_cache=vc)
    return o, conv, h, kc, vc


def token_pass(t, i, conv, h, kc, vc, pos):
    y = la.la_conv_decode_step(t["x"][:, i], t["w"], conv, bias=t["bias"])
    y = la.la_ssm_decode_step(y, t["delta"][:, i], t["A"], t["Bm"][:, :, i], t["Cm"][:, :, i], h, D=t["D"], z=t["z"][:, i], delta_bias=t["dt_bias"])
    q = torch.cat([y, y], -1).unflatten(-1, (4, 32))
    return la.la_swa_biased_decode_step(q, t["k"][:, :, i].contiguous(), t["v"][:, :, i].contiguous(), kc, vc, pos, softcap=20.0,
                                        slopes=t["D"][:4].abs().contiguous())


def test_layers_together_prompt_then_tokens():
    """A prompt through convolution, scan and attention, then tokens one by one: the same as the longer prompt at once."""
    dev = cuda_device()
    B, N, steps, window = 2, 150, 5, 40
    t = hybrid(dev, B, N + steps, 4)
    whole, conv_w, h_w, kc_w, vc_w = prompt_pass(t, N + steps, window)
    o, conv, h, kc, vc = prompt_pass(t, N, window)
    assert torch.equal(o, whole[:, :, :N])  # causal: later tokens change nothing, bit for bit
    for i in range(N, N + steps):
        out = token_pass(t, i, conv, h, kc, vc, torch.full((B,), i, dtype=torch.int64, device=dev))
        # both sides round the scan's output and the result to bf16; the weights' rounding is one more
        assert (out.float() - whole[:, :, i].float()).abs().max() < 4 * 2 ** -8 * whole.float().abs().max()
    assert torch.equal(conv, conv_w) and torch.equal(kc, kc_w) and torch.equal(vc, vc_w)
    assert (h - h_w).abs().max() <= 1e-5 * h_w.abs().max()
    assert la.la_device_status() == la.LA_OK


def test_layers_captured_replayed_and_on_another_stream():
    dev = cuda_device()
    B, N, window = 1, 1200, 40
    t = hybrid(dev, B, N, 6)
    eager = prompt_pass(t, N, window)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = prompt_pass(t, N, window)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = prompt_pass(t, N, window)
    x0 = t["x"].clone()
    t["x"].zero_()
    graph.replay()
    t["x"].copy_(x0)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(eager, other, captured):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_steps_captured_and_replayed():
    dev = cuda_device()
    B, N, window = 2, 30, 16
    t = hybrid(dev, B, N + 1, 8)
    _, conv, h, kc, vc = prompt_pass(t, N, window)
    saved = [x.clone() for x in (conv, h, kc, vc)]
    pos = torch.full((B,), N, dtype=torch.int64, device=dev)
    want = token_pass(t, N, conv, h, kc, vc, pos)
    after = [x.clone() for x in (conv, h, kc, vc)]
    for x, s in zip((conv, h, kc, vc), saved):
        x.copy_(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token_pass(t, N, conv, h, kc, vc, pos)
    for x, s in zip((conv, h, kc, vc), saved):
        x.copy_(s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for x, s in zip((conv, h, kc, vc), after):
        assert torch.equal(x, s)


# ------------------------------------------------------------------------------------------ larger, repeated, shared
@pytest.mark.parametrize("B,H,Hkv,N,d,window,softcap,slopes", [
    (1, 4, 2, 3001, 128, 0, 0.0, False), (1, 4, 2, 2500, 64, 0, 0.0, False), (2, 4, 1, 2049, 128, 0, 30.0, False),
    (1, 4, 4, 3000, 64, 100, 0.0, False), (1, 2, 2, 2600, 96, 700, 0.0, True), (1, 4, 4, 2300, 64, 0, 4.0, True)])
def test_swa_long_prompts_sampled_and_repeated(B, H, Hkv, N, d, window, softcap, slopes):
    """Many blocks a query tile: sampled rows against the definition in fp64, and the same bits every time."""
    dev = cuda_device()
    q, k, v = swa_case(B, H, Hkv, N, N, d, BF, N)
    sl = slopes_of(H) if slopes else None
    qd, kd, vd, sld = on(dev, q, k, v, sl)
    o = la.la_swa_prefill(qd, kd, vd, window=window, softcap=softcap, slopes=sld)
    for _ in range(10):
        assert torch.equal(la.la_swa_prefill(qd, kd, vd, window=window, softcap=softcap, slopes=sld), o)
    assert la.la_device_status() == la.LA_OK
    sample = sorted(set(np.random.default_rng(N).choice(N, 24, replace=False).tolist()) | {0, 127, 128, 255, 256, N - 1})
    rows = ref.spans(N, N, B, window, None, None, 0, None)
    rows = [[r if i in sample else None for i, r in enumerate(rb)] for rb in rows]
    o_ref, bound = ref.swa(q, k, v, d ** -0.5, softcap, sl, rows, 0, BF)
    ref.check(o, o_ref, bound)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_swa_keys_shared_by_sequences_and_strided_views(dtype):
    """Keys and values expanded over the batch (stride 0) and heads taken out of one wide projection."""
    dev = cuda_device()
    B, H, Hkv, N, d = 3, 4, 2, 200, 64
    g = gen(2)
    wide = randn(g, B, N, (H + 2 * Hkv) * d, dtype=dtype, scale=1.5).to(dev)
    heads = wide.unflatten(-1, (H + 2 * Hkv, d)).transpose(1, 2)
    q, k, v = heads[:, :H], heads[:, H:H + Hkv], heads[:, H + Hkv:]
    o = la.la_swa_prefill(q, k, v, window=70)
    want = la.la_swa_prefill(q.contiguous(), k.contiguous(), v.contiguous(), window=70)
    assert torch.equal(o, want)
    ks, vs = k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1)
    o = la.la_swa_prefill(q, ks, vs, window=70)
    rows = ref.spans(N, N, B, 70, None, None, 0, None)
    o_ref, bound = ref.swa(q.cpu(), ks.cpu(), vs.cpu(), d ** -0.5, 0.0, None, rows, 0, dtype)
    ref.check(o, o_ref, bound)


def test_ssm_repeated_gives_the_same_bits():
    """Two channels per lane (many blocks), one channel, and time segments."""
    dev = cuda_device()
    for B, N, C in ((4, 700, 2048), (1, 500, 512), (1, 4000, 96)):
        t = ssm_inputs(B, N, C, 16, 1, BF, True, N)
        u, delta, z, A, Bm, Cm, D, bias = on(dev, *(t[k] for k in ("u", "delta", "z", "A", "Bm", "Cm", "D", "bias")))
        y, h = la.la_ssm_prefill(u, delta, A, Bm, Cm, D=D, z=z, delta_bias=bias)
        for _ in range(5):
            y2, h2 = la.la_ssm_prefill(u, delta, A, Bm, Cm, D=D, z=z, delta_bias=bias)
            assert torch.equal(y, y2) and torch.equal(h, h2)
        # a slice of the channels alone takes another schedule: the same recurrence
        c = slice(0, 64)
        ys, hs = la.la_ssm_prefill(u[..., c], delta[..., c], A[c].contiguous(), Bm, Cm, D=D[c].contiguous(), z=z[..., c],
                                   delta_bias=bias[c].contiguous())
        assert (hs - h[:, c]).abs().max() <= 2e-5 * h.abs().max()
        assert (ys.float() - y[..., c].float()).abs().max() <= 2 * 2 ** -8 * y.float().abs().max()


@pytest.mark.parametrize("n,G", [(16, 1), (8, 2), (4, 1), (24, 1), (64, 2)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_ssm_two_channels_per_lane_meets_the_definition(dtype, n, G):
    """Enough channels and sequences for two channels a lane; a few of them against fp64."""
    dev = cuda_device()
    lanes = 1 if n <= 4 else 2 if n <= 8 else 4 if n <= 16 else 8 if n <= 32 else 16
    B, N, C = 2, 67, 80 * (128 // lanes)
    t = ssm_inputs(B, N, C, n, G, dtype, True, n)
    lens = [N, 40]
    u, delta, z, A, Bm, Cm, D, bias, h0 = on(dev, *(t[k] for k in ("u", "delta", "z", "A", "Bm", "Cm", "D", "bias", "h")))
    y, h = la.la_ssm_prefill(u, delta, A, Bm, Cm, D=D, z=z, delta_bias=bias, h_in=h0, lens=torch.tensor(lens, device=dev))
    pick = torch.tensor(sorted({0, 1, C // G - 1, C // G % C, C // 2, C - 2, C - 1}))
    group = pick // (C // G)
    sub = {k: t[k][..., pick] for k in ("u", "delta", "z")}
    for i, c in enumerate(pick.tolist()):  # one channel at a time: its group's B and C
        b1, c1 = t["Bm"][:, group[i]:group[i] + 1], t["Cm"][:, group[i]:group[i] + 1]
        y_ref, bound, h_ref, h_bound = ref.ssm(sub["u"][..., i:i + 1], sub["delta"][..., i:i + 1], t["A"][c:c + 1], b1, c1, t["D"][c:c + 1],
                                               sub["z"][..., i:i + 1], t["bias"][c:c + 1], True, t["h"][:, c:c + 1], lens, dtype)
        ref.check(h[:, c:c + 1], h_ref, h_bound)
        ref.check(y[..., c:c + 1], y_ref, bound)


def test_two_streams_at_once():
    """The same calls on two streams without an order between them: each has its own workspace and flags."""
    dev = cuda_device()
    t = [hybrid(dev, 1, 1500, s) for s in (11, 12)]
    want = [prompt_pass(x, 1500, 64) for x in t]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in t]
    for _ in range(4):
        got = []
        for s, x in zip(streams, t):
            with torch.cuda.stream(s):
                got.append(prompt_pass(x, 1500, 64))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, b in zip(g, w):
                assert torch.equal(a, b)
    assert la.la_device_status() == la.LA_OK


@pytest.mark.parametrize("C", [24, 5120])
def test_ssm_step_of_zero_length_keeps_the_state(C):
    """dt = 0 is the identity to the bit, for any decay rate: neither the exponential nor its argument may move it."""
    dev = cuda_device()
    B, N, n = 1, 70, 16
    t = ssm_inputs(B, N, C, n, 1, FP, False, 3)
    A = t["A"].clone()
    A[:, 0], A[:, 1], A[:, 2] = 0.0, torch.finfo(torch.float32).min, -1e-30
    u, z, Bm, Cm, h0 = on(dev, t["u"], t["z"], t["Bm"], t["Cm"], t["h"])
    _, h = la.la_ssm_prefill(u, torch.zeros_like(u), A.to(dev), Bm, Cm, h_in=h0, delta_softplus=False)
    assert torch.equal(h, h0)


def test_swa_bad_values_are_seen_by_their_own_queries_only():
    """Nine query tiles per block of the grid, seven of which see nothing: the notes that the first and the last
    one's masked values are not finite must not take each other's place."""
    dev = cuda_device()
    H, N, d = 152, 9 * 256, 16
    q, k, v = swa_case(1, H, 2, N, N, d, BF, 77)
    lo, hi = torch.zeros(1, N, dtype=torch.int32), torch.zeros(1, N, dtype=torch.int32)
    lo[0, :256], hi[0, :256] = 10, 256
    lo[0, -256:], hi[0, -256:] = N - 246, N
    clean = la.la_swa_prefill(*on(dev, q, k, v), key_lo=lo.to(dev), key_hi=hi.to(dev))
    v[:, :, 5], v[:, :, N - 251] = float("nan"), float("inf")
    for _ in range(5):
        o = la.la_swa_prefill(*on(dev, q, k, v), key_lo=lo.to(dev), key_hi=hi.to(dev))
        assert torch.isfinite(o.float()).all()
        assert (o.float() - clean.float()).abs().max() <= 2 ** -7 * clean.float().abs().max()
    assert not o[:, :, 256:-256].any()
    assert la.la_device_status() == la.LA_OK


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("scale,softcap,slope", [(-0.3, 0.0, 0.0), (0.0, 0.0, 0.0), (-0.3, 3.0, 0.0), (0.2, 1e6, 0.0), (0.2, 1e-3, 0.0),
                                                 (0.2, 2e3, 0.01), (0.2, 0.0, -0.02), (2.0, 1.5, -0.5)])
def test_swa_unusual_scales_caps_and_slopes(dtype, scale, softcap, slope):
    """Negative and zero scales, caps far above and below the scores, biases that grow with the distance."""
    dev = cuda_device()
    B, H, Hkv, N, d = 1, 2, 1, 300, 64
    q, k, v = swa_case(B, H, Hkv, N, N, d, dtype, 55)
    sl = torch.full((H,), slope) if slope else None
    for window in (0, 90):  # wide and narrow blocks
        o = la.la_swa_prefill(*on(dev, q, k, v), scale=scale, softcap=softcap, slopes=None if sl is None else sl.to(dev), window=window)
        rows = ref.spans(N, N, B, window, None, None, 0, None)
        o_ref, bound = ref.swa(q, k, v, scale, softcap, sl, rows, 0, dtype)
        ref.check(o, o_ref, bound)
    # the step at the last position, over a ring of the last 90 tokens
    w = 90
    kc, vc = (torch.zeros(B, Hkv, w, d, dtype=dtype) for _ in range(2))
    for p in range(N - w, N - 1):
        kc[:, :, p % w], vc[:, :, p % w] = k[:, :, p], v[:, :, p]
    last = [x[:, :, -1].contiguous() for x in (q, k, v)]
    out = la.la_swa_biased_decode_step(*on(dev, *last, kc, vc), torch.tensor([N - 1], device=dev), softcap=softcap,
                                       slopes=None if sl is None else sl.to(dev), scale=scale)
    ref.check(out, o_ref[:, :, -1], bound[:, :, -1])


def test_time_major_activations():
    """[N, B, C] activations as [B, N, C] views, outputs too: sequences lie within a token's row."""
    dev = cuda_device()
    B, N, C, n = 3, 150, 64, 8
    t = ssm_inputs(B, N, C, n, 1, BF, True, 5)
    u, delta, z, A, Bm, Cm = on(dev, *(t[k] for k in ("u", "delta", "z", "A", "Bm", "Cm")))
    w = randn(gen(1), C, 4, dtype=BF).to(dev)
    major = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    empty = lambda: torch.empty(N, B, C, dtype=BF, device=dev).transpose(0, 1)  # noqa: E731
    y, s = la.la_conv_prefill(u, w)
    y2, s2 = la.la_conv_prefill(major(u), w, y=empty())
    assert torch.equal(y, y2) and torch.equal(s, s2)
    y, h = la.la_ssm_prefill(u, delta, A, Bm, Cm, z=z)
    y2, h2 = la.la_ssm_prefill(major(u), major(delta), A, Bm, Cm, z=major(z), y=empty())
    assert torch.equal(y, y2) and torch.equal(h, h2)


def test_stream_argument_orders_the_whole_call():
    """Outputs with zeros for padding, copies of states, workspaces: all of a call's work is on the stream it is given."""
    dev = cuda_device()
    B, N, C, n = 1, 4000, 64, 16
    t = ssm_inputs(B, N, C, n, 1, FP, False, 6)
    u, delta, A, Bm, Cm, h0 = on(dev, *(t[k] for k in ("u", "delta", "A", "Bm", "Cm", "h")))
    lens = torch.tensor([N - 100], device=dev)
    w = randn(gen(1), C, 4, dtype=FP).to(dev)
    s0 = randn(gen(2), B, 3, C, dtype=FP).to(dev)
    q, k, v = on(dev, *swa_case(1, 2, 1, N, N, 64, BF, 9))
    calls = (lambda s: la.la_conv_prefill(u, w, state_in=s0, lens=lens, stream=s),
             lambda s: la.la_ssm_prefill(u, delta, A, Bm, Cm, h_in=h0, lens=lens, stream=s),
             lambda s: (la.la_swa_prefill(q=q, k=k, v=v, lens=lens, window=300, stream=s),))
    want = [c(None) for c in calls]
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream())
    big = torch.randn(8192, 8192, device=dev)
    for handle in (side, side.cuda_stream):
        busy = big
        for _ in range(6):
            busy = busy @ big  # the current stream is behind: what a call put on it would come too late
        got = [c(handle) for c in calls]
        side.synchronize()
        for g, x in zip(got, want):
            for a, b in zip(g, x):
                assert torch.equal(a.cpu(), b.cpu())
    torch.cuda.synchronize()
    with pytest.raises(TypeError):
        la.la_conv_prefill(u, w, None, None, None, True, None, None, None, side)  # by name only


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("Nq,Nk,d,window,softcap,slopes,lens", [
    (1, 1, 64, 0, 0.0, False, None), (1, 2000, 128, 0, 0.0, False, None), (7, 1501, 40, 0, 0.0, True, None), (133, 1333, 64, 0, 5.0, False, None),
    (300, 2300, 96, 900, 0.0, True, None), (65, 700, 128, 0, 0.0, False, [640, 700]), (40, 4000, 8, 2000, 3.0, True, [3990, 1000])])
def test_swa_few_queries_share_their_keys(dtype, Nq, Nk, d, window, softcap, slopes, lens):
    """Few query tiles over long caches: clusters of blocks share a tile's keys."""
    dev = cuda_device()
    B, H, Hkv = (len(lens) if lens else 1), 2, 1
    q, k, v = swa_case(B, H, Hkv, Nq, Nk, d, dtype, Nq + Nk)
    sl = slopes_of(H) if slopes else None
    dlens = None if lens is None else torch.tensor(lens, device=dev)
    rows = ref.spans(Nq, Nk, B, window, None, None, Nk - Nq, lens)
    o_ref, bound = ref.swa(q, k, v, d ** -0.5, softcap, sl, rows, Nk - Nq, dtype)
    qd, kd, vd, sld = on(dev, q, k, v, sl)
    o = la.la_swa_prefill(qd, kd, vd, window=window, softcap=softcap, slopes=sld, lens=dlens)
    ref.check(o, o_ref, bound)
    for _ in range(3):
        assert torch.equal(la.la_swa_prefill(qd, kd, vd, window=window, softcap=softcap, slopes=sld, lens=dlens), o)
    # values that no query sees, and rows that see nothing but one share's keys
    lo = torch.full((B, Nq), max(0, Nk // 2 - 3), dtype=torch.int32)
    hi = torch.minimum(lo + 1 + torch.arange(Nq, dtype=torch.int32) % 5, torch.tensor(Nk, dtype=torch.int32))
    hi[:, ::3] = lo[:, ::3]
    seen = torch.zeros(Nk, dtype=torch.bool)
    seen[int(lo[0, 0]):int(lo[0, 0]) + 5] = True
    k[:, :, ~seen], v[:, :, ~seen] = float("nan"), float("inf")
    rows = ref.spans(Nq, Nk, B, 0, lo.numpy(), hi.numpy(), Nk - Nq, lens)
    o_ref, bound = ref.swa(q, k, v, d ** -0.5, softcap, sl, rows, Nk - Nq, dtype)
    o = la.la_swa_prefill(*on(dev, q, k, v), softcap=softcap, slopes=sld, lens=dlens, key_lo=lo.to(dev), key_hi=hi.to(dev))
    ref.check(o, o_ref, bound)
    assert la.la_device_status() == la.LA_OK


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("C", [13, 64])
def test_new_outputs_have_zeros_for_padding_and_the_incoming_state_of_skipped_sequences(dtype, C):
    dev = cuda_device()
    B, N, n = 4, 150, 5
    lens = torch.tensor([0, 70, N + 1, N], device=dev)
    t = ssm_inputs(B, N, C, n, 1, dtype, True, C)
    u, delta, z = (pad_rows(t[k], dev) for k in ("u", "delta", "z"))
    A, Bm, Cm, h0 = on(dev, *(t[k] for k in ("A", "Bm", "Cm", "h")))
    w, s0 = randn(gen(1), C, 4, dtype=dtype).to(dev), randn(gen(2), B, 3, C, dtype=dtype).to(dev)
    q, k, v = on(dev, *swa_case(B, 2, 1, N - 20, N, 16, dtype, 3))

    def poison():  # what the next outputs are made of
        for shape in ((B, N, 16), (B, N, 64), (B, 3, C), (B, C, n), (B, 2, N - 20, 16)):
            for dt in (dtype, FP):
                torch.full(shape, float("nan"), dtype=dt, device=dev)
    for state in (False, True):
        poison()
        y, s = la.la_conv_prefill(u, w, state_in=s0 if state else None, lens=lens)
        assert not y[0].any() and not y[1, 70:].any() and not y[2].any() and torch.isfinite(y.float()).all() and y[1, :70].any()
        assert torch.equal(s[2], s0[2] if state else torch.zeros_like(s0[2])) and torch.equal(s[0], s[2] if not state else s0[0])
        poison()
        y, h = la.la_ssm_prefill(u, delta, A, Bm, Cm, z=z, h_in=h0 if state else None, lens=lens)
        assert not y[0].any() and not y[1, 70:].any() and not y[2].any() and torch.isfinite(y.float()).all() and y[3, N - 1].any()
        assert torch.equal(h[2], h0[2] if state else torch.zeros_like(h0[2])) and torch.isfinite(h).all()
    poison()
    o = la.la_swa_prefill(q, k, v, lens=lens)  # queries stand at 20..149
    assert not o[0].any() and not o[1, :, 50:].any() and not o[2].any() and torch.isfinite(o.float()).all() and o[1, :, :50].any()
    assert la.la_device_status() == la.LA_ERR_INVALID_ARGUMENT


def test_offsets_beyond_32_bits():
    """Sequences, heads and states more than 2^31 elements apart give what they give side by side."""
    dev = cuda_device()
    far = (1 << 31) + (1 << 12)
    N, C, n, H, d = 70, 64, 16, 2, 64
    t = ssm_inputs(2, N, C, n, 1, BF, True, 8)
    u, delta, z, A, Bm, Cm = on(dev, *(t[k] for k in ("u", "delta", "z", "A", "Bm", "Cm")))
    w = randn(gen(1), C, 4, dtype=BF).to(dev)
    q, k, v = on(dev, *swa_case(2, H, H, N, N, d, BF, 4))
    room = torch.empty(far + (1 << 22), dtype=BF, device=dev)
    at = 0

    def apart(x, make=True):  # the same values, the sequences `far` elements apart
        nonlocal at
        y = room.as_strided(x.shape, (far, *x[0].contiguous().stride()), at)
        at += -(-x[0].numel() // 64) * 64
        if make:
            y.copy_(x)
        return y
    assert all(torch.equal(a, b) for a, b in zip(la.la_conv_prefill(apart(u), w, y=apart(u, False)), la.la_conv_prefill(u, w)))
    got = la.la_ssm_prefill(apart(u), apart(delta), A, apart(Bm), apart(Cm), z=apart(z), y=apart(u, False))
    assert all(torch.equal(a, b) for a, b in zip(got, la.la_ssm_prefill(u, delta, A, Bm, Cm, z=z)))
    for x in (BF, FP):
        if x is FP:
            q, k, v = (i.float() for i in (q, k, v))
            room, at = torch.empty(far + (1 << 22), dtype=FP, device=dev), 0
        assert torch.equal(la.la_swa_prefill(apart(q), apart(k), apart(v), window=40, o=apart(q, False)), la.la_swa_prefill(q, k, v, window=40))
        # heads and tokens apart: one sequence, the far axis inside it
        side = apart(k.transpose(0, 1)).transpose(0, 1)
        assert torch.equal(la.la_swa_prefill(q, side, v, window=40), la.la_swa_prefill(q, k, v, window=40))
    del room
    # rings and states of so many sequences that the last one lies beyond 2^31 elements
    S, ring = (1 << 31) // (256 * 128) + 3, (256, 128)
    kc, vc = (torch.zeros((S, 1, *ring), dtype=BF, device=dev) for _ in range(2))
    qs, ks, vs = (randn(gen(i), S, 1, 128, dtype=BF).to(dev) for i in (5, 6, 7))
    kc[-1], vc[-1] = randn(gen(8), 1, *ring, dtype=BF).to(dev), randn(gen(9), 1, *ring, dtype=BF).to(dev)
    last = [i[-1:].clone() for i in (qs, ks, vs, kc, vc)]
    pos = torch.full((S,), 300, device=dev)
    out = la.la_swa_biased_decode_step(qs, ks, vs, kc, vc, pos)
    assert torch.equal(out[-1:], la.la_swa_biased_decode_step(*last, pos[:1]))
    assert torch.equal(kc[-1:], last[3]) and torch.equal(vc[-1, 0, 300 % 256], vs[-1, 0])
    del kc, vc
    S, C, n = 8200, 4096, 64
    h = torch.zeros((S, C, n), device=dev)
    h[-1] = randn(gen(3), C, n).to(dev)
    us, ds = (randn(gen(i), S, C, dtype=BF).to(dev) for i in (1, 2))
    bc = randn(gen(4), S, 1, n, dtype=BF).to(dev)
    A = -torch.rand((C, n), device=dev)
    h_last = h[-1:].clone()
    y = la.la_ssm_decode_step(us, ds, A, bc, bc, h)
    y_last = la.la_ssm_decode_step(us[-1:], ds[-1:], A, bc[-1:], bc[-1:], h_last)
    assert torch.equal(y[-1:], y_last) and torch.equal(h[-1:], h_last)
    assert la.la_device_status() == la.LA_OK
