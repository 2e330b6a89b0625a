"""The layers' calls at the ends of what their documentation allows: ranges of scores, far keys, shared keys, growing
states, counts and streams, against fp64 definitions."""
import numpy as np
import pytest
import torch

import linear_attention_recurrence_chunked_gb300 as la
from tests import layers_oracle as ref
from tests.helpers import cuda_device
from tests.test_gpu_layers import gen, on, pad_rows, randn, slopes_of, ssm_inputs, swa_case

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("H,Hkv,d,window,softcap,slopes", [
    (4, 4, 64, 64, 0.0, False), (16, 4, 128, 256, 30.0, True), (16, 1, 72, 100, 0.0, True), (3, 3, 8, 33, 5.0, False)])
def test_swa_step_weights_hold_more_than_bf16(H, Hkv, d, window, softcap, slopes):
    """bf16 rings, fp32 outputs: the weights meet their values in two bf16 parts, off by 2^-17 of a weight."""
    dev = cuda_device()
    S = 5
    g = gen(H + d)
    q, k, v = randn(g, S, H, d, dtype=BF, scale=1.5), randn(g, S, Hkv, d, dtype=BF, scale=1.5), randn(g, S, Hkv, d, dtype=BF)
    kc, vc = randn(g, S, Hkv, window, d, dtype=BF, scale=1.5), randn(g, S, Hkv, window, d, dtype=BF)
    sl = slopes_of(H) if slopes else None
    pos = torch.tensor([0, 7, window - 1, window, 1000 * window + 5])
    out = la.la_swa_biased_decode_step(*on(dev, q, k, v, kc, vc, pos), softcap=softcap, slopes=None if sl is None else sl.to(dev), out_dtype=FP)
    for s in range(S):
        p = int(pos[s])
        n = min(p + 1, window)
        order = [(p - i) % window for i in range(n - 1, 0, -1)]  # oldest first, the new token behind them
        keys = torch.cat([kc[s][:, order], k[s][:, None]], 1)[None].float()
        values = torch.cat([vc[s][:, order], v[s][:, None]], 1)[None].float()
        # fp32 copies: the definition's bound then has no term for weights in bf16
        want, bound = ref.swa(q[s][None, :, None].float(), keys, values, d ** -0.5, softcap, sl, [[(0, n)]], n - 1, FP)
        ref.check(out[s][None, :, None], want, bound + 2 ** -17 * values.abs().max().item())


def test_swa_biased_step_and_plain_step_agree_beyond_bf16():
    dev = cuda_device()
    S, H, d, w = 7, 4, 64, 64
    g = gen(1)
    q, k, v = (randn(g, S, H, d, dtype=BF).to(dev) for _ in range(3))
    kc, vc = (randn(g, S, H, w, d, dtype=BF).to(dev) for _ in range(2))
    pos = torch.tensor([0, 1, 63, 64, 65, 1000, 1 << 40], dtype=torch.int64, device=dev)
    a = la.la_swa_decode_step(q, k, v, kc.clone(), vc.clone(), pos, out_dtype=FP)
    b = la.la_swa_biased_decode_step(q, k, v, kc.clone(), vc.clone(), pos, out_dtype=FP)
    # two-part weights: 2^-17 of the weighted mean of |v|; beside that both sum up to 64 fp32 terms in their own order
    largest = max(vc.float().abs().max(), v.float().abs().max())
    assert (a - b).abs().max() < (2 ** -17 + 64 * 2 ** -23) * largest


@pytest.mark.parametrize("d,first,later", [(64, 41, 46.5), (128, 41, 46.5), (64, 27.5, 35), (128, 27.5, 35), (64, 20, 36)])
def test_swa_capped_scores_far_below_zero(d, first, later):
    """Scores that are all far below zero, under a cap far above them: a block's bound on its maximum lies as far above
    zero, and what later blocks hold must still count beside it."""
    dev = cuda_device()
    H, N = 4, 8192
    q = torch.ones((1, H, N, d), dtype=BF)
    per = torch.full((N,), -later / d)
    per[:128] = -first / d  # exact in bf16
    k = per.to(BF)[None, None, :, None].expand(1, 1, N, d).contiguous()
    v = randn(gen(d), 1, 1, N, d, dtype=BF) + 1
    v[:, :, :128] -= 2
    o = la.la_swa_prefill(*on(dev, q, k, v), scale=1.0, softcap=1000.0)
    rows = [[(0, i + 1) if i in (5, 127, 128, 500, 4000, N - 1) else None for i in range(N)]]
    o_ref, bound = ref.swa(q, k, v, 1.0, 1000.0, None, rows, 0, BF)
    ref.check(o, o_ref, bound)


@pytest.mark.parametrize("B,H,Hkv,Nq,N,d,window,softcap", [
    (3, 4, 2, 200, 200, 64, 70, 0.0), (2, 8, 4, 300, 300, 128, 0, 20.0), (4, 40, 4, 260, 260, 72, 0, 0.0), (2, 4, 2, 10, 1500, 64, 0, 0.0)])
def test_swa_repeated_axes_give_what_copies_give(B, H, Hkv, Nq, N, d, window, softcap):
    """Keys, values and queries expanded over sequences or heads (stride 0): the same kernel, to the bit."""
    dev = cuda_device()
    q, k, v = (t.to(dev) for t in swa_case(B, H, Hkv, Nq, N, d, BF, N + d))
    kw = dict(window=window, softcap=softcap)
    for ks, vs in ((k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1)), (k[:, :1].expand(-1, Hkv, -1, -1), v),
                   (k[:1, :1].expand(B, Hkv, -1, -1), v[:, :1].expand(-1, Hkv, -1, -1))):
        assert torch.equal(la.la_swa_prefill(q, ks, vs, **kw), la.la_swa_prefill(q, ks.contiguous(), vs.contiguous(), **kw))
    qs = q[:1, :1].expand(B, H, -1, -1)
    assert torch.equal(la.la_swa_prefill(qs, k, v, **kw), la.la_swa_prefill(qs.contiguous(), k, v, **kw))
    assert la.la_device_status() == la.LA_OK


def test_swa_rows_computed_again_over_long_prompts_time_nothing_out():
    """A value that is not finite in a partly seen block has its item's rows computed again key by key, here for seconds,
    while the products of the block's next item wait: work that goes on is not a wait that has expired."""
    dev = cuda_device()
    B, H, Nq, Nk, d = 20, 8, 256, 1_200_000, 8  # 160 items on 152 SMs: those of sequence 19 come behind sequence 18's
    g = gen(6)
    q = randn(g, B, H, Nq, d, dtype=BF).to(dev)
    k, v = (torch.randn((B, 1, Nk, d), device=dev, generator=torch.Generator(dev).manual_seed(s)).to(BF) for s in (1, 2))
    lens = torch.full((B,), Nk - Nq, device=dev)  # every query is padding
    lens[18:] = Nk
    clean = la.la_swa_prefill(q, k, v, lens=lens)
    v[18, 0, -1, 3] = float("nan")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    o = la.la_swa_prefill(q, k, v, lens=lens)
    end.record()
    assert la.la_device_status() == la.LA_OK
    print(f"computed again in {start.elapsed_time(end):.0f} ms")
    assert torch.equal(o[19], clean[19]) and not o[:18].any()
    assert (o[18, :, :-1].float() - clean[18, :, :-1].float()).abs().max() <= 2 ** -7 * clean[18].float().abs().max() + 1e-4
    assert torch.isnan(o[18, :, -1, 3]).all() and torch.isfinite(o[18, :, -1, 4]).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("H,Nq", [(2, 3), (160, 200)])
def test_swa_biased_rows_far_from_all_their_keys(dtype, H, Nq):
    """Rows whose keys all lie far behind or far ahead of them: the bias is the same for all of a row's keys but for
    their distance from the nearest one, and what they share must not cost the scores their accuracy."""
    dev = cuda_device()
    Nk, d, seen = 70000, 64, 300
    q, k, v = swa_case(1, H, 1, Nq, Nk, d, dtype, H)
    sl = torch.full((H,), 0.7)
    for q_pos0, lo, hi, nearest in ((Nk - Nq, 40, 40 + seen, seen - 1), (0, Nk - seen, Nk, 0)):
        key_lo, key_hi = (torch.full((1, Nq), x, dtype=torch.int32, device=dev) for x in (lo, hi))
        o = la.la_swa_prefill(*on(dev, q, k, v), slopes=sl.to(dev), key_lo=key_lo, key_hi=key_hi, q_pos0=q_pos0)
        for h, i in ((0, 0), (H - 1, 1), (H // 2, Nq - 1)):
            want, bound = ref.swa(q[:, h:h + 1, i:i + 1], k[:, :, lo:hi], v[:, :, lo:hi], d ** -0.5, 0.0, sl[:1], [[(0, seen)]], nearest, dtype)
            ref.check(o[:, h:h + 1, i:i + 1], want, bound)
    assert la.la_device_status() == la.LA_OK


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_swa_biased_rows_far_from_their_keys_computed_again(bad):
    """The same where a masked value of a partly seen block is not finite."""
    dev = cuda_device()
    Nk, d, Nq = 70000, 64, 5
    q, k, v = swa_case(1, 2, 1, Nq, Nk, d, BF, 3)
    v[:, :, 39] = bad
    sl = torch.full((2,), 0.7)
    key_lo, key_hi = (torch.full((1, Nq), x, dtype=torch.int32, device=dev) for x in (40, 340))
    o = la.la_swa_prefill(*on(dev, q, k, v), slopes=sl.to(dev), key_lo=key_lo, key_hi=key_hi)
    for i in (0, 4):
        want, bound = ref.swa(q[:, :, i:i + 1], k[:, :, 40:340], v[:, :, 40:340], d ** -0.5, 0.0, sl, [[(0, 300)]], 299, BF)
        ref.check(o[:, :, i:i + 1], want, bound)


@pytest.mark.parametrize("h0,lens", [(0.0, None), (1e-30, [170])])
def test_ssm_segments_of_growing_states(h0, lens):
    """Time segments over which exp(A sum dt) leaves fp32's range: a state of zero stays zero, a small one grows."""
    dev = cuda_device()
    B, N, C, n = 1, 2000, 48, 16
    g = gen(4)
    A = 0.8 + 0.2 * torch.rand((C, n), generator=g)
    delta = 0.6 + 0.1 * torch.rand((B, N, C), generator=g)
    u, Bm, Cm = randn(g, B, N, C), randn(g, B, 1, N, n), randn(g, B, 1, N, n)
    u[:, :N - 40] = 0  # what enters grows by 2^40 at most
    h_in = torch.full((B, C, n), h0)
    ln = None if lens is None else torch.tensor(lens, device=dev)
    assert la.la_ssm_prefill_workspace_size(*on(dev, u, delta, A, Bm, Cm)) > 0
    y, h = la.la_ssm_prefill(*on(dev, u, delta, A, Bm, Cm), h_in=h_in.to(dev), delta_softplus=False, lens=ln)
    y_ref, bound, h_ref, h_bound = ref.ssm(u, delta, A, Bm, Cm, None, None, None, False, h_in, lens, FP, segment=160)
    ref.check(h, h_ref, h_bound)
    ref.check(y, y_ref, bound)


@pytest.mark.parametrize("handle,runs_on", [(0, 0), (1, 0), (2, 2)])
def test_stream_handles_of_the_default_streams(monkeypatch, handle, runs_on):
    """0 and cudaStreamLegacy (1) are the legacy default stream, cudaStreamPerThread (2) is the thread's own."""
    dev = cuda_device()
    x, w = torch.randn((1, 9, 16), device=dev), torch.randn((16, 4), device=dev)
    want = la.la_conv_prefill(x, w)
    torch.cuda.synchronize()
    used = []
    call = la._call
    monkeypatch.setattr(la, "_call", lambda name, index, *a: (used.append(torch.cuda.current_stream(dev).cuda_stream), call(name, index, *a)))
    with torch.cuda.stream(torch.cuda.Stream(dev)):
        got = la.la_conv_prefill(x, w, stream=handle)
        torch.cuda.synchronize()
    assert used == [runs_on]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_swa_step_at_the_last_position(dtype):
    dev = cuda_device()
    g = gen(3)
    q, k, v = (randn(g, 2, 4, 64, dtype=dtype).to(dev) for _ in range(3))
    kc, vc = (randn(g, 2, 4, 40, 64, dtype=dtype).to(dev) for _ in range(2))
    far = torch.tensor([(1 << 63) - 1, (1 << 63) - 2], device=dev)
    near = 40 + far % 40  # the same slots of a full ring
    a = la.la_swa_biased_decode_step(q, k, v, kc.clone(), vc.clone(), far)
    b = la.la_swa_biased_decode_step(q, k, v, kc.clone(), vc.clone(), near)
    assert torch.isfinite(a.float()).all() and torch.equal(a, b)


def test_ssm_slow_decays_add_up_to_no_bias():
    """One pass over 20000 tokens with memories of about 800 to 6000: a state takes one rounded factor per token, and the
    mean of their errors must stay near zero where factors are close to 1 too."""
    dev = cuda_device()
    B, N, C, n = 1, 20000, 3328, 16
    g = torch.Generator(dev).manual_seed(5)
    draw = lambda *shape: torch.randn(shape, device=dev, generator=g)  # noqa: E731
    u, delta, Bm, Cm = (draw(*s).to(BF) for s in ((B, N, C), (B, N, C), (B, 1, N, n), (B, 1, N, n)))
    A = -torch.linspace(0.2, 1.5, n, device=dev).expand(C, n).contiguous()
    bias = torch.full((C,), -7.6, device=dev)  # steps near 5e-4
    assert la.la_ssm_prefill_workspace_size(u, delta, A, Bm, Cm) == 0
    _, h = la.la_ssm_prefill(u, delta, A, Bm, Cm, delta_bias=bias, out_dtype=FP)
    pick = torch.tensor([0, 1, 1700, C - 1], device=dev)
    h_ref = ref.ssm(u[..., pick], delta[..., pick], A[pick], Bm, Cm, None, None, bias[pick], True, None, None, FP)[2]
    err = np.linalg.norm(h[:, pick].double().cpu().numpy() - h_ref) / np.linalg.norm(h_ref)
    # a mean of 2.5e-9 a token over 6000 tokens of memory, 0.7 of which weigh: 1.1e-5; a factor's and a state's rounding of
    # 2^-24 enter at random: 2.5e-6
    assert err < 2e-5


@pytest.mark.parametrize("B,N,C,n,G,dtype,out,z,softplus", [
    (2, 37, 40, 16, 2, BF, BF, True, True), (2, 70, 33, 4, 1, FP, FP, False, True), (3, 129, 24, 24, 3, FP, FP, True, True),
    (1, 100, 10, 64, 2, BF, FP, False, True), (2, 31, 7, 1, 1, FP, FP, True, True), (1, 40, 21, 7, 3, BF, FP, True, False),
    (1, 300, 16, 16, 1, FP, FP, True, True)])
def test_ssm_prefill_in_one_segment_within_single_roundings(B, N, C, n, G, dtype, out, z, softplus):
    """No time segments: a token's decay has the errors of its own product and exponential alone."""
    dev = cuda_device()
    t = ssm_inputs(B, N, C, n, G, dtype, z, 2 * N + C)
    if not softplus:
        t["delta"], t["bias"] = t["delta"].abs() * 0.2, t["bias"].abs() * 0.1
    names = ("u", "delta", "A", "Bm", "Cm", "D", "z", "bias", "h")
    args = [t[k] for k in names]
    y_ref, bound, h_ref, h_bound = ref.ssm(*args[:8], softplus, t["h"], None, out)
    u, delta, A, Bm, Cm, D, zd, bias, h0 = on(dev, *args)
    u, delta, zd = (None if x is None else pad_rows(x, dev) for x in (u, delta, zd))
    assert la.la_ssm_prefill_workspace_size(u, delta, A, Bm, Cm) == 0
    y, h = la.la_ssm_prefill(u, delta, A, Bm, Cm, D=D, z=zd, delta_bias=bias, delta_softplus=softplus, h_in=h0, out_dtype=out)
    ref.check(h, h_ref, h_bound)
    ref.check(y, y_ref, bound)


@pytest.mark.parametrize("B,N,C,n,dtype,length", [(1, 2000, 48, 16, BF, 160), (2, 1500, 24, 8, FP, 160), (1, 4000, 96, 16, FP, 160)])
def test_ssm_prefill_in_segments_joins_them_within_a_segments_roundings(B, N, C, n, dtype, length):
    """Time segments: a state that enters one decays by exp(A sum dt), whose sum has a rounding per token of the segment.
    That error enters once per segment, on top of the single pass's."""
    dev = cuda_device()
    t = ssm_inputs(B, N, C, n, 1, dtype, False, N)
    args = [t[k] for k in ("u", "delta", "A", "Bm", "Cm", "D", "z", "bias")]
    y_ref, bound, h_ref, h_bound = ref.ssm(*args, True, t["h"], None, FP)
    # what a segment's end holds of the states that entered it, times the error of the decay that carried it there
    dt = np.logaddexp(ref.f64(t["delta"]) + ref.f64(t["bias"]), 0)
    A, e, states = ref.f64(t["A"]), 0.0, ref.f64(t["h"])
    for s in range(0, N, length):
        total = dt[:, s:s + length].sum(1)[..., None] * A  # [B, C, n]
        a = np.exp(total)
        e = a * e + a * np.abs(states) * (np.abs(total) * (length + 4) * ref.U + 2.0 ** -21)
        cut = [x[:, s:s + length] for x in (t["u"], t["delta"])]
        bc = [x[:, :, s:s + length] for x in (t["Bm"], t["Cm"])]
        states = ref.ssm(*cut, t["A"], *bc, t["D"], None, t["bias"], True, torch.from_numpy(states), None, FP)[2]
    u, delta, Ad, Bm, Cm, D, _, bias, h0 = on(dev, *args, t["h"])
    assert la.la_ssm_prefill_workspace_size(u, delta, Ad, Bm, Cm) > 0
    y, h = la.la_ssm_prefill(u, delta, Ad, Bm, Cm, D=D, delta_bias=bias, h_in=h0, out_dtype=FP)
    ref.check(h, h_ref, h_bound + e)
    # the first segment enters without a join
    assert N > 2 * length
    first = np.full_like(y_ref, np.nan)
    first[:, :length] = y_ref[:, :length]
    ref.check(y, first, bound)


@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,d,window,q_pos0", [
    (2, 4, 1, 253, 561, 72, 0, 272), (3, 10, 2, 237, 283, 24, 345, 25), (2, 15, 3, 246, 257, 24, 59, 2), (3, 3, 3, 1242, 1976, 72, 620, 109)])
def test_swa_values_that_are_not_finite_give_the_same_bits_every_time(B, H, Hkv, Nq, Nk, d, window, q_pos0):
    """Values behind the last query are not finite: they have the rows of the last queries' tile computed again, and no
    other tile's, however far along those are when the values are found."""
    dev = cuda_device()
    q, k, v = swa_case(B, H, Hkv, Nq, Nk, d, BF, Nq)
    k[:, :, q_pos0 + Nq:], v[:, :, q_pos0 + Nq:] = float("nan"), float("inf")
    q, k, v = on(dev, q, k, v)
    first = la.la_swa_prefill(q, k, v, window=window, q_pos0=q_pos0)
    assert torch.isfinite(first.float()).all()
    for _ in range(200):
        assert torch.equal(la.la_swa_prefill(q, k, v, window=window, q_pos0=q_pos0), first)
    # values that are finite change the last tile's rows by their weights' roundings alone, and no other row
    clean = la.la_swa_prefill(q, k, torch.nan_to_num(v, 0, 0, 0), window=window, q_pos0=q_pos0)
    kept = (Nq - 1) // 128 * 128
    assert torch.equal(clean[:, :, :kept], first[:, :, :kept])
    assert la.la_device_status() == la.LA_OK


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (16, 2), (12, 1)])
def test_swa_step_of_infinite_values(H, Hkv, dtype):
    """A seen value of infinity with the only weight is the output, as in the plain step; its neighbours stay finite."""
    dev = cuda_device()
    g = gen(H)
    q, k, v = (randn(g, 2, n, 64, dtype=dtype).to(dev) for n in (H, Hkv, Hkv))
    kc, vc = (randn(g, 2, Hkv, 40, 64, dtype=dtype).to(dev) for _ in range(2))
    v[0, :, 5], v[1, :, 7] = float("inf"), -float("inf")
    pos = torch.tensor([0, 100], device=dev)  # alone, and beside a full ring
    out = la.la_swa_biased_decode_step(q, k, v, kc, vc, pos, out_dtype=FP)
    assert (out[0, :, 5] == float("inf")).all() and (out[1, :, 7] == -float("inf")).all()
    out[0, :, 5], out[1, :, 7] = 0, 0
    assert torch.isfinite(out).all()


def test_tensors_freed_behind_a_call_on_another_stream():
    """Inputs that are gone when a call on another stream gets to them, and outputs that are while their reader has not:
    neither's memory goes to the next tensor before that."""
    dev = cuda_device()
    N, C = 700, 256
    x, w = randn(gen(1), 2, N, C).to(dev), randn(gen(2), C, 4).to(dev)
    q, k, v = on(dev, *swa_case(1, 2, 1, 300, 300, 64, BF, 9))
    want = la.la_conv_prefill(x, w)[0], la.la_swa_prefill(q, k, v)
    side, big = torch.cuda.Stream(dev), torch.randn(8192, 8192, device=dev)
    torch.cuda.synchronize()

    def keep_busy():
        busy = big
        for _ in range(6):
            busy = busy @ big

    with torch.cuda.stream(side):
        keep_busy()
    got = [la.la_conv_prefill(x.clone(), w.clone(), stream=side)[0], la.la_swa_prefill(q.clone(), k=k.clone(), v=v.clone(), stream=side)]
    spoil = [torch.full_like(t, float("nan")) for t in (x, w, q, k, v)]  # where the copies were, were they free
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(spoil) == 5
    # outputs: read on this stream, behind long work, and dropped
    side.wait_stream(torch.cuda.current_stream())
    y = la.la_conv_prefill(x, w, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    keep_busy()
    copy = y * 1
    del y
    with torch.cuda.stream(side):
        spoil = [torch.full_like(x, float("nan")) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want[0])
