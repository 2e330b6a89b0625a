"""GPU parity of the queries' and keys' norms with the position rotation, and of the paged caches: appends, reads and a
step's attention, against fp64 definitions with per-entry error bounds."""
import numpy as np
import pytest
import torch

import linear_attention_recurrence_chunked_gb300 as la
from tests import layers_oracle
from tests import paged_oracle as ref
from tests.helpers import cuda_device

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=FP, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def on(dev, *ts):
    return [None if t is None else t.to(dev) for t in ts]


def longs(dev, xs):
    return torch.tensor(xs, dtype=torch.int64, device=dev)


def fused(g, dev, B, N, heads, d, dtype):
    """A projection's output [B, N, sum(heads), d] and its parts as [B, H, N, d] views."""
    x = randn(g, B, N, sum(heads), d, dtype=dtype).to(dev)
    parts, at = [], 0
    for h in heads:
        parts.append(x[:, :, at:at + h].transpose(1, 2))
        at += h
    return parts


def table_of(g, totals, page, spare_columns=1, spare_pages=2):
    """A table of pages in no order, -1 where no token needs one, and the pool's size."""
    need = [-(-t // page) for t in totals]
    count = sum(need) + spare_pages
    order = torch.randperm(count, generator=g)
    table = torch.full((len(totals), max(need) + spare_columns), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].int()
        at += n
    return table, count


def pack(x):
    """4-bit pages of bf16 rows [P, H, page, d], written from the layout in the header."""
    P, H, page, d = x.shape
    q, scale, lo = ref.quantise(x.double().numpy())
    codes = np.clip(np.rint(q), 0, 15).astype(np.uint32)
    words = np.zeros((P, H, page, d // 8), dtype=np.uint32)
    for w in range(d // 8):
        g, e = w % (d // 64), w // (d // 64)
        for j in range(8):
            words[..., w] |= codes[..., 64 * g + 8 * e + j] << np.uint32(4 * j)
    half = lambda t: torch.from_numpy(t).float().to(torch.bfloat16).view(torch.int16).numpy().astype(np.uint16)  # noqa: E731
    meta = half(scale).astype(np.uint32) | half(lo).astype(np.uint32) << np.uint32(16)
    raw = np.concatenate([words.reshape(P, H, -1), meta.reshape(P, H, -1)], -1)
    return torch.from_numpy(raw.view(np.uint8).reshape(P, H, page, d * 9 // 16).copy())


# ------------------------------------------------------------------------------------------ norms and rotation
@pytest.mark.parametrize("B,N,H,Hkv,d,rot,norm,interleaved,dtype,out,w_dtype,lens,pos", [
    (1, 1, 1, 1, 8, 0, "rms", False, BF, BF, None, None, None),
    (2, 5, 3, 1, 16, 16, "rms", False, FP, FP, FP, None, "first"),
    (1, 7, 2, 2, 128, 0, "l2", False, BF, BF, None, None, None),
    (3, 33, 16, 4, 128, 128, "rms", False, BF, BF, BF, [33, 0, 5], "first"),
    (2, 19, 6, 2, 96, 32, "rms", True, FP, BF, FP, [19, 1], "each"),
    (2, 40, 5, 5, 40, 32, "l2", False, BF, FP, FP, None, "each"),
    (1, 65, 9, 3, 256, 256, "rms", True, BF, BF, BF, None, None),
    (1, 21, 7, 7, 200, 48, "rms", False, FP, FP, None, [20], "first"),
    (2, 30, 4, 2, 64, 64, None, False, BF, BF, None, None, "first"),
    (1, 12, 33, 1, 72, 64, None, True, FP, FP, None, [11], "each"),
    (70, 1, 8, 2, 128, 64, "rms", False, BF, BF, FP, None, "first"),
    (1, 600, 40, 8, 128, 128, "rms", False, BF, BF, FP, None, None),
])
def test_qk_norm_rope(B, N, H, Hkv, d, rot, norm, interleaved, dtype, out, w_dtype, lens, pos):
    dev = cuda_device()
    g = gen(B + N + d + rot)
    q, k = fused(g, dev, B, N, (H, Hkv), d, dtype)
    wq, wk = (None, None) if w_dtype is None else ((1 + randn(g, d, scale=0.3)).to(w_dtype) for _ in range(2))
    cos, sin = ref.tables(900, rot) if rot else (None, None)
    at = np.tile(np.arange(N), (B, 1))
    p = None
    if rot and pos == "first":
        first = torch.randint(0, 900 - N, (B,), generator=g)
        at, p = at + first.numpy()[:, None], first.to(dev)
    elif rot and pos == "each":
        p = torch.randint(0, 900, (B, N), generator=g)
        at, p = p.numpy(), p.to(dev)
    want = [ref.norm_rope(x, w, norm, 1e-6, cos, sin, at, interleaved, lens, out) for x, w in ((q, wq), (k, wk))]
    for b, n in enumerate(lens or []):
        q[b, :, n:], k[b, :, n:] = float("nan"), float("nan")  # padding reaches nothing
    ln = None if lens is None else longs(dev, lens)
    wqd, wkd, cd, sd = on(dev, wq, wk, cos, sin)
    more = dict(q_weight=wqd, k_weight=wkd, norm=norm, cos=cd, sin=sd, pos=p, interleaved=interleaved, lens=ln)
    got = la.la_qk_norm_rope(q, k, out_dtype=out, **more)
    for (y, bound), x in zip(want, got):
        assert x.dtype == out
        ref.check(x, y, bound)
        for b, n in enumerate(lens or []):
            assert torch.all(x[b, :, n:] == 0)
    # outputs that are there: views, padding stays
    qo, ko = fused(g, dev, B, N, (H, Hkv), d, out)
    qo.fill_(5), ko.fill_(5)
    a, b = la.la_qk_norm_rope(q, k, q_out=qo, k_out=ko, **more)
    assert a is qo and b is ko
    for x, y in zip((qo, ko), got):
        for s in range(B):
            n = N if lens is None else lens[s]
            assert torch.equal(x[s, :, :n], y[s, :, :n]) and torch.all(x[s, :, n:] == 5)
    assert torch.equal(la.la_qk_norm_rope(k, q_weight=wkd, out_dtype=out, **{n: v for n, v in more.items() if not n.endswith("weight")})[0],
                       got[1])  # one of them alone
    if dtype == out:  # in place, inside the projection
        la.la_qk_norm_rope(q, k, q_out=q, k_out=k, **more)
        for x, y in zip((q, k), got):
            for s in range(B):
                n = N if lens is None else lens[s]
                assert torch.equal(x[s, :, :n], y[s, :, :n]) and torch.all(torch.isnan(x[s, :, n:]))
    assert la.la_device_status() == la.LA_OK


def test_qk_steps_are_the_prompts_tokens():
    dev = cuda_device()
    g = gen(2)
    S, H, Hkv, d = 5, 12, 4, 96
    x = randn(g, S, H + Hkv, d, dtype=BF).to(dev)
    cos, sin = on(dev, *ref.tables(100, 64))
    pos = longs(dev, [0, 99, 3, 50, 7])
    q, k = la.la_qk_norm_rope(x[:, :H], x[:, H:], cos=cos, sin=sin, pos=pos)
    assert q.shape == (S, H, d) and k.shape == (S, Hkv, d)
    q4, k4 = la.la_qk_norm_rope(x[:, :H, None], x[:, H:, None], cos=cos, sin=sin, pos=pos)
    assert torch.equal(q, q4[:, :, 0]) and torch.equal(k, k4[:, :, 0])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_norms_of_rows_at_the_ends(dtype):
    """Zeros, squares beyond fp32, NaN and infinities: a row's own affair."""
    dev = cuda_device()
    d = 64
    x = randn(gen(5), 1, 8, 1, d, dtype=dtype)
    plain = x.clone()
    x[0, 1] = 0
    x[0, 2] *= 1e30
    x[0, 3] *= 1e-30
    x[0, 4, 0, 3] = float("nan")
    x[0, 5, 0, 63] = float("inf")
    for norm in ("rms", "l2"):
        y, bound = ref.norm_rope(x[:, [0, 1, 2, 3, 6, 7]], None, norm, 1e-6, None, None, None, False, None, dtype)
        got = la.la_qk_norm_rope(x.to(dev), norm=norm)[0]
        ref.check(got[:, [0, 1, 2, 3, 6, 7]], y, bound)
        assert torch.isnan(got[0, 4]).all() and torch.isnan(got[0, 5, 0, 63]) and torch.all(got[0, 5, 0, :63] == 0)
        assert torch.equal(got[:, [0, 6, 7]], la.la_qk_norm_rope(plain.to(dev), norm=norm)[0][:, [0, 6, 7]])


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [8, 96, 256])
def test_norms_of_the_largest_rows(dtype, norm, d):
    """Rows whose length passes fp32, so that its reciprocal is a subnormal number, beside ordinary ones and small elements."""
    dev = cuda_device()
    g = gen(d)
    size = torch.tensor([1.0, 1e18, 2e19, 1e30, 1e37, 1.2e38, 2.1e38, 3.2e38, 3.3e38, 2.7e38, 1e-3, 1e38]).view(1, 12, 1, 1)
    x = (torch.rand((1, 12, 5, d), generator=g) * 0.3 + 0.7) * size * (1 - 2.0 * torch.randint(0, 2, (1, 12, 5, d), generator=g))
    x[..., 3] *= 2.0 ** -60
    x = x.to(dtype)
    y, bound = ref.norm_rope(x, None, norm, 1e-6, None, None, None, False, None, FP)
    ref.check(la.la_qk_norm_rope(x.to(dev), norm=norm, out_dtype=FP)[0], y, bound)


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("d", [64, 256])
def test_a_large_eps_counts_beside_squares_beyond_fp32(norm, d):
    """Sums of squares just below and beyond fp32's range."""
    dev = cuda_device()
    x = randn(gen(d), 2, 8, 3, d) / d ** 0.5
    x = x / x.norm(dim=-1, keepdim=True) * torch.tensor([0.9, 0.95, 0.99, 0.995, 1.01, 1.05, 1.3, 20.0]).view(1, 8, 1, 1) * 2.0 ** 64
    for eps in (1e37, 1e33, 1e-6):
        y, bound = ref.norm_rope(x, None, norm, eps, None, None, None, False, None, FP)
        ref.check(la.la_qk_norm_rope(x.to(dev), norm=norm, eps=eps)[0], y, bound)


def test_positions_outside_the_tables_are_skipped_and_reported():
    dev = cuda_device()
    cos, sin = on(dev, *ref.tables(10, 16))
    q = randn(gen(6), 3, 2, 4, 16).to(dev)
    for pos, dead in ((longs(dev, [0, 8, -2]), {(1, 2), (1, 3), (2, 0), (2, 1)}),
                      (longs(dev, [[0, 10, 2, 3], [-1, 9, 1 << 40, 0], [1, 2, 3, 4]]), {(0, 1), (1, 0), (1, 2)}),
                      (longs(dev, [(1 << 63) - 1, 0, -(1 << 63)]), {(0, n) for n in range(4)} | {(2, n) for n in range(4)})):
        out = torch.full_like(q, 7.0)
        la.la_qk_norm_rope(q, cos=cos, sin=sin, pos=pos, q_out=out)
        assert la.la_device_status() == la.LA_ERR_INVALID_ARGUMENT and la.la_device_status() == la.LA_OK
        made = la.la_qk_norm_rope(q, cos=cos, sin=sin, pos=pos)[0]  # zeros in an output made by the call
        assert torch.equal(made, torch.where(out == 7.0, torch.zeros_like(out), out))
        la.la_device_status()
        for b in range(3):
            for n in range(4):
                assert bool(torch.all(out[b, :, n] == 7.0)) == ((b, n) in dead)
    with pytest.raises(ValueError):
        la.la_qk_norm_rope(q, q, cos=cos, sin=sin, k_out=torch.full_like(q, 7.0))
    out = torch.full_like(q, 7.0)
    la.la_qk_norm_rope(q, lens=longs(dev, [5, 4, -1]), q_out=out)
    assert la.la_device_status() == la.LA_ERR_INVALID_ARGUMENT
    assert torch.all(out[0] == 7.0) and torch.all(out[2] == 7.0) and not torch.any(out[1] == 7.0)


# ------------------------------------------------------------------------------------------ appends and reads
@pytest.mark.parametrize("B,N,Hkv,d,page,rot,interleaved,dtype,bits,seen,lens", [
    (1, 1, 1, 8, 16, 0, False, FP, 0, [0], None),
    (2, 37, 3, 64, 16, 64, False, BF, 0, [5, 0], [37, 20]),
    (3, 18, 2, 40, 48, 32, True, FP, 0, [100, 47, 48], [18, 0, 1]),
    (2, 50, 5, 128, 32, 128, False, FP, 0, [31, 64], None),
    (1, 100, 8, 96, 64, 48, False, BF, 0, [3], None),
    (1, 1, 1, 64, 16, 0, False, BF, 4, [0], None),
    (2, 37, 3, 64, 16, 64, False, BF, 4, [5, 0], [37, 20]),
    (3, 18, 2, 128, 48, 96, True, BF, 4, [100, 47, 48], [18, 0, 1]),
    (2, 50, 5, 128, 32, 128, False, BF, 4, [31, 64], None),
    (40, 1, 4, 128, 64, 64, False, BF, 4, list(range(20, 60)), None),
    (40, 1, 4, 128, 64, 128, False, BF, 0, list(range(20, 60)), None),
])
def test_paged_append_and_read(B, N, Hkv, d, page, rot, interleaved, dtype, bits, seen, lens):
    dev = cuda_device()
    g = gen(N + d + rot + bits)
    k, v = fused(g, dev, B, N, (Hkv, Hkv), d, dtype)
    new = lens or [N] * B
    totals = [s + n for s, n in zip(seen, new)]
    table, count = table_of(g, totals, page)
    before = [randn(g, count, Hkv, page, d, dtype=dtype) for _ in range(2)]
    if bits:
        before = [pack(x) for x in before]
    pools = [x.to(dev) for x in before]
    cos, sin = ref.tables(max(totals) + 1, rot) if rot else (None, None)
    rows = [k.cpu().clone(), v.cpu().clone()]
    for b, n in enumerate(new):
        k[b, :, n:], v[b, :, n:] = float("nan"), float("nan")  # padding is not stored
    cd, sd, td = on(dev, cos, sin, table)
    if N == 1 and B > 1:
        k, v = k[:, :, 0], v[:, :, 0]
    out = la.la_paged_append(k, v, *pools, td, longs(dev, seen), cos=cd, sin=sd, interleaved=interleaved,
                             lens=None if lens is None else longs(dev, lens))
    assert out[0] is pools[0] and out[1] is pools[1]
    longest = max(totals) + 2
    back = la.la_paged_read(*pools, td, longs(dev, totals), longest)
    assert la.la_device_status() == la.LA_OK
    for which in range(2):
        was, now = (ref.values(x, d)[0] for x in (before[which], pools[which].cpu()))
        touched = np.zeros(now.shape[:1] + now.shape[2:3], dtype=bool)
        for b, (past, n) in enumerate(zip(seen, new)):
            x = rows[which][b, :, :n].double().numpy()
            mag = np.abs(x)
            p = np.arange(past, past + n)
            if which == 0 and rot:
                x, mag = ref.turn(x, cos.double().numpy()[p], sin.double().numpy()[p], interleaved)
            at = table[b].numpy()[p // page]
            touched[at, p % page] = True
            got = now[at, :, p % page].transpose(1, 0, 2)
            if not bits:
                # the two products' and the sum's roundings; values are copied
                bound = (2 * ref.U * mag + ref.half_step(dtype) * np.abs(x)) * (which == 0 and rot > 0)
                assert np.all(np.abs(got - x) <= bound)
                continue
            x = torch.from_numpy(x).float().to(BF).double().numpy()
            quotient, scale, lo = ref.quantise(x)
            codes, s_got, lo_got = (t[at, :, p % page].transpose(1, 0, 2) for t in ref.split(pools[which], d))
            assert np.array_equal(lo_got, lo)
            assert np.all(np.abs(s_got - scale) <= 2.0 ** -7 * scale)  # twice rounded to fp32 before: at a tie the next bf16
            exact = (x - np.repeat(lo, 64, -1)) / np.where(s_got > 0, s_got, 1).repeat(64, -1)
            # half a code, and the quotient's two fp32 roundings at most beside it
            assert np.all((np.abs(codes - exact) <= 0.5 + 16 * 2 * ref.U) | ((codes == 15) & (exact > 15)))
        assert np.array_equal(now[~touched.any(1)], was[~touched.any(1)])  # other pages
        stay = ~touched[:, None, :, None] & np.ones(now.shape, dtype=bool)
        assert np.array_equal(now[stay], was[stay])  # other slots
        for b, n in enumerate(totals):  # the cache as rows
            want = ref.gather(now, table, b, 0, n)
            assert torch.equal(back[which][b, :, :n].cpu(), torch.from_numpy(want).float().to(dtype))
            assert torch.all(back[which][b, :, n:] == 0)
    kept = [torch.full((B, longest, Hkv, d), 3.0, dtype=FP, device=dev).transpose(1, 2) for _ in range(2)]
    la.la_paged_read(*pools, td, longs(dev, totals), longest, k=kept[0], v=kept[1])
    for which in range(2):
        for b, n in enumerate(totals):
            want = ref.gather(ref.values(pools[which].cpu(), d)[0], table, b, 0, n)
            assert torch.equal(kept[which][b, :, :n].cpu(), torch.from_numpy(want).float())
            assert torch.all(kept[which][b, :, n:] == 3.0)


@pytest.mark.parametrize("dtype,bits,d", [(t, 0, d) for t in (BF, FP) for d in (8, 16, 24, 32, 40, 72, 128)] + [(BF, 4, 64), (BF, 4, 128)])
@pytest.mark.parametrize("page,N", [(16, 16), (16, 51), (48, 48), (48, 32)])
def test_reads_stay_within_their_rows(dtype, bits, d, page, N):
    """Lengths at, below and beyond whole tiles of 16 tokens, into views with other rows on every side of them."""
    dev = cuda_device()
    g = gen(d + page + N + bits)
    Hkv = 3
    lens = [n for n in (16, 0, 48, 17, 32, 15, 33, 1, 31, 51) if n <= N]
    lens.append(lens[0])  # a whole tile at the end
    table, count = table_of(g, lens, page, spare_pages=1)
    pools = [randn(g, count, Hkv, page, d, dtype=dtype) for _ in range(2)]
    if bits:
        pools = [pack(x) for x in pools]
    want = [ref.values(x, d)[0] for x in pools]
    given = [on(dev, x)[0] for x in (*pools, table)]
    B = len(lens)
    for out in (BF, FP):
        around = [torch.full((B + 2, Hkv + 2, N + 64, d + 8), 3.0, dtype=out, device=dev) for _ in range(2)]
        k, v = (x[1:-1, 1:-1, 32:32 + N, :d] for x in around)
        la.la_paged_read(*given, longs(dev, lens), N, k=k, v=v)
        made = la.la_paged_read(*given, longs(dev, lens), N, out_dtype=out)
        for which in range(2):
            rows = torch.full(tuple(around[which].shape), 3.0, dtype=out)
            alone = torch.zeros((B, Hkv, N, d), dtype=out)
            for b, n in enumerate(lens):
                x = torch.from_numpy(ref.gather(want[which], table, b, 0, n)).float().to(out)
                rows[1 + b, 1:-1, 32:32 + n, :d], alone[b, :, :n] = x, x
            assert torch.equal(around[which].cpu(), rows) and torch.equal(made[which].cpu(), alone)
    assert la.la_device_status() == la.LA_OK


def test_4bit_groups_at_the_ends():
    """Equal elements, tiny spreads, spreads beyond fp32, NaN and infinities: a group's own affair."""
    dev = cuda_device()
    d, page = 128, 16
    x = randn(gen(8), 1, 9, 1, d, dtype=BF)  # nine heads of one token
    x[0, 0] = 2.5
    x[0, 1, 0, :64] = 0
    x[0, 2, 0, :64] = torch.linspace(0, 1, 64).to(BF) * 2.0 ** -130
    x[0, 3, 0, 5] = float("nan")
    x[0, 4, 0, 70] = float("inf")
    x[0, 5, 0, 70] = -float("inf")
    x[0, 6, 0, :2] = torch.tensor([3e38, -3e38]).to(BF)
    x[0, 7, 0, :64] = -7.0
    x[0, 7, 0, 3] = 8.0
    pools = [torch.zeros((1, 9, page, d * 9 // 16), dtype=torch.uint8, device=dev) for _ in range(2)]
    table = torch.zeros((1, 1), dtype=torch.int32, device=dev)
    la.la_paged_append(x.to(dev), x.to(dev), *pools, table, longs(dev, [0]))
    k, v = la.la_paged_read(*pools, table, None, 1, out_dtype=FP)
    assert torch.equal(pools[0], pools[1]) and torch.equal(k.nan_to_num(1e9), v.nan_to_num(1e9))
    k = k.cpu()
    assert torch.all(k[0, 0] == 2.5) and torch.all(k[0, 1, 0, :64] == 0)
    for h, half in ((3, 0), (4, 1), (5, 1), (6, 0)):
        assert torch.isnan(k[0, h, 0, 64 * half:64 * half + 64]).all() and torch.isfinite(k[0, h, 0, 64 - 64 * half:128 - 64 * half]).all()
    assert torch.all(k[0, 7, 0, :64] == x[0, 7, 0, :64].float())  # a spread of 15: the codes are exact
    tiny = x[0, 2, 0, :64].float()
    assert (k[0, 2, 0, :64] - tiny).abs().max() <= 2.0 ** -130 / 15 * (0.5 + 15 * 2.0 ** -7) + 2.0 ** -133


def test_tokens_without_a_place_are_skipped_and_reported():
    dev = cuda_device()
    g = gen(9)
    Hkv, d, page = 2, 64, 16
    k = randn(g, 4, Hkv, 20, d, dtype=BF).to(dev)
    cos, sin = on(dev, *ref.tables(100, 32))
    table = torch.tensor([[0, 1, -1], [2, 7, 3], [4, 5, 6], [-5, 2 ** 31 - 1, 8]], dtype=torch.int32, device=dev)
    for bits in (0, 4):
        fresh = lambda: [torch.zeros((9, Hkv, page, d * 9 // 16 if bits else d), dtype=torch.uint8 if bits else BF, device=dev) for _ in range(2)]  # noqa: E731
        pools = fresh()
        # 0: to the table's hole; 1: behind the table; 2: a bad length; 3: pages that are none
        la.la_paged_append(k, k, *pools, table, longs(dev, [20, 40, 0, 8]), cos=cos, sin=sin, lens=longs(dev, [20, 20, 21, 20]))
        assert la.la_device_status() == la.LA_ERR_INVALID_ARGUMENT and la.la_device_status() == la.LA_OK
        row = d * 9 // 16 if bits else d
        pages = [p.reshape(9, Hkv, page, row) for p in pools]
        for p in (0, 2, 4, 5, 6, 7, 8):
            assert not pages[0][p].any() and not pages[1][p].any()
        assert pages[0][1].any() and pages[0][3].any()
        pools = fresh()
        for seen in ([-1, -30, -(1 << 62), (1 << 63) - 1], [95, 99, 1 << 33, 48]):  # before the first, behind the last position
            la.la_paged_append(k[:, :, :1], k[:, :, :1], *pools, table, longs(dev, seen), cos=cos[:48], sin=sin[:48])
            assert la.la_device_status() == la.LA_ERR_INVALID_ARGUMENT
        assert not pools[0].any() and not pools[1].any()
        pools = [torch.randint(0, 100, p.shape, device=dev).to(p.dtype) for p in pools]
        a, b = la.la_paged_read(*pools, table, longs(dev, [48, 48, 99, 16]), 48)
        assert la.la_device_status() == la.LA_ERR_INVALID_ARGUMENT
        assert not a[0, :, 32:].any() and a[0, :, :32].any() and a[1].any() and not a[2].any() and not a[3].any() and not b[3].any()


# ------------------------------------------------------------------------------------------ steps
def cache(g, lens, page, Hkv, d, dtype, bits, scale=1.0):
    """Pools whose unneeded slots hold NaN where a type has one, and the table."""
    table, count = table_of(g, lens, page)
    pools = []
    for _ in range(2):
        x = randn(g, count, Hkv, page, d, dtype=dtype, scale=scale)
        used = torch.zeros((count, page), dtype=torch.bool)
        for b, n in enumerate(lens):
            p = torch.arange(n)
            used[table[b].long()[p // page], p % page] = True
        if bits:
            raw = pack(x)
            flat = raw.view(count, Hkv, -1)
            meta = flat[..., page * d // 2:].reshape(count, Hkv, page, d // 16)
            meta[(~used)[:, None, :, None].expand(meta.shape)] = 255  # NaN scales and offsets
            flat[..., page * d // 2:] = meta.reshape(count, Hkv, -1)
            pools.append(flat.view(raw.shape))
        else:
            x[(~used)[:, None, :, None].expand(x.shape)] = float("nan")
            pools.append(x)
    return pools, table


STEPS = [
    (1, 1, 1, 8, 16, 0, 0.0, False, FP, FP, 0, [1]),
    (4, 6, 2, 40, 16, 0, 0.0, False, FP, FP, 0, [0, 1, 17, 90]),
    (3, 8, 1, 128, 48, 50, 20.0, True, FP, BF, 0, [49, 50, 333]),
    (2, 32, 2, 96, 32, 0, 0.0, True, FP, FP, 0, [300, 31]),
    (2, 5, 5, 64, 64, 7, 5.0, False, FP, FP, 0, [64, 65]),
    (4, 4, 4, 64, 16, 0, 0.0, False, BF, BF, 0, [0, 1, 16, 90]),
    (3, 8, 2, 128, 32, 0, 0.0, False, BF, FP, 0, [300, 15, 33]),
    (2, 16, 1, 128, 16, 100, 30.0, True, BF, FP, 0, [257, 99]),
    (3, 7, 1, 72, 48, 0, 0.0, True, BF, FP, 0, [48, 49, 200]),
    (2, 18, 2, 40, 64, 33, 0.0, False, BF, BF, 0, [500, 12]),
    (2, 3, 1, 8, 16, 0, 0.0, False, BF, FP, 0, [77, 2]),
    (4, 4, 4, 64, 16, 0, 0.0, False, BF, BF, 4, [0, 1, 16, 90]),
    (3, 8, 2, 128, 32, 0, 0.0, False, BF, FP, 4, [300, 15, 33]),
    (2, 16, 1, 128, 16, 100, 30.0, True, BF, FP, 4, [257, 99]),
    (3, 10, 1, 64, 48, 0, 0.0, True, BF, FP, 4, [48, 49, 200]),
    (2, 18, 2, 64, 64, 33, 0.0, False, BF, BF, 4, [500, 12]),
]


@pytest.mark.parametrize("S,H,Hkv,d,page,window,softcap,slopes,dtype,out,bits,lens", STEPS)
def test_paged_decode_step(S, H, Hkv, d, page, window, softcap, slopes, dtype, out, bits, lens):
    dev = cuda_device()
    g = gen(H + d + page + window)
    pools, table = cache(g, lens, page, Hkv, d, dtype, bits, 1.3)
    qkv = randn(g, S, H + Hkv, d, dtype=dtype, scale=1.3)
    sl = torch.exp2(-8.0 * torch.arange(1, H + 1) / H) if slopes else None
    o, bound = ref.step(qkv[:, :H], *pools, table, lens, window, d ** -0.5, softcap, sl, out)
    qd, kd, vd, td, sld = on(dev, qkv, *pools, table, sl)
    got = la.la_paged_decode_step(qd[:, :H], kd, vd, td, longs(dev, lens), window=window, softcap=softcap, slopes=sld, out_dtype=out)
    ref.check(got, o, bound)
    wide = torch.full((S, H + 3, d + 8), 5.0, dtype=out, device=dev)  # a view as the output
    la.la_paged_decode_step(qd[:, :H], kd, vd, td, longs(dev, lens), window=window, softcap=softcap, slopes=sld, out=wide[:, 1:H + 1, :d])
    assert torch.equal(wide[:, 1:H + 1, :d], got) and torch.all(wide[:, :1] == 5) and torch.all(wide[:, H + 1:] == 5) and torch.all(wide[..., d:] == 5)
    assert la.la_device_status() == la.LA_OK


@pytest.mark.parametrize("dtype,bits,H,Hkv,d,window,softcap", [
    (FP, 0, 4, 2, 64, 0, 0.0), (BF, 0, 8, 1, 128, 0, 0.0), (BF, 0, 12, 1, 96, 3001, 25.0), (BF, 4, 8, 1, 128, 0, 0.0), (BF, 4, 16, 1, 64, 3001, 0.0)])
def test_split_sequences(dtype, bits, H, Hkv, d, window, softcap):
    """Long sequences beside short ones: the tokens are split, and the parts joined."""
    dev = cuda_device()
    g = gen(d + bits + window)
    lens = [5000, 0, 1, 255, 256, 257, 1025]
    pools, table = cache(g, lens, 32, Hkv, d, dtype, bits, 1.2)
    q = randn(g, len(lens), H, d, dtype=dtype, scale=1.2)
    o, bound = ref.step(q, *pools, table, lens, window, d ** -0.5, softcap, None, FP)
    qd, kd, vd, td = on(dev, q, *pools, table)
    size = la.la_paged_decode_workspace_size(qd, kd, vd, td, window)
    assert size > 0
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device=dev)  # NaN where nothing is written
    got = la.la_paged_decode_step(qd, kd, vd, td, longs(dev, lens), window=window, softcap=softcap, out_dtype=FP, workspace=ws[:size])
    ref.check(got, o, bound)
    assert torch.all(ws[size:] == 255)
    assert torch.equal(got, la.la_paged_decode_step(qd, kd, vd, td, longs(dev, lens), window=window, softcap=softcap, out_dtype=FP))
    with pytest.raises(la.LAError):
        la.la_paged_decode_step(qd, kd, vd, td, longs(dev, lens), window=window, workspace=ws[:size - 16])


@pytest.mark.parametrize("bits,d,H,Hkv", [(0, 128, 8, 4), (0, 40, 40, 4), (4, 64, 4, 4), (4, 128, 16, 4), (4, 128, 64, 4)])
def test_many_short_sequences(bits, d, H, Hkv):
    """Enough of them for blocks of one warp."""
    dev = cuda_device()
    g = gen(d + H)
    S, page = 640, 16
    lens = [(7 * s) % 61 for s in range(S)]
    pools, table = cache(g, lens, page, Hkv, d, BF, bits, 1.2)
    q = randn(g, S, H, d, dtype=BF, scale=1.2)
    sl = torch.exp2(-8.0 * torch.arange(1, H + 1) / H)
    for window in (0, 19):
        got = la.la_paged_decode_step(*on(dev, q, *pools, table), longs(dev, lens), window=window, slopes=sl.to(dev), out_dtype=FP)
        some = list(range(0, S, 23)) + [S - 1]
        o, bound = ref.step(q[some], *pools, table[some], [lens[s] for s in some], window, d ** -0.5, 0.0, sl, FP)
        ref.check(got[some], o, bound)
        assert torch.isfinite(got).all() and torch.all(got[[s for s in range(S) if lens[s] == 0]] == 0)
    assert la.la_device_status() == la.LA_OK


@pytest.mark.parametrize("bits,d,H", [(0, 128, 4), (4, 64, 4), (4, 128, 16)])
def test_means_of_many_values_keep_their_bits(bits, d, H):
    """A flat softmax over 40000 tokens gives means of 1 / sqrt(n) of a value's size, which sums that drift would drown.  Each
    weight is off by up to 2^-17 of itself, independently, and adds 2^-17 / sqrt(n) of a value, 2^-17 of the mean's size; fp32
    sums of n / 1000 terms a warp and their join stay below that.  Four times as much is allowed."""
    dev = cuda_device()
    g = torch.Generator(device=dev).manual_seed(d + H)
    n, page = 40000, 64
    P = n // page
    x = [torch.randn((P, 1, page, d), generator=g, device=dev).to(BF) for _ in range(2)]
    table = torch.randperm(P, generator=g, device=dev).to(torch.int32)[None]
    q = (0.05 * torch.randn((1, H, d), generator=g, device=dev)).to(BF)
    pools = [torch.zeros((P, 1, page, d * 9 // 16), dtype=torch.uint8, device=dev) for _ in range(2)] if bits else x
    rows = [t[table[0].long()].permute(1, 0, 2, 3).reshape(1, 1, n, d) for t in x]
    if bits:
        la.la_paged_append(*rows, *pools, table, longs(dev, [0]))
        rows = la.la_paged_read(*pools, table, None, n, out_dtype=FP)
    out = la.la_paged_decode_step(q, *pools, table, longs(dev, [n]), out_dtype=FP).double()
    k, v = (t[0, 0].double() for t in rows)
    want = torch.softmax(q[0].double() @ k.T * d ** -0.5, -1) @ v
    assert (out[0] - want).norm() <= 2.0 ** -15 * want.norm()


def two_tokens(g, dev, S, H, d, bits, low, high):
    """S sequences of two tokens: a key of zeros with values of zeros, and one whose score x, low <= -x <= high, fp32 holds
    exactly, with whole numbers as values, which 4 bits hold exactly.  Returns (x [S, H], values [d], the call's inputs)."""
    k, v = torch.zeros((S, 1, 16, d)), torch.zeros((S, 1, 16, d))
    c = (1 + torch.rand(S, generator=g)).to(BF)
    u = (low + (high / 2 - low) * torch.rand((S, H), generator=g)).to(BF)
    k[:, 0, 1] = c.float()[:, None]
    v[:, 0, 1] = (torch.arange(d) % 16).float()
    q = torch.zeros((S, H, d))
    q[:, :, 0] = -u.float()
    pools = [t.to(BF) for t in (k, v)]
    if bits:
        pools = [pack(t) for t in pools]
    table = torch.randperm(S, generator=g).int()[:, None]
    x = q[:, :, 0].double() * c.double()[table[:, 0].long()][:, None]
    return x.numpy(), v[0, 0, 1].double().numpy(), [*on(dev, q.to(BF), *pools, table), longs(dev, [2] * S)]


def check_two_tokens(got, s, es, v, bits):
    """got [S, H, d] against the softmax of scores 0 and s, which is off by es; the rest of the bound is counted here."""
    U = ref.U
    p = np.exp(s)[..., None]
    # of the second weight: the score in units of log2 (its factor's rounding and the product's), 2 ulp of the exponential;
    # of the sum: the first weight is one, their sum's rounding; then the weight's three parts together (2^-26), four
    # additions on the tensor cores that may cut off (2 U), the parts' and warps' sums, the quotient and its rounding
    bound = es + 2 * U * np.abs(s) + (4 + 1 + 0.25 + 8 + 2 + 2) * U
    mag = (np.abs(v - 8) + 8 if bits else v) * p / (1 + p)  # 4 bits: centred codes and what they were centred by
    ref.check(got, p * v / (1 + p), bound[..., None] * mag)


@pytest.mark.parametrize("bits,d,H", [(0, 64, 8), (0, 128, 3), (0, 128, 16), (0, 40, 9), (4, 64, 8), (4, 128, 2), (4, 128, 16)])
def test_weights_of_fp32_outputs_keep_their_bits(bits, d, H):
    """Weights that two bf16 parts would leave off by up to 2^-17, 128 half steps of fp32."""
    dev = cuda_device()
    x, v, inputs = two_tokens(gen(d + H), dev, 100, H, d, bits, 0.5, 3.0)
    got = la.la_paged_decode_step(*inputs, scale=1.0, out_dtype=FP)
    check_two_tokens(got, x, 0.0, v, bits)
    rounded = la.la_paged_decode_step(*inputs, scale=1.0)  # bf16 outputs: two parts, less than a hundredth of their half step
    p = np.exp(x)[..., None]
    mag = (np.abs(v - 8) + 8 if bits else v) * p / (1 + p)
    ref.check(rounded, p * v / (1 + p), 2.0 ** -8 * p * v / (1 + p) + 2.0 ** -16 * mag)


@pytest.mark.parametrize("bits,d,H", [(0, 64, 8), (0, 128, 16), (4, 64, 8), (4, 128, 16)])
@pytest.mark.parametrize("low,high", [(4.0, 14.9), (15.5, 60.0)])
def test_capped_scores_of_fp32_outputs_keep_their_bits(bits, d, H, low, high):
    """Scores up to half of the cap, and beyond."""
    dev = cuda_device()
    U, cap = ref.U, 30.0
    x, v, inputs = two_tokens(gen(d + H + int(low)), dev, 100, H, d, bits, low, high)
    z = x / cap
    s, a, r = cap * np.tanh(z), np.abs(z), 1 / (1 + np.exp(2 * np.abs(z)))
    # up to half of the cap: the polynomial's 2.6e-8, and an argument off by 2 U twice, which reaches the value with a twelfth;
    # its last term's rounding and the product's.  Beyond: an exponent off by 8 a U, 2 ulp of its exponential, a sum, 1 ulp of the
    # reciprocal, and the difference's rounding.
    near = (2.6e-8 + (5 / 12 + 0.1 + 2) * U) * np.abs(s)
    far = 2 * cap * r * (8 * a + 4 + 1 + 2) * U + U * np.abs(s)
    got = la.la_paged_decode_step(*inputs, scale=1.0, softcap=cap, out_dtype=FP)
    check_two_tokens(got, s, np.where(a <= 0.5, near, far), v, bits)


@pytest.mark.parametrize("dtype,bits", [(FP, 0), (BF, 0), (BF, 4)])
def test_steps_report_bad_lengths_and_pages(dtype, bits):
    dev = cuda_device()
    g = gen(3)
    lens = [40, 40, 40, 40]
    pools, table = cache(g, lens, 16, 2, 64, dtype, bits)
    q = randn(g, 4, 4, 64, dtype=dtype)
    qd, kd, vd, td = on(dev, q, *pools, table)
    out = torch.full((4, 4, 64), 7.0, device=dev)
    la.la_paged_decode_step(qd, kd, vd, td, longs(dev, [40, -1, td.shape[1] * 16 + 1, 1 << 40]), out=out)
    assert la.la_device_status() == la.LA_ERR_INVALID_ARGUMENT and la.la_device_status() == la.LA_OK
    assert torch.all(out[1:] == 7.0) and not torch.any(out[0] == 7.0)
    bad = table.clone()
    bad[1, 1], bad[2, 0] = 10 ** 6, -1
    got = la.la_paged_decode_step(qd, kd, vd, bad.to(dev), longs(dev, lens), out_dtype=FP)
    assert la.la_device_status() == la.LA_ERR_INVALID_ARGUMENT
    # the other pages' tokens are seen: the same as sequences without the page
    o, bound = ref.step(q[:1], *pools, table[:1], lens[:1], 0, 0.125, 0.0, None, FP)
    ref.check(got[:1], o, bound)
    short = torch.stack([table[1][[0, 2, 1, 1]], table[2][[1, 2, 0, 0]]])
    o, bound = ref.step(q[1:3], *pools, short, [24, 24], 0, 0.125, 0.0, None, FP)
    ref.check(got[1:3], o, bound)


@pytest.mark.parametrize("dtype,bits", [(FP, 0), (BF, 0), (BF, 4)])
@pytest.mark.parametrize("width", [2, 100])
def test_no_weight_gives_zeros(dtype, bits, width):
    """Sequences none of whose pages is there, empty ones, and scores of -infinity alone."""
    dev = cuda_device()
    g = gen(17)
    pools, table = cache(g, [32, 32, 32], 16, 1, 64, dtype, bits)
    wide = torch.full((3, width), -1, dtype=torch.int32)
    wide[:, :2] = table[:, :2]
    wide[0, :2] = -1
    q = torch.ones((3, 4, 64), dtype=dtype)
    if not bits:
        pools[0][table[2, :2].long()] = -float("inf")
    qd, kd, vd, td = on(dev, q, *pools, wide)
    got = la.la_paged_decode_step(qd, kd, vd, td, longs(dev, [32, 0, 32]), out_dtype=FP)
    assert la.la_device_status() == la.LA_ERR_INVALID_ARGUMENT
    assert torch.all(got[:2] == 0) and (bits or torch.all(got[2] == 0))


@pytest.mark.parametrize("dtype,bits", [(FP, 0), (BF, 0), (BF, 4)])
def test_scores_far_apart(dtype, bits):
    """One key that takes all the weight, first or last, and scores beyond what exp holds."""
    dev = cuda_device()
    g = gen(4)
    H, d, n = 4, 64, 200
    pools, table = cache(g, [n, n, n], 16, 1, d, dtype, bits)
    q = randn(g, 3, H, d, dtype=dtype, scale=60.0)
    for s, at in ((0, 0), (1, n - 1), (2, 100)):
        if not bits:
            pools[0][table[s, at // 16], 0, at % 16] = q[s, 0]
    o, bound = ref.step(q, *pools, table, [n] * 3, 0, d ** -0.5, 0.0, None, FP)
    got = la.la_paged_decode_step(*on(dev, q, *pools, table), longs(dev, [n] * 3), out_dtype=FP)
    ref.check(got, o, bound)


@pytest.mark.parametrize("dtype,bits,H,d", [(FP, 0, 4, 64), (BF, 0, 4, 64), (BF, 0, 16, 128), (BF, 4, 4, 64), (BF, 4, 8, 128), (BF, 4, 16, 128)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
def test_a_heads_query_is_its_own(dtype, bits, H, d, value):
    """Small queries of large keys, beside a head whose query is huge or not finite: it reaches no other head."""
    dev = cuda_device()
    g = gen(31)
    n, odd = 150, 1
    pools, table = cache(g, [n], 16, 1, d, dtype, bits, scale=128.0)
    q = randn(g, 1, H, d, dtype=dtype, scale=2.0 ** -7)
    others = [h for h in range(H) if h != odd]
    o, bound = ref.step(q[:, others], *pools, table, [n], 0, d ** -0.5, 0.0, None, FP)
    q[:, odd] = value
    got = la.la_paged_decode_step(*on(dev, q, *pools, table), longs(dev, [n]), out_dtype=FP)
    ref.check(got[:, others], o, bound)


@pytest.mark.parametrize("H", [4, 16])
@pytest.mark.parametrize("dtype", [FP, BF])
def test_values_that_are_not_finite(dtype, H):
    """An infinite value of a token that is seen reaches its column alone, a NaN too; what is not seen reaches nothing."""
    dev = cuda_device()
    g = gen(14)
    d, n = 64, 90
    pools, table = cache(g, [n], 16, 1, d, dtype, 0)
    q = randn(g, 1, H, d, dtype=dtype)
    clean = la.la_paged_decode_step(*on(dev, q, *pools, table), longs(dev, [n]), window=50, out_dtype=FP)
    v = pools[1]
    v[table[0, 80 // 16], 0, 80 % 16, 5] = float("inf")
    v[table[0, 80 // 16], 0, 80 % 16, 6] = float("nan")
    v[table[0, 10 // 16], 0, 10 % 16, 7] = float("inf")  # behind the window
    v[table[0, 39 // 16], 0, 39 % 16] = float("nan")     # behind the window, in its first tile
    pools[0][table[0, 39 // 16], 0, 39 % 16] = float("nan")
    got = la.la_paged_decode_step(*on(dev, q, *pools, table), longs(dev, [n]), window=50, out_dtype=FP)
    assert torch.all(got[0, :, 5] == float("inf")) and torch.all(torch.isnan(got[0, :, 6]))
    rest = [c for c in range(d) if c not in (5, 6)]
    assert torch.isfinite(got[0][:, rest]).all() and torch.equal(got[0][:, rest], clean[0][:, rest])


@pytest.mark.parametrize("dtype,bits", [(FP, 0), (BF, 0), (BF, 4)])
def test_repeated_axes_full_tables_and_single_tokens(dtype, bits):
    """Heads or sequences repeated with stride 0, sequences that fill their table to the last slot, windows of one token."""
    dev = cuda_device()
    g = gen(61 + bits)
    B, H, Hkv, N, d, page = 3, 6, 2, 32, 64, 16
    cos, sin = ref.tables(N, 64)
    x = randn(g, 1, 1, N, d, dtype=dtype)
    y, bound = ref.norm_rope(x, None, "l2", 1e-6, cos, sin, np.arange(N)[None], False, None, dtype)
    cd, sd = on(dev, cos, sin)
    got, alone = la.la_qk_norm_rope(x.to(dev).expand(B, H, N, d), x.to(dev).expand(B, Hkv, N, d), norm="l2", cos=cd, sin=sd)
    ref.check(got, np.broadcast_to(y, got.shape), np.broadcast_to(bound, got.shape))
    assert torch.equal(got[:, :Hkv], alone)
    table, count = table_of(g, [N] * B, page, spare_columns=0, spare_pages=0)
    assert table.shape[1] * page == N
    pools = [torch.zeros((count, Hkv, page, d * 9 // 16 if bits else d), dtype=torch.uint8 if bits else dtype, device=dev) for _ in range(2)]
    v = randn(g, B, 1, N, d, dtype=dtype).to(dev).expand(B, Hkv, N, d)
    la.la_paged_append(alone[:1].expand(B, Hkv, N, d), v, *pools, table.to(dev), longs(dev, [0] * B))
    q = randn(g, 1, H, d, dtype=dtype)
    for window in (0, 1):
        o, bound = ref.step(q.expand(B, H, d), *pools, table, [N, N, N - 1], window, d ** -0.5, 0.0, None, FP)
        got = la.la_paged_decode_step(q.to(dev).expand(B, H, d), *pools, table.to(dev), longs(dev, [N, N, N - 1]), window=window, out_dtype=FP)
        ref.check(got, o, bound)
    if not bits:
        assert torch.equal(got[0, 0], v[0, 0, N - 1].float()) and torch.equal(got[2, 5], v[2, 1, N - 2].float())
    assert la.la_device_status() == la.LA_OK


# ------------------------------------------------------------------------------------------ together, streams, graphs
@pytest.mark.parametrize("bits,window,interleaved", [(0, 0, False), (4, 0, False), (0, 40, True)])
def test_a_layer_over_a_prompt_and_steps(bits, window, interleaved):
    """Norms and rotation, the prompt's attention, its keys and values into pages, a second chunk that reads them back, then
    single tokens: each equal to attention over the rows that the cache stands for."""
    dev = cuda_device()
    g = gen(20 + bits)
    B, H, Hkv, d, page = 3, 8, 2, 64, 16
    first, second, steps = [33, 20, 1], [10, 17, 16], 4
    total = [a + b for a, b in zip(first, second)]
    N = max(total) + steps
    q, k, v = fused(g, dev, B, N, (H, Hkv, Hkv), d, BF)
    wq, wk = ((1 + randn(g, d, scale=0.2)).to(dev) for _ in range(2))
    cos, sin = on(dev, *ref.tables(N, 32))
    table, count = table_of(g, [t + steps for t in total], page)
    td = table.to(dev)
    pools = [torch.zeros((count, Hkv, page, d * 9 // 16 if bits else d), dtype=torch.uint8 if bits else BF, device=dev) for _ in range(2)]
    kw = dict(q_weight=wq, k_weight=wk, cos=cos, sin=sin, interleaved=interleaved)

    def rows_of(start, lens, width):  # each sequence's tokens from its own start, padded
        out = []
        for x in (q, k, v):
            y = torch.zeros((B, x.shape[1], width, d), dtype=BF, device=dev)
            for b in range(B):
                y[b, :, :lens[b]] = x[b, :, start[b]:start[b] + lens[b]]
            out.append(y)
        return out

    # the first chunk
    qc, kc, vc = rows_of([0] * B, first, max(first))
    qn, kn = la.la_qk_norm_rope(qc, kc, lens=longs(dev, first), **kw)
    la.la_swa_prefill(qn, kn, vc, window=window, lens=longs(dev, first))
    la.la_paged_append(kn, vc, *pools, td, longs(dev, [0] * B), lens=longs(dev, first))
    # the second one: queries at their positions over everything so far
    qc, kc, vc = rows_of(first, second, max(second))
    qn, kn = la.la_qk_norm_rope(qc, kc, pos=longs(dev, first), lens=longs(dev, second), **kw)
    la.la_paged_append(kn, vc, *pools, td, longs(dev, first), lens=longs(dev, second))
    for b in range(B):
        t = longs(dev, [total[b]])
        kr, vr = la.la_paged_read(*pools, td[b:b + 1], t, total[b])
        o = la.la_swa_prefill(qn[b:b + 1, :, :second[b]], kr, vr, window=window, out_dtype=FP)
        spans = layers_oracle.spans(second[b], total[b], 1, window, None, None, first[b], None)
        want, bound = layers_oracle.swa(qn[b:b + 1, :, :second[b]], kr, vr, d ** -0.5, 0.0, None, spans, first[b], FP)
        ref.check(o, want, bound)
    # single tokens: keys without the norm's call are rotated by the append
    for t in range(steps):
        n = [x + t for x in total]
        qt, kt, vt = (x[:, :, 0] for x in rows_of(n, [1] * B, 1))
        qn, _ = la.la_qk_norm_rope(qt, q_weight=wq, cos=cos, sin=sin, pos=longs(dev, n), interleaved=interleaved)
        kn, _ = la.la_qk_norm_rope(kt, q_weight=wk)
        la.la_paged_append(kn, vt, *pools, td, longs(dev, n), cos=cos, sin=sin, interleaved=interleaved)
        o = la.la_paged_decode_step(qn, *pools, td, longs(dev, n) + 1, window=window, out_dtype=FP)
        want, bound = ref.step(qn, *pools, table, [x + 1 for x in n], window, d ** -0.5, 0.0, None, FP)
        ref.check(o, want, bound)
    if not bits:  # the cache holds the normed and rotated keys, whichever call turned them
        _, kn = la.la_qk_norm_rope(q, k, **kw)
        kr, vr = la.la_paged_read(*pools, td, longs(dev, [t + steps for t in total]), max(total) + steps)
        for b in range(B):
            m = total[b] + steps
            assert torch.equal(kr[b, :, :total[b]], kn[b, :, :total[b]]) and torch.equal(vr[b, :, :m], v[b, :, :m])
            # the steps' keys were rounded to bf16 once more between norm and rotation: a half step each, of the pair's length
            far = (kr[b, :, total[b]:m].float() - kn[b, :, total[b]:m].float()).abs().max()
            assert far <= 4 * 2.0 ** -8 * kn[b].float().abs().max()
    assert la.la_device_status() == la.LA_OK


def step_layer(q, k, v, pools, table, seen, cos, sin, workspace=None):
    qn, kn = la.la_qk_norm_rope(q, k, cos=cos, sin=sin, pos=seen)
    la.la_paged_append(kn, v, *pools, table, seen)
    return la.la_paged_decode_step(qn, *pools, table, seen + 1, workspace=workspace)


@pytest.mark.parametrize("bits", [0, 4])
def test_captured_layers_that_share_a_workspace_replay(bits):
    """Two layers' steps in two graphs, one workspace: replayed with new inputs they give what eager calls give."""
    dev = cuda_device()
    g = gen(31 + bits)
    S, H, Hkv, d, page = 2, 8, 2, 128, 32
    lens = [900, 1500]
    cos, sin = on(dev, *ref.tables(2000, 64))
    layers, q, k, v = [], *(randn(g, S, h, d, dtype=BF).to(dev) for h in (H, Hkv, Hkv))
    seen = longs(dev, lens)
    for _ in range(2):
        pools, table = cache(g, [n + 8 for n in lens], page, Hkv, d, BF, bits)
        layers.append(([p.to(dev) for p in pools], table.to(dev)))
    size = max(la.la_paged_decode_workspace_size(q, *pools, table) for pools, table in layers)
    assert size > 0
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    for pools, table in layers:
        step_layer(q, k, v, pools, table, seen, cos, sin, ws)  # warm
    graphs, outs = [], []
    for pools, table in layers:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step_layer(q, k, v, pools, table, seen, cos, sin, ws))
        graphs.append(graph)
    for t in range(3):
        for x, h in ((q, H), (k, Hkv), (v, Hkv)):
            x.copy_(randn(g, S, h, d, dtype=BF))
        seen.copy_(longs(dev, [n + t for n in lens]))
        for graph in graphs + graphs:  # appending a token again changes nothing
            graph.replay()
        got = [o.clone() for o in outs]
        for (pools, table), o in zip(layers, got):
            copy = [p.clone() for p in pools]
            assert torch.equal(step_layer(q, k, v, copy, table, seen, cos, sin), o)
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(copy, pools))  # NaN among them
    assert la.la_device_status() == la.LA_OK


def test_calls_on_a_given_stream():
    dev = cuda_device()
    g = gen(41)
    S, H, Hkv, d, page = 3, 4, 2, 64, 16
    lens = [700, 3, 1000]
    pools, table = cache(g, [n + 1 for n in lens], page, Hkv, d, BF, 0)
    pools, table = [p.to(dev) for p in pools], table.to(dev)
    q, k, v = (randn(g, S, h, d, dtype=BF).to(dev) for h in (H, Hkv, Hkv))
    cos, sin = on(dev, *ref.tables(2000, 64))
    seen = longs(dev, lens)
    want = step_layer(q, k, v, pools, table, seen, cos, sin)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        qn, kn = la.la_qk_norm_rope(q, k, cos=cos, sin=sin, pos=seen, stream=s)
        alone, none = la.la_qk_norm_rope(q, cos=cos, sin=sin, pos=seen, stream=s)
        assert none is None
        la.la_paged_append(kn, v, *pools, table, seen, stream=s)
        with torch.cuda.stream(side):
            n = seen + 1
        out = la.la_paged_decode_step(qn, *pools, table, n, stream=s)
        kr, vr = la.la_paged_read(*pools, table, n, 1001, stream=s)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want) and torch.equal(alone, qn)
        assert torch.equal(kr[0, :, 700], kn[0]) and torch.equal(vr[2, :, 1000], v[2])


def test_calls_at_once_on_two_streams():
    """Calls share nothing but the status word: each with its own workspace, on streams of their own."""
    dev = cuda_device()
    g = gen(43)
    H, Hkv, d, page, lens = 8, 2, 128, 32, [3000, 2500]
    jobs = []
    for bits in (0, 4, 0, 4):
        pools, table = cache(g, lens, page, Hkv, d, BF, bits)
        q = randn(g, 2, H, d, dtype=BF)
        jobs.append(on(dev, q, *pools, table))
    n = longs(dev, lens)
    want = [la.la_paged_decode_step(*j, n) for j in jobs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for i, j in enumerate(jobs):
            got.append((i, la.la_paged_decode_step(*j, n, stream=streams[i % 2])))
    torch.cuda.synchronize()
    for i, o in got:
        assert torch.equal(o, want[i])


@pytest.mark.parametrize("dtype,bits,page", [(BF, 0, 64), (BF, 4, 4096), (FP, 0, 16)])
def test_offsets_beyond_32_bits(dtype, bits, page):
    """A pool of more than 2^32 bytes (and 2^31 elements): tokens of its last pages are stored, read back and seen."""
    dev = cuda_device()
    Hkv, d, S, H = 2, 128, 2, 4
    row = d * 9 // 16 if bits else d * (2 if dtype == BF else 4)
    count = (5 << 30) // (Hkv * page * row) + 3
    if not bits:
        count = max(count, (1 << 31) // (Hkv * page * d) + 3)
    pools = [torch.empty((count, Hkv, page, d * 9 // 16 if bits else d), dtype=torch.uint8 if bits else dtype, device=dev) for _ in range(2)]
    g = gen(51)
    N = 50
    table = torch.full((S, 4), -1, dtype=torch.int32)
    need = -(-N // page)
    for s in range(S):
        table[s, :need] = torch.arange(count - 1 - s, count - 1 - s - 2 * need, -2)[:need].int()
    k, v, q = (randn(g, S, h, n, d, dtype=dtype).to(dev) for h, n in ((Hkv, N), (Hkv, N), (H, 1)))
    td, lens = table.to(dev), longs(dev, [N, N - 7])
    la.la_paged_append(k, v, *pools, td, longs(dev, [0, 0]), lens=lens)
    small = [p[table[:, :need].flatten().long().to(dev)].cpu() for p in pools]  # the used pages as a pool of their own
    near = torch.arange(S * need, dtype=torch.int32).view(S, need)
    out = la.la_paged_decode_step(q[:, :, 0], *pools, td, lens, out_dtype=FP)
    o, bound = ref.step(q[:, :, 0], *small, near, [N, N - 7], 0, d ** -0.5, 0.0, None, FP)
    ref.check(out, o, bound)
    kr, _ = la.la_paged_read(*pools, td, lens, N)
    if not bits:
        assert torch.equal(kr[0], k[0]) and torch.equal(kr[1, :, :N - 7], k[1, :, :N - 7])
    assert la.la_device_status() == la.LA_OK


@pytest.mark.parametrize("dtype,bits,page", [(BF, 0, 64), (BF, 4, 4096), (FP, 0, 16)])
def test_tokens_beyond_32_bits_are_where_the_table_says(dtype, bits, page):
    """Appends into a pool of more than 2^32 bytes whose used pages held a pattern: the same bytes as in a small pool, in their
    slots and nowhere else on these pages; read back, the same rows."""
    dev = cuda_device()
    Hkv, d, S, N = 2, 128, 2, 50
    row = d * 9 // 16 if bits else d * (2 if dtype == BF else 4)
    count = (5 << 30) // (Hkv * page * row) + 3
    if not bits:
        count = max(count, (1 << 31) // (Hkv * page * d) + 3)
    need = -(-N // page)
    assert (count - 2 * S * need) * Hkv * page * row > 1 << 32
    g = gen(53)
    far = torch.full((S, need + 1), -1, dtype=torch.int32)
    for s in range(S):
        far[s, :need] = torch.arange(count - 1 - s, count - 1 - s - 2 * need, -2).int()
    near = torch.full((S, need + 1), -1, dtype=torch.int32)
    near[:, :need] = torch.arange(S * need, dtype=torch.int32).view(S, need)
    k, v = (randn(g, S, Hkv, N, d, dtype=dtype).to(dev) for _ in range(2))
    lens, zero = longs(dev, [N, N - 7]), longs(dev, [0, 0])
    last = row if bits else d
    kind = torch.uint8 if bits else dtype
    used = far[:, :need].flatten().long().to(dev)
    large = [torch.empty((count, Hkv, page, last), dtype=kind, device=dev) for _ in range(2)]
    small = [torch.empty((S * need, Hkv, page, last), dtype=kind, device=dev) for _ in range(2)]
    for x, y in zip(large, small):
        y.view(torch.uint8).fill_(0x5a)
        x[used] = y
    la.la_paged_append(k, v, *large, far.to(dev), zero, lens=lens)
    la.la_paged_append(k, v, *small, near.to(dev), zero, lens=lens)
    for x, y in zip(large, small):
        assert torch.equal(x[used].view(torch.uint8), y.view(torch.uint8))
    rows = la.la_paged_read(*large, far.to(dev), lens, N), la.la_paged_read(*small, near.to(dev), lens, N)
    for x, y, given in zip(*rows, (k, v)):
        assert torch.equal(x, y)
        for b, n in enumerate((N, N - 7)):
            if bits:  # half a step of a fifteenth of the spread, the scale's rounding for 15 codes, and the row's own
                want = given[b, :, :n].float()
                groups = want.unflatten(-1, (2, 64))
                spread = (groups.amax(-1) - groups.amin(-1)).repeat_interleave(64, -1)
                off = spread * (0.5 / 15 * (1 + 2.0 ** -8) + 2.0 ** -8)
                assert torch.all((x[b, :, :n].float() - want).abs() <= off + (want.abs() + off) * 2.0 ** -8)
            else:
                assert torch.equal(x[b, :, :n], given[b, :, :n])
            assert not x[b, :, n:].any()
    assert la.la_device_status() == la.LA_OK
