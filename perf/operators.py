"""The operators around the recurrences that a hybrid model's other layers need, as cases to measure.

Three operators, each for prompts and for single tokens:

  conv   the short causal depthwise convolution with its optional SiLU, in front of q, k, v of a gated-delta-rule
         layer or of a state space scan (``la_conv_prefill``, ``la_conv_decode_step``)
  ssm    the selective state space scan, h_t = exp(dt A) h_{t-1} + dt u B_t, y = (C_t h_t + D u) silu(z)
         (``la_ssm_prefill``, ``la_ssm_decode_step``)
  swa    softmax attention over a window or a whole prompt with capped scores, a distance bias and one key
         interval per query, which expresses documents, prefixes and rows that see nothing
         (``la_swa_prefill``, ``la_swa_biased_decode_step``)

``own`` selects the library's calls; otherwise ``run`` computes the same in elementary torch operations in fp32.
Rows behind a sequence's length are left as they were in both (the output buffers of ``prepare`` hold zeros there).
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------------------ the cases


def listed():
    return [
        # q, k or v of a gated-delta-rule layer (16 heads x 128) in front of its prefill: 4 x 16384 tokens
        {"name": "conv_prompt", "op": "conv", "B": 4, "N": 16384, "C": 2048, "W": 4, "dtype": "bf16", "silu": True,
         "bias": False, "ragged": 0, "state": False},
        # a padded fp32 batch that goes on from earlier tokens, 3 taps, lengths down to none
        {"name": "conv_ragged_fp32", "op": "conv", "B": 5, "N": 1001, "C": 520, "W": 3, "dtype": "fp32", "silu": False,
         "bias": True, "ragged": 250, "state": True},
        # one token of each of 256 sequences
        {"name": "conv_step", "op": "conv_step", "S": 256, "C": 2048, "W": 4, "dtype": "bf16", "silu": True,
         "bias": True},
        # a short question: latency
        {"name": "ssm_short", "op": "ssm", "B": 1, "N": 77, "C": 2048, "n": 16, "G": 1, "dtype": "bf16", "z": True,
         "ragged": 0, "state": True},
        # a batch of long prompts through one layer
        {"name": "ssm_prompt", "op": "ssm", "B": 4, "N": 16384, "C": 2048, "n": 16, "G": 1, "dtype": "bf16", "z": True,
         "ragged": 0, "state": False},
        # grouped B, C in fp32, an odd number of tokens, ragged lengths
        {"name": "ssm_groups_fp32", "op": "ssm", "B": 3, "N": 777, "C": 496, "n": 24, "G": 2, "dtype": "fp32",
         "z": False, "ragged": 259, "state": True},
        # one token of each of 256 sequences; the states (67 MB read, 67 MB written) exceed L2
        {"name": "ssm_step", "op": "ssm_step", "S": 256, "C": 4096, "n": 16, "G": 1, "dtype": "bf16", "z": True},
        # BASED's window layers on its prefill shape (8 x 16 x 4096, window 64), filling the decode rings
        {"name": "swa_window", "op": "swa", "B": 8, "H": 16, "Hkv": 16, "Nq": 4096, "Nk": 4096, "d": 64, "window": 64,
         "softcap": 0.0, "slopes": False, "doc": 0, "prefix": 0, "ragged": 0, "cache": True, "dtype": "bf16"},
        # whole prompts, grouped heads, capped scores
        {"name": "swa_capped", "op": "swa", "B": 2, "H": 16, "Hkv": 4, "Nq": 8192, "Nk": 8192, "d": 128, "window": 0,
         "softcap": 30.0, "slopes": False, "doc": 0, "prefix": 0, "ragged": 0, "cache": False, "dtype": "bf16"},
        # packed documents with bidirectional prefixes, a distance bias, rows that see nothing, odd sizes
        {"name": "swa_documents", "op": "swa", "B": 2, "H": 8, "Hkv": 2, "Nq": 4099, "Nk": 4099, "d": 96, "window": 1024,
         "softcap": 0.0, "slopes": True, "doc": 700, "prefix": 90, "ragged": 500, "cache": False, "dtype": "bf16"},
        # the last part of a prompt against all of it, fp32
        {"name": "swa_continued_fp32", "op": "swa", "B": 1, "H": 6, "Hkv": 3, "Nq": 133, "Nk": 333, "d": 40,
         "window": 200, "softcap": 20.0, "slopes": True, "doc": 0, "prefix": 0, "ragged": 0, "cache": True,
         "dtype": "fp32"},
        # one token of each of 256 sequences over 256-token rings, grouped heads, capped and biased scores
        {"name": "swa_step", "op": "swa_step", "S": 256, "H": 16, "Hkv": 4, "d": 128, "window": 256, "softcap": 30.0,
         "slopes": True, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "ssm", "ssm", "ssm_step", "swa", "swa", "swa_step"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op == "conv":
        C = 8 * _log(rng, 1, 1024)
        B = rng.randint(1, 8)
        N = _log(rng, 1, min(32768, (1 << 26) // (B * C)))
        return {"op": op, "B": B, "N": N, "C": C, "W": rng.randint(2, 4), "dtype": dtype, "silu": flag(), "bias": flag(),
                "ragged": rng.choice([0, N // 3]), "state": flag()}
    if op == "conv_step":
        return {"op": op, "S": _log(rng, 1, 512), "C": 8 * _log(rng, 8, 1024), "W": rng.randint(2, 4), "dtype": dtype,
                "silu": flag(), "bias": flag()}
    if op in ("ssm", "ssm_step"):
        n = rng.choice([4, 8, 16, 16, 16, 24, 32, 64])
        G = rng.choice([1, 1, 2, 4])
        C = 8 * G * _log(rng, 2, 1024 // G)
        if op == "ssm_step":
            S = _log(rng, 1, min(512, (1 << 24) // (C * n)))
            return {"op": op, "S": S, "C": C, "n": n, "G": G, "dtype": dtype, "z": flag()}
        B = rng.randint(1, 4)
        N = _log(rng, 1, min(65536, (1 << 30) // (B * C * n)))
        return {"op": op, "B": B, "N": N, "C": C, "n": n, "G": G, "dtype": dtype, "z": flag(),
                "ragged": rng.choice([0, N // 3]), "state": flag()}
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 3, 4, 8])
    d = 8 * rng.randint(4, 16)
    softcap = rng.choice([0.0, 0.0, 20.0, 50.0])
    if op == "swa_step":
        window = _log(rng, 16, 256)
        S = _log(rng, 1, min(512, (1 << 28) // (Hkv * window * d * 4)))
        return {"op": op, "S": S, "H": H, "Hkv": Hkv, "d": d, "window": window, "softcap": softcap, "slopes": flag(),
                "dtype": dtype}
    B = rng.randint(1, 4)
    pairs = (1 << 30) if dtype == "bf16" else (1 << 27)
    Nq = _log(rng, 1, int(math.sqrt(pairs // (B * H))))
    Nk = Nq if flag() else Nq + rng.randint(0, max(1, Nq // 2))
    window = rng.choice([0, 0, _log(rng, 16, 256), _log(rng, 16, 4096)])
    docs = flag() and Nq == Nk
    return {"op": op, "B": B, "H": H, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "d": d, "window": window, "softcap": softcap,
            "slopes": flag(), "doc": _log(rng, 16, 2048) if docs else 0, "prefix": rng.choice([0, 40]) if docs else 0,
            "ragged": rng.choice([0, Nk // 5]) if Nq == Nk else 0, "cache": 0 < window <= 256, "dtype": dtype}


# ------------------------------------------------------------------------------------------------ inputs


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lens(case, N):
    """Tokens of each sequence of a padded batch, or None where all are full."""
    if not case["ragged"]:
        return None
    return [max(0, N - b * case["ragged"]) for b in range(case["B"])]


def _spans(case):
    """(lo, hi) int64 [B, Nq]: the keys that each query sees, everything that masks it taken together; and the two
    arrays that a call gets (documents, prefixes and separators), None where there are none."""
    B, Nq, Nk = case["B"], case["Nq"], case["Nk"]
    pos = np.arange(Nk - Nq, Nk, dtype=np.int64)
    lens = np.array(_lens(case, Nk) or [Nk] * B, dtype=np.int64)
    key_lo = key_hi = None
    if case["doc"]:
        cuts = [0]  # documents of 1/2, 1 and 3/2 times the stated length in turn
        while cuts[-1] < Nk:
            cuts.append(min(Nk, cuts[-1] + max(1, case["doc"] * (1 + (len(cuts) - 1) % 3) // 2)))
        cuts = np.array(cuts, dtype=np.int64)
        k = np.searchsorted(cuts, pos, side="right") - 1
        lo1 = cuts[k]
        hi1 = np.maximum(pos + 1, np.minimum(lo1 + case["prefix"], cuts[k + 1]))
        hi1 = np.where(pos % 97 == 96, lo1, hi1)  # separators see nothing
        key_lo, key_hi = np.tile(lo1, (B, 1)), np.tile(hi1, (B, 1))
    lo = key_lo if key_lo is not None else np.zeros((B, Nq), dtype=np.int64)
    if case["window"]:
        lo = np.maximum(lo, pos - case["window"] + 1)
    hi = key_hi if key_hi is not None else np.tile(pos + 1, (B, 1))
    hi = np.minimum(hi, lens[:, None])
    hi = np.where(pos < lens[:, None], hi, 0)
    return np.maximum(lo, 0), hi, key_lo, key_hi


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, dev, op = _dtype(case), "cuda", case["op"]

    def randn(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=dev)

    st = {"case": case}
    if op in ("conv", "conv_step"):
        C, W = case["C"], case["W"]
        st["w"] = randn(C, W, scale=W ** -0.5)
        st["bias"] = randn(C, scale=0.1) if case["bias"] else None
        if op == "conv":
            B, N = case["B"], case["N"]
            st["x"] = randn(B, N, C)
            st["state"] = randn(B, W - 1, C) if case["state"] else None
            lens = _lens(case, N)
            st["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int64, device=dev)
            st["y"] = torch.zeros((B, N, C), dtype=dt, device=dev)
        else:
            st["x"] = randn(case["S"], C)
            st["state"] = randn(case["S"], W - 1, C)
            st["state_out"] = torch.empty_like(st["state"])
        return st
    if op in ("ssm", "ssm_step"):
        C, n, G = case["C"], case["n"], case["G"]
        # A = -(1..n) spread by a factor, steps around softplus(bias) in 0.001 .. 0.1: the usual ranges at use
        st["A"] = -(torch.arange(1, n + 1, device=dev, dtype=torch.float32) * torch.exp(0.3 * randn(C, n, dtype=torch.float32)))
        st["A"] = st["A"].contiguous()
        step0 = torch.exp(rand(C) * math.log(100.0) + math.log(0.001))
        st["dt_bias"] = (step0 + torch.log(-torch.expm1(-step0))).contiguous()
        st["D"] = 1 + randn(C, scale=0.1, dtype=torch.float32)
        if op == "ssm":
            B, N = case["B"], case["N"]
            st["u"], st["delta"] = randn(B, N, C), randn(B, N, C, scale=0.5)
            st["z"] = randn(B, N, C) if case["z"] else None
            bc = randn(B, N, 2, G, n)  # one projection's output: B and C are views of it
            st["Bm"], st["Cm"] = bc[:, :, 0].transpose(1, 2), bc[:, :, 1].transpose(1, 2)  # [B, G, N, n]
            st["h"] = randn(B, C, n, dtype=torch.float32) if case["state"] else None
            lens = _lens(case, N)
            st["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int64, device=dev)
            st["y"] = torch.zeros((B, N, C), dtype=dt, device=dev)
        else:
            S = case["S"]
            st["u"], st["delta"] = randn(S, C), randn(S, C, scale=0.5)
            st["z"] = randn(S, C) if case["z"] else None
            bc = randn(S, 2, G, n)
            st["Bm"], st["Cm"] = bc[:, 0], bc[:, 1]
            st["h"] = randn(S, C, n, dtype=torch.float32)
            st["h_out"] = torch.empty_like(st["h"])
        return st
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    st["scale"] = d ** -0.5
    st["slopes"] = (torch.exp2(-8.0 * torch.arange(1, H + 1, device=dev, dtype=torch.float32) / H)
                    if case["slopes"] else None)
    if op == "swa_step":
        S, w = case["S"], case["window"]
        st["q"], st["k"], st["v"] = randn(S, H, d, scale=1.5), randn(S, Hkv, d, scale=1.5), randn(S, Hkv, d)
        st["k_cache"], st["v_cache"] = randn(S, Hkv, w, d, scale=1.5), randn(S, Hkv, w, d)
        # most rings are full, some sequences are new
        st["pos"] = torch.randint(0, 4 * w, (S,), generator=g, device=dev)
        return st
    B, Nq, Nk = case["B"], case["Nq"], case["Nk"]
    # token-major projections [B, N, H, d], as a layer makes them, seen as [B, H, N, d]
    st["q"] = randn(B, Nq, H, d, scale=1.5).transpose(1, 2)
    st["k"] = randn(B, Nk, Hkv, d, scale=1.5).transpose(1, 2)
    st["v"] = randn(B, Nk, Hkv, d).transpose(1, 2)
    lens = _lens(case, Nk)
    st["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int64, device=dev)
    _, _, lo, hi = _spans(case)
    st["key_lo"] = None if lo is None else torch.from_numpy(lo.astype(np.int32)).to(dev)
    st["key_hi"] = None if hi is None else torch.from_numpy(hi.astype(np.int32)).to(dev)
    st["o"] = torch.zeros((B, Nq, H, d), dtype=dt, device=dev).transpose(1, 2)
    w = case["window"]
    st["k_cache"] = torch.zeros((B, Hkv, w, d), dtype=dt, device=dev) if case["cache"] else None
    st["v_cache"] = torch.zeros((B, Hkv, w, d), dtype=dt, device=dev) if case["cache"] else None
    return st


# ------------------------------------------------------------------------------------------------ one pass


def _alive(lens, B, N, dev):
    """[B, N, 1] truth values: the token is one of its sequence's."""
    t = torch.arange(N, device=dev)
    return (t[None, :] < lens[:, None])[..., None] if lens is not None else torch.ones((B, N, 1), dtype=torch.bool, device=dev)


def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _plain_conv(st, c):
    x = st["x"].float()
    B, N, C = x.shape
    W = c["W"]
    prev = st["state"].float() if st["state"] is not None else torch.zeros((B, W - 1, C), device=x.device)
    xx = torch.cat([prev, x], 1)
    y = (xx.unfold(1, W, 1) * st["w"].float()).sum(-1)
    if st["bias"] is not None:
        y = y + st["bias"].float()
    if c["silu"]:
        y = _silu(y)
    y = torch.where(_alive(st["lens"], B, N, x.device), y, torch.zeros_like(y))
    at = (st["lens"] if st["lens"] is not None else torch.full((B,), N, device=x.device))[:, None] + torch.arange(W - 1, device=x.device)
    last = torch.gather(xx, 1, at[..., None].expand(B, W - 1, C))
    return {"y": y.to(st["x"].dtype), "state": last.to(st["x"].dtype)}


def _plain_conv_step(st, c):
    xx = torch.cat([st["state"].float(), st["x"].float()[:, None]], 1)  # [S, W, C]
    y = (xx * st["w"].float().t()).sum(1)
    if st["bias"] is not None:
        y = y + st["bias"].float()
    if c["silu"]:
        y = _silu(y)
    return {"y": y.to(st["x"].dtype), "state": xx[:, 1:].to(st["x"].dtype)}


def _plain_ssm(st, c):
    """The recurrence by doubling: after pass p every token holds the map of the 2^p tokens that end at it."""
    u = st["u"].float()
    B, N, C = u.shape
    G, n = c["G"], c["n"]
    dt = _softplus(st["delta"].float() + st["dt_bias"])
    dt = torch.where(_alive(st["lens"], B, N, u.device), dt, torch.zeros_like(dt))  # a padded token changes nothing
    Bt = st["Bm"].float().transpose(1, 2)  # [B, N, G, n]
    Ct = st["Cm"].float().transpose(1, 2)
    a = torch.exp(dt[..., None] * st["A"])  # [B, N, C, n]
    h = ((dt * u).view(B, N, G, C // G, 1) * Bt[:, :, :, None]).view(B, N, C, n)
    if st["h"] is not None:
        h[:, 0] += a[:, 0] * st["h"]
    span = 1
    while span < N:
        h[:, span:] += a[:, span:] * h[:, :-span].clone()
        if 2 * span < N:
            a[:, span:] *= a[:, :-span].clone()
        span *= 2
    y = (h.view(B, N, G, C // G, n) * Ct[:, :, :, None]).sum(-1).view(B, N, C) + st["D"] * u
    if st["z"] is not None:
        y = y * _silu(st["z"].float())
    y = torch.where(_alive(st["lens"], B, N, u.device), y, torch.zeros_like(y))
    return {"y": y.to(st["u"].dtype), "h": h[:, -1].contiguous()}


def _plain_ssm_step(st, c):
    u = st["u"].float()
    S, C = u.shape
    G, n = c["G"], c["n"]
    dt = _softplus(st["delta"].float() + st["dt_bias"])
    Bt = st["Bm"].float()[:, :, None].expand(S, G, C // G, n).reshape(S, C, n)
    Ct = st["Cm"].float()[:, :, None].expand(S, G, C // G, n).reshape(S, C, n)
    h = torch.exp(dt[..., None] * st["A"]) * st["h"] + (dt * u)[..., None] * Bt
    y = (h * Ct).sum(-1) + st["D"] * u
    if st["z"] is not None:
        y = y * _silu(st["z"].float())
    return {"y": y.to(st["u"].dtype), "h": h}


def _plain_softmax(s, seen, v):
    """softmax over the seen keys times v; rows that see nothing give zeros."""
    s = s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = s.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    return torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_swa(st, c):
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    B, H, Nq, d = q.shape
    Nk, group = k.shape[2], H // c["Hkv"]
    dev = q.device
    j = torch.arange(Nk, device=dev)
    p = torch.arange(Nk - Nq, Nk, device=dev)
    lens = st["lens"] if st["lens"] is not None else torch.full((B,), Nk, device=dev)
    lo = st["key_lo"].long() if st["key_lo"] is not None else torch.zeros((B, Nq), dtype=torch.long, device=dev)
    hi = st["key_hi"].long() if st["key_hi"] is not None else (p + 1).expand(B, Nq)
    seen = (j >= lo[..., None]) & (j < hi[..., None]) & (j < lens[:, None, None]) & (p[:, None] < lens[:, None, None])
    if c["window"]:
        seen = seen & (p[:, None] - j < c["window"])
    s = torch.matmul(q, k.repeat_interleave(group, 1).transpose(2, 3)) * st["scale"]
    if c["softcap"]:
        s = s.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    if st["slopes"] is not None:
        s = s.sub_(st["slopes"][:, None, None] * (p[:, None] - j).abs())
    out = {"o": _plain_softmax(s, seen[:, None], v.repeat_interleave(group, 1)).to(st["q"].dtype)}
    if c["cache"]:
        w = c["window"]
        slot = torch.arange(w, device=dev)
        at = lens[:, None] - 1 - (lens[:, None] - 1 - slot) % w  # the newest token of each slot
        held = (at >= 0)[:, None, :, None]
        idx = at.clamp(min=0)[:, None, :, None].expand(B, c["Hkv"], w, d)
        out["k_cache"] = torch.where(held, torch.gather(st["k"], 2, idx), torch.zeros_like(st["k_cache"]))
        out["v_cache"] = torch.where(held, torch.gather(st["v"], 2, idx), torch.zeros_like(st["v_cache"]))
    return out


def _plain_swa_step(st, c):
    S, H, d = st["q"].shape
    w, group = c["window"], H // c["Hkv"]
    dev, pos = st["q"].device, st["pos"]
    slot = torch.arange(w, device=dev)
    new = (slot == (pos % w)[:, None])[:, None, :, None]
    kc = torch.where(new, st["k"][:, :, None], st["k_cache"])
    vc = torch.where(new, st["v"][:, :, None], st["v_cache"])
    age = (pos[:, None] - slot) % w  # how long ago the slot's token came
    seen = (age <= pos[:, None])[:, None, None]
    s = torch.matmul(st["q"].float().view(S, c["Hkv"], group, d), kc.float().transpose(2, 3)) * st["scale"]
    if c["softcap"]:
        s = s.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    if st["slopes"] is not None:
        s = s - st["slopes"].view(c["Hkv"], group, 1) * age[:, None, None]
    o = _plain_softmax(s, seen, vc.float())
    return {"o": o.view(S, H, d).to(st["q"].dtype), "k_cache": kc, "v_cache": vc}


def _own_run(st, c):
    import linear_attention_recurrence_chunked_gb300 as la
    op = c["op"]
    if op == "conv":
        y, state = la.la_conv_prefill(st["x"], st["w"], bias=st["bias"], state_in=st["state"], lens=st["lens"],
                                      silu=c["silu"], y=st["y"])
        return {"y": y, "state": state}
    if op == "conv_step":
        y = la.la_conv_decode_step(st["x"], st["w"], st["state"], bias=st["bias"], silu=c["silu"],
                                   state_out=st["state_out"])
        return {"y": y, "state": st["state_out"]}
    if op == "ssm":
        y, h = la.la_ssm_prefill(st["u"], st["delta"], st["A"], st["Bm"], st["Cm"], D=st["D"], z=st["z"],
                                 delta_bias=st["dt_bias"], delta_softplus=True, h_in=st["h"], lens=st["lens"],
                                 y=st["y"])
        return {"y": y, "h": h}
    if op == "ssm_step":
        y = la.la_ssm_decode_step(st["u"], st["delta"], st["A"], st["Bm"], st["Cm"], st["h"], D=st["D"], z=st["z"],
                                  delta_bias=st["dt_bias"], delta_softplus=True, state_out=st["h_out"])
        return {"y": y, "h": st["h_out"]}
    if op == "swa":
        o = la.la_swa_prefill(st["q"], st["k"], st["v"], window=c["window"], scale=st["scale"], softcap=c["softcap"],
                              slopes=st["slopes"], key_lo=st["key_lo"], key_hi=st["key_hi"], lens=st["lens"],
                              o=st["o"], k_cache=st["k_cache"], v_cache=st["v_cache"])
        return {"o": o, "k_cache": st["k_cache"], "v_cache": st["v_cache"]} if c["cache"] else {"o": o}
    o = la.la_swa_biased_decode_step(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["pos"],
                                     scale=st["scale"], softcap=c["softcap"], slopes=st["slopes"])
    return {"o": o, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def run(state):
    c = state["case"]
    if own:
        return _own_run(state, c)
    return {"conv": _plain_conv, "conv_step": _plain_conv_step, "ssm": _plain_ssm, "ssm_step": _plain_ssm_step,
            "swa": _plain_swa, "swa_step": _plain_swa_step}[c["op"]](state, c)


# ------------------------------------------------------------------------------------------------ work


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("conv", "conv_step"):
        C, W = case["C"], case["W"]
        if op == "conv":
            tokens = sum(_lens(case, case["N"]) or [case["N"]] * case["B"])
            states = case["B"] * (2 if case["state"] else 1)
        else:
            tokens, states = case["S"], 2 * case["S"]
        return {"bytes": e * C * (2 * tokens + states * (W - 1) + W + case["bias"]), "flops": tokens * C * (2 * W + 4 * case["silu"])}
    if op in ("ssm", "ssm_step"):
        C, n, G = case["C"], case["n"], case["G"]
        if op == "ssm":
            tokens = sum(_lens(case, case["N"]) or [case["N"]] * case["B"])
            states = case["B"] * (2 if case["state"] else 1)
        else:
            tokens, states = case["S"], 2 * case["S"]
        rows = 3 + case["z"]  # u, delta, y and z
        # an exponential, its argument, dt u B, the update and the readout per state; the gates per channel
        return {"bytes": e * tokens * (rows * C + 2 * G * n) + 4 * (states * C * n + C * n + 2 * C),
                "flops": tokens * C * (7 * n + 8)}
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    extra = 1 + 3 * bool(case["softcap"]) + 2 * case["slopes"]  # per score: the exponential, the cap, the bias
    if op == "swa_step":
        S, w = case["S"], case["window"]
        return {"bytes": e * S * (2 * H * d + 2 * Hkv * d * (w + 2)), "flops": S * H * w * (4 * d + extra)}
    lo, hi, _, _ = _spans(case)
    pairs = int(np.maximum(hi - lo, 0).sum()) * H
    lens = _lens(case, case["Nk"]) or [case["Nk"]] * case["B"]
    keys, rows = sum(lens), sum(max(0, n - (case["Nk"] - case["Nq"])) for n in lens)
    ring = 2 * sum(min(n, case["window"]) for n in lens) * Hkv * d if case["cache"] else 0
    return {"bytes": e * (2 * rows * H * d + 2 * keys * Hkv * d + ring) + (8 * rows if case["doc"] else 0),
            "flops": pairs * (4 * d + extra)}


# ------------------------------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    """The definitions in fp64, token by token or row block by row block."""
    st = prepare(case, seed)
    op, f = case["op"], torch.float64
    sig = lambda t: torch.sigmoid(t)  # noqa: E731
    if op == "conv":
        B, N, C, W = case["B"], case["N"], case["C"], case["W"]
        y = torch.zeros((B, N, C), dtype=f, device="cuda")
        state = torch.zeros((B, W - 1, C), dtype=f, device="cuda")
        for b in range(B):
            n = N if st["lens"] is None else int(st["lens"][b])
            head = st["state"][b].to(f) if st["state"] is not None else torch.zeros((W - 1, C), dtype=f, device="cuda")
            seq = torch.cat([head, st["x"][b, :n].to(f)])
            acc = torch.zeros((n, C), dtype=f, device="cuda")
            for i in range(W):
                acc += seq[i:i + n] * st["w"][:, i].to(f)
            if st["bias"] is not None:
                acc += st["bias"].to(f)
            y[b, :n] = acc * sig(acc) if case["silu"] else acc
            state[b] = seq[n:]
        return {"y": y, "state": state}
    if op == "conv_step":
        acc = st["x"].to(f) * st["w"][:, -1].to(f)
        for i in range(case["W"] - 1):
            acc += st["state"][:, i].to(f) * st["w"][:, i].to(f)
        if st["bias"] is not None:
            acc += st["bias"].to(f)
        new = torch.cat([st["state"][:, 1:], st["x"][:, None]], 1).to(f)
        return {"y": acc * sig(acc) if case["silu"] else acc, "state": new}
    if op in ("ssm", "ssm_step"):
        C, n, G = case["C"], case["n"], case["G"]
        u, delta = st["u"].to(f), st["delta"].to(f)
        Bm, Cm = st["Bm"].to(f), st["Cm"].to(f)
        if op == "ssm_step":
            u, delta, Bm, Cm = u[:, None], delta[:, None], Bm[:, :, None], Cm[:, :, None]
        R, N = u.shape[:2]
        dt = torch.logaddexp(delta + st["dt_bias"].to(f), torch.zeros((), dtype=f, device="cuda"))
        A = st["A"].to(f)
        h = st["h"].to(f) if st["h"] is not None else torch.zeros((R, C, n), dtype=f, device="cuda")
        y = torch.zeros((R, N, C), dtype=f, device="cuda")
        lens = st.get("lens")
        of = torch.arange(C, device="cuda") // (C // G)
        for t in range(N):
            new = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * u[:, t])[..., None] * Bm[:, of, t]
            out = torch.einsum("rcn,rcn->rc", new, Cm[:, of, t])
            if lens is None:
                h, y[:, t] = new, out
            else:
                on = lens > t
                h = torch.where(on[:, None, None], new, h)
                y[:, t] = torch.where(on[:, None], out, torch.zeros_like(out))
        full = y + st["D"].to(f) * u
        if st["z"] is not None:
            z = st["z"].to(f).view(full.shape)
            full = full * z * sig(z)
        if lens is not None:
            full = full * (torch.arange(N, device="cuda")[None, :] < lens[:, None])[..., None]
        return {"y": full[:, 0] if op == "ssm_step" else full, "h": h}
    H, Hkv, d, w = case["H"], case["Hkv"], case["d"], case["window"]
    slopes = st["slopes"].to(f) if st["slopes"] is not None else None

    def attend(q, k, v, seen, dist, head):
        s = q.to(f) @ k.to(f).T * st["scale"]
        if case["softcap"]:
            s = case["softcap"] * torch.tanh(s / case["softcap"])
        if slopes is not None:
            s = s - slopes[head] * dist.abs()
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
        p = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)
        return p @ v.to(f)

    if op == "swa_step":
        S, pos = case["S"], st["pos"].tolist()
        o = torch.zeros((S, H, d), dtype=f, device="cuda")
        kc, vc = st["k_cache"].clone(), st["v_cache"].clone()
        if S * H > 8192:
            return None
        for s in range(S):
            kc[s, :, pos[s] % w], vc[s, :, pos[s] % w] = st["k"][s], st["v"][s]
            first = max(0, pos[s] - w + 1)
            tok = torch.arange(first, pos[s] + 1, device="cuda")
            every = torch.ones((1, len(tok)), dtype=torch.bool, device="cuda")
            for h in range(H):
                kv = h // (H // Hkv)
                o[s, h] = attend(st["q"][s, h][None], kc[s, kv, tok % w], vc[s, kv, tok % w], every,
                                 (pos[s] - tok)[None].to(f), h)[0]
        return {"o": o, "k_cache": kc.to(f), "v_cache": vc.to(f)}
    B, Nq, Nk = case["B"], case["Nq"], case["Nk"]
    lo, hi, _, _ = _spans(case)
    lo, hi = torch.from_numpy(lo).cuda(), torch.from_numpy(hi).cuda()
    o = torch.zeros((B, H, Nq, d), dtype=f, device="cuda")
    for b in range(B):
        for r in range(0, Nq, 2048):
            e = min(Nq, r + 2048)
            first, last = int(lo[b, r:e].min()), int(hi[b, r:e].max())
            if last <= first:
                continue
            j = torch.arange(first, last, device="cuda")
            p = torch.arange(Nk - Nq + r, Nk - Nq + e, device="cuda")
            seen = (j >= lo[b, r:e, None]) & (j < hi[b, r:e, None])
            dist = (p[:, None] - j).to(f)
            for h in range(H):
                kv = h // (H // Hkv)
                o[b, h, r:e] = attend(st["q"][b, h, r:e], st["k"][b, kv, first:last], st["v"][b, kv, first:last], seen, dist, h)
    out = {"o": o}
    if case["cache"]:
        out["k_cache"] = torch.zeros((B, Hkv, w, d), dtype=f, device="cuda")
        out["v_cache"] = torch.zeros((B, Hkv, w, d), dtype=f, device="cuda")
        for b in range(B):
            n = Nk if st["lens"] is None else int(st["lens"][b])
            tok = torch.arange(max(0, n - w), n, device="cuda")
            out["k_cache"][b, :, tok % w] = st["k"][b][:, tok].to(f)
            out["v_cache"][b, :, tok % w] = st["v"][b][:, tok].to(f)
    return out
