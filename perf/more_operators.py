"""What a hybrid model's full attention layers need beside the recurrences, as cases to measure.

Three operators, each for prompts and for single tokens:

  qk      norms of queries and keys for each head with the position rotation in the same pass: root mean square with
          weights in front of attention, unit length in front of the gated delta rule (``la_qk_norm_rope``)
  append  keys and values of new tokens into a paged cache, the keys rotated on the way, in the model's type or in
          4 bits (``la_paged_append``), and the cache read back as the values it stands for (``la_paged_read``), as a
          prompt's next chunk needs it
  step    attention of one token of each sequence over a paged cache, in the model's type or in 4 bits, with grouped
          heads, windows, capped scores and a distance bias (``la_paged_decode_step``)

A page holds ``page`` tokens of every key head; ``table[b, i]`` is the page of tokens i page .. (i + 1) page - 1 of
sequence b, and entries that no token needs are -1.  In 4 bits, 64 neighbouring elements of a row share a bf16 scale and
a bf16 offset: element = offset + scale code, offset = the least of the 64, scale = a fifteenth of their spread.

``own`` selects the library's calls; otherwise ``run`` computes the same in elementary torch operations in fp32.
"""
import math

import torch

own = False


# ------------------------------------------------------------------------------------------------ the cases


def listed():
    return [
        # the 16 heads x 128 of a gated-delta-rule layer's queries and keys to unit length, 4 prompts of 16384
        {"name": "qk_unit_prompt", "op": "qk", "B": 4, "N": 16384, "H": 16, "Hkv": 16, "d": 128, "norm": "l2", "rot": 0,
         "interleaved": False, "dtype": "bf16", "ragged": 0, "weights": False, "packed": False},
        # grouped heads of an attention layer over prompts of a length that nothing divides
        {"name": "qk_rope_prompt", "op": "qk", "B": 3, "N": 8191, "H": 32, "Hkv": 4, "d": 128, "norm": "rms", "rot": 128,
         "interleaved": False, "dtype": "bf16", "ragged": 0, "weights": True, "packed": False},
        # a padded fp32 batch of packed documents (positions start anew), neighbours rotated, a third of the width
        {"name": "qk_ragged_fp32", "op": "qk", "B": 5, "N": 1001, "H": 6, "Hkv": 2, "d": 96, "norm": "rms", "rot": 32,
         "interleaved": True, "dtype": "fp32", "ragged": 250, "weights": True, "packed": True},
        # one token of each of 256 sequences
        {"name": "qk_step", "op": "qk", "B": 256, "N": 1, "H": 32, "Hkv": 4, "d": 128, "norm": "rms", "rot": 64,
         "interleaved": False, "dtype": "bf16", "ragged": 0, "weights": True, "packed": False},
        # eight padded prompts into empty pages
        {"name": "append_prompt", "op": "append", "B": 8, "N": 4096, "Hkv": 4, "d": 128, "page": 64, "seen": 0, "rot": 128,
         "interleaved": False, "dtype": "bf16", "ragged": 301, "bits": 0},
        # one token of each of 256 sequences: latency
        {"name": "append_step", "op": "append", "B": 256, "N": 1, "Hkv": 4, "d": 128, "page": 64, "seen": 400, "rot": 128,
         "interleaved": False, "dtype": "bf16", "ragged": 0, "bits": 0},
        # a prompt's next chunk into 4 bits, and the whole context read back for the chunk's attention
        {"name": "append_chunk_4bit", "op": "append", "B": 4, "N": 2048, "Hkv": 8, "d": 128, "page": 32, "seen": 14000,
         "rot": 64, "interleaved": False, "dtype": "bf16", "ragged": 0, "bits": 4},
        # 256 sequences of mixed lengths, the usual batch of a server
        {"name": "step_batch", "op": "step", "S": 256, "L": 8192, "H": 32, "Hkv": 4, "d": 128, "page": 64, "window": 0,
         "softcap": 0.0, "slopes": False, "dtype": "bf16", "bits": 0, "short": False},
        # a few sequences of 256K tokens: the key axis has to be split
        {"name": "step_long", "op": "step", "S": 2, "L": 262144, "H": 32, "Hkv": 4, "d": 128, "page": 64, "window": 0,
         "softcap": 0.0, "slopes": False, "dtype": "bf16", "bits": 0, "short": False},
        # five sequences, one of them empty and one of a single token, fp32, capped and biased scores in a window: latency
        {"name": "step_small_fp32", "op": "step", "S": 5, "L": 700, "H": 6, "Hkv": 2, "d": 40, "page": 16, "window": 333,
         "softcap": 20.0, "slopes": True, "dtype": "fp32", "bits": 0, "short": True},
        # the server's batch over a cache held in 4 bits
        {"name": "step_batch_4bit", "op": "step", "S": 256, "L": 16384, "H": 32, "Hkv": 4, "d": 128, "page": 64,
         "window": 0, "softcap": 0.0, "slopes": False, "dtype": "bf16", "bits": 4, "short": False},
        # long contexts in 4 bits, capped scores, half the width
        {"name": "step_long_4bit", "op": "step", "S": 3, "L": 131071, "H": 16, "Hkv": 8, "d": 64, "page": 128, "window": 0,
         "softcap": 30.0, "slopes": False, "dtype": "bf16", "bits": 4, "short": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["qk", "qk", "append", "append", "step", "step", "step"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "qk":
        H = Hkv * rng.choice([1, 2, 3, 4, 8])
        d = 8 * rng.randint(4, 32)
        rot = 16 * rng.randint(0, d // 16)
        B = rng.choice([1, 2, 3, 5, 8, _log(rng, 1, 512)])
        N = 1 if B > 8 else _log(rng, 1, min(32768, (1 << 27) // (B * (H + Hkv) * d)))
        norm = rng.choice(["rms", "rms", "l2", "none"] if rot else ["rms", "l2"])
        return {"op": op, "B": B, "N": N, "H": H, "Hkv": Hkv, "d": d, "norm": norm, "rot": rot, "interleaved": flag(),
                "dtype": dtype, "ragged": rng.choice([0, N // 3]), "weights": norm != "none" and flag(), "packed": flag()}
    page = rng.choice([16, 32, 48, 64, 128, 256])
    bits = rng.choice([0, 4])
    d = rng.choice([64, 128]) if bits else 8 * rng.randint(4, 16)
    dtype = "bf16" if bits else dtype
    if op == "append":
        B = rng.choice([1, 2, 3, 5, 8, _log(rng, 1, 512)])
        N = 1 if B > 8 else _log(rng, 1, min(16384, (1 << 25) // (B * Hkv * d)))
        seen = rng.choice([0, _log(rng, 1, min(16384, (1 << 26) // (B * Hkv * d)))])
        return {"op": op, "B": B, "N": N, "Hkv": Hkv, "d": d, "page": page, "seen": seen, "rot": 16 * rng.randint(0, d // 16),
                "interleaved": flag(), "dtype": dtype, "ragged": rng.choice([0, N // 3]), "bits": bits}
    H = Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    S = _log(rng, 1, 512)
    L = _log(rng, 1, min(131072, (1 << 28) // (S * Hkv * d)))
    return {"op": op, "S": S, "L": L, "H": H, "Hkv": Hkv, "d": d, "page": page, "window": rng.choice([0, 0, _log(rng, 1, 8192)]),
            "softcap": rng.choice([0.0, 0.0, 20.0, 50.0]), "slopes": rng.random() < 0.3, "dtype": dtype, "bits": bits,
            "short": S >= 2 and flag()}


# ------------------------------------------------------------------------------------------------ inputs


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _new_tokens(case):
    """Tokens of each sequence of a padded batch."""
    if case["B"] > 8:
        return [case["N"]] * case["B"]
    return [max(0, case["N"] - b * case["ragged"]) for b in range(case["B"])]


def _lengths(case):
    """Tokens of each cached sequence: a quarter to the whole of L, one of them L, spread evenly in no order."""
    S, L = case["S"], case["L"]
    lens = [max(1, round(L * (1 - 0.75 * ((s * 0.6180339887498949) % 1.0)))) for s in range(S)]
    if case["short"]:
        lens[-1] = 0
        if S > 2:
            lens[-2] = 1
    return lens


def _seen(case):
    """Tokens in the cache before the append: half of `seen` to all of it, in no order."""
    return [round(case["seen"] * (1 - 0.5 * ((b * 0.6180339887498949) % 1.0))) for b in range(case["B"])]


def _angles(rows, rot, dev):
    """cos and sin fp32 [rows, rot / 2] of position x base^(-2 i / rot), the angles in 64 bits."""
    freq = 10000.0 ** (-2.0 * torch.arange(rot // 2, device=dev, dtype=torch.float64) / rot)
    angle = torch.arange(rows, device=dev, dtype=torch.float64)[:, None] * freq
    return torch.cos(angle).float(), torch.sin(angle).float()


def _pages(totals, page, g, dev, spare):
    """A table int32 [B, width] of distinct pages in no order, and the number of pages; -1 where no token needs one."""
    need = [-(-t // page) for t in totals]
    width = max(1, max(need) + spare)
    count = sum(need)
    order = torch.randperm(max(1, count), generator=g, device=dev).to(torch.int32)
    table = torch.full((len(totals), width), -1, dtype=torch.int32, device=dev)
    slot = torch.arange(width, device=dev)[None, :] < torch.tensor(need, device=dev)[:, None]
    table[slot] = order[:count]
    return table, max(1, count)


def _code(x, scale, offset, wide):
    """The codes of bf16 rows [..., d] under the scales and offsets bf16 [..., d / 64], fp32 (64 bits if `wide`)."""
    t = torch.float64 if wide else torch.float32
    y = x.unflatten(-1, (x.shape[-1] // 64, 64)).to(t) - offset[..., None].to(t)
    s = scale[..., None].to(t)
    y = torch.where(s > 0, y / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    return torch.clamp(torch.round(y), 0, 15).to(torch.uint8).reshape(x.shape)


def _quantise(x, wide=False):
    """bf16 rows [..., d] -> (codes uint8 [..., d], scales bf16 [..., d / 64], offsets bf16 [..., d / 64])."""
    t = torch.float64 if wide else torch.float32
    y = x.unflatten(-1, (x.shape[-1] // 64, 64))
    lo, hi = y.amin(-1), y.amax(-1)
    scale = ((hi.to(t) - lo.to(t)) / 15).to(torch.float32).to(torch.bfloat16)
    return _code(x, scale, lo, wide), scale, lo


def _pack(codes, scale, offset):
    """Rows of whole pages [P, Hkv, page, d] in the cache's bytes: the page's codes, then its scales and offsets.  A row's
    32-bit words take eight elements each, of its 64-element halves in turn."""
    P, Hkv, page, d = codes.shape
    w = codes.view(P, Hkv, page, d // 64, 8, 4, 2).transpose(3, 4)
    row = (w[..., 0] | (w[..., 1] << 4)).reshape(P, Hkv, page * d // 2)
    meta = torch.stack([scale, offset], -1).contiguous().view(torch.uint8).reshape(P, Hkv, page * d // 16)
    return torch.cat([row, meta], -1).view(P, Hkv, page, d * 9 // 16)


def _unpack(pages, d):
    """The cache's bytes -> (codes uint8 [P, Hkv, page, d], scales, offsets bf16 [P, Hkv, page, d / 64])."""
    P, Hkv, page, _ = pages.shape
    flat = pages.reshape(P, Hkv, page * d * 9 // 16)
    row = flat[..., :page * d // 2].reshape(P, Hkv, page, 8, d // 64, 4)
    codes = torch.stack([row & 15, row >> 4], -1).transpose(3, 4).reshape(P, Hkv, page, d)
    meta = flat[..., page * d // 2:].contiguous().view(torch.bfloat16).view(P, Hkv, page, d // 64, 2)
    return codes, meta[..., 0], meta[..., 1]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, dev, op = _dtype(case), "cuda", case["op"]

    def randn(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)

    def pool(P, page, scale):
        x = randn(P, case["Hkv"], page, case["d"], scale=scale)
        return _pack(*_quantise(x)) if case["bits"] else x

    st = {"case": case}
    d, Hkv = case["d"], case["Hkv"]
    if op == "qk":
        B, N, H, rot = case["B"], case["N"], case["H"], case["rot"]
        qkv = randn(B, N, H + 2 * Hkv, d)  # one projection's output: q and k are views of it
        st["q"], st["k"] = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hkv].transpose(1, 2)
        st["q_weight"] = 1 + randn(d, scale=0.2, dtype=torch.float32) if case["weights"] else None
        st["k_weight"] = 1 + randn(d, scale=0.2, dtype=torch.float32) if case["weights"] else None
        st["lens"] = torch.tensor(_new_tokens(case), dtype=torch.int64, device=dev) if case["ragged"] and B <= 8 else None
        st["cos"] = st["sin"] = st["pos"] = None
        if rot:
            if case["packed"]:  # documents of 300 tokens
                st["pos"] = (torch.arange(N, device=dev) % 300).expand(B, N).contiguous()
            else:  # prompts and steps that go on from earlier tokens
                st["pos"] = torch.randint(0, 4000, (B,), generator=g, device=dev)
            st["cos"], st["sin"] = _angles(N + 4000, rot, dev)
        return st
    if op == "append":
        B, N, page, rot = case["B"], case["N"], case["page"], case["rot"]
        seen, new = _seen(case), _new_tokens(case)
        kv = randn(B, N, 2, Hkv, d)  # one projection's output
        st["k"], st["v"] = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
        st["seen"] = torch.tensor(seen, dtype=torch.int64, device=dev)
        st["lens"] = torch.tensor(new, dtype=torch.int64, device=dev) if case["ragged"] and B <= 8 else None
        st["total"] = torch.tensor([s + n for s, n in zip(seen, new)], dtype=torch.int64, device=dev)
        st["longest"] = max(s + n for s, n in zip(seen, new))
        st["table"], P = _pages([s + n for s, n in zip(seen, new)], page, g, dev, 3)
        st["k_pages"], st["v_pages"] = pool(P, page, 1.0), pool(P, page, 1.0)
        st["cos"], st["sin"] = _angles(st["longest"] + 1, rot, dev) if rot else (None, None)
        return st
    S, H, page = case["S"], case["H"], case["page"]
    lens = _lengths(case)
    st["q"] = randn(S, H + 2 * Hkv, d, scale=1.5)[:, :H]  # the queries of one projection's output
    st["lens"] = torch.tensor(lens, dtype=torch.int64, device=dev)
    st["table"], P = _pages(lens, page, g, dev, 2)
    st["k_pages"], st["v_pages"] = pool(P, page, 1.5), pool(P, page, 1.0)
    st["scale"] = d ** -0.5
    st["slopes"] = (torch.exp2(-8.0 * torch.arange(1, H + 1, device=dev, dtype=torch.float32) / H)
                    if case["slopes"] else None)
    return st


# ------------------------------------------------------------------------------------------------ one pass


def _turn(x, cos, sin, interleaved):
    """The first 2 x cos.shape[-1] elements of each row turned; cos, sin broadcast against [..., rot / 2]."""
    rot = 2 * cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _positions(st, N, dev):
    pos = st["pos"]
    return pos if pos.dim() == 2 else pos[:, None] + torch.arange(N, device=dev)


def _plain_qk(st, c):
    out = {}
    for name in ("q", "k"):
        x = st[name].float()
        if c["norm"] != "none":
            ss = (x * x).sum(-1, keepdim=True)
            x = x * torch.rsqrt((ss / c["d"] if c["norm"] == "rms" else ss) + 1e-6)
            if st[name + "_weight"] is not None:
                x = x * st[name + "_weight"]
        if c["rot"]:
            at = _positions(st, c["N"], x.device)
            x = _turn(x, st["cos"][at][:, None], st["sin"][at][:, None], c["interleaved"])
        if st["lens"] is not None:  # padding of an output made by the call: zeros
            alive = torch.arange(c["N"], device=x.device) < st["lens"][:, None]
            x = torch.where(alive[:, None, :, None], x, torch.zeros_like(x))
        out[name] = x.to(st[name].dtype)
    return out


def _slots(st, c):
    """(b, i, page, slot) of every new token: its sequence, its number in the call, where it goes."""
    dev, N = st["seen"].device, c["N"]
    i = torch.arange(N, device=dev).expand(c["B"], N)
    new = i < st["lens"][:, None] if st["lens"] is not None else torch.ones_like(i, dtype=torch.bool)
    b, i = new.nonzero(as_tuple=True)
    p = st["seen"][b] + i
    return b, i, st["table"][b, p // c["page"]].long(), p % c["page"], p


def _dense(pages, table, lens, longest, d, bits):
    """fp32 rows [B, Hkv, longest, d] of the cached tokens, zeros behind each sequence."""
    page = pages.shape[2]
    width = -(-longest // page)
    at = table[:, :width].long().clamp(min=0)
    x = pages[at]  # [B, width, Hkv, page, ...]
    B, W, Hkv = x.shape[:3]
    if bits:
        codes, scale, offset = _unpack(x.reshape(B * W, Hkv, page, -1), d)
        x = (codes.view(B * W, Hkv, page, d // 64, 64).float() * scale.float()[..., None] + offset.float()[..., None])
    x = x.reshape(B, W, Hkv, page, d).float().transpose(1, 2).reshape(B, Hkv, W * page, d)[:, :, :longest]
    alive = torch.arange(longest, device=x.device) < lens[:, None]
    return torch.where(alive[:, None, :, None], x, torch.zeros((), device=x.device))


def _plain_append(st, c):
    b, i, at, slot, p = _slots(st, c)
    dt, d = st["k"].dtype, c["d"]
    v = st["v"].transpose(1, 2)[b, i]  # [tokens, Hkv, d]
    k = st["k"].transpose(1, 2)[b, i]
    if c["rot"]:
        # in 4 bits a rounding of a key next to a border is a whole code: 64 bits up to the key's own rounding
        t = torch.float64 if c["bits"] else torch.float32
        k = _turn(k.to(t), st["cos"][p][:, None].to(t), st["sin"][p][:, None].to(t), c["interleaved"]).float().to(dt)
    if not c["bits"]:
        heads = torch.arange(c["Hkv"], device=k.device)
        st["k_pages"][at[:, None], heads, slot[:, None]] = k
        st["v_pages"][at[:, None], heads, slot[:, None]] = v
        return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    out = {}
    for name, x in (("k", k), ("v", v)):
        codes, scale, offset = _unpack(st[name + "_pages"], d)
        heads = torch.arange(c["Hkv"], device=k.device)
        codes, scale, offset = codes.clone(), scale.clone(), offset.clone()
        for whole, rows in zip((codes, scale, offset), _quantise(x)):
            whole[at[:, None], heads, slot[:, None]] = rows
        st[name + "_pages"].copy_(_pack(codes, scale, offset))
        out[name] = _dense(st[name + "_pages"], st["table"], st["total"], st["longest"], d, 4).to(dt)
    return out


def _plain_step(st, c):
    S, H, d = st["q"].shape
    Hkv, group, L = c["Hkv"], H // c["Hkv"], c["L"]
    lens, dev = st["lens"], st["q"].device
    out = torch.empty((S, H, d), dtype=st["q"].dtype, device=dev)
    many = max(1, (1 << 30) // (Hkv * L * d))  # sequences at a time: a few GB of fp32 rows
    for s in range(0, S, many):
        n = lens[s:s + many]
        k = _dense(st["k_pages"], st["table"][s:s + many], n, L, d, c["bits"])
        x = torch.matmul(st["q"][s:s + many].float().reshape(-1, Hkv, group, d), k.transpose(2, 3)) * st["scale"]
        del k
        if c["softcap"]:
            x = torch.tanh(x / c["softcap"]) * c["softcap"]
        age = (n[:, None] - 1 - torch.arange(L, device=dev))[:, None, None]
        if st["slopes"] is not None:
            x = x - st["slopes"].view(Hkv, group, 1) * age
        seen = age >= 0
        if c["window"]:
            seen = seen & (age < c["window"])
        x = torch.where(seen, x, torch.full((), -math.inf, device=dev))
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
        total = e.sum(-1, keepdim=True)
        v = _dense(st["v_pages"], st["table"][s:s + many], n, L, d, c["bits"])
        o = torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))
        out[s:s + many] = o.reshape(-1, H, d).to(out.dtype)
    return {"o": out}


def _own_run(st, c):
    import linear_attention_recurrence_chunked_gb300 as la
    if c["op"] == "qk":
        q, k = la.la_qk_norm_rope(st["q"], st["k"], q_weight=st["q_weight"], k_weight=st["k_weight"],
                                  norm=None if c["norm"] == "none" else c["norm"], eps=1e-6, cos=st["cos"], sin=st["sin"],
                                  pos=st["pos"], interleaved=c["interleaved"], lens=st["lens"])
        return {"q": q, "k": k}
    if c["op"] == "append":
        la.la_paged_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["seen"], cos=st["cos"],
                           sin=st["sin"], interleaved=c["interleaved"], lens=st["lens"])
        if not c["bits"]:
            return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}
        k, v = la.la_paged_read(st["k_pages"], st["v_pages"], st["table"], st["total"], st["longest"],
                                out_dtype=st["k"].dtype)
        return {"k": k, "v": v}
    o = la.la_paged_decode_step(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"], window=c["window"],
                                scale=st["scale"], softcap=c["softcap"], slopes=st["slopes"])
    return {"o": o}


def run(state):
    c = state["case"]
    if own:
        return _own_run(state, c)
    return {"qk": _plain_qk, "append": _plain_append, "step": _plain_step}[c["op"]](state, c)


# ------------------------------------------------------------------------------------------------ work and the definition


def work(case):
    e, d, Hkv = (2 if case["dtype"] == "bf16" else 4), case["d"], case["Hkv"]
    row = d * 9 // 16 if case.get("bits") else d * e  # bytes of a cached row
    if case["op"] == "qk":
        heads = case["H"] + Hkv
        tokens = sum(_new_tokens(case)) if case["ragged"] else case["B"] * case["N"]
        positions = min(case["N"], 300) if case["packed"] else min(4000 + case["N"], tokens)
        table = 4 * case["rot"] * min(positions, tokens)
        written = case["B"] * case["N"]  # padding is zeroed
        return {"bytes": heads * d * e * (tokens + written) + table, "flops": 8 * heads * d * tokens}
    if case["op"] == "append":
        tokens = sum(_new_tokens(case)) if case["ragged"] else case["B"] * case["N"]
        n = max(s + t for s, t in zip(_seen(case), _new_tokens(case)))
        total = sum(_seen(case)) + tokens
        back = 2 * Hkv * (total * row + case["B"] * n * d * e) if case["bits"] else 0
        table = 4 * case["rot"] * min(n, tokens)
        return {"bytes": 2 * Hkv * tokens * (d * e + row) + back + table, "flops": Hkv * d * (8 * tokens + (2 * total if case["bits"] else 0))}
    keys = sum(min(n, case["window"]) if case["window"] else n for n in _lengths(case))
    heads = case["H"] * case["S"]
    return {"bytes": 2 * keys * Hkv * row + 2 * heads * d * e, "flops": 4 * keys * case["H"] * d}


def _exact_qk(st, c):
    out = {}
    half = c["rot"] // 2
    for name in ("q", "k"):
        y = st[name].double()
        if c["norm"] != "none":
            length = y.square().sum(-1, keepdim=True)
            length = length / c["d"] if c["norm"] == "rms" else length
            y = y / (length + 1e-6).sqrt()
            if st[name + "_weight"] is not None:
                y = y * st[name + "_weight"].double()
        if half:
            at = _positions(st, c["N"], y.device)
            z = torch.complex(st["cos"].double(), st["sin"].double())[at][:, None]
            if c["interleaved"]:
                y[..., :2 * half] = torch.view_as_real(torch.view_as_complex(y[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * z).flatten(-2)
            else:
                w = torch.complex(y[..., :half].contiguous(), y[..., half:2 * half].contiguous()) * z
                y[..., :half], y[..., half:2 * half] = w.real, w.imag
        for b, n in enumerate(_new_tokens(c) if st["lens"] is not None else []):
            y[b, :, n:] = 0
        out[name] = y
    return out


def _exact_append(st, c):
    d, page, half = c["d"], c["page"], c["rot"] // 2
    new = _new_tokens(c) if st["lens"] is not None else [c["N"]] * c["B"]
    out = {}
    for name in ("k", "v"):
        if c["bits"]:
            codes, scale, offset = _unpack(st[name + "_pages"], d)
            cache = codes.double().unflatten(-1, (d // 64, 64)).mul_(scale.double()[..., None]).add_(offset.double()[..., None]).flatten(-2)
        else:
            cache = st[name + "_pages"].double()
        rows = torch.zeros((c["B"], c["Hkv"], st["longest"], d), dtype=torch.float64, device=cache.device)
        for b, (past, n) in enumerate(zip(_seen(c), new)):
            x = st[name][b, :, :n].double()
            p = torch.arange(past, past + n, device=x.device)
            if name == "k" and half:
                z = torch.complex(st["cos"].double(), st["sin"].double())[p]
                if c["interleaved"]:
                    x[..., :2 * half] = torch.view_as_real(torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * z).flatten(-2)
                else:
                    w = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * z
                    x[..., :half], x[..., half:2 * half] = w.real, w.imag
            if c["bits"]:
                codes, scale, offset = _quantise(x.float().to(torch.bfloat16), wide=True)
                x = codes.double().unflatten(-1, (d // 64, 64)).mul(scale.double()[..., None]).add(offset.double()[..., None]).flatten(-2)
            at = st["table"][b].long()
            cache[at[p // page], :, p % page] = x.transpose(0, 1)
            if c["bits"]:
                p = torch.arange(past + n, device=x.device)
                rows[b, :, :past + n] = cache[at[p // page], :, p % page].transpose(0, 1)
        out[name if c["bits"] else name + "_pages"] = rows if c["bits"] else cache
    return out


def _exact_step(st, c):
    S, H, d = st["q"].shape
    Hkv, page = c["Hkv"], c["page"]
    out = torch.zeros((S, H, d), dtype=torch.float64, device=st["q"].device)
    for s, n in enumerate(_lengths(c)):
        if n == 0:
            continue
        first = max(0, n - c["window"]) if c["window"] else 0
        p = torch.arange(first, n, device=out.device)
        at, slot = st["table"][s].long()[p // page], p % page
        rows = []
        for name in ("k_pages", "v_pages"):
            if c["bits"]:
                used = st["table"][s, first // page:-(-n // page)].long()
                codes, scale, offset = _unpack(st[name][used], d)
                x = codes.double().unflatten(-1, (d // 64, 64)).mul_(scale.double()[..., None]).add_(offset.double()[..., None]).flatten(-2)
                x = x.transpose(0, 1).reshape(Hkv, -1, d)[:, first % page:first % page + n - first]
            else:
                x = st[name][at, :, slot].transpose(0, 1).double()
            rows.append(x)
        x = st["q"][s].double().reshape(Hkv, H // Hkv, d) @ rows[0].transpose(1, 2) * st["scale"]
        if c["softcap"]:
            x = c["softcap"] * torch.tanh(x / c["softcap"])
        if st["slopes"] is not None:
            x = x - st["slopes"].double().reshape(Hkv, -1, 1) * (n - 1 - p)
        out[s] = (torch.softmax(x, -1) @ rows[1]).reshape(H, d)
    return {"o": out}


def exact(case, seed):
    st = prepare(case, seed)
    return {"qk": _exact_qk, "append": _exact_append, "step": _exact_step}[case["op"]](st, case)
