"""Cases and plain forms of the decode-step operators between two projection GEMVs.

Four operators of ``quantized_decode_gemv_q4_gb300``:

* ``qk_norm_rope``: RMSNorm of every query and key head and the rotary position rotation, in one pass.
* ``kv4_write``: new keys and values quantised into a paged cache of planar Q4 rows (measured with the read-back of
  the rows it wrote, because what is held in 4 bits comes back as the values it stands for).
* ``kv4_read``: cached rows back as values.
* ``kv4_attention``: attention of the newest tokens of each sequence over that cache.

A case's ``op`` names the operator. With ``own`` false, ``run`` computes the same thing from elementary torch
operations.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ELEM = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------

def listed():
    return [
        # One token of one stream in the library's own fp32, 28 query heads over 4 key heads of 128 (a 3584-wide
        # projection): pure latency.
        dict(name="rope f32 T1", op="rope", dtype="f32", T=1, Hq=28, Hkv=4, D=128, rot=128, interleaved=False, norm=True),
        # A decode batch whose q and k are columns of one q/k/v projection output (strided rows), partial rotation.
        dict(name="rope bf16 T67", op="rope", dtype="bf16", T=67, Hq=32, Hkv=8, D=128, rot=64, interleaved=True, norm=True),
        # A prompt of 8191 tokens: bound by memory.
        dict(name="rope bf16 T8191", op="rope", dtype="bf16", T=8191, Hq=32, Hkv=8, D=128, rot=128, interleaved=False,
             norm=True),
        # The new token of each of 8 streams goes into the cache.
        dict(name="write f32 T8", op="write", dtype="f32", T=8, Hkv=4, D=128, page=16, pad=0),
        # A packed batch of prompts whose last rows are padding (no slot): the rows' slots lie on shuffled pages.
        dict(name="write bf16 T16384", op="write", dtype="bf16", T=16384, Hkv=8, D=128, page=16, pad=100),
        # A short shared prefix is read back to be re-encoded.
        dict(name="read f32 T500", op="read", dtype="f32", T=500, Hkv=4, D=128, page=16, pad=0),
        # A long document's cache is read back.
        dict(name="read bf16 T50001", op="read", dtype="bf16", T=50001, Hkv=8, D=128, page=64, pad=0),
        # One stream, a hundred tokens in: pure latency.
        dict(name="attn f32 B1 L100", op="attn", dtype="f32", B=1, M=1, Hq=28, Hkv=4, D=128, page=16, longest=100,
             ragged=False, window=0, lse=False),
        # One stream far into a document, in the library's own fp32: a few rows, one long axis.
        dict(name="attn f32 B1 L16384", op="attn", dtype="f32", B=1, M=1, Hq=28, Hkv=4, D=128, page=16, longest=16384,
             ragged=False, window=0, lse=True),
        # A serving batch of ragged lengths (some empty, some one token long).
        dict(name="attn bf16 B64 ragged", op="attn", dtype="bf16", B=64, M=1, Hq=32, Hkv=8, D=128, page=16, longest=8192,
             ragged=True, window=0, lse=False),
        # One very long stream.
        dict(name="attn f16 B1 L131001", op="attn", dtype="f16", B=1, M=1, Hq=32, Hkv=8, D=128, page=64, longest=131001,
             ragged=False, window=0, lse=False),
        # Draft tokens of a batch checked in one call, with a sliding window.
        dict(name="attn bf16 B16 M4 window", op="attn", dtype="bf16", B=16, M=4, Hq=64, Hkv=8, D=64, page=32,
             longest=6000, ragged=True, window=2048, lse=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn", "attn", "attn"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    if op == "rope":
        D = rng.choice([32, 64, 96, 128, 160, 192, 256])
        rot = rng.choice([D, D, D // 2])
        Hq = Hkv * rng.choice([1, 3, 4, 7, 8])
        T = _spread(rng, 1, min(8191, 8191 * 40 * 128 * 2 // ((Hq + Hkv) * D * ELEM[dtype])))
        return dict(op=op, dtype=dtype, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.8)
    if op in ("write", "read"):
        D = rng.choice([32, 64, 96, 128, 256])
        most = 16384 if op == "write" else 50001
        T = _spread(rng, 1, min(most, most * 8 * 128 * 2 // (Hkv * D * ELEM[dtype])))
        return dict(op=op, dtype=dtype, T=T, Hkv=Hkv, D=D, page=rng.choice([1, 8, 16, 32, 64, 256]),
                    pad=rng.choice([0, min(T - 1, 7)]))
    B = _spread(rng, 1, 64)
    M, Hq, D = rng.choice([1, 1, 1, 2, 3, 5, 8]), Hkv * rng.choice([1, 3, 4, 7, 8]), rng.choice([64, 128, 128, 256])
    # no more bytes and no more arithmetic than the largest listed case
    longest = _spread(rng, 1, max(1, min(131000, 260_000_000 // (B * Hkv * D), 1_000_000_000 // (B * M * Hq * D))))
    return dict(op=op, dtype=dtype, B=B, M=M, Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([1, 8, 16, 32, 64, 256]), longest=longest,
                ragged=rng.random() < 0.6, window=rng.choice([0, 0, _spread(rng, 1, 4096)]), lse=rng.random() < 0.5)


def lengths(case):
    """The sequences' lengths: ragged ones spread over 0..longest, the same for every seed."""
    B, longest = case["B"], case["longest"]
    if not case["ragged"]:
        return [longest] * B
    out = [int(longest * ((b + 1) * 0.6180339887498949 % 1.0)) for b in range(B)]
    out[0] = longest
    if B > 2:
        out[1], out[2] = 0, 1
    return out


def work(case):
    if case["op"] == "rope":
        rows = case["T"] * (case["Hq"] + case["Hkv"])
        table = case["T"] * case["rot"] * 4
        return {"bytes": 2 * rows * case["D"] * ELEM[case["dtype"]] + table, "flops": rows * case["D"] * 7}
    if case["op"] in ("write", "read"):
        n = (case["T"] - case["pad"]) * case["Hkv"] * case["D"] * 2
        packed = n * 9 // 16
        values = n * ELEM[case["dtype"]]
        if case["op"] == "write":  # values in, 4 bits out, 4 bits in again, values out
            return {"bytes": 2 * packed + 2 * values + 8 * case["T"], "flops": 6 * n}
        return {"bytes": packed + values + 4 * case["T"], "flops": 2 * n}
    seen = [min(n, case["window"] + case["M"] - 1) if case["window"] else n for n in lengths(case)]
    rows = case["B"] * case["M"] * case["Hq"] * case["D"]
    return {"bytes": sum(seen) * case["Hkv"] * case["D"] * 2 * 9 // 16 + 2 * rows * ELEM[case["dtype"]],
            "flops": 4 * sum(seen) * case["M"] * case["Hq"] * case["D"]}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _keys(g, *shape):
    """Key-like rows: a few channels many times larger than the rest."""
    x = _normal(g, *shape)
    D = shape[-1]
    x *= torch.where(torch.rand(D, generator=g, device="cuda") < 0.04, 6.0, 1.0)
    return x * 0.8


def _pack(x):
    """Planar Q4 rows of fp32 values: (codes uint8 [..., D/2], scales f16 [..., D/32])."""
    blocks = x.unflatten(-1, (-1, 32)).double()
    # the largest of scale, code and value are the definition's: d = amax / 7 in f16, code = nearest of x / d
    d = (blocks.abs().amax(-1) / 7).clamp(max=65504.0).float().half()
    dd = d.double().unsqueeze(-1)
    q = torch.where(dd > 0, blocks / torch.where(dd > 0, dd, 1.0), 0.0).round().clamp(-7, 7) + 8
    q = q.to(torch.uint8)
    return (q[..., :16] | (q[..., 16:] << 4)).flatten(-2), d


def _unpack(qs, d):
    """fp32 values of planar Q4 rows."""
    b = qs.unflatten(-1, (-1, 16))
    q = torch.cat([b & 15, b >> 4], -1).float() - 8.0
    return (q * d.float().unsqueeze(-1)).flatten(-2)


def _empty_cache(pages, Hkv, page, D):
    """Pages as a server keeps them: what nobody has written holds any bits, NaN scales among them."""
    made = []
    for _ in range(2):
        made.append(torch.full((pages, Hkv, page, D // 2), 255, dtype=torch.uint8, device="cuda"))
        made.append(torch.full((pages, Hkv, page, D // 32), float("nan"), dtype=torch.float16, device="cuda"))
    return dict(zip(("k_qs", "k_d", "v_qs", "v_d"), made))


def _put(cache, which, slots, values):
    qs, d = cache[which + "_qs"], cache[which + "_d"]
    page = qs.shape[2]
    for at in range(0, slots.numel(), 1 << 17):  # in parts, so that the 64-bit temporaries stay small
        sl = slots[at:at + (1 << 17)]
        c, s = _pack(values[at:at + (1 << 17)])
        qs[sl // page, :, sl % page] = c
        d[sl // page, :, sl % page] = s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    dt = DTYPES[case["dtype"]]
    Hkv, D = case["Hkv"], case["D"]
    s = {"case": case}
    if case["op"] == "rope":
        T, Hq, rot = case["T"], case["Hq"], case["rot"]
        # q and k are columns of the projection's output [T, (Hq + 2 Hkv) D]
        qkv = _normal(g, T, Hq + 2 * Hkv, D).to(dt)
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        s["q_out"], s["k_out"] = torch.empty(T, Hq, D, dtype=dt, device="cuda"), torch.empty(T, Hkv, D, dtype=dt, device="cuda")
        s["q_gamma"] = (1 + 0.1 * _normal(g, D)) if case["norm"] else None
        s["k_gamma"] = (1 + 0.1 * _normal(g, D)) if case["norm"] else None
        far = 32768
        angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot))
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], -1).float()
        s["positions"] = torch.randint(0, far, (T,), generator=g, device="cuda", dtype=torch.int32)
        return s
    if case["op"] in ("write", "read"):
        T, page = case["T"], case["page"]
        pages = -(-T // page) + 3
        s.update(_empty_cache(pages, Hkv, page, D))
        order = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        slots = order[t // page] * page + t % page
        if case["op"] == "write":
            kv = torch.cat([_keys(g, T, Hkv, D), _normal(g, T, Hkv, D)], 1).to(dt)
            s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
        else:
            _put(s, "k", slots, _keys(g, T, Hkv, D))
            _put(s, "v", slots, _normal(g, T, Hkv, D))
        if case["pad"]:
            slots[T - case["pad"]:] = -1
        s["slots"] = slots.to(torch.int32)
        s["k_out"] = torch.zeros(T, Hkv, D, dtype=dt, device="cuda")
        s["v_out"] = torch.zeros(T, Hkv, D, dtype=dt, device="cuda")
    else:
        B, M, Hq, page = case["B"], case["M"], case["Hq"], case["page"]
        lens = lengths(case)
        per = [-(-n // page) for n in lens]
        pages = sum(per) + 5
        s.update(_empty_cache(pages, Hkv, page, D))
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        width = max(per) + 1
        firsts = torch.tensor([sum(per[:b]) for b in range(B)], device="cuda")
        at = torch.arange(width, device="cuda")
        used = at[None, :] < torch.tensor(per, device="cuda")[:, None]
        s["block_table"] = torch.where(used, order[(firsts[:, None] + at).clamp(max=pages - 1)], 0).contiguous()
        for b, n in enumerate(lens):
            t = torch.arange(n, device="cuda")
            slots = s["block_table"][b].long()[t // page] * page + t % page
            _put(s, "k", slots, _keys(g, n, Hkv, D))
            _put(s, "v", slots, _normal(g, n, Hkv, D))
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = (1.2 * _normal(g, B, M, Hq, D)).to(dt)
        s["out"] = torch.empty(B, M, Hq, D, dtype=dt, device="cuda")
        s["lse"] = torch.empty(B, M, Hq, device="cuda") if case["lse"] else None
    if own:  # the handle that a user's program keeps beside the cache's tensors, and the call's workspace
        import quantized_decode_gemv_q4_gb300 as q4

        s["cache"] = q4.KV4Cache(s["k_qs"], s["k_d"], s["v_qs"], s["v_d"])
        if case["op"] == "attn":
            s["workspace"] = q4.kv4_attention_workspace(s["q"], s["cache"])
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import quantized_decode_gemv_q4_gb300 as q4

        if op == "rope":
            q4.qk_norm_rope(s["q_out"], s["k_out"], s["q"], s["k"], s["q_gamma"], s["k_gamma"], s["cos_sin"], s["positions"],
                            eps=EPS, interleaved=s["case"]["interleaved"])
            return [s["q_out"], s["k_out"]]
        if op == "attn":
            q4.kv4_attention(s["out"], s["q"], s["cache"], s["block_table"], s["seq_lens"], window=s["case"]["window"],
                             lse=s["lse"], workspace=s["workspace"])
            return [s["out"]] if s["lse"] is None else [s["out"], s["lse"]]
        if op == "write":
            q4.kv4_write(s["cache"], s["k"], s["v"], s["slots"])
        q4.kv4_read(s["k_out"], s["v_out"], s["cache"], s["slots"])
        return [s["k_out"], s["v_out"]]
    if op == "rope":
        return [_rope(s, s["q"], s["q_gamma"]), _rope(s, s["k"], s["k_gamma"])]
    if op == "attn":
        return _attention(s)
    if op == "write":
        _write(s, "k")
        _write(s, "v")
    return [_read(s, "k"), _read(s, "v")]


def _rope(s, x, gamma):
    c = s["case"]
    rot = c["rot"]
    y = x.float()
    if gamma is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * gamma
    row = s["cos_sin"][s["positions"].long()].unsqueeze(1)
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    if c["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _write(s, which):
    n = s["case"]["T"] - s["case"]["pad"]  # the rows behind it have no slot
    sl = s["slots"][:n].long()
    page = s["case"]["page"]
    qs, d = _pack(s[which][:n].float())
    s[which + "_qs"][sl // page, :, sl % page] = qs
    s[which + "_d"][sl // page, :, sl % page] = d


def _read(s, which):
    n = s["case"]["T"] - s["case"]["pad"]
    sl = s["slots"][:n].long()
    page = s["case"]["page"]
    out = s[which + "_out"]
    out[:n] = _unpack(s[which + "_qs"][sl // page, :, sl % page], s[which + "_d"][sl // page, :, sl % page]).to(out.dtype)
    return out


def _attention(s):
    c = s["case"]
    B, M, Hkv, D, page = c["B"], c["M"], c["Hkv"], c["D"], c["page"]
    t = torch.arange(max(c["longest"], 1), device="cuda")
    pages, offs = s["block_table"][:, t // page].long(), (t % page).expand(B, -1)
    there = (t < s["seq_lens"][:, None])[..., None, None]
    k = torch.where(there, _unpack(s["k_qs"][pages, :, offs], s["k_d"][pages, :, offs]), 0.0)
    v = torch.where(there, _unpack(s["v_qs"][pages, :, offs], s["v_d"][pages, :, offs]), 0.0)
    q = s["q"].float().reshape(B, M, Hkv, -1, D)
    logits = torch.einsum("bmhgd,blhd->bmhgl", q, k) * D ** -0.5
    last = s["seq_lens"][:, None] - M + torch.arange(M, device="cuda")  # the position of each query
    seen = t <= last[..., None]
    if c["window"]:
        seen &= t > last[..., None] - c["window"]
    logits = logits.masked_fill(~seen[:, :, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bmhgl,blhd->bmhgd", p, v) / torch.where(total == 0, 1.0, total)
    out = out.reshape(s["q"].shape).to(s["q"].dtype)
    if not c["lse"]:
        return [out]
    return [out, (top + torch.log(total)).reshape(B, M, -1)]


# ------------------------------------------------------------------------------------------------
# the same from the definitions in 64 bits
# ------------------------------------------------------------------------------------------------

def _table():
    """The 16 values of a code in units of its scale."""
    return torch.arange(-8.0, 8.0, dtype=torch.float64, device="cuda")


def _rows64(qs, d):
    """Rows [n, D/2] of codes and [n, D/32] of scales as 64-bit values [n, D]."""
    n, D = qs.shape[0], qs.shape[1] * 2
    out = torch.empty(n, D // 32, 2, 16, dtype=torch.float64, device="cuda")
    by = qs.reshape(n, D // 32, 16).long()
    out[:, :, 0] = _table()[by % 16]
    out[:, :, 1] = _table()[by // 16]
    return (out * d.double()[:, :, None, None]).reshape(n, D)


def exact(case, seed):
    s = prepare(case, seed)
    D = case["D"]
    if case["op"] == "rope":
        rot, half = case["rot"], case["rot"] // 2
        where = s["positions"].long()
        turn = torch.complex(s["cos_sin"][where, :half].double(), s["cos_sin"][where, half:].double())[:, None]
        outs = []
        for name in ("q", "k"):
            x = s[name].double()
            if case["norm"]:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * s[name + "_gamma"].double()
            i = torch.arange(half, device="cuda")
            first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            z = torch.complex(x[..., first], x[..., second]) * turn
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            outs.append(y)
        return outs
    if case["op"] == "write":
        outs = []
        n = case["T"] - case["pad"]
        for name in ("k", "v"):
            x = s[name].double().reshape(case["T"], case["Hkv"], D // 32, 32)
            d = (x.abs().max(-1, keepdim=True).values / 7).float().half().double()
            y = d * torch.clamp(torch.round(x / d), -7, 7)
            y[n:] = 0
            outs.append(y.reshape(case["T"], case["Hkv"], D))
        return outs
    if case["op"] == "read":
        outs = []
        n = case["T"] - case["pad"]
        for name in ("k", "v"):
            y = torch.zeros(case["T"], case["Hkv"], D, dtype=torch.float64, device="cuda")
            for h in range(case["Hkv"]):
                sl = s["slots"][:n].long()
                y[:n, h] = _rows64(s[name + "_qs"][:, h].reshape(-1, D // 2)[sl], s[name + "_d"][:, h].reshape(-1, D // 32)[sl])
            outs.append(y)
        return outs
    B, M, Hq, Hkv, page = case["B"], case["M"], case["Hq"], case["Hkv"], case["page"]
    out = torch.zeros(B, M, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, M, Hq), -math.inf, dtype=torch.float64, device="cuda")
    group = Hq // Hkv
    for b, n in enumerate(lengths(case)):
        for h in range(Hkv):
            which = s["block_table"][b, :-(-n // page)].long()
            k, v = (_rows64(s[x + "_qs"][which, h].reshape(-1, D // 2)[:n], s[x + "_d"][which, h].reshape(-1, D // 32)[:n])
                    for x in ("k", "v"))
            for m in range(M):
                end = n - M + m + 1
                start = max(0, end - case["window"]) if case["window"] else 0
                if end <= start:
                    continue
                q = s["q"][b, m, h * group:(h + 1) * group].double()
                a = q @ k[start:end].T / math.sqrt(D)
                lse[b, m, h * group:(h + 1) * group] = torch.logsumexp(a, -1)
                out[b, m, h * group:(h + 1) * group] = torch.softmax(a, -1) @ v[start:end]
    return [out, lse] if case["lse"] else [out]
