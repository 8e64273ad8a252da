"""Cases and plain forms of the operators around and inside a mixture-of-experts block.

Three operators of ``quantized_decode_gemv_q4_gb300``:

* ``residual_norm``: the norm behind a block, its gate and scales, the residual sum and the norm before the next block,
  in one pass.
* ``moe_q4_down_gemv``: the selected experts' down projections (planar Q4) and their weighted sum per token.
* ``moe_q4_layer``: a whole mixture-of-experts layer for a few tokens: norm, router, gate and up projections, SwiGLU, down
  projections, weighted sum and residual.

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
        # One token of one stream between two blocks, plain pre-norm residual: pure latency.
        dict(name="norm f32 T1 K2048", op="norm", dtype="f32", T=1, K=2048, post=False, pre=True, gate="none", rs=1.0, bs=1.0),
        # A decode batch with norms on both sides of the block and a per-channel gate; x are columns of a wider tensor.
        dict(name="norm bf16 T67 K3584", op="norm", dtype="bf16", T=67, K=3584, post=True, pre=True, gate="channel", rs=1.0,
             bs=1.0),
        # An odd number of tokens of an odd width, gated element by element.
        dict(name="norm f16 T1023 K1416", op="norm", dtype="f16", T=1023, K=1416, post=True, pre=True, gate="element", rs=0.8,
             bs=0.25),
        # A prompt: bound by memory.
        dict(name="norm bf16 T8191 K4096", op="norm", dtype="bf16", T=8191, K=4096, post=True, pre=True, gate="none", rs=1.0,
             bs=1.0),
        # The library's own mixture of experts (64 experts of 1408 x 2048, top 8), finished behind its SwiGLU call: one token,
        # its 8 tokens, and a batch whose tokens meet at the experts.
        dict(name="down f32 T1 E64", op="down", dtype="f32", T=1, topk=8, E=64, N=1408, K=2048, residual=False),
        dict(name="down f32 T8 E64", op="down", dtype="f32", T=8, topk=8, E=64, N=1408, K=2048, residual=True),
        dict(name="down bf16 T64 E64", op="down", dtype="bf16", T=64, topk=8, E=64, N=1408, K=2048, residual=True),
        # Few large experts (the library's 14336 x 4096 matrices), two for each of 7 tokens.
        dict(name="down bf16 T7 E8 large", op="down", dtype="bf16", T=7, topk=2, E=8, N=14336, K=4096, residual=True),
        # The whole layer: one token, the library's 8 tokens, a batch, and a small odd-sized one.
        dict(name="layer f32 T1 E64", op="layer", dtype="f32", T=1, topk=8, E=64, N=1408, K=2048, norm=True, normalize=True),
        dict(name="layer f32 T8 E64", op="layer", dtype="f32", T=8, topk=8, E=64, N=1408, K=2048, norm=True, normalize=True),
        dict(name="layer bf16 T64 E64", op="layer", dtype="bf16", T=64, topk=8, E=64, N=1408, K=2048, norm=True,
             normalize=True),
        dict(name="layer f16 T5 E10 odd", op="layer", dtype="f16", T=5, topk=3, E=10, N=1056, K=672, norm=False,
             normalize=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "down", "layer", "layer"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "norm":
        K = 8 * _spread(rng, 8, 1024)
        T = _spread(rng, 1, max(1, min(8191, 8191 * 4096 * 2 // (K * ELEM[dtype] * 2))))
        post = rng.random() < 0.6
        return dict(op=op, dtype=dtype, T=T, K=K, post=post, pre=rng.random() < 0.8,
                    gate=rng.choice(["none", "channel", "token", "element"]), rs=rng.choice([1.0, 0.7]),
                    bs=rng.choice([1.0, 0.22]))
    E = _spread(rng, 4, 128)
    topk = min(E, rng.choice([1, 2, 3, 4, 6, 8]))
    K = 32 * _spread(rng, 8, 128)
    # no more weights than the library's own experts hold
    N = 32 * _spread(rng, 8, max(8, min(448, 64 * 1408 * 2048 // (E * K * 32))))
    T = _spread(rng, 1, min(64, 512 // topk))
    case = dict(op=op, dtype=dtype, T=T, topk=topk, E=E, N=N, K=K)
    if op == "down":
        return dict(case, residual=rng.random() < 0.5)
    return dict(case, norm=rng.random() < 0.7, normalize=rng.random() < 0.7)


def _experts_met(case):
    """How many experts T tokens select between them, on average."""
    return case["E"] * (1 - (1 - case["topk"] / case["E"]) ** case["T"])


def work(case):
    if case["op"] == "norm":
        n, e = case["T"] * case["K"], ELEM[case["dtype"]]
        passes = 3 + (1 if case["pre"] else 0) + (1 if case["gate"] == "element" else 0)
        return {"bytes": passes * n * e + 8 * case["K"], "flops": 12 * n}
    T, topk, N, K = case["T"], case["topk"], case["N"], case["K"]
    e = ELEM[case["dtype"]]
    weights = _experts_met(case) * N * K
    if case["op"] == "down":
        return {"bytes": weights * 9 / 16 + T * topk * (N * 4 + 8) + T * K * e * (2 if case["residual"] else 1),
                "flops": 2 * T * topk * N * K}
    return {"bytes": 3 * weights * 9 / 16 + case["E"] * K * 9 / 16 + 2 * T * K * e,
            "flops": 6 * T * topk * N * K + 2 * T * case["E"] * K}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _hidden(g, T, K):
    """Hidden states: a few channels many times larger than the rest."""
    return _normal(g, T, K) * torch.where(torch.rand(K, generator=g, device="cuda") < 0.02, 8.0, 1.0)


def _weights(g, rows, K):
    """Planar Q4 rows: (codes uint8 [rows, K/32, 16], scales f16 [rows, K/32]); outputs of about the inputs' size."""
    qs = torch.empty(rows, K // 32, 16, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // K)
    for at in range(0, rows, step):  # in parts, so that the temporaries stay small
        part = qs[at:at + step]
        codes = (torch.randn(2, *part.shape, generator=g, device="cuda") * 2.3 + 8).round_().clamp_(1, 15).to(torch.uint8)
        part.copy_(codes[0] | (codes[1] << 4))
    d = (0.7 + 0.6 * torch.rand(rows, K // 32, generator=g, device="cuda")) / (2.3 * math.sqrt(K))
    return qs, d.half()


def _unpack(qs, d):
    """fp32 values [..., K] of planar Q4 rows."""
    q = torch.cat([qs & 15, qs >> 4], -1).float() - 8.0
    return (q * d.float().unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    dt = DTYPES[case["dtype"]]
    T, K = case["T"], case["K"]
    s = {"case": case}
    if case["op"] == "norm":
        s["x"] = _normal(g, T, 2, K).to(dt)[:, 0]  # columns of a wider tensor, where there is more than one token
        s["residual"] = (2 * _hidden(g, T, K)).to(dt)
        s["post_gamma"] = (1 + 0.2 * _normal(g, K)) if case["post"] else None
        s["pre_gamma"] = (1 + 0.2 * _normal(g, K)) if case["pre"] else None
        shape = {"none": None, "channel": (K,), "token": (T, 1), "element": (T, K)}[case["gate"]]
        s["gate"] = None if shape is None else torch.tanh(_normal(g, *shape)).to(dt)
        s["h"] = torch.empty(T, K, dtype=dt, device="cuda")
        s["y"] = torch.empty(T, K, dtype=dt, device="cuda") if case["pre"] else None
        return s
    topk, E, N = case["topk"], case["E"], case["N"]
    s["down_qs"], s["down_d"] = (t.unflatten(0, (E, K)) for t in _weights(g, E * K, N))
    s["out"] = torch.empty(T, K, dtype=dt, device="cuda")
    if case["op"] == "down":
        s["residual"] = _hidden(g, T, K).to(dt) if case["residual"] else None
        gate = _normal(g, T, topk, N)
        s["h"] = gate * torch.sigmoid(gate) * _normal(g, T, topk, N)
        scores = _normal(g, T, E)
        top, ids = torch.sort(scores, dim=-1, descending=True, stable=True)
        s["ids"] = ids[:, :topk].to(torch.int32).contiguous()
        s["w"] = torch.softmax(2 * top[:, :topk], -1).contiguous()
        if own:
            import quantized_decode_gemv_q4_gb300 as q4

            s["workspace"] = q4.moe_q4_down_workspace(s["out"], s["h"])
        return s
    s["router_qs"], s["router_d"] = _weights(g, E, K)
    for name in ("gate", "up"):
        s[name + "_qs"], s[name + "_d"] = (t.unflatten(0, (E, N)) for t in _weights(g, E * N, K))
    s["gamma"] = (1 + 0.2 * _normal(g, K)) if case["norm"] else None
    x = _hidden(g, T, K).to(dt)
    if topk < E:
        # A token whose last chosen and first rejected experts lie closer than 32 bits can tell has two right answers:
        # such tokens are drawn again.
        router = _unpack(s["router_qs"], s["router_d"]).double().T
        for _ in range(20):
            v = x.double() if s["gamma"] is None else x.double() * s["gamma"].double()
            top = torch.sort(v @ router, dim=-1, descending=True).values
            close = top[:, topk - 1] - top[:, topk] < 1e-4 * top.std(-1)
            x = torch.where(close[:, None], _hidden(g, T, K).to(dt), x)
    s["x"] = x
    if own:  # the handle that a user's program keeps beside the weights, and the call's workspace
        import quantized_decode_gemv_q4_gb300 as q4

        s["moe"] = q4.MoEWeights(s["router_qs"], s["router_d"], s["gate_qs"], s["gate_d"], s["up_qs"], s["up_d"],
                                 s["down_qs"], s["down_d"])
        s["workspace"] = q4.moe_q4_layer_workspace(s["moe"], s["x"], topk)
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        import quantized_decode_gemv_q4_gb300 as q4

        if c["op"] == "norm":
            q4.residual_norm(s["h"], s["y"], s["x"], s["residual"], post_gamma=s["post_gamma"], gate=s["gate"],
                             pre_gamma=s["pre_gamma"], eps=EPS, residual_scale=c["rs"], branch_scale=c["bs"])
            return [s["h"]] if s["y"] is None else [s["h"], s["y"]]
        if c["op"] == "down":
            q4.moe_q4_down_gemv(s["out"], s["down_qs"], s["down_d"], s["h"], s["ids"], s["w"], residual=s["residual"],
                                workspace=s["workspace"])
            return s["out"]
        # the hidden states go through the layer's norm and are its residual
        q4.moe_q4_layer(s["out"], s["x"], s["moe"], c["topk"], gamma=s["gamma"], eps=EPS, residual=s["x"],
                        normalize=c["normalize"], workspace=s["workspace"])
        return s["out"]
    if c["op"] == "norm":
        return _residual_norm(s)
    if c["op"] == "down":
        total = 0.0 if s["residual"] is None else s["residual"].float()
        return (total + _down(s, s["h"], s["ids"].long(), s["w"])).to(s["out"].dtype)
    return _layer(s)


def _rms(x, gamma):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma


def _residual_norm(s):
    c = s["case"]
    b = s["x"].float()
    if s["post_gamma"] is not None:
        b = _rms(b, s["post_gamma"])
    if s["gate"] is not None:
        b = b * s["gate"].float()
    h = c["rs"] * s["residual"].float() + c["bs"] * b
    out = [h.to(s["x"].dtype)]
    if s["pre_gamma"] is not None:
        out.append(_rms(h, s["pre_gamma"]).to(s["x"].dtype))
    return out


def _per_expert(c, ids, apply, outs):
    """Fills outs [T * topk, rows] with apply(expert, its slots): each expert once where the slots are many, else each slot."""
    E, flat = c["E"], ids.reshape(-1)
    if flat.numel() >= E:
        for e in range(E):
            outs += apply(slice(e, e + 1), slice(None)) * (flat == e)[:, None]
    else:
        for i in range(flat.numel()):
            outs[i:i + 1] = apply(flat[i:i + 1], slice(i, i + 1))
    return outs


def _down(s, h, ids, w):
    c = s["case"]
    h = h.reshape(-1, c["N"])
    z = torch.zeros(h.shape[0], c["K"], device="cuda")
    _per_expert(c, ids, lambda e, at: h[at] @ _unpack(s["down_qs"][e][0], s["down_d"][e][0]).T, z)
    return (z.unflatten(0, ids.shape) * w.unsqueeze(-1)).sum(1)


def _layer(s):
    c = s["case"]
    x = s["x"].float()
    v = x if s["gamma"] is None else _rms(x, s["gamma"])
    # which experts a token goes to is a border: the logits are taken in 64 bits
    logits = v.double() @ _unpack(s["router_qs"], s["router_d"]).double().T
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, ids = top[:, :c["topk"]], ids[:, :c["topk"]]
    share = torch.exp(top - logits.amax(-1, keepdim=True))
    w = share / (share if c["normalize"] else torch.exp(logits - logits.amax(-1, keepdim=True))).sum(-1, keepdim=True)
    rows = v.repeat_interleave(c["topk"], 0)
    h = torch.zeros(rows.shape[0], c["N"], device="cuda")

    def gated(e, at):
        gate = rows[at] @ _unpack(s["gate_qs"][e][0], s["gate_d"][e][0]).T
        return gate / (1 + torch.exp(-gate)) * (rows[at] @ _unpack(s["up_qs"][e][0], s["up_d"][e][0]).T)

    _per_expert(c, ids, gated, h)
    return (x + _down(s, h, ids, w.float())).to(s["x"].dtype)


# ------------------------------------------------------------------------------------------------
# the same from the definitions in 64 bits
# ------------------------------------------------------------------------------------------------

def _matrix64(qs, d):
    """64-bit values [rows, K] of planar Q4 rows, from the 16 values of a code in units of its scale."""
    rows, blocks, _ = qs.shape
    values = torch.arange(-8.0, 8.0, dtype=torch.float64, device="cuda")
    out = torch.empty(rows, blocks, 2, 16, dtype=torch.float64, device="cuda")
    out[:, :, 0] = values[(qs % 16).long()]
    out[:, :, 1] = values[(qs // 16).long()]
    out *= d.double()[:, :, None, None]
    return out.reshape(rows, blocks * 32)


def _unit64(x):
    """x over its root mean square."""
    return x / torch.sqrt(EPS + (x * x).sum(-1, keepdim=True) / x.shape[-1])


def _sum64(s, rows, ids, w):
    """Sum over a token's picks of weight * down projection; rows(t, i, e): the vector that goes into expert e."""
    T, topk = ids.shape
    total = torch.zeros(T, s["case"]["K"], dtype=torch.float64, device="cuda")
    where = ids.cpu()
    for e in sorted(set(where.flatten().tolist())):
        t, i = torch.nonzero(where == e, as_tuple=True)
        t, i = t.cuda(), i.cuda()
        z = _matrix64(s["down_qs"][e], s["down_d"][e]) @ rows(t, i, e).T
        total.index_add_(0, t, z.T * w[t, i].double()[:, None])
    return total


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        branch = s["x"].double()
        if case["post"]:
            branch = _unit64(branch) * s["post_gamma"].double()
        if case["gate"] != "none":
            branch = branch * s["gate"].double().expand_as(branch)
        h = s["residual"].double() * case["rs"] + branch * case["bs"]
        return [h, _unit64(h) * s["pre_gamma"].double()] if case["pre"] else [h]
    if case["op"] == "down":
        total = _sum64(s, lambda t, i, e: s["h"][t, i].double(), s["ids"], s["w"])
        return total if s["residual"] is None else total + s["residual"].double()
    x = s["x"].double()
    v = _unit64(x) * s["gamma"].double() if case["norm"] else x
    logits = v @ _matrix64(s["router_qs"], s["router_d"]).T
    shares = torch.softmax(logits, -1)
    # the picks one after the other: the largest that is left, the lowest index of equal ones
    left, ids = logits.clone(), []
    for _ in range(case["topk"]):
        best = (left == left.max(-1, keepdim=True).values).to(torch.int8).argmax(-1)
        ids.append(best)
        left.scatter_(1, best[:, None], -math.inf)
    ids = torch.stack(ids, 1)
    w = shares.gather(1, ids)
    if case["normalize"]:
        w = w / w.sum(-1, keepdim=True)

    def hidden(t, i, e):
        a = v[t] @ _matrix64(s["gate_qs"][e], s["gate_d"][e]).T
        return a * torch.sigmoid(a) * (v[t] @ _matrix64(s["up_qs"][e], s["up_d"][e]).T)

    return x + _sum64(s, hidden, ids, w)
