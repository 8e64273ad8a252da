"""64-bit references of the block norm, the experts' down projections and the whole layer, with the error that fp32 arithmetic
may leave in each (numpy and torch float64; no code of the library).

U is half a step of fp32. An fp32 sum of n terms, in whatever order, is off by at most (n - 1) U times the sum of their sizes.

A product of a planar Q4 row with a vector, here: blocks of 32 are summed exactly enough on matrix instructions and the block
sums are added in fp32. One matrix instruction adds 16 exact products and its accumulator, each cut off no higher than 2^-23
of the largest of them: at most 17 * 2 U of the block's sum of sizes, four instructions a block (two parts of the vector), so
136 U; the parts hold an element to 2^-22 (4 U); 20 U are left for the scale's product, the joins of warps and unscaling.
The block sums themselves add (blocks) U: DOT(blocks) = (blocks + 160) U times sum |w| |x|. What the parts do not hold of
small elements is 2^-33 of the vector's largest element: 2^-33 max|x| sum |w| more.

bf16 layers hold a vector in one f16 part: half a step of f16 (2^-11) of each element instead of 4 U, so 2^-11 sum |w| |x| more,
and nothing else changes (two instructions a block instead of four).
"""

import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half a step of subnormals


def rounded(ref, dtype):
    return HALF_STEP[dtype] * ref.abs() + TINY[dtype]


def q4_matrix(qs, d):
    """Values [..., K] of codes [..., K/32, 16] and scales [..., K/32]."""
    q = torch.cat([qs & 15, qs >> 4], -1).double() - 8
    return (q * d.double().unsqueeze(-1)).flatten(-2)


def rms(x, err, gamma, eps):
    """(norm of x, its error), for x that is off by err: the sum of squares has K terms, added in at most 64 steps a thread
    and 10 across threads (74 U, halved by the root), rsqrt two units (4 U), three products and the mean (5 U)."""
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y = x * r * gamma
    off = (err.square().mean(-1, keepdim=True)).sqrt() * r  # how far err moves r, as a share of it
    return y, y.abs() * (46 * U + off) + err * r * gamma.abs()


def residual_norm(x, residual, post, gate, pre, eps, rs, bs):
    """(h, its error), (y, its error) before rounding to the type; y None without pre."""
    b, err = x.double(), torch.zeros_like(x, dtype=torch.float64)
    if post is not None:
        b, err = rms(b, err, post.double(), eps)
    g = bs if gate is None else bs * gate.double()
    b, err = b * g, err * abs(g) + 3 * U * (b * g).abs()
    h = b
    if residual is not None:
        h = b + rs * residual.double()
        err = err + 2 * U * (rs * residual.double()).abs() + U * h.abs()
    if pre is None:
        return (h, err), (None, None)
    return (h, err), rms(h, err, pre.double(), eps)


def dot(w, x, err, part=0.0):
    """(w x, error) for a matrix [rows, cols], a vector [cols] that is off by err; part: what its f16 parts lose of an element."""
    size = w.abs()
    blocks = w.shape[1] // 32
    return w @ x, ((blocks + 160) * U + part) * (size @ x.abs()) + size @ err + 2.0 ** -33 * x.abs().max() * size.sum(1)


def one_part(dtype):
    return 2.0 ** -11 if dtype == torch.bfloat16 else 0.0


def down(h, h_err, w_of, ids, weights, w_err, residual, rows, part=0.0):
    """(out, error before rounding): w_of(e) the expert's matrix; invalid ids make the token NaN."""
    T, topk = ids.shape
    out = torch.zeros(T, rows, dtype=torch.float64, device=h.device)
    err = torch.zeros_like(out)
    size = torch.zeros_like(out)
    for e in sorted(set(ids.flatten().tolist())):
        m = w_of(e)
        for t, s in torch.nonzero(ids == e).tolist():
            if m is None:
                out[t] = float("nan")
                continue
            z, dz = dot(m, h[t, s], h_err[t, s], part)
            out[t] += weights[t, s] * z
            err[t] += weights[t, s].abs() * dz + w_err[t, s] * z.abs()
            size[t] += (weights[t, s] * z).abs()
    if residual is not None:
        out = out + residual.double()
        size = size + residual.double().abs()
    return out, err + (topk + 2) * U * size


def layer(x, m, gamma, eps, residual, ids, normalize):
    """(out, error), (weights, error), logits and their error, for the picks `ids`. m: the layer's matrices by name, [E, rows,
    cols] in float64."""
    v, verr = x.double(), torch.zeros_like(x, dtype=torch.float64)
    if gamma is not None:
        v, verr = rms(v, verr, gamma.double(), eps)
    part = one_part(x.dtype)
    T, topk = ids.shape
    logits = torch.empty(T, m["router"].shape[0], dtype=torch.float64, device=x.device)
    lerr = torch.empty_like(logits)
    for t in range(T):
        logits[t], lerr[t] = dot(m["router"], v[t], verr[t])
    p = torch.softmax(logits, -1).gather(1, ids)
    w = p / p.sum(-1, keepdim=True) if normalize else p
    # a share's exponent is off by twice the largest logit error; exp, the sums of E and of topk terms and two quotients
    werr = w * (2 * lerr.amax(-1, keepdim=True) + (logits.shape[1] + topk + 10 + 2 * logits.abs().amax(-1, keepdim=True)) * U)
    h = torch.empty(T, topk, m["gate"].shape[1], dtype=torch.float64, device=x.device)
    herr = torch.empty_like(h)
    for e in sorted(set(ids.flatten().tolist())):
        for t, s in torch.nonzero(ids == e).tolist():
            g, dg = dot(m["gate"][e], v[t], verr[t], part)
            u, du = dot(m["up"][e], v[t], verr[t], part)
            a = g * torch.sigmoid(g)
            h[t, s] = a * u
            # silu's slope is at most 1.1; exp's argument is off by |g| U, its value by 2 U
            herr[t, s] = (1.1 * dg + (8 + g.abs()) * U * a.abs()) * (u.abs() + du) + a.abs() * du + U * h[t, s].abs()
    return down(h, herr, lambda e: m["down"][e], ids, w, werr, residual, x.shape[1], part), (w, werr), (logits, lerr)
