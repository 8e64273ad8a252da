"""The experts' products where precision or a range ends: sums that cancel, vectors of which more than f16's bits matter."""

import pytest
import torch

import moe_ref as ref
from test_gpu_moe_layer import Rand, check_down, check_layer, down_case, layer_case, run_layer

pytestmark = pytest.mark.gpu

import quantized_decode_gemv_q4_gb300 as q4  # noqa: E402

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def pairs(*shape, second=7):
    """Rows [..., K] (K = 32 n) of which only weights 2r and 2r + 1 (mod K) of row r are not zero: 1 and -1 (or second - 8)."""
    *lead, rows, K = shape
    qs = torch.full((*lead, rows, K // 32, 16), 0x88, dtype=torch.uint8, device="cuda")
    for r in range(rows):
        for k, code in ((2 * r % K, 9), ((2 * r + 1) % K, second)):
            byte = qs[..., r, k // 32, k % 16]
            byte.copy_((byte & 0xF0) | code if k % 32 < 16 else (byte & 0x0F) | code << 4)
    return qs, torch.ones(*lead, rows, K // 32, dtype=torch.float16, device="cuda")


@pytest.mark.parametrize("T,topk,E", [(1, 1, 1), (3, 2, 2), (8, 2, 3), (40, 1, 2), (64, 4, 4)])
@pytest.mark.parametrize("dt", DTYPES)
def test_down_of_vectors_that_all_but_cancel(T, topk, E, dt):
    """out = h[2r] - h[2r + 1], which differ from the 13th bit on: 22 bits of each leave a difference to 2^-9 of itself,
    11 bits leave none of it."""
    K, N = 96, 48
    r = Rand(T)
    qs, d = pairs(E, N, K)
    h = r.normal(T, topk, K).abs() + 1
    h[..., 1::2] = h[..., 0::2] * (1 + 2.0 ** -12 * (1 + torch.rand(T, topk, K // 2, generator=r.g, device="cuda")))
    a = dict(qs=qs, d=d, h=h, expert_ids=r.picks(T, topk, E), expert_weights=torch.softmax(r.normal(T, topk), -1))
    out = torch.empty(T, N, dtype=dt, device="cuda")
    q4.moe_q4_down_gemv(out, **a)
    z = h[..., 0::2].double() - h[..., 1::2].double()
    w = a["expert_weights"].double().unsqueeze(-1)
    want = (w * z).sum(1)
    # each element is held to 2^-22, their difference and the sums add at most topk + 4 half steps of fp32
    held = 2.0 ** -22 * (h[..., 0::2] + h[..., 1::2]).double()
    lim = (w * (held + (topk + 4) * ref.U * z.abs())).sum(1) + ref.rounded(want, dt) * (1 + 2.0 ** -7)
    off = (out.double() - want).abs()
    assert bool((off <= lim).all()), f"{float((off / lim).max()):.2f} of the limit"


@pytest.mark.parametrize("T,topk,E,N,K", [(1, 8, 8, 64, 96), (8, 8, 64, 256, 512), (64, 8, 16, 136, 352), (9, 2, 2, 72, 4128),
                                          (33, 1, 1, 200, 224)])
@pytest.mark.parametrize("dt", DTYPES)
def test_down_behind_a_residual_that_takes_it_away(T, topk, E, N, K, dt):
    """The residual is the sum's rounded opposite, so that the output shows what its own rounding hides otherwise."""
    a = down_case(T, topk, E, N, K, dt, residual=False)
    args = (a["h"].double(), torch.zeros_like(a["h"], dtype=torch.float64), lambda e: ref.q4_matrix(a["qs"][e], a["d"][e]),
            a["expert_ids"].long(), a["expert_weights"].double(), torch.zeros_like(a["expert_weights"], dtype=torch.float64))
    a["residual"] = -ref.down(*args, None, N)[0].to(dt)
    out = torch.empty(T, N, dtype=dt, device="cuda")
    q4.moe_q4_down_gemv(out, **a)
    want, err = ref.down(*args, a["residual"], N)
    off, lim = (out.double() - want).abs(), err + ref.rounded(want, dt) * (1 + 2.0 ** -7)
    assert bool((off <= lim).all()), f"{float((off / lim).max()):.2f} of the limit"


@pytest.mark.parametrize("T,topk,E,N,K", [(1, 1, 1, 32, 32), (5, 2, 3, 32, 64), (24, 1, 2, 64, 32), (64, 2, 2, 32, 32)])
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("norm", [True, False])
def test_layer_behind_a_residual_that_takes_it_away(T, topk, E, N, K, dt, norm):
    """As above, with the products' precision the same for every type of the layer."""
    a = layer_case(T, topk, E, N, K, dt, norm)
    a["residual"] = None
    _, ids, _ = run_layer(a)

    def exact(residual):  # x by its values: fp32 holds every type's
        return ref.layer(a["x"].float(), a["mats"], a["gamma"], 1e-6, residual, ids.long(), True)[0]

    a["residual"] = -exact(None)[0].to(dt)
    out, again, _ = run_layer(a)
    assert torch.equal(ids, again)
    want, err = exact(a["residual"])
    off, lim = (out.double() - want).abs(), err + ref.rounded(want, dt) * (1 + 2.0 ** -7)
    assert bool((off <= lim).all()), f"{float((off / lim).max()):.2f} of the limit"


@pytest.mark.parametrize("T", [1, 3, 40])
def test_bf16_layer_of_inputs_that_all_but_cancel(T):
    """A norm with weights of 24 bits in front of gate and up whose rows take differences of neighbouring elements."""
    K, N = 96, 32
    r = Rand(T)
    parts = dict(router=pairs(1, K), gate=pairs(1, N, K), up=pairs(1, N, K), down=pairs(1, K, N))
    parts["gate"][1].mul_(2048), parts["up"][1].mul_(2048)
    moe = q4.MoEWeights(*(t for pair in parts.values() for t in pair))
    x = (r.normal(T, K).abs() + 1).to(torch.bfloat16)
    x[:, 1::2] = x[:, 0::2]
    gamma = torch.ones(K, device="cuda")
    gamma[1::2] += 2.0 ** -12 * (1 + torch.rand(K // 2, generator=r.g, device="cuda"))
    out = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    q4.moe_q4_layer(out, x, moe, 1, gamma=gamma)
    v, _ = ref.rms(x.double(), torch.zeros(T, K, dtype=torch.float64, device="cuda"), gamma.double(), 1e-6)
    g = 2048 * (v[:, 0::2] - v[:, 1::2])[:, torch.arange(N) % (K // 2)]
    # v is off by 46 U (one number for a row, which the differences keep) and 4 U of its own, and held to 2^-22 (4 U)
    dg = 46 * ref.U * g.abs() + 2048 * 8 * ref.U * 2 * v.abs().amax(-1, keepdim=True)
    a = g * torch.sigmoid(g)
    h = a * g
    dh = 1.1 * dg * (g.abs() + dg) + a.abs() * dg + (10 + g.abs()) * ref.U * h.abs()
    down = torch.cat([h[:, 0::2] - h[:, 1::2]] * (K // (N // 2)), -1)[:, :K]
    err = torch.cat([(dh + 2.0 ** -22 * h.abs())[:, 0::2] + (dh + 2.0 ** -22 * h.abs())[:, 1::2]] * (K // (N // 2)), -1)[:, :K]
    lim = err + 6 * ref.U * down.abs() + ref.rounded(down, torch.bfloat16) * (1 + 2.0 ** -7)
    off = (out.double() - down).abs()
    assert bool((off <= lim).all()), f"{float((off / lim).max()):.2f} of the limit"


@pytest.mark.parametrize("T", [1, 40])
def test_norm_of_a_long_row_whose_first_squares_are_the_largest(T):
    """A large element in the first vector that a thread adds, and squares behind it that are less than half a step of it: one
    after the other they would all be lost, 127 half steps of the sum and as many again in silu(g) * u."""
    K, N = 32768, 32
    parts = {}
    for name, rows, cols in (("router", 1, K), ("gate", N, K), ("up", N, K), ("down", K, N)):
        qs = torch.full((1, rows, cols // 32, 16), 0x88, dtype=torch.uint8, device="cuda")
        qs[0, :, 0, 0] = 0x89  # each row takes its vector's first element
        parts[name] = qs, torch.ones(1, rows, cols // 32, dtype=torch.float16, device="cuda")
    parts["router"] = tuple(t[0] for t in parts["router"])
    x = torch.full((T, K), 2.0 ** -12 * (1 - 2.0 ** -10), device="cuda")
    x[:, :2048:8] = 1
    gamma, out = torch.ones(K, device="cuda"), torch.empty(T, K, device="cuda")
    q4.moe_q4_layer(out, x, q4.MoEWeights(*(t for pair in parts.values() for t in pair)), 1, gamma=gamma)
    g = 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6)
    want = g * torch.sigmoid(g) * g
    # The sum: at most 47 steps (halved by the root), 9 U for the root and the products, 4 U as it is held and 3 U more in each
    # of gate and up (41 U); their product has both, silu's slope being 1 here, and 10 U of its own; 7 U more in down.
    lim = (2 * (47 / 2 + 9 + 4 + 3) + 10 + 7) * ref.U * want
    assert bool(((out.double() - want).abs() <= lim).all()), f"{float(((out.double() - want).abs() / want).max() / ref.U):.1f} U"


@pytest.mark.parametrize("topk", [2, 4])
@pytest.mark.parametrize("T", [3, 64])
def test_infinite_logits(T, topk):
    """-infinity beside other logits: a share of zero, and the row that a very low logit gives. +infinity, or -infinity alone: a
    NaN row, of valid picks."""
    a = layer_case(T, topk, 4, 64, 96, torch.float32, norm=False)
    m = a["moe"]
    a["x"].abs_().add_(0.1)  # so that a block of equal codes has a sum of their sign
    m.router_qs[1] = 0x99
    m.router_d[1] = -60000.0  # a logit far below where a share is exactly zero
    want = run_layer(a)
    m.router_d[1, 0] = float("-inf")
    got = run_layer(a)
    assert all(torch.equal(g, w) for g, w in zip(got, want)) and bool(got[0].isfinite().all())
    assert bool((got[2][got[1] == 1] == 0).all()) and bool((got[1] == 1).any()) == (topk == 4)
    m.router_d[1, 0] = float("inf")
    out, ids, _ = run_layer(a)
    assert bool(out.isnan().all()) and bool(((ids >= 0) & (ids < 4)).all())
    m.router_qs[:] = 0x99
    m.router_d[:] = float("-inf")
    out, ids, _ = run_layer(a)
    assert bool(out.isnan().all()) and bool(((ids >= 0) & (ids < 4)).all())
    assert q4.q4_device_faults() == 0


def test_down_of_the_smallest_numbers():
    """Slots whose largest element lies near the least of fp32's range, subnormal ones among them."""
    a = down_case(9, 2, 3, 64, 288, torch.float32, residual=False)
    a["d"] = (a["d"].float() * 2.0 ** 21).half()  # whole numbers: what stays subnormal is exact but for the weighted sum
    top = a["h"].abs().amax(-1, keepdim=True)
    exponents = torch.tensor([-149, -140, -130, -127, -126, -125, -121, -118, -112], device="cuda", dtype=torch.float64)
    a["h"] = (a["h"].double() / top * torch.exp2(exponents)[:, None, None]).float()
    assert bool((a["h"].abs().amax(-1) > 0).all())
    out = torch.empty(9, 64, device="cuda")
    q4.moe_q4_down_gemv(out, **a)
    check_down(a, out)


@pytest.mark.parametrize("exponent", [-148, -140, -126, -125, -119, -112, 0, 100])
def test_down_holds_small_elements_beside_large_ones(exponent):
    """One element of 2^exponent or so, which scales its slot, beside smaller ones that the rows take alone."""
    K, N, T = 96, 48, 8
    r = Rand(exponent + 200)
    qs, d = pairs(1, N, K, second=8)
    d.mul_(8192)
    h = torch.rand(T, 1, K, generator=r.g, device="cuda", dtype=torch.float64) + 0.5
    h *= torch.exp2(torch.randint(-36, 1, h.shape, generator=r.g, device="cuda").double())
    h[..., 1] = 1.9
    h = (h * 2.0 ** exponent).float()
    out = torch.empty(T, N, device="cuda")
    one = torch.ones(T, 1, device="cuda")
    q4.moe_q4_down_gemv(out, qs, d, h, torch.zeros(T, 1, dtype=torch.int32, device="cuda"), one)
    want = 8192 * h[:, 0, 0::2].double()
    top = h.abs().amax(-1).double()
    # held to 2^-22 of itself or 2^-33 of the largest; one product, with 4 half steps for what is done to it
    lim = torch.maximum(2.0 ** -22 * want.abs(), 8192 * 2.0 ** -33 * top) + 4 * ref.U * want.abs() + 2 * ref.TINY[torch.float32]
    off = (out.double() - want).abs()
    assert bool((off <= lim).all()), f"{float((off / lim).max()):.2f} of the limit"


# Gate and up in every ring, with copies of 16, 8 and 2 bytes of scales and of few and many slots an expert. K of 4096 and 4224:
# two stages where slots are many, three where they are few; rows of an odd number of 128-column chunks (4224, 896, 1152, 1920),
# so that warps start and end on either half of a pair of chunks; enough rows that a ring goes round many times; parts of x
# that fit once (15360, 15488) or four times (7680, 7808).
FORMS = [(64, 4, 4, 512, 4096), (64, 4, 4, 512, 4224), (64, 2, 3, 256, 4128), (3, 1, 1, 1024, 4224), (2, 1, 1, 1024, 4096),
         (1, 2, 2, 512, 4224), (1, 2, 2, 512, 4096), (100, 2, 64, 96, 4224), (64, 8, 16, 64, 896), (64, 8, 16, 320, 1408),
         (48, 8, 16, 256, 1024), (5, 2, 6, 96, 1152), (12, 3, 40, 256, 1920), (12, 3, 40, 256, 2048), (24, 8, 32, 288, 640),
         (7, 2, 2, 64, 15360), (7, 2, 2, 64, 15488), (1, 1, 4, 96, 15488), (9, 2, 2, 96, 7680), (9, 2, 2, 96, 7808),
         (6, 1, 1, 32, 30976), (6, 1, 1, 32, 30848)]


@pytest.mark.parametrize("T,topk,E,N,K", FORMS)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_layer_in_every_form_of_its_products(T, topk, E, N, K, dt):
    a = layer_case(T, topk, E, N, K, dt, norm=False)
    out, ids, w = run_layer(a)
    by_value = dict(a, x=a["x"].float())  # the same precision for every type
    check_layer(by_value, out, ids, w, keep=list(range(0, T, max(1, T * topk // 48))))
    assert torch.equal(run_layer(a)[0], out)


@pytest.mark.parametrize("T,topk,E,N,K", [(12, 2, 6, 256, 1024), (13, 2, 8, 256, 1152), (9, 3, 8, 96, 672), (40, 3, 64, 96, 1920)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_layer_whose_tokens_meet_at_few_of_many_experts(T, topk, E, N, K, dt):
    """Tokens that are multiples of one another pick the same experts: full segments in the form for few slots an expert."""
    a = layer_case(T, topk, E, N, K, dt, norm=False)
    a["x"] = (a["x"][:1].float() * torch.linspace(0.5, 2, T, device="cuda")[:, None]).to(dt)
    out, ids, w = run_layer(a)
    assert bool((ids[0].sort().values == ids.sort(-1).values).all(-1).sum() > 8)
    check_layer(dict(a, x=a["x"].float()), out, ids, w)
    assert torch.equal(run_layer(a)[0], out)


@pytest.mark.parametrize("T,topk,E,N,K", [(5, 2, 6, 96, 1024), (48, 4, 4, 96, 1024), (64, 4, 4, 64, 4096)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_layer_with_scales_at_any_alignment(T, topk, E, N, K, dt):
    """Scales of one matrix 2, 4 and 8 bytes past a 16-byte boundary: other copies, the same bits."""
    a = layer_case(T, topk, E, N, K, dt, norm=False)
    m, want = a["moe"], run_layer(a)
    names = [f"{n}_{part}" for n in ("router", "gate", "up", "down") for part in ("qs", "d")]
    for name in ("gate_d", "up_d", "down_d"):
        for shift in (1, 2, 4):
            d = getattr(m, name)
            moved = torch.empty(d.numel() + 8, dtype=torch.float16, device="cuda")[shift:shift + d.numel()].view(d.shape)
            moved.copy_(d)
            moe = q4.MoEWeights(**dict({n: getattr(m, n) for n in names}, **{name: moved}))
            got = run_layer(dict(a, moe=moe))
            assert all(torch.equal(g, v) for g, v in zip(got, want)), (name, shift)
