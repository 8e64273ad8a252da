"""qk_norm_rope on the GPU against the 64-bit formula.

Tolerance, with u = 2^-24: the sum of D squares is off by at most D u of itself (half of it after the root), the mean,
eps and root add 6 u, the factors r, gamma, cos and the difference 4 u: (D / 2 + 10) u of |a cos| + |b sin|, and the
stored value half a step of its type."""

import numpy as np
import pytest
import torch

import kv4_ref as ref

pytestmark = pytest.mark.gpu

import quantized_decode_gemv_q4_gb300 as q4  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def table(rot, far=5000, base=10000.0):
    a = np.arange(far)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def check(got, x, gamma, eps, cs, pos, inter, dtype, what):
    y, size = ref.rope(x, gamma, eps, cs, pos, inter)
    got = got.double().cpu().numpy()
    D = x.shape[-1]
    tol = (D / 2 + 10) * ref.U * size + ref.half_step(dtype) * (1 + 1e-3) * np.abs(y) + ref.subnormal(dtype)
    bad = ~(np.abs(got - y) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} off, first {got[bad][:3]} for {y[bad][:3]}"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,norm", [
    (1, 28, 4, 128, 128, False, True), (3, 4, 4, 64, 64, True, True), (5, 7, 1, 96, 96, False, True),
    (2, 3, 1, 32, 16, True, True), (7, 8, 2, 256, 256, False, True), (4, 6, 3, 160, 80, False, False),
    (33, 40, 8, 128, 64, True, False), (2, 5, 5, 192, 176, False, True), (600, 2, 1, 64, 32, False, True),
    (3, 2, 1, 224, 224, True, True),
    (4099, 28, 6, 128, 128, False, True), (5001, 9, 3, 256, 64, True, True), (12345, 13, 1, 64, 64, False, False)])  # many rows
def test_matches_the_formula(dtype, T, Hq, Hkv, D, rot, inter, norm):
    g = torch.Generator().manual_seed(T * 1000 + D + rot)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda()
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]  # strided rows
    gq = (1 + 0.2 * torch.randn(D, generator=g)).cuda() if norm else None
    gk = (1 + 0.2 * torch.randn(D, generator=g)).cuda() if norm else None
    cs = table(rot)
    pos = torch.randint(0, cs.shape[0], (T,), generator=g, dtype=torch.int32)
    pos[0], pos[-1] = 0, cs.shape[0] - 1
    qo, ko = torch.full((T, Hq, D), 7.0, dtype=dtype, device="cuda"), torch.full((T + 1, Hkv, D), 7.0, dtype=dtype, device="cuda")
    before = qkv.clone()
    q4.qk_norm_rope(qo, ko[:T], q, k, gq, gk, torch.from_numpy(cs).cuda(), pos.cuda(), eps=1e-5, interleaved=inter)
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    for got, x, gam, what in ((qo, q, gq, "q"), (ko[:T], k, gk, "k")):
        check(got, host(x), None if gam is None else gam.cpu().numpy(), 1e-5, cs, pos.numpy(), inter, dtype, what)
    assert torch.equal(qkv, before) and torch.all(ko[T] == 7.0)
    # the same in place, and without a rotation
    q4.qk_norm_rope(q, k, q, k, gq, gk, torch.from_numpy(cs).cuda(), pos.cuda(), eps=1e-5, interleaved=inter)
    assert torch.equal(q, qo) and torch.equal(k, ko[:T]) and torch.equal(qkv[:, Hq + Hkv:], before[:, Hq + Hkv:])
    x = before[:, :Hq]
    q4.qk_norm_rope(qo, ko[:T], x, before[:, Hq:Hq + Hkv], gq, gk, None, None, eps=1e-5)
    check(qo, host(x), None if gq is None else gq.cpu().numpy(), 1e-5, None, None, False, dtype, "norm alone")


def test_zero_rows_infinities_and_bad_positions():
    T, H, D = 4, 2, 64
    x = torch.randn(T, H, D, device="cuda")
    x[0] = 0
    x[1, 0, 40] = float("inf")
    cs = torch.from_numpy(table(32)).cuda()
    gamma = torch.ones(D, device="cuda")
    pos = torch.tensor([3, 4, -1, cs.shape[0]], dtype=torch.int32, device="cuda")
    out, k_out = torch.empty_like(x), torch.empty_like(x)
    assert q4.q4_device_faults() == 0
    q4.qk_norm_rope(out, k_out, x, x, None, None, cs, pos)
    assert q4.q4_device_faults() == q4.FAULT_BAD_POSITION
    assert torch.all(out[0] == 0) and torch.isnan(out[2:]).all()
    assert out[1, 0, 40] == float("inf") and torch.isfinite(out[1]).sum() == H * D - 1  # behind rot_dim: as it came
    q4.qk_norm_rope(out, k_out, x, x, gamma, gamma, cs, pos.clamp(0, 5), eps=1e-6)
    assert torch.all(out[0] == 0) and q4.q4_device_faults() == 0
    assert torch.isfinite(out[2:]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("side", ["q", "k"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter", [
    (1, 7, 1, 128, 128, False), (3, 5, 3, 64, 32, True), (5, 1, 1, 32, 32, False), (2, 3, 2, 96, 96, True), (4, 2, 1, 256, 256, False),
    (9, 1, 6, 160, 0, False), (4099, 30, 6, 128, 128, False), (12345, 13, 1, 64, 64, True), (5001, 9, 3, 256, 64, False)])  # many rows
def test_a_norm_on_one_side_only(dtype, T, Hq, Hkv, D, rot, inter, side):
    """Query and key heads that share a warp, one of them without a norm."""
    g = torch.Generator().manual_seed(T + Hq + D)
    q, k = (torch.randn(T, H, D, generator=g).to(dtype).cuda() for H in (Hq, Hkv))
    gamma = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    gq, gk = (gamma, None) if side == "q" else (None, gamma)
    cs = table(rot) if rot else None
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    q4.qk_norm_rope(qo, ko, q, k, gq, gk, None if cs is None else torch.from_numpy(cs).cuda(), None if cs is None else pos.cuda(),
                    eps=1e-5, interleaved=inter)
    for got, x, gam, what in ((qo, q, gq, "q"), (ko, k, gk, "k")):
        check(got, x.double().cpu().numpy(), None if gam is None else gam.cpu().numpy(), 1e-5, cs, pos.numpy(), inter, dtype, what)
