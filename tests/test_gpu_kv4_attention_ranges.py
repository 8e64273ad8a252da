"""kv4_attention where its values, scores and scales lie far apart, and 16-bit types against what their roundings allow.

Tolerance of an output, with u = 2^-24, p = exp(score - largest), W = sum p 16 d over the scales d of the element's own
block, S = scale sum |q_i| 16 d_i of the token's key scales:
  - scores: off by e = (2 D + 32) u max S + 4 u max |score|, so weights by a factor within exp(+-2 e): 2 e sum p |v| / sum p;
  - the fp32 sum over n tokens, 16 or fewer at a step: (n / 4 + 64) u W / sum p, in which everything that is lost below the
    last bits of the terms lies too (n 2^-29 of the largest term, which is at most W / 16);
  - 16-bit types: a weight times its scale is one f16, half a step off, 2^-11 of it: 2^-11 sum p |v| / sum p;
  - half a step of the stored value."""

import numpy as np
import pytest
import torch

import kv4_ref as ref
from test_gpu_kv4_attention import Case

pytestmark = pytest.mark.gpu

import quantized_decode_gemv_q4_gb300 as q4  # noqa: E402

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ALL = [F32, F16, BF16]


def check(c, out):
    q, got = c.q.double().cpu().numpy(), out.double().cpu().numpy()
    B, M, Hq, D = q.shape
    g = Hq // c.Hkv
    for b, n in enumerate(c.lens):
        if n == 0:
            assert (got[b] == 0).all()
            continue
        t = np.arange(n)
        pages, offs = c.table[b][t // c.page], t % c.page
        for h in range(c.Hkv):
            k, v = (ref.cache_rows(qs, d, pages, offs, h) for qs, d in ((c.k_qs, c.k_d), (c.v_qs, c.v_d)))
            kd, vd = (np.repeat(np.abs(d[pages, h, offs]).astype(np.float64), 32, -1) for d in (c.k_d, c.v_d))
            for m in range(M):
                end = n - M + m + 1
                start = max(0, end - c.window) if c.window else 0
                rows = slice(h * g, h * g + g)
                if end <= start:
                    assert (got[b, m, rows] == 0).all()
                    continue
                x = q[b, m, rows]
                s = c.scale * (x @ k[start:end].T)
                e = (2 * D + 32) * ref.U * c.scale * 16 * (np.abs(x) @ kd[start:end].T).max(1) + 4 * ref.U * np.abs(s).max(1)
                p = np.exp(s - s.max(1, keepdims=True))
                total = p.sum(1, keepdims=True)
                y, size = p @ v[start:end] / total, p @ np.abs(v[start:end]) / total
                tol = 2 * e[:, None] * size + ((end - start) / 4 + 64) * ref.U * (p @ (16 * vd[start:end])) / total
                if c.dtype != F32:
                    tol = tol + 2.0 ** -11 * size
                tol = tol * (1 + 1e-2) + ref.half_step(c.dtype) * np.abs(y) + ref.subnormal(c.dtype)
                bad = ~(np.abs(got[b, m, rows] - y) <= tol)
                assert not bad.any(), (f"sequence {b}, query {m}, key head {h}: {bad.sum()} of {bad.size} off, e.g. "
                                       f"{got[b, m, rows][bad][:3]} for {y[bad][:3]} (tolerance {tol[bad][:3]})")


def every_token(c, b):
    t = np.arange(c.lens[b])
    return c.table[b][t // c.page], t % c.page


def put_key(c, b, t, score):
    """Token t's keys of every head give every query about this score (the queries are positive)."""
    pg, of = c.table[b][t // c.page], t % c.page
    x = abs(score) / (c.scale * c.q.double().sum(-1).mean().item())
    c.k_qs[pg, :, of] = 0xFF if score > 0 else 0x11  # codes 15 and 1: 7 and -7 times the scale
    c.k_d[pg, :, of] = np.float16(x / 7)


def positive(c):
    c.q = (c.q.abs() + 0.25).to(c.dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("spare", [1, 300, 2000])
@pytest.mark.parametrize("lens,M,Hq,Hkv,D,page,window", [
    ([4100, 9], 1, 8, 2, 128, 16, 0), ([4100, 64, 333], 1, 16, 1, 128, 16, 0), ([1500, 3000], 3, 4, 2, 64, 8, 0),
    ([2500], 4, 8, 2, 64, 16, 900), ([2100, 50], 1, 6, 2, 256, 32, 0), ([700, 31, 95, 64], 2, 10, 2, 256, 16, 500)])
def test_16_bit_types_are_off_by_their_roundings_only(lens, M, Hq, Hkv, D, page, window, spare, dtype):
    c = Case(lens, M, Hq, Hkv, D, page, dtype, window, spare=spare)
    check(c, c.run()[0])


GROUPS = [(1, 1), (1, 4), (3, 4)]  # queries of a sequence, heads of a group: one and two groups of 8 rows


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("spare", [1, 800])
@pytest.mark.parametrize("M,group", GROUPS)
@pytest.mark.parametrize("at", [3, 40, 98])  # in the first tile, a later one, among the last tokens
def test_a_large_value_of_no_weight(at, M, group, spare, D, dtype):
    """The other tokens' values keep their precision, whatever the scale of a token that weighs nothing."""
    c = Case([100, 700], M, 2 * group, 2, D, 16, dtype, spare=spare)
    positive(c)
    for b in range(2):
        pg, of = every_token(c, b)
        c.v_d[pg, :, of] *= np.float16(2.0 ** -9)
        put_key(c, b, at, -60.0)
        c.v_d[c.table[b][at // 16], :, at % 16] = 60000.0
    c.upload()
    check(c, c.run()[0])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("spare", [1, 800])
@pytest.mark.parametrize("M,group", GROUPS)
@pytest.mark.parametrize("at", [3, 40, 95])
def test_a_token_that_outweighs_the_rest_has_no_values_in_a_block(at, M, group, spare, D, dtype):
    """What is left in that block comes from weights of 1e-9 and keeps its own precision."""
    c = Case([100, 700], M, 2 * group, 2, D, 16, dtype, spare=spare)
    positive(c)
    for b in range(2):
        put_key(c, b, at, 24.0)
        c.v_d[c.table[b][at // 16], :, at % 16, 1] = 0.0
    c.upload()
    check(c, c.run()[0])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("spare", [1, 800])
@pytest.mark.parametrize("M,group", GROUPS)
@pytest.mark.parametrize("window", [0, 90])
def test_blocks_and_tokens_of_very_different_scales(window, M, group, spare, D, dtype):
    c = Case([100, 700], M, 2 * group, 2, D, 16, dtype, window, spare=spare)
    for b in range(2):
        pg, of = every_token(c, b)
        c.v_d[pg, :, of, 0] = np.float16(20000.0)
        c.v_d[pg, :, of, 1] *= np.float16(2.0 ** -12)
        c.v_d[pg[::7], :, of[::7]] = 0.0
        c.v_d[pg[1::7], :, of[1::7], 1] = np.float16(2.0 ** -24)
        c.v_d[pg[2::7], :, of[2::7]] *= np.float16(-1.0)  # a cache that something else filled
    c.upload()
    check(c, c.run()[0])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("spare", [1, 800])
@pytest.mark.parametrize("M,group", GROUPS)
@pytest.mark.parametrize("window", [0, 90])
def test_blocks_of_zeros_in_all_tokens_and_in_some(window, M, group, spare, D, dtype):
    """A block that is always zero (a padded head), and one that is zero in the first half, where the weight lies, or behind it."""
    for lo, hi in ((0, 10 ** 6), (0, 50), (50, 10 ** 6), (0, 32), (32, 64), (64, 10 ** 6)):
        c = Case([100, 700], M, 2 * group, 2, D, 16, dtype, window, spare=spare)
        positive(c)
        for b in range(2):
            pg, of = every_token(c, b)
            put_key(c, b, 30, 24.0)
            put_key(c, b, c.lens[b] - 20, 12.0)
            c.v_d[pg[lo:hi], :, of[lo:hi], 1] = 0.0
        c.upload()
        check(c, c.run()[0])


def test_a_cache_of_zero_and_of_subnormal_scales():
    for scale in (0.0, 2.0 ** -24, 2.0 ** -17):
        c = Case([100, 300], 1, 4, 2, 128, 16, F32)
        c.v_d[:] = np.where(np.isfinite(c.v_d), np.float16(scale), c.v_d)
        c.upload()
        check(c, c.run()[0])


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -20, 2.0 ** -8, 300.0])
@pytest.mark.parametrize("spare", [1, 100, 800])
@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 128), (F32, 256), (BF16, 64), (BF16, 128), (BF16, 256)])
@pytest.mark.parametrize("group", [1, 4])
def test_scales_and_scores_that_a_query_does_not_see_change_no_bit(group, dtype, D, spare, scale):
    """Tokens behind a query or before its window with any value scale, that weigh nothing or outweigh all others."""
    c = Case([50, 300], 3, 2 * group, 2, D, 16, dtype, window=80, spare=spare)
    positive(c)
    c.upload()
    out, lse = c.run()
    check(c, out)
    saved = [a.copy() for a in (c.k_qs, c.k_d, c.v_qs, c.v_d)]
    for back, others in ((1, [0, 1]), (80 + 2, [1, 2])):  # the newest token, seen by query 2; the oldest, seen by query 0
        for score in (-30.0, 30.0):
            for b, n in enumerate(c.lens):
                if n < back:
                    continue
                put_key(c, b, n - back, score)
                at = c.table[b][(n - back) // 16], slice(None), (n - back) % 16
                c.v_qs[at], c.v_d[at] = 0x1E, scale
            c.upload()
            got, got_lse = c.run()
            assert torch.equal(got[:, others], out[:, others]) and torch.equal(got_lse[:, others], lse[:, others])
            check(c, got)
            c.k_qs, c.k_d, c.v_qs, c.v_d = (a.copy() for a in saved)


@pytest.mark.parametrize("dtype", ALL)
def test_a_crowd_of_items_of_two_row_groups(dtype):
    """More than eight items an SM, each of more than 8 rows."""
    c = Case([(i * 13) % 90 for i in range(430)], 3, 12, 3, 64, 16, dtype)
    out, lse = c.run()
    c.check(out, lse)
    check(c, out)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("spare", [1, 800])
@pytest.mark.parametrize("group", [1, 12])
def test_scores_above_the_range_of_fp32_give_nan(group, spare, dtype):
    """In out and in lse, however the work is divided; other queries are as they were."""
    c = Case([90, 200], 2, 2 * group, 2, 64, 16, dtype, spare=spare, scale=0.125)
    positive(c)
    put_key(c, 1, 70, 1.0)
    c.upload()
    out, lse = c.run()
    check(c, out)
    c.q[1, 1, 1] *= 3e37
    put = c.table[1][70 // 16], slice(None), 70 % 16
    c.k_d[put] = 60000.0  # a score of 1e44 and more for that query
    c.upload()
    got, got_lse = c.run()
    assert torch.isnan(got[1, 1, 1]).all() and torch.isnan(got_lse[1, 1, 1])
    assert torch.equal(got[0], out[0]) and torch.equal(got_lse[0], lse[0])
    assert torch.isfinite(got[1, 0]).all() and torch.isfinite(got[1, 1, 0]).all()


def test_windows_past_the_c_abi_s_integers():
    c = Case([40, 300], 2, 4, 2, 64, 16, F32)
    out, _ = c.run()
    for window in (2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 70):
        c.window = window
        assert torch.equal(c.run()[0], out)
    for window in (-1, -2 ** 32 + 5, -2 ** 40):
        c.window = window
        with pytest.raises(q4.Q4Error, match="window"):
            c.run()
