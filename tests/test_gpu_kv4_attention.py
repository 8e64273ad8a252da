"""kv4_attention on the GPU against attention in 64 bits over the same cached values (tolerances: kv4_ref.attention,
plus the weights' half step in fp16 for 16-bit types and half a step of the stored value)."""

import numpy as np
import pytest
import torch

import kv4_ref as ref

pytestmark = pytest.mark.gpu

import quantized_decode_gemv_q4_gb300 as q4  # noqa: E402

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


class Case:
    def __init__(self, lens, M, Hq, Hkv, D, page, dtype, window=0, seed=0, scale=None, spread=1.0, spare=2):
        rng = np.random.default_rng(seed + sum(lens) + D)
        B = len(lens)
        per = [-(-n // page) for n in lens]
        pages = sum(per) + 3
        order = rng.permutation(pages).astype(np.int32)
        width = max(per) + spare
        # entries past a sequence's pages are never looked at
        self.table = np.full((B, width), 2 ** 30, np.int32)
        self.k_qs = rng.integers(0, 256, (pages, Hkv, page, D // 2), dtype=np.uint8)
        self.v_qs = rng.integers(0, 256, (pages, Hkv, page, D // 2), dtype=np.uint8)
        self.k_d = np.full((pages, Hkv, page, D // 32), np.nan, np.float16)  # what no sequence has written
        self.v_d = np.full((pages, Hkv, page, D // 32), np.inf, np.float16)
        at = 0
        for b, n in enumerate(lens):
            self.table[b, :per[b]] = order[at:at + per[b]]
            at += per[b]
            t = np.arange(n)
            pg, of = self.table[b][t // page], t % page
            for qs, d, size in ((self.k_qs, self.k_d, spread), (self.v_qs, self.v_d, 1.0)):
                x = rng.standard_normal((n, Hkv, D)) * size
                x[..., rng.integers(0, D, 2)] *= 5
                qs[pg, :, of], d[pg, :, of] = ref.quantise(x)
        self.lens, self.M, self.Hq, self.Hkv, self.D, self.page, self.dtype, self.window = lens, M, Hq, Hkv, D, page, dtype, window
        self.scale = D ** -0.5 if scale is None else scale
        self.q = torch.from_numpy(rng.standard_normal((B, M, Hq, D))).to(dtype).cuda()
        self.upload()

    def upload(self):
        self.cache = q4.KV4Cache(*(torch.from_numpy(a).cuda() for a in (self.k_qs, self.k_d, self.v_qs, self.v_d)))
        self.dtable = torch.from_numpy(self.table).cuda()
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        B = len(self.lens)
        buf = torch.full((B * self.M + 2, self.Hq, self.D), 9.0, dtype=self.dtype, device="cuda")
        out = buf[1:-1].view(B, self.M, self.Hq, self.D)
        lse = torch.full((B, self.M, self.Hq), 9.0, device="cuda")
        q4.kv4_attention(out, self.q, self.cache, self.dtable, self.dlens, scale=self.scale, window=self.window, lse=lse, **kw)
        torch.cuda.synchronize()
        assert (buf[0] == 9).all() and (buf[-1] == 9).all(), "written outside the output"
        return out, lse

    def check(self, out, lse, rows=slice(None)):
        y, l, tol, tol_lse = ref.attention(self.q.double().cpu().numpy(), self.k_qs, self.k_d, self.v_qs, self.v_d, self.table,
                                           self.lens, self.scale, self.window)
        if self.dtype != F32:
            # 16-bit types: the weights are rounded to f16 (2^-12 of the largest |v| a weight meets, 8 steps)
            vd = np.nan_to_num(np.where(np.isfinite(self.v_d), self.v_d, 0)).astype(np.float64).max()
            tol = tol + 2.0 ** -12 * np.where(np.isinf(l), 0, 8 * vd)[..., None]
        tol = tol + ref.half_step(self.dtype) * 1.001 * np.abs(y) + ref.subnormal(self.dtype)
        got = out.double().cpu().numpy()
        bad = ~(np.abs(got - y) <= tol)[rows]
        assert not bad.any(), f"{bad.sum()} of {bad.size} off, e.g. {got[rows][bad][:3]} for {y[rows][bad][:3]} (tolerance {tol[rows][bad][:3]})"
        g = lse.double().cpu().numpy()
        empty = np.isinf(l)
        assert np.array_equal(g[rows][empty[rows]], l[rows][empty[rows]])
        seen = ~empty[rows]
        assert (np.abs(g[rows][seen] - l[rows][seen]) <= tol_lse[rows][seen]).all(), "lse"
        assert (got[rows][empty[rows]] == 0).all()


SHAPES = [
    # lens, M, Hq, Hkv, D, page, window
    ([1], 1, 1, 1, 64, 16, 0),
    ([100], 1, 28, 4, 128, 16, 0),
    ([0, 1, 2, 31, 32, 33, 64, 65, 127, 128, 129], 1, 8, 2, 128, 16, 0),
    ([5, 0, 300], 1, 7, 1, 256, 1, 0),
    ([777, 12], 1, 32, 4, 64, 64, 0),
    ([257, 1, 3], 4, 8, 8, 128, 8, 0),       # queries that see nothing: M > length
    ([500, 40, 2], 5, 14, 2, 64, 32, 37),     # a sliding window
    ([90], 16, 16, 2, 128, 256, 1),           # a window of one token, 128 rows a key head
    ([1000], 3, 40, 1, 256, 2, 0),            # 120 rows on one key head
    ([4100, 9], 1, 16, 1, 128, 16, 4000),
    ([3000, 2999], 2, 5, 5, 64, 16, 0),
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("wide", [0, 5000, 20000])  # tokens that the page table admits beyond the longest sequence
@pytest.mark.parametrize("lens,M,Hq,Hkv,D,page,window", SHAPES)
def test_matches_64_bits(lens, M, Hq, Hkv, D, page, window, wide, dtype):
    assert q4.q4_device_faults() == 0
    c = Case(lens, M, Hq, Hkv, D, page, dtype, window, spare=wide // page + 1)
    out, lse = c.run()
    c.check(out, lse)
    assert q4.q4_device_faults() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("spare", [1, 100, 800])
def test_many_sequences_of_all_lengths(dtype, spare):
    lens = [(i * 37) % 211 for i in range(150)]
    c = Case(lens, 1, 6, 2, 64, 16, dtype, spare=spare)
    out, lse = c.run(workspace=q4.kv4_attention_workspace(c.q, c.cache))
    c.check(out, lse)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,M,Hq,Hkv,D", [(120, 1, 12, 4, 128), (330, 1, 8, 4, 128), (200, 3, 12, 3, 64), (410, 2, 6, 3, 64),
                                          (160, 1, 8, 8, 256)])
def test_many_and_crowded_items(B, M, Hq, Hkv, D, dtype):
    """Hundreds to thousands of (sequence, key head) items of short sequences, in whole items and as streams."""
    c = Case([(i * 13) % 90 for i in range(B)], M, Hq, Hkv, D, 16, dtype)
    out, lse = c.run()
    c.check(out, lse)
    c.table = np.concatenate([c.table, np.full((B, 600), 2 ** 30, np.int32)], 1)
    c.upload()
    c.check(*c.run())


@pytest.mark.parametrize("spare", [1, 100, 800])
def test_the_most_sequences(spare):
    c = Case([(i * 7) % 40 for i in range(1024)], 1, 2, 1, 64, 16, F32, spare=spare)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", [F32, F16])
def test_sharp_softmax_and_a_wide_range_of_values(dtype):
    """Scores tens apart, and value scales 2^20 apart between tokens."""
    c = Case([700, 45], 1, 8, 2, 128, 16, dtype, spread=12.0)
    c.check(*c.run())
    for b, n in enumerate(c.lens):
        t = np.arange(n)
        pg, of = c.table[b][t // c.page], t % c.page
        c.v_d[pg, :, of] *= (2.0 ** ((t * 5) % 21 - 14)).astype(np.float16)[:, None, None]
    c.upload()
    c.check(*c.run())


def test_zero_queries_and_zero_values():
    c = Case([90], 1, 4, 2, 128, 16, F32)
    c.q.zero_()
    c.check(*c.run())
    c.v_qs[:] = 0x88
    c.v_d[:] = np.where(np.isfinite(c.v_d), c.v_d, 1.0)
    c.upload()
    out, _ = c.run()
    assert (out.abs() <= 1e-5).all()
    c.v_d[:] = 0
    c.upload()
    out, lse = c.run()
    assert (out == 0).all()
    c.check(out, lse)


def test_large_and_small_queries():
    for size in (1e-20, 1e15):
        c = Case([60], 1, 4, 2, 64, 16, F32, scale=0.125 / size)
        c.q.mul_(size)
        c.check(*c.run())


@pytest.mark.parametrize("spare", [1, 100, 800])
def test_a_nan_reaches_only_the_queries_that_see_it(spare):
    c = Case([50, 50], 3, 4, 2, 128, 16, BF16, window=20, spare=spare)
    b, t = 0, 48  # the newest but one: query 0 does not see it, nor does a token behind the window count
    c.k_d[c.table[b][t // 16], 1, t % 16, 2] = np.nan
    c.v_d[c.table[1][49 // 16], 0, 49 % 16, 0] = np.nan
    for bb in (0, 1):
        c.k_d[c.table[bb][3 // 16], :, 3] = np.nan
        c.v_d[c.table[bb][3 // 16], :, 3] = np.inf
    c.upload()
    out, lse = c.run()
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros((2, 3, 4, 128), bool)
    want[0, 1:, 2:] = True  # heads of key head 1
    want[1, 2, :2, :32] = True  # values: only the block whose scale it is
    assert np.array_equal(nan[0], want[0])
    assert nan[1][want[1]].all() and not nan[1, :2].any() and not nan[1, 2, 2:].any()
    c.q[1, 0, 0, 5] = float("inf")
    c.q[1, 1, 1, 6] = float("nan")
    out, _ = c.run()
    assert torch.isnan(out[1, 0, 0]).all() and torch.isnan(out[1, 1, 1]).all() and torch.isfinite(out[1, 0, 1:]).all()


@pytest.mark.parametrize("scale", [np.nan, 65504.0])
@pytest.mark.parametrize("spare", [1, 100, 800])
@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 128), (F32, 256), (BF16, 64), (BF16, 128), (BF16, 256)])
@pytest.mark.parametrize("group", [1, 4])
def test_what_a_query_does_not_see_changes_no_bit(group, dtype, D, spare, scale):
    """Values of about 1e-3, and tokens behind a query or before its window with any scales, codes and NaN."""
    c = Case([50, 300], 3, 2 * group, 2, D, 16, dtype, window=20, spare=spare)
    c.v_d[:] = np.where(np.isfinite(c.v_d), c.v_d * np.float16(2.0 ** -9), c.v_d)
    c.upload()
    out, lse = c.run()
    c.check(out, lse)
    for back, others in ((1, [0, 1]), (20 + 2, [1, 2])):  # the newest token, seen by query 2; the oldest, seen by query 0
        saved = [a.copy() for a in (c.k_qs, c.k_d, c.v_qs, c.v_d)]
        for b, n in enumerate(c.lens):
            at = c.table[b][(n - back) // 16], slice(None), (n - back) % 16
            c.k_qs[at], c.v_qs[at], c.k_d[at], c.v_d[at] = 0xF0, 0x1E, scale, scale
        c.upload()
        got, got_lse = c.run()
        assert torch.equal(got[:, others], out[:, others]) and torch.equal(got_lse[:, others], lse[:, others])
        c.k_qs, c.k_d, c.v_qs, c.v_d = saved


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_nan_block_of_values_leaves_the_other_blocks_as_accurate(dtype):
    c = Case([70], 1, 4, 2, 128, 16, dtype)
    c.v_d[:] = np.where(np.isfinite(c.v_d), c.v_d * np.float16(2.0 ** -9), c.v_d)
    c.v_d[c.table[0][2], 1, 5, 2] = np.nan
    c.upload()
    out, lse = c.run()
    assert torch.isnan(out[:, :, 2:, 64:96]).all()
    out[:, :, 2:, 64:96] = 0
    c.v_d[:, 1, :, 2] = 0  # the expected values of that block are zeros
    c.check(out, lse)


@pytest.mark.parametrize("spare", [1, 100, 800])
def test_bad_pages_and_lengths_are_recorded(spare):
    c = Case([100, 60, 40, 70], 1, 4, 2, 64, 16, F32, spare=spare)
    c.check(*c.run())
    assert q4.q4_device_faults() == 0
    c.dtable[1, 2] = -1
    out, lse = c.run()
    assert q4.q4_device_faults() == q4.FAULT_BAD_PAGE
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    c.check(out, lse, rows=[0, 2, 3])
    c.dtable[1, 2] = c.cache.num_pages
    out, lse = c.run()
    assert q4.q4_device_faults() == q4.FAULT_BAD_PAGE and torch.isnan(out[1]).all()
    c.upload()
    c.dlens[2], c.dlens[0] = -3, c.table.shape[1] * c.page + 1
    out, lse = c.run()
    assert q4.q4_device_faults() == q4.FAULT_BAD_LENGTH
    assert torch.isnan(out[[0, 2]]).all()
    c.check(out, lse, rows=[1, 3])


@pytest.mark.parametrize("spare", [1, 800])
def test_windows_past_every_sequence_are_none(spare):
    c = Case([1, 40, 0, 9], 16, 2, 1, 64, 16, F32, spare=spare)
    out, lse = c.run()
    c.check(out, lse)
    for window in (c.table.shape[1] * c.page, 2 ** 30, 2 ** 31 - 1):
        c.window = window
        again, lse2 = c.run()
        assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,M,Hq,Hkv,D,longest,window", [
    (52, 3, 12, 4, 64, 2700, 1400),   # many items of more than a thousand tokens each
    (45, 1, 8, 4, 128, 1600, 1030),
    (3, 2, 4, 2, 64, 9300, 8300),     # few, of more tokens than are split between CTAs
    (3, 2, 4, 2, 64, 9300, 700),
    (40, 2, 10, 5, 128, 1500, 1023),  # most that is read: 1024 tokens
    (40, 2, 10, 5, 128, 1500, 1024),
])
def test_windows_over_many_and_long_sequences(B, M, Hq, Hkv, D, longest, window, dtype):
    lens = [longest * ((7 * i) % B + 1) // B for i in range(B)]
    lens[0], lens[1] = longest, 1
    c = Case(lens, M, Hq, Hkv, D, 16, dtype, window)
    c.check(*c.run())


def test_many_heads_and_rows():
    """More query heads than a CTA's rows many times over, and a key head for each query head."""
    c = Case([70, 3], 2, 192, 2, 64, 16, BF16)
    c.check(*c.run())
    c = Case([45], 1, 96, 96, 64, 16, F16)
    c.check(*c.run())


def test_strided_queries_and_one_token_form():
    c = Case([130, 7], 1, 8, 2, 64, 16, BF16)
    out, _ = c.run()
    wide = torch.zeros(2, 12, 64, dtype=BF16, device="cuda")
    wide[:, :8] = c.q[:, 0]
    res = torch.zeros(2, 9, 64, dtype=BF16, device="cuda")
    q4.kv4_attention(res[:, 1:], wide[:, :8], c.cache, c.dtable, c.dlens)
    assert torch.equal(res[:, 1:], out[:, 0]) and (res[:, 0] == 0).all()


def test_twice_the_same_bits_on_another_stream_and_in_a_graph():
    c = Case([2000, 0, 333, 1], 2, 16, 4, 128, 16, BF16)
    out, lse = c.run()
    again, lse2 = c.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other, olse = torch.empty_like(out), torch.empty_like(lse)
    q4.kv4_attention(other, c.q, c.cache, c.dtable, c.dlens, scale=c.scale, lse=olse, stream=s)
    q4.kv4_attention(other, c.q, c.cache, c.dtable, c.dlens, scale=c.scale, lse=olse, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(out, other) and torch.equal(lse, olse)
    # two graphs over one workspace, replayed in turn; the lengths change between replays
    ws = q4.kv4_attention_workspace(c.q, c.cache)
    outs, graphs = [torch.empty_like(out) for _ in range(2)], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q4.kv4_attention(o, c.q, c.cache, c.dtable, c.dlens, scale=c.scale, workspace=ws)
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)
    c.lens = [1500, 0, 3, 1]
    c.dlens.copy_(torch.tensor(c.lens, dtype=torch.int32))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    c.check(*c.run())
    assert torch.equal(outs[0], c.run()[0])


def test_two_calls_at_once_with_a_workspace_each():
    cases = [Case([3000, 500], 1, 28, 4, 128, 16, F32), Case([2500, 900, 17], 1, 16, 8, 64, 32, F32)]
    alone = [c.run()[0] for c in cases]
    spaces = [q4.kv4_attention_workspace(c.q, c.cache) for c in cases]
    outs = [[torch.empty_like(a) for _ in range(8)] for a in alone]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for i in range(8):
        for c, ws, o, s in zip(cases, spaces, outs, streams):
            q4.kv4_attention(o[i], c.q, c.cache, c.dtable, c.dlens, scale=c.scale, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for a, os_ in zip(alone, outs):
        assert all(torch.equal(a, o) for o in os_)


def test_pages_behind_2_to_the_32_bytes():
    H, D, page = 8, 256, 4
    pages = (1 << 32) // (H * D // 2 * page) + 40
    cache = q4.KV4Cache.allocate(pages, page, H, D)
    n = 50
    where = np.concatenate([np.arange(pages - 7, pages), np.arange(0, 6)]).astype(np.int32)
    table = torch.from_numpy(where[None].copy()).cuda()
    k, v = torch.randn(n, H, D, device="cuda"), torch.randn(n, H, D, device="cuda")
    t = torch.arange(n, device="cuda")
    q4.kv4_write(cache, k, v, (table[0][t // page] * page + t % page).int())
    small = q4.KV4Cache.allocate(len(where), page, H, D)
    q4.kv4_write(small, k, v, t.int())
    q = torch.randn(1, 8, D, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, want = torch.empty_like(q), torch.empty_like(q)
    q4.kv4_attention(out, q, cache, table, lens)
    q4.kv4_attention(want, q, small, torch.arange(len(where), dtype=torch.int32, device="cuda")[None], lens)
    assert torch.equal(out, want) and torch.isfinite(out).all()
