"""kv4_write and kv4_read on the GPU: bytes equal the 64-bit definition's, values equal the stored ones rounded once."""

import numpy as np
import pytest
import torch

import kv4_ref as ref

pytestmark = pytest.mark.gpu

import quantized_decode_gemv_q4_gb300 as q4  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def junk_cache(pages, page, H, D):
    c = q4.KV4Cache.allocate(pages, page, H, D)
    for t in (c.k_qs, c.v_qs):
        t.fill_(0xA5)
    for t in (c.k_d, c.v_d):
        t.fill_(3.0)
    return c


def host(c):
    return [t.cpu().numpy().copy() for t in (c.k_qs, c.k_d, c.v_qs, c.v_d)]


def same_halves(a, b):
    nan = np.isnan(a) & np.isnan(b)
    return np.array_equal(a.view(np.uint16)[~nan], b.view(np.uint16)[~nan])


def expect(before, k, v, slots, page):
    k_qs, k_d, v_qs, v_d = before
    for x, qs, d in ((k, k_qs, k_d), (v, v_qs, v_d)):
        c, s = ref.quantise(x.double().cpu().numpy())
        for t, slot in enumerate(slots):
            if 0 <= slot < qs.shape[0] * page:
                qs[slot // page, :, slot % page] = c[t]
                d[slot // page, :, slot % page] = s[t]
    return k_qs, k_d, v_qs, v_d


def roundtrip(k, v, slots, pages, page):
    T, H, D = k.shape
    cache = junk_cache(pages, page, H, D)
    want = expect(host(cache), k, v, slots, page)
    sl = torch.tensor(slots, dtype=torch.int32, device="cuda")
    q4.kv4_write(cache, k, v, sl)
    got = host(cache)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[2], want[2]), "codes"
    assert same_halves(got[1], want[1]) and same_halves(got[3], want[3]), "scales"
    for dtype in TYPES:
        ko, vo = (torch.full((T, H, D), 9.0, dtype=dtype, device="cuda") for _ in range(2))
        q4.kv4_read(ko, vo, cache, sl)
        for out, qs, d in ((ko, want[0], want[1]), (vo, want[2], want[3])):
            y = np.full((T, H, D), 9.0)
            for t, slot in enumerate(slots):
                if slot >= 0:
                    y[t] = ref.values(qs[slot // page, :, slot % page], d[slot // page, :, slot % page])
            y = torch.from_numpy(y).float().to(dtype)  # (code - 8) d has 15 bits: exact in fp32, then one rounding
            assert torch.equal(torch.nan_to_num(out.cpu(), nan=-1), torch.nan_to_num(y, nan=-1))
        only = torch.full((T, H, D), 9.0, dtype=dtype, device="cuda")
        q4.kv4_read(None, only, cache, sl)
        assert torch.equal(torch.nan_to_num(only, nan=-1), torch.nan_to_num(vo, nan=-1))
    return cache


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 32, 1), (1, 4, 128, 16), (5, 1, 32, 4), (37, 5, 32, 8), (19, 8, 128, 16),
                                        (9, 3, 96, 64), (130, 2, 256, 32), (3, 31, 160, 2), (301, 1, 64, 256)])
def test_write_and_read(dtype, T, H, D, page):
    rng = np.random.default_rng(T + H + D + page)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].tolist()
    if T > 3:
        slots[1] = slots[-1] = -1
    kv = torch.from_numpy(rng.standard_normal((T, 2 * H + 1, D))).to(dtype).cuda()  # k and v as strided columns
    roundtrip(kv[:, :H], kv[:, H + 1:], slots, pages, page)


@pytest.mark.parametrize("dtype", TYPES)
def test_values_at_the_borders(dtype):
    """Ties, values a rounding away from them, zeros, subnormals, the largest and non-finite values."""
    rng = np.random.default_rng(5)
    x = np.zeros((64, 2, 64), np.float64)
    for t in range(40):
        for h in range(2):
            for b in range(2):
                d = np.float64(np.float16(rng.uniform(0.01, 4) * 2.0 ** rng.integers(-12, 8)))
                y = (rng.integers(-7, 7, 32) + 0.5) * d  # ties
                y = y.astype(np.float32)
                if t % 2:
                    y = np.nextafter(y, np.where(rng.random(32) < 0.5, -1e30, 1e30).astype(np.float32))
                y[rng.integers(32)] = 7 * d * rng.choice([-1, 1])
                x[t, h, 32 * b:32 * b + 32] = y
    x[41] = 1e-30
    x[42] = 2.0 ** -25 * 7 * rng.choice([-1, 0.49, 0.5, 0.51, 1], (2, 64))
    x[43] = rng.standard_normal((2, 64)) * 1e-7
    x[44, 0, 3] = np.inf
    x[45, 1, 40] = -np.inf
    x[46, 0, 33] = np.nan
    x[47] = rng.standard_normal((2, 64)) * (3e38 if dtype != torch.float16 else 3e4)
    x[48] = 6e4 * rng.choice([-1, 1, 0.3], (2, 64))
    x[49, 0, 5] = -1.0
    k = torch.from_numpy(x).to(dtype).cuda()
    v = torch.from_numpy(x[::-1].copy()).to(dtype).cuda()
    roundtrip(k, v, list(range(63, -1, -1)), 8, 8)


def test_a_million_values_round_as_in_64_bits():
    rng = np.random.default_rng(6)
    x = rng.standard_normal((1024, 8, 128)).astype(np.float32)
    roundtrip(torch.from_numpy(x).cuda(), torch.from_numpy(x[::-1].copy() * 1e-3).cuda(), list(range(1024)), 64, 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,D,page", [(8211, 8, 128, 16), (33001, 1, 256, 64), (5003, 21, 96, 4)])
def test_many_rows(dtype, T, H, D, page):
    """Enough rows for several tokens a thread, a last group that is not full, some without a slot."""
    rng = np.random.default_rng(T)
    pages = -(-T // page) + 1
    slots = rng.permutation(pages * page)[:T]
    slots[rng.integers(0, T, 50)] = -1
    kv = torch.from_numpy(rng.standard_normal((T, 2 * H, D)).astype(np.float32)).to(dtype).cuda()
    cache = junk_cache(pages, page, H, D)
    before = host(cache)
    sl = torch.from_numpy(slots.astype(np.int32)).cuda()
    q4.kv4_write(cache, kv[:, :H], kv[:, H:], sl)
    got, there = host(cache), slots >= 0
    pg, of = slots[there] // page, slots[there] % page
    outs = [torch.full((T, H, D), 9.0, dtype=dtype, device="cuda") for _ in range(2)]
    q4.kv4_read(*outs, cache, sl)
    for x, qs, d, was_qs, was_d, out in ((kv[:, :H], got[0], got[1], before[0], before[1], outs[0]),
                                         (kv[:, H:], got[2], got[3], before[2], before[3], outs[1])):
        c, s = ref.quantise(x.double().cpu().numpy()[there])
        was_qs[pg, :, of], was_d[pg, :, of] = c, s
        assert np.array_equal(qs, was_qs) and same_halves(d, was_d)
        want = torch.full((T, H, D), 9.0, dtype=dtype)
        want[torch.from_numpy(there)] = torch.from_numpy(ref.values(c, s)).float().to(dtype)
        assert torch.equal(out.cpu(), want)


def test_bad_slots_are_recorded_and_written_nowhere():
    H, D, page, pages = 2, 64, 8, 3
    k = torch.randn(4, H, D, device="cuda")
    assert q4.q4_device_faults() == 0
    cache = junk_cache(pages, page, H, D)
    want = expect(host(cache), k, k, [3, 24, -5, 2 ** 31 - 1], page)
    sl = torch.tensor([3, 24, -5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    q4.kv4_write(cache, k, k, sl)
    assert q4.q4_device_faults() == q4.FAULT_BAD_SLOT
    got = host(cache)
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    out = torch.full((4, H, D), 9.0, device="cuda")
    q4.kv4_read(out, None, cache, sl)
    assert q4.q4_device_faults() == q4.FAULT_BAD_SLOT
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1]).all() and (out[2] == 9).all() and torch.isnan(out[3]).all()


def test_the_same_slot_read_twice_and_the_dequant_dump():
    H, D, page, pages = 3, 128, 16, 4
    cache = q4.KV4Cache.allocate(pages, page, H, D)
    k = torch.randn(pages * page, H, D, device="cuda")
    q4.kv4_write(cache, k, 2 * k, torch.arange(pages * page, dtype=torch.int32, device="cuda"))
    out = torch.empty(6, H, D, device="cuda")
    q4.kv4_read(out, None, cache, torch.tensor([5, 5, 60, 5, 0, 60], dtype=torch.int32, device="cuda"))
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[3]) and torch.equal(out[2], out[5])
    W = torch.empty(pages * H * page, D, device="cuda")
    q4.q4_dequant(W, cache.k_qs.view(-1, D // 2), cache.k_d.view(-1, D // 32))
    assert torch.equal(W.view(pages, H, page, D)[0, :, 5], out[0])


def test_rows_behind_2_to_the_32_bytes():
    """Slots whose code bytes lie past 2^32: 2.2 million pages of one 4 KB row set."""
    H, D, page = 8, 256, 4
    pages = (1 << 32) // (H * D // 2 * page) + 40
    cache = q4.KV4Cache.allocate(pages, page, H, D)
    k = torch.randn(3, H, D, device="cuda")
    slots = [pages * page - 1, 2, (1 << 32) // (H * D // 2) + 5]
    q4.kv4_write(cache, k, -k, torch.tensor(slots, dtype=torch.int32, device="cuda"))
    out, v = torch.empty_like(k), torch.empty_like(k)
    q4.kv4_read(out, v, cache, torch.tensor(slots, dtype=torch.int32, device="cuda"))
    want = torch.from_numpy(ref.values(*ref.quantise(k.cpu().numpy()))).float().cuda()
    assert torch.equal(out, want) and torch.equal(v, -want)
    rows = [cache.k_qs[s // page, :, s % page].cpu().numpy() for s in slots]
    assert np.array_equal(np.stack(rows), ref.quantise(k.cpu().numpy())[0])
    assert int((cache.k_qs != 0x88).any(-1).sum()) == 3 * H


def test_a_cache_keeps_the_tensors_that_its_struct_points_to():
    cache = q4.KV4Cache.allocate(2, 16, 2, 64)
    for name in ("k_qs", "k_d", "v_qs", "v_d"):
        with pytest.raises(AttributeError):
            setattr(cache, name, torch.zeros_like(getattr(cache, name)))
    with pytest.raises(AttributeError):
        cache.num_pages = 3
    assert cache._struct.k_qs == cache.k_qs.data_ptr() and cache._struct.v_d == cache.v_d.data_ptr()
