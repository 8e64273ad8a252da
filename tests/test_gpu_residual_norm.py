"""residual_norm against 64 bits: types, widths, gates, scales, strides, in place, streams and graphs."""

import pytest
import torch

import moe_ref as ref

pytestmark = pytest.mark.gpu

import quantized_decode_gemv_q4_gb300 as q4  # noqa: E402

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def make(T, K, dt, post, pre, gate, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    shape = {"none": None, "channel": (K,), "token": (T, 1), "element": (T, K)}[gate]
    return dict(x=rand(T, K).to(dt), residual=(3 * rand(T, K)).to(dt), post=1 + 0.3 * rand(K) if post else None,
                pre=1 + 0.3 * rand(K) if pre else None, gate=None if shape is None else rand(*shape).to(dt))


def call(a, h, y, rs=1.0, bs=1.0, eps=1e-6, **kw):
    q4.residual_norm(h, y, a["x"], a["residual"], post_gamma=a["post"], gate=a["gate"], pre_gamma=a["pre"], eps=eps,
                     residual_scale=rs, branch_scale=bs, **kw)


def check(a, h, y, rs=1.0, bs=1.0, eps=1e-6):
    (rh, eh), (ry, ey) = ref.residual_norm(a["x"], a["residual"], a["post"], a["gate"], a["pre"], eps, rs, bs)
    for got, want, err, name in ((h, rh, eh, "h"), (y, ry, ey, "y")):
        if want is None:
            continue
        lim = (1 + 2.0 ** -7) * err + ref.rounded(want, got.dtype)
        off = (got.double() - want).abs()
        assert bool((off <= lim).all()), f"{name}: {float((off / lim).max()):.2f} of the limit"


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,K", [(1, 8), (1, 2048), (3, 24), (5, 136), (7, 264), (2, 1032), (67, 3584), (9, 4104), (2, 8200),
                                 (3, 16384), (2, 32768), (1025, 96), (300, 2048)])
@pytest.mark.parametrize("post,pre,gate", [(False, True, "none"), (True, True, "channel"), (True, False, "token"),
                                           (True, True, "element"), (False, False, "none")])
def test_against_64_bits(dt, T, K, post, pre, gate):
    a = make(T, K, dt, post, pre, gate)
    h, y = torch.empty_like(a["x"]), torch.empty_like(a["x"]) if pre else None
    call(a, h, y, 0.75, -0.22)
    check(a, h, y, 0.75, -0.22)


@pytest.mark.parametrize("dt", DTYPES)
def test_no_residual_and_zero_rows(dt):
    a = make(4, 256, dt, True, True, "none")
    a["residual"] = None
    a["x"][1] = 0
    h, y = torch.empty_like(a["x"]), torch.empty_like(a["x"])
    call(a, h, y)
    check(a, h, y)
    assert not h[1].any() and not y[1].any()


@pytest.mark.parametrize("dt", DTYPES)
def test_strided_rows_and_broadcast_gate(dt):
    """Columns of wider tensors on every side; what lies between them stays as it was."""
    T, K = 37, 264
    a = make(T, K, dt, True, True, "channel")
    wide = {n: torch.full((T, K + 24), 7.0, device="cuda", dtype=dt) for n in ("x", "residual", "h", "y")}
    for n in ("x", "residual"):
        wide[n][:, 8:8 + K] = a[n]
    cut = {n: t[:, 8:8 + K] for n, t in wide.items()}
    b = dict(a, x=cut["x"], residual=cut["residual"], gate=a["gate"].expand(T, K))
    call(b, cut["h"], cut["y"])
    check(a, cut["h"], cut["y"])
    for n in ("h", "y"):
        assert bool((wide[n][:, :8] == 7).all()) and bool((wide[n][:, 8 + K:] == 7).all())


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("K", [64, 2048, 16384])
def test_in_place(dt, K):
    a = make(33, K, dt, True, True, "element")
    h, y = torch.empty_like(a["x"]), torch.empty_like(a["x"])
    call(a, h, y)
    b = {n: None if t is None else t.clone() for n, t in a.items()}
    call(b, b["residual"], b["x"])  # the residual stream is updated, the norm replaces the branch
    assert torch.equal(b["residual"], h) and torch.equal(b["x"], y)
    b = {n: None if t is None else t.clone() for n, t in a.items()}
    call(b, b["x"], b["residual"])
    assert torch.equal(b["x"], h) and torch.equal(b["residual"], y)


def test_nan_and_infinity_stay_in_their_rows():
    a = make(5, 512, torch.float32, True, True, "none")
    a["x"][1, 3], a["residual"][3, 500] = float("inf"), float("nan")
    h, y = torch.empty_like(a["x"]), torch.empty_like(a["x"])
    call(a, h, y)
    assert bool(y[1].isnan().all()) and bool(y[3].isnan().all()) and bool(h[1, 3].isnan())
    keep = [0, 2, 4]
    for n in ("x", "residual"):
        a[n] = a[n][keep]
    check(a, h[keep], y[keep])


def test_large_and_small_values():
    a = make(2, 1024, torch.float32, True, True, "none")
    for n in ("x", "residual"):
        a[n][0] *= 1e15
        a[n][1] *= 1e-15
    h, y = torch.empty_like(a["x"]), torch.empty_like(a["x"])
    call(a, h, y, eps=0.0)
    check(a, h, y, eps=0.0)


def test_offsets_past_32_bits():
    """Rows far apart: the last one's offset in elements does not fit 32 bits."""
    K, T = 64, 3
    step = (1 << 31) // 2 + 64
    big = torch.empty((T - 1) * step + K, dtype=torch.float16, device="cuda")
    rows = big.as_strided((T, K), (step, 1))
    a = make(T, K, torch.float16, False, True, "none")
    rows.copy_(a["x"])
    h, y = torch.empty_like(a["x"]), torch.empty_like(a["x"])
    call(dict(a, x=rows), h, y)
    check(a, h, y)
    call(a, rows, y)
    check(a, rows, y)


def test_stream_overlap_and_graph_give_the_same_bits():
    a = make(130, 1032, torch.bfloat16, True, True, "token")
    h, y = torch.empty_like(a["x"]), torch.empty_like(a["x"])

    def run(stream=None):
        call(a, h, y, stream=stream)
        call(dict(a, x=y, residual=h), h, y, stream=stream)  # the next block's, in place

    run()
    torch.cuda.synchronize()
    want = h.clone(), y.clone()
    side = torch.cuda.Stream()
    q4.q4_set_launch_overlap(True)
    try:
        side.wait_stream(torch.cuda.current_stream())
        run(side)
        side.synchronize()
        assert torch.equal(h, want[0]) and torch.equal(y, want[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            run()
        for _ in range(2):
            h.zero_(), y.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    finally:
        q4.q4_set_launch_overlap(False)
