"""The experts' down projections with their weighted sum, and the whole mixture-of-experts layer, against 64 bits."""

import pytest
import torch

import moe_ref as ref

pytestmark = pytest.mark.gpu

import quantized_decode_gemv_q4_gb300 as q4  # noqa: E402

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


class Rand:
    def __init__(self, seed=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *s):
        return torch.randn(*s, generator=self.g, device="cuda")

    def weights(self, *shape):
        """Codes over the whole range and scales of both signs, [..., K/32, 16] and [..., K/32]."""
        *rows, K = shape
        qs = torch.randint(0, 256, (*rows, K // 32, 16), generator=self.g, device="cuda", dtype=torch.uint8)
        d = (0.5 + torch.rand(*rows, K // 32, generator=self.g, device="cuda")) / (4.6 * K ** 0.5)
        return qs, (d * torch.where(torch.rand(d.shape, generator=self.g, device="cuda") < 0.2, -1.0, 1.0)).half()

    def picks(self, T, topk, E):
        return torch.rand(T, E, generator=self.g, device="cuda").argsort(-1)[:, :topk].to(torch.int32).contiguous()


def down_case(T, topk, E, N, K, dt, seed=0, residual=True):
    r = Rand(seed)
    qs, d = r.weights(E, N, K)
    return dict(qs=qs, d=d, h=r.normal(T, topk, K) * r.normal(T, topk, 1).exp(), expert_ids=r.picks(T, topk, E),
                expert_weights=torch.softmax(r.normal(T, topk), -1), residual=r.normal(T, N).to(dt) if residual else None)


def check_down(a, out, keep=None):
    E = a["d"].shape[0]
    want, err = ref.down(a["h"].double(), torch.zeros_like(a["h"], dtype=torch.float64),
                         lambda e: ref.q4_matrix(a["qs"][e], a["d"][e]) if 0 <= e < E else None, a["expert_ids"].long(),
                         a["expert_weights"].double(), torch.zeros_like(a["expert_weights"], dtype=torch.float64), a["residual"],
                         out.shape[1], ref.one_part(out.dtype))
    lim = err + ref.rounded(want, out.dtype) * (1 + 2.0 ** -7)
    if keep is not None:
        out, want, lim = out[keep], want[keep], lim[keep]
    off = (out.double() - want).abs()
    assert bool((off <= lim).all()), f"{float((off / lim).max()):.2f} of the limit"


DOWN = [(1, 1, 1, 8, 32), (1, 8, 8, 64, 96), (2, 2, 3, 24, 256), (1, 8, 64, 520, 1408), (5, 3, 10, 672, 1056),
        (8, 8, 64, 256, 512), (17, 4, 5, 40, 288), (64, 8, 16, 136, 352), (170, 3, 6, 24, 64), (512, 1, 2, 16, 128),
        (3, 2, 4, 16, 16384), (9, 2, 2, 72, 4128), (2, 1, 2, 8, 65536), (4, 100, 128, 32, 64), (2, 3, 5000, 8, 32),
        (33, 1, 1, 200, 224), (16, 1, 1, 304, 2048), (12, 2, 2, 1000, 160)]


@pytest.mark.parametrize("T,topk,E,N,K", DOWN)
@pytest.mark.parametrize("dt", DTYPES)
def test_down_against_64_bits(T, topk, E, N, K, dt):
    a = down_case(T, topk, E, N, K, dt)
    out = torch.empty(T, N, dtype=dt, device="cuda")
    q4.moe_q4_down_gemv(out, **a)
    check_down(a, out)
    again = torch.empty_like(out)
    q4.moe_q4_down_gemv(again, **a)
    assert torch.equal(out, again)
    assert q4.q4_device_faults() == 0


def test_down_strided_rows_in_place_and_workspace():
    T, N = 9, 200
    a = down_case(T, 3, 7, N, 288, torch.bfloat16)
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    ws = q4.moe_q4_down_workspace(out, a["h"])
    guarded = torch.full((ws.numel() + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    q4.moe_q4_down_gemv(out, **a, workspace=guarded[:ws.numel()])
    check_down(a, out)
    assert bool((guarded[ws.numel():] == 0xA5).all())
    wide = torch.full((T, N + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + N] = a["residual"]
    q4.moe_q4_down_gemv(wide[:, 8:8 + N], **dict(a, residual=wide[:, 8:8 + N]), workspace=ws)
    assert torch.equal(wide[:, 8:8 + N], out) and bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + N:] == 7).all())


def test_down_bad_ids_make_their_tokens_nan():
    T, E, N = 20, 6, 48
    a = down_case(T, 3, E, N, 96, torch.float32)
    a["expert_ids"][3, 1], a["expert_ids"][9, 0], a["expert_ids"][19, 2] = -1, E, 2147483647
    out = torch.empty(T, N, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q4.moe_q4_down_gemv(out, **a, dev_status=status)
    bad = [3, 9, 19]
    assert bool(out[bad].isnan().all()) and status.item() == q4.FAULT_BAD_EXPERT
    assert q4.q4_device_faults() == q4.FAULT_BAD_EXPERT
    check_down(a, out, [t for t in range(T) if t not in bad])
    a["expert_ids"].fill_(-5)
    q4.moe_q4_down_gemv(out, **a)
    assert bool(out.isnan().all()) and q4.q4_device_faults() == q4.FAULT_BAD_EXPERT


def test_down_same_expert_twice_zero_weights_and_zero_rows():
    a = down_case(7, 4, 5, 64, 160, torch.float32)
    a["expert_ids"][2] = 3
    a["expert_ids"][4, 1:3] = 0
    a["expert_weights"][5] = 0
    a["h"][6] = 0
    out = torch.empty(7, 64, device="cuda")
    q4.moe_q4_down_gemv(out, **a)
    check_down(a, out)
    assert torch.equal(out[5:], a["residual"][5:])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_down_nan_and_infinity_stay_in_their_tokens(value):
    a = down_case(12, 2, 2, 64, 288, torch.float32)
    a["h"][5, 1, 77] = value
    out = torch.empty(12, 64, device="cuda")
    q4.moe_q4_down_gemv(out, **a)
    assert not bool(out[5].isfinite().any())
    check_down(a, out, [t for t in range(12) if t != 5])


def test_down_values_far_apart():
    """Elements 2^-20 to 2^20 apart within a slot, slots 2^80 apart, and blocks of zero scales."""
    a = down_case(10, 2, 3, 64, 512, torch.float32, residual=False)
    a["h"] *= torch.exp2(torch.randint(-20, 20, a["h"].shape, device="cuda").float())
    a["h"][3] *= 2.0 ** 60
    a["h"][4] *= 2.0 ** -80
    a["d"][:, :, 3] = 0
    out = torch.empty(10, 64, device="cuda")
    q4.moe_q4_down_gemv(out, **a)
    check_down(a, out)


def test_down_weights_past_32_bits():
    """Experts whose codes lie more than 2^32 bytes from the first's, among memory that is never read."""
    E, N, K, T = 1200, 1024, 8192, 3
    qs = torch.empty(E, N, K // 32, 16, dtype=torch.uint8, device="cuda")
    d = torch.empty(E, N, K // 32, dtype=torch.float16, device="cuda")
    assert qs.numel() > 1 << 32
    r = Rand(4)
    ids = torch.tensor([[0, E - 1], [E - 2, E - 1], [E // 2, 1]], dtype=torch.int32)
    for e in sorted(set(ids.flatten().tolist())):
        qs[e], d[e] = r.weights(N, K)
    a = dict(qs=qs, d=d, h=r.normal(T, 2, K), expert_ids=ids.cuda(), expert_weights=torch.rand(T, 2, device="cuda"), residual=None)
    out = torch.empty(T, N, device="cuda")
    q4.moe_q4_down_gemv(out, **a)
    check_down(a, out)


def test_down_scales_at_any_alignment():
    """Scales 2, 4 and 8 bytes past a 16-byte boundary: other copies, the same bits."""
    a = down_case(5, 3, 7, 96, 1024, torch.float32)
    out, again = torch.empty(5, 96, device="cuda"), torch.empty(5, 96, device="cuda")
    q4.moe_q4_down_gemv(out, **a)
    check_down(a, out)
    for shift in (1, 2, 4):
        d = torch.empty(a["d"].numel() + 8, dtype=torch.float16, device="cuda")[shift:shift + a["d"].numel()].view(a["d"].shape)
        d.copy_(a["d"])
        q4.moe_q4_down_gemv(again, **dict(a, d=d))
        assert torch.equal(out, again), shift


# ------------------------------------------------------------------------------------------------

def layer_case(T, topk, E, N, K, dt, norm=True, seed=0):
    r = Rand(seed + 100)
    parts = dict(router=r.weights(E, K), gate=r.weights(E, N, K), up=r.weights(E, N, K), down=r.weights(E, K, N))
    moe = q4.MoEWeights(*(t for pair in parts.values() for t in pair))
    x = (r.normal(T, K) * torch.where(torch.rand(K, generator=r.g, device="cuda") < 0.03, 8.0, 1.0)).to(dt)
    return dict(moe=moe, x=x, topk=topk, gamma=1 + 0.2 * r.normal(K) if norm else None, residual=r.normal(T, K).to(dt),
                mats={n: ref.q4_matrix(*p) for n, p in parts.items()})


def run_layer(a, out=None, **kw):
    T = a["x"].shape[0]
    out = torch.empty_like(a["x"]) if out is None else out
    ids = torch.full((T, a["topk"]), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, a["topk"]), -7.0, device="cuda")
    q4.moe_q4_layer(out, a["x"], a["moe"], a["topk"], gamma=a["gamma"], residual=a["residual"], expert_ids=ids,
                    expert_weights=w, **kw)
    return out, ids, w


def check_layer(a, out, ids, w, normalize=True, keep=None):
    keep = slice(None) if keep is None else keep
    x, res = a["x"][keep], None if a["residual"] is None else a["residual"][keep]
    out, ids, w = out[keep], ids[keep], w[keep]
    assert bool(((ids >= 0) & (ids < a["moe"].E)).all())
    (want, err), (rw, werr), (logits, lerr) = ref.layer(x, a["mats"], a["gamma"], 1e-6, res, ids.long(), normalize)
    # the picks: every one's logit may not lie below a rejected one's, nor the order be turned, by more than the errors
    slack = 2 * lerr.amax(-1, keepdim=True)
    got = logits.gather(1, ids.long())
    best = logits.sort(-1, descending=True).values[:, :a["topk"]]
    assert bool((got >= best - slack).all()) and all(len(set(r)) == a["topk"] for r in ids.tolist())
    assert bool(((w.double() - rw).abs() <= werr).all())
    off, lim = (out.double() - want).abs(), err + ref.rounded(want, out.dtype) * (1 + 2.0 ** -7)
    assert bool((off <= lim).all()), f"{float((off / lim).max()):.2f} of the limit"


LAYER = [(1, 1, 1, 32, 32), (1, 8, 64, 96, 256), (5, 3, 10, 1056, 672), (8, 8, 64, 320, 512), (64, 8, 16, 64, 2048),
         (31, 2, 4, 32, 4128), (512, 1, 3, 32, 64), (2, 2, 200, 32, 64), (1, 2, 2, 32, 32768), (1, 1, 1, 65536, 32),
         (6, 4, 4, 288, 8224), (40, 1, 2, 160, 96), (64, 8, 64, 32, 256), (19, 8, 128, 64, 224)]


@pytest.mark.parametrize("T,topk,E,N,K", LAYER)
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("norm", [True, False])
def test_layer_against_64_bits(T, topk, E, N, K, dt, norm):
    a = layer_case(T, topk, E, N, K, dt, norm)
    out, ids, w = run_layer(a, normalize=norm)
    check_layer(a, out, ids, w, norm)
    assert torch.equal(run_layer(a, normalize=norm)[0], out)


def test_layer_of_the_longest_vectors_and_most_slots():
    a = layer_case(128, 4, 5, 32, 24576, torch.float32)
    a["residual"] = None
    out, ids, w = run_layer(a)
    keep = list(range(0, 128, 9))
    check_layer(a, out, ids, w, keep=keep)


def test_two_graphs_and_streams_at_the_same_time():
    """Calls that run at the same time, each with its workspace."""
    cases = [layer_case(T, 4, 16, 256, 512, dt, seed=T) for T, dt in ((3, torch.bfloat16), (30, torch.float32))]
    outs, want, graphs, streams = [], [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for a, side in zip(cases, streams):
        ws = q4.moe_q4_layer_workspace(a["moe"], a["x"], 4)
        out = torch.empty_like(a["x"])
        call = lambda: q4.moe_q4_layer(out, a["x"], a["moe"], 4, gamma=a["gamma"], residual=a["residual"], workspace=ws)  # noqa: E731
        call()
        torch.cuda.synchronize()
        want.append(out.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            for _ in range(20):
                call()
        outs.append(out.zero_())
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, side in zip(graphs, streams):
            with torch.cuda.stream(side):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_everything_written_directly_before_the_calls():
    """With launch overlap off, the kernel before a call may write all that the call reads, weights among it."""
    sets = [layer_case(6, 3, 8, 640, 1024, torch.float32, seed=s) for s in (1, 2)]
    hid = [Rand(s).normal(6, 3, 640) for s in (1, 2)]
    names = [f"{m}_{part}" for m in ("router", "gate", "up", "down") for part in ("qs", "d")]
    live = {n: torch.empty_like(getattr(sets[0]["moe"], n)) for n in names}
    moe = q4.MoEWeights(**live)
    x, res, h = torch.empty(6, 1024, device="cuda"), torch.empty(6, 1024, device="cuda"), torch.empty_like(hid[0])
    out, down = torch.empty_like(x), torch.empty_like(x)
    ids, w = torch.empty(6, 3, dtype=torch.int32, device="cuda"), torch.empty(6, 3, device="cuda")
    ws, ws2 = q4.moe_q4_layer_workspace(moe, x, 3), q4.moe_q4_down_workspace(down, h)

    def load(a, hidden, wait):
        for src, dst in [(a["x"], x), (a["residual"], res), *((getattr(a["moe"], n), live[n]) for n in names)]:
            dst.copy_(src)
            if wait:
                torch.cuda.synchronize()
        q4.moe_q4_layer(out, x, moe, 3, gamma=a["gamma"], residual=res, expert_ids=ids, expert_weights=w, workspace=ws)
        first = out.clone()
        h.copy_(hidden)
        live["down_d"].mul_(2)
        if wait:
            torch.cuda.synchronize()
        q4.moe_q4_down_gemv(down, live["down_qs"], live["down_d"], h, ids, w, residual=res, workspace=ws2)
        q4.residual_norm(out, res, down, res, pre_gamma=a["gamma"])
        return first, down.clone(), out.clone(), res.clone()

    want = [load(a, hd, True) for a, hd in zip(sets, hid)]
    torch.cuda.synchronize()
    for i in range(40):
        got = load(sets[i % 2], hid[i % 2], False)
        assert all(torch.equal(g, v) for g, v in zip(got, want[i % 2])), i


@pytest.mark.parametrize("overlap", [False, True])
def test_graphs_whose_calls_follow_copies_fills_and_joined_streams(overlap):
    """What a captured call may follow: another library's kernel, a copy, a fill, two streams that meet."""
    a = layer_case(5, 2, 6, 96, 256, torch.bfloat16)
    src = {n: t.clone() for n, t in (("x", a["x"]), ("residual", a["residual"]))}
    h, y, out, down = (torch.empty_like(a["x"]) for _ in range(4))
    hid, ids, w = Rand(2).normal(5, 2, 96), Rand(3).picks(5, 2, 6), torch.rand(5, 2, device="cuda")
    moved = torch.empty_like(hid)
    ws, ws2 = q4.moe_q4_layer_workspace(a["moe"], a["x"], 2), q4.moe_q4_down_workspace(down, hid)
    other = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            a["residual"].copy_(src["residual"])
            moved.zero_()
            moved.add_(hid)
        a["x"].copy_(src["x"])
        here.wait_stream(other)
        q4.residual_norm(h, y, a["x"], a["residual"], pre_gamma=a["gamma"])
        y.mul_(2)
        q4.moe_q4_layer(out, y, a["moe"], 2, gamma=a["gamma"], residual=h, workspace=ws)
        other.wait_stream(here)
        with torch.cuda.stream(other):
            q4.moe_q4_down_gemv(down, a["moe"].down_qs, a["moe"].down_d, moved, ids, w, residual=out, workspace=ws2)
        h.fill_(1)
        q4.residual_norm(h, y, out, h, pre_gamma=a["gamma"])
        here.wait_stream(other)
        q4.residual_norm(down, y, down, h, pre_gamma=a["gamma"])

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (h, y, out, down)]

    q4.q4_set_launch_overlap(overlap)
    try:
        step()
        want = results()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
        for _ in range(3):
            for t in (a["x"], a["residual"], h, y, out, down, moved):
                t.fill_(-3)
            g.replay()
            assert all(torch.equal(r, v) for r, v in zip(results(), want))
    finally:
        q4.q4_set_launch_overlap(False)
    assert q4.q4_device_faults() == 0


def test_layer_in_place_strides_and_workspace():
    T, K = 7, 288
    a = layer_case(T, 2, 5, 96, K, torch.float16)
    a["residual"] = a["x"]
    out, ids, w = run_layer(a)
    check_layer(a, out, ids, w)
    ws = q4.moe_q4_layer_workspace(a["moe"], a["x"], 2)
    guarded = torch.full((ws.numel() + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    wide = torch.full((T, K + 16), 7.0, dtype=torch.float16, device="cuda")
    cut = wide[:, 8:8 + K]
    cut.copy_(a["x"])
    q4.moe_q4_layer(cut, cut, a["moe"], 2, gamma=a["gamma"], residual=cut, workspace=guarded[:ws.numel()])
    assert torch.equal(cut, out) and bool((guarded[ws.numel():] == 0xA5).all())
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + K:] == 7).all())
    no = run_layer(dict(a, residual=None))
    check_layer(dict(a, residual=None), *no)


def test_layer_nan_tokens_touch_no_other():
    a = layer_case(12, 2, 3, 64, 256, torch.float32)
    want = run_layer(a)
    a["x"][4, 9], a["x"][7, 100] = float("nan"), float("inf")
    out, ids, w = run_layer(a)
    assert bool(out[4].isnan().all()) and bool(out[7].isnan().all())
    assert bool(((ids >= 0) & (ids < 3)).all())
    keep = [t for t in range(12) if t not in (4, 7)]
    check_layer(a, out, ids, w, keep=keep)
    assert torch.equal(ids[keep], want[1][keep])


def test_layer_is_the_router_the_experts_and_the_down_projection():
    """The same layer from the separate calls, which a user may put together differently."""
    T, topk, E, N, K = 8, 4, 16, 192, 512
    a = layer_case(T, topk, E, N, K, torch.float32, norm=False)
    m = a["moe"]
    ids = torch.empty(T, topk, dtype=torch.int32, device="cuda")
    w = torch.empty(T, topk, device="cuda")
    h = torch.empty(T, topk, N, device="cuda")
    out = torch.empty(T, K, device="cuda")
    q4.moe_router_q4(ids, w, m.router_qs, m.router_d, a["x"], topk)
    flat = lambda t: t.flatten(0, 1)  # noqa: E731
    q4.moe_q4_swiglu_gemv(h, flat(m.gate_qs), flat(m.gate_d), flat(m.up_qs), flat(m.up_d), a["x"], ids, E)
    q4.moe_q4_down_gemv(out, m.down_qs, m.down_d, h, ids, w, residual=a["residual"])
    check_layer(a, out, ids, w)
    whole, ids2, w2 = run_layer(a)
    check_layer(a, whole, ids2, w2)
    assert torch.equal(ids, ids2)


def block(a, s, stream=None):
    """Between attention and the next block: residual and norm, the layer, its own norm behind it and the next one's."""
    q4.residual_norm(s["h"], s["y"], a["x"], a["residual"], pre_gamma=a["gamma"], stream=stream)
    q4.moe_q4_layer(s["m"], s["y"], a["moe"], a["topk"], workspace=s["ws"], stream=stream)
    q4.residual_norm(s["h"], s["y"], s["m"], s["h"], post_gamma=a["gamma"], gate=s["gate"], pre_gamma=a["gamma"], stream=stream)
    q4.moe_q4_layer(s["h"], s["y"], a["moe"], a["topk"], residual=s["h"], workspace=s["ws"], stream=stream)
    q4.moe_q4_down_gemv(s["h"], a["moe"].down_qs, a["moe"].down_d, s["hid"], s["ids"], s["w"], residual=s["h"],
                        workspace=s["ws2"], stream=stream)


@pytest.mark.parametrize("T", [1, 11, 60])
def test_a_block_on_streams_with_overlap_and_in_graphs(T):
    a = layer_case(T, 4, 8, 256, 512, torch.bfloat16)
    r = Rand(5)
    empty = lambda: torch.empty_like(a["x"])  # noqa: E731
    s = dict(h=empty(), y=empty(), m=empty(), gate=torch.tanh(r.normal(512)).to(torch.bfloat16), hid=r.normal(T, 4, 256),
             ids=r.picks(T, 4, 8), w=torch.rand(T, 4, device="cuda"), ws=q4.moe_q4_layer_workspace(a["moe"], a["x"], 4))
    s["ws2"] = q4.moe_q4_down_workspace(s["h"], s["hid"])
    block(a, s)
    torch.cuda.synchronize()
    want = s["h"].clone(), s["y"].clone()
    # stage by stage: the first norm, and the layer on its actual input
    (rh, eh), (ry, ey) = ref.residual_norm(a["x"], a["residual"], None, None, a["gamma"], 1e-6, 1.0, 1.0)
    q4.residual_norm(s["h"], s["y"], a["x"], a["residual"], pre_gamma=a["gamma"])
    assert bool(((s["y"].double() - ry).abs() <= ey + ref.rounded(ry, torch.bfloat16) * (1 + 2.0 ** -7)).all())
    b = dict(a, x=s["y"], gamma=None, residual=None)
    check_layer(b, *run_layer(b))

    def same(what):
        torch.cuda.synchronize()
        assert torch.equal(s["h"], want[0]) and torch.equal(s["y"], want[1]), what

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for overlap in (False, True):
        q4.q4_set_launch_overlap(overlap)
        try:
            s["h"].zero_(), s["y"].zero_()
            torch.cuda.synchronize()
            block(a, s, side)
            same("a given stream")
            with torch.cuda.stream(side):
                block(a, s)
            same("another current stream")
            block(a, dict(s, ws=None, ws2=None))
            same("workspaces of the calls")
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                block(a, s)
            for _ in range(3):
                s["h"].zero_(), s["y"].zero_()
                g.replay()
                same("graph")
        finally:
            q4.q4_set_launch_overlap(False)
    assert q4.q4_device_faults() == 0
