"""A decode step's operators as they are used: q/k/v projection GEMVs (fused RMSNorm + Q4_K), q/k norm and rotation in place
on the projection's output, the cache write, attention over the cache and the output projection (planar Q4).

Each stage is checked against its own 64-bit reference on the stage's actual inputs; then the whole step must give the same
bits with launch overlap on, from a captured graph replayed over growing sequences, and on another stream."""

import numpy as np
import pytest
import torch

import kv4_ref as ref
import synth
from gpu_util import assert_close, cu

pytestmark = pytest.mark.gpu

import quantized_decode_gemv_q4_gb300 as q4  # noqa: E402

B, HQ, HKV, D, K, PAGE, PAGES = 3, 7, 1, 128, 1024, 16, 24
WIDTH = (HQ + 2 * HKV) * D


class Step:
    def __init__(self, spare=0):
        rng = np.random.default_rng(11)
        self.w_qkv = synth.q4k_weights(rng, WIDTH, K)
        self.gamma = synth.gamma(rng, K)
        self.w_o = synth.q4_weights(rng, K, HQ * D)
        self.d_qkv, self.d_gamma, self.d_o = cu(self.w_qkv), cu(self.gamma), [cu(a) for a in self.w_o]
        self.qg, self.kg = cu(synth.gamma(rng, D)), cu(synth.gamma(rng, D))
        a = np.arange(512)[:, None] * 10000.0 ** (-np.arange(0, D, 2) / D)
        self.cos_sin = cu(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))
        self.cache = q4.KV4Cache.allocate(PAGES, PAGE, HKV, D)
        order = rng.permutation(PAGES).astype(np.int32).reshape(B, -1)
        self.table = cu(np.concatenate([order, np.full((B, spare), -1, np.int32)], 1))
        self.xs = [cu(synth.activations(rng, B, K)) for _ in range(5)]
        self.x = torch.empty(B, K, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.start = torch.tensor([0, 30, 100], dtype=torch.int32, device="cuda")
        old = torch.randn(128, HKV, D, generator=torch.Generator().manual_seed(3)).cuda()
        for b, n in enumerate(self.start.tolist()):  # what earlier steps left in the cache
            if n:
                t = torch.arange(n, device="cuda")
                q4.kv4_write(self.cache, old[:n], old[:n] * 2, (self.table[b][t // PAGE] * PAGE + t % PAGE).int())
        self.saved = [t.clone() for t in (self.cache.k_qs, self.cache.k_d, self.cache.v_qs, self.cache.v_d)]
        self.qkv = torch.empty(B, HQ + 2 * HKV, D, device="cuda")
        self.att = torch.empty(B, HQ, D, device="cuda")
        self.y = torch.empty(B, K, device="cuda")
        self.ws = q4.kv4_attention_workspace(self.att, self.cache)

    def reset(self):
        for t, s in zip((self.cache.k_qs, self.cache.k_d, self.cache.v_qs, self.cache.v_d), self.saved):
            t.copy_(s)
        self.lens.copy_(self.start)

    def run(self, stream=None):
        q, k, v = self.qkv[:, :HQ], self.qkv[:, HQ:HQ + HKV], self.qkv[:, HQ + HKV:]
        pos = self.lens.clone()
        slots = (torch.gather(self.table, 1, (pos // PAGE).long()[:, None])[:, 0] * PAGE + pos % PAGE).int()
        self.lens += 1
        for b in range(B):
            q4.fused_rmsnorm_q4k_gemv(self.qkv[b], self.d_qkv, self.x[b], self.d_gamma, 1e-5, stream=stream)
        q4.qk_norm_rope(q, k, q, k, self.qg, self.kg, self.cos_sin, pos, stream=stream)
        q4.kv4_write(self.cache, k, v, slots, stream=stream)
        q4.kv4_attention(self.att, q, self.cache, self.table, self.lens, workspace=self.ws, stream=stream)
        q4.q4_gemv_batched(self.y, *self.d_o, self.att.view(B, -1), stream=stream)

    def outputs(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.qkv, self.att, self.y, self.cache.k_qs, self.cache.k_d)]


@pytest.mark.parametrize("spare", [0, 100])
def test_every_stage_against_64_bits(spare, oracle_lib):
    s = Step(spare)
    s.reset()
    for x in s.xs:
        s.x.copy_(x)
        pos = s.lens.cpu().numpy().copy()
        s.run()
        torch.cuda.synchronize()
        host = [t.cpu().numpy() for t in (s.qkv, s.att, s.y, s.cache.k_qs, s.cache.k_d, s.cache.v_qs, s.cache.v_d, s.table)]
        qkv, att, y, k_qs, k_d, v_qs, v_d, table = host
        for b in range(B):
            proj, bound = oracle_lib.fused_rmsnorm_q4k_gemv(s.w_qkv, x[b].cpu().numpy(), s.gamma, np.float32(1e-5))
            lim = 1e-3 * bound + 1e-5  # the projection's tolerance; its q and k are normalised in place, v is as it came
            assert np.all(np.abs(qkv[b].reshape(-1)[(HQ + HKV) * D:] - proj[(HQ + HKV) * D:]) <= lim[(HQ + HKV) * D:])
            slot = table[b, pos[b] // PAGE], pos[b] % PAGE
            for rows, qs, d in ((qkv[b, HQ:HQ + HKV], k_qs, k_d), (qkv[b, HQ + HKV:], v_qs, v_d)):
                c, sc = ref.quantise(rows)
                assert np.array_equal(qs[slot[0], :, slot[1]], c) and np.array_equal(d[slot[0], :, slot[1]], sc)
        out, _, tol, _ = ref.attention(qkv[:, None, :HQ].astype(np.float64), k_qs, k_d, v_qs, v_d, table, pos + 1, D ** -0.5, 0)
        assert np.all(np.abs(att - out[:, 0]) <= tol[:, 0] + 2.0 ** -24 * np.abs(out[:, 0]))
        r, bound = oracle_lib.q4_gemv_batched(*s.w_o, att.reshape(B, -1))
        assert_close(y, r, bound, "output projection")
    assert q4.q4_device_faults() == 0


def test_the_norm_and_rotation_of_the_projection(oracle_lib):
    """The rotated heads of the step, from the projection's own values."""
    s = Step()
    s.reset()
    s.x.copy_(s.xs[0])
    s.run()
    rotated = s.qkv.clone()
    for b in range(B):
        q4.fused_rmsnorm_q4k_gemv(s.qkv[b], s.d_qkv, s.x[b], s.d_gamma, 1e-5)
    raw = s.qkv.double().cpu().numpy()
    for lo, hi, g in ((0, HQ, s.qg), (HQ, HQ + HKV, s.kg)):
        y, size = ref.rope(raw[:, lo:hi], g.cpu().numpy(), 1e-6, s.cos_sin.cpu().numpy(), s.start.cpu().numpy(), False)
        got = rotated[:, lo:hi].double().cpu().numpy()
        assert np.all(np.abs(got - y) <= (D / 2 + 12) * ref.U * size)


@pytest.mark.parametrize("spare", [0, 100])
def test_overlap_graph_and_stream_give_the_same_bits(spare):
    s = Step(spare)

    def eager(stream=None):
        s.reset()
        outs = []
        for x in s.xs:
            s.x.copy_(x)
            s.run(stream)
            outs.append(s.outputs())
        return outs

    def same(a, b, what):
        for i, (u, v) in enumerate(zip(a, b)):
            for j, (x, y) in enumerate(zip(u, v)):
                assert torch.equal(x, y), f"{what}: step {i}, output {j}"

    want = eager()
    q4.q4_set_launch_overlap(True)
    try:
        same(eager(), want, "overlap")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        s.reset()
        with torch.cuda.stream(side):
            s.run()  # warm-up
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        s.reset()
        with torch.cuda.graph(g, stream=side):
            s.run()
        s.reset()
        outs = []
        for x in s.xs:
            s.x.copy_(x)
            g.replay()
            outs.append(s.outputs())
        same(outs, want, "graph")
        with torch.cuda.stream(side):
            same(eager(), want, "another current stream")
            same(eager(side), want, "a given stream")
    finally:
        q4.q4_set_launch_overlap(False)
    assert q4.q4_device_faults() == 0
