"""Refusals of the block norm, the down projection and the layer, without a GPU: through the C ABI on fake addresses (nothing
is dereferenced before an argument is refused), and through the Python binding on CPU tensors."""

import ctypes

import pytest
import torch

import quantized_decode_gemv_q4_gb300 as q4
from quantized_decode_gemv_q4_gb300 import build as lib_build

A = 1 << 20  # a fake, 16-byte aligned address
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    if lib_build.is_stale():
        lib_build.build()
    return q4.load()


_kept = []


def weights(**kw):
    f = {n: A for n, _ in q4.MoEWeights._Struct._fields_}
    f.update(E=4, N=64, K=96)
    f.update(kw)
    _kept.append(q4.MoEWeights._Struct(*f.values()))
    return ctypes.addressof(_kept[-1])


NORM = dict(h=A, y=2 * A, x=A, residual=A, post=A, gate=A, pre=A, eps=1e-6, rs=1.0, bs=1.0, T=2, K=64, width=64, hs=64, ys=64,
            xs=64, ress=64, gs=64, dtype=0, stream=None)
DOWN = dict(out=A, qs=A, d=A, h=A, ids=A, w=A, residual=A, T=2, topk=2, E=4, N=64, K=96, os=64, rs=64, dtype=0, status=None,
            ws=A, ws_bytes=1 << 40, stream=None)
LAYER = dict(out=A, x=A, weights=None, gamma=A, eps=1e-6, residual=A, ids=A, w=A, T=2, topk=2, normalize=1, os=96, xs=96, rs=96,
             dtype=0, ws=A, ws_bytes=1 << 40, stream=None)
E, L = q4.Q4_EINVAL, q4.Q4_EALIGN


def refused(lib, name, base, code, text, **kw):
    f = dict(base)
    if "weights" in f and "weights" not in kw:
        f["weights"] = weights()
    f.update(kw)
    assert getattr(lib, name)(*f.values()) == code, f"{name} {kw}"
    said = lib.q4_last_error().decode()
    assert said.startswith(name) and text in said, said


@pytest.mark.parametrize("kw,code,text", [
    (dict(T=0), E, "T must"), (dict(T=-1), E, "T must"), (dict(K=0), E, "K must"), (dict(K=60), E, "multiple of 8"),
    (dict(K=32776), E, "32768"), (dict(dtype=3), E, "dtype"), (dict(x=None), E, "null x"), (dict(h=None), E, "null h_out"),
    (dict(y=None), E, "come together"), (dict(pre=None), E, "come together"), (dict(y=A), E, "the same"),
    (dict(x=A + 8), L, "row of x"), (dict(xs=62), E, "token stride of x"), (dict(xs=66), L, "row of x"),
    (dict(hs=0), E, "token stride of h_out"), (dict(ys=63), E, "token stride of y_out"), (dict(residual=A + 4), L, "row of residual"),
    (dict(ress=-64), E, "token stride of residual"), (dict(post=A + 4), L, "post_gamma"), (dict(pre=A + 8), L, "pre_gamma"),
    (dict(width=2), E, "gate_width"), (dict(width=0), E, "gate_width"), (dict(gs=63), E, "token stride of gate"),
    (dict(gs=-64), E, "token stride of gate"), (dict(gate=A + 8), L, "gate"), (dict(gs=65), L, "gate"),
    (dict(gate=A + 2, width=1, gs=1), L, "gate"), (dict(eps=-1.0), E, "eps"), (dict(eps=NAN), E, "eps"), (dict(eps=INF), E, "eps"),
    (dict(rs=INF), E, "scales"), (dict(bs=NAN), E, "scales")])
def test_residual_norm_refusals(lib, kw, code, text):
    refused(lib, "residual_norm", NORM, code, text, **kw)


SLOTS = [(dict(T=0), E, "T and topk"), (dict(topk=0), E, "T and topk"), (dict(topk=5), E, "exceeds E"),
         (dict(T=257), E, "exceeds 512"), (dict(T=1 << 30, topk=4), E, "exceeds 512"), (dict(dtype=-1), E, "dtype"),
         (dict(ws=None), E, "null workspace"), (dict(ws=A + 8), L, "workspace"), (dict(ws_bytes=16), E, "are needed"),
         (dict(residual=A + 8), L, "row of residual"), (dict(rs=63), E, "token stride of residual"), (dict(out=None), E, "null out"),
         (dict(out=A + 4), L, "row of out"), (dict(os=32), E, "token stride of out")]


@pytest.mark.parametrize("kw,code,text", SLOTS + [
    (dict(E=0), E, "E must"), (dict(N=0), E, "multiple of 8"), (dict(N=60), E, "multiple of 8"), (dict(K=0), E, "multiple of 32"),
    (dict(K=80), E, "multiple of 32"), (dict(K=65568), E, "65536"), (dict(E=1 << 27, N=64), E, "2^31-1"),
    (dict(qs=None), E, "null weight"), (dict(d=None), E, "null weight"), (dict(qs=A + 8), L, "qs"), (dict(d=A + 1), L, "d "),
    (dict(h=None), E, "null h"), (dict(h=A + 4), L, "h must"), (dict(ids=None), E, "null expert_ids"),
    (dict(ids=A + 2), L, "expert_ids"), (dict(w=None), E, "null expert_weights"), (dict(w=A + 2), L, "expert_weights"),
    (dict(status=A + 2), L, "dev_status")])
def test_down_refusals(lib, kw, code, text):
    refused(lib, "moe_q4_down_gemv", DOWN, code, text, **kw)


@pytest.mark.parametrize("kw,code,text", SLOTS + [
    (dict(weights=None), E, "null weights"), (dict(x=None), E, "null x"), (dict(x=A + 8), L, "row of x"),
    (dict(xs=90), E, "token stride of x"), (dict(gamma=A + 4), L, "gamma"), (dict(eps=NAN), E, "eps"),
    (dict(ids=A + 2), L, "expert_ids"), (dict(w=A + 1), L, "expert_ids")])
def test_layer_refusals(lib, kw, code, text):
    refused(lib, "moe_q4_layer", LAYER, code, text, **kw)


@pytest.mark.parametrize("kw,code,text", [
    (dict(E=0), E, "E must"), (dict(E=4097), E, "4096"), (dict(N=16), E, "multiple of 32"), (dict(N=0), E, "multiple of 32"),
    (dict(N=65568), E, "65536"), (dict(K=112), E, "multiple of 32"), (dict(K=32800), E, "32768"),
    (dict(router_qs=None), E, "null weight"), (dict(gate_d=None), E, "null weight"), (dict(up_qs=A + 8), L, "qs"),
    (dict(down_d=A + 1), L, "d ")])
def test_layer_weight_refusals(lib, kw, code, text):
    refused(lib, "moe_q4_layer", LAYER, code, text, weights=weights(**kw))


def test_workspace_refusals(lib):
    need = ctypes.c_size_t(0)
    for name, good in (("moe_q4_down_workspace", (2, 2, 64, 96)), ("moe_q4_layer_workspace", (2, 2, 4, 64, 96))):
        fn = getattr(lib, name)
        assert fn(None, *good) == E
        assert fn(ctypes.byref(need), *good) == q4.Q4_OK and need.value > 0
        for i in range(len(good)):
            bad = list(good)
            bad[i] = 0
            assert fn(ctypes.byref(need), *bad) == E
        assert fn(ctypes.byref(need), 513, 1, *good[2:]) == E


def q4_pair(*shape):
    *rows, K = shape
    return torch.zeros(*rows, K // 32, 16, dtype=torch.uint8), torch.zeros(*rows, K // 32, dtype=torch.float16)


def test_binding_refuses_cpu_tensors_and_shapes():
    x = torch.zeros(2, 96)
    with pytest.raises(TypeError, match="CUDA"):
        q4.residual_norm(x, None, x)
    with pytest.raises(TypeError, match="CUDA"):
        q4.moe_q4_down_gemv(x, *q4_pair(4, 96, 64), torch.zeros(2, 2, 64), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2))
    with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
        q4.residual_norm(x.double(), None, x.double())
    good = [q4_pair(4, 96), q4_pair(4, 64, 96), q4_pair(4, 64, 96), q4_pair(4, 96, 64)]
    for i, pair in [(0, q4_pair(4, 64)), (0, q4_pair(5, 96)), (1, q4_pair(4, 32, 96)), (2, q4_pair(4, 64, 64)),
                    (3, q4_pair(4, 64, 96)), (3, q4_pair(3, 96, 64))]:
        bad = list(good)
        bad[i] = pair
        with pytest.raises(ValueError, match="expected codes"):
            q4.MoEWeights(*(t for p in bad for t in p))
    with pytest.raises(ValueError, match="multiple of 32"):
        q4.MoEWeights(*good[0], *q4_pair(4, 48, 96), *q4_pair(4, 48, 96), *good[3])
    with pytest.raises(TypeError, match="CUDA"):
        q4.MoEWeights(*(t for p in good for t in p))


@pytest.mark.parametrize("handle", [q4.MoEWeights, q4.KV4Cache])
def test_handles_keep_what_their_structs_point_to(handle):
    made = object.__new__(handle)  # without a GPU: only what guards the attributes
    made.__dict__["tensor"] = torch.zeros(1)
    for change in (lambda: setattr(made, "tensor", None), lambda: delattr(made, "tensor"), lambda: delattr(made, "_struct")):
        with pytest.raises(AttributeError, match="make another one"):
            change()
    assert made.tensor is not None
