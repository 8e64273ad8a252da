"""Refusals of the norm/rotation, cache and attention calls, without a GPU: through the C ABI on fake addresses (nothing
is dereferenced before an argument is refused), and through the Python binding on CPU tensors."""

import ctypes

import pytest
import torch

import quantized_decode_gemv_q4_gb300 as q4
from quantized_decode_gemv_q4_gb300 import build as lib_build

P = ctypes.c_void_p
A = 1 << 20  # a fake, 16-byte aligned address


@pytest.fixture(scope="module")
def lib():
    if lib_build.is_stale():
        lib_build.build()
    return q4.load()


def cache(**kw):
    f = dict(k_qs=A, k_d=A, v_qs=A, v_d=A, num_pages=4, num_kv_heads=2, page_size=16, head_dim=64)
    f.update(kw)
    return ctypes.addressof(keep(q4.KV4Cache._Struct(*[f[n] for n, _ in q4.KV4Cache._Struct._fields_])))


_kept = []


def keep(x):
    _kept.append(x)
    return x


ROPE = dict(q_out=A, k_out=A, q=A, k=A, q_gamma=A, k_gamma=A, eps=1e-6, cos_sin=A, positions=A, T=2, Hq=4, Hkv=2, D=64, rot=64,
            max_pos=10, interleaved=0, qs=256, ks=128, qos=256, kos=128, dtype=0, stream=None)
WRITE = dict(cache=None, k=A, v=A, slots=A, T=2, ks=128, vs=128, dtype=0, stream=None)
READ = dict(k=A, v=A, cache=None, slots=A, T=2, ks=128, vs=128, dtype=0, stream=None)
ATTN = dict(out=A, lse=None, q=A, cache=None, table=A, lens=A, B=2, M=1, Hq=4, max_pages=4, qs=256, os=256, scale=0.1, window=0,
            dtype=0, ws=A, ws_bytes=1 << 40, stream=None)


def refused(lib, name, base, code, text, **kw):
    f = dict(base)
    if "cache" in f:
        f["cache"] = cache()
    f.update(kw)
    assert getattr(lib, name)(*f.values()) == code, f"{name} {kw}"
    said = lib.q4_last_error().decode()
    assert said.startswith(name) and text in said, said


def test_rope_refusals(lib):
    for kw, code, text in [
            (dict(q=None), q4.Q4_EINVAL, "null q"), (dict(k_out=None), q4.Q4_EINVAL, "null k_out"),
            (dict(T=0), q4.Q4_EINVAL, "T must"), (dict(T=1 << 30), q4.Q4_EINVAL, "2^31-1"), (dict(D=48), q4.Q4_EINVAL, "multiple of 32"),
            (dict(D=288, qs=2000, ks=2000, qos=2000, kos=2000), q4.Q4_EINVAL, "up to 256"),
            (dict(Hq=0), q4.Q4_EINVAL, "heads"), (dict(Hkv=0), q4.Q4_EINVAL, "key heads"),
            (dict(Hq=70000), q4.Q4_EINVAL, "heads"), (dict(rot=24), q4.Q4_EINVAL, "multiple of 16"),
            (dict(rot=80), q4.Q4_EINVAL, "rot_dim"), (dict(rot=-16), q4.Q4_EINVAL, "rot_dim"),
            (dict(max_pos=0), q4.Q4_EINVAL, "max_pos"), (dict(positions=None), q4.Q4_EINVAL, "null positions"),
            (dict(cos_sin=None), q4.Q4_EINVAL, "null cos_sin"), (dict(cos_sin=A + 4), q4.Q4_EALIGN, "cos_sin"),
            (dict(q_gamma=A + 8), q4.Q4_EALIGN, "q_gamma"), (dict(eps=-1.0), q4.Q4_EINVAL, "eps"),
            (dict(eps=float("nan")), q4.Q4_EINVAL, "eps"), (dict(q=A + 8), q4.Q4_EALIGN, "row of q"),
            (dict(qs=255), q4.Q4_EINVAL, "token stride"), (dict(qs=258), q4.Q4_EALIGN, "row of q"),
            (dict(dtype=2, kos=132), q4.Q4_EALIGN, "row of k_out"), (dict(dtype=3), q4.Q4_EINVAL, "dtype")]:
        refused(lib, "qk_norm_rope", ROPE, code, text, **kw)


def test_cache_refusals(lib):
    bad = [(dict(k_qs=None), q4.Q4_EINVAL, "null cache pointer"), (dict(v_d=None), q4.Q4_EINVAL, "null cache pointer"),
           (dict(num_pages=0), q4.Q4_EINVAL, "num_pages"), (dict(page_size=12), q4.Q4_EINVAL, "power of two"),
           (dict(page_size=0), q4.Q4_EINVAL, "power of two"), (dict(head_dim=40), q4.Q4_EINVAL, "multiple of 32"),
           (dict(head_dim=512), q4.Q4_EINVAL, "up to 256"), (dict(num_kv_heads=0), q4.Q4_EINVAL, "key heads"),
           (dict(num_kv_heads=1 << 20), q4.Q4_EINVAL, "2^20"), (dict(num_pages=1 << 30), q4.Q4_EINVAL, "rows"),
           (dict(k_qs=A + 8), q4.Q4_EALIGN, "k_qs"), (dict(v_d=A + 2), q4.Q4_EALIGN, "v_d")]
    for name, base in (("kv4_write", WRITE), ("kv4_read", READ), ("kv4_attention", ATTN)):
        refused(lib, name, base, q4.Q4_EINVAL, "null cache", cache=None)
        for kw, code, text in bad:
            refused(lib, name, base, code, text, cache=cache(**kw))
    for name, base in (("kv4_write", WRITE), ("kv4_read", READ)):
        refused(lib, name, base, q4.Q4_EINVAL, "T must", T=0)
        refused(lib, name, base, q4.Q4_EINVAL, "T must", T=(1 << 30) + 1)
        refused(lib, name, base, q4.Q4_EINVAL, "null slots", slots=None)
        refused(lib, name, base, q4.Q4_EALIGN, "slots", slots=A + 2)
        refused(lib, name, base, q4.Q4_EINVAL, "token stride", ks=127)
        refused(lib, name, base, q4.Q4_EALIGN, "row of v", v=A + 8)
        refused(lib, name, base, q4.Q4_EINVAL, "dtype", dtype=-1)
    refused(lib, "kv4_write", WRITE, q4.Q4_EINVAL, "null k", k=None)
    refused(lib, "kv4_read", READ, q4.Q4_EINVAL, "null k_out and v_out", k=None, v=None)


def test_attention_refusals(lib):
    for kw, code, text in [
            (dict(M=0), q4.Q4_EINVAL, "outside 1..16"), (dict(M=17), q4.Q4_EINVAL, "outside 1..16"),
            (dict(B=0), q4.Q4_EINVAL, "1..1024"), (dict(B=1025), q4.Q4_EINVAL, "1..1024"),
            (dict(Hq=5), q4.Q4_EINVAL, "multiple of the key heads"), (dict(Hq=0), q4.Q4_EINVAL, "multiple of the key heads"),
            (dict(max_pages=0), q4.Q4_EINVAL, "max_pages"), (dict(max_pages=1 << 28), q4.Q4_EINVAL, "2^30"),
            (dict(scale=0.0), q4.Q4_EINVAL, "scale"), (dict(scale=float("inf")), q4.Q4_EINVAL, "scale"),
            (dict(scale=float("nan")), q4.Q4_EINVAL, "scale"), (dict(scale=2e30), q4.Q4_EINVAL, "scale"), (dict(window=-1), q4.Q4_EINVAL, "window"),
            (dict(q=None), q4.Q4_EINVAL, "null q"), (dict(out=None), q4.Q4_EINVAL, "null out"),
            (dict(out=A + 8), q4.Q4_EALIGN, "row of out"), (dict(lse=A + 2), q4.Q4_EALIGN, "lse"),
            (dict(table=None), q4.Q4_EINVAL, "null block_table"), (dict(lens=None), q4.Q4_EINVAL, "null seq_lens"),
            (dict(qs=250), q4.Q4_EINVAL, "token stride"), (dict(dtype=7), q4.Q4_EINVAL, "dtype")]:
        refused(lib, "kv4_attention", ATTN, code, text, **kw)
    refused(lib, "kv4_attention", ATTN, q4.Q4_EINVAL, "64, 128 or 256", cache=cache(head_dim=96))
    n = ctypes.c_size_t(0)
    assert lib.kv4_attention_workspace(None, 1, 4, 2, 64, 0) == q4.Q4_EINVAL
    assert lib.kv4_attention_workspace(ctypes.byref(n), 17, 4, 2, 64, 0) == q4.Q4_EINVAL
    assert lib.kv4_attention_workspace(ctypes.byref(n), 1, 4, 2, 32, 0) == q4.Q4_EINVAL


def test_the_binding_refuses_before_it_calls():
    qs, d = torch.zeros(2, 2, 16, 32, dtype=torch.uint8), torch.zeros(2, 2, 16, 2, dtype=torch.float16)
    with pytest.raises(TypeError, match="CUDA"):
        q4.KV4Cache(qs, d, qs, d)
    with pytest.raises(ValueError, match="head_dim"):
        q4.KV4Cache(qs, d, qs, d[..., :1])
    with pytest.raises(ValueError, match="num_pages"):
        q4.KV4Cache(qs[0], d, qs, d)
    x = torch.zeros(3, 2, 64)
    with pytest.raises(TypeError, match="CUDA"):
        q4.qk_norm_rope(x, x, x, x, None, None, None, None)
    with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
        q4.qk_norm_rope(x, x, x.double(), x, None, None, None, None)


def test_token_rows():
    rows = lambda t: q4._rows(t, t.shape[-2] * t.shape[-1], torch.float32, -1, "t")[1]  # noqa: E731
    base = torch.zeros(4, 3, 10, 32)
    assert rows(base) == 320 and rows(base[:, :, 2:7]) == 320
    assert rows(base[:, :1]) == 960 and rows(base[:1, :1]) == 320
    assert rows(base[0]) == 320 and rows(base[:, 0, :4]) == 960
    for bad in (base[:, :2], base[..., ::2, :], base.transpose(-1, -2), base[..., :16]):
        with pytest.raises(ValueError):
            rows(bad)
    with pytest.raises(TypeError):
        q4._rows(base, 320, torch.float16, -1, "t")


def test_a_cache_of_too_many_rows_is_refused_by_the_binding():
    """Sizes past 32 bits, which the struct would take modulo 2^32."""
    for pages in (1 << 26, (1 << 32) + 4):
        qs, d = (torch.empty(pages, 2, 16, n, dtype=t, device="meta") for n, t in ((32, torch.uint8), (2, torch.float16)))
        with pytest.raises(ValueError, match="rows"):
            q4.KV4Cache(qs, d, qs, d)
