"""The paged 8-bit cache without a GPU: refusals of the entry points and the binding, the host
tensors' refusal, and the 64-bit reference forms of tests/kv_reference.py against torch."""
import ctypes
import math

import numpy as np
import pytest
import torch

from gated_linear_attention_liger_b200 import build as libbuild
from gated_linear_attention_liger_b200 import ops
from tests import kv_reference as ref


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return ops.load()


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


def _assign(lib, **kw):
    a = dict(new=16, lens=16, table=16, ring=16, span=16, slots=16, cu=16, lo=16, so=16, B=2, width=4, n=8, bs=16, N=4)
    a.update(kw)
    return lib.liger_kv_cache_assign(*(_p(a[x]) for x in ("new", "lens", "table", "ring", "span", "slots", "cu", "lo", "so")),
                                     a["B"], a["width"], a["n"], a["bs"], a["N"], None)


def _append(lib, **kw):
    a = dict(k=16, v=16, slots=16, cache=16, scales=16, N=2, Hkv=2, d=64, n=8, bs=16, ks=128, vs=128, dt=0, kv=0)
    a.update(kw)
    return lib.liger_kv_cache_append(*(_p(a[x]) for x in ("k", "v", "slots", "cache", "scales")), a["N"], a["Hkv"], a["d"],
                                     a["n"], a["bs"], a["ks"], a["vs"], a["dt"], a["kv"], None)


def _attend(lib, **kw):
    a = dict(q=16, cache=16, scales=16, table=16, lens=16, out=16, B=2, nq=1, Hq=4, Hkv=2, d=64, width=4, n=8, bs=16, qs=256,
             dt=0, kv=0, ws=16, wsb=1 << 30)
    a.update(kw)
    return lib.liger_attn_cached(*(_p(a[x]) for x in ("q", "cache", "scales", "table", "lens", "out")), a["B"], a["nq"], a["Hq"],
                                 a["Hkv"], a["d"], a["width"], a["n"], a["bs"], a["qs"], a["dt"], a["kv"], _p(a["ws"]),
                                 a["wsb"], None)


INVALID, UNSUPPORTED = ops.LIGER_ERR_INVALID_ARG, ops.LIGER_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(width=0), INVALID), (dict(n=0), INVALID), (dict(bs=0), INVALID), (dict(N=-1), INVALID),
    (dict(new=None), INVALID), (dict(slots=None), INVALID), (dict(so=None), INVALID), (dict(slots=20), INVALID),
    (dict(lens=18), INVALID), (dict(bs=48), UNSUPPORTED), (dict(bs=256), UNSUPPORTED), (dict(B=8193), UNSUPPORTED),
    (dict(n=1 << 27, bs=16), UNSUPPORTED), (dict(width=1 << 27, bs=16), UNSUPPORTED), (dict(N=2 ** 31 - 1), UNSUPPORTED),
])
def test_assign_rejects(lib, kw, status):
    assert _assign(lib, **kw) == status
    assert lib.liger_last_error().decode() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INVALID), (dict(Hkv=0), INVALID), (dict(dt=5), INVALID), (dict(kv=2), INVALID), (dict(ks=64), INVALID),
    (dict(vs=132), INVALID), (dict(k=None), INVALID), (dict(cache=8), INVALID), (dict(scales=4), INVALID), (dict(slots=2), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(n=1 << 28), UNSUPPORTED), (dict(Hkv=70000, ks=1 << 23, vs=1 << 23), UNSUPPORTED),
])
def test_append_rejects(lib, kw, status):
    assert _append(lib, **kw) == status
    assert lib.liger_last_error().decode() != ""


def test_append_of_nothing_is_ok(lib):
    assert _append(lib, N=0, k=None, v=None, slots=None) == ops.LIGER_OK


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=3), INVALID), (dict(Hkv=0), INVALID), (dict(nq=0), INVALID), (dict(B=0), INVALID), (dict(qs=128), INVALID),
    (dict(qs=260), INVALID), (dict(dt=2), INVALID), (dict(kv=-1), INVALID), (dict(q=None), INVALID), (dict(out=8), INVALID),
    (dict(ws=None), INVALID), (dict(wsb=1024), INVALID), (dict(scales=4), INVALID), (dict(lens=2), INVALID),
    (dict(nq=17), UNSUPPORTED), (dict(d=32), UNSUPPORTED), (dict(bs=512), UNSUPPORTED), (dict(B=9000), UNSUPPORTED),
    (dict(Hkv=256, Hq=256, qs=256 * 64, n=1 << 24, bs=16), UNSUPPORTED),
    (dict(B=8192, width=1 << 20, bs=128), UNSUPPORTED),
])
def test_attention_rejects(lib, kw, status):
    assert _attend(lib, **kw) == status
    assert lib.liger_last_error().decode() != ""


def test_workspace_size(lib):
    assert ops.cached_attention_workspace_size(96) == 0
    assert 0 < ops.cached_attention_workspace_size(64) < ops.cached_attention_workspace_size(128)


def _cache(n=4, Hkv=2, bs=16, d=64, dtype=torch.int8):
    c = ops.kv_cache_new(n, Hkv, d, bs, 3, 40, dtype=dtype, device="cpu")
    return c


def test_new_cache_is_empty():
    c = _cache()
    assert c["cache"].shape == (4, 2, 2, 16, 64) and c["scales"].shape == (4, 2, 2)
    assert c["block_table"].shape == (3, 3) and c["free_blocks"].tolist() == [0, 1, 2, 3]
    assert c["free_span"].tolist() == [0, 4] and int(c["seq_lens"].sum()) == 0
    with pytest.raises(TypeError, match="cache dtype"):
        _cache(dtype=torch.uint8)


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    c = _cache()
    i32 = dict(dtype=torch.int32)
    new = torch.ones(3, **i32)
    state = (c["seq_lens"], c["block_table"], c["free_blocks"], c["free_span"], 16, 8)
    with pytest.raises(ValueError, match="CUDA"):
        ops.kv_cache_assign(new, *state)
    with pytest.raises(ValueError, match="int32"):
        ops.kv_cache_assign(new.long(), *state)
    with pytest.raises(ValueError, match="seq_lens must have shape"):
        ops.kv_cache_assign(new[:2], *state)
    with pytest.raises(ValueError, match="slot_map must have shape"):
        ops.kv_cache_assign(new, *state, slot_map=torch.zeros(7, **i32))
    with pytest.raises(ValueError, match="free_span_out must be"):
        ops.kv_cache_assign(new, *state, free_span_out=torch.zeros(2))
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(5, **i32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.kv_cache_append(k, k, slots, c["cache"], c["scales"])
    with pytest.raises(ValueError, match="v must have shape"):
        ops.kv_cache_append(k, k[:4], slots, c["cache"], c["scales"])
    with pytest.raises(ValueError, match="v must be"):
        ops.kv_cache_append(k, k.float(), slots, c["cache"], c["scales"])
    with pytest.raises(ValueError, match="slot_map must be"):
        ops.kv_cache_append(k, k, slots.long(), c["cache"], c["scales"])
    with pytest.raises(ValueError, match="strides"):
        ops.kv_cache_append(k.transpose(0, 1).contiguous().transpose(0, 1), k, slots, c["cache"], c["scales"])
    with pytest.raises(ValueError, match="contiguous"):
        ops.kv_cache_append(k, k, slots, c["cache"].transpose(1, 2).contiguous().transpose(1, 2), c["scales"])
    with pytest.raises(ValueError, match="scales must have shape"):
        ops.kv_cache_append(k, k, slots, c["cache"], c["scales"][:2])
    with pytest.raises(TypeError, match="float16"):
        ops.kv_cache_append(k.half(), k.half(), slots, c["cache"], c["scales"])
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    args = (c["cache"], c["scales"], c["block_table"], c["seq_lens"])
    with pytest.raises(ValueError, match="CUDA"):
        ops.cached_attention(q, *args)
    with pytest.raises(ValueError, match="q must be"):
        ops.cached_attention(q[..., :32], *args)
    with pytest.raises(ValueError, match="block_table must"):
        ops.cached_attention(q[:2], *args)
    with pytest.raises(ValueError, match="out must"):
        ops.cached_attention(q, *args, out=torch.zeros(3, 4, 64))


def test_token_strides():
    x = torch.zeros(6, 10, 64)
    assert ops._token_stride(x[:, 2:4], "k", 2, 64) == 640
    assert ops._token_stride(x.view(2, 3, 10, 64)[:, :, :4], "q", 4, 64) == 640
    assert ops._token_stride(x.view(2, 3, 10, 64)[:, :1, :4], "q", 4, 64) == 1920
    assert ops._token_stride(x[:1, :2], "k", 2, 64) == 128       # one token
    with pytest.raises(ValueError):
        ops._token_stride(x.view(2, 3, 10, 64)[:, :2, :4], "q", 4, 64)
    with pytest.raises(ValueError):
        ops._token_stride(x[:, ::2], "k", 5, 64)


def test_reference_codes_match_torch():
    x = np.concatenate([np.linspace(-500, 500, 4001), np.linspace(-0.1, 0.1, 4001), [np.inf, -np.inf, 0.0]])
    t = torch.tensor(np.clip(x, -448, 448), dtype=torch.float32)
    got = ref.to_code_values(t.double().numpy(), torch.float8_e4m3fn)
    np.testing.assert_array_equal(got, ref.decode(t.to(torch.float8_e4m3fn)))
    assert ref.scale_of(448.0, torch.float8_e4m3fn) == 1.0 and ref.scale_of(448.1, torch.float8_e4m3fn) == 2.0
    assert ref.scale_of(0.0, torch.int8) == 2.0 ** -64 and ref.scale_of(127.0, torch.int8) == 1.0


def test_reference_attention_matches_torch():
    rng = np.random.default_rng(1)
    B, nq, Hq, Hkv, d, bs = 3, 2, 4, 2, 64, 16
    values, scales = np.rint(rng.normal(0, 30, (9, Hkv, 2, bs, d))), np.exp2(rng.integers(-7, -3, (9, Hkv, 2)).astype(float))
    table = rng.permutation(9).reshape(B, 3)
    lens = [48, 17, 1]
    q = rng.normal(size=(B, nq, Hq, d))
    out = ref.attention(q, values, scales, table, lens)[0]
    for s, n in enumerate(lens):
        kv = (values * scales[..., None, None])[table[s]].transpose(2, 1, 0, 3, 4).reshape(2, Hkv, 48, d)[:, :, :n]
        kv = torch.tensor(np.repeat(kv, Hq // Hkv, 1))
        for i in range(nq):
            e = n - nq + i + 1
            want = np.zeros((Hq, d)) if e <= 0 else torch.nn.functional.scaled_dot_product_attention(
                torch.tensor(q[s, i])[:, None], kv[0, :, :e], kv[1, :, :e])[:, 0].numpy()
            np.testing.assert_allclose(out[s, i], want, atol=1e-12)


def test_reference_assign_hands_out_each_block_once():
    rng = np.random.default_rng(2)
    B, width, bs, n = 5, 6, 16, 14
    table, ring, span, lens = [[-1] * width for _ in range(B)], list(range(n)), [3, n], [0] * B
    for _ in range(60):
        new = [int(x) for x in rng.choice([-1, 0, 1, 5, 20, 40], B)]
        _, _, lens, span = ref.assign(new, lens, table, ring, span, bs, 100)
        used = [table[s][j] for s in range(B) for j in range(-(-lens[s] // bs))]
        free = [ring[(span[0] + i) % n] for i in range(span[1])]
        assert sorted(used + free) == list(range(n))
