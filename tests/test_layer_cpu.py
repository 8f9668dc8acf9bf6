"""The layer's operators without a GPU: their oracle, and what they refuse before touching CUDA."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import layer as L
from sparse_attention_token_02_b200 import _lib, api


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from sparse_attention_token_02_b200 import build
        build.build()
    return _lib.load()


# ------------------------------------------------------------------------------------------- the oracle


def test_oracle_norm_by_hand():
    s, y = L.rmsnorm([[3.0, 4.0]], [1.0, 2.0], 0.0, [[0.0, 0.0]])
    assert np.allclose(s, [[3, 4]]) and np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    assert np.array_equal(L.group_scales(np.array([[448.0, -896.0, 0.0]]), 2), [[2.0, 1.0]])
    assert np.array_equal(L.group_scales(np.array([[448.0, -896.0, 0.0]]), 0), [[2.0]])


def test_oracle_pow2_scale_and_rows():
    assert [L.pow2_scale(a) for a in (448.0, 448.5, 224.0, 0.0, 1.75, 1.76)] == [1.0, 2.0, 0.5, 1.0, 2.0 ** -8, 2.0 ** -7]
    table = np.array([[2, -1], [0, 9]])
    rows = [L.page_row(table, 4, 3, s, p) for s, p in ((0, 0), (0, 3), (0, 4), (1, 2), (1, 5), (1, 8), (2, 0), (0, -1))]
    assert rows == [8, 11, -1, 2, -1, -1, -1, -1]


def test_oracle_attention_by_hand():
    q, keys = np.array([[1.0, 0.0]]), np.array([[0.0, 5.0], [np.log(3.0), 1.0]])
    out, lse, mag, _ = L.attend(q, keys, 2, 1.0)
    assert np.allclose(out, [[0.75 * np.log(3.0), 0.25 * 5 + 0.75]]) and np.allclose(lse, np.log(4.0))
    assert np.allclose(mag, np.abs(out))
    out, lse, _, _ = L.attend(q, keys[:0], 2, 1.0)
    assert not out.any() and np.isneginf(lse).all()


# ------------------------------------------------------------------------------------------- refusals

P = ctypes.c_void_p


def _name(st):
    return _lib.STATUS_NAMES[st]


NORM = dict(x=0x10000, dtype=_lib.DSA_BF16, x_stride=256, residual=0x20000, residual_out=0x30000, weight=0x40000,
            weight_dtype=_lib.DSA_BF16, rows=4, d=256, eps=1e-6, group=128, codes=0x50000, scale=0x60000, normed=None)


@pytest.mark.parametrize("change,expect", [
    (dict(rows=-1), "INVALID_ARG"), (dict(d=0), "INVALID_ARG"), (dict(d=24), "INVALID_ARG"),
    (dict(d=32784, x_stride=32784), "UNSUPPORTED"), (dict(group=64), "UNSUPPORTED"), (dict(eps=-1.0), "INVALID_ARG"),
    (dict(eps=float("nan")), "INVALID_ARG"), (dict(dtype=_lib.DSA_FP8_E4M3), "INVALID_ARG"),
    (dict(weight_dtype=_lib.DSA_FP8_E4M3), "INVALID_ARG"), (dict(x=None), "INVALID_ARG"), (dict(weight=None), "INVALID_ARG"),
    (dict(codes=None), "INVALID_ARG"), (dict(scale=None), "INVALID_ARG"), (dict(residual_out=None), "INVALID_ARG"),
    (dict(residual=None), "INVALID_ARG"), (dict(x_stride=240), "INVALID_ARG"), (dict(x_stride=260), "INVALID_ARG"),
    (dict(x=0x10008), "INVALID_ARG"), (dict(normed=0x70002), "INVALID_ARG"), (dict(codes=0x50008), "INVALID_ARG"),
])
def test_norm_refusals(lib, change, expect):
    a = {**NORM, **change}
    v = [P(a[k]) if k in ("x", "residual", "residual_out", "weight", "codes", "scale", "normed") else a[k]
         for k in ("x", "dtype", "x_stride", "residual", "residual_out", "weight", "weight_dtype", "rows", "d", "eps",
                   "group", "codes", "scale", "normed")]
    assert _name(lib.dsa_rmsnorm_fp8(*v, None)) == "DSA_ERR_" + expect, lib.dsa_get_last_error()
    assert lib.dsa_get_last_error()


def test_norm_of_no_rows_touches_nothing(lib):
    assert lib.dsa_rmsnorm_fp8(None, 0, 0, None, None, None, 0, 0, 256, 1e-6, 128, None, None, None, None) == 0


def _cache(**change):
    a = dict(latent=0x100000, scale=None, rope=0x200000, num_pages=8, page_size=64, d_c=512, d_r=64, dtype=_lib.DSA_BF16)
    a.update(change)
    return _lib.LatentCacheView(*a.values())


def _table(**change):
    a = dict(pages=0x300000, num_seqs=2, max_pages=4)
    a.update(change)
    return _lib.PageTable(*a.values())


CACHES = [
    (dict(latent=None), {}, "INVALID_ARG"), ({}, dict(pages=None), "INVALID_ARG"), (dict(dtype=_lib.DSA_F32), {}, "INVALID_ARG"),
    (dict(dtype=_lib.DSA_FP8_E4M3), {}, "INVALID_ARG"), (dict(d_c=256), {}, "UNSUPPORTED"), (dict(d_r=32), {}, "UNSUPPORTED"),
    (dict(rope=None), {}, "INVALID_ARG"), (dict(num_pages=0), {}, "INVALID_ARG"), (dict(page_size=0), {}, "INVALID_ARG"),
    (dict(num_pages=1 << 25, page_size=64), {}, "INVALID_ARG"), ({}, dict(num_seqs=0), "INVALID_ARG"),
    ({}, dict(max_pages=0), "INVALID_ARG"), (dict(latent=0x100008), {}, "INVALID_ARG"), (dict(rope=0x200008), {}, "INVALID_ARG"),
]


@pytest.mark.parametrize("cache,table,expect", CACHES)
def test_cache_refusals(lib, cache, table, expect):
    c, t, r = _cache(**cache), _table(**table), _lib.Rope(64, 1, 10000.0)
    q = _lib.LatentQuery(0x400000, 65536, 512, 0x500000, 8192, 64, 4, 128)
    got = [lib.dsa_latent_append_rope(ctypes.byref(c), ctypes.byref(t), P(0x600000), 576, P(0x700000), 576, 0, P(0x800000),
                                      P(0x900000), 4, ctypes.byref(r), None),
           lib.dsa_sparse_attention(ctypes.byref(q), ctypes.byref(c), ctypes.byref(t), P(0x600000), P(0x700000), 16, 0.1,
                                    P(0x800000), None, None, 0, None),
           lib.dsa_prefix_attention(ctypes.byref(q), ctypes.byref(c), ctypes.byref(t), P(0x600000), P(0x700000), 4, 0, 16,
                                    0.1, P(0x800000), None, None, 0, None)]
    assert [_name(s) for s in got] == ["DSA_ERR_" + expect] * 3, lib.dsa_get_last_error()


@pytest.mark.parametrize("change,expect", [
    (dict(n=-1), "INVALID_ARG"), (dict(dtype=_lib.DSA_FP8_E4M3), "INVALID_ARG"), (dict(c=None), "INVALID_ARG"),
    (dict(kr=None), "INVALID_ARG"), (dict(seq=None), "INVALID_ARG"), (dict(pos=None), "INVALID_ARG"),
    (dict(c=0x600008), "INVALID_ARG"), (dict(c_stride=516), "INVALID_ARG"), (dict(c_stride=504), "INVALID_ARG"),
    (dict(kr_stride=32), "INVALID_ARG"), (dict(rope_dim=66), "UNSUPPORTED"), (dict(rope_dim=3), "UNSUPPORTED"),
    (dict(rope_dim=-2), "UNSUPPORTED"), (dict(base=0.0), "INVALID_ARG"), (dict(base=float("inf")), "INVALID_ARG"),
])
def test_append_refusals(lib, change, expect):
    a = dict(c=0x600000, c_stride=576, kr=0x700000, kr_stride=576, dtype=_lib.DSA_BF16, seq=0x800000, pos=0x900000, n=4,
             rope_dim=64, base=10000.0)
    a.update(change)
    c, t, r = _cache(), _table(), _lib.Rope(a["rope_dim"], 1, a["base"])
    st = lib.dsa_latent_append_rope(ctypes.byref(c), ctypes.byref(t), P(a["c"]), a["c_stride"], P(a["kr"]), a["kr_stride"],
                                    a["dtype"], P(a["seq"]), P(a["pos"]), a["n"], ctypes.byref(r), None)
    assert _name(st) == "DSA_ERR_" + expect, lib.dsa_get_last_error()


@pytest.mark.parametrize("change,expect", [
    (dict(T=-1), "INVALID_ARG"), (dict(H=0), "UNSUPPORTED"), (dict(H=129), "UNSUPPORTED"), (dict(latent=None), "INVALID_ARG"),
    (dict(qrope=None), "INVALID_ARG"), (dict(latent=0x400008), "INVALID_ARG"), (dict(st=65532), "INVALID_ARG"),
    (dict(sh=516), "INVALID_ARG"), (dict(T=1 << 24, H=128), "UNSUPPORTED"), (dict(seq=None), "INVALID_ARG"),
    (dict(idx=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(out=0x800008), "INVALID_ARG"),
    (dict(scale=float("nan")), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
    (dict(scale=0.0), "INVALID_ARG"), (dict(scale=-0.1), "INVALID_ARG"),
])
def test_attention_refusals(lib, change, expect):
    a = dict(T=4, H=128, latent=0x400000, qrope=0x500000, st=65536, sh=512, seq=0x600000, idx=0x700000, out=0x800000, scale=0.1)
    a.update(change)
    c, t = _cache(), _table()
    q = _lib.LatentQuery(a["latent"], a["st"], a["sh"], a["qrope"], 8192, 64, a["T"], a["H"])
    got = [lib.dsa_sparse_attention(ctypes.byref(q), ctypes.byref(c), ctypes.byref(t), P(a["seq"]), P(a["idx"]), 16, a["scale"],
                                    P(a["out"]), None, None, 0, None),
           lib.dsa_prefix_attention(ctypes.byref(q), ctypes.byref(c), ctypes.byref(t), P(a["seq"]), P(a["idx"]), 4, 0, 16,
                                    a["scale"], P(a["out"]), None, None, 0, None)]
    assert [_name(s) for s in got] == ["DSA_ERR_" + expect] * 2, lib.dsa_get_last_error()


def test_attention_sizes_refused(lib):
    c, t = _cache(), _table()
    q = _lib.LatentQuery(0x400000, 65536, 512, 0x500000, 8192, 64, 4, 128)
    for top_k in (0, -1, (1 << 30) + 1):
        st = lib.dsa_sparse_attention(ctypes.byref(q), ctypes.byref(c), ctypes.byref(t), P(0x600000), P(0x700000), top_k, 0.1,
                                      P(0x800000), None, None, 0, None)
        assert _name(st) == "DSA_ERR_INVALID_ARG"
    for prefix, seq, most in ((-1, 0, 16), (20, 0, 16), (4, 2, 16), (4, -1, 16), (4, 0, (1 << 30) + 1)):
        st = lib.dsa_prefix_attention(ctypes.byref(q), ctypes.byref(c), ctypes.byref(t), P(0x600000), P(0x700000), prefix, seq,
                                      most, 0.1, P(0x800000), None, None, 0, None)
        assert _name(st) == "DSA_ERR_INVALID_ARG", (prefix, seq, most)
    q.T = 0                                                  # nothing to do: no pointer is touched
    assert lib.dsa_sparse_attention(ctypes.byref(q), ctypes.byref(c), ctypes.byref(t), None, None, 4, 0.1, None, None, None, 0,
                                    None) == 0
    assert lib.dsa_prefix_attention(ctypes.byref(q), ctypes.byref(c), ctypes.byref(t), None, None, 0, 0, 0, 0.1, None, None,
                                    None, 0, None) == 0
    assert lib.dsa_sparse_attention_workspace_bytes(0, 128, 16, _lib.DSA_BF16) == 0
    assert lib.dsa_prefix_attention_workspace_bytes(64, 16, 32768, 33792, _lib.DSA_BF16) > 0    # parts to be joined
    assert lib.dsa_prefix_attention_workspace_bytes(4, 128, 100, 50, _lib.DSA_BF16) == 0


def test_binding_refusals():
    cache = api.LatentCache.empty(2, 64, device="cpu")
    ids = torch.zeros(3, dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32)
    q, qr = torch.zeros(3, 4, 512, dtype=torch.bfloat16), torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="seq_ids must be int32"):
        api.dsa_sparse_attention(q, qr, cache, table, ids.long(), torch.zeros(3, 4, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError, match="idx must have shape"):
        api.dsa_sparse_attention(q, qr, cache, table, ids, torch.zeros(2, 4, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError, match="q_latent must be"):
        api.dsa_prefix_attention(q[:, :, :256], qr, cache, table, ids, ids, 0.1)
    with pytest.raises(TypeError, match="q_rope must be bf16"):
        api.dsa_prefix_attention(q, qr.float(), cache, table, ids, ids, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        api.dsa_prefix_attention(q, qr, cache, table, ids, ids, 0.1)
    with pytest.raises(ValueError, match="kr_new must be"):
        api.dsa_latent_append_rope(cache, table, torch.zeros(3, 512), None, ids, ids)
    with pytest.raises(TypeError, match="one dtype"):
        api.dsa_latent_append_rope(cache, table, torch.zeros(3, 512), torch.zeros(3, 64, dtype=torch.bfloat16), ids, ids)
    with pytest.raises(ValueError, match="contiguous rows"):
        api.dsa_rmsnorm_fp8(torch.zeros(16, 32).t(), torch.zeros(16))
    with pytest.raises(ValueError, match="group"):
        api.dsa_rmsnorm_fp8(torch.zeros(16, 32), torch.zeros(32), group=64)


def test_compiled_calls_answer_only_plain_ones():
    # built with the library; a call that it does not make itself is left to the Python form, without an error of its own
    calls = api._layer_calls
    assert calls is not None
    _lib.load()
    x = torch.zeros(2, 128)
    assert calls.rmsnorm(x, x[0], 1e-6, None, 128, None, None, None, None) is None
    assert calls.rmsnorm(None, 3, "eps", x, [], None, None, None, None) is None
    assert calls.rmsnorm() is None and calls.append(1) is None and calls.sparse(x) is None and calls.prefix() is None
    idx = torch.zeros(2, 1, dtype=torch.int32)
    ids = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 16, 512, dtype=torch.bfloat16)
    assert calls.sparse(q, q[:, :, :64], x, None, None, 64, idx, ids, idx, 1.0, None, None, None) is None
    with pytest.raises(TypeError):
        calls.bind(1, 2)
