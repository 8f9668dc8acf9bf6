"""The layer's operators on the GPU (RMS norm to FP8, paged latent append, attention over a selection and over
a shared prefix) against oracle/layer.py in fp64.

Tolerances, from the formats (half a step: bf16 2^-8, E4M3 2^-4 of the value, fp32 2^-24):
* norm: a row's sum of squares takes at most 32 + 10 fp32 additions on any path, halved by the root, and five
  more roundings follow: below 2^-18 relative for y and the scales.
* rotation: fp32 products of fp32 sines: 2^-21 of the pair's magnitudes beside bf16's half step.
* attention: a score is 36 accumulations of 16 products, each within two fp32 steps of the sum of magnitudes A
  (ds = 36 * 2^-22 A, and 2^-22 of the score for its scaling); weights carry exp(ds) and bf16's half step, so
  |out - exact| <= (2^-8 + 2 ds + 2^-18) * sum |w_j c_j| + 2^-8 |out|, and lse is within ds + 2^-20 (1 + |lse|).
"""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from oracle import e4m3_decode, e4m3_encode
from oracle import layer as L
from sparse_attention_token_02_b200 import _lib, api

pytestmark = pytest.mark.gpu

SM = 1.0 / np.sqrt(192.0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    api.dsa_version()
    yield
    api.dsa_check_device_errors()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------------------------------------ norm


@pytest.mark.parametrize("rows,d,dtype,wdtype,residual,group,pad", [
    (1, 16, "bf16", "bf16", False, 128, 0), (3, 112, "bf16", "f32", True, 128, 16), (5, 128, "f32", "bf16", True, 0, 0),
    (4, 7168, "bf16", "bf16", True, 128, 0), (2, 7168, "f32", "f32", True, 128, 64), (7, 1536, "f32", "bf16", False, 0, 576),
    (9, 2064, "bf16", "bf16", True, 128, 48), (2, 16384, "bf16", "bf16", False, 0, 0), (1, 32768, "bf16", "f32", True, 128, 0),
    (1, 32752, "f32", "bf16", False, 128, 0), (300, 576, "bf16", "bf16", True, 0, 8),
])
def test_norm(rows, d, dtype, wdtype, residual, group, pad):
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    g = gen(rows * d)
    x = torch.randn(rows, d + pad, generator=g).to(dt[dtype])[:, :d]
    x[0, d // 2:] = 0                                       # groups of zeros (where there is no residual)
    res = (4 * torch.randn(rows, d, generator=g)).to(dt[dtype]) if residual else None
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(dt[wdtype])
    xc = x.cuda() if not pad else torch.nn.functional.pad(x, (0, pad)).cuda()[:, :d]
    assert xc.stride(0) == d + pad or rows == 1
    normed = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    codes, scale, out = api.dsa_rmsnorm_fp8(xc, w.cuda(), 1e-6, residual=None if res is None else res.cuda(), group=group,
                                            normed=normed)
    s, y = L.rmsnorm(f64(x), f64(w), 1e-6, None if res is None else f64(res))
    ref = L.group_scales(y, group)
    assert np.all(np.abs(f64(scale) - ref) <= 2.0 ** -18 * ref)
    assert np.all(np.abs(f64(normed) - y) <= (2.0 ** -8 + 2.0 ** -17) * np.abs(y))
    wide = np.repeat(f64(scale), group or d, axis=1)[:, :d]
    got = e4m3_decode(codes.cpu().numpy()) * wide
    step = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * wide)   # half a step; below 2^-6 of the scale steps are equal
    assert np.all(np.abs(got - y) <= step + 2.0 ** -17 * np.abs(y))
    if residual:
        assert torch.equal(out.cpu(), (x.float() + res.float()).to(dt[dtype]))
    else:
        assert out is None


def test_norm_in_place_residual_zero_rows_and_a_nan_row():
    d = 1024
    x, r = torch.randn(5, d, generator=gen(1)), torch.randn(5, d, generator=gen(2))
    x[1], r[1] = 0, 0
    x[3, 7] = float("nan")
    w = torch.ones(d)
    res = r.cuda()
    codes, scale, out = api.dsa_rmsnorm_fp8(x.cuda(), w.cuda(), 1e-6, residual=res, residual_out=res)
    assert out is res and torch.equal(res[:3].cpu(), (x + r)[:3])
    assert not codes[1].any() and (scale[1] == 1).all()
    clean = [0, 2, 4]
    c2, s2, _ = api.dsa_rmsnorm_fp8(x[clean].cuda(), w.cuda(), 1e-6, residual=r[clean].cuda())
    assert torch.equal(codes[clean], c2) and torch.equal(scale[clean], s2)
    empty = api.dsa_rmsnorm_fp8(torch.empty(0, d, device="cuda"), w.cuda())
    assert empty[0].shape == (0, d) and empty[1].shape == (0, 8)


def test_norm_agrees_with_the_row_quantiser():
    # the FP8 rows are those of the framework's quantiser on the same fp32 rows, up to a code where a product
    # with the reciprocal and a quotient fall on two sides of a border
    x = torch.randn(64, 2048, generator=gen(3)).cuda()
    w = torch.ones(2048, device="cuda")
    codes, scale, _ = api.dsa_rmsnorm_fp8(x, w, 0.0, group=0)
    y = (x.double() / x.double().square().mean(1, keepdim=True).sqrt()).float()
    c2, s2 = api.dsa_quantize_rows_fp8(y)
    assert torch.allclose(scale[:, 0], s2, rtol=2.0 ** -18, atol=0)
    assert (codes != c2).float().mean() < 1e-3


# ------------------------------------------------------------------------------------------------ append


def make_table(seqs, pages, num_pages, seed):
    return torch.randperm(num_pages, generator=gen(seed))[:seqs * pages].view(seqs, pages).to(torch.int32)


@pytest.mark.parametrize("n,page,fp8,src,rope_dim,interleaved,d_r", [
    (1, 64, False, "bf16", 64, True, 64), (9, 1, True, "bf16", 64, False, 64), (33, 16, True, "f32", 64, True, 64),
    (33, 48, False, "f32", 32, False, 64), (17, 16, False, "bf16", 2, True, 64), (17, 16, True, "bf16", 0, True, 64),
    (40, 256, True, "bf16", 64, True, 0), (24, 64, False, "bf16", 64, False, 0), (25, 16, False, "f32", 6, False, 64),
])
def test_append(n, page, fp8, src, rope_dim, interleaved, d_r):
    g = gen(n * page + rope_dim)
    dt = torch.bfloat16 if src == "bf16" else torch.float32
    seqs, pages = 4, -(-2 * n // page) + 3
    num_pages = seqs * pages + 2
    table = make_table(seqs, pages, num_pages, 5)
    both = (torch.randn(n, 512 + 64 + 16, generator=g) * torch.exp(4 * torch.randn(n, 1, generator=g))).to(dt)
    both[0, :512] = 0
    if n > 4:                                               # absmax on a power of two times 448, and just above it
        both[1, :512] = both[1, :512].clamp(-3.5, 3.5)
        both[1, 5] = 3.5
        both[2, :512] = both[2, :512].clamp(-3.5, 3.5)
        both[2, 9] = -3.53125
        both[3, :512] *= 1e-36
    seq = torch.arange(n) % seqs
    pos = (torch.arange(n) // seqs) * 2 + page                # every other position, from the second page on
    cache = api.LatentCache.empty(num_pages, page, fp8=fp8, d_r=d_r)
    cache.latent.fill_(3)
    if d_r:
        cache.rope.fill_(7)
    dev = both.cuda()
    api.dsa_latent_append_rope(cache, table.cuda(), dev[:, :512], dev[:, 520:584] if d_r else None, seq.to(torch.int32).cuda(),
                               pos.to(torch.int32).cuda(), rope_dim=rope_dim, interleaved=interleaved)
    api.dsa_check_device_errors()
    rows = [L.page_row(table.numpy(), page, num_pages, int(s), int(p)) for s, p in zip(seq, pos)]
    assert len(set(rows)) == n and min(rows) >= 0
    lat, scale, rot = L.append_values(f64(both[:, :512]), f64(both[:, 520:584]), pos.numpy(), fp8, rope_dim, 10000.0, interleaved)
    if fp8:
        assert np.array_equal(cache.latent.cpu().numpy()[rows], lat)
        assert np.array_equal(f64(cache.scale)[rows], scale)
    else:
        assert torch.equal(cache.latent.cpu()[rows], both[:, :512].to(torch.bfloat16))
    if d_r:
        mag = np.abs(f64(both[:, 520:584])).max(1, keepdims=True)
        assert np.all(np.abs(f64(cache.rope)[rows] - rot) <= 2.0 ** -8 * np.abs(rot) + 2.0 ** -20 * mag)
    others = np.setdiff1d(np.arange(num_pages * page), rows)
    assert (cache.latent.cpu()[others] == 3).all() and (not d_r or (cache.rope.cpu()[others] == 7).all())


def test_append_far_positions():
    n, page = 8, 64
    pos = torch.tensor([0, 1, 131071, 1000003, 9999991, 16777217, 33554431, 40000000], dtype=torch.int32)
    pages = 40000000 // page + 1
    table = torch.full((1, pages), -1, dtype=torch.int32)
    table[0, (pos // page).unique()] = torch.arange(len((pos // page).unique()), dtype=torch.int32)
    cache = api.LatentCache.empty(n, page)
    c, kr = torch.randn(n, 512, generator=gen(8)), torch.randn(n, 64, generator=gen(9))
    api.dsa_latent_append_rope(cache, table.cuda(), c.cuda(), kr.cuda(), torch.zeros(n, dtype=torch.int32).cuda(), pos.cuda())
    api.dsa_check_device_errors()
    rows = [L.page_row(table.numpy(), page, n, 0, int(p)) for p in pos]
    _, _, rot = L.append_values(f64(c), f64(kr), pos.numpy(), False, 64, 10000.0, True)
    assert np.all(np.abs(f64(cache.rope)[rows] - rot) <= 2.0 ** -8 * np.abs(rot) + 2.0 ** -20 * f64(kr.abs().amax(1, keepdim=True)))


def test_append_skips_padding_and_reports_what_has_no_page():
    page, num_pages = 16, 6
    table = torch.tensor([[0, 1, -1], [5, 6, 2]], dtype=torch.int32)
    # good, padding, no page, page past the cache, past the table, negative position, no such sequence, good
    seq = torch.tensor([0, -1, 0, 1, 1, 0, 2, 1], dtype=torch.int32)
    pos = torch.tensor([17, 3, 33, 20, 48, -1, 0, 40], dtype=torch.int32)
    c, kr = torch.randn(8, 512, generator=gen(1)).bfloat16(), torch.randn(8, 64, generator=gen(2)).bfloat16()
    cache = api.LatentCache.empty(num_pages, page)
    args = (table.cuda(), c.cuda(), kr.cuda(), seq.cuda(), pos.cuda())
    api.dsa_latent_append_rope(cache, *args)
    with pytest.raises(RuntimeError, match="DEVICE_CHECK.*page table for token [2-6]"):
        api.dsa_check_device_errors()
    want = torch.zeros(num_pages * page, 512, dtype=torch.bfloat16)
    want[17], want[2 * 16 + 8] = c[0], c[7]
    assert torch.equal(cache.latent.cpu(), want)
    keep = [0, 1, 7]                                         # padding alone is no fault
    api.dsa_latent_append_rope(cache, args[0], *(t[keep] for t in args[1:]))
    api.dsa_check_device_errors()
    assert torch.equal(cache.latent.cpu(), want)
    api.dsa_latent_append_rope(cache, args[0], *(t[:0] for t in args[1:]))


# ------------------------------------------------------------------------------------------------ attention


def make_cache(rows, page, fp8, seed, d_r=64):
    """(cache, its values in fp64 [rows, 512 + d_r])."""
    g = gen(seed)
    lat, rope = torch.randn(rows, 512, generator=g), torch.randn(rows, 64, generator=g).bfloat16()
    cache = api.LatentCache.empty(rows // page, page, fp8=fp8, d_r=d_r)
    if fp8:
        scale = np.array([L.pow2_scale(a) for a in f64(lat.abs().amax(1))])
        codes = e4m3_encode(f64(lat) / scale[:, None])
        cache.latent.copy_(torch.from_numpy(codes))
        cache.scale.copy_(torch.from_numpy(scale).float())
        vals = e4m3_decode(codes) * scale[:, None]
    else:
        cache.latent.copy_(lat.bfloat16())
        vals = f64(lat.bfloat16())
    if d_r:
        cache.rope.copy_(rope)
        vals = np.concatenate([vals, f64(rope)], 1)
    return cache, vals


def queries(T, H, seed, mult=1.0):
    g = gen(seed)
    return (mult * torch.randn(T, H, 512, generator=g)).bfloat16(), (mult * torch.randn(T, H, 64, generator=g)).bfloat16()


def check_token(got, got_lse, q, keys, sm, what):
    out, lse, mag, A = L.attend(q, keys, 512, sm)
    ds = 36 * 2.0 ** -22 * A + 2.0 ** -22 * A
    if len(keys) == 0:
        assert not got.any() and np.isneginf(got_lse).all(), what
        return
    err = np.abs(got - out) - ((2.0 ** -8 + 2 * ds + 2.0 ** -18) * mag + 2.0 ** -8 * np.abs(out))
    assert err.max() <= 0, (what, float(err.max()))
    lerr = np.abs(got_lse - lse) - (ds + 2.0 ** -20 * (1 + np.abs(lse)))
    assert lerr.max() <= 0, (what, float(lerr.max()))


SELECT = [
    # T, H, k, page, fp8, d_r, length, mult
    (1, 1, 1, 64, False, 64, 70, 1), (1, 128, 2048, 64, False, 64, 4100, 1), (3, 128, 65, 16, False, 64, 300, 1),
    (2, 16, 64, 1, True, 64, 130, 1), (5, 24, 129, 48, True, 64, 1000, 1), (4, 64, 513, 64, True, 64, 700, 1),
    (2, 96, 200, 256, False, 0, 500, 1), (3, 65, 63, 64, True, 0, 200, 1), (2, 128, 300, 64, False, 64, 400, 30),
    (160, 8, 70, 64, False, 64, 200, 1), (2, 33, 4099, 64, True, 64, 5000, 1),
]


@pytest.mark.parametrize("T,H,k,page,fp8,d_r,length,mult", SELECT)
def test_sparse_attention(T, H, k, page, fp8, d_r, length, mult):
    rng = np.random.default_rng(T * k + H)
    seqs = min(T, 3)
    pages = -(-length // page)
    num_pages = seqs * pages + 1
    cache, vals = make_cache(num_pages * page, page, fp8, T + k, d_r)
    table = make_table(seqs, pages, num_pages, 4)
    seq = torch.from_numpy(rng.integers(0, seqs, T).astype(np.int32))
    idx = np.stack([rng.permutation(length)[:k] for _ in range(T)]).astype(np.int32)
    idx[rng.random(idx.shape) < 0.2] = -1                    # holes anywhere
    idx[0, -1] = length - 1
    if T > 1:
        idx[1] = -1                                          # a row that selects nothing
    if T > 2:
        idx[2, 1:] = -1                                      # and one that selects a single key
        idx[2, 0] = 0
    ql, qr = queries(T, H, k, mult)
    out, lse = api.dsa_sparse_attention(ql.cuda(), qr.cuda() if d_r else None, cache, table.cuda(), seq.cuda(),
                                        torch.from_numpy(idx).cuda(), SM)
    api.dsa_check_device_errors()
    q = f64(torch.cat([ql, qr], 2) if d_r else ql)
    out, lse = f64(out), f64(lse)
    for t in list(range(min(T, 6))) + [T - 1]:
        rows = [L.page_row(table.numpy(), page, num_pages, int(seq[t]), int(p)) for p in idx[t] if p >= 0]
        check_token(out[t], lse[t], q[t], vals[rows], SM, t)


def test_sparse_attention_masked_places_hold_anything():
    # keys that no query names are NaN and infinite; whole tiles of the selection are empty; positions repeat
    cache, vals = make_cache(512, 64, False, 1)
    bad = np.arange(256, 512)
    cache.latent[bad[:128]] = float("nan")
    cache.latent[bad[128:]] = float("inf")
    cache.rope[bad] = float("nan")
    table = torch.arange(8, dtype=torch.int32).view(1, 8)
    idx = np.full((3, 320), -1, np.int32)
    idx[0, 200] = 5                                          # only the fourth tile has an entry
    idx[1, ::7] = np.arange(46)
    idx[2, :6] = [9, 9, 9, 200, 200, 3]
    ql, qr = queries(3, 40, 2)
    out, lse = api.dsa_sparse_attention(ql.cuda(), qr.cuda(), cache, table.cuda(), torch.zeros(3, dtype=torch.int32).cuda(),
                                        torch.from_numpy(idx).cuda(), SM)
    q = f64(torch.cat([ql, qr], 2))
    for t in range(3):
        check_token(f64(out)[t], f64(lse)[t], q[t], vals[[p for p in idx[t] if p >= 0]], SM, t)


def test_sparse_attention_rising_scores():
    # one query direction, keys along it with growing lengths: the running maximum rises in every tile, by far
    # more than any head start that the sums allow, and falls in the other order
    n = 640
    cache, _ = make_cache(n, 64, False, 3)
    cache.latent.zero_()
    cache.rope.zero_()
    cache.latent[:, 0] = torch.arange(n).bfloat16().cuda() / 4
    cache.latent[:, 1] = (torch.arange(n) % 5).bfloat16().cuda()
    vals = np.concatenate([f64(cache.latent), f64(cache.rope)], 1)
    ql, qr = torch.zeros(2, 70, 512).bfloat16(), torch.zeros(2, 70, 64).bfloat16()
    ql[:, :, 0] = (torch.arange(70) + 1) / 4                   # up to 17.5 * 160 = 2800 in the exponent
    idx = torch.stack([torch.arange(n), torch.arange(n).flip(0)]).to(torch.int32)
    table = torch.arange(10, dtype=torch.int32).view(1, 10)
    out, lse = api.dsa_sparse_attention(ql.cuda(), qr.cuda(), cache, table.cuda(), torch.zeros(2, dtype=torch.int32).cuda(),
                                        idx.cuda(), 1.0)
    for t in range(2):
        check_token(f64(out)[t], f64(lse)[t], f64(torch.cat([ql, qr], 2))[t], vals[idx[t].numpy()], 1.0, t)


def test_sparse_attention_padding_and_faults():
    cache, vals = make_cache(8 * 16, 16, True, 6)
    table = torch.tensor([[0, 1, 2, 3], [4, -1, 8, 5]], dtype=torch.int32)      # page 8 does not exist
    seq = torch.tensor([-1, 0, 1], dtype=torch.int32)
    idx = torch.tensor([[0, 1, 2], [60, -1, 0], [15, 50, -1]], dtype=torch.int32)
    ql, qr = queries(3, 20, 5)
    q = f64(torch.cat([ql, qr], 2))

    def run(s, i):
        o, l = api.dsa_sparse_attention(ql.cuda(), qr.cuda(), cache, table.cuda(), s.cuda(), i.cuda(), SM)
        return f64(o), f64(l)

    out, lse = run(seq, idx)
    api.dsa_check_device_errors()
    rows = [[], [60, 0], [4 * 16 + 15, 5 * 16 + 2]]
    for t in range(3):
        check_token(out[t], lse[t], q[t], vals[rows[t]], SM, t)
    for bad in (17, 40, 64, 10 ** 9):                        # no page, a page past the cache, past the table
        i = idx.clone()
        i[2, 2] = bad
        out, lse = run(seq, i)
        with pytest.raises(RuntimeError, match="DEVICE_CHECK.*page table for token 2"):
            api.dsa_check_device_errors()
        check_token(out[2], lse[2], q[2], vals[rows[2]], SM, bad)    # the key is left out
    out, lse = run(torch.tensor([0, 2, 1], dtype=torch.int32), idx)  # no such sequence
    with pytest.raises(RuntimeError, match="DEVICE_CHECK.*page table for token 1"):
        api.dsa_check_device_errors()
    assert not out[1].any() and np.isneginf(lse[1]).all()


def test_sparse_attention_far_rows():
    # byte offsets past 2^32: a 5.4 GB cache, the page table naming its last pages
    page, num_pages = 64, 82000
    cache = api.LatentCache(torch.zeros(num_pages * page, 512, dtype=torch.bfloat16, device="cuda"),
                            torch.zeros(num_pages * page, 64, dtype=torch.bfloat16, device="cuda"), None, page)
    table = torch.tensor([[num_pages - 1, num_pages - 2, 65536, 65535]], dtype=torch.int32)
    n = 4 * page
    c, kr = torch.randn(n, 512, generator=gen(1)).bfloat16(), torch.randn(n, 64, generator=gen(2)).bfloat16()
    api.dsa_latent_append_rope(cache, table.cuda(), c.cuda(), kr.cuda(), torch.zeros(n, dtype=torch.int32).cuda(),
                               torch.arange(n, dtype=torch.int32).cuda(), rope_dim=0)
    ql, qr = queries(1, 128, 3)
    out, lse = api.dsa_sparse_attention(ql.cuda(), qr.cuda(), cache, table.cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
                                        torch.arange(n, dtype=torch.int32).cuda()[None], SM)
    api.dsa_check_device_errors()
    check_token(f64(out)[0], f64(lse)[0], f64(torch.cat([ql, qr], 2))[0], f64(torch.cat([c, kr], 1)), SM, 0)


def test_attention_strides():
    cache, vals = make_cache(256, 64, False, 2)
    table = torch.arange(4, dtype=torch.int32).view(1, 4).cuda()
    T, H = 3, 72
    ql, qr = queries(T, H, 1)
    idx = torch.stack([torch.randperm(256, generator=gen(t))[:100] for t in range(T)]).to(torch.int32).cuda()
    seq = torch.zeros(T, dtype=torch.int32).cuda()
    ref = api.dsa_sparse_attention(ql.cuda(), qr.cuda(), cache, table, seq, idx, SM)
    lt = ql.transpose(0, 1).contiguous().cuda().transpose(0, 1)           # heads outermost, as a batched product leaves them
    joint = torch.cat([qr, torch.zeros(T, H, 40).bfloat16()], 2).cuda()[:, :, :64]
    got = api.dsa_sparse_attention(lt, joint, cache, table, seq, idx, SM)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    again = api.dsa_sparse_attention(lt, joint, cache, table, seq, idx, SM)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    no_lse = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda")
    lib = _lib.load()                                        # no lse wanted, the stream's own workspace
    q = _lib.LatentQuery(lt.data_ptr(), lt.stride(0), lt.stride(1), joint.data_ptr(), joint.stride(0), joint.stride(1), T, H)
    cc, pt = cache.c(), _lib.PageTable(table.data_ptr(), 1, 4)
    V = ctypes.c_void_p
    _lib.check(lib.dsa_sparse_attention(ctypes.byref(q), ctypes.byref(cc), ctypes.byref(pt), V(seq.data_ptr()),
                                        V(idx.data_ptr()), 100, SM, V(no_lse.data_ptr()), None, None, 0,
                                        V(torch.cuda.current_stream().cuda_stream)))
    assert torch.equal(no_lse, ref[0])


PREFIX = [
    # T, H, prefix, longest own part, page, fp8, d_r
    (1, 128, 0, 1, 64, False, 64), (1, 16, 1, 1, 16, False, 64), (3, 128, 130, 70, 64, False, 64), (5, 24, 1000, 64, 48, True, 64),
    (9, 16, 64, 300, 64, True, 64), (4, 8, 500, 0, 1, False, 64), (2, 96, 77, 200, 256, True, 0), (70, 1, 200, 5, 64, False, 64),
    (2, 128, 5000, 3000, 64, False, 64),
]


@pytest.mark.parametrize("T,H,prefix,own,page,fp8,d_r", PREFIX)
def test_prefix_attention(T, H, prefix, own, page, fp8, d_r):
    rng = np.random.default_rng(T * H + prefix)
    full = prefix // page                                    # whole pages that all sequences share
    pages = -(-(prefix + own) // page) + 1
    num_pages = full + T * (pages - full)
    cache, vals = make_cache(num_pages * page, page, fp8, prefix + own, d_r)
    table = torch.cat([torch.arange(full).expand(T, full),
                       full + torch.randperm(T * (pages - full), generator=gen(1)).view(T, pages - full)], 1).to(torch.int32)
    src = table[T - 1, full].item() * page                   # each sequence's copy of the page that the prefix ends in
    for t in range(T):
        dst = table[t, full].item() * page
        for x in (cache.latent, cache.scale, cache.rope):
            if x is not None:
                x[dst:dst + prefix % page] = x[src:src + prefix % page].clone()
        vals[dst:dst + prefix % page] = vals[src:src + prefix % page]
    lens = prefix + rng.integers(0, own + 1, T)
    lens[0] = prefix + own
    if T > 2:
        lens[1] = prefix // 2                                # stops inside the shared part
        lens[2] = 0
    seq = torch.arange(T, dtype=torch.int32)
    if T > 4:
        seq[4] = -1
    ql, qr = queries(T, H, prefix)
    args = (ql.cuda(), qr.cuda() if d_r else None, cache, table.cuda(), seq.cuda(), torch.from_numpy(lens.astype(np.int32)).cuda(), SM)
    out, lse = api.dsa_prefix_attention(*args, prefix_len=prefix, prefix_seq=T - 1, max_keys=prefix + own)
    api.dsa_check_device_errors()
    q = f64(torch.cat([ql, qr], 2) if d_r else ql)
    o64, l64 = f64(out), f64(lse)
    for t in sorted(set(range(min(T, 6))) | {T - 1}):
        n = lens[t] if seq[t] >= 0 else 0
        rows = [L.page_row(table.numpy(), page, num_pages, t, p) for p in range(n)]
        check_token(o64[t], l64[t], q[t], vals[rows], SM, t)
    again = api.dsa_prefix_attention(*args, prefix_len=prefix, prefix_seq=T - 1, max_keys=prefix + own)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    alone = api.dsa_prefix_attention(*args)                  # nothing shared, the page table's own bound
    for t in sorted(set(range(min(T, 6))) | {T - 1}):
        n = lens[t] if seq[t] >= 0 else 0
        rows = [L.page_row(table.numpy(), page, num_pages, t, p) for p in range(n)]
        check_token(f64(alone[0])[t], f64(alone[1])[t], q[t], vals[rows], SM, t)


def test_prefix_attention_cuts_and_reports_a_length_past_its_bound():
    cache, vals = make_cache(256, 64, False, 4)
    table = torch.arange(4, dtype=torch.int32).view(1, 4).expand(3, 4).contiguous()
    ql, qr = queries(3, 16, 1)
    lens = torch.tensor([100, 120, -7], dtype=torch.int32)
    out, lse = api.dsa_prefix_attention(ql.cuda(), qr.cuda(), cache, table.cuda(), torch.arange(3, dtype=torch.int32).cuda(),
                                        lens.cuda(), SM, prefix_len=64, max_keys=100)
    with pytest.raises(RuntimeError, match="DEVICE_CHECK.*page table for token 1"):
        api.dsa_check_device_errors()
    for t, n in enumerate((100, 100, 0)):
        check_token(f64(out)[t], f64(lse)[t], f64(torch.cat([ql, qr], 2))[t], vals[:n], SM, t)


def test_prefix_attention_of_no_keys():
    cache, _ = make_cache(64, 64, False, 4)
    table = torch.zeros(3, 1, dtype=torch.int32).cuda()
    ql, qr = (t.cuda() for t in queries(3, 70, 1))
    out = torch.full((3, 70, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32).cuda()
    _, lse = api.dsa_prefix_attention(ql, qr, cache, table, lens, lens, SM, max_keys=0, out=out)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("T,H,prefix,own,hole", [(40, 16, 8000, 30, False), (40, 16, 8000, 30, True), (5, 128, 8100, 0, False)])
def test_prefix_attention_fp8_prefix_of_many_rows(T, H, prefix, own, hole):
    # enough rows read the prefix for it to be expanded once; a page that does not exist is left out and reported
    page = 64
    full = prefix // page
    pages = -(-(prefix + own) // page)
    num_pages = full + T * (pages - full) + 1
    cache, vals = make_cache(num_pages * page, page, True, T)
    table = torch.cat([torch.arange(full).expand(T, full), full + torch.arange(T * (pages - full)).view(T, pages - full)], 1).to(torch.int32)
    if hole:
        table[0, 3] = -1
    src = table[0, full].item() * page if prefix % page else 0
    for t in range(1, T):
        dst = table[t, full].item() * page if prefix % page else 0
        for x in (cache.latent, cache.scale, cache.rope):
            x[dst:dst + prefix % page] = x[src:src + prefix % page].clone()
        vals[dst:dst + prefix % page] = vals[src:src + prefix % page]
    lens = torch.full((T,), prefix + own, dtype=torch.int32)
    lens[1] = prefix + own // 2
    lens[2] = 100
    seq = torch.arange(T, dtype=torch.int32)
    seq[3] = -1
    ql, qr = queries(T, H, 5)
    out, lse = api.dsa_prefix_attention(ql.cuda(), qr.cuda(), cache, table.cuda(), seq.cuda(), lens.cuda(), SM, prefix_len=prefix,
                                        max_keys=prefix + own)
    if hole:
        with pytest.raises(RuntimeError, match="DEVICE_CHECK.*page table"):
            api.dsa_check_device_errors()
    else:
        api.dsa_check_device_errors()
    q = f64(torch.cat([ql, qr], 2))
    for t in (0, 1, 2, 3, T - 1):
        n = int(lens[t]) if seq[t] >= 0 else 0
        rows = [L.page_row(table.numpy(), page, num_pages, 0 if p < prefix else t, p) for p in range(n)]
        check_token(f64(out)[t], f64(lse)[t], q[t], vals[[r for r in rows if r >= 0]], SM, t)


def test_prefix_attention_many_parts():
    # one token's few heads over a long cache: more parts than the joining kernel's threads take in one round
    n, page = 70001, 64
    cache, vals = make_cache(-(-n // page) * page, page, False, 3)
    table = torch.randperm(-(-n // page), generator=gen(1)).to(torch.int32).view(1, -1)
    ql, qr = queries(1, 9, 2)
    lens = torch.tensor([n], dtype=torch.int32)
    out, lse = api.dsa_prefix_attention(ql.cuda(), qr.cuda(), cache, table.cuda(), torch.zeros(1, dtype=torch.int32).cuda(), lens.cuda(),
                                        SM, max_keys=n)
    api.dsa_check_device_errors()
    rows = (table[0].long()[torch.arange(n) // page] * page + torch.arange(n) % page).numpy()
    check_token(f64(out)[0], f64(lse)[0], f64(torch.cat([ql, qr], 2))[0], vals[rows], SM, 0)


def test_fp8_nan_codes_reach_the_rows_that_read_them():
    cache, vals = make_cache(128, 64, True, 5)
    cache.latent[70, 17] = 0x7F
    cache.latent[71, 300] = 0xFF
    table = torch.arange(2, dtype=torch.int32).view(1, 2).cuda()
    ql, qr = queries(3, 12, 3)
    idx = torch.tensor([[1, 2, 3], [1, 70, 3], [71, -1, 2]], dtype=torch.int32)
    out, lse = api.dsa_sparse_attention(ql.cuda(), qr.cuda(), cache, table, torch.zeros(3, dtype=torch.int32).cuda(), idx.cuda(), SM)
    check_token(f64(out)[0], f64(lse)[0], f64(torch.cat([ql, qr], 2))[0], vals[[1, 2, 3]], SM, 0)
    assert torch.isnan(lse[1:]).all() and torch.isnan(out[1:]).all()


# ------------------------------------------------------------------------------------------------ together


def test_layer_step_as_used():
    """Two decode steps of a layer: norm, append to both caches, score and select, attend; graph-captured for the
    second, replayed on another stream than the one that captured it."""
    S, L0, H, k, page = 3, 300, 128, 128, 64
    g = gen(11)
    pages = -(-(L0 + 8) // page)
    table = make_table(S, pages, S * pages, 3).cuda()
    cache = api.LatentCache.empty(S * pages, page, fp8=True)
    cap = L0 + 8
    icache = api.IndexerKCache.empty(S * cap, 128, fp8=False)
    hist = torch.randn(S, L0 + 2, 512 + 64, generator=g).bfloat16()
    ikeys = torch.randn(S, L0 + 2, 128, generator=g).bfloat16()
    iq = torch.randn(2, S, 64, 128, generator=g).bfloat16()
    iw = torch.softmax(torch.randn(2, S, 64, generator=g), 2)
    ql, qr = queries(2 * S, H, 12)
    hidden, resid = torch.randn(2, S, 7168, generator=g).bfloat16(), torch.randn(S, 7168, generator=g).bfloat16()
    w = torch.ones(7168).bfloat16().cuda()
    seq = torch.arange(S, dtype=torch.int32).cuda()
    # the prompt
    allseq = torch.arange(S, dtype=torch.int32).repeat_interleave(L0).cuda()
    allpos = torch.arange(L0, dtype=torch.int32).repeat(S).cuda()
    h = hist[:, :L0].reshape(S * L0, 576).cuda()
    api.dsa_latent_append_rope(cache, table, h[:, :512], h[:, 512:], allseq, allpos)
    dst = (torch.arange(S)[:, None] * cap + torch.arange(L0)).reshape(-1).cuda()
    api.dsa_indexer_kcache_append(icache, ikeys[:, :L0].reshape(S * L0, 128).contiguous().cuda(), dst)
    res = resid.cuda()
    base = np.arange(S, dtype=np.int64) * cap
    outs = []
    bufs = dict(c=torch.empty(S, 576, dtype=torch.bfloat16, device="cuda"), ik=torch.empty(S, 128, dtype=torch.bfloat16, device="cuda"),
                row=torch.empty(S, dtype=torch.int64, device="cuda"), pos=torch.empty(S, dtype=torch.int32, device="cuda"),
                iq=torch.empty(S, 64, 128, dtype=torch.bfloat16, device="cuda"), iw=torch.empty(S, 64, device="cuda"),
                ql=torch.empty(S, H, 512, dtype=torch.bfloat16, device="cuda"), qr=torch.empty(S, H, 64, dtype=torch.bfloat16, device="cuda"),
                x=torch.empty(S, 7168, dtype=torch.bfloat16, device="cuda"))

    def fill(step):
        bufs["c"].copy_(hist[:, L0 + step])
        bufs["ik"].copy_(ikeys[:, L0 + step])
        bufs["row"].copy_(torch.from_numpy(base) + L0 + step)
        bufs["pos"].fill_(L0 + step)
        bufs["iq"].copy_(iq[step])
        bufs["iw"].copy_(iw[step])
        bufs["ql"].copy_(ql[step * S:(step + 1) * S])
        bufs["qr"].copy_(qr[step * S:(step + 1) * S])
        bufs["x"].copy_(hidden[step])

    def step(length):
        codes, scale, _ = api.dsa_rmsnorm_fp8(bufs["x"], w, residual=res, residual_out=res)
        api.dsa_latent_append_rope(cache, table, bufs["c"][:, :512], bufs["c"][:, 512:], seq, bufs["pos"])
        api.dsa_indexer_kcache_append(icache, bufs["ik"], bufs["row"])
        idx, _ = api.dsa_indexer_decode(bufs["iq"], icache, bufs["iw"], [length] * S, [1] * S, k, k_base=base)
        o, l = api.dsa_sparse_attention(bufs["ql"], bufs["qr"], cache, table, seq, idx, SM)
        return codes, scale, idx, o, l

    fill(0)
    outs.append([t.clone() for t in step(L0 + 1)])
    side = torch.cuda.Stream()
    fill(1)
    side.wait_stream(torch.cuda.current_stream())
    saved = (res.clone(), cache.latent.clone(), icache.k.clone())
    with torch.cuda.stream(side):
        step(L0 + 2)                                         # the uncaptured call that the indexer wants before a capture
        res.copy_(saved[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            captured = step(L0 + 2)
    torch.cuda.synchronize()
    res.copy_(saved[0])
    cache.latent.copy_(saved[1])
    icache.k.copy_(saved[2])
    graph.replay()
    torch.cuda.synchronize()
    outs.append(list(captured))
    api.dsa_check_device_errors()
    with torch.cuda.stream(side):
        api.dsa_check_device_errors()
    lat, scale, rot = L.append_values(f64(hist[:, :, :512]).reshape(-1, 512), f64(hist[:, :, 512:]).reshape(-1, 64),
                                      np.tile(np.arange(L0 + 2), S), True, 64, 10000.0, True)
    vals = np.concatenate([e4m3_decode(lat) * scale[:, None], f64(torch.from_numpy(rot).bfloat16())], 1).reshape(S, L0 + 2, 576)
    s = f64(resid)
    for n, (codes, sc, idx, o, l) in enumerate(outs):
        s, y = L.rmsnorm(f64(hidden[n]), np.ones(7168), 1e-6, s)
        s = f64(torch.from_numpy(s).float().bfloat16())
        got = e4m3_decode(codes.cpu().numpy()) * np.repeat(f64(sc), 128, axis=1)
        assert np.all(np.abs(got - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * np.repeat(f64(sc), 128, axis=1)) + 2.0 ** -17 * np.abs(y))
        for b in range(S):
            pos = idx[b].cpu().numpy()
            assert pos.min() >= 0 and pos.max() <= L0 + n and len(set(pos)) == k
            # the cache's rotated parts are bf16 roundings of fp32 rotations: their own half step, times |q_r|, enters the scores
            q = f64(torch.cat([ql, qr], 2))[n * S + b]
            out, lse, mag, A = L.attend(q, vals[b][pos], 512, SM)
            ds = 37 * 2.0 ** -22 * A + SM * 2.0 ** -7 * np.abs(q[:, 512:]).sum(1).max() * 4 * 2.0 ** -10
            assert np.all(np.abs(f64(o)[b] - out) <= (2.0 ** -8 + 2 * ds + 2.0 ** -18) * mag + 2.0 ** -8 * np.abs(out))
            assert np.all(np.abs(f64(l)[b] - lse) <= ds + 2.0 ** -20 * (1 + np.abs(lse)))


def test_two_graphs_at_once_and_another_stream():
    # two captures of split attentions, replayed at the same time on two streams, against eager results
    cache, _ = make_cache(64 * 64, 64, False, 9)
    table = torch.arange(64, dtype=torch.int32).view(1, 64).cuda()
    seq = torch.zeros(2, dtype=torch.int32).cuda()
    idx = torch.stack([torch.randperm(4096, generator=gen(t))[:2048] for t in range(2)]).to(torch.int32).cuda()
    lens = torch.tensor([4096, 4000], dtype=torch.int32).cuda()
    ql, qr = (t.cuda() for t in queries(2, 128, 3))
    want = (api.dsa_sparse_attention(ql, qr, cache, table, seq, idx, SM),
            api.dsa_prefix_attention(ql, qr, cache, table, seq, lens, SM, prefix_len=2000, max_keys=4096))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    graphs, got = [], []
    for s, call in zip(streams, (lambda: api.dsa_sparse_attention(ql, qr, cache, table, seq, idx, SM),
                                 lambda: api.dsa_prefix_attention(ql, qr, cache, table, seq, lens, SM, prefix_len=2000, max_keys=4096))):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=streams[0]):
            got.append(call())
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with torch.cuda.stream(streams[1]):                      # eager on a stream that is handed over, twice in a row
        pass
    outs = [api.dsa_sparse_attention(ql, qr, cache, table, seq, idx, SM, stream=streams[1]) for _ in range(2)]
    streams[1].synchronize()
    assert all(torch.equal(o[0], want[0][0]) for o in outs)
    for s in streams:
        api.dsa_check_device_errors(s)


def test_first_calls_on_a_stream_may_be_captured():
    # a stream the library has not seen: the call's context and its own workspace appear inside the capture
    cache, vals = make_cache(64 * 64, 64, False, 9)
    table = torch.arange(64, dtype=torch.int32).view(1, 64).cuda()
    ids, lens = torch.zeros(40, dtype=torch.int32).cuda(), torch.full((40,), 4096, dtype=torch.int32).cuda()
    ql, qr = (t.cuda() for t in queries(40, 16, 3))
    want = api.dsa_prefix_attention(ql, qr, cache, table, ids, lens, SM, prefix_len=3000, max_keys=4096)[0]
    out = torch.zeros_like(want)
    lib, side, graph = _lib.load(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    q = _lib.LatentQuery(ql.data_ptr(), ql.stride(0), ql.stride(1), qr.data_ptr(), qr.stride(0), qr.stride(1), 40, 16)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        _lib.check(lib.dsa_prefix_attention(q, cache.c(), _lib.PageTable(table.data_ptr(), 1, 64), ids.data_ptr(), lens.data_ptr(), 3000, 0,
                                            4096, SM, out.data_ptr(), None, None, 0, side.cuda_stream))
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    api.dsa_check_device_errors(side)


def test_selection_of_everything_is_dense_attention():
    # the two attentions meet where a selection holds every position (the short-sequence bypass)
    S, n, H = 2, 150, 128
    cache, _ = make_cache(S * 192, 64, True, 7)
    table = make_table(S, 3, 6, 2).cuda()
    seq = torch.arange(S, dtype=torch.int32).cuda()
    ql, qr = (t.cuda() for t in queries(S, H, 4))
    icache = api.IndexerKCache.empty(S * n, 128, fp8=False)
    zq = torch.zeros(S, 64, 128, dtype=torch.bfloat16, device="cuda")
    idx, _ = api.dsa_indexer_decode(zq, icache, torch.ones(S, 64, device="cuda"), [n] * S, [1] * S, 256, scores=False)
    a = api.dsa_sparse_attention(ql, qr, cache, table, seq, idx, SM)
    lens = torch.full((S,), n, dtype=torch.int32, device="cuda")
    b = api.dsa_prefix_attention(ql, qr, cache, table, seq, lens, SM, max_keys=n)
    assert torch.allclose(a[0].float(), b[0].float(), rtol=2.0 ** -6, atol=2.0 ** -7)
    assert torch.allclose(a[1], b[1], rtol=0, atol=2.0 ** -12)


# ------------------------------------------------------------------------------------------------ many rows
# Sizes at which two CTAs share a tile's keys; the tests above reach one CTA, clusters and groups of 16 heads.


@pytest.mark.parametrize("T,H,k,page,fp8,d_r,length,mult", [
    (50, 128, 512, 64, False, 64, 900, 1), (60, 65, 200, 16, False, 64, 500, 1), (60, 96, 130, 64, False, 0, 300, 30),
    (40, 128, 640, 1, False, 64, 700, 1), (75, 100, 300, 48, False, 64, 400, 1),
])
def test_sparse_attention_of_many_rows(T, H, k, page, fp8, d_r, length, mult):
    test_sparse_attention(T, H, k, page, fp8, d_r, length, mult)


@pytest.mark.parametrize("T,H,prefix,own,page,fp8,d_r", [
    (70, 24, 6000, 64, 64, False, 64), (16, 24, 9000, 100, 48, False, 64), (9, 128, 3000, 0, 64, False, 0),
    (23, 128, 3000, 100, 64, True, 64), (40, 128, 500, 1, 16, False, 64),
])
def test_prefix_attention_of_many_rows(T, H, prefix, own, page, fp8, d_r):
    test_prefix_attention(T, H, prefix, own, page, fp8, d_r)


def test_many_rows_of_rising_scores():
    # as above, and a token without a key between the others
    n, T, H = 640, 44, 128
    cache, _ = make_cache(n, 64, False, 3)
    cache.latent.zero_()
    cache.rope.zero_()
    cache.latent[:, 0] = torch.arange(n).bfloat16().cuda() / 4
    cache.latent[:, 300] = (torch.arange(n) % 5).bfloat16().cuda()
    vals = np.concatenate([f64(cache.latent), f64(cache.rope)], 1)
    ql, qr = torch.zeros(T, H, 512).bfloat16(), torch.zeros(T, H, 64).bfloat16()
    ql[:, :, 0] = (torch.arange(H) + 1) / 8                    # up to 16 * 160 = 2560 in the exponent
    idx = torch.stack([torch.arange(n) if t % 2 else torch.arange(n).flip(0) for t in range(T)]).to(torch.int32)
    idx[2] = -1
    table = torch.arange(10, dtype=torch.int32).view(1, 10)
    out, lse = api.dsa_sparse_attention(ql.cuda(), qr.cuda(), cache, table.cuda(), torch.zeros(T, dtype=torch.int32).cuda(),
                                        idx.cuda(), 1.0)
    q = f64(torch.cat([ql, qr], 2))
    for t in (0, 1, 2, T - 1):
        check_token(f64(out)[t], f64(lse)[t], q[t], vals[[p for p in idx[t].tolist() if p >= 0]], 1.0, t)


def test_many_rows_with_anything_in_masked_places():
    cache, vals = make_cache(512, 64, False, 1)
    bad = np.arange(256, 512)
    cache.latent[bad[:128]] = float("nan")
    cache.latent[bad[128:]] = float("inf")
    cache.rope[bad] = float("nan")
    T, H = 48, 128
    table = torch.arange(8, dtype=torch.int32).view(1, 8)
    idx = np.full((T, 330), -1, np.int32)
    idx[0, 200] = 5
    idx[1, ::7] = np.arange(48)
    idx[3:, :40] = np.arange(40)
    idx[T - 1, :6] = [9, 9, 9, 200, 200, 3]
    seq = torch.zeros(T, dtype=torch.int32)
    seq[5] = -1
    ql, qr = queries(T, H, 2)
    args = (ql.cuda(), qr.cuda(), cache, table.cuda(), seq.cuda(), torch.from_numpy(idx).cuda(), SM)
    out, lse = api.dsa_sparse_attention(*args)
    q = f64(torch.cat([ql, qr], 2))
    for t in (0, 1, 2, 3, 5, T - 1):
        keys = [p for p in idx[t] if p >= 0] if seq[t] >= 0 else []
        check_token(f64(out)[t], f64(lse)[t], q[t], vals[keys], SM, t)
    # rows that a page table does not hold are left out and reported; the queries' strides; a captured call
    lens = torch.full((T,), 200, dtype=torch.int32).cuda()
    holes = table.clone()
    holes[0, 1] = -1
    o, l = api.dsa_prefix_attention(args[0], args[1], cache, holes.cuda(), args[4], lens, SM, prefix_len=130, max_keys=500)
    with pytest.raises(_lib.DsaError):
        api.dsa_check_device_errors()
    keys = [p for p in range(200) if not 64 <= p < 128]
    check_token(f64(o)[0], f64(l)[0], q[0], vals[keys], SM, "holes")
    lt = ql.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    joint = torch.cat([qr, torch.zeros(T, H, 40).bfloat16()], 2).cuda()[:, :, :64]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = api.dsa_sparse_attention(lt, joint, *args[2:])
    for _ in range(2):
        got[0].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got[0]) and torch.equal(lse, got[1])


def test_compiled_and_python_calls_agree(monkeypatch):
    # the compiled calls and their Python forms: the same results, given and new outputs, and the same refusals
    assert api._layer_calls is not None
    cache, _ = make_cache(512, 64, False, 1)
    fp8, _ = make_cache(512, 64, True, 2)
    table = torch.arange(8, dtype=torch.int32).view(1, 8).cuda()
    T, H = 3, 40
    ql, qr = (x.cuda() for x in queries(T, H, 2))
    seq = torch.tensor([0, -1, 0], dtype=torch.int32).cuda()
    idx = torch.stack([torch.randperm(512, generator=gen(t))[:200] for t in range(T)]).to(torch.int32).cuda()
    lens = torch.tensor([300, 5, 512], dtype=torch.int32).cuda()
    x, w = torch.randn(5, 320, generator=gen(3)).cuda(), torch.randn(256, generator=gen(4)).bfloat16().cuda()
    pos = torch.tensor([1, 70, 200], dtype=torch.int32).cuda()
    new = torch.randn(3, 700, generator=gen(5)).cuda()

    def calls():
        res = torch.ones(5, 256).cuda()
        given = torch.empty(5, 256, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(5, device="cuda")
        got = [*api.dsa_rmsnorm_fp8(x[:, :256], w, 1e-5, residual=res), *api.dsa_rmsnorm_fp8(x[:, 64:], w, group=0)[:2]]
        codes, scale, out = api.dsa_rmsnorm_fp8(x[:, :256], w, residual=res, residual_out=res, group=0, codes=given[0], scale=given[1],
                                                normed=torch.empty(5, 256, dtype=torch.bfloat16, device="cuda"))
        assert codes is given[0] and scale is given[1] and out is res
        got += [codes.view(torch.uint8), scale, out.clone()]
        for c in (cache, fp8):
            for kw in (dict(rope_dim=32, interleaved=False), dict(base=500.0)):
                api.dsa_latent_append_rope(c, table, new[:, 4:516], new[:, 600:664], seq, pos, **kw)
            got += [c.latent.clone(), c.rope.clone()]
            got += api.dsa_sparse_attention(ql, qr, c, table, seq, idx, SM)
            got += api.dsa_prefix_attention(ql, qr, c, table, seq, lens, SM)
            out, lse = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, device="cuda")
            ws = torch.empty(api.dsa_prefix_attention_workspace_bytes(T, H, 64, 512, c.fp8), dtype=torch.uint8, device="cuda")
            r = api.dsa_prefix_attention(ql, qr, c, table, seq, lens, SM, 64, 0, 512, out=out, lse=lse, workspace=ws)
            assert r[0] is out and r[1] is lse
            got += r
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got += api.dsa_sparse_attention(ql, qr, cache, table, seq, idx, SM, stream=side)
        side.synchronize()
        return got

    def refusals():
        small = torch.empty(16, dtype=torch.uint8, device="cuda")
        for f, kind in (
            (lambda: api.dsa_rmsnorm_fp8(x[:, :200].half(), w[:200]), TypeError),
            (lambda: api.dsa_rmsnorm_fp8(x[:, :200], w[:200]), _lib.DsaError),                   # d % 16
            (lambda: api.dsa_rmsnorm_fp8(x[:, :256], w, residual=torch.ones(5, 255).cuda()), ValueError),
            (lambda: api.dsa_sparse_attention(ql, qr, cache, table, seq, idx.long(), SM), TypeError),
            (lambda: api.dsa_sparse_attention(ql, qr[:, :, ::2], cache, table, seq, idx, SM), ValueError),
            (lambda: api.dsa_sparse_attention(ql, qr, cache, table, seq, idx.cpu(), SM), ValueError),
            (lambda: api.dsa_sparse_attention(ql, qr, cache, table, seq, idx, float("nan")), _lib.DsaError),
            (lambda: api.dsa_prefix_attention(ql, qr, fp8, table, seq, lens, SM, 400, 0, 512, workspace=small), _lib.DsaError),
            (lambda: api.dsa_latent_append_rope(cache, table, new[:, :512], new[:, 600:664], seq[:2], pos), ValueError),
        ):
            with pytest.raises(kind):
                f()

    a = calls()
    refusals()
    monkeypatch.setattr(api, "_layer_calls", None)
    b = calls()
    refusals()
    assert len(a) == len(b) and all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))


@pytest.mark.parametrize("rows,d,dtype,residual,group", [
    (1400, 128, "bf16", True, 128), (900, 2064, "bf16", False, 128), (700, 4112, "f32", True, 128), (650, 4112, "f32", True, 0),
    (640, 8192, "bf16", True, 128), (620, 8176, "f32", False, 0), (5000, 48, "f32", False, 128), (300, 8208, "bf16", True, 128),
])
def test_norm_of_more_rows_than_stay_resident(rows, d, dtype, residual, group):
    # a block takes several rows, the next one's loads under way: each is what it is alone, in place too
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    g = gen(rows + d)
    x, w = torch.randn(rows, d, generator=g).to(dt).cuda(), (1 + 0.2 * torch.randn(d, generator=g)).to(dt).cuda()
    res = (4 * torch.randn(rows, d, generator=g)).to(dt).cuda() if residual else None
    x[rows // 2] = 0
    if residual:
        res[rows // 2] = 0
    x[rows - 2, 3] = float("inf")
    pick = torch.tensor([0, 1, rows // 2, rows // 2 + 1, rows - 3, rows - 2, rows - 1])
    alone = api.dsa_rmsnorm_fp8(x[pick].contiguous(), w, 1e-6, residual=res[pick].contiguous() if residual else None, group=group)
    inplace = res.clone() if residual else None
    codes, scale, out = api.dsa_rmsnorm_fp8(x, w, 1e-6, residual=inplace, residual_out=inplace, group=group)
    assert torch.equal(codes[pick], alone[0]) and torch.equal(scale[pick].view(torch.int32), alone[1].view(torch.int32))
    if residual:
        assert out is inplace and torch.equal(out[pick], alone[2]) and torch.equal(out, (x.float() + res.float()).to(dt))
    finite = torch.arange(rows) != rows - 2
    s, y = L.rmsnorm(f64(x[finite]), f64(w), 1e-6, f64(res[finite]) if residual else None)
    ref = L.group_scales(y, group)
    assert np.all(np.abs(f64(scale)[finite] - ref) <= 2.0 ** -18 * ref)
    wide = np.repeat(f64(scale)[finite], group or d, axis=1)[:, :d]
    got = e4m3_decode(codes.cpu().numpy()[finite]) * wide
    assert np.all(np.abs(got - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * wide) + 2.0 ** -17 * np.abs(y))


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("mag", [2.0 ** -122, 2.0 ** -104, 2.0 ** -98, 2.0 ** 60])
def test_norm_of_small_and_large_values(mag, group):
    # the codes keep their precision where 448 / max|t| would overflow, and a group of such values beside ordinary ones.
    # A sum of squares that underflows to nothing is as far off as eps is large against it: nothing here.
    x = (torch.rand(3, 384, generator=gen(7)) + 0.5) * torch.sign(torch.randn(3, 384, generator=gen(8)))
    x[:2] *= mag
    x[1, 128:256] /= mag if mag < 1 else 1
    x[2, 256:] = 0
    w = torch.ones(384)
    codes, scale, _ = api.dsa_rmsnorm_fp8(x.cuda(), w.cuda(), 1e-6, group=group)
    s, y = L.rmsnorm(f64(x), f64(w), 1e-6)
    ref = L.group_scales(y, group)
    assert np.all(np.abs(f64(scale) - ref) <= 2.0 ** -18 * ref + 2.0 ** -149)      # and half a step of subnormal numbers
    wide = np.repeat(f64(scale), group or 384, axis=1)
    got = e4m3_decode(codes.cpu().numpy()) * wide
    assert np.all(np.abs(got - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * wide) + 2.0 ** -17 * np.abs(y) + 448 * 2.0 ** -149)


def test_calls_from_two_threads():
    # the host path gives up the interpreter's lock while the library works: each thread has its own stream
    import threading

    cache, _ = make_cache(2048, 64, False, 1)
    table = torch.arange(32, dtype=torch.int32).view(1, 32).cuda()
    sizes = [(1, 128, 700), (50, 128, 500), (3, 16, 90)]
    args = []
    for T, H, k in sizes:
        ql, qr = (x.cuda() for x in queries(T, H, k))
        idx = torch.stack([torch.randperm(2048, generator=gen(t))[:k] for t in range(T)]).to(torch.int32).cuda()
        args.append((ql, qr, cache, table, torch.zeros(T, dtype=torch.int32).cuda(), idx, SM))
    x, w = torch.randn(400, 1024, generator=gen(2)).cuda(), torch.ones(1024, device="cuda")
    want = [api.dsa_sparse_attention(*a)[0] for a in args], api.dsa_rmsnorm_fp8(x, w)[0]
    torch.cuda.synchronize()
    bad = []

    def work(order):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got = {i: api.dsa_sparse_attention(*args[i])[0] for i in order}
                    codes = api.dsa_rmsnorm_fp8(x, w)[0]
                    torch.cuda.current_stream().synchronize()
                    if not torch.equal(codes, want[1]) or any(not torch.equal(got[i], want[0][i]) for i in order):
                        bad.append(order)
        except Exception as e:                               # reported by the main thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(o,)) for o in ([0, 1, 2], [2, 1, 0], [1, 0, 2])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    api.dsa_check_device_errors()
