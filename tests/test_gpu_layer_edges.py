"""The layer's operators on the GPU where calls meet: host threads, captures, and rows whose neighbours hold anything.

Results are compared with the same call made alone, bit for bit, or with oracle/layer.py in fp64 under the tolerances
that tests/test_gpu_layer.py derives.
"""

from __future__ import annotations

import ctypes
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import e4m3_decode
from oracle import layer as L
from sparse_attention_token_02_b200 import _lib, api
from .test_gpu_layer import SM, check_token, f64, gen, make_cache, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    api.dsa_version()
    yield
    api.dsa_check_device_errors()


def test_threads_on_one_stream_share_its_workspace():
    # calls without a workspace, in parts: neither thread's parts may land between the other's kernels, and the second
    # sizes need a larger buffer than the first left behind
    cache, _ = make_cache(4096, 64, False, 1)
    table = torch.arange(64, dtype=torch.int32).view(1, 64).cuda()
    lib, stream = _lib.load(), torch.cuda.Stream()
    view, pages = cache.c(), _lib.PageTable(table.data_ptr(), 1, 64)

    def prepare(T, prefix, n):
        ql, qr = (x.cuda() for x in queries(T, 16, T))
        ids, lens = torch.zeros(T, dtype=torch.int32).cuda(), torch.full((T,), n, dtype=torch.int32).cuda()
        want = api.dsa_prefix_attention(ql, qr, cache, table, ids, lens, SM, prefix_len=prefix, max_keys=n)[0]
        assert lib.dsa_prefix_attention_workspace_bytes(T, 16, prefix, n, _lib.DSA_BF16) > 0
        q = _lib.LatentQuery(ql.data_ptr(), ql.stride(0), ql.stride(1), qr.data_ptr(), qr.stride(0), qr.stride(1), T, 16)
        return (ql, qr, ids, lens), q, prefix, n, want

    calls = [prepare(T, prefix, n) for T, prefix, n in ((2, 500, 600), (40, 3000, 4096), (5, 1000, 1500), (64, 3500, 4096))]
    torch.cuda.synchronize()
    bad = []

    def work(order):
        try:
            for _ in range(25):
                outs = {}
                for i in order:
                    (_, _, ids, lens), q, prefix, n, want = calls[i]
                    outs[i] = torch.empty_like(want)
                    _lib.check(lib.dsa_prefix_attention(ctypes.byref(q), ctypes.byref(view), ctypes.byref(pages), ids.data_ptr(),
                                                        lens.data_ptr(), prefix, 0, n, SM, outs[i].data_ptr(), None, None, 0,
                                                        stream.cuda_stream))
                stream.synchronize()
                if any(not torch.equal(outs[i], calls[i][4]) for i in order):
                    bad.append(order)
        except Exception as e:                               # reported by the main thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(o,)) for o in ([0, 1], [2, 3], [3, 0])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    api.dsa_check_device_errors(stream)


@pytest.mark.parametrize("T,H,prefix,own,fp8,d_r", [
    (5, 16, 500, 40, False, 64), (6, 24, 1000, 64, False, 0), (9, 96, 700, 30, False, 64), (64, 16, 4096, 40, False, 64),
    (16, 24, 9000, 100, False, 64), (5, 24, 1000, 64, True, 64), (40, 16, 8000, 30, True, 64), (9, 128, 3000, 10, False, 64),
])
def test_prefix_a_token_does_not_read_may_hold_anything(T, H, prefix, own, fp8, d_r):
    # tokens that end inside the shared prefix, beside others that read on: what lies behind their end must not reach
    # them, though all are rows of the same products (one CTA, pairs, FP8 as it is and expanded, a token's own items)
    page = 64
    full, pages = prefix // page, -(-(prefix + own) // page) + 1
    num_pages = full + T * (pages - full)
    cache, vals = make_cache(num_pages * page, page, fp8, T, d_r)
    table = torch.cat([torch.arange(full).expand(T, full), full + torch.arange(T * (pages - full)).view(T, pages - full)], 1).to(torch.int32)
    n = prefix // 2 - 5
    behind = [n, n + 1, n + 9, n + 64, n + 130, full * page - 1]
    nan, inf = (0x7F, 0xFF) if fp8 else (float("nan"), float("inf"))
    for j, p in enumerate(behind):
        cache.latent[p, (j * 97 + 3) % 512] = nan
        cache.latent[p, 511] = inf
        cache.latent[p + 1, 200 + j] = -inf if not fp8 else nan
    if d_r:
        cache.rope[n:full * page:50] = float("nan")
    lens = torch.full((T,), prefix + own, dtype=torch.int32)
    lens[1], lens[2], lens[3], lens[4] = n, 0, n, n - 100
    ids = torch.arange(T, dtype=torch.int32)
    ql, qr = queries(T, H, 7)
    out, lse = api.dsa_prefix_attention(ql.cuda(), qr.cuda() if d_r else None, cache, table.cuda(), ids.cuda(), lens.cuda(), SM,
                                        prefix_len=full * page, max_keys=prefix + own)
    api.dsa_check_device_errors()
    q = f64(torch.cat([ql, qr], 2) if d_r else ql)
    for t in (1, 2, 3, 4):
        check_token(f64(out)[t], f64(lse)[t], q[t], vals[:int(lens[t])], SM, t)
    reads = [t for t in range(T) if t not in (1, 2, 3, 4)]
    assert torch.isnan(out[reads]).all() and torch.isnan(lse[reads]).all()


FIRST = """
import torch
from sparse_attention_token_02_b200 import api

cache = api.LatentCache.empty(64, 64, fp8={fp8})
cache.rope.normal_()
table = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64)
ids, lens = (torch.full(({T},), n, dtype=torch.int32, device="cuda") for n in (0, 4096))
ql, qr = torch.randn({T}, {H}, 512, device="cuda").bfloat16(), torch.randn({T}, {H}, 64, device="cuda").bfloat16()
idx = torch.arange(2048, dtype=torch.int32, device="cuda").repeat({T}, 1)
x, w = torch.randn(400, 1024, device="cuda"), torch.ones(1024, device="cuda")
torch.cuda.synchronize()


def call():
    return [*api.dsa_prefix_attention(ql, qr, cache, table, ids, lens, 0.1, prefix_len=3000, max_keys=4096),
            *api.dsa_sparse_attention(ql, qr, cache, table, ids, idx, 0.1), *api.dsa_rmsnorm_fp8(x, w)[:2]]


graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, call()))
api.dsa_check_device_errors()
print("equal")
"""


@pytest.mark.parametrize("T,H,fp8", [(1, 128, False), (40, 16, False), (30, 128, True)])
def test_a_process_first_call_may_be_captured(T, H, fp8):
    # nothing has asked for a workspace, a cluster's room or a kernel before the capture begins
    r = subprocess.run([sys.executable, "-c", FIRST.format(T=T, H=H, fp8=fp8)], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-2000:]


def test_an_argument_whose_truth_raises_is_an_error():
    class Undecided:
        def __bool__(self):
            raise ValueError("undecided")

    cache = api.LatentCache.empty(2, 64)
    table, ids = torch.arange(2, dtype=torch.int32).view(1, 2).cuda(), torch.zeros(3, dtype=torch.int32).cuda()
    new = torch.ones(3, 576, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="undecided"):
        api.dsa_latent_append_rope(cache, table, new[:, :512], new[:, 512:], ids, torch.arange(3, dtype=torch.int32).cuda(),
                                   interleaved=Undecided())
    assert not cache.latent.any() and not cache.rope.any()


LAZY = """
import torch
from sparse_attention_token_02_b200 import api

x, w = torch.randn(1 << 15, 8192, dtype=torch.bfloat16, device="cuda"), torch.ones(8192, device="cuda")
want = api.dsa_rmsnorm_fp8(x, w)[0]
lazy = x._lazy_clone()                                       # copied when it is written, or its address asked for
total = torch.cuda.get_device_properties(0).total_memory
torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + x.numel() * 1.25) / total)
got = api.dsa_rmsnorm_fp8(lazy, w)[0]                        # there is room for the results, not for a copy
assert torch._C._is_cow_tensor(lazy) and all(torch.equal(got[i:i + 4096], want[i:i + 4096]) for i in range(0, 1 << 15, 4096))
torch.cuda.set_per_process_memory_fraction(1.0)
lazy = x._lazy_clone()
out = api.dsa_rmsnorm_fp8(x, w, residual=lazy, residual_out=lazy)[2]       # written: its own now
assert out is lazy and not torch._C._is_cow_tensor(lazy) and torch.equal(api.dsa_rmsnorm_fp8(x, w)[0], want)
assert torch.equal(out[:64], (x[:64].float() + x[:64].float()).bfloat16())
print("equal")
"""


def test_what_is_only_read_is_not_copied_first():
    # a copy inside a call could run out of memory there, while other threads run Python
    r = subprocess.run([sys.executable, "-c", LAZY], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "equal" in r.stdout, (r.returncode, r.stdout, r.stderr[-2000:])


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("d", [384, 4112, 16384])
@pytest.mark.parametrize("mag,weight,residual", [(2.0 ** 126, 40.0, True), (2.0 ** 127, 2.0 ** 60, False), (2.0 ** 100, 2.0 ** -60, False),
                                                 (2.0 ** 47, 1.0, True)])
def test_norm_whose_weighted_values_would_overflow(mag, weight, residual, d, group):
    # s * weight is past fp32 where the normed value is not: whole rows of such values, and groups of them beside
    # ordinary and small ones.  Bounds as for every norm, half a step of subnormal numbers with them.
    x = (torch.rand(5, d, generator=gen(7)) / 2 + 0.25) * torch.sign(torch.randn(5, d, generator=gen(8)))
    res = x.flip(0) / 2 if residual else None
    w = weight * (torch.rand(d, generator=gen(9)) + 0.5)
    unit = torch.ones(5, d)
    unit[0] = mag
    unit[1, 128:256] = mag
    unit[2, :128], unit[2, 256:] = mag, 2.0 ** -40
    unit[3, 5] = mag
    x = x * unit
    res = res * unit if residual else None
    normed = torch.empty(5, d, dtype=torch.bfloat16, device="cuda")
    codes, scale, _ = api.dsa_rmsnorm_fp8(x.cuda(), w.cuda(), 1e-6, residual=res.cuda() if residual else None, group=group, normed=normed)
    s, y = L.rmsnorm(f64(x), f64(w), 1e-6, f64(res) if residual else None)
    ref = L.group_scales(y, group)
    # fp32 holds nothing below 2^-149: a group whose y are smaller is one of zeros (at most half of that rounds up)
    zeros = (448 * ref < 2.0 ** -149) & (f64(scale) == 1)
    assert np.all(zeros | (np.abs(f64(scale) - ref) <= 2.0 ** -18 * ref + 2.0 ** -149))
    assert np.all(np.abs(f64(normed) - y) <= (2.0 ** -8 + 2.0 ** -17) * np.abs(y) + 2.0 ** -134)
    wide = np.repeat(f64(scale), group or d, axis=1)[:, :d]
    got = e4m3_decode(codes.cpu().numpy()) * wide
    assert np.all(np.abs(got - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * wide) + 2.0 ** -17 * np.abs(y) + 448 * 2.0 ** -149)


@pytest.mark.parametrize("T,H,prefix,own", [(3, 16, 300, 40), (40, 16, 8000, 30)])
def test_fp8_scales_of_another_writer(T, H, prefix, own):
    # scales that are not powers of two: every value is the bf16 nearest to code times scale, expanded once or on the way
    page, full = 64, prefix // 64
    pages = full + 2
    num_pages = full + 2 * T
    cache, vals = make_cache(num_pages * page, page, True, T)
    scale = torch.rand(num_pages * page, generator=gen(3)) / 100 + 0.002
    cache.scale.copy_(scale)
    latent = e4m3_decode(cache.latent.cpu().numpy()) * f64(scale)[:, None]
    vals[:, :512] = f64(torch.from_numpy(latent).float().bfloat16())
    table = torch.cat([torch.arange(full).expand(T, full), full + torch.arange(2 * T).view(T, 2)], 1).to(torch.int32)
    lens = torch.full((T,), prefix + own, dtype=torch.int32)
    ql, qr = queries(T, H, 7)
    out, lse = api.dsa_prefix_attention(ql.cuda(), qr.cuda(), cache, table.cuda(), torch.arange(T, dtype=torch.int32).cuda(), lens.cuda(),
                                        SM, prefix_len=full * page, max_keys=prefix + own)
    api.dsa_check_device_errors()
    q = f64(torch.cat([ql, qr], 2))
    for t in (0, 1, T - 1):
        rows = [L.page_row(table.numpy(), page, num_pages, t, p) for p in range(prefix + own)]
        check_token(f64(out)[t], f64(lse)[t], q[t], vals[rows], SM, t)
