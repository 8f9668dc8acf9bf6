"""The layer's operators without a GPU: what their sources, builds and bindings promise beyond test_layer_cpu.py."""

import ctypes
import glob
import importlib.machinery
import importlib.util
import os
import re
import subprocess

import pytest
import torch

from sparse_attention_token_02_b200 import _lib, api, build


def _sources():
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu*"))):
        with open(path) as f:
            yield os.path.basename(path), f.read()


def test_arrivals_on_a_neighbours_barrier_have_cluster_scope():
    # an arrival's default scope is its own CTA, which orders nothing for the CTA that waits
    arrivals = [(name, op) for name, text in _sources() for op in re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*", text)]
    assert arrivals
    for name, op in arrivals:
        assert ".release.cluster." in op or ".relaxed.cluster." in op, (name, op)
    # a relaxed one orders through the fence in front of it
    for name, text in _sources():
        for at in re.finditer(r"mbarrier\.arrive\.relaxed\.cluster", text):
            assert re.search(r"fence\.release[\w.:]*\.cluster;", text[max(0, at.start() - 120):at.start()]), name


def test_waits_for_a_neighbours_arrivals_acquire_at_cluster_scope():
    # barriers of the pair kernel that the other CTA's threads or products arrive on; the rest are a CTA's own
    text = dict(_sources())["kernels_attention.cu"]
    pair = text[text.index("attention_pair_kernel(AttnArgs a, AttnPlan p) {"):text.index("expand_kernel(LatentView kv")]
    waits = re.findall(r"(mbar_wait\w*)(?:<true>)?\(&sh\.(\w+)", pair)
    own = {"keys", "values", "listed", "moved"}
    assert {bar for _, bar in waits} >= {"scores", "taken", "weights", "queries", "peer_keys", "peer_values", "used", "drained"}
    for call, bar in waits:
        assert call == ("mbar_wait" if bar in own else "mbar_wait_cluster"), (call, bar)


FAKE_DEVICE = """
#include <cuda_runtime.h>
#include "internal.h"
static int device = 0, rooms[2] = {16, 16};
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
namespace dsa {
int cluster_room(int cluster, int, bool* answered) {     // CTAs in clusters of up to rooms[device]; negative: no answer
  if (rooms[device] < 0) *answered = false;
  return rooms[device] >= cluster ? 148 / cluster * cluster : 0;
}
}
extern "C" void set(int d, int room0, int room1) { device = d; rooms[0] = room0; rooms[1] = room1; }
extern "C" int cluster_of(long T, int H, long own) { return dsa::plan_attention(T, H, 0, own, false, 148).cluster; }
"""


@pytest.fixture(scope="module")
def planner(tmp_path_factory):
    """The planner of attention calls on a fake of the device's answers."""
    tmp = tmp_path_factory.mktemp("plan")
    (tmp / "fake.cpp").write_text(FAKE_DEVICE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wl,-Bsymbolic", f"-I{cuda}", f"-I{build.INCLUDE}", f"-I{build.CSRC}", "-x", "c++",
                    os.path.join(build.CSRC, "attention_plan.cu"), str(tmp / "fake.cpp"), "-o", str(tmp / "plan.so")], check=True)
    return ctypes.CDLL(str(tmp / "plan.so"))


def test_a_plan_belongs_to_its_device(planner):
    # two devices with as many SMs, only the first with room for clusters: one query over 2048 keys is cut into
    # a cluster there and through memory on the other, whichever was asked before
    planner.set(0, 16, 0)
    assert planner.cluster_of(1, 128, 2048) > 1
    planner.set(1, 16, 0)
    assert planner.cluster_of(1, 128, 2048) == 1
    planner.set(0, 16, 0)
    assert planner.cluster_of(1, 128, 2048) > 1


def test_a_plan_without_the_devices_answer_is_not_kept(planner):
    planner.set(0, -1, 0)
    assert planner.cluster_of(2, 128, 2048) == 1
    planner.set(0, 16, 0)
    assert planner.cluster_of(2, 128, 2048) > 1


def test_numbers_that_do_not_fit_32_bits_are_refused():
    # ctypes would pass their low 32 bits on: a rotation of 64 values for 2^32 + 64, a bound of 100 keys for 2^32 + 100
    over = 2 ** 32
    cache = api.LatentCache.empty(2, 64, device="cpu")
    ids = torch.zeros(3, dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32)
    q, qr = torch.zeros(3, 4, 512, dtype=torch.bfloat16), torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rope_dim must fit 32 bits"):
        api.dsa_latent_append_rope(cache, table, torch.zeros(3, 512), torch.zeros(3, 64), ids, ids, rope_dim=over + 64)
    for name in ("prefix_len", "prefix_seq", "max_keys"):
        with pytest.raises(ValueError, match=f"{name} must fit 32 bits"):
            api.dsa_prefix_attention(q, qr, cache, table, ids, ids, 0.1, **{name: over + 100})
    wide = torch.zeros(1, 1, dtype=torch.int32).expand(1, 2 ** 26 + 1)          # pages of 64 rows: 2^32 positions and more
    with pytest.raises(ValueError, match="max_keys must fit 32 bits"):
        api.dsa_prefix_attention(q, qr, cache, wide, ids, ids, 0.1)
    with pytest.raises(ValueError, match="max_pages must fit 32 bits"):
        api.dsa_prefix_attention(q, qr, cache, torch.zeros(1, 1, dtype=torch.int32).expand(1, over + 1), ids, ids, 0.1, max_keys=64)
    with pytest.raises(ValueError, match="top_k must fit 32 bits"):
        api.dsa_sparse_attention(q, qr, cache, table, ids, torch.zeros(1, 1, dtype=torch.int32).expand(3, over + 1), 0.1)
    one = torch.zeros(1, 1, 512, dtype=torch.bfloat16).expand(over + 3, 4, 512)
    with pytest.raises(ValueError, match="T must fit 32 bits"):
        api.dsa_sparse_attention(one, one[:, :, :64], cache, table, ids, ids, 0.1)
    long = torch.empty(1, over + 16, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="d must fit 32 bits"):
        api.dsa_rmsnorm_fp8(long, long[0])
    with pytest.raises(ValueError, match="top_k must fit 32 bits"):
        api.dsa_sparse_attention_workspace_bytes(1, 16, over + 64)
    with pytest.raises(ValueError, match="prefix_len must fit 32 bits"):
        api.dsa_prefix_attention_workspace_bytes(1, 16, over, 4096)


@pytest.fixture
def calls_at(tmp_path, monkeypatch):
    """Builds of the compiled calls go to another place."""
    path = str(tmp_path / "_layer_calls.so")
    monkeypatch.setattr(build, "CALLS", path)
    monkeypatch.setattr(build, "CALLS_COMMAND", str(tmp_path / "command"))
    return path


def test_compiled_calls_that_cannot_be_built_are_done_without(calls_at, monkeypatch, capsys):
    with open(calls_at, "w") as f:
        f.write("of an earlier build")
    for command in (["g++", "--no-such-flag"], ["no-such-compiler"], None):
        monkeypatch.setattr(build, "_calls_command", lambda src, command=command: command)
        assert os.path.exists(build.build()) and not os.path.exists(calls_at)
        assert (command is None) == ("Python forms" not in capsys.readouterr().err)


def test_compiled_calls_follow_torchs_version(calls_at, monkeypatch):
    made = []

    def run(command):
        made.append(command)
        with open(calls_at, "w") as f:
            f.write("module")

    for _ in range(2):                                       # the second finds it as it should be
        build._build_calls(run)
    assert len(made) == 1 and any(torch.__version__ in part for part in made[0])
    place, version = build._torch()
    monkeypatch.setattr(build, "_torch", lambda: (place, "0.0"))
    build._build_calls(run)
    assert len(made) == 2


def test_a_torch_that_names_no_version_is_no_torch_to_build_for(calls_at, tmp_path, monkeypatch):
    spec = importlib.machinery.ModuleSpec("torch", None, is_package=True)
    spec.submodule_search_locations.append(str(tmp_path))
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: spec)
    assert build._torch() is None and build._calls_command("layer_calls.cpp") is None


def test_compiled_calls_for_another_torch_are_declined(monkeypatch):
    assert build.CALLS.endswith(importlib.machinery.EXTENSION_SUFFIXES[0])
    monkeypatch.setattr(torch, "__version__", "0.0")
    assert api._compiled_calls() is None


def test_a_softmax_scale_that_overflows_in_base_2_is_refused():
    # scores are held times log2(e): 2^127.5 times it is past fp32, and 0 times infinity a NaN
    lib = _lib.load()
    cache = _lib.LatentCacheView(0x100000, None, 0x200000, 8, 64, 512, 64, _lib.DSA_BF16)
    table, q = _lib.PageTable(0x300000, 2, 4), _lib.LatentQuery(0x400000, 65536, 512, 0x500000, 8192, 64, 4, 128)
    P = ctypes.c_void_p
    for scale in (2.0 ** 127.5, 3.4e38):
        got = [lib.dsa_sparse_attention(ctypes.byref(q), ctypes.byref(cache), ctypes.byref(table), P(0x600000), P(0x700000), 16, scale,
                                        P(0x800000), None, None, 0, None),
               lib.dsa_prefix_attention(ctypes.byref(q), ctypes.byref(cache), ctypes.byref(table), P(0x600000), P(0x700000), 4, 0, 16,
                                        scale, P(0x800000), None, None, 0, None)]
        assert [_lib.STATUS_NAMES[s] for s in got] == ["DSA_ERR_INVALID_ARG"] * 2
        assert b"sm_scale" in lib.dsa_get_last_error()


def test_pointers_that_are_not_aligned_to_their_values_are_refused():
    # a device fault otherwise; torch's tensors are always aligned, other callers' buffers may not be
    lib, P = _lib.load(), ctypes.c_void_p
    bad = []

    def norm(scale=0x60000):
        return lib.dsa_rmsnorm_fp8(P(0x10000), _lib.DSA_BF16, 256, None, None, P(0x40000), _lib.DSA_BF16, 4, 256, 1e-6, 128, P(0x50000),
                                   P(scale), None, None)

    def append(scale=0x900000, pages=0x300000, kr=0x700000, seq=0x600000, pos=0x800000, dtype=_lib.DSA_F32):
        cache = _lib.LatentCacheView(0x100000, scale, 0x200000, 8, 64, 512, 64, _lib.DSA_FP8_E4M3)
        return lib.dsa_latent_append_rope(ctypes.byref(cache), ctypes.byref(_lib.PageTable(pages, 2, 4)), P(0xA00000), 512, P(kr), 64, dtype,
                                          P(seq), P(pos), 4, ctypes.byref(_lib.Rope(64, 1, 10000.0)), None)

    def attention(prefix, seq=0x600000, keys=0x700000, lse=0x900000):
        cache, table = _lib.LatentCacheView(0x100000, None, 0x200000, 8, 64, 512, 64, _lib.DSA_BF16), _lib.PageTable(0x300000, 2, 4)
        q = _lib.LatentQuery(0x400000, 65536, 512, 0x500000, 8192, 64, 4, 128)
        args = [ctypes.byref(q), ctypes.byref(cache), ctypes.byref(table), P(seq), P(keys)]
        args += [4, 0, 16] if prefix else [16]
        return (lib.dsa_prefix_attention if prefix else lib.dsa_sparse_attention)(*args, 0.1, P(0x800000), P(lse), None, 0, None)

    for call, name, at in ((norm, "scale", 0x60002), (append, "scale", 0x900002), (append, "pages", 0x300002), (append, "kr", 0x700002),
                           (append, "seq", 0x600001), (append, "pos", 0x800002)):
        bad.append((name, call(**{name: at}), lib.dsa_get_last_error()))
    for prefix in (False, True):
        for name, at in (("seq", 0x600002), ("keys", 0x700001), ("lse", 0x900002)):
            bad.append((name, attention(prefix, **{name: at}), lib.dsa_get_last_error()))
    assert append(kr=0x700001, dtype=_lib.DSA_BF16) == 1
    assert all(status == 1 and b"aligned" in message for _, status, message in bad), bad     # DSA_ERR_INVALID_ARG
