"""The layer's operators without a GPU: what their sources, builds and bindings promise beyond test_layer_cpu.py."""

import glob
import os
import re

from sparse_attention_token_02_b200 import build


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
