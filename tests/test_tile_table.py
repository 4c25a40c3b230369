"""The committed tile table: one entry a shape and format, swept for the shapes that the benchmark's
workloads name. Any other shape takes the compiled-in rule, or a sweep of the user's own; the table is
not the place to tune single calls."""
import json
import os

import bench
from block_scaled_w8a8_amd import build


def _entries():
    with open(os.path.join(build.TABLE_PATH)) as f:
        return json.load(f)["entries"]


def test_dense_entries_are_the_workloads_shapes():
    known = {s for w in bench.WORKLOADS.values() if w.get("kind") != "moe" for s in w["shapes"]}
    assert {(e["N"], e["K"]) for e in _entries() if "E" not in e} == known


def test_entries_are_distinct():
    keys = [(e["N"], e["K"], e["dtype"], e.get("E"), tuple(e.get("block_shape", (128, 128))),
             e.get("w_layout"), e.get("scales")) for e in _entries()]
    assert len(keys) == len(set(keys))
