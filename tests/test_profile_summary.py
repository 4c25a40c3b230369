"""The source hash on the profile summaries covers the kernels that they describe."""
import glob
import os

from block_scaled_w8a8_amd import profile_summary as ps

# host code, and the matrix-core probe, which no summary describes
NOT_KERNELS = {"api_common.h", "tile_table.h", "probe.hip"}


def test_every_kernel_source_is_hashed():
    csrc = os.path.join(ps.HERE, "csrc")
    found = {os.path.basename(p) for pat in ("*.hip", "*.h") for p in glob.glob(os.path.join(csrc, pat))}
    assert {os.path.basename(p) for p in ps.FEED_FORWARD_SOURCES} == found - NOT_KERNELS


def test_the_stamp_changes_with_any_of_them(tmp_path, monkeypatch):
    for rel in ps.FEED_FORWARD_SOURCES:
        os.makedirs(tmp_path / os.path.dirname(rel), exist_ok=True)
        (tmp_path / rel).write_text(rel)
    monkeypatch.setattr(ps, "HERE", str(tmp_path))
    seen = {ps.source_hash(ps.FEED_FORWARD_SOURCES)}
    for rel in ps.FEED_FORWARD_SOURCES:
        (tmp_path / rel).write_text("changed")
        seen.add(ps.source_hash(ps.FEED_FORWARD_SOURCES))
    assert len(seen) == 1 + len(ps.FEED_FORWARD_SOURCES)


def test_stats_stamp(tmp_path, capsys):
    csv = tmp_path / "run_kernel_stats.csv"
    csv.write_text("Name,Calls,AverageNs,MinNs,MaxNs,TotalDurationNs,Percentage\nk,1,1000,1000,1000,1000,100\n")
    import sys
    for flags, sources in (([], ps.KERNEL_SOURCES), (["--feed-forward"], ps.FEED_FORWARD_SOURCES)):
        argv, sys.argv = sys.argv, ["profile_summary", "stats", str(csv), *flags]
        try:
            ps.main()
        finally:
            sys.argv = argv
        assert f"# kernel sources: {ps.source_hash(sources)}\n" in capsys.readouterr().out
