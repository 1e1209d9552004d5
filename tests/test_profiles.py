"""Summaries under profiles/ say which kernel sources they were taken of."""
import glob
import os
import re

from weight_scans_amd import profiling


def test_every_summary_says_its_sources():
    files = glob.glob(os.path.join(profiling.ROOT, "profiles", "*.md"))
    assert any(os.path.basename(p).startswith("delta_") for p in files)
    for p in files:
        assert re.search(r"^Kernel source hash: `[0-9a-f]{16}`$", open(p).read(), re.M), p


def test_stale_summaries_are_told(monkeypatch, tmp_path):
    """Each family by the hash of its own sources."""
    (tmp_path / "profiles").mkdir()
    scans, delta = profiling.kernel_source_hash(), profiling.delta_source_hash()
    assert scans != delta
    for name, h in (("delta_a.md", delta), ("delta_b.md", scans), ("scan_a.md", scans), ("scan_b.md", delta)):
        (tmp_path / "profiles" / name).write_text(f"# x\n\nKernel source hash: `{h}`\n")
    (tmp_path / "profiles" / "scan_c.md").write_text("# x\n")
    monkeypatch.setattr(profiling, "ROOT", str(tmp_path))
    assert profiling.stale_profiles() == ["delta_b.md", "scan_b.md", "scan_c.md"]
    assert profiling.main(["stale"]) == 1
