"""The hash that ties the stored counter measurements to the sources they were taken of (no GPU)."""

import os
import shutil

import pytest

from norm_rope_cache_amd import build


@pytest.mark.parametrize("name,changes", [("api.cpp", True), ("kv_project.hip", True), ("device_common.h", True),
                                          ("status.h", True), ("tree_attention.hip", False), ("cache_api.cpp", False)])
def test_the_hash_follows_the_chain(tmp_path, monkeypatch, name, changes):
    """A change to the chain's kernels, or to the entry points that choose among them, is another hash; a comment is none."""
    before = build.source_hash()
    copy = tmp_path / "csrc"
    shutil.copytree(build.CSRC, copy)
    monkeypatch.setattr(build, "CSRC", str(copy))
    with open(os.path.join(copy, name), "a") as f:
        f.write("// a comment\n")
    assert build.source_hash() == before
    with open(os.path.join(copy, name), "a") as f:
        f.write("static int changed;\n")
    assert (build.source_hash() != before) == changes
