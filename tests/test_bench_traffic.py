"""When bench.py reports a stored traffic figure: while the sources of the
kernels that it times are the ones it was measured on."""
import json
import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402

CSRC = os.path.join("gemm_w4a16_group_gb300", "csrc")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(ROOT, CSRC), tmp_path / CSRC)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    monkeypatch.setattr(bench, "TRAFFIC_FILE", str(tmp_path / "traffic.json"))
    (tmp_path / "traffic.json").write_text(json.dumps({"source_hash": bench.kernel_source_hash(), "bytes_per_launch": {"a": 7}}))
    return tmp_path / CSRC


def change(path):
    path.write_text(path.read_text() + "\n// changed\n")


def test_figures_count_while_the_sources_stand(tree):
    assert bench.stored_traffic("a") == 7 and bench.stored_traffic("b") is None


@pytest.mark.parametrize("name", ["kv_pages.cu", "tree_attn.cu", "tree_attn.cuh", "tree_attn_tc.cu"])
def test_the_cache_operators_are_no_part_of_them(tree, name):
    change(tree / name)
    assert bench.stored_traffic("a") == 7


@pytest.mark.parametrize("name", ["decode.cu", "decode_tc.cu", "prompt.cu", "repack.cu", "api.cu", "w4a16_common.cuh", "w4a16_internal.h"])
def test_a_changed_product_makes_them_stale(tree, name):
    change(tree / name)
    assert bench.stored_traffic("a") is None


def test_a_new_source_makes_them_stale(tree):
    (tree / "another.cu").write_text("// new\n")
    assert bench.stored_traffic("a") is None
