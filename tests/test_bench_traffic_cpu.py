"""CPU tests of what keys the bench's recorded HBM traffic: the code of the GEMM's
own units and the flags that they are built with, not what else the library holds."""
import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

BUILD = "communication_tensor_gemm_amd/build.py"


@pytest.fixture
def source_copy(tmp_path, monkeypatch):
    for f in bench.KERNEL_SOURCES:
        (tmp_path / f).parent.mkdir(parents=True, exist_ok=True)
        shutil.copy(os.path.join(ROOT, f), tmp_path / f)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return tmp_path


def change(path, old, new):
    text = path.read_text()
    assert old in text
    path.write_text(text.replace(old, new))


@pytest.mark.parametrize("workload", ["c2_blog_overlap_f32", "c3_ag_rot_a_bf16_tp8", "c4_rs_tile_a_rot_c_bf16_tp8", "c5_ag_rot_b_e4m3_tp8"])
def test_the_record_is_of_these_sources(workload):
    assert bench.recorded_traffic(workload) > 1e9


def test_where_the_tree_lies_does_not_count(source_copy):
    here = bench.kernel_source_hash()
    bench.ROOT = ROOT
    assert bench.kernel_source_hash() == here


def test_other_units_do_not_count(source_copy):
    h0 = bench.kernel_source_hash()
    change(source_copy / BUILD, '"distgemm.hip",', '"distgemm.hip", "another.hip",')
    change(source_copy / BUILD, 'EXTRA = {', 'EXTRA = {\n    "another.hip": ["-O1"],')
    assert bench.kernel_source_hash() == h0


@pytest.mark.parametrize("old,new", [('"-O3"', '"-O2"'), ('"gfx950"', '"gfx942"'),
                                     ('"gemm_mfma16.hip": ["-mllvm", "-pragma-unroll-threshold=1000000"]', '"gemm_mfma16.hip": []')])
def test_their_flags_count(source_copy, old, new):
    h0 = bench.kernel_source_hash()
    change(source_copy / BUILD, old, new)
    assert bench.kernel_source_hash() != h0
