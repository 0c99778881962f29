"""The benchmark's DRAM traffic figure holds while the sources of the kernels it
was counted on are unchanged, and only theirs."""
import importlib.util
import os
import shutil

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def bench(tmp_path, monkeypatch):
    """bench.py over a copy of the kernel sources."""
    spec = importlib.util.spec_from_file_location("bench_copy", os.path.join(ROOT, "bench.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    csrc = tmp_path / "gqa_kv_head_gb300" / "csrc"
    shutil.copytree(os.path.join(ROOT, "gqa_kv_head_gb300", "csrc"), csrc)
    monkeypatch.setattr(m, "ROOT", str(tmp_path))
    return m, csrc


def test_the_paged_kernels_do_not_void_the_figure(bench):
    m, csrc = bench
    before = m.kernel_source_hash()
    for name in ("fr_paged.cu", "fr_paged_tc.cu", "fr_paged_attn.cuh", "fr_paged_append.cu"):
        with open(csrc / name, "a") as f:
            f.write("static int added;\n")
    (csrc / "fr_paged_more.cuh").write_text("static int more;\n")
    assert m.kernel_source_hash() == before


@pytest.mark.parametrize("name", ["fr_attn_tc.cu", "fr_attn_sw.cu", "fr_decode_attn.cu", "fr_qkv_post.cu", "fr_sm100.cuh",
                                  "fr_common.cuh", "fr_split_merge.cuh"])
def test_the_counted_kernels_do(bench, name):
    m, csrc = bench
    before = m.kernel_source_hash()
    src = (csrc / name).read_text()
    (csrc / name).write_text(src + "// a comment\n")
    assert m.kernel_source_hash() == before
    (csrc / name).write_text(src + "static int added;\n")
    assert m.kernel_source_hash() != before
