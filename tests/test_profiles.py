"""CPU tests that the committed counter summaries describe the kernels that are
built: the benchmark reports a workload's measured memory traffic only while the
hash in its summary is the sources' own."""
import os
import shutil

import pytest

import bench

WORKLOADS = [n for n in bench.CONFIGS if os.path.exists(bench.pmc_summary_path(n))]


@pytest.mark.parametrize("workload", WORKLOADS)
def test_the_benchmark_has_its_traffic(workload):
    traffic, note = bench.read_pmc_traffic(bench.pmc_summary_path(workload))
    assert traffic is not None, note


def test_the_benchmarks_workloads_have_summaries():
    assert {"sq1024", "sq2048", "ragged", "sq8192"} <= set(WORKLOADS)


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the sources that the hash covers."""
    for part in ("include", os.path.join("register_lds_tiled_amd", "csrc")):
        shutil.copytree(os.path.join(bench.ROOT, part), tmp_path / part)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return tmp_path


def test_another_familys_header_changes_no_hash(tree):
    was = {p: bench.source_hash(p) for p in bench.PATH_SOURCES}
    header = tree / "include" / "sgemm.h"
    text = header.read_text()
    more = "#define SGEMM_NEW 99\n/* another family;\n * SGEMM_API int sgemm_f32(void); */\nSGEMM_API int gemm_new_f32(int M,\n    const void *A);\n"
    at = text.index("SGEMM_API int gemm_mxfp4_quantize_f32")
    header.write_text(text[:at] + more + text[at:])
    assert {p: bench.source_hash(p) for p in bench.PATH_SOURCES} == was


@pytest.mark.parametrize("old,new", [("SGEMM_API int sgemm_f32(int M,", "SGEMM_API int sgemm_f32(long M,"),
                                     ("#define SGEMM_PATH_AUTO       0", "#define SGEMM_PATH_AUTO       9")])
def test_its_own_declarations_do(tree, old, new):
    was = bench.source_hash("f32")
    header = tree / "include" / "sgemm.h"
    assert old in header.read_text()
    header.write_text(header.read_text().replace(old, new))
    assert bench.source_hash("f32") != was


@pytest.mark.parametrize("path", list(bench.PATH_SOURCES))
def test_a_paths_sources_do(tree, path):
    was = bench.source_hash(path)
    with open(tree / "register_lds_tiled_amd" / "csrc" / bench.PATH_SOURCES[path][0], "a") as f:
        f.write("// more\n")
    assert bench.source_hash(path) != was
