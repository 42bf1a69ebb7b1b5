"""The DRAM bytes that bench.py reports beside its roofline are those of the kernel that it runs: they were captured from
the sources as they are (an entry of other sources is left out of the report)."""
import importlib.util
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_dominant_kernels_traffic_is_of_these_sources():
    spec = importlib.util.spec_from_file_location("bench_of_traffic", os.path.join(ROOT, "bench.py"))
    bench = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bench)
    with open(os.path.join(ROOT, "profiles", "dram_traffic.txt")) as f:
        entries = [line.split() for line in f if line.strip() and not line.startswith("#")]
    assert [e[0] for e in entries] == ["gemm_dw1_mxfp8"]
    for name, size, sha in entries:
        assert int(size) > 0 and sha == bench.source_sha(name), name
