"""bench.py's command-line contract, checked on the CPU (no GPU is touched):
more than one GPU is refused with exit status 2 and a message, before torch or the
library is loaded."""
import os
import re
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_more_than_one_gpu_is_refused():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--gpus", "2", "--steps", "3"],
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 2
    assert "one GPU" in r.stderr
    assert r.stdout == ""


def test_help_names_the_default_workload():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--help"], capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0
    assert "dense expert" in r.stdout


def bench():
    import importlib.util
    spec = importlib.util.spec_from_file_location("bench_for_its_sources", os.path.join(ROOT, "bench.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_traffic_hash_covers_every_header_of_the_products():
    """Whatever the products' sources include from csrc/ is hashed too."""
    m = bench()
    csrc = os.path.join(ROOT, "fp8_rowwise_scaled_amd", "csrc")
    for f in m.GEMM_SOURCES:
        for name in re.findall(r'#include "(\w+\.h)"', open(os.path.join(csrc, f)).read()):
            assert name in m.GEMM_SOURCES or not os.path.exists(os.path.join(csrc, name)), f"{f} includes {name}"


def test_the_measured_traffic_is_that_of_the_sources_here():
    """profiles/traffic.json was measured on the kernels as they are: bench.py's JSON has a figure for each workload."""
    m = bench()
    for w in m.WORKLOADS:
        assert m.measured_traffic(w, m.kernel_source_hash()), f"{w}: counters of other sources; measure them again"
