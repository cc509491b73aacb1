"""What a process's first call costs beyond its work."""
import os

from tests.gpu_harness import ensure_built


def test_device_code_is_not_compressed():
    """Unpacking it took 17 ms of a process's first call."""
    ensure_built()
    from persistent_micro_dispatch_gb300 import build
    report = open(os.path.join(build.BUILD, "gpuos_device.ptxas.txt")).read()
    assert "--no-compress" in report.splitlines()[0].split()
