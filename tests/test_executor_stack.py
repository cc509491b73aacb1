"""What an executor's launch costs beyond its work."""
import os
import re

from tests.gpu_harness import ensure_built


def test_stacks_fit_what_a_context_keeps_for_each_thread():
    """1,024 bytes unless set otherwise. A kernel that needs more has the device's local memory made larger at its launch,
    which waits until nothing runs."""
    ensure_built()
    from persistent_micro_dispatch_gb300 import build
    report = open(os.path.join(build.BUILD, "gpuos_device.ptxas.txt")).read()
    stacks = [int(n) for n in re.findall(r"(\d+) bytes cumulative stack size", report)]
    assert len(stacks) > 4 and max(stacks) <= 1024
