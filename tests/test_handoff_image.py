"""What a hand-off links anew each time, the relocatable build of the
executor, holds the executor's kernel and its ops, and nothing besides."""
import os
import re

from tests.gpu_harness import ensure_built


def test_relocatable_image_holds_one_kernel_and_no_line_tables():
    ensure_built()
    from persistent_micro_dispatch_gb300 import build
    report = open(os.path.join(build.BUILD, "gpuos_exec_rdc.ptxas.txt")).read()
    assert set(re.findall(r"Compiling entry function '(\w+)'", report)) == {"gpuos_executor_kernel"}
    assert "-lineinfo" not in report.splitlines()[0].split()
    with open(build.EXEC_RDC, "rb") as f:
        image = f.read()
    assert image[:4] == b"\x7fELF" and b"debug_line" not in image


def test_library_itself_keeps_its_line_tables():
    ensure_built()
    from persistent_micro_dispatch_gb300 import build
    report = open(os.path.join(build.BUILD, "gpuos_device.ptxas.txt")).read()
    assert "-lineinfo" in report.splitlines()[0].split()
    assert {"gpuos_executor_kernel", "gpuos_eager_kernel"} <= set(re.findall(r"Compiling entry function '(\w+)'", report))
