"""The digest under which bench.py reports DRAM traffic covers every source of
the executor's image, what those include among them (CPU)."""
import re
import shutil

import pytest

import bench


@pytest.fixture
def copy(tmp_path, monkeypatch):
    for f in bench.TRAFFIC_SOURCES + bench.TRAFFIC_INCLUDES:
        (tmp_path / f).parent.mkdir(parents=True, exist_ok=True)
        shutil.copy(f"{bench.ROOT}/{f}", tmp_path / f)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return tmp_path


@pytest.mark.parametrize("f", bench.TRAFFIC_SOURCES + bench.TRAFFIC_INCLUDES)
def test_digest_follows_each_file(copy, f):
    before = bench.sources_digest()
    with open(copy / f, "a") as fh:
        fh.write("\n")
    assert bench.sources_digest() != before
    assert all(bench.launch_traffic(w, 100) is None for w in bench.TRAFFIC)


def test_no_own_include_is_left_out():
    """Every file of csrc that a device source includes is in the digest."""
    known = {f.rsplit("/", 1)[1] for f in bench.TRAFFIC_SOURCES + bench.TRAFFIC_INCLUDES}
    for f in bench.TRAFFIC_SOURCES + bench.TRAFFIC_INCLUDES:
        for inc in re.findall(r'#include "([^"]+)"', open(f"{bench.ROOT}/{f}").read()):
            assert inc in known or inc == "gpuos.h", (f, inc)
