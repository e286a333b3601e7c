"""tests/kernel_meta.py reads the library and leaves it as it was: a process may have it mapped."""

import os
import shutil

import pytest

from tests import kernel_meta as KM

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "latency_collectives_amd", "libar.so")


def test_reading_the_code_objects_does_not_write_the_library(tmp_path):
    if not os.path.exists(LIB) or not KM.tools_available():
        pytest.skip("the library is not built, or ROCm's LLVM tools are not there")
    lib = tmp_path / "lib.so"
    shutil.copy(LIB, lib)
    os.utime(lib, ns=(10 ** 18, 10 ** 18))
    before, held = os.stat(lib), open(lib, "rb")
    work = tmp_path / "work"
    work.mkdir()
    assert KM.code_objects(str(lib), str(work))
    after = os.stat(lib)
    assert (after.st_ino, after.st_mtime_ns, after.st_size) == (before.st_ino, before.st_mtime_ns, before.st_size)
    with held, open(LIB, "rb") as f:
        assert held.read() == f.read()
