"""CPU-only: every helper calls the library that was loaded."""
import os
import shutil

import pytest

from quant_dequant_gemv_amd import binding as b

pytestmark = pytest.mark.skipif(not os.path.exists(b.LIB_PATH),
                                reason="libqkgemv.so not built (run __graft_entry__.build())")


def test_packed_calls_are_the_loaded_librarys(monkeypatch, tmp_path):
    path = str(tmp_path / "libother.so")
    shutil.copy(b.LIB_PATH, path)
    monkeypatch.setattr(b, "_lib", None)
    b._packed_calls.cache_clear()
    try:
        assert b.load_library(path)._name == path
        assert b._packed_calls()._name == path
    finally:
        b._packed_calls.cache_clear()
