"""Versions of the header, the binding and the library (no GPU)."""
import os
import re

import pytest

from chunked_prefill_hybrid_tau_gb300 import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_header_binding_and_library_agree(lib):
    with open(os.path.join(ROOT, "include", "hb.h")) as f:
        header = int(re.search(r"#define HB_VERSION (\d+)", f.read()).group(1))
    assert header == L.HB_VERSION == lib.hb_version()


def test_binding_refuses_a_library_of_another_version(lib, monkeypatch):
    """Its structures may have other sizes."""
    monkeypatch.setattr(L, "_lib", None)
    monkeypatch.setattr(L, "HB_VERSION", L.HB_VERSION - 100, raising=False)
    with pytest.raises(RuntimeError, match="version"):
        L.load()
    assert L._lib is None
