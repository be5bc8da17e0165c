"""The build entry point fails where any compiled part does not load (CPU)."""
import pytest

import __graft_entry__ as entry
import bitwise_deterministic_exact_amd.build as lib_build
import oracle.build as oracle_build
from bitwise_deterministic_exact_amd import _lib


@pytest.mark.parametrize("part", ["load", "ops"])
def test_build_loads_every_library(part, monkeypatch):
    monkeypatch.setattr(lib_build, "build", lambda: None)
    monkeypatch.setattr(oracle_build, "build", lambda: None)
    entry.build()

    def broken():
        raise ImportError(f"{part} does not load")
    monkeypatch.setattr(_lib, part, broken)
    with pytest.raises(ImportError, match="does not load"):
        entry.build()
