"""What each library is rebuilt for (no GPU, nothing compiled beyond the first build)."""
import os
import re

import pytest

from depthwise_causal_short_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()


def _included(path, seen):
    """The repository's files that `path` includes, and so on."""
    if path in seen:
        return seen
    seen.add(path)
    for name in re.findall(r'^\s*#include\s+"([^"]+)"', path.read_text(), re.M):
        found = (path.parent / name).resolve()
        assert found.exists(), f"{path}: {name}"
        _included(found, seen)
    return seen


@pytest.mark.parametrize("lib,sources", [
    (_build.LIB, _build.sources()), (_build.ATTN_LIB, _build.attn_sources()),
    (_build.ATTN_PY, [_build.attn_binding()]),
], ids=["libcconv", "libcattn", "_cattn"])
def test_every_included_file_is_an_input(lib, sources):
    inputs = {p.resolve() for p in _build._inputs(lib)}
    for src in sources:
        assert _included(src.resolve(), set()) <= inputs


def test_a_newer_header_makes_its_library_stale():
    assert _build.up_to_date()
    header = _build.CSRC / "attn" / "attn_chunk_host.h"
    old = header.stat()
    try:
        later = _build.ATTN_LIB.stat().st_mtime + 10
        os.utime(header, (later, later))
        assert not _build._newer(_build.ATTN_LIB) and _build._newer(_build.LIB)
    finally:
        os.utime(header, ns=(old.st_atime_ns, old.st_mtime_ns))
    assert _build.up_to_date()


def test_the_binding_is_stale_for_another_torch(monkeypatch):
    import torch
    assert _build._newer(_build.ATTN_PY)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert not _build._newer(_build.ATTN_PY) and _build._newer(_build.ATTN_LIB)
