"""Kernels that start beside the launch before theirs (programmatic serialization) read no memory by the read-only path: it
may only serve what nobody writes while the kernel runs, and the wait for the earlier launch does not order it."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parent.parent / "ulysses_qkv_proj_gb300" / "csrc"
OVERLAPPED = sorted(p.name for p in CSRC.glob("*.cu") if "cudaLaunchAttributeProgrammaticStreamSerialization" in p.read_text())


def _with_headers(name, seen):
    if name in seen or not (CSRC / name).exists():
        return seen
    seen[name] = (CSRC / name).read_text()
    for header in re.findall(r'#include "([\w./]+)"', seen[name]):
        _with_headers(header, seen)
    return seen


def test_there_are_such_kernels():
    assert {"rope_table.cu", "sample.cu", "verify_tree.cu", "qk_norm_rope.cu", "tree_attention.cu"} <= set(OVERLAPPED)


@pytest.mark.parametrize("name", OVERLAPPED)
def test_no_read_only_loads(name):
    for file, text in _with_headers(name, {}).items():
        assert not re.search(r"\b__ldg\s*\(|ld\.global(\.\w+)*\.nc", text), file
        assert "griddepcontrol.wait" in text or file != name
