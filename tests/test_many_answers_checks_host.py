"""More refusals of the calls for many answers: the cache's own state, tables whose numbers leave their range."""
import ctypes

import pytest

from test_decode_host import A, MB, cache, lib  # noqa: F401
from test_many_answers_host import attention
from ulysses_qkv_proj_gb300 import binding as qb


@pytest.mark.parametrize("name", ["out", "lse", "ws"])
@pytest.mark.parametrize("state", [dict(page_refs=0), dict(scratch=0), dict(scratch=-16 * 4 - 12)])
def test_outputs_keep_off_page_counts_and_scratch(lib, name, state):
    """No output may lie over page_refs or scratch (the last case: over its last word alone)."""
    at = dict(out=A + 220 * MB, lse=A + 230 * MB, ws=A + 240 * MB)[name]
    assert attention(lib, c=cache(**{k: at + x for k, x in state.items()})) == 4


@pytest.mark.parametrize("state", [dict(page_refs=0), dict(scratch=0), dict(scratch=-16 * 4 - 12)])
def test_common_lengths_keep_off_page_counts_and_scratch(lib, state):
    c = cache(**{k: A + 202 * MB + x for k, x in state.items()})
    assert lib.qnre_cache_shared_prefix(ctypes.byref(c), A + 200 * MB, 4, A + 201 * MB, 2, A + 202 * MB, None) == 4


@pytest.mark.parametrize("kw", [
    dict(kind=1, factor=1e-310), dict(kind=3, factor=1e-310, original=100.0), dict(kind=4, factor=1e-310, original=10.0),
    dict(magnitude=1e39), dict(magnitude=-3.5e38), dict(kind=2, factor=1e-310, theta=1.5),
])
def test_tables_out_of_range(lib, kw):
    """Frequencies or a magnitude that no float holds."""
    f = dict(kind=0, factor=2.0, original=4096.0, low=1.0, high=32.0, magnitude=1.0, theta=1e4)
    f.update(kw)
    s = qb._RopeScaling(*[f[k] for k in ("kind", "factor", "original", "low", "high", "magnitude")])
    assert lib.qnre_rope_table(A, 8, 64, 0, f["theta"], ctypes.byref(s), None) == 1
