"""Refusals of ember_paged_decode_shared, answered before any device work (no GPU needed)."""
import ctypes as C

import pytest

from gqa_transformer_decode_gb300 import ember as E
from test_paged_host import A, ATTENTION, CACHE, INVALID, UNSUPPORTED, cache


def shared(c=None, **over):
    d = dict(q=A, ld_q=256, B=2, heads=4, seqs=None, lens=A, groups=A, shared=A, prefixes=A, n_groups=1, scale=0.1, out=A,
             ld_out=256, lse=None, ws=A, ws_bytes=1 << 40, status=None)
    d.update(over)
    return E.ember_paged_decode_shared(C.byref(c or cache()), d["q"], d["ld_q"], d["B"], d["heads"], d["seqs"], d["lens"],
                                       d["groups"], d["shared"], d["prefixes"], d["n_groups"], d["scale"], d["out"], d["ld_out"],
                                       d["lse"], d["ws"], d["ws_bytes"], d["status"], None)


@pytest.mark.parametrize("over,status,msg", CACHE)
def test_bad_caches(over, status, msg):
    assert shared(cache(**over)) == status and msg in E.last_error(), E.last_error()


@pytest.mark.parametrize("over,status,msg", [x for x in ATTENTION if not {"window", "sinks"} & set(x[0])] + [
    (dict(n_groups=0), INVALID, "n_groups"), (dict(n_groups=3), INVALID, "n_groups"), (dict(groups=None), INVALID, "groups"),
    (dict(shared=None), INVALID, "groups"), (dict(prefixes=None), INVALID, "groups"), (dict(groups=A + 2), INVALID, "4-byte"),
    (dict(shared=A + 1), INVALID, "4-byte"), (dict(prefixes=A + 3), INVALID, "4-byte"), (dict(status=A + 2), INVALID, "4-byte"),
    (dict(lse=A + 2), INVALID, "4-byte"), (dict(B=5), INVALID, "n_seqs"), (dict(B=70000, seqs=A), UNSUPPORTED, "65535"),
])
def test_bad_arguments(over, status, msg):
    assert shared(**over) == status and msg in E.last_error(), E.last_error()


def test_no_rows_and_bad_queries():
    assert shared(B=0, q=None, out=None, lens=None, groups=None, ws=None) == 0
    f = E.ember_paged_decode_shared_workspace
    assert f(None, 1, 4, 1) == 0 and f(C.byref(cache()), 2, 4, 0) == 0 and f(C.byref(cache()), 2, 4, 3) == 0
