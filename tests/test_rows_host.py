"""Refusals of the operators on rows: every call here is answered before any device work, so the pointers are
never followed (no GPU needed)."""
import pytest

from gqa_transformer_decode_gb300 import ember as E

INVALID, CAPACITY, UNSUPPORTED = 1, 2, 8
A = 1 << 20          # stands for an aligned buffer; never dereferenced


def logprobs(**over):
    d = dict(logits=A, dtype=E.F32, n=3, V=100, ldl=100, t=1.0, ids=A, top=5, logprob=A, rank=A, entropy=A, top_ids=A,
             top_logprobs=A)
    d.update(over)
    return E.ember_logprobs(d["logits"], d["dtype"], d["n"], d["V"], d["ldl"], d["t"], d["ids"], d["top"], d["logprob"],
                            d["rank"], d["entropy"], d["top_ids"], d["top_logprobs"], None)


@pytest.mark.parametrize("over,status,msg", [
    (dict(dtype=3), INVALID, "dtype"), (dict(n=-1), INVALID, "rows"), (dict(V=0), INVALID, "V must"),
    (dict(V=(1 << 30) + 1, ldl=1 << 31), INVALID, "V must"), (dict(ldl=99), INVALID, "ldl"),
    (dict(t=0.0), INVALID, "temperature"), (dict(t=-1.0), INVALID, "temperature"),
    (dict(t=float("nan")), INVALID, "temperature"), (dict(t=float("inf")), INVALID, "temperature"),
    (dict(t=9e-7), INVALID, "temperature"), (dict(t=1.1e6), INVALID, "temperature"), (dict(top=-1), INVALID, "top"), (dict(top=101), INVALID, "top"),
    (dict(top=33), UNSUPPORTED, "top > 32"), (dict(top_ids=None), INVALID, "top_ids"),
    (dict(top_logprobs=None), INVALID, "top_ids"), (dict(ids=None), INVALID, "need ids"),
    (dict(logits=None), INVALID, "logits is NULL"), (dict(logits=A + 2), INVALID, "aligned"),
    (dict(dtype=E.BF16, logits=A + 1), INVALID, "aligned"), (dict(rank=A + 2), INVALID, "4-byte"),
])
def test_logprobs_refuses(over, status, msg):
    assert logprobs(**over) == status and msg in E.last_error(), E.last_error()


def test_nothing_to_do_is_fine():
    assert logprobs(n=0, logits=None) == 0


def test_the_limit_is_the_headers():
    import os
    import re
    with open(os.path.join(os.path.dirname(__file__), "..", "include", "ember.h")) as f:
        assert int(re.search(r"EMBER_LOGPROBS_MAX_TOP (\d+)", f.read()).group(1)) == E.LOGPROBS_MAX_TOP
