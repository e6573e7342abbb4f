"""Refusals of the operators on rows: every call here is answered before any device work, so the pointers are
never followed (no GPU needed)."""
import ctypes as C

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


def project(**over):
    d = dict(a=A, b=A, scale=A, n_adapters=3, rank=8, x=A, ld_x=64, w=A, bias=None, dtype=E.BF16, n=3, N=128, K=64, ids=A, out=A,
             out_dtype=E.F32, ld_out=128, ws=A, ws_bytes=1 << 30, status=None)
    d.update(over)
    ad = E.ember_adapters(a=d["a"], b=d["b"], scale=d["scale"], n_adapters=d["n_adapters"], rank=d["rank"])
    return E.ember_adapter_project(C.byref(ad), d["x"], d["ld_x"], d["w"], d["bias"], d["dtype"], d["n"], d["N"], d["K"], d["ids"],
                                   d["out"], d["out_dtype"], d["ld_out"], d["ws"], d["ws_bytes"], d["status"], None)


@pytest.mark.parametrize("over,status,msg", [
    (dict(dtype=E.F32), INVALID, "dtype"), (dict(out_dtype=E.F16), INVALID, "out_dtype"), (dict(n=-1), INVALID, "rows"),
    (dict(N=0), INVALID, "multiples of 8"), (dict(N=132), INVALID, "multiples of 8"), (dict(K=60), INVALID, "multiples of 8"),
    (dict(n_adapters=0), INVALID, "n_adapters"), (dict(rank=0), INVALID, "rank"), (dict(rank=12), INVALID, "rank"),
    (dict(rank=136), UNSUPPORTED, "rank"), (dict(a=None), INVALID, "a and b"), (dict(b=A + 8), INVALID, "a and b"),
    (dict(w=None), INVALID, "w must"), (dict(bias=A + 2), INVALID, "bias"), (dict(ids=None), INVALID, "ids is NULL"),
    (dict(ids=A + 2), INVALID, "4-byte"), (dict(scale=A + 2), INVALID, "4-byte"), (dict(status=A + 1), INVALID, "4-byte"),
    (dict(x=None), INVALID, "x is NULL"), (dict(x=A + 8), INVALID, "x must be"), (dict(ld_x=56), INVALID, "of x"),
    (dict(ld_x=68), INVALID, "of x"), (dict(out=None), INVALID, "out is NULL"), (dict(ld_out=120), INVALID, "of out"),
    (dict(ws=None), INVALID, "workspace"), (dict(ws=A + 8), INVALID, "workspace"), (dict(ws_bytes=3 * 2 * 16 * 2 - 1), CAPACITY, "workspace"),
])
def test_project_refuses(over, status, msg):
    assert project(**over) == status and msg in E.last_error(), E.last_error()


def test_the_adapters_workspace():
    assert E.ember_adapter_workspace(3, 8) == 3 * 2 * 16 * 2 and E.ember_adapter_workspace(100, 128) == 100 * 2 * 128 * 2
    assert [E.ember_adapter_workspace(*x) for x in ((0, 8), (-1, 8), (3, 0), (3, 12), (3, 136))] == [0] * 5


def test_nothing_to_do_is_fine():
    assert logprobs(n=0, logits=None) == 0 and project(n=0, x=None, ws=None) == 0


def test_the_limit_is_the_headers():
    import os
    import re
    with open(os.path.join(os.path.dirname(__file__), "..", "include", "ember.h")) as f:
        assert int(re.search(r"EMBER_LOGPROBS_MAX_TOP (\d+)", f.read()).group(1)) == E.LOGPROBS_MAX_TOP


def test_the_torch_side_refuses_tensors_of_the_host():
    import torch
    from gqa_transformer_decode_gb300 import runtime
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        runtime.logprobs(x, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="logits"):
        runtime.logprobs([1.0])
    a, b = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="a must be a tensor on a CUDA device"):
        runtime.Adapters(a, b)
