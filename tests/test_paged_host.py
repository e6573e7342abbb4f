"""Refusals of the paged-cache entry points: every call here is answered before
any device work, so the pointers are never followed (no GPU needed)."""
import ctypes as C

import pytest

from gqa_transformer_decode_gb300 import ember as E

INVALID, CAPACITY, UNSUPPORTED = 1, 2, 8
A = 1 << 20          # stands for an aligned buffer; never dereferenced


def cache(**over):
    c = E.ember_paged_kv()
    d = dict(k=A, v=A, table=A, dtype=E.BF16, n_pages=8, page_size=16, n_kv_heads=2, head_dim=64, n_seqs=4,
             table_width=4, page_stride=2 * 16 * 64, head_stride=16 * 64, row_stride=64)
    d.update(over)
    for k, v in d.items():
        setattr(c, k, v)
    return c


def append(c=None, **over):
    d = dict(q=A, k=A, v=A, src=E.F32, ld_q=256, ld_k=128, ld_v=128, n=3, heads=4, seqs=A, positions=A, qn=None,
             kn=None, eps=1e-6, cos=A, sin=A, n_pos=64, q_out=A, ld_out=256)
    d.update(over)
    return E.ember_paged_append(C.byref(c or cache()), d["q"], d["k"], d["v"], d["src"], d["ld_q"], d["ld_k"],
                                d["ld_v"], d["n"], d["heads"], d["seqs"], d["positions"], d["qn"], d["kn"],
                                d["eps"], d["cos"], d["sin"], d["n_pos"], d["q_out"], d["ld_out"], None, None)


def prefill(c=None, **over):
    d = dict(q=A, ld_q=256, n=5, B=2, heads=4, seqs=None, cu=A, lens=A, window=0, sinks=0, scale=0.1, out=A,
             ld_out=256, lse=None)
    d.update(over)
    return E.ember_paged_prefill(C.byref(c or cache()), d["q"], d["ld_q"], d["n"], d["B"], d["heads"], d["seqs"],
                                 d["cu"], d["lens"], d["window"], d["sinks"], d["scale"], d["out"], d["ld_out"],
                                 d["lse"], None, None)


def decode(c=None, **over):
    d = dict(q=A, ld_q=256, B=2, heads=4, seqs=None, lens=A, window=0, sinks=0, scale=0.1, out=A, ld_out=256,
             lse=None, ws=A, ws_bytes=1 << 40)
    d.update(over)
    return E.ember_paged_decode(C.byref(c or cache()), d["q"], d["ld_q"], d["B"], d["heads"], d["seqs"], d["lens"],
                                d["window"], d["sinks"], d["scale"], d["out"], d["ld_out"], d["lse"], d["ws"],
                                d["ws_bytes"], None, None)


CACHE = [
    (dict(k=None), INVALID, "NULL pages"), (dict(table=None), INVALID, "NULL pages"),
    (dict(dtype=E.F32), INVALID, "dtype"), (dict(dtype=7), INVALID, "dtype"),
    (dict(n_pages=0), INVALID, "> 0"), (dict(n_seqs=-1), INVALID, "> 0"), (dict(table_width=0), INVALID, "> 0"),
    (dict(head_dim=48), UNSUPPORTED, "head_dim"), (dict(head_dim=256), UNSUPPORTED, "head_dim"),
    (dict(page_size=24), UNSUPPORTED, "page_size"), (dict(page_size=8), UNSUPPORTED, "page_size"),
    (dict(page_size=2048), UNSUPPORTED, "page_size"),
    (dict(table_width=1 << 30), UNSUPPORTED, "2^30"),
    (dict(k=A + 8), INVALID, "aligned"), (dict(table=A + 2), INVALID, "aligned"),
    (dict(row_stride=60), INVALID, "strides"), (dict(row_stride=68), INVALID, "strides"),
    (dict(page_stride=-64), INVALID, "strides"), (dict(head_stride=0), INVALID, "strides"),
]


@pytest.mark.parametrize("call", [append, decode, prefill])
@pytest.mark.parametrize("over,status,msg", CACHE)
def test_bad_caches_are_refused_by_every_operator(call, over, status, msg):
    assert call(cache(**over)) == status and msg in E.last_error(), E.last_error()


@pytest.mark.parametrize("over,status,msg", [
    (dict(n=-1), INVALID, "tokens"), (dict(src=3), INVALID, "src_dtype"), (dict(eps=-1.0), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"), (dict(n_pos=0), INVALID, "n_pos"),
    (dict(seqs=None), INVALID, "seqs"), (dict(positions=None), INVALID, "positions"),
    (dict(cos=None), INVALID, "cos_t"), (dict(sin=A + 4), INVALID, "cos_t"), (dict(qn=A + 2), INVALID, "q_norm"),
    (dict(k=None), INVALID, "k is NULL"), (dict(v=A + 4), INVALID, "v must be"), (dict(ld_k=120), INVALID, "of k"),
    (dict(ld_v=132), INVALID, "of v"), (dict(q_out=None), INVALID, "go together"),
    (dict(q=None), INVALID, "go together"), (dict(heads=3), INVALID, "multiple of n_kv_heads"),
    (dict(heads=34, ld_q=34 * 64, ld_out=34 * 64), UNSUPPORTED, "GQA"), (dict(ld_out=128), INVALID, "q_out"),
])
def test_append_refuses(over, status, msg):
    assert append(**over) == status and msg in E.last_error(), E.last_error()


ATTENTION = [
    (dict(heads=0), INVALID, "multiple of n_kv_heads"), (dict(heads=5), INVALID, "multiple of n_kv_heads"),
    (dict(heads=34, ld_q=34 * 64, ld_out=34 * 64), UNSUPPORTED, "GQA"),
    (dict(window=-1), INVALID, "window"), (dict(sinks=-2), INVALID, "window and sinks"),
    (dict(scale=float("inf")), INVALID, "scale"), (dict(scale=float("nan")), INVALID, "scale"),
    (dict(q=None), INVALID, "q is NULL"), (dict(out=None), INVALID, "out is NULL"), (dict(lens=None), INVALID, "lens"),
    (dict(q=A + 8), INVALID, "aligned"), (dict(ld_q=250), INVALID, "of q"), (dict(ld_out=248), INVALID, "of out"),
]


@pytest.mark.parametrize("call", [decode, prefill])
@pytest.mark.parametrize("over,status,msg", ATTENTION)
def test_attentions_refuse(call, over, status, msg):
    assert call(**over) == status and msg in E.last_error(), E.last_error()


def test_batches_beyond_the_table_are_refused():
    assert decode(B=5) == INVALID and "n_seqs" in E.last_error()
    assert prefill(B=5) == INVALID and "n_seqs" in E.last_error()
    assert decode(B=-1) == INVALID and decode(B=70000, seqs=A) == UNSUPPORTED
    assert prefill(n=70000, B=70000, seqs=A) == UNSUPPORTED
    assert prefill(n=-1) == INVALID and prefill(B=-1) == INVALID and prefill(cu=None) == INVALID


def test_calls_without_rows_do_nothing():
    assert append(n=0, seqs=None, positions=None) == 0
    assert decode(B=0, q=None, out=None, lens=None, ws=None) == 0
    assert prefill(n=0, q=None, out=None) == 0 and prefill(B=0, q=None, cu=None, lens=None) == 0


def test_the_workspace_query_answers_zero_for_bad_arguments():
    f = E.ember_paged_decode_workspace
    assert f(None, 1, 4) == 0 and f(C.byref(cache()), 0, 4) == 0 and f(C.byref(cache()), 2, 3) == 0


def torch_side():
    """The compiled marshalling over a cache that is never reached."""
    from gqa_transformer_decode_gb300 import runtime
    t = runtime._paged_torch()
    return t, t.cache(C.addressof(cache()), A, 0)


def test_the_torch_side_refuses_before_any_device_work():
    import torch
    t, c = torch_side()
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    lens = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError, match="arguments"):
        t.decode(c, q)
    with pytest.raises(TypeError, match="q must be a tensor"):
        t.decode(c, 3, lens, None, 0, 0, None, None, None, False, None)
    with pytest.raises(ValueError, match="q must be on cuda:0, not cpu"):
        t.decode(c, q, lens, None, 0, 0, None, None, None, False, None)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        t.append(c, lens, lens, lens, lens, q, q, None, None, None, 1e-6, None)
    with pytest.raises(ValueError, match="k must be on cuda"):
        t.append(c, q, q, lens, lens, q, q, None, None, None, 1e-6, None)
    with pytest.raises(TypeError, match="lens must be a tensor"):
        t.prefill(c, q, lens, None, None, 0, 0, None, None, None, False)
    with pytest.raises(ValueError):
        t.decode("no cache", q, lens, None, 0, 0, None, None, None, False, None)


def test_the_torch_side_refuses_to_lose_a_gradient():
    import torch
    t, c = torch_side()
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, requires_grad=True)
    x = q.detach()
    lens = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="q requires a gradient"):
        t.decode(c, q, lens, None, 0, 0, None, None, None, False, None)
    with pytest.raises(ValueError, match="q requires a gradient"):
        t.prefill(c, q * 2, lens, lens, None, 0, 0, None, None, None, False)
    with pytest.raises(ValueError, match="v requires a gradient"):
        t.append(c, x, q, lens, lens, x, x, None, None, None, 1e-6, None)
    with torch.no_grad(), pytest.raises(ValueError, match="q must be on cuda:0, not cpu"):
        t.decode(c, q, lens, None, 0, 0, None, None, None, False, None)


def test_the_torch_side_refuses_pages_whose_gradient_would_be_lost():
    import torch
    from gqa_transformer_decode_gb300 import runtime
    t = runtime._paged_torch()
    k, v = (torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16) for _ in range(2))
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    x = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="v_pages requires a gradient"):
        t.cache(C.addressof(cache()), A, 0, k, v.clone().requires_grad_())
    c = t.cache(C.addressof(cache()), A, 0, k, v)
    calls = [lambda: t.decode(c, q, x, None, 0, 0, None, None, None, False, None),
             lambda: t.prefill(c, q, x, x, None, 0, 0, None, None, None, False),
             lambda: t.append(c, q, q, x, x, q, q, None, None, None, 1e-6, None)]
    for call in calls:
        with pytest.raises(ValueError, match="must be on cuda:0, not cpu"):
            call()
    k.requires_grad_()                       # asked for after the cache was made
    for call in calls:
        with pytest.raises(ValueError, match="k_pages requires a gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="must be on cuda:0, not cpu"):
            call()


def test_the_torch_side_refuses_to_lose_a_forward_mode_tangent():
    import torch
    import torch.autograd.forward_ad as fw
    from gqa_transformer_decode_gb300 import runtime
    t = runtime._paged_torch()
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    x = torch.zeros(1, dtype=torch.int32)
    pages = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    _, c = torch_side()
    with fw.dual_level():
        d = fw.make_dual(q, torch.ones_like(q))
        with pytest.raises(ValueError, match="q has a forward-mode tangent"):
            t.decode(c, d, x, None, 0, 0, None, None, None, False, None)
        with pytest.raises(ValueError, match="q has a forward-mode tangent"):
            t.prefill(c, d * 2, x, x, None, 0, 0, None, None, None, False)
        with pytest.raises(ValueError, match="v has a forward-mode tangent"):
            t.append(c, q, d, x, x, q, q, None, None, None, 1e-6, None)
        with pytest.raises(ValueError, match="k_pages has a forward-mode tangent"):
            t.cache(C.addressof(cache()), A, 0, fw.make_dual(pages, pages + 1), pages)
    with pytest.raises(ValueError, match="q must be on cuda:0, not cpu"):      # outside there is none
        t.decode(c, q, x, None, 0, 0, None, None, None, False, None)

    def through(x):                                                            # torch.func's own tensors
        return t.decode(c, x, torch.zeros(1, dtype=torch.int32), None, 0, 0, None, None, None, False, None)
    with pytest.raises((ValueError, RuntimeError)):
        torch.func.jvp(through, (q,), (torch.ones_like(q),))
    with pytest.raises((ValueError, RuntimeError)):
        torch.func.vmap(through)(q[None])


def test_the_status_word_is_taken_from_valid_pointers_only():
    f = E.ember_paged_take_status
    for a, b, msg in ((None, A, "NULL"), (A, None, "NULL"), (A + 2, A, "4-byte"), (A, A + 1, "4-byte")):
        assert f(a, b, None) == INVALID and msg in E.last_error()


def test_index_arrays_that_are_not_aligned_are_refused():
    """They would be read by loads, and the status word by atomics, of 4 bytes."""
    kv = C.byref(cache())
    for over in (dict(seqs=A + 2), dict(positions=A + 1)):
        assert append(**over) == INVALID and "4-byte" in E.last_error()
    for over in (dict(seqs=A + 2), dict(lens=A + 3), dict(lse=A + 2)):
        assert decode(**over) == INVALID and "4-byte" in E.last_error()
    for over in (dict(seqs=A + 1), dict(cu=A + 2), dict(lens=A + 2), dict(lse=A + 1)):
        assert prefill(**over) == INVALID and "4-byte" in E.last_error()
    bad = A + 2                              # the status word
    assert E.ember_paged_append(kv, None, A, A, E.F32, 0, 128, 128, 3, 0, A, A, None, None, 1e-6, A, A, 64, None, 0,
                                bad, None) == INVALID and "4-byte" in E.last_error()
    assert E.ember_paged_decode(kv, A, 256, 2, 4, None, A, 0, 0, 0.1, A, 256, None, A, 1 << 40, bad, None) == INVALID
    assert "4-byte" in E.last_error()
    assert E.ember_paged_prefill(kv, A, 256, 5, 2, 4, None, A, A, 0, 0, 0.1, A, 256, None, bad, None) == INVALID
    assert "4-byte" in E.last_error()


def test_rows_too_long_for_32_bit_offsets_are_refused():
    """Without q nothing else bounds the kv heads of a row: 2^25 heads of 64 pass 2^31 elements."""
    for nkv in (1 << 25, (1 << 31) - 1, (1 << 14) + 1):
        c = cache(n_kv_heads=nkv)
        assert append(c, q=None, q_out=None, ld_k=64 * nkv, ld_v=64 * nkv) == UNSUPPORTED and "2^20" in E.last_error()
    for call in (decode, prefill):
        assert call(heads=1 << 15, ld_q=1 << 21, ld_out=1 << 21, c=cache(n_kv_heads=1 << 15)) == UNSUPPORTED
    c = cache(n_kv_heads=1024, head_dim=16, n_seqs=70000, table_width=1 << 20)
    assert decode(c, B=2048, heads=1024, ld_q=1 << 14, ld_out=1 << 14) == UNSUPPORTED and "2^34" in E.last_error()
