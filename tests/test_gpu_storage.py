"""Objects that keep tensors (runtime.Adapters, runtime.PagedKV) read them where they lie at each call: a tensor that was given
other storage (t.data = .., as a module that is moved or loaded does) is read there, not in the old storage, which may be
somebody else's by then; one that has another type, shape or device is refused."""
import gc

import pytest
import torch

from test_gpu_adapters import Case
from test_gpu_paged import ints

pytestmark = pytest.mark.gpu


def filled(*like):
    """Tensors in what the allocator has free now, not finite."""
    return [torch.full_like(t, float("nan")) for t in like for _ in range(4)]


def test_adapters_in_other_storage():
    c, d = Case(40, 256, 512, 16, 4), Case(40, 256, 512, 16, 4, seed=9)
    want = d.ad.project(c.x, c.w, c.ids)
    first = c.run()
    assert not torch.equal(first, want)
    for mine, other in ((c.a, d.a), (c.b, d.b), (c.scale, d.scale)):
        mine.data = other.clone()
    gc.collect()
    junk = filled(c.a, c.b, c.scale)
    assert torch.equal(c.run(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = c.run(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and len(junk) == 12


@pytest.mark.parametrize("name,new", [("a", lambda t: t.half()), ("a", lambda t: t[:3].clone()), ("b", lambda t: t[:, :128].clone()),
                                      ("b", lambda t: t.cpu()), ("b", lambda t: t.transpose(1, 2)), ("scale", lambda t: t.double()),
                                      ("scale", lambda t: t[:2].clone())])
def test_adapters_that_became_others(name, new):
    c = Case(40, 256, 512, 16, 4)
    c.run()
    t = getattr(c, name)
    was = t.data
    t.data = new(t)
    with pytest.raises(ValueError, match=f"{name} must be"):
        c.run()
    t.data = was
    c.check(c.run())


def test_adapters_are_not_replaced_behind_the_objects_back():
    c = Case(8, 128, 64, 8, 2)
    for name in ("a", "b", "scale"):
        assert getattr(c.ad, name) is getattr(c, name)
        with pytest.raises(AttributeError):
            setattr(c.ad, name, None)
    c.check(c.run())


class Paged:
    """A cache of four sequences, and calls of each operator on it."""

    def __init__(self, seed, row_major=False):
        from gqa_transformer_decode_gb300 import runtime
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.k, self.v = ((r(16, 16, 2, 64).transpose(1, 2) if row_major else r(16, 2, 16, 64)) for _ in range(2))
        self.table = torch.arange(16, dtype=torch.int32, device="cuda").view(4, 4).flip(seed % 2).contiguous()
        self.cache = runtime.PagedKV(self.k, self.v, self.table)

    def calls(self, q):
        c = self.cache
        cos = torch.ones(64, 32, device="cuda")
        c.append(q[:, :2], q[:, 2:4], ints([0, 1, 2, 3]), ints([5, 6, 7, 8]), cos, torch.zeros_like(cos))
        return [c.decode(q, ints([64, 33, 20, 9])), c.prefill(q, ints([0, 2, 4]), ints([50, 64])),
                c.decode_shared(q, ints([64, 33, 40, 50]), ints([0, 4]), ints([32]), ints([0]))]


@pytest.mark.parametrize("row_major", [False, True])
def test_a_cache_in_other_storage(row_major):
    p, o = Paged(0, row_major), Paged(1, row_major)
    q = torch.randn(4, 8, 64, device="cuda").bfloat16()
    want = o.calls(q)
    assert not torch.equal(p.calls(q)[0], want[0])
    old = Paged(1, row_major)                    # as o was before its append
    for name in ("k", "v", "table"):
        src = getattr(old, name)
        new = torch.empty_like(src)              # of the same strides
        new.copy_(src)
        getattr(p, name).data = new
    gc.collect()
    junk = filled(p.k, p.v) + [torch.full_like(p.table, -5) for _ in range(4)]
    got = p.calls(q)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(junk) == 12
    assert p.cache.sync_status() == 0 and torch.equal(p.k, o.k) and torch.equal(p.v, o.v)


@pytest.mark.parametrize("name,new,says", [
    ("k", lambda t: t.half(), "k_pages must keep"), ("v", lambda t: t[:8].clone(), "v_pages must keep"),
    ("v", lambda t: t.transpose(1, 2).contiguous().transpose(1, 2), "v_pages must keep"), ("k", lambda t: t.cpu(), "k_pages must be on cuda"),
    ("table", lambda t: t.long(), "table must be"), ("table", lambda t: t[:2].clone(), "table must be")])
def test_a_cache_that_became_another(name, new, says):
    p = Paged(0)
    q = torch.randn(4, 8, 64, device="cuda").bfloat16()
    want = p.calls(q)
    t = getattr(p, name)
    was = t.data
    t.data = new(t)
    for call in (lambda: p.calls(q), lambda: p.cache.decode(q, ints([64, 33, 20, 9])),
                 lambda: p.cache.prefill(q, ints([0, 2, 4]), ints([50, 64]))):
        with pytest.raises(ValueError, match=says):
            call()
    t.data = was
    assert all(torch.equal(a, b) for a, b in zip(p.calls(q), want))


def test_page_dimensions_of_one_have_any_stride():
    from gqa_transformer_decode_gb300 import runtime
    k = torch.randn(4, 1, 16, 64, device="cuda").bfloat16()
    v = torch.as_strided(k.clone(), k.shape, (16 * 64, 8, 64, 1))
    cache = runtime.PagedKV(k, v, torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4))
    q = torch.randn(1, 4, 64, device="cuda").bfloat16()
    assert cache.decode(q, ints([50])).isfinite().all()
