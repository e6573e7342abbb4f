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
