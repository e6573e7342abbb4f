"""The tensors that runtime.logprobs returns are each their own: on storage of their type and size, so that keeping, saving or
growing one has nothing to do with the others."""
import io

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,top,given", [(1, 5, True), (37, 20, True), (37, 0, True), (2000, 32, True), (37, 3, False), (0, 4, True)])
def test_each_output_has_storage_of_its_own(n, top, given):
    from gqa_transformer_decode_gb300 import runtime
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, 1000, generator=g, device="cuda")
    ids = torch.randint(1000, (n,), generator=g, device="cuda").to(torch.int32) if given else None
    r = runtime.logprobs(x, ids, top=top)
    some = [t for t in r if t is not None]
    assert len(some) == (5 if given else 3) and [t.dtype for t in some[-3:]] == [torch.float32, torch.int32, torch.float32]
    for t in some:
        assert t.is_contiguous() and t.storage_offset() == 0 and not t._is_view()
        assert t.untyped_storage().nbytes() == t.numel() * 4
        f = io.BytesIO()
        torch.save(t, f)
        assert f.tell() <= 4 * t.numel() + 4096
    at = [t.untyped_storage().data_ptr() for t in some if t.numel()]
    assert len(set(at)) == len(at)
    if n == 0:
        return
    want = [t.clone() for t in some]
    some[0].resize_(4 * n + 64).fill_(9)         # growing one leaves the others as they are
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(some[1:], want[1:]))
