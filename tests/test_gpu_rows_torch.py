"""What the operators for many requests on one base model (runtime.Adapters, runtime.logprobs, PagedKV.decode_shared) owe
torch: version counters of what they write, refused gradients and tangents, inference mode, memory kept for other streams,
streams that are being captured, no errors left behind by launches that fail."""
import ctypes as C
import gc

import pytest
import torch
from torch.autograd import forward_ad

from test_gpu_paged import ints

pytestmark = pytest.mark.gpu


class Small:
    """One call of each, on inputs of its own."""

    def __init__(self):
        from gqa_transformer_decode_gb300 import runtime
        g = torch.Generator(device="cuda").manual_seed(3)

        def rand(*s):
            return torch.randn(*s, generator=g, device="cuda").bfloat16()
        self.x, self.w, self.a, self.b = rand(12, 256), rand(192, 256), rand(3, 16, 256), rand(3, 192, 16)
        self.ids = torch.tensor([0, 1, 2, -1] * 3, dtype=torch.int32, device="cuda")
        self.ad = runtime.Adapters(self.a, self.b)
        self.k, self.v = rand(16, 2, 16, 64), rand(16, 2, 16, 64)
        self.table = torch.arange(16, dtype=torch.int32, device="cuda").view(4, 4)
        self.cache = runtime.PagedKV(self.k, self.v, self.table)
        self.q = rand(3, 8, 64)
        self.shared = [ints([33, 40, 64]), ints([0, 3]), ints([32]), ints([0])]
        self.seqs = ints([1, 2, 3])
        self.logits = torch.randn(5, 1000, generator=g, device="cuda")
        self.given = torch.arange(5, dtype=torch.int32, device="cuda")
        self.lib = runtime

    def project(self, x=None, **k):
        return self.ad.project(self.x if x is None else x, self.w, self.ids, **k)

    def decode(self, q=None, **k):
        return self.cache.decode_shared(self.q if q is None else q, *self.shared, seqs=self.seqs, **k)

    def logprobs(self, x=None, **k):
        return self.lib.logprobs(self.logits if x is None else x, self.given, top=3, **k)

    def calls(self):
        """Each operator as a function of its floating input, that input, and what of its answer to look at."""
        return [(self.project, self.x, lambda y: [y]), (self.decode, self.q, lambda y: [y]), (self.logprobs, self.logits, list)]


def test_writes_raise_the_version_counters():
    s = Small()
    out, att, lse = (torch.zeros(12, 400, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 8, 64, dtype=torch.bfloat16, device="cuda"),
                     torch.zeros(3, 8, device="cuda"))
    read = [s.x, s.w, s.a, s.b, s.ids, s.k, s.v, s.table, s.q, s.seqs, s.logits, s.given, *s.shared]
    was = [t._version for t in read + [out, att, lse]]
    s.project(out=out[:, 8:200])                         # a view counts with its base
    s.decode(out=att, lse=lse)
    s.logprobs()
    assert [t._version for t in read] == was[:-3]
    assert [t._version for t in (out, att, lse)] == [v + 1 for v in was[-3:]]


def test_gradients_and_tangents_are_refused():
    s = Small()
    for call, x, _ in s.calls():
        with pytest.raises(ValueError, match="gradient"):
            call(x.clone().requires_grad_())
        with forward_ad.dual_level():
            with pytest.raises(ValueError, match="tangent"):
                call(forward_ad.make_dual(x, torch.ones_like(x)))
        with torch.no_grad():
            call(x.clone().requires_grad_())
    s.w.requires_grad_()
    with pytest.raises(ValueError, match="w requires a gradient"):
        s.project()
    s.w.requires_grad_(False)
    s.b.requires_grad_()
    with pytest.raises(ValueError, match="b requires a gradient"):
        s.project()


def test_inference_mode():
    s = Small()
    want = [look(call()) for call, _, look in s.calls()]
    with torch.inference_mode():
        t = Small()
        got = [look(call()) for call, _, look in t.calls()]
        out = torch.empty(12, 192, dtype=torch.bfloat16, device="cuda")
        t.project(out=out)
    got2 = [look(call()) for call, _, look in t.calls()]  # outside the mode as well
    for a, b, c in zip(want, got, got2):
        assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))
    assert torch.equal(out, want[0][0])
    t.ids = torch.full_like(s.ids, 7)
    t.project()
    assert t.ad.sync_status() == 1 and t.ad.sync_status() == 0


def busy(stream):
    """Work on the stream that outlasts the host's next calls."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(200_000_000)                   # a tenth of a second


@pytest.mark.parametrize("op", range(3))
def test_inputs_freed_after_a_call_on_another_stream_are_kept_for_it(op):
    s = Small()
    call, data, look = s.calls()[op]
    other = torch.cuda.Stream()
    want = [t.clone() for t in look(call())]
    x = data.clone()
    at = x.data_ptr()
    torch.cuda.synchronize()
    busy(other)
    got = call(x, stream=other)
    del x
    reused = [torch.zeros_like(data) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(t.data_ptr() != at for t in reused)
    assert all(torch.equal(a, b) for a, b in zip(want, look(got)))


@pytest.mark.parametrize("op", range(3))
def test_a_stream_that_is_being_captured_can_be_passed(op):
    s = Small()
    call, data, look = s.calls()[op]
    want = [t.clone() for t in look(call())]
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        x = data.clone()                                 # of the graph's own memory, gone before its replay
        got = call(x, stream=side)
        del x
    for t in look(got):
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, look(got)))


def test_two_graphs_with_memory_of_their_own_run_at_once():
    s = Small()
    want = [[t.clone() for t in look(call())] for call, _, look in s.calls()]
    torch.cuda.synchronize()
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], []
    for side in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got = [[look(call()) for call, _, look in s.calls()] for _ in range(6)]
        graphs.append((g, got))
    torch.cuda.synchronize()
    for _ in range(20):
        for side, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(side):
                g.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        for one in got:
            assert all(torch.equal(a, b) for w, y in zip(want, one) for a, b in zip(w, y))


def test_the_status_word_outlives_its_adapters_while_a_stream_may_raise_an_error():
    s = Small()
    at = s.ad.status.data_ptr()
    bad = torch.full_like(s.ids, 99)
    x, w, a, b = s.x, s.w, s.a, s.b
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    busy(other)
    with torch.cuda.stream(other):
        s.ad.project(x, w, bad)
    s.ad = None
    gc.collect()
    words = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    assert all(int(t) == 0 and t.data_ptr() != at for t in words) and a.is_cuda and b.is_cuda


def test_a_launch_that_fails_leaves_no_error_behind():
    """Launches into a capture that a synchronize has invalidated are refused by the runtime; the next caller's check of
    the last error does not see it."""
    from gqa_transformer_decode_gb300 import ember as E
    with open("/proc/self/maps") as f:
        rt = C.CDLL(next(line.split()[-1] for line in f if "libcudart" in line))
    s = Small()
    want = [[t.clone() for t in look(call())] for call, _, look in s.calls()]
    p = lambda t: C.c_void_p(t.data_ptr())  # noqa: E731
    ad = E.ember_adapters(a=s.a.data_ptr(), b=s.b.data_ptr(), scale=None, n_adapters=3, rank=16)
    kv = E.ember_paged_kv(k=s.k.data_ptr(), v=s.v.data_ptr(), table=s.table.data_ptr(), dtype=E.BF16, n_pages=16, page_size=16,
                          n_kv_heads=2, head_dim=64, n_seqs=4, table_width=4, page_stride=2 * 16 * 64, head_stride=16 * 64,
                          row_stride=64)
    out, att, H = torch.empty_like(s.x), torch.empty_like(s.q), torch.empty(5, device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    stream, graph = C.c_void_p(), C.c_void_p()
    assert rt.cudaStreamCreate(C.byref(stream)) == 0
    calls = [
        lambda: E.ember_adapter_project(C.byref(ad), p(s.x), 256, p(s.w), None, E.BF16, 12, 192, 256, p(s.ids), p(out), E.BF16,
                                        192, p(ws), 1 << 22, None, stream),
        lambda: E.ember_logprobs(p(s.logits), E.F32, 5, 1000, 1000, 1.0, None, 0, None, None, p(H), None, None, stream),
        lambda: E.ember_paged_decode_shared(C.byref(kv), p(s.q), 512, 3, 8, p(s.seqs), p(s.shared[0]), p(s.shared[1]),
                                            p(s.shared[2]), p(s.shared[3]), 1, 0.125, p(att), 512, None, p(ws), 1 << 22, None,
                                            stream)]
    for call in calls:
        assert rt.cudaStreamBeginCapture(stream, 2) == 0             # relaxed: only this stream's
        assert rt.cudaStreamSynchronize(stream) != 0                 # not while it is captured: invalidates it
        rt.cudaGetLastError()
        assert call() == 6 and "launch failed" in E.last_error()
        left = rt.cudaPeekAtLastError()
        assert rt.cudaStreamEndCapture(stream, C.byref(graph)) != 0
        rt.cudaGetLastError()
        assert left == 0
    assert rt.cudaStreamDestroy(stream) == 0
    torch.cuda.synchronize()
    for (call, _, look), w in zip(s.calls(), want):                  # all as before
        assert all(torch.equal(a, b) for a, b in zip(w, look(call())))
