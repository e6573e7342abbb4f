"""What runtime.PagedKV owes torch: version counters of what it writes, gradients refused, streams and
the status word."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Small:
    """One sequence of up to 64 keys on four pages; 2 kv heads, 4 query heads of 64."""

    def __init__(self):
        from gqa_transformer_decode_gb300 import runtime
        self.k, self.v = (torch.randn(6, 2, 16, 64, device="cuda").bfloat16() for _ in range(2))
        self.table = ints(3, 1, 0, 5)[None].contiguous()
        self.cache = runtime.PagedKV(self.k, self.v, self.table)
        self.cos, self.sin = torch.ones(64, 32, device="cuda"), torch.zeros(64, 32, device="cuda")
        self.q = torch.randn(3, 4, 64, device="cuda").bfloat16()
        self.x = torch.randn(3, 2, 64, device="cuda").bfloat16()

    def append(self, **kw):
        return self.cache.append(self.x, self.x, ints(0, 0, 0), ints(40, 41, 42), self.cos, self.sin, **kw)


def test_writes_raise_the_version_counters():
    s = Small()
    versions = lambda *ts: [t._version for t in ts]  # noqa: E731
    before = versions(s.k, s.v, s.q, s.x, s.table)
    s.append()
    assert versions(s.k, s.v, s.q, s.x, s.table) == [before[0] + 1, before[1] + 1, *before[2:]]
    buf, lse = torch.zeros(3, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 4, device="cuda")
    at = versions(buf, lse)
    s.append(q=s.q, q_out=buf[:, 2:6])                   # a view counts with its base
    s.cache.prefill(s.q, ints(0, 3), ints(43), out=buf[:, :4], lse=lse)
    s.cache.decode(s.q[:1], ints(43), out=buf[:1, 4:], lse=lse[:1])
    assert versions(buf, lse) == [at[0] + 3, at[1] + 2]
    at = versions(s.k, buf)
    s.cache.prefill(s.q[:0], ints(0), ints(), out=buf[:0, :4])   # nothing to do, nothing written
    assert versions(s.k, buf) == at


def test_autograd_notices_that_a_saved_tensor_was_overwritten():
    s = Small()
    w = torch.ones_like(s.k).requires_grad_()
    y = (w * s.k).sum()                                  # saves the pages for w's gradient
    s.append()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_inference_tensors_are_written_too():
    with torch.inference_mode():
        s = Small()
        out = torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda")
        s.append(q=s.q, q_out=out)
    assert torch.equal(out, s.q)
    s.cache.prefill(s.q, ints(0, 3), ints(43), out=out)  # outside the mode as well
    assert torch.equal(out, s.cache.prefill(s.q, ints(0, 3), ints(43)))


def test_pages_that_require_a_gradient_are_refused():
    from gqa_transformer_decode_gb300 import runtime
    s = Small()
    with pytest.raises(ValueError, match="k_pages requires a gradient"):
        runtime.PagedKV(s.k.clone().requires_grad_(), s.v, s.table)
    want = s.cache.decode(s.q[:1], ints(43))
    s.v.requires_grad_()
    with pytest.raises(ValueError, match="v_pages requires a gradient"):
        s.cache.decode(s.q[:1], ints(43))
    with torch.no_grad():
        assert torch.equal(want, s.cache.decode(s.q[:1], ints(43)))


def test_an_error_raised_while_the_status_is_read_is_kept():
    s = Small()
    word = s.cache.status
    raised = []

    class Raised:
        """The status word; as soon as the host has read it, a call on another stream raises 2 (a length beyond
        the table's)."""

        def data_ptr(self):
            return word.data_ptr()

        def item(self):
            got = word.item()
            s.cache.decode(s.q[:1], ints(65))
            raised.append(2)
            torch.cuda.synchronize()
            return got

        def zero_(self):
            word.zero_()

    s.cache.decode(s.q[:1], ints(43), seqs=ints(9))      # raises 1
    s.cache.status = Raised()
    got = [s.cache.sync_status()]
    if not raised:                                       # (where the word is taken on the device)
        s.cache.decode(s.q[:1], ints(65))
    s.cache.status = word
    got.append(s.cache.sync_status())
    assert got == [1, 2] and s.cache.sync_status() == 0


def test_no_error_is_lost_between_streams():
    """One stream raises an error again and again while another takes the word: whatever it takes is 0 or that
    error, and the last one is still there at the end."""
    s = Small()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    bad, n = ints(65), ints(43)
    with torch.cuda.stream(other):
        for _ in range(300):
            s.cache.decode(s.q[:1], bad)
    got = [s.cache.sync_status() for _ in range(30)]
    assert set(got) <= {0, 2}
    other.synchronize()
    with torch.cuda.stream(other):
        s.cache.decode(s.q[:1], bad)
    assert s.cache.sync_status(other) == 2 and s.cache.sync_status() == 0
    s.cache.decode(s.q[:1], n)
    assert s.cache.sync_status() == 0


def test_the_status_of_a_cache_made_in_inference_mode():
    with torch.inference_mode():
        s = Small()
    s.cache.decode(s.q[:1], ints(65))
    assert s.cache.sync_status() == 2 and s.cache.sync_status() == 0


def busy(stream):
    """Work on the stream that outlasts the host's next calls."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(200_000_000)                   # a tenth of a second


@pytest.mark.parametrize("op", ["decode", "prefill", "append"])
def test_inputs_freed_after_a_call_on_another_stream_are_kept_for_it(op):
    s = Small()
    other = torch.cuda.Stream()
    side = lambda *a, **k: getattr(s.cache, op)(*a, stream=other, **k)  # noqa: E731
    n = {"decode": 1}.get(op, 3)
    lens, cu, seqs, pos = ints(43), ints(0, 3), ints(0, 0, 0), ints(40, 41, 42)
    call = {"decode": lambda q: side(q, lens), "prefill": lambda q: side(q, cu, lens),
            "append": lambda q: side(s.x, s.x, seqs, pos, s.cos, s.sin, q=q)}[op]
    data = torch.randn(n, 4, 64, device="cuda").bfloat16()
    q = data.clone()
    at = q.data_ptr()
    other.wait_stream(torch.cuda.current_stream())
    want = call(q).clone()
    torch.cuda.synchronize()
    busy(other)
    got = call(q)
    del q
    new = [torch.full((n, 4, 64), 100.0, device="cuda").bfloat16() for _ in range(4)]   # into memory that is free
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(t.data_ptr() != at for t in new)


def test_the_status_word_outlives_its_cache_while_a_stream_may_raise_an_error():
    s = Small()
    at = s.cache.status.data_ptr()
    k, v, table, q, bad = s.k, s.v, s.table, s.q[:1], ints(65)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    busy(other)
    with torch.cuda.stream(other):
        s.cache.decode(q, bad)
    s.cache = None
    words = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    assert all(int(w) == 0 and w.data_ptr() != at for w in words) and k.is_cuda and v.is_cuda and table.is_cuda


def test_a_launch_that_fails_leaves_no_error_behind():
    """Launches into a capture that a synchronize has invalidated are refused by the runtime; the next caller's
    check of the last error does not see it."""
    import ctypes as C
    from gqa_transformer_decode_gb300 import ember as E
    with open("/proc/self/maps") as f:
        rt = C.CDLL(next(line.split()[-1] for line in f if "libcudart" in line))
    s = Small()
    kv = E.ember_paged_kv(k=s.k.data_ptr(), v=s.v.data_ptr(), table=s.table.data_ptr(), dtype=E.BF16, n_pages=6,
                          page_size=16, n_kv_heads=2, head_dim=64, n_seqs=1, table_width=4, page_stride=2 * 16 * 64,
                          head_stride=16 * 64, row_stride=64)
    zeros, lens, cu = ints(0, 0, 0), ints(43), ints(0, 3)
    out = torch.empty_like(s.q)
    p = lambda t: C.c_void_p(t.data_ptr())  # noqa: E731
    torch.cuda.synchronize()
    stream, graph = C.c_void_p(), C.c_void_p()
    assert rt.cudaStreamCreate(C.byref(stream)) == 0
    calls = [
        lambda: E.ember_paged_append(C.byref(kv), None, p(s.x), p(s.x), E.BF16, 0, 128, 128, 3, 0, p(zeros), p(zeros),
                                     None, None, 1e-6, p(s.cos), p(s.sin), 64, None, 0, None, stream),
        lambda: E.ember_paged_decode(C.byref(kv), p(s.q), 256, 1, 4, None, p(lens), 0, 0, 0.1, p(out), 256, None, None,
                                     0, None, stream),
        lambda: E.ember_paged_prefill(C.byref(kv), p(s.q), 256, 3, 1, 4, None, p(cu), p(lens), 0, 0, 0.1, p(out), 256,
                                      None, None, stream),
        lambda: E.ember_paged_take_status(p(zeros), p(lens), stream)]
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
    s.cache.decode(s.q[:1], lens)                                    # all as before
    assert s.cache.sync_status() == 0


def test_a_stream_that_is_being_captured_can_be_passed():
    s = Small()
    lens, cu = ints(43), ints(0, 3)
    want = s.cache.decode(s.q[:1], lens), s.cache.prefill(s.q, cu, lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        q = s.q.clone()                                  # of the graph's own memory, gone before its replay
        got = s.cache.decode(q[:1], lens, stream=side), s.cache.prefill(q, cu, lens, stream=side)
        del q
    for t in got:
        t.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and s.cache.sync_status(side) == 0
