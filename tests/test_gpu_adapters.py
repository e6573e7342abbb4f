"""ember_adapter_project through runtime.Adapters against oracle/rows.py in 64 bits.

Tolerance, per output y: each of the f32 sums (of W x, of A x, of B t over both terms, of the split parts) adds in
steps of 16 products, each step off by at most 2^-22 of the magnitudes summed (its products are exact; the sum of 17
numbers is kept to f32, cut off); so (K / 16 + R / 8 + 9) 2^-22 of |w||x| + 2 |s||b||a||x|.  t's two terms: bf16 2^-16
of |s||b||a||x|; f16 2^-21 of it and 2^-24 of sum |b|.  The scale's product 2^-23.  The output's rounding, half a step:
eps / 2 of |y|, and f32's 2^-24."""
import numpy as np
import pytest
import torch

from oracle import rows as O

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def adapters(*a, **k):
    from gqa_transformer_decode_gb300 import runtime
    return runtime.Adapters(*a, **k)


class Case:
    def __init__(self, n, N, K, R, A, dtype="bf16", seed=0, scale=True, bias=False, ids=None):
        g = torch.Generator().manual_seed(seed + 7 * n + N + K + R)
        dt = TYPES[dtype]
        r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(dt).cuda()  # noqa: E731
        self.x, self.w = r(n, K), r(N, K, scale=0.05)
        self.a, self.b = r(A, R, K, scale=K ** -0.5), r(A, N, R, scale=0.3)
        self.scale = (torch.rand(A, generator=g) * 3 - 1).cuda() if scale else None
        self.bias = r(N) if bias else None
        if ids is None:
            ids = torch.randint(-1, A, (n,), generator=g)
        self.ids = torch.as_tensor(ids, dtype=torch.int32).cuda()
        self.ad = adapters(self.a, self.b, self.scale)

    def run(self, **k):
        return self.ad.project(self.x, self.w, self.ids, bias=self.bias, **k)

    def check(self, y, only=None):
        f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        want, size, low, ranks = O.project(f(self.x), f(self.w), f(self.a), f(self.b), f(self.scale), self.ids.cpu().numpy(),
                                           f(self.bias))
        K, R = self.x.shape[1], self.a.shape[1]
        tol = (K / 16 + R / 8 + 9) * 2.0 ** -22 * (size + 2 * low) + 2.0 ** -23 * low
        tol += 2.0 ** -16 * low if self.x.dtype == torch.bfloat16 else 2.0 ** -21 * low + 2.0 ** -24 * ranks
        tol += (np.abs(want) + tol) * (2.0 ** -24 + (0.0 if y.dtype == torch.float32 else torch.finfo(y.dtype).eps / 2))
        tol += torch.finfo(y.dtype).tiny
        err = np.abs(f(y) - want)
        if only is not None:
            err, tol = err[only], tol[only]
        assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
        assert self.ad.sync_status() == 0


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,N,K,R,A", [
    (1, 8, 8, 8, 1), (1, 1152, 896, 8, 4), (2, 136, 72, 16, 3), (7, 896, 896, 32, 5), (15, 256, 2048, 24, 9), (16, 128, 64, 128, 2),
    (17, 384, 520, 40, 6), (31, 2048, 1024, 16, 40), (33, 896, 4864, 64, 33), (64, 1024, 2048, 16, 64), (65, 512, 320, 72, 20),
    (100, 264, 136, 128, 64), (128, 4096, 64, 8, 200), (129, 640, 512, 48, 7), (200, 1024, 1024, 56, 300), (257, 2056, 264, 32, 3),
    (600, 896, 896, 16, 5), (777, 1152, 896, 128, 11), (1500, 2048, 128, 64, 4)])
def test_shapes(dtype, n, N, K, R, A):
    c = Case(n, N, K, R, A, dtype, bias=n % 2 == 0, scale=n % 3 > 0)
    y = c.run()
    c.check(y)
    z = c.run(out_dtype=torch.float32)
    c.check(z)
    assert torch.equal(y, c.run()) and torch.equal(z, c.run(out_dtype=torch.float32))


@pytest.mark.parametrize("n", [5, 64, 300, 1030])
def test_orders_of_adapters(n):
    A = 6
    base = torch.arange(n) * 5 // n
    for ids in (torch.full((n,), -1), torch.full((n,), 3), base, base.flip(0), torch.arange(n) % A, torch.arange(n) % (A + 1) - 1,
                torch.where(torch.arange(n) == n - 1, 5, -1), torch.where(torch.arange(n) % 16 == 15, 2, -7)):
        c = Case(n, 520, 320, 16, A, ids=ids)
        c.check(c.run(out_dtype=torch.float32))


def test_rows_in_another_order():
    """The same rows in another order give the same outputs up to rounding: which CTA of a cluster adds an adapter's
    products goes by the adapter's place among its tile's, so the sums may be joined in another order."""
    c = Case(300, 640, 512, 32, 4, ids=torch.arange(300) * 4 // 300)
    y = c.run(out_dtype=torch.float32)
    c.check(y)
    p = torch.randperm(300, generator=torch.Generator().manual_seed(1)).cuda()
    c.x, c.ids = c.x[p].contiguous(), c.ids[p].contiguous()
    c.check(c.run(out_dtype=torch.float32))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_strides_and_outputs_of_the_callers(dtype):
    c = Case(37, 264, 136, 16, 5, dtype, bias=True)
    want = c.run()
    wide = torch.full((37, 200), float("nan"), dtype=TYPES[dtype], device="cuda")
    wide[:, 32:168] = c.x
    c.x = wide[:, 32:168]
    for ot in (TYPES[dtype], torch.float32):
        buf = torch.full((40, 400), 7.0, dtype=ot, device="cuda")
        out = buf[1:38, 64:328]
        at = buf._version
        assert c.run(out=out).data_ptr() == out.data_ptr() and buf._version == at + 1
        c.check(out)
        if ot != torch.float32:
            assert torch.equal(out, want)
        buf[1:38, 64:328] = 7.0
        assert (buf == 7.0).all()
    ws = torch.empty(c.ad.workspace_bytes(37) + 64, dtype=torch.uint8, device="cuda").fill_(0xff)
    assert torch.equal(c.run(workspace=ws), want)


def test_one_rows_values_stay_its_own():
    """A row that is not finite, and an adapter's a, spoil only the rows that read them."""
    c = Case(90, 256, 128, 16, 5)
    y = c.run()
    own = (c.ids == 2).nonzero()[:, 0]
    c.x[10] = float("nan")
    c.x[11, 5] = float("inf")
    c.a[2, 3] = float("nan")
    z = c.run()
    bad = torch.zeros(90, dtype=torch.bool, device="cuda")
    bad[own] = True
    bad[10:12] = True
    assert torch.equal(z[~bad], y[~bad]) and not z[bad].isfinite().any(-1).all()
    assert not z[10].isfinite().any()


def test_errors_of_device_data():
    c = Case(40, 128, 64, 8, 3)
    y = c.run()
    ids = c.ids.clone()
    c.ids[7], c.ids[9] = 3, 1 << 30
    z = c.run()
    assert c.ad.sync_status() == 1 and c.ad.sync_status() == 0
    c.ids[7], c.ids[9] = -1, -5
    assert torch.equal(c.run(), z)
    c.ids = ids
    assert torch.equal(c.run(), y)
    c = Case(40, 128, 64, 8, 3, "f16", ids=torch.arange(40) % 3)
    c.check(c.run())
    c.x[4] = 60000.0
    c.a[1] = 10.0
    c.run()
    assert c.ad.sync_status() == 9


def test_small_and_large_values_of_f16():
    for size in (1e-3, 100.0):
        c = Case(50, 256, 512, 32, 4, "f16")
        c.x.mul_(size)
        c.check(c.run(out_dtype=torch.float32))


def test_graphs_and_streams():
    c = Case(70, 1024, 1024, 16, 9)
    d = Case(70, 1024, 1024, 16, 9, seed=50)
    want = [c.run(), c.ad.project(d.x, c.w, d.ids)]
    assert not torch.equal(*want)
    x, ids = c.x.clone(), c.ids.clone()
    c.ad.project(x, c.w, ids)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = c.ad.project(x, c.w, ids)
        again = c.ad.project(x, c.w, ids, out_dtype=torch.float32)
    for k, src in ((0, c), (1, d), (0, c)):
        x.copy_(src.x)
        ids.copy_(src.ids)
        g.replay()
        assert torch.equal(got, want[k]) and torch.equal(again.bfloat16(), want[k])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both = []
    for _ in range(20):      # calls that overlap, each with its own workspace
        both.append((c.ad.project(d.x, c.w, d.ids, stream=side), c.run()))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[1]) and torch.equal(b, want[0]) for a, b in both)
    assert c.ad.sync_status(side) == 0


def test_inputs_straight_from_a_kernel_before():
    """x and ids written by the kernel just before: the second launch starts early and must not read them sooner."""
    c = Case(64, 2048, 2048, 16, 8)
    want = c.run()
    keep_x, keep_ids = c.x.clone(), c.ids.clone()
    for _ in range(30):
        c.x.zero_()
        c.ids.fill_(-1)
        big = torch.randn(1 << 22, device="cuda")
        c.x.copy_(keep_x)
        c.ids.copy_(keep_ids)
        assert torch.equal(c.run(), want)
        del big


def test_refusals():
    c = Case(4, 128, 64, 8, 3)
    x, w, ids, p = c.x, c.w, c.ids, c.ad.project
    f = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    for bad, err in [(lambda: p(x.half(), w, ids), "x must be"), (lambda: p(x[:, :56], w, ids), "x must be"),
                     (lambda: p(x, w[:64], ids), "w must be"), (lambda: p(x, w.t().contiguous().t(), ids), "w must be"),
                     (lambda: p(x, w, ids[:3]), "ids"), (lambda: p(x, w, ids.long()), "ids"),
                     (lambda: p(x, w, ids, bias=f(64)), "bias"), (lambda: p(x, w, ids, out=f(4, 64)), "out must"),
                     (lambda: p(x, w, ids, out=f(4, 128, d=torch.float16)), "out must"),
                     (lambda: p(x, w, ids, out_dtype=torch.float16), "out_dtype"), (lambda: p(x, w, ids, out_dtype=3), "out_dtype"),
                     (lambda: p(x, w, ids, workspace=f(64, d=torch.uint8)), "workspace"),
                     (lambda: p(x, w, ids, out=f(4, 132)[:, :128]), "row stride"),
                     (lambda: p(x.clone().requires_grad_(), w, ids), "gradient"), (lambda: p(x.cpu(), w, ids), "cuda"),
                     (lambda: adapters(c.a, c.b[:2]), "b must"), (lambda: adapters(c.a, c.b, c.scale[:2]), "scale"),
                     (lambda: adapters(c.a.float(), c.b.float()), "bfloat16"), (lambda: adapters(c.a.cpu(), c.b.cpu()), "CUDA"),
                     (lambda: adapters(f(2, 4, 64), f(2, 128, 4)).project(x, w, ids), "rank"),
                     (lambda: adapters(f(2, 136, 64), f(2, 128, 136)).project(x, w, ids), "rank")]:
        with pytest.raises((ValueError, TypeError, RuntimeError), match=err):
            bad()
    assert p(x[:0], w, ids[:0]).shape == (0, 128)
    c.a.requires_grad_()
    with pytest.raises(ValueError, match="a requires a gradient"):
        c.run()
    with torch.no_grad():
        c.run()


def test_offsets_beyond_2_31():
    """Rows far apart, in x and in out: 64-bit offsets in both launches and every form of the output."""
    for n, R in ((3, 16), (200, 64)):
        far = (1 << 31) // n + 64
        far -= far % 8
        c = Case(n, 136, 64, R, 3)
        base = torch.empty((n - 1) * far + 200, dtype=torch.bfloat16, device="cuda")
        x = torch.as_strided(base, (n, 64), (far, 1))
        x.copy_(c.x)
        out = torch.as_strided(base, (n, 136), (far, 1), 64)
        want = c.run()
        c.x = x
        assert torch.equal(c.run(out=out), want)


def test_calls_that_share_a_workspace_in_turn():
    c, d = Case(20, 256, 512, 16, 4), Case(300, 256, 512, 16, 4, seed=9)
    ws = torch.empty(d.ad.workspace_bytes(300), dtype=torch.uint8, device="cuda").fill_(0x7f)
    want = [c.run(), d.run()]
    for _ in range(10):
        assert torch.equal(c.run(workspace=ws), want[0]) and torch.equal(d.run(workspace=ws), want[1])


def test_status_word_and_inputs_outlive_a_call_on_another_stream():
    c = Case(64, 512, 512, 16, 4)
    want = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    x, ids = c.x.clone(), c.ids.clone()
    torch.cuda.current_stream().synchronize()
    y = c.ad.project(x, c.w, ids, stream=side)
    del x, ids
    junk = [torch.full((64, 512), 9.0, device="cuda").bfloat16() for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(y, want) and len(junk) == 4


def test_forms_of_the_first_launch():
    """More adapters than rows, rows of a tile that all name different adapters, one adapter for all of many rows."""
    for n, N, K, R, A in ((64, 128, 2048, 64, 3), (64, 128, 2056, 64, 3), (65, 128, 64, 8, 200), (300, 264, 512, 8, 300),
                          (257, 128, 4096, 32, 1), (16, 1024, 8192, 128, 16), (33, 8, 8, 8, 40)):
        c = Case(n, N, K, R, A, ids=np.random.default_rng(n).permutation(max(n, A))[:n] % A)
        c.check(c.run())
        c.check(c.run(out_dtype=torch.float32))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,N,K,R,A", [
    (5, 72, 65544, 128, 3), (16, 128, 40968, 128, 40), (33, 136, 16456, 128, 5), (64, 64, 16384, 64, 2), (100, 200, 9000, 56, 4),
    (128, 128, 8200, 72, 3), (129, 136, 8192, 40, 7), (300, 128, 2056, 64, 8), (300, 64, 4104, 128, 300), (1030, 264, 1032, 64, 12),
    (2100, 128, 520, 128, 60), (4100, 72, 1096, 16, 1),
])
def test_the_first_launch_on_tensor_cores(dtype, n, N, K, R, A):
    """Enough multiplications (2^25, 2^26 from 16 adapters on) that A x goes on tcgen05: each width of its tiles, several
    row tiles, K split over clusters of every size, runs of rows, rows in any order and without adapters."""
    assert n * R * K > (1 << 25) * (2 if min(n, A) >= 16 else 1)
    g = np.random.default_rng(n)
    for ids in (g.integers(-1, A, n), np.sort(g.integers(0, A, n)), np.full(n, A - 1), np.where(g.random(n) < 0.02, 0, -1)):
        c = Case(n, N, K, R, A, dtype, ids=ids)
        y = c.run()
        c.check(y)
        assert torch.equal(c.run(), y)


def test_errors_of_the_first_launch_on_tensor_cores():
    c = Case(300, 128, 2056, 64, 8)
    ids = c.ids.clone()
    ids[7], ids[200] = 8, 1 << 30
    y = c.ad.project(c.x, c.w, ids)
    assert c.ad.sync_status() == 1
    c.ids = torch.where(ids >= 8, -1, ids)
    c.check(y)
    c = Case(300, 128, 2056, 64, 8, "f16")
    c.ad = adapters(c.a, c.b, torch.full((8,), 1e5, device="cuda"))
    c.ids[:] = 3
    y = c.run()
    assert c.ad.sync_status() == 9 and not torch.isfinite(y).all()


def test_a_graph_sees_new_ids_and_new_adapters():
    """What a captured call reads is read at every replay: ids, adapters, scales, x and W."""
    for n, N, K, R, A in ((6, 256, 512, 16, 4), (300, 128, 2056, 64, 8)):
        c = Case(n, N, K, R, A)
        c.run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = c.run()
        d = Case(n, N, K, R, A, seed=77)
        for mine, new in ((c.x, d.x), (c.w, d.w), (c.a, d.a), (c.b, d.b), (c.scale, d.scale), (c.ids, d.ids)):
            mine.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        d.check(y)
        c.ids.fill_(-1)
        g.replay()
        torch.cuda.synchronize()
        c.check(y)


@pytest.mark.parametrize("A", [20, 3])           # A x row by row and on tensor cores
def test_more_rows_than_65535(A):
    c = Case(70000, 64, 64, 8, A)
    c.check(c.run())
