"""Adapters of many requests in one batch: values that are not finite in one adapter's b reach the rows that name it, by the
formula, and no other row (a product of a tile's adapter takes in neighbouring rows as zeros, and zero times an infinity is NaN).
Tolerances as derived in test_gpu_adapters.py."""
import numpy as np
import pytest
import torch

from oracle import rows as O
from test_gpu_adapters import TYPES, Case

pytestmark = pytest.mark.gpu
INF = float("inf")


def check(c, y):
    """All outputs against the formula in 64 bits: finite ones within the tolerance, infinities and NaN in their places."""
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    with np.errstate(invalid="ignore"):
        want, size, low, ranks = O.project(f(c.x), f(c.w), f(c.a), f(c.b), f(c.scale), c.ids.cpu().numpy(), f(c.bias))
    got = f(y)
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fine), np.argwhere(np.isfinite(got) != fine)[:8]
    assert np.array_equal(np.nan_to_num(got[~fine], nan=7.0), np.nan_to_num(want[~fine], nan=7.0))
    K, R = c.x.shape[1], c.a.shape[1]
    want, size, low, ranks = (t[fine] for t in (want, size, low, ranks))
    tol = (K / 16 + R / 8 + 9) * 2.0 ** -22 * (size + 2 * low) + 2.0 ** -23 * low
    tol += 2.0 ** -16 * low if c.x.dtype == torch.bfloat16 else 2.0 ** -21 * low + 2.0 ** -24 * ranks
    tol += (np.abs(want) + tol) * (2.0 ** -24 + (0.0 if y.dtype == torch.float32 else torch.finfo(y.dtype).eps / 2))
    tol += torch.finfo(y.dtype).tiny
    err = np.abs(got[fine] - want)
    assert (err <= tol).all(), float((err / tol).max())
    assert c.ad.sync_status() == 0
    return int((~fine).sum())


# One tile a CTA, K shared out over clusters, tiles one after another of several widths, f32 sums added up in between; ranks that
# are filled up to a product's.
SHAPES = [(4, 128, 64, 8, 3), (7, 896, 4864, 32, 5), (16, 24576, 2064, 16, 5), (33, 264, 8, 8, 9), (90, 256, 128, 16, 5),
          (200, 640, 2056, 24, 4), (300, 128, 2056, 64, 8), (777, 1152, 896, 40, 11), (640, 5000, 1096, 16, 6), (1300, 2048, 72, 128, 3)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,N,K,R,A", SHAPES)
def test_an_adapters_infinities_stay_with_its_rows(n, N, K, R, A, dtype):
    g = torch.Generator().manual_seed(n)
    mixed = torch.randint(-1, A, (n,), generator=g)
    mixed[0] = A - 1
    one = torch.full((n,), -1)
    one[min(3, n - 1)] = A - 1                   # the only row that names it, among rows without
    for ids in (mixed, one, mixed.sort().values):
        c = Case(n, N, K, R, A, dtype, ids=ids, bias=n % 2 == 0)
        c.b[A - 1, 5, 3], c.b[A - 1, N - 1, R - 1], c.b[A - 1, 7, 0] = INF, -INF, float("nan")
        if A > 3:
            c.b[1, 5, 0], c.b[1, 77, 2] = -INF, INF
        for out in (None, torch.float32):
            y = c.run(out_dtype=out)
            assert check(c, y) > 0
            assert torch.equal(c.run(out_dtype=out).nan_to_num(nan=7.0), y.nan_to_num(nan=7.0))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_a_whole_adapter_that_is_not_finite(dtype):
    """Its rows lose all their outputs, the others none; with rows of x that are not finite among them."""
    for n, N, K in ((40, 384, 512), (600, 2048, 128)):
        c = Case(n, N, K, 16, 6, dtype, ids=torch.arange(n) % 7 - 1)
        clean = c.run(out_dtype=torch.float32)
        c.b[2] = float("nan")
        c.x[8], c.x[9, 3] = float("nan"), INF
        y = c.run(out_dtype=torch.float32)
        spoilt = c.ids == 2
        spoilt[8:10] = True
        assert not y[spoilt][:, :].isfinite().any() and y[~spoilt].isfinite().all()
        # taken again in another order of sums: each within the bound of test_gpu_adapters.py, so twice that apart
        size = c.x[~spoilt].double().abs() @ c.w.double().abs().T + 2 * 3 * 16 * 0.3 * 4 * 4
        assert ((y[~spoilt] - clean[~spoilt]).abs() <= 2 * (K / 16 + 11) * 2.0 ** -22 * size + 2.0 ** -15).all()
        assert c.ad.sync_status() == (9 if dtype == "f16" else 0)    # A x of rows 8 and 9 is beyond f16's range


def test_a_graph_and_outputs_of_the_callers():
    c = Case(50, 264, 320, 16, 5, bias=True)
    buf = torch.full((52, 400), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:51, 64:328]
    c.run(out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=out)
    c.b[1, 9, 2] = INF
    graph.replay()
    torch.cuda.synchronize()
    assert check(c, out) > 0
    buf[1:51, 64:328] = 7.0
    assert (buf == 7.0).all()
    c.b[1, 9, 2] = 0.5
    graph.replay()
    torch.cuda.synchronize()
    assert check(c, out) == 0
