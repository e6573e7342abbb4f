"""Norms of the errors of ember_adapter_project's f32 outputs against 64 bits: what single outputs' bounds, which have to allow
for the worst of every step, let pass.

The tensor cores cut their f32 sums off at each step of 16 products, by up to one unit of the last place, on average half of
one, which is 2^-24 to 2^-23 of the sum so far, on average 0.72 2^-23; and the sum grows with the root of the steps.  So s steps
lose about 0.36 2^-23 (2/3) s of the final sum's norm, at most 2.8 times as much.  The second launch takes at most 48 steps in
one accumulator (1.4e-6) and adds the accumulators' rounded to nearest (2^-24 of a part of the norm each): 3e-6 is twice what is
expected.  A x as W x; its two terms are off by 2^-18 (bf16) or 2^-22 (f16), and by the mean of that in a norm; B t takes R / 8 steps.
A lost second term would be off by 1e-3 / sqrt(3) (bf16) or 1.4e-4 (f16), a lost block or share of K by its share."""
import pytest
import torch

from test_gpu_adapters import TYPES, Case

pytestmark = pytest.mark.gpu


def relative(y, want):
    return ((y.double() - want).norm() / want.norm()).item()


def exact(c):
    """The adapters' contributions alone, in 64 bits."""
    y = torch.zeros(c.x.shape[0], c.w.shape[0], dtype=torch.float64, device="cuda")
    for a in range(c.a.shape[0]):
        at = (c.ids == a).nonzero()[:, 0]
        y[at] = c.x[at].double() @ c.a[a].double().T @ c.b[a].double().T * (1.0 if c.scale is None else c.scale[a].double())
    return y


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,N,K", [
    (1, 1152, 896), (4, 896, 4864), (16, 24576, 4096), (64, 20480, 2048), (33, 896, 4864), (130, 20480, 1032), (200, 640, 4096),
    (256, 4096, 8192), (777, 4096, 1024), (1024, 2048, 4096), (1300, 5000, 520), (4096, 2048, 8192),
])
def test_sums_over_k(n, N, K, dtype):
    """No adapters: lone tiles, split K, tiles one after another of every width, K from one run of blocks to sixteen."""
    c = Case(n, N, K, 8, 2, dtype, ids=[-1] * n)
    y = c.run(out_dtype=torch.float32)
    want = c.x.double() @ c.w.double().T
    assert relative(y, want) <= 3e-6
    assert c.ad.sync_status() == 0
    assert torch.equal(c.run(out_dtype=torch.float32), y)
    # of 16 bits: the rounding's norm, of values each anywhere in half a step, and the sums' 2^-15 at most (K / 16 steps)
    bare = (want.to(c.x.dtype).double() - want).norm().item()
    assert (c.run().double() - want).norm().item() <= (1.0 + 3.0 / (n * N) ** 0.5) * bare + 2.0 ** -15 * want.norm().item()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,N,K,R,A", [
    (1, 1152, 896, 8, 4), (2, 136, 72, 16, 3), (4, 256, 2048, 24, 3), (5, 72, 65544, 128, 3), (15, 256, 2048, 24, 9), (16, 128, 40968, 128, 40),
    (33, 896, 4864, 64, 33), (64, 1024, 2048, 16, 64), (64, 64, 16384, 64, 2), (300, 128, 2056, 64, 8), (300, 64, 4104, 128, 300),
    (777, 1152, 896, 128, 11), (1030, 264, 1032, 64, 12), (2100, 128, 520, 128, 60), (4096, 2048, 4096, 16, 5),
    (300, 64, 16384, 128, 300), (4096, 256, 8192, 64, 3), (2100, 128, 4096, 128, 60),
])
def test_adapters_alone(n, N, K, R, A, dtype):
    """W is zero: what is left is s B A x, of which every block, share of K and term counts.  Its magnitudes are summed apart
    from the adapters of others, so each row's own error is bounded by the call's."""
    g = torch.Generator().manual_seed(n)
    ids = torch.randint(0, A, (n,), generator=g)
    c = Case(n, N, K, R, A, dtype, ids=ids)
    c.w.zero_()
    want = exact(c)
    bound = 3e-6 + (2.0 ** -18 if dtype == "bf16" else 2.0 ** -22) + 0.36 * (2 / 3) * R / 8 * 2.0 ** -23
    y = c.run(out_dtype=torch.float32)
    assert relative(y, want) <= bound
    for r in {0, n // 3, n - 1}:                 # a single row's few outputs vary more
        assert relative(y[r], want[r]) <= 4 * bound, r
    assert c.ad.sync_status() == 0


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,N,K,R,A,ids", [
    (1, 1152, 896, 8, 4, [3]), (1, 128, 128, 8, 4, [0]), (1, 128, 256, 16, 4, [2]), (1, 128, 8192, 64, 4, [1]), (2, 136, 72, 16, 3, [2, -1]),
    (2, 896, 4864, 32, 3, [-1, 1]), (3, 264, 512, 128, 5, [4, 0, 4]), (4, 16384, 2048, 16, 40, [39, -1, 0, 39]), (4, 896, 896, 8, 4, [-1, -1, -1, 2]),
])
def test_few_rows_that_name_adapters(n, N, K, R, A, ids, dtype):
    """K in one share and in clusters of two, four and eight; the adapter in the first share, and in another."""
    for bias in (False, True):
        c = Case(n, N, K, R, A, dtype, ids=ids, bias=bias)
        assert (c.ids >= 0).any()
        c.check(c.run())
        y = c.run(out_dtype=torch.float32)
        c.check(y)
        c.ids.fill_(-1)
        own = (y - c.run(out_dtype=torch.float32)).double()      # the adapters' part, and both sums' errors
        c.ids[:] = torch.tensor(ids)
        want = exact(c)
        size = (c.x.double() @ c.w.double().T).norm() + want.norm() + (0.0 if c.bias is None else c.bias.double().norm() * n ** 0.5)
        assert (own - want).norm() <= 2e-5 * want.norm() + 6e-6 * size
