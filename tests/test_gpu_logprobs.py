"""ember_logprobs through runtime.logprobs against oracle/rows.py in 64 bits.

Tolerances.  The kernel's f32 sums: a thread adds at most c = ceil(V / 512) + 8 terms one after another (fewer where a
row is split), then 9 + 4 + 3 times two sums, so that S and U are off by (c + 16) 2^-24 of their size; each term's
exponential by 2^-22 (the approximation) and by its argument's error, 3 roundings of (x - m) / t log2 e, which
weighs |y| e^y 2^-24 * 3 <= 1.2 * 2^-24 of the largest term and on average E[|y|] 3 * 2^-24 of S, E[|y|] <= entropy.
With c' = c + 16 + 4 + 3: log S is off by (c' + 3 H) 2^-24 + its own rounding; a log probability besides by 3
roundings of itself and of (x - m) / t, which is no larger than it and log S together.  The entropy log S - U / (S t)
by both sums' errors: c'(1 + H) 2^-24 and, for the arguments, 6 (1 + E[y^2]) 2^-24.
Token ids and ranks are compared for equality: they rest on comparisons alone."""
import numpy as np
import pytest
import torch

from oracle import rows as O

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 2.0 ** -24


def logprobs(*a, **k):
    from gqa_transformer_decode_gb300 import runtime
    return runtime.logprobs(*a, **k)


def check(logits, ids, top, t, got):
    x = logits.double().cpu().numpy()
    n, V = x.shape
    lp, H = O.logprobs(x, t)
    if ids is None:
        assert got.logprob is None and got.rank is None
    for r in range(n):
        order = O.order(x[r])
        h = 0.0 if np.isnan(H[r]) else H[r]
        c = -(-V // 512) + 8 + 23
        with np.errstate(invalid="ignore", over="ignore"):
            y = np.where(np.isfinite(x[r]), x[r] - x[r].max(), 0.0) / float(np.float32(t))
            y2 = float(np.nansum(np.exp(lp[r]) * np.minimum(y * y, 1e30)))
        log_s = (c + 3 * h + 2) * EPS + 2 * np.log(V) * EPS

        def near(a, want, tol):
            a = float(a)
            if abs(want) > 2.0 ** 128:  # beyond f32, whose nearest value is infinite: a lowest logit at a temperature below 1
                want = np.copysign(np.inf, want)
            if not np.isfinite(want):
                assert (np.isnan(a) and np.isnan(want)) or a == want, (r, a, want)
            else:
                assert abs(a - want) <= tol, (r, a, want, abs(a - want) / tol)
        near(got.entropy[r], H[r], (c * (1 + h) + 6 * (1 + y2)) * 2 * EPS)
        if ids is not None:
            i = int(ids[r])
            if 0 <= i < V:
                near(got.logprob[r], lp[r, i], log_s + 8 * EPS * abs(lp[r, i]))
                assert int(got.rank[r]) == int(np.nonzero(order == i)[0][0]), r
            else:
                assert np.isnan(float(got.logprob[r])) and int(got.rank[r]) == -1
        best = got.top_ids[r].cpu().numpy()
        assert np.array_equal(best, order[:top]), (r, best, order[:top])
        for k in range(top):
            near(got.top_logprobs[r, k], lp[r, best[k]], log_s + 8 * EPS * abs(lp[r, best[k]]))


def rows(n, V, dtype, seed=0, pad=0, offset=0):
    """Rows in a wider buffer of NaN, from an element on."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((n, V + pad + offset), float("nan"), dtype=TYPES[dtype])
    x = torch.randn(n, V, generator=g) * 2
    x[torch.arange(n), torch.randint(V, (n,), generator=g)] += 8.0
    buf[:, offset:offset + V] = x.to(TYPES[dtype])
    ids = torch.randint(V, (n,), generator=g, dtype=torch.int32)
    return buf.cuda()[:, offset:offset + V], ids.cuda()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,V,top,pad,offset", [
    (1, 1, 1, 0, 0), (3, 2, 2, 0, 0), (5, 7, 7, 1, 0), (2, 31, 20, 0, 1), (4, 32, 32, 3, 0), (3, 33, 32, 0, 3), (2, 255, 5, 1, 0),
    (3, 4093, 32, 0, 0), (2, 4111, 31, 5, 2), (7, 8192, 1, 0, 0), (1, 50257, 20, 0, 0), (70, 9001, 3, 7, 1), (400, 1000, 10, 0, 0),
    (1, 151936, 32, 0, 0), (2, 128257, 0, 1, 1), (33, 40000, 20, 0, 0), (155, 20011, 32, 5, 0)])
def test_shapes(dtype, n, V, top, pad, offset):
    x, ids = rows(n, V, dtype, n + V, pad, offset)
    got = logprobs(x, ids, top=top)
    check(x, ids, top, 1.0, got)
    assert all(torch.equal(a, b) for a, b in zip(got, logprobs(x, ids, top=top)))


@pytest.mark.parametrize("t", [0.05, 0.7, 1.3, 50.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_temperatures(dtype, t):
    for n, V in ((3, 333), (2, 30011)):
        x, ids = rows(n, V, dtype, 5)
        check(x, ids, 8, t, logprobs(x, ids, top=8, temperature=t))


@pytest.mark.parametrize("n", [4, 330])          # a row split over CTAs, and a CTA of its own
@pytest.mark.parametrize("dtype", list(TYPES))
def test_rows_of_every_kind(dtype, n):
    V, dt = 20000, TYPES[dtype]
    low = torch.finfo(dt).min
    g = torch.Generator().manual_seed(3)
    base = (torch.randn(V, generator=g) * 3).to(dt)
    some = torch.randperm(V, generator=g)[:9]
    kinds = []

    def kind(f):
        x = base.clone()
        f(x)
        kinds.append(x)

    def masked(value, keep):
        def f(x):
            kept = x[keep].clone()
            x[:] = value
            x[keep] = kept
        return f
    kind(lambda x: x.fill_(float("-inf")))
    for value in (float("-inf"), low):
        kind(masked(value, some))
        kind(masked(value, some[:1]))
        kind(masked(value, torch.arange(V - 40, V)))
        kind(masked(value, torch.arange(0, V, 2)))
    kind(lambda x: x.fill_(1.5))                                  # all equal
    kind(lambda x: x.copy_((torch.arange(V) / 100.0).to(dt)))     # rising, with equal ones
    kind(lambda x: x.copy_((-torch.arange(V) / 100.0).to(dt)))
    kind(lambda x: x.copy_(torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0).to(dt)))
    kind(lambda x: x[12345:12346].fill_(float("nan")))
    kind(lambda x: x[some].fill_(float("nan")))
    kind(lambda x: x.fill_(float("nan")))
    kind(lambda x: x[777:779].fill_(float("inf")))
    kind(lambda x: x[::1000].fill_(torch.finfo(dt).max))
    kind(lambda x: x[5000:9000].fill_(40.0))                      # thousands of equal largest ones
    x = torch.stack(kinds)
    given = torch.tensor([int(some[0]), 0, V - 1, 12345], dtype=torch.int32)
    for k in range(0, len(kinds), 4):
        part = x[k:k + 4]
        part = part.repeat(-(-n // len(part)), 1)[:n].cuda()
        ids = given.roll(k).repeat(-(-n // 4))[:n].cuda()
        for top in (32, 1):
            got = logprobs(part, ids, top=top)
            few = min(n, 8)
            check(part[:few], ids[:few], top, 1.0, type(got)(*(y[:few] for y in got)))


def test_infinite_given_tokens_and_none():
    x, _ = rows(6, 5000, "f32", 9)
    x[:, 100:200] = float("-inf")
    x[3, 150] = float("nan")
    ids = torch.tensor([150, 100, 199, 150, -1, 5000], dtype=torch.int32, device="cuda")
    check(x, ids, 4, 1.0, logprobs(x, ids, top=4))
    check(x, None, 4, 1.0, logprobs(x, top=4))
    empty = logprobs(x[:0], ids[:0], top=3)
    assert empty.logprob.shape == (0,) and empty.top_ids.shape == (0, 3)


def test_largest_temperatures_and_values():
    x = torch.tensor([[3e38, -3e38, 1e38, 0.0], [1e-38, 2e-38, 0.0, -1e-38]], device="cuda")
    ids = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    for t in (1e-6, 1.0, 1e6):
        got = logprobs(x, ids, top=4, temperature=t)
        assert got.top_ids.tolist() == [[0, 2, 3, 1], [1, 0, 2, 3]]
        assert not got.entropy.isnan().any() and not got.logprob.isnan().any() and not got.top_logprobs.isnan().any()
        assert (got.entropy >= 0).all() and (got.top_logprobs <= 0).all()
    assert got.entropy[1].item() == pytest.approx(np.log(4), rel=1e-6)


def test_graphs_and_streams():
    x, ids = rows(9, 30000, "bf16", 1)
    y, _ = rows(9, 30000, "bf16", 2)
    want = [logprobs(z, ids, top=7) for z in (x, y)]
    buf = x.clone()
    logprobs(buf, ids, top=7)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = logprobs(buf, ids, top=7)
    for z, w in ((x, want[0]), (y, want[1]), (x, want[0])):
        buf.copy_(z)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, w))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = logprobs(y, ids, top=7, stream=side)
    here = logprobs(x, ids, top=7)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want[1])) and all(torch.equal(a, b) for a, b in zip(here, want[0]))


def test_the_greedy_token_of_the_sampler_is_the_first():
    from gqa_transformer_decode_gb300 import ember as E
    x, _ = rows(6, 151936, "f32", 4)
    x[2, 500], x[2, 400] = 60.0, 60.0
    tok = torch.empty(6, dtype=torch.int32, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert E.ember_sample(x.data_ptr(), 6, 151936, 151936, 0.0, 0, 0.0, None, tok.data_ptr(), s) == 0
    got = logprobs(x, tok, top=1)
    assert torch.equal(got.top_ids[:, 0], tok) and int(tok[2]) == 400 and not got.rank.any()
    assert torch.equal(got.logprob, got.top_logprobs[:, 0])


def test_refusals():
    x, ids = rows(2, 64, "f32")
    for bad, err in [(lambda: logprobs(x, ids, top=33), "top > 32"), (lambda: logprobs(x, ids, top=-1), "top"),
                     (lambda: logprobs(x, ids, temperature=0.0), "temperature"),
                     (lambda: logprobs(x, ids, temperature=float("nan")), "temperature"),
                     (lambda: logprobs(x.double(), ids), "float32"), (lambda: logprobs(x[0], ids), "two dimensions"),
                     (lambda: logprobs(x, ids.long()), "ids"), (lambda: logprobs(x, ids[:1]), "ids"),
                     (lambda: logprobs(x.t(), ids), "side by side"), (lambda: logprobs(x.cpu(), ids), "CUDA"),
                     (lambda: logprobs(x[:, :3], ids, top=4), "top"), (lambda: logprobs(x[:1].expand(2, 64), ids), "ldl"),
                     (lambda: logprobs(x.clone().requires_grad_(), ids), "gradient")]:
        with pytest.raises((ValueError, TypeError, RuntimeError), match=err):
            bad()
    with torch.no_grad():
        logprobs(x.clone().requires_grad_(), ids)


def test_rows_beyond_2_31_elements():
    """Offsets of 64 bits: the last of 16800 rows of 128256 bf16 (4.3 GB)."""
    n, V = 16800, 128256
    x = torch.empty(n, V, dtype=torch.bfloat16, device="cuda").fill_(-3.0)
    few, ids = rows(3, V, "bf16", 8)
    x[-3:] = few
    all_ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    all_ids[-3:] = ids
    got = logprobs(x, all_ids, top=5)
    check(few, ids, 5, 1.0, type(got)(*(y[-3:] for y in got)))
    assert got.top_ids[0].tolist() == [0, 1, 2, 3, 4] and got.entropy[7].item() == pytest.approx(np.log(V), rel=1e-6)


def test_masks_of_the_types_lowest_value():
    """A grammar's mask: a handful of tokens, all others at the type's lowest value or -inf, in one call with open rows."""
    for dtype in TYPES:
        x, ids = rows(40, 32000, dtype, 6)
        for r in range(0, 40, 3):
            keep = torch.randperm(32000, generator=torch.Generator().manual_seed(r))[:1 + r // 3].cuda()
            kept = x[r, keep].clone()
            x[r] = torch.finfo(x.dtype).min if r % 2 else float("-inf")
            x[r, keep] = kept
        check(x, ids, 20, 1.0, logprobs(x, ids, top=20))
        check(x, ids, 3, 0.5, logprobs(x, ids, top=3, temperature=0.5))


@pytest.mark.parametrize("n", [3, 40, 200])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_given_tokens_that_a_mask_excludes(dtype, n):
    """-inf and the lowest value as the given token's logit: its rank counts the equal ones before it, in every part of a
    row, in the row's ends and beside what stands for vectors beyond a part."""
    V = 33001
    x, _ = rows(n, V, dtype, 11, pad=3, offset=1)
    g = torch.Generator().manual_seed(n)
    for r in range(n):
        keep = torch.rand(V, generator=g) < (0.5, 0.01, 0.999)[r % 3]
        x[r, ~keep.cuda()] = float("-inf") if r % 2 else torch.finfo(x.dtype).min
    ids = torch.randint(V, (n,), generator=g)
    ids[::5], ids[1::5], ids[2::5] = 0, V - 1, V - 2
    for r in range(0, n, 2):
        x[r, ids[r]] = x[r].min()
    few = list(range(0, n, max(1, n // 24)))
    got = logprobs(x, ids.int().cuda(), top=6)
    check(x[few], ids[few].int(), 6, 1.0, type(got)(*(y[few] for y in got)))


def test_more_rows_than_65535():
    x, ids = rows(70001, 13, "bf16", 5)
    got = logprobs(x, ids, top=3)
    few = list(range(0, 70001, 700))
    check(x[few], ids[few], 3, 1.0, type(got)(*(y[few] for y in got)))
