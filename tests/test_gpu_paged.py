"""The paged-cache operators (through runtime.PagedKV, so through the C ABI)
against oracle/paged.py in 64 bits.

Tolerances, elementwise, from the arithmetic (u = half a step of the type,
2^-8 bf16, 2^-11 f16, 2^-24 f32):
  scores   a product of D terms accumulated in f32, scaled and shifted:
           ds = (D + 4) 2^-23 S, S the largest sum_d |q_d k_d| scale; the tensor
           cores may truncate where f32 addition would round, hence 2^-23
  weights  e^x to 2^-21 relative, two scores' errors in each normalised weight;
           P as the second product's operand: u of its type (bf16 decode: two
           bf16 terms, 2^-16)
  sums     n/16 + 64 partial sums of 2^-23 relative to sum p |v| = A
  output   one rounding: u |out| (and half a subnormal step, 2^-25, for f16)
so |out - exact| <= A (2 ds + 2^-21 + u_P + (n/16 + 64) 2^-23) + u |out| + 2^-25 and
|lse - exact| <= ds + 2^-21 + (n/16 + 64) 2^-23 + 2^-22 |lse|.
append without a norm is exact in f32 (each product and sum rounded by itself),
so it must equal numpy's f32 evaluation bit for bit; with a norm the f32 factor
rsqrt(mean + eps) w is off by at most (D/16 + 16) 2^-23 relative."""
import numpy as np
import pytest
import torch

from oracle import paged as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def runtime():
    from gqa_transformer_decode_gb300 import runtime as R
    return R


class Pool:
    """Pages dealt out in random order; what no sequence holds is NaN."""

    def __init__(self, seed, lens, NKV, D, P, dtype="bf16", row_major=False, extra=3, kscale=1.0):
        g = np.random.default_rng(seed)
        self.P, self.D, self.NKV, self.dtype, self.lens = P, D, NKV, dtype, lens
        per = [-(-n // P) for n in lens]
        pages = sum(per) + extra
        self.table_np = np.full((len(lens), max(per + [1]) + 1), -1, np.int32)
        order = g.permutation(pages)
        shape = (pages, P, NKV, D) if row_major else (pages, NKV, P, D)
        ts = []
        for s in (kscale, 1.0):
            t = torch.full(shape, float("nan"), dtype=DT[dtype])
            ts.append(t.transpose(1, 2) if row_major else t)
        at = 0
        for b, n in enumerate(lens):
            self.table_np[b, :per[b]] = order[at:at + per[b]]
            at += per[b]
            for t, s in zip(ts, (kscale, 1.0)):
                for i in range(per[b]):
                    rows = min(P, n - i * P)
                    t[int(self.table_np[b, i]), :, :rows] = torch.from_numpy(
                        g.standard_normal((NKV, rows, D)) * s).to(DT[dtype])
        self.k, self.v = (self._cuda(t, row_major) for t in ts)
        self.rng = g
        self.remake()

    @staticmethod
    def _cuda(t, row_major):
        return t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if row_major else t.cuda()

    def remake(self):
        self.table = torch.from_numpy(self.table_np).cuda()
        self.cache = runtime().PagedKV(self.k, self.v, self.table)

    def f64(self):
        return self.k.cpu().double().numpy(), self.v.cpu().double().numpy()

    def queries(self, n, NH, scale=1.0):
        return (torch.from_numpy(self.rng.standard_normal((n, NH, self.D)) * scale)).to(DT[self.dtype]).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check_rows(got, lse, want, u_p, u, D, n_keys):
    out, wl, mean, big = want
    ds = (D + 4) * 2.0 ** -23 * big
    sums = (n_keys / 16 + 64) * 2.0 ** -23
    tol = mean * (2 * ds + 2.0 ** -21 + u_p + sums) + u * np.abs(out) + 2.0 ** -25
    err = np.abs(got.double().cpu().numpy() - out)
    assert np.isfinite(err).all() and (err <= tol).all(), (np.nanmax(err / tol), np.unravel_index(np.nanargmax(err / tol), err.shape))
    if lse is not None:
        lse = lse.double().cpu().numpy()
        empty = np.isneginf(wl)
        assert (np.isneginf(lse) == empty).all()
        d = np.abs(lse[~empty] - wl[~empty])
        assert (d <= ds + 2.0 ** -21 + sums + 2.0 ** -22 * np.abs(wl[~empty])).all(), d.max()


def u_decode(dtype):
    return 2.0 ** -16 if dtype == "bf16" else U[dtype]


def check_decode(p, q, got, lse, lens=None, seqs=None, window=0, sinks=0, scale=None):
    k, v = p.f64()
    lens = p.lens if lens is None else lens
    qq = q.double().cpu().numpy()
    for b in range(q.shape[0]):
        s = b if seqs is None else seqs[b]
        if s < 0:
            continue
        n = lens[b]
        want = O.attend(qq[b:b + 1], k, v, p.table_np[s], n, [n - 1], window, sinks, scale)
        check_rows(got[b:b + 1], None if lse is None else lse[b:b + 1], want, u_decode(p.dtype), U[p.dtype], p.D, n)


HEADS = [(14, 2, 64), (32, 8, 64), (8, 8, 128), (16, 1, 128), (4, 2, 16), (6, 2, 32), (3, 3, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("NH,NKV,D", HEADS)
@pytest.mark.parametrize("P,row_major", [(16, False), (64, True)])
def test_decode_over_ragged_lengths(NH, NKV, D, P, row_major, dtype):
    lens = [1, 2, 15, 16, 17, 0, 63, 64, 65, 130, 257]
    p = Pool(NH * 7 + D, lens, NKV, D, P, dtype, row_major)
    q = p.queries(len(lens), NH, 2.0)
    out, lse = p.cache.decode(q, ints(lens), return_lse=True)
    assert p.cache.sync_status() == 0
    check_decode(p, q, out, lse)
    assert (out[5] == 0).all()


@pytest.mark.parametrize("NH,NKV,D,P,lens", [
    (14, 2, 64, 16, [5000]), (8, 1, 128, 128, [4099]), (4, 4, 128, 32, [3001, 5, 2048, 0, 777]),
    (32, 8, 64, 1024, [1500, 1025]), (2, 1, 16, 16, [9000]),
])
def test_decode_split_over_long_sequences(NH, NKV, D, P, lens):
    p = Pool(sum(lens), lens, NKV, D, P)
    q = p.queries(len(lens), NH, 1.5)
    out, lse = p.cache.decode(q, ints(lens), return_lse=True, scale=0.2)
    check_decode(p, q, out, lse, scale=0.2)
    again = p.cache.decode(q, ints(lens), scale=0.2)
    assert torch.equal(out, again)              # no order of arrival in it


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (100, 1), (33, 50), (1000, 17), (7, 5000), (5000, 3)])
def test_decode_window_and_sinks(window, sinks):
    lens = [1, 16, 40, 101, 700, 1999]
    p = Pool(window + sinks, lens, 2, 64, 16)
    # pages without a visible key are given back: their entries are invalid, their rows NaN
    for b, n in enumerate(lens):
        ok = O.visible(n - 1, n, window, sinks)
        for i in range(-(-n // 16)):
            if not ok[i * 16:(i + 1) * 16].any():
                p.k[int(p.table_np[b, i])] = float("nan")
                p.v[int(p.table_np[b, i])] = float("nan")
                p.table_np[b, i] = -1 if i % 2 else 10 ** 9
    p.remake()
    # rows a query does not see inside pages that it reads may hold anything too
    q = p.queries(len(lens), 6, 2.0)
    out, lse = p.cache.decode(q, ints(lens), window=window, sinks=sinks, return_lse=True)
    assert p.cache.sync_status() == 0
    check_decode(p, q, out, lse, window=window, sinks=sinks)


def test_decode_ignores_whatever_lies_in_hidden_rows():
    lens = [50, 333]
    p = Pool(5, lens, 2, 128, 32, "f16")
    q = p.queries(2, 8)
    want = p.cache.decode(q, ints(lens), window=20, sinks=3)
    for b, n in enumerate(lens):
        ok = O.visible(n - 1, n, 20, 3)
        for j in np.nonzero(~ok)[0]:
            for t, x in ((p.k, float("inf")), (p.v, float("nan"))):
                t[int(p.table_np[b, j // 32]), :, j % 32] = x
    assert torch.equal(want, p.cache.decode(q, ints(lens), window=20, sinks=3))


def test_decode_extreme_scores():
    lens = [70, 40]
    p = Pool(9, lens, 1, 64, 16)
    low = torch.finfo(torch.bfloat16).min
    k = p.k
    k[int(p.table_np[0, 1]), :, 3] = 0
    k[int(p.table_np[0, 1]), :, 3, 0] = low               # score -inf or +huge with q
    q = p.queries(2, 2, 3.0)
    q[:, :, 0] = 4.0                                       # 4 * low overflows f32: the score is -inf
    out, lse = p.cache.decode(q, ints(lens), return_lse=True)
    check_decode(p, q, out, lse)
    # every score far below zero, and far above
    for s in (-300.0, 300.0):
        q2 = torch.zeros_like(q)
        q2[:, :, 1] = s
        p.k[:, :, :, 1] = torch.where(p.k[:, :, :, 1].isnan(), p.k[:, :, :, 1], 8.0 + p.k[:, :, :, 1].abs())
        p.k[int(p.table_np[0, 1]), :, 3, 0] = 0
        out, lse = p.cache.decode(q2, ints(lens), return_lse=True)
        check_decode(p, q2, out, lse)
    # only scores of -inf: no weight anywhere
    p.k[int(p.table_np[1, 0]), :, :1] = 0
    p.k[int(p.table_np[1, 0]), :, :1, 0] = low
    out, lse = p.cache.decode(q[1:], ints([1]), seqs=ints([1]), return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    # a value that is not finite and seen shows
    p.v[int(p.table_np[1, 1]), :, 0, 5] = float("nan")
    out = p.cache.decode(q, ints(lens))
    assert out[1, :, 5].isnan().all() and out[0].isfinite().all()


def test_decode_strides_sequence_order_and_padding():
    lens = [33, 200, 64]
    p = Pool(11, lens, 2, 64, 16)
    order = [2, -1, 0, 1, -1, 2]
    want_lens = [64, 7, 20, 200, 10 ** 9, 1]
    wide = p.queries(6, 10)
    q = wide[:, 2:8]                                       # 6 heads out of rows of 10
    buf = torch.full((6, 9, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((6, 6), 5.0, device="cuda")
    out, _ = p.cache.decode(q, ints(want_lens), seqs=ints(order), out=buf[:, 1:7], lse=lse)
    assert p.cache.sync_status() == 0
    check_decode(p, q, out, lse, lens=want_lens, seqs=order)
    assert (buf[:, 0] == 7).all() and (buf[:, 7:] == 7).all()
    for b in (1, 4):
        assert (buf[b] == 7).all() and (lse[b] == 5).all()


def test_decode_device_errors_are_reported_and_leave_the_rest_right():
    lens = [30, 40, 50]
    p = Pool(13, lens, 1, 64, 16)
    q = p.queries(3, 2)
    buf = torch.full((3, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    cap = p.table_np.shape[1] * 16
    for bad_lens, seqs, code in (([30, cap + 1, 50], None, 2), ([30, -1, 50], None, 2), ([30, 40, 50], [0, 3, 2], 1)):
        buf.fill_(7.0)
        p.cache.decode(q, ints(bad_lens), seqs=None if seqs is None else ints(seqs), out=buf)
        assert p.cache.sync_status() == code
        assert p.cache.sync_status() == 0
        assert (buf[1] == 7).all()
        for b in (0, 2):
            check_decode(p, q, buf, None, lens=[30, 40, 50], seqs=[-1 if x != b else b for x in range(3)])
    # a page outside the pool among the visible ones: reported, read as zeros
    for bad in (-1, p.k.shape[0], 2 ** 31 - 1):
        p.table_np[1, 1] = bad
        p.remake()
        out = p.cache.decode(q, ints(lens))
        assert p.cache.sync_status() == 1
        check_decode(p, q, out, None, seqs=[0, -1, 2])
        assert out[1].isfinite().all()


def test_decode_many_short_sequences():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 40, 300)]
    p = Pool(17, lens, 2, 16, 16, extra=0)
    q = p.queries(300, 4, 2.0)
    out, lse = p.cache.decode(q, ints(lens), return_lse=True)
    check_decode(p, q, out, lse)


@pytest.mark.parametrize("B,most,NH,NKV,D", [
    (40, 900, 4, 2, 64), (90, 400, 2, 2, 64), (130, 330, 12, 1, 128), (260, 480, 2, 2, 64), (500, 250, 3, 1, 128),
])
def test_decode_batches_of_every_size_of_cluster(B, most, NH, NKV, D):
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, most, B)]
    lens[0], lens[1] = most, most - 15
    p = Pool(B, lens, NKV, D, 16)
    q = p.queries(B, NH, 2.0)
    out, lse = p.cache.decode(q, ints(lens), return_lse=True)
    check_decode(p, q, out, lse)
    assert torch.equal(out, p.cache.decode(q, ints(lens)))
    out, lse = p.cache.decode(q, ints(lens), window=70, sinks=5, return_lse=True)
    check_decode(p, q, out, lse, window=70, sinks=5)


@pytest.mark.parametrize("at", [0, 151, 299])
def test_decode_one_long_sequence_among_many_short_ones(at):
    rng = np.random.default_rng(at)
    lens = [int(x) for x in rng.integers(0, 40, 300)]
    lens[at] = 6000
    p = Pool(at + 23, lens, 2, 64, 16)
    q = p.queries(300, 4, 2.0)
    seqs = [b if b % 7 != 3 or b == at else -1 for b in range(300)]
    buf = torch.full((300, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    bad = list(lens)
    bad[5] = 10 ** 6
    out, lse = p.cache.decode(q, ints(bad), seqs=ints(seqs), out=buf, return_lse=True)
    assert p.cache.sync_status() == 2
    seqs[5] = -1
    check_decode(p, q, out, lse, seqs=seqs)
    for b in range(300):
        if seqs[b] < 0:
            assert (buf[b] == 7).all()


@pytest.mark.parametrize("lens", [[300, 1000], [9000, 700]])   # joined in a cluster; over the workspace
def test_decode_captured_replayed_and_on_other_streams(lens):
    p = Pool(19, lens, 2, 64, 16)
    q = p.queries(2, 14)
    ln = ints(lens)
    want = p.cache.decode(q, ln)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = p.cache.decode(q, ln, stream=other)
    other.synchronize()
    assert torch.equal(want, got)
    graphs = []
    for _ in range(2):                                     # each allocates a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = p.cache.decode(q, ln)
        graphs.append((g, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (g, _), s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert torch.equal(want, out)
    # new lengths and queries in the same buffers
    ln.copy_(ints([17, 444]))
    q.copy_(p.queries(2, 14))
    graphs[0][0].replay()
    check_decode(p, q, graphs[0][1], None, lens=[17, 444])
    need = p.cache.workspace_bytes(2, 14)
    assert (need > 0) == (lens[0] == 9000)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")      # NaN: any content will do
    assert torch.equal(graphs[0][1], p.cache.decode(q, ln, workspace=ws))
    if need:
        with pytest.raises(RuntimeError, match="workspace"):
            p.cache.decode(q, ln, workspace=ws[:-16])


def test_page_numbers_and_offsets_beyond_32_bits():
    """Pages whose element offsets pass 2^31 (a pool of 5 GB) give the same rows."""
    P, D, NKV, n = 64, 128, 8, 200
    pages = (5 << 29) // (P * D * NKV)
    small = Pool(23, [n], NKV, D, P)
    k = torch.empty((pages, NKV, P, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    far = [pages - 1, pages - 7, 3, pages // 2 + 1]
    for i, f in enumerate(far):
        k[f], v[f] = small.k[int(small.table_np[0, i])], small.v[int(small.table_np[0, i])]
    big = runtime().PagedKV(k, v, ints([far]))
    assert far[0] * NKV * P * D > 2 ** 31
    q = small.queries(1, 16)
    assert torch.equal(small.cache.decode(q, ints([n])), big.decode(q, ints([n])))
    qs = small.queries(20, 16)
    a = small.cache.prefill(qs, ints([0, 20]), ints([n]))
    assert torch.equal(a, big.prefill(qs, ints([0, 20]), ints([n])))
    x = torch.randn(3, NKV, D, device="cuda")
    cos = torch.ones(256, D // 2, device="cuda")
    big.append(x, x, ints([0, 0, 0]), ints([10, 63, 64]), cos, cos * 0)
    assert torch.equal(k[far[0], :, 10], x[0].bfloat16()) and torch.equal(v[far[1], :, 0], x[2].bfloat16())


# ---- prefill ------------------------------------------------------------------------------------------------

def check_prefill(p, q, got, lse, cu, lens, seqs=None, window=0, sinks=0, scale=None, rows=None):
    k, v = p.f64()
    qq = q.double().cpu().numpy()
    for b in range(len(lens)):
        s = b if seqs is None else seqs[b]
        nq = cu[b + 1] - cu[b]
        if s < 0 or nq == 0:
            continue
        pick = np.arange(nq) if rows is None or nq <= rows else np.unique(np.linspace(0, nq - 1, rows).astype(int))
        at = cu[b] + pick
        want = O.attend(qq[at], k, v, p.table_np[s], lens[b], lens[b] - nq + pick, window, sinks, scale)
        ti = torch.from_numpy(at).cuda()
        check_rows(got[ti], None if lse is None else lse[ti], want, U[p.dtype], U[p.dtype], p.D, lens[b])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("NH,NKV,D", HEADS)
@pytest.mark.parametrize("P,row_major", [(16, False), (64, True), (256, False)])
def test_prefill_ragged(NH, NKV, D, P, row_major, dtype):
    new = [1, 9, 0, 33, 64, 70]
    lens = [1, 150, 20, 33, 65, 131]
    p = Pool(NH * 5 + D, lens, NKV, D, P, dtype, row_major)
    cu = [0] + [int(x) for x in np.cumsum(new)]
    q = p.queries(cu[-1], NH, 2.0)
    out, lse = p.cache.prefill(q, ints(cu), ints(lens), return_lse=True)
    assert p.cache.sync_status() == 0
    check_prefill(p, q, out, lse, cu, lens, rows=12)


@pytest.mark.parametrize("NH,NKV,D,P,new,lens", [
    (4, 2, 64, 16, [700], [700]), (8, 8, 128, 128, [300], [1300]), (7, 1, 64, 32, [513, 130], [600, 2000]),
    (16, 1, 128, 64, [250], [250]), (12, 4, 128, 16, [257], [999]),
])
def test_prefill_long(NH, NKV, D, P, new, lens):
    p = Pool(sum(lens), lens, NKV, D, P)
    cu = [0] + [int(x) for x in np.cumsum(new)]
    q = p.queries(cu[-1], NH, 1.5)
    out, lse = p.cache.prefill(q, ints(cu), ints(lens), return_lse=True, scale=0.15)
    check_prefill(p, q, out, lse, cu, lens, scale=0.15, rows=24)
    assert torch.equal(out, p.cache.prefill(q, ints(cu), ints(lens), scale=0.15))


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (100, 1), (33, 50), (300, 17), (7, 5000), (128, 128)])
@pytest.mark.parametrize("D,NH,NKV", [(64, 8, 2), (128, 3, 1)])
def test_prefill_window_and_sinks(window, sinks, D, NH, NKV):
    new, lens = [5, 400, 130], [300, 400, 900]
    p = Pool(window + sinks, lens, NKV, D, 16)
    for b, n in enumerate(lens):                           # pages that no row sees are given back
        ok = np.zeros(n, bool)
        for i in range(n - new[b], n):
            ok |= O.visible(i, n, window, sinks)
        for i in range(-(-n // 16)):
            if not ok[i * 16:(i + 1) * 16].any():
                p.k[int(p.table_np[b, i])] = float("nan")
                p.v[int(p.table_np[b, i])] = float("nan")
                p.table_np[b, i] = -1 if i % 2 else 10 ** 9
    p.remake()
    cu = [0] + [int(x) for x in np.cumsum(new)]
    q = p.queries(cu[-1], NH, 2.0)
    out, lse = p.cache.prefill(q, ints(cu), ints(lens), window=window, sinks=sinks, return_lse=True)
    assert p.cache.sync_status() == 0
    check_prefill(p, q, out, lse, cu, lens, window=window, sinks=sinks, rows=16)


def test_prefill_rows_before_the_sequence_see_nothing_and_rows_outside_stay():
    lens = [4, 0, 37]
    p = Pool(29, [4, 1, 37], 2, 64, 16)
    cu, seqs = [3, 13, 15, 20], [0, 1, 2]                  # ten rows on four keys: six before its start
    n = 26
    wide = p.queries(n, 9)
    q = wide[:, 1:7]
    buf = torch.full((n, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, 6), 5.0, device="cuda")
    out, _ = p.cache.prefill(q, ints(cu), ints(lens), out=buf[:, 2:], lse=lse)
    assert p.cache.sync_status() == 0
    check_prefill(p, q, out, lse, cu, lens)
    assert (out[3:9] == 0).all() and torch.isneginf(lse[3:9]).all() and (out[13:15] == 0).all()
    assert (buf[:, :2] == 7).all()
    for r in (slice(0, 3), slice(20, n)):
        assert (buf[r] == 7).all() and (lse[r] == 5).all()
    # padding sequences and another order of the table's rows
    buf.fill_(7.0)
    lens = [37, 2, 3]
    out = p.cache.prefill(q, ints(cu), ints(lens), seqs=ints([2, -1, 0]), out=buf[:, 2:])
    check_prefill(p, q, out, None, cu, lens, seqs=[2, -1, 0])
    assert (out[13:15] == 7).all() and p.cache.sync_status() == 0


def test_prefill_device_errors_are_reported_and_leave_the_rest_right():
    lens = [30, 40, 50]
    p = Pool(31, lens, 1, 64, 16)
    q = p.queries(60, 2)
    cu = [0, 20, 40, 60]
    cap = p.table_np.shape[1] * 16
    for bad_cu, bad_lens, seqs, code, skipped in (
            (cu, [30, cap + 1, 50], [0, 1, 2], 2, 1), (cu, [30, -5, 50], [0, 1, 2], 2, 1),
            (cu, lens, [0, 9, 2], 1, 1), ([0, 20, 40, 61], lens, [0, 1, 2], 1, 2), ([-1, 20, 40, 60], lens, [0, 1, 2], 1, 0)):
        buf = torch.full((60, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        p.cache.prefill(q, ints(bad_cu), ints(bad_lens), seqs=ints(seqs), out=buf)
        assert p.cache.sync_status() == code
        assert (buf[cu[skipped]:cu[skipped + 1]] == 7).all()
        check_prefill(p, q, buf, None, cu, lens, seqs=[-1 if b == skipped else b for b in range(3)])
    p.table_np[1, 1] = p.k.shape[0]
    p.remake()
    out = p.cache.prefill(q, ints(cu), ints(lens))
    assert p.cache.sync_status() == 1
    check_prefill(p, q, out, None, cu, lens, seqs=[0, -1, 2])
    assert out.isfinite().all()


def test_prefill_captured_and_on_another_stream():
    lens, cu = [300, 90], [0, 100, 131]
    p = Pool(37, lens, 2, 64, 16)
    q = p.queries(131, 8)
    c, ln = ints(cu), ints(lens)
    want = p.cache.prefill(q, c, ln)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = p.cache.prefill(q, c, ln, stream=other)
    other.synchronize()
    assert torch.equal(want, got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = p.cache.prefill(q, c, ln)
    c.copy_(ints([0, 31, 131]))
    g.replay()
    check_prefill(p, q, out, None, [0, 31, 131], lens, rows=10)
    c.copy_(ints(cu))
    g.replay()
    assert torch.equal(want, out)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-4])
def test_other_scales(scale):
    lens, new = [300, 70], [130, 20]
    p = Pool(67, lens, 2, 64, 16)
    q = p.queries(2, 8, 2.0)
    out, lse = p.cache.decode(q, ints(lens), window=100, sinks=3, scale=scale, return_lse=True)
    check_decode(p, q, out, lse, window=100, sinks=3, scale=scale)
    cu = [0, 130, 150]
    q = p.queries(150, 8, 2.0)
    out, lse = p.cache.prefill(q, ints(cu), ints(lens), window=100, sinks=3, scale=scale, return_lse=True)
    check_prefill(p, q, out, lse, cu, lens, window=100, sinks=3, scale=scale, rows=20)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form", ["decode", "prefill", "prefill with scale < 0", "prefill at the end"])
def test_many_small_weights_beside_a_large_one(form, dtype):
    """250000 keys of weight 2^-25.1 with value 1 beside one of weight 1 with value
    0: out is what the small ones sum to, 0.7 %.  Each weight may be off by u_P of
    itself and, for f16, whose step is fixed below a point, by 2^-32 of the largest
    one, which with n keys of |v| <= 1 is n 2^-32 in out and in lse."""
    n = 250000
    p = Pool(3, [n], 1, 16, 1024, dtype)
    sign = -1.0 if "scale" in form else 1.0
    p.k[...] = 0
    p.k[..., 0] = -25.1 * np.log(2.0) * sign
    p.v[...] = 1
    at = (n - 1 if "end" in form else 1234)
    p.k[int(p.table_np[0, at // 1024]), 0, at % 1024, 0] = 0
    p.v[int(p.table_np[0, at // 1024]), 0, at % 1024] = 0
    new = 1 if form == "decode" else 3 if "end" not in form else 200
    q = torch.zeros((new, 2, 16), dtype=p.k.dtype, device="cuda")
    q[..., 0] = 1
    if form == "decode":
        out, lse = p.cache.decode(q, ints([n]), scale=1.0, return_lse=True)
        u_p = 2.0 ** -16 if dtype == "bf16" else 2.0 ** -22
    else:
        out, lse = p.cache.prefill(q, ints([0, new]), ints([n]), scale=sign, return_lse=True)
        u_p = U[dtype]
    k, v = p.f64()
    pos = list(range(n - new, n))
    want = O.attend(q.double().cpu().numpy(), k, v, p.table_np[0], n, pos, 0, 0, sign)
    flush = n * 2.0 ** -32 if dtype == "f16" else 0.0
    ex, _, mean, big = want
    ds, sums = 20 * 2.0 ** -23 * big, (n / 16 + 64) * 2.0 ** -23
    tol = mean * (2 * ds + 2.0 ** -21 + u_p + sums) + flush + U[dtype] * np.abs(ex) + 2.0 ** -25
    err = np.abs(out.double().cpu().numpy() - ex)
    assert (err <= tol).all(), (err / tol).max()
    assert np.abs(lse.double().cpu().numpy() - want[1]).max() <= (ds + 2.0 ** -21 + sums + 2.0 ** -22 * np.abs(want[1])).max()


def test_one_row_of_prefill_is_decode():
    lens = [1, 64, 300]
    p = Pool(41, lens, 2, 128, 32, "f16")
    q = p.queries(3, 8)
    a, la = p.cache.decode(q, ints(lens), window=50, sinks=2, return_lse=True)
    b, lb = p.cache.prefill(q, ints([0, 1, 2, 3]), ints(lens), window=50, sinks=2, return_lse=True)
    check_decode(p, q, a, la, window=50, sinks=2)
    check_prefill(p, q, b, lb, [0, 1, 2, 3], lens, window=50, sinks=2)


# ---- append -------------------------------------------------------------------------------------------------

def tables(n, D, seed=0):
    ang = np.arange(n)[:, None] * (1e4 ** (-np.arange(0, D, 2) / D))[None]
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("NH,NKV,D,P,row_major", [(14, 2, 64, 16, False), (8, 8, 128, 64, True), (4, 2, 16, 16, False),
                                                  (5, 1, 32, 32, True), (32, 8, 64, 128, False)])
@pytest.mark.parametrize("norm", [False, True])
def test_append(NH, NKV, D, P, row_major, dtype, src, norm):
    lens = [40, 170, 1]
    p = Pool(NH + D, lens, NKV, D, P, dtype, row_major)
    seqs = [0] * 12 + [-1] + [1] * 33 + [2] + [-1]
    pos = list(range(28, 40)) + [5] + list(range(131, 164)) + [0] + [-9]
    n = len(seqs)
    qkv = torch.from_numpy(p.rng.standard_normal((n, NH + 2 * NKV, D)) * 3).to(src).cuda()
    cos, sin = tables(170, D)
    wq, wk = (torch.from_numpy(1 + 0.1 * p.rng.standard_normal(D)).bfloat16().cuda() if norm else None for _ in range(2))
    before = [t.clone() for t in (p.k, p.v)]
    q_out = torch.full((n, NH + 1, D), 7.0, dtype=DT[dtype], device="cuda")
    q, k, v = qkv.split((NH, NKV, NKV), 1)
    got = p.cache.append(k, v, ints(seqs), ints(pos), torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda(),
                         q=q, q_norm=wq, k_norm=wk, eps=1e-5, q_out=q_out[:, :NH])
    assert p.cache.sync_status() == 0
    live = np.nonzero(np.array(seqs) >= 0)[0]
    x = qkv.float().cpu().numpy()
    c, s = cos[np.maximum(pos, 0)], sin[np.maximum(pos, 0)]
    parts = []
    for a, w in ((x[:, :NH], wq), (x[:, NH:NH + NKV], wk)):
        if not norm:
            z = torch.from_numpy(O.norm_rope(a, None, 0, c, s, np.float32)).to(DT[dtype])
            parts.append((z.double().numpy(), None))
        else:
            w64 = w.double().cpu().numpy()
            z = O.norm_rope(a, w64, 1e-5, c, s)
            size = np.abs(O.norm_rope(a, w64, 1e-5, np.ones_like(c), np.zeros_like(c)))
            h = D // 2
            pair = np.concatenate([size[..., :h] + size[..., h:]] * 2, -1)
            parts.append((z, U[dtype] * np.abs(z) + pair * (1 + U[dtype]) * (D / 16 + 16) * 2.0 ** -23 + 2.0 ** -25))
    parts.append((v.to(DT[dtype]).double().cpu().numpy(), None))
    rows = [got.double().cpu().numpy()]
    for t in (p.k, p.v):
        t = t.double().cpu().numpy()
        rows.append(np.stack([t[p.table_np[max(b, 0), max(i, 0) // P], :, max(i, 0) % P] for b, i in zip(seqs, pos)]))
    for have, (want, tol) in zip(rows, parts):
        if tol is None:
            assert np.array_equal(have[live], want[live])
        else:
            assert (np.abs(have - want)[live] <= tol[live]).all()
    assert (q_out[:, NH] == 7).all() and (q_out[12] == 7).all() and (q_out[n - 1] == 7).all()
    # every other row of the pool is as it was
    for t, old in zip((p.k, p.v), before):
        t, old = t.clone(), old
        for b, i in zip(seqs, pos):
            if b >= 0:
                t[int(p.table_np[b, i // P]), :, i % P] = 0
                old[int(p.table_np[b, i // P]), :, i % P] = 0
        assert torch.equal(t.view(torch.int16), old.view(torch.int16))


def test_append_equals_the_rope_store_entry_point_bit_for_bit():
    import ctypes as C
    from gqa_transformer_decode_gb300 import ember as E
    p = Pool(43, [64], 4, 64, 16)
    x = torch.randn(64, 4, 64, device="cuda") * 5
    cos, sin = (torch.from_numpy(t).cuda() for t in tables(64, 64))
    p.cache.append(x, x, ints([0] * 64), ints(list(range(64))), cos, sin)
    out = torch.empty(64, 4 * 64, dtype=torch.int16, device="cuda")
    ptr = lambda t: C.c_void_p(t.data_ptr())  # noqa: E731
    assert E.ember_rope_store(ptr(x), 64, 4, 64, ptr(cos), ptr(sin), ptr(out),
                              C.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    rows = torch.cat([p.k[int(i)].transpose(0, 1) for i in p.table_np[0, :4]])
    assert torch.equal(rows.reshape(64, 256).view(torch.int16), out)


def test_append_device_errors_skip_the_token():
    p = Pool(47, [20, 20], 2, 32, 16)
    before = [t.clone() for t in (p.k, p.v)]
    cos, sin = (torch.from_numpy(t).cuda() for t in tables(30, 32))
    x = torch.randn(1, 4, 32, device="cuda")
    cap = p.table_np.shape[1] * 16
    for seq, pos, code in ((2, 0, 1), (0, -1, 2), (0, cap, 2), (0, 30, 2), (1, 2 ** 31 - 1, 2), (0, 2 * 16, 1)):
        out = torch.full((1, 4, 32), 7.0, dtype=torch.bfloat16, device="cuda")
        if (seq, pos) == (0, 32):                          # position within the tables, page entry -1
            c, s = (torch.from_numpy(t).cuda() for t in tables(64, 32))
        else:
            c, s = cos, sin
        p.cache.append(x[:, :2], x[:, :2], ints([seq]), ints([pos]), c, s, q=x, q_out=out)
        assert p.cache.sync_status() == code, (seq, pos)
        assert (out == 7).all()
    for t, old in zip((p.k, p.v), before):
        assert torch.equal(t.view(torch.int16), old.view(torch.int16))


def test_append_many_heads_and_captured():
    NH, NKV, D = 160, 10, 128                              # more threads to a token than a block has
    p = Pool(53, [300], NKV, D, 16)
    x = torch.randn(300, NH + 2 * NKV, D, device="cuda")
    q, k, v = x.split((NH, NKV, NKV), 1)
    cos, sin = (torch.from_numpy(t).cuda() for t in tables(300, D))
    sq, ps = ints([0] * 300), ints(list(range(300)))
    want = p.cache.append(k, v, sq, ps, cos, sin, q=q)
    kk, vv = p.k.clone(), p.v.clone()
    c, s = cos[:, None], sin[:, None]
    a, b = q[..., :64], q[..., 64:]
    assert torch.equal(want, torch.cat((a * c - b * s, b * c + a * s), -1).bfloat16())
    p.k.zero_()
    p.v.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = p.cache.append(k, v, sq, ps, cos, sin, q=q)
    got.zero_()
    g.replay()
    rows = torch.from_numpy(p.table_np[0, :18].astype(np.int64)).cuda()
    assert torch.equal(got, want) and torch.equal(p.k[rows], kk[rows]) and torch.equal(p.v[rows], vv[rows])


# ---- together -----------------------------------------------------------------------------------------------

@pytest.mark.parametrize("NH,NKV,D,window,sinks", [(14, 2, 64, 0, 0), (8, 2, 128, 40, 4)])
def test_a_prompt_in_chunks_then_single_tokens_equals_one_whole_pass(NH, NKV, D, window, sinks):
    """A serving run: two sequences' prompts appended and attended in chunks, then
    tokens one at a time, on growing tables; every row against the oracle on the
    rows that the cache holds at the end."""
    R = runtime()
    rng = np.random.default_rng(59)
    P, total = 16, [150, 97]
    pages = 30
    order = rng.permutation(pages)
    k = torch.full((pages, NKV, P, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, float("nan"))
    table_np = np.full((2, 12), -1, np.int32)
    table = torch.from_numpy(table_np).cuda()
    cache = R.PagedKV(k, v, table)
    cos, sin = (torch.from_numpy(t).cuda() for t in tables(160, D))
    x = [torch.randn(n, NH + 2 * NKV, D, device="cuda") for n in total]
    done, used = [0, 0], 0
    outs = [[], []]
    qs = [[], []]
    wn = torch.from_numpy(1 + 0.1 * rng.standard_normal(D)).bfloat16().cuda()
    steps = [(60, 33), (40, 14)] + [(1, 1)] * 50
    for new in steps:
        for b in range(2):
            while table_np[b].tolist().index(-1) * P < done[b] + new[b]:
                table_np[b, table_np[b].tolist().index(-1)] = order[used]
                used += 1
        table.copy_(torch.from_numpy(table_np))
        rows = torch.cat([x[b][done[b]:done[b] + new[b]] for b in range(2)])
        seqs = [b for b in range(2) for _ in range(new[b])]
        pos = [done[b] + i for b in range(2) for i in range(new[b])]
        q, kk, vv = rows.split((NH, NKV, NKV), 1)
        q = cache.append(kk, vv, ints(seqs), ints(pos), cos, sin, q=q, q_norm=wn, k_norm=wn)
        done = [done[b] + new[b] for b in range(2)]
        if new == (1, 1):
            out = cache.decode(q, ints(done), window=window, sinks=sinks)
        else:
            out = cache.prefill(q, ints([0, new[0], sum(new)]), ints(done), window=window, sinks=sinks)
        for b in range(2):
            sl = slice(0, new[0]) if b == 0 else slice(new[0], sum(new))
            outs[b].append(out[sl])
            qs[b].append(q[sl])
    assert cache.sync_status() == 0 and done == total
    kn, vn = k.double().cpu().numpy(), v.double().cpu().numpy()
    for b in range(2):
        got, q = torch.cat(outs[b]), torch.cat(qs[b])
        want = O.attend(q.double().cpu().numpy(), kn, vn, table_np[b], total[b], np.arange(total[b]), window, sinks)
        check_rows(got, None, want, U["bf16"], U["bf16"], D, total[b])


def test_wrapper_refuses_what_does_not_fit():
    p = Pool(61, [20], 2, 64, 16)
    q = p.queries(1, 4)
    ln = ints([20])
    with pytest.raises(ValueError):
        p.cache.decode(q.half(), ln)
    with pytest.raises(ValueError):
        p.cache.decode(q, ln.long())
    with pytest.raises(ValueError):
        p.cache.decode(q, ints([20, 20]))
    with pytest.raises(ValueError):
        p.cache.decode(q.transpose(1, 2).contiguous().transpose(1, 2), ln)
    with pytest.raises(ValueError):
        p.cache.decode(q, ln, out=torch.empty(1, 3, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        p.cache.decode(q.cpu(), ln)
    with pytest.raises(RuntimeError, match="multiple of n_kv_heads"):
        p.cache.decode(p.queries(1, 3), ln)
    with pytest.raises(RuntimeError, match="window"):
        p.cache.prefill(q, ints([0, 1]), ln, window=-1)
    with pytest.raises(ValueError):
        runtime().PagedKV(p.k, p.v[:, :, :8], p.table)
    with pytest.raises(TypeError):
        runtime().PagedKV(p.k.float(), p.v.float(), p.table)
    assert p.cache.decode(q[:0], ln[:0]).shape == (0, 4, 64)
    assert p.cache.prefill(q[:0], ints([0]), ln[:0]).shape == (0, 4, 64)
