"""Attention of one token per sequence under shared prefixes (ember_paged_decode_shared through
runtime.PagedKV.decode_shared) against oracle/paged.py in 64 bits.

Tolerances as derived in test_gpu_paged.py, with the weights of the second product rounded once to the cache's type
(u_P = U, as in prefill): the prefix may be multiplied so."""
import numpy as np
import pytest
import torch

from oracle import paged as O
from test_gpu_paged import DT, U, check_rows, ints, runtime

pytestmark = pytest.mark.gpu


class Shared:
    """Groups (shared keys, lengths of their rows) on pages dealt out in random order; what nobody reads is NaN, and
    entries of pages that hold only shared keys, in the rows' own tables, are invalid."""

    def __init__(self, groups, NKV, D, P, dtype="bf16", row_major=False, seed=0, kscale=1.0, extra_width=0):
        g = np.random.default_rng(seed + NKV * D + P)
        self.groups, self.dtype, self.D, self.P = groups, dtype, D, P
        spans = [(0, s) for s, _ in groups]
        self.start, self.lens = [], []
        for s, lens in groups:
            for n in lens:
                spans.append((min(s, n), n))
                self.start.append(min(s, n))
                self.lens.append(n)
        per = [(a // P, max(a // P, -(-b // P))) if b > a else (0, 0) for a, b in spans]
        pages = sum(b - a for a, b in per) + 2
        order = g.permutation(pages)
        self.table_np = np.where(g.random((len(spans), max(b for _, b in per) + 1 + extra_width)) < 0.5, -1, 10 ** 9).astype(np.int32)
        shape = (pages, P, NKV, D) if row_major else (pages, NKV, P, D)
        pool = [torch.full(shape, float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2)]
        if row_major:
            pool = [t.transpose(1, 2) for t in pool]
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.held, at = [], 0
        for r, ((a, b), (p0, p1)) in enumerate(zip(spans, per)):
            self.table_np[r, p0:p1] = order[at:at + p1 - p0]
            at += p1 - p0
            i = torch.arange(a, b, device="cuda")
            page = torch.from_numpy(self.table_np[r].astype(np.int64)).cuda()[i // P]
            kv = [(torch.randn(len(i), NKV, D, generator=gen, device="cuda") * s).to(DT[dtype]) for s in (kscale, 1.0)]
            for t, x in zip(pool, kv):
                t[page, :, i % P] = x
            self.held.append(kv)
        self.k, self.v = pool
        self.table = torch.from_numpy(self.table_np).cuda()
        self.cache = runtime().PagedKV(self.k, self.v, self.table)
        cu = np.cumsum([0] + [len(x) for _, x in groups])
        self.args = (ints(self.lens), ints(cu.tolist()), ints([s for s, _ in groups]), ints(list(range(len(groups)))))
        self.seqs = ints([len(groups) + b for b in range(len(self.lens))])
        self.rng = g

    def queries(self, NH, scale=1.5):
        return torch.from_numpy(self.rng.standard_normal((len(self.lens), NH, self.D)) * scale).to(DT[self.dtype]).cuda()

    def run(self, q, **k):
        return self.cache.decode_shared(q, *self.args, seqs=self.seqs, **k)

    def check(self, q, out, lse, rows=None, scale=None):
        b = 0
        for g, (s, lens) in enumerate(self.groups):
            for n in lens:
                if rows is None or b in rows:
                    kv = [torch.cat((p[:min(s, n)], t)).double() for p, t in zip(self.held[g], self.held[len(self.groups) + b])]
                    want = O.attend_all(q[b:b + 1].double(), *kv, torch.tensor([n - 1], device="cuda"), scale=scale)
                    w = [x.cpu().numpy() for x in want]
                    if n == 0:
                        assert (out[b] == 0).all() and (lse is None or torch.isneginf(lse[b]).all())
                    else:
                        check_rows(out[b:b + 1], None if lse is None else lse[b:b + 1], w[:3] + [w[3].max()], U[self.dtype],
                                   U[self.dtype], self.D, n)
                b += 1
        assert self.cache.sync_status() == 0


HEADS = [(14, 2, 64), (32, 8, 64), (8, 8, 128), (16, 1, 128), (4, 2, 16), (6, 2, 32), (3, 3, 64)]
RAGGED = [(37, [38, 40, 90, 37, 20, 0, 1]), (0, [5, 64]), (64, [65, 128, 129]), (300, [301])]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("NH,NKV,D", HEADS)
@pytest.mark.parametrize("P,row_major", [(16, False), (64, True)])
def test_ragged_groups(NH, NKV, D, P, row_major, dtype):
    p = Shared(RAGGED, NKV, D, P, dtype, row_major)
    q = p.queries(NH)
    p.check(q, *p.run(q, return_lse=True))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("NH,NKV,D", HEADS)
def test_ragged_groups_on_a_wide_table(NH, NKV, D, dtype):
    """A table with room for many keys: the prefixes go by themselves, however short they are."""
    p = Shared(RAGGED + [(1, [1, 2, 3]), (63, [70] * 3), (130, [128, 131, 500] * 20)], NKV, D, 16, dtype, extra_width=20000)
    q = p.queries(NH)
    p.check(q, *p.run(q, return_lse=True))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("NH,NKV,D,P,groups", [
    (14, 2, 64, 16, [(1000, [1001] * 5)]), (32, 8, 64, 32, [(2049, list(range(2050, 2050 + 70)))]),
    (16, 8, 128, 64, [(777, [800] * 20), (3000, [3001, 4100, 2900] * 9), (65, [66] * 3)]),
    (8, 8, 128, 128, [(4000, [4001 + 3 * i for i in range(130)])]), (4, 2, 16, 16, [(513, [600] * 150)]),
    (32, 2, 64, 16, [(1500, [1501, 1600, 0, 700, 1500] * 8)]), (9, 3, 32, 16, [(100, [120] * 33), (5000, [5010] * 2)]),
    (3, 3, 64, 1024, [(1023, [1024, 1025, 2050] * 50)]),
])
def test_larger_groups(NH, NKV, D, P, groups, dtype):
    p = Shared(groups, NKV, D, P, dtype)
    q = p.queries(NH)
    out, lse = p.run(q, return_lse=True)
    n = len(p.lens)
    p.check(q, out, lse, rows=set(range(0, n, max(1, n // 24))) | {n - 1})
    again, lse2 = p.run(q, return_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    p.check(q, p.run(q, scale=0.3), None, rows={0, n // 2}, scale=0.3)


def test_the_same_as_decode_on_a_table_that_spells_the_prefixes_out():
    """Rows whose own tables hold the prefix's pages too: decode on them sees the same keys."""
    p = Shared([(640, [700 + i for i in range(40)]), (96, [100, 333])], 2, 64, 32)
    table = p.table_np.copy()
    b = 0
    for g, (s, lens) in enumerate(p.groups):
        for _ in lens:
            table[len(p.groups) + b, :s // 32] = table[g, :s // 32]
            b += 1
    q = p.queries(8)
    whole = runtime().PagedKV(p.k, p.v, torch.from_numpy(table).cuda())
    a, la = whole.decode(q, p.args[0], seqs=p.seqs, return_lse=True)
    out, lse = p.run(q, return_lse=True)
    p.check(q, out, lse)
    p.check(q, a, la)


def test_scores_that_rise_fall_and_overflow():
    """Prefix and tail far apart in either direction, scores of -inf, and one key that outweighs all."""
    for dtype in ("bf16", "f16"):
        for up, lo in ((0, 40.0), (1, 40.0)):
            p = Shared([(700, [760] * 40)], 2, 64, 16, dtype, seed=up)
            q = p.queries(8, 1.0)
            q[..., 0] = 8.0
            for r, x in enumerate(p.held):           # the first component sets the level
                x[0][:, :, 0] = lo if (r == 0) == bool(up) else -lo
                if r == 0:
                    x[0][350, :, 0] = -lo if up else lo
                s = 0 if r == 0 else 700
                i = torch.arange(s, s + len(x[0]), device="cuda")
                p.k[p.table[r].long()[i // 16], :, i % 16] = x[0]
            p.check(q, *p.run(q, return_lse=True), rows={0, 13, 39})
    p = Shared([(300, [350] * 30)], 1, 64, 16)
    q = p.queries(4)
    i = torch.arange(300, device="cuda")
    p.held[0][0][:] = float("-inf")
    p.k[p.table[0].long()[i // 16], :, i % 16] = p.held[0][0]
    q[:] = q.abs()                                   # every prefix score is -inf
    p.check(q, *p.run(q, return_lse=True), rows={0, 29})


def test_padding_strides_and_outputs_of_the_callers():
    p = Shared([(200, [210, 220, 230] * 12), (50, [51, 60])], 2, 64, 16)
    q = p.queries(8)
    want, wl = p.run(q, return_lse=True)
    n = len(p.lens)
    wide = torch.full((n, 16, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 4:12] = q
    buf = torch.full((n + 2, 10, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, 8), 5.0, device="cuda")
    seqs = p.seqs.clone()
    seqs[[3, 17, n - 1]] = -1
    ws = torch.empty(p.cache.shared_workspace_bytes(n, 8, 2) + 16, dtype=torch.uint8, device="cuda").fill_(0xff)
    versions = buf._version, lse._version
    r = p.cache.decode_shared(wide[:, 4:12], *p.args, seqs=seqs, out=buf[1:n + 1, :8], lse=lse, workspace=ws)
    assert r[0].data_ptr() == buf[1].data_ptr() and (buf._version, lse._version) == (versions[0] + 1, versions[1] + 1)
    live = torch.ones(n, dtype=torch.bool, device="cuda")
    live[[3, 17, n - 1]] = False
    assert torch.equal(buf[1:n + 1, :8][live], want[live]) and torch.equal(lse[live], wl[live])
    assert (buf[1:n + 1, :8][~live] == 7).all() and (lse[~live] == 5).all() and (buf[[0, n + 1]] == 7).all() and (buf[:, 8:] == 7).all()
    assert p.cache.sync_status() == 0


def test_errors_of_device_data():
    p = Shared([(200, [210] * 30), (50, [51, 60])], 2, 64, 16)
    q = p.queries(8)
    want = p.run(q)
    lens, cu, shared, prefixes = p.args

    def run(code, skipped, **over):
        out = torch.full_like(want, 3.0)
        a = dict(lens=lens, groups=cu, shared=shared, prefixes=prefixes, seqs=p.seqs)
        a.update(over)
        p.cache.decode_shared(q, a["lens"], a["groups"], a["shared"], a["prefixes"], seqs=a["seqs"], out=out)
        assert p.cache.sync_status() == code
        keep = torch.ones(32, dtype=torch.bool, device="cuda")
        keep[skipped] = False
        assert torch.equal(out[keep], want[keep]) and (out[~keep] == 3).all()

    def put(t, i, x):
        t = t.clone()
        t[i] = x
        return t
    width = p.table.shape[1] * 16
    run(0, [], lens=lens)
    run(1, [5], seqs=put(p.seqs, 5, len(p.table)))
    run(2, [6], lens=put(lens, 6, width + 1))
    run(2, [7], lens=put(lens, 7, -1))
    run(1, [30, 31], prefixes=put(prefixes, 1, len(p.table)))
    run(1, [30, 31], prefixes=put(prefixes, 1, -1))
    run(2, [30, 31], shared=put(shared, 1, -1))
    run(2, [30, 31], shared=put(shared, 1, width + 1))
    run(1, [31], groups=put(cu, 2, 31))
    # a page that does not exist: its keys read as zeros
    p.table[0, 2] = 10 ** 9
    p.run(q)
    assert p.cache.sync_status() == 1


def test_graphs_and_streams():
    p = Shared([(500, [600 + i for i in range(50)])], 2, 64, 16)
    qs = [p.queries(8) for _ in range(2)]
    want = [p.run(q) for q in qs]
    buf = qs[0].clone()
    p.run(buf)
    one, first = ints([500]), ints([0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = p.run(buf)
        plain = p.cache.decode(buf[:1], one, seqs=first)     # another call right behind it
    for k in (0, 1, 0):
        buf.copy_(qs[k])
        g.replay()
        assert torch.equal(got, want[k])
    assert plain.shape == (1, 8, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both = [(p.run(qs[1], stream=side), p.run(qs[0])) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[1]) and torch.equal(b, want[0]) for a, b in both)


def test_inputs_straight_from_the_kernels_before():
    """q, lens and the last page row written just before the call, as a decode step has it."""
    p = Shared([(800, [850] * 64)], 2, 64, 16)
    q = p.queries(8)
    want = p.run(q)
    lens = p.args[0].clone()
    buf, n = torch.empty_like(q), torch.empty_like(lens)
    for _ in range(20):
        buf.zero_()
        n.zero_()
        buf.copy_(q)
        n.copy_(lens)
        assert torch.equal(p.cache.decode_shared(buf, n, *p.args[1:], seqs=p.seqs), want)


def test_refusals():
    p = Shared([(40, [50, 60])], 2, 64, 16)
    q = p.queries(4)
    lens, cu, shared, prefixes = p.args
    run = p.cache.decode_shared
    for bad, err in [(lambda: run(q.half(), *p.args), "q must"), (lambda: run(q, lens[:1], cu, shared, prefixes), "lens"),
                     (lambda: run(q, lens, cu[:1], shared, prefixes), "groups"), (lambda: run(q, lens, cu, shared, prefixes.long()), "prefixes"),
                     (lambda: run(q, lens, cu[:1], shared[:0], prefixes[:0]), "n_groups"),
                     (lambda: run(q, lens, ints([0, 1, 2, 2]), ints([1, 1, 1]), ints([0, 0, 0])), "n_groups"),
                     (lambda: run(q, *p.args, scale=float("nan")), "scale"), (lambda: run(q.clone().requires_grad_(), *p.args), "gradient"),
                     (lambda: run(q, *p.args, out=q[:1]), "out"), (lambda: run(q[:, :3], *p.args), "n_kv_heads")]:
        with pytest.raises((ValueError, TypeError, RuntimeError), match=err):
            bad()
    assert run(q[:0], lens[:0], ints([0]), shared[:0], prefixes[:0]).shape == (0, 4, 64)


@pytest.mark.parametrize("NH,NKV,D,n_groups,per", [(14, 2, 64, 100, 13), (8, 8, 128, 40, 33), (4, 2, 64, 700, 2)])
def test_many_rows_in_many_groups(NH, NKV, D, n_groups, per):
    """Batches of several chunks of rows, groups found among many; two rows a group read their keys each for itself."""
    g = np.random.default_rng(n_groups)
    groups = []
    for i in range(n_groups):
        s = int(g.integers(0, 300))
        groups.append((s, [int(s + g.integers(-s // 4, 60)) if g.random() < 0.9 else 0 for _ in range(int(g.integers(0, 2 * per + 1)))]))
    p = Shared([(s, [max(0, n) for n in lens]) for s, lens in groups], NKV, D, 16, extra_width=40)
    q = p.queries(NH)
    out, lse = p.run(q, return_lse=True)
    n = len(p.lens)
    p.check(q, out, lse, rows=set(range(0, n, max(1, n // 150))) | {n - 1})
    minus, lse = p.run(q, return_lse=True, scale=-0.2)
    p.check(q, minus, lse, rows=set(range(0, n, max(1, n // 40))), scale=-0.2)


def test_groups_out_of_order_touch_nothing():
    """What the header forbids and only the device can see: no row outside the call's buffers is written, and rows of
    groups that are in order before it are right."""
    p = Shared([(200, [220 + i for i in range(60)]), (300, [310 + i for i in range(90)]), (64, [70] * 50)], 2, 64, 16, extra_width=4000)
    q = p.queries(8)
    lens, cu, sh, pre = p.args
    n = len(p.lens)
    buf = torch.full((n + 2, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for bad in ([0, 60, 20, 200], [0, 60, 900, 200], [0, -5, 150, 200], [5, 60, 150, 200], [0, 60, 150, 180]):
        ws = torch.full((p.cache.shared_workspace_bytes(n, 8, 3) + 256,), 0x5a, dtype=torch.uint8, device="cuda")
        p.cache.decode_shared(q, lens, ints(bad), sh, pre, seqs=p.seqs, out=buf[1:-1], workspace=ws[:-256])
        assert (buf[0] == 7).all() and (buf[-1] == 7).all() and (ws[-256:] == 0x5a).all()
        assert p.cache.sync_status() == 1
    out = p.run(q)
    p.check(q, out, None, rows={0, 61, n - 1})


@pytest.mark.parametrize("width", [0, 6000])     # read for each row, and for the group
def test_the_same_rows_and_prefixes_twice(width):
    """Several groups on one prefix, with different numbers of its keys, and sequences that stand in several rows."""
    p = Shared([(300, [310, 420, 300]), (64, [70, 75])], 2, 64, 16, extra_width=width)
    q = p.queries(8)
    first, lse = p.run(q, return_lse=True)
    p.check(q, first, lse)
    rows = [0, 1, 2, 0, 1, 2, 1, 3, 4, 3]
    q2 = q[rows].contiguous()
    lens = p.args[0][rows].contiguous()
    out, lse2 = p.cache.decode_shared(q2, lens, ints([0, 3, 6, 7, 10]), ints([300, 300, 300, 64]), ints([0, 0, 0, 1]),
                                      seqs=p.seqs[rows].contiguous(), return_lse=True)
    tol = 2.0 ** -8 * first.float().abs().max()  # one rounding of the output, and one of the weights, either way
    assert ((out.float() - first[rows].float()).abs() <= 4 * tol).all() and (lse2 - lse[rows]).abs().max() <= 1e-4
    assert p.cache.sync_status() == 0


def test_nothing_but_padding():
    p = Shared([(300, [310, 420, 300])], 2, 64, 16, extra_width=6000)
    q = p.queries(8)
    out = torch.full_like(q, 3.0)
    p.cache.decode_shared(q, *p.args, seqs=torch.full_like(p.seqs, -1), out=out)
    assert (out == 3).all() and p.cache.sync_status() == 0


def test_twenty_thousand_rows():
    p = Shared([(40, [41 + i % 9 for i in range(12000)]), (33, [30 + i % 19 for i in range(8000)])], 1, 16, 16)
    q = p.queries(4)
    out, lse = p.run(q, return_lse=True)
    p.check(q, out, lse, rows=set(range(0, 20000, 251)) | {11999, 12000, 19999})
