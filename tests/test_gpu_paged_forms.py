"""The forms of the paged-cache kernels that only large calls run in, against
oracle/paged.py's attend_all in 64 bits: prefill with more tile pairs than SMs
(CTAs that take over waiting ones), many sequences, scores that move the
reference maximum; decode along the line with groups of 9 to 16 heads and its
join; append with a token's heads in turn; weights whose rounding shows.

Tolerances as in test_gpu_paged.py, with the largest product taken per row and
head: with u half a step of the type, ds = (D + 4) 2^-23 sum_d |q_d k_d| scale,
    |out - exact| <= A (2 ds + 2^-21 + u_P + (n/16 + 64) 2^-23) + u |out| + 2^-25,
    |lse - exact| <= ds + 2^-21 + (n/16 + 64) 2^-23 + 2^-22 |lse|,
A = sum p |v|.  u_P is the rounding of a weight for the second product: prefill on
tcgen05 u of the type; decode and the warp-product prefill two terms, 2^-16 for
bf16 and 2^-22 for f16.  An f16 weight is also off by up to 2^-32 of its row's
largest (its step is fixed below 2^-14), over n keys at most n 2^-32 max |v|."""
import numpy as np
import pytest
import torch

from oracle import paged as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TWO = {"bf16": 2.0 ** -16, "f16": 2.0 ** -22}      # two terms


def runtime():
    from gqa_transformer_decode_gb300 import runtime as R
    return R


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Held:
    """Sequences' keys and values, laid into pages dealt out in random order; rows that no
    sequence holds are NaN."""

    def __init__(self, seed, lens, NKV, D, P, dtype="bf16", row_major=False, wide=1):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.P, self.D, self.NKV, self.dtype, self.row_major = lens, P, D, NKV, dtype, row_major
        self.keys = [self.normal(n, NKV, D) for n in lens]
        self.values = [self.normal(n, NKV, D) for n in lens]
        per = [-(-n // P) for n in lens]
        order = np.random.default_rng(seed).permutation(sum(per) + 2)
        self.table_np = np.full((len(lens), max(per + [1]) + wide), -1, np.int32)
        at = 0
        for b, n in enumerate(per):
            self.table_np[b, :n] = order[at:at + n]
            at += n
        self.n_pages = sum(per) + 2
        self.lay()

    def normal(self, *shape, scale=1.0):
        return (torch.randn(shape, generator=self.g, device="cuda") * scale).to(DT[self.dtype])

    def lay(self):
        shape = (self.n_pages, self.P, self.NKV, self.D)
        pools = []
        for rows in (self.keys, self.values):
            t = torch.full(shape, float("nan"), dtype=DT[self.dtype], device="cuda")
            for b, x in enumerate(rows):
                i = torch.arange(x.shape[0], device="cuda")
                t[torch.from_numpy(self.table_np[b].astype(np.int64)).cuda()[i // self.P], i % self.P] = x
            t = t.transpose(1, 2)
            pools.append(t if self.row_major else t.contiguous())
        self.k, self.v = pools
        self.table = torch.from_numpy(self.table_np).cuda()
        self.cache = runtime().PagedKV(self.k, self.v, self.table)

    def check(self, b, q, pos, out, lse, u_p, window=0, sinks=0, scale=None):
        """Rows q at positions pos of sequence b."""
        k, v = self.keys[b].double(), self.values[b].double()
        want, wl, mean, big = O.attend_all(q.double(), k, v, pos, window, sinks, scale)
        n = k.shape[0]
        u = U[self.dtype]
        ds = (self.D + 4) * 2.0 ** -23 * big
        sums = (n / 16 + 64) * 2.0 ** -23
        flush = n * 2.0 ** -32 * v.abs().max() if self.dtype == "f16" and n else 0.0
        tol = mean * (2 * ds[..., None] + 2.0 ** -21 + u_p + sums) + flush + u * want.abs() + 2.0 ** -25
        err = (out.double() - want).abs()
        assert (err <= tol).all(), (b, (err / tol).nan_to_num(nan=torch.inf).max().item(), err.isnan().any().item())
        if lse is not None:
            empty = torch.isneginf(wl)
            assert torch.equal(torch.isneginf(lse), empty), b
            d = (lse.double() - wl).abs()[~empty]
            assert (d <= (ds + 2.0 ** -21 + sums + 2.0 ** -22 * wl.abs())[~empty]).all(), (b, d.max().item())

    def check_prefill(self, q, cu, out, lse, u_p=None, seqs=None, **mask):
        for i in range(len(cu) - 1):
            b = i if seqs is None else seqs[i]
            nq = cu[i + 1] - cu[i]
            if b < 0 or nq == 0:
                continue
            pos = torch.arange(self.lens[b] - nq, self.lens[b], device="cuda")
            r = slice(cu[i], cu[i + 1])
            self.check(b, q[r], pos, out[r], None if lse is None else lse[r], U[self.dtype] if u_p is None else u_p, **mask)

    def check_decode(self, q, out, lse, **mask):
        for b, n in enumerate(self.lens):
            self.check(b, q[b:b + 1], torch.tensor([n - 1], device="cuda"), out[b:b + 1], lse[b:b + 1], TWO[self.dtype], **mask)


def cumulated(new):
    return [0] + [int(x) for x in np.cumsum(new)]


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def pairs_of(new, NH, NKV):
    """Tile pairs that have rows."""
    per = 2 * (128 // (NH // NKV))
    return sum(-(-n // per) for n in new) * NKV


# ---- prefill with more tile pairs than SMs --------------------------------------------------------------------

def uneven(per, count):
    """New tokens and keys before them: whole pairs, a pair and a token, the first tile alone (the second
    without tokens), one token, none, and many; on nothing, on a little and on many key tiles.  Sequences
    without keys and with fewer keys than rows among them."""
    news = [3 * per + 5, 1, per // 2, per + 1, 0, 2 * per, per // 2 + 1, 5 * per - 1, per // 4]
    pasts = [0, 700, 63, 1409, 64, 0, 1, 130, 2000, 17, 1100]
    new = [news[i % len(news)] for i in range(count)]
    lens = [new[i] + pasts[i * 7 % len(pasts)] for i in range(count)]
    new[3], lens[3] = per + 9, 0
    new[7], lens[7] = per * 2, per - 13
    return new, lens


@pytest.mark.parametrize("NH,NKV,D,P,dtype,row_major,mask", [
    (32, 8, 64, 16, "bf16", False, {}), (32, 8, 64, 64, "f16", True, {}),
    (16, 8, 128, 32, "f16", False, {}), (16, 8, 128, 128, "bf16", True, {}),
    (16, 8, 128, 64, "bf16", False, dict(window=300, sinks=4)), (32, 8, 64, 32, "f16", False, dict(window=90, sinks=70)),
    (56, 8, 64, 16, "bf16", False, dict(window=1000)), (24, 8, 128, 16, "bf16", False, {}),
    (16, 8, 16, 16, "bf16", False, {}), (8, 8, 32, 64, "f16", True, dict(window=500, sinks=1)),
])
def test_prefill_with_more_tile_pairs_than_sms(NH, NKV, D, P, dtype, row_major, mask):
    per = 2 * (128 // (NH // NKV))
    new, lens = uneven(per, 37)
    pairs = pairs_of(new, NH, NKV)
    assert pairs > 2 * sms() and max(lens) > 16 * 64   # rounds of CTAs; key tiles past the K / V ring's slots
    p = Held(NH + D + P, lens, NKV, D, P, dtype, row_major)
    cu = cumulated(new)
    q = p.normal(cu[-1], NH, D, scale=2.0)
    out, lse = p.cache.prefill(q, ints(cu), ints(lens), return_lse=True, **mask)
    assert p.cache.sync_status() == 0
    p.check_prefill(q, cu, out, lse, **mask)
    again, lse2 = p.cache.prefill(q, ints(cu), ints(lens), return_lse=True, **mask)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("NH,NKV,D,dtype", [(32, 8, 64, "bf16"), (16, 8, 128, "f16")])
def test_prefill_of_one_long_prompt_over_several_rounds(NH, NKV, D, dtype):
    per = 2 * (128 // (NH // NKV))
    n = per * (3 * sms() // NKV) + per // 2 + 3
    p = Held(D, [n], NKV, D, 64, dtype)
    q = p.normal(n, NH, D, scale=2.0)
    out, lse = p.cache.prefill(q, ints([0, n]), ints([n]), return_lse=True)
    assert p.cache.sync_status() == 0
    p.check_prefill(q, [0, n], out, lse)


@pytest.mark.parametrize("NH,NKV,D", [(32, 8, 64), (16, 8, 128)])
def test_prefill_of_several_rounds_with_padding_captured_and_beside_another(NH, NKV, D):
    """Two graphs of the same call replayed at once on two streams, then with other rows."""
    per = 2 * (128 // (NH // NKV))
    new, lens = uneven(per, 30)
    p = Held(5 * D, lens, NKV, D, 32)
    cu = cumulated(new)
    q = p.normal(cu[-1], NH, D, scale=2.0)
    seqs = [-1 if b % 6 == 2 else b for b in range(30)]
    c, ln, sq = ints(cu), ints(lens), ints(seqs)
    graphs = []
    for _ in range(2):
        out = torch.full((cu[-1], NH, D), 7.0, dtype=q.dtype, device="cuda")
        lse = torch.full((cu[-1], NH), 5.0, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.cache.prefill(q, c, ln, seqs=sq, out=out, lse=lse)
        graphs.append((g, out, lse, torch.cuda.Stream()))
    for _ in range(3):
        for g, _, _, s in graphs:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert p.cache.sync_status() == 0
    for _, out, lse, _ in graphs:
        p.check_prefill(q, cu, out, lse, seqs=seqs)
        for b in range(30):
            if seqs[b] < 0:
                assert (out[cu[b]:cu[b + 1]] == 7).all() and (lse[cu[b]:cu[b + 1]] == 5).all()
    assert torch.equal(graphs[0][1], graphs[1][1])
    q.copy_(p.normal(cu[-1], NH, D, scale=2.0))
    graphs[1][0].replay()
    assert p.cache.sync_status() == 0
    p.check_prefill(q, cu, graphs[1][1], graphs[1][2], seqs=seqs)


def test_prefill_errors_among_several_rounds_leave_the_rest_right():
    NH, NKV, D = 16, 8, 128
    new, lens = uneven(128, 30)
    p = Held(77, lens, NKV, D, 64)
    cu = cumulated(new)
    q = p.normal(cu[-1], NH, D, scale=2.0)
    bad = list(lens)
    bad[11] = p.table_np.shape[1] * 64 + 1
    out = torch.full((cu[-1], NH, D), 7.0, dtype=q.dtype, device="cuda")
    p.cache.prefill(q, ints(cu), ints(bad), out=out)
    assert p.cache.sync_status() == 2 and p.cache.sync_status() == 0
    assert new[11] > 0 and (out[cu[11]:cu[12]] == 7).all()
    p.check_prefill(q, cu, out, None, seqs=[-1 if b == 11 else b for b in range(30)])
    out = torch.full((cu[-1], NH, D), 7.0, dtype=q.dtype, device="cuda")
    p.cache.prefill(q, ints(cu), ints(lens), seqs=ints([30 if b == 20 else b for b in range(30)]), out=out)
    assert p.cache.sync_status() == 1
    assert new[20] > 0 and (out[cu[20]:cu[21]] == 7).all()
    p.check_prefill(q, cu, out, None, seqs=[-1 if b == 20 else b for b in range(30)])


# ---- prefill of many sequences ----------------------------------------------------------------------------------

@pytest.mark.parametrize("B", [33, 100, 300])
@pytest.mark.parametrize("most,NH,NKV,D", [(900, 8, 2, 64), (260, 4, 2, 128), (40, 6, 2, 64)])   # tcgen05 twice; warp products
def test_prefill_of_many_sequences(B, most, NH, NKV, D):
    rng = np.random.default_rng(B + most)
    new = [int(x) for x in rng.integers(0, 12, B)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, most - 12, B))]
    new[31], new[32] = 0, 5                            # on both sides of the 32 that a warp looks through at once
    lens[32], lens[5], new[5] = most, 0, 0
    p = Held(B, lens, NKV, D, 16)
    cu = cumulated(new)
    q = p.normal(cu[-1], NH, D, scale=2.0)
    seqs = [-1 if b % 9 == 4 and b != 32 else b for b in range(B)]
    out = torch.full((cu[-1], NH, D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((cu[-1], NH), 5.0, device="cuda")
    p.cache.prefill(q, ints(cu), ints(lens), seqs=ints(seqs), out=out, lse=lse)
    assert p.cache.sync_status() == 0
    p.check_prefill(q, cu, out, lse, seqs=seqs)
    for b in range(B):
        if seqs[b] < 0:
            assert (out[cu[b]:cu[b + 1]] == 7).all() and (lse[cu[b]:cu[b + 1]] == 5).all()


# ---- scores that move the reference maximum ---------------------------------------------------------------------

FORMS = {"several rounds": ([700] * 5, [900] * 5), "keys split": ([40], [900]), "warp products": ([40, 3], [120, 90])}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("course", ["rising", "falling", "waves", "far below", "far above"])
def test_prefill_scores_that_move_the_maximum(course, form, dtype, D):
    new, lens = FORMS[form]
    NH, NKV = (16, 8) if form == "several rounds" else (4, 2)
    if form == "several rounds":
        assert pairs_of(new, NH, NKV) * 2 > sms()
    p = Held(len(course) + D, lens, NKV, D, 16, dtype, wide=0 if form == "warp products" else 1)
    for k in p.keys:
        j = torch.arange(k.shape[0], device="cuda", dtype=torch.float32)[:, None]
        k[..., 0] = {"rising": j * 0.5, "falling": -j * 0.5, "waves": 40 * torch.sin(j * 0.05),
                     "far below": -300 + 0 * j, "far above": 300 + 0 * j}[course]
    p.lay()
    cu = cumulated(new)
    q = p.normal(cu[-1], NH, D, scale=0.5)
    q[..., 0] = 1.0 + torch.arange(NH, device="cuda") % 3       # heads of different slopes
    out, lse = p.cache.prefill(q, ints(cu), ints(lens), scale=0.5, return_lse=True)
    assert p.cache.sync_status() == 0
    p.check_prefill(q, cu, out, lse, scale=0.5)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_scores_of_minus_infinity(form, D):
    """Keys at the type's lowest value, whose scores overflow to -inf: without weight, and a row that sees
    no others gives 0 and -inf."""
    new, lens = FORMS[form]
    NH, NKV = (16, 8) if form == "several rounds" else (4, 2)
    p = Held(D, lens, NKV, D, 16, wide=0 if form == "warp products" else 1)
    low = torch.finfo(torch.bfloat16).min
    for b, k in enumerate(p.keys):
        n = k.shape[0]
        first = n - new[b] + 3                              # the first rows see only such keys in sequence 0
        for j in range(first) if b == 0 else range(0, n, 3):
            k[j] = 0
            k[j, :, 0] = low
    p.lay()
    for k in p.keys:                                        # for the oracle, whose f64 would hold the products
        k[k == low] = -torch.inf
    cu = cumulated(new)
    q = p.normal(cu[-1], NH, D, scale=2.0)
    q[..., 0] = 4.0
    out, lse = p.cache.prefill(q, ints(cu), ints(lens), scale=1.0, return_lse=True)
    assert p.cache.sync_status() == 0
    p.check_prefill(q, cu, out, lse, scale=1.0)
    assert (out[:3] == 0).all() and torch.isneginf(lse[:3]).all() and torch.isfinite(lse[3:]).all()


@pytest.mark.parametrize("above", [7.96875, 8.9375])                # just no move in decode, in prefill
@pytest.mark.parametrize("form", [*FORMS, "decode", "decode in a cluster"])
def test_values_as_large_as_a_lagging_maximum_allows(form, above):
    """The first 64 keys score `above` (log2) below all others, which moves no maximum: weights of up to 2^9 for each
    key meet values of 3.4e38 / (2^9 (keys + 63)), and nothing overflows."""
    new, lens = FORMS.get(form, ([1], [9000 if form == "decode" else 700]))
    if form in ("several rounds", "keys split"):
        lens = [n + 4000 for n in lens]
    NH, NKV, D = (16, 8, 64) if form == "several rounds" else (4, 2, 64)
    p = Held(7, lens, NKV, D, 16, wide=0 if form == "warp products" else 1)
    largest = torch.tensor(3.4e38 / (2.0 ** 9 * (max(lens) + 63))).bfloat16()
    largest = (largest.float() * (1 - 2.0 ** -7)).bfloat16()         # (not above it after its rounding)
    for k, v in zip(p.keys, p.values):
        k.zero_()
        k[64:, :, 0] = above
        v.fill_(largest.item())
        v[:, :, 1] *= -1
    p.lay()
    cu = cumulated(new)
    q = torch.zeros(cu[-1], NH, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    scale = float(np.log(2.0))
    if "decode" in form:
        assert (p.cache.workspace_bytes(1, NH) > 0) == (form == "decode")
        out, lse = p.cache.decode(q, ints(lens), scale=scale, return_lse=True)
        p.check_decode(q, out, lse, scale=scale)
    else:
        out, lse = p.cache.prefill(q, ints(cu), ints(lens), scale=scale, return_lse=True)
        p.check_prefill(q, cu, out, lse, scale=scale)
    assert p.cache.sync_status() == 0


# ---- decode along the line: groups of more than eight heads ---------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("G", [9, 12, 16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("count,NKV", [(1, 1), (24, 2), (160, 2)])   # the join takes single heads; groups; records by CTA
def test_decode_line_and_join_of_large_groups(count, NKV, D, G, dtype):
    rng = np.random.default_rng(count + G)
    lens = [9001] if count == 1 else [int(x) for x in rng.integers(0, 3000, count)]
    lens[-1] = max(lens[-1], 2500)
    p = Held(count + D + G, lens, NKV, D, 64, dtype)
    assert p.cache.workspace_bytes(count, G * NKV) > 0               # the line, not clusters
    q = p.normal(count, G * NKV, D, scale=2.0)
    out, lse = p.cache.decode(q, ints(lens), return_lse=True)
    assert p.cache.sync_status() == 0
    p.check_decode(q, out, lse)
    assert torch.equal(out, p.cache.decode(q, ints(lens)))


def test_a_workspace_shared_by_mistake_leads_out_of_no_buffer():
    """Two calls of different sizes at once on one workspace: their rows may be wrong, all else stays as it was."""
    many, few = Held(1, [int(x) for x in np.random.default_rng(1).integers(2000, 3000, 40)], 2, 64, 64), Held(2, [9001], 1, 64, 64)
    ws = torch.empty(max(many.cache.workspace_bytes(40, 8), few.cache.workspace_bytes(1, 4)), dtype=torch.uint8, device="cuda")
    jobs = []
    for p, NH in ((many, 8), (few, 4)):
        B = len(p.lens)
        q, lens = p.normal(B, NH, 64), ints(p.lens)
        room = torch.full((B + 80, NH, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        jobs.append((p, q, lens, room, room[40:40 + B], stream))
    for _ in range(200):
        for p, q, lens, _, out, stream in jobs:
            p.cache.decode(q, lens, out=out, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for p, q, lens, room, out, _ in jobs:
        B = len(p.lens)
        assert (room[:40] == 7).all() and (room[40 + B:] == 7).all() and p.cache.sync_status() == 0
        out, lse = p.cache.decode(q, lens, workspace=ws, return_lse=True)      # alone: right again
        p.check_decode(q, out, lse)


# ---- weights whose rounding shows ------------------------------------------------------------------------------

def nearly_cancelling(n, dtype, wide=1):
    """A sequence of n keys with values +1 and -1 in equal numbers, whose weights are so close that the sum nearly
    cancels but round to different values of the type: with one term half a step of the weight would remain, A u / 2."""
    D, u = 16, U[dtype]
    p = Held(n, [n], 1, D, 16, dtype, wide=wide)
    k, v = p.keys[0], p.values[0]
    k.zero_()
    v.zero_()
    # every 16th key weighs 1, so that the others weigh 2^-3 (1 + u / 2) and 2^-3 (1 + 3 u / 2) in every block:
    # one term rounds them down and up to multiples of 2 u; a score is the sum of three of the type's values
    j = torch.arange(n, device="cuda")
    for odd, w, sign in ((0, 1 + u / 2, -1.0), (1, 1 + 3 * u / 2, 1.0)):
        at = (j % 16 > 0) & ((j - j // 16) % 2 == odd)
        s = torch.tensor(np.log(w / 8.0), dtype=torch.float64)
        for d in range(3):
            part = s.to(DT[dtype])
            k[at, 0, d] = part.item()
            s = s - part.double()
        v[at, 0] = sign
    p.lay()
    q = torch.zeros(1, 2, D, dtype=DT[dtype], device="cuda")
    q[..., :3] = 1.0
    return p, q


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [101, 9001])                          # in a cluster; along the line
def test_decode_weights_keep_both_terms(n, dtype):
    p, q = nearly_cancelling(n, dtype)
    out, lse = p.cache.decode(q, ints([n]), scale=1.0, return_lse=True)
    p.check(0, q, torch.tensor([n - 1], device="cuda"), out, lse, TWO[dtype], scale=1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,sign", [(101, 1.0), (120, 1.0), (700, -1.0)])   # short; scale < 0 at any length
def test_weights_of_warp_product_prefill_keep_both_terms(n, sign, dtype):
    p, q = nearly_cancelling(n, dtype, wide=0)                       # tables of at most 128 keys: warp products
    assert sign < 0 or p.table_np.shape[1] * p.P <= 128
    q *= sign
    out, lse = p.cache.prefill(q, ints([0, 1]), ints([n]), scale=sign, return_lse=True)
    p.check(0, q, torch.tensor([n - 1], device="cuda"), out, lse, TWO[dtype], scale=sign)


# ---- append: a token's heads in turn -----------------------------------------------------------------------------

@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("NH,NKV,D,n,norm", [
    (16, 8, 128, 1300, True), (14, 2, 64, 4400, True), (5, 1, 128, 5700, True), (4, 2, 16, 40000, True),
    (6, 2, 32, 16000, True), (14, 2, 64, 4400, False), (0, 8, 128, 2500, True),
])
def test_append_with_a_tokens_heads_in_turn(NH, NKV, D, n, norm, dtype, src):
    assert n * (NH + 2 * NKV) * (D // 16) >= 152 * 2048              # items: a full chip of threads
    P = 64
    lens = [n // 2, n - n // 2 - 40]
    p = Held(NH + D, lens, NKV, D, P, dtype)
    seqs = [0] * lens[0] + [1] * lens[1] + [-1] * 40                 # padding at the end
    pos = list(range(lens[0])) + list(range(lens[1])) + [0] * 40
    qkv = (torch.randn(n, NH + 2 * NKV, D, generator=p.g, device="cuda") * 3).to(src)
    ang = torch.arange(max(lens), dtype=torch.float64)[:, None] * (1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D))
    cos, sin = ang.cos().float().cuda(), ang.sin().float().cuda()
    wq, wk = ((1 + 0.1 * torch.randn(D, generator=p.g, device="cuda")).bfloat16() if norm else None for _ in range(2))
    q, k, v = qkv.split((NH, NKV, NKV), 1)
    q_out = torch.full((n, NH, D), 7.0, dtype=DT[dtype], device="cuda")
    p.cache.append(k, v, ints(seqs), ints(pos), cos, sin, q=q if NH else None, q_norm=wq if NH else None, k_norm=wk,
                   eps=1e-5, q_out=q_out if NH else None)
    assert p.cache.sync_status() == 0
    live = n - 40
    at = torch.from_numpy(p.table_np.astype(np.int64)).cuda()[ints(seqs[:live]).long(), ints(pos[:live]).long() // P]
    row = ints(pos[:live]).long() % P
    x = qkv.float().cpu().numpy()
    c, s = cos.cpu().numpy()[pos], sin.cpu().numpy()[pos]
    u = U[dtype]
    for have, part, w in ((q_out[:live], x[:live, :NH], wq), (p.k[at, :, row], x[:live, NH:NH + NKV], wk)):
        have = have.double().cpu().numpy()
        if not norm:
            assert np.array_equal(have, torch.from_numpy(O.norm_rope(part, None, 0, c[:live], s[:live], np.float32))
                                  .to(DT[dtype]).double().numpy())
            continue
        w64 = w.double().cpu().numpy()
        z = O.norm_rope(part, w64, 1e-5, c[:live], s[:live])
        size = np.abs(O.norm_rope(part, w64, 1e-5, np.ones_like(c[:live]), np.zeros_like(s[:live])))
        pair = np.concatenate([size[..., :D // 2] + size[..., D // 2:]] * 2, -1)
        tol = u * np.abs(z) + pair * (1 + u) * (D / 16 + 16) * 2.0 ** -23 + 2.0 ** -25
        assert (np.abs(have - z) <= tol).all()
    assert torch.equal(p.v[at, :, row], v[:live].to(DT[dtype])) and (q_out[live:] == 7).all()
    assert int(p.k.isnan().any(-1).any(1).sum()) == p.n_pages * P - live      # every other row as it was
