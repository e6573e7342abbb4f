"""What a shared prefix may cost in exactness: nothing.  ember_paged_decode_shared takes a weight of the softmax as the sum of
two values of the cache's type in all of its forms, as ember_paged_decode does, so it is held to the bounds that
test_gpu_paged_forms.py derives for two terms (2^-16 of a weight for bf16, 2^-22 for f16)."""
import pytest
import torch

from oracle import paged as O
from test_gpu_paged_forms import TWO, Held, ints, nearly_cancelling, runtime

pytestmark = pytest.mark.gpu


def shared(p, q, rows, n, scale=1.0, wide=0):
    """`rows` copies of the query on one prefix of all n keys of sequence 0: no keys of their own."""
    table = torch.full((1 + rows, p.table.shape[1] + wide), -1, dtype=torch.int32, device="cuda")
    table[0, :p.table.shape[1]] = p.table[0]
    cache = runtime().PagedKV(p.k, p.v, table)
    out, lse = cache.decode_shared(q.expand(rows, -1, -1).contiguous(), ints([n] * rows), ints([0, rows]), ints([n]), ints([0]),
                                   seqs=ints(list(range(1, rows + 1))), scale=scale, return_lse=True)
    assert cache.sync_status() == 0
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,wide", [(1, 0), (40, 0), (3, 40000), (40, 40000), (200, 40000)])
@pytest.mark.parametrize("n", [101, 3001])
def test_both_terms_of_a_prefixs_weights(n, rows, wide, dtype):
    """Each row for itself (narrow tables, few rows), and the prefix multiplied for its group (tables wide enough)."""
    p, q = nearly_cancelling(n, dtype)
    out, lse = shared(p, q, rows, n, wide=wide)
    for r in {0, rows // 2, rows - 1}:
        p.check(0, q, torch.tensor([n - 1], device="cuda"), out[r:r + 1], lse[r:r + 1], TWO[dtype], scale=1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("NH,NKV,D", [(32, 8, 64), (16, 8, 128), (4, 2, 16)])
def test_as_exact_as_without_sharing(NH, NKV, D, dtype):
    """Norm of the error against 64 bits, of decode_shared and of decode on tables that spell the prefix out, beside that of
    the exact result rounded to the type.  Before its rounding an output is off by some 2^-17 of the norm (weights 2^-17,
    sums and scores less), and the roundings' norm, of n values each anywhere in half a step, varies by about n^-1/2 of
    itself, 1 % for 7680.  With weights of one value it was 1.4 times the bare rounding's."""
    n, rows = 4000, 60
    p = Held(NH + D, [n], NKV, D, 16, dtype)
    q = p.normal(rows, NH, D, scale=1.0)
    want = O.attend_all(q.double(), p.keys[0].double(), p.values[0].double(), torch.full((rows,), n - 1, device="cuda"))[0]
    table = torch.full((1 + rows, p.table.shape[1] + 4000), -1, dtype=torch.int32, device="cuda")
    table[:, :p.table.shape[1]] = p.table[0]
    cache = runtime().PagedKV(p.k, p.v, table)
    lens, seqs = ints([n] * rows), ints(list(range(1, rows + 1)))
    one = cache.decode(q, lens, seqs=seqs)
    two = cache.decode_shared(q, lens, ints([0, rows]), ints([n]), ints([0]), seqs=seqs)
    bare = (want.to(q.dtype).double() - want).norm().item()
    off = [(x.double() - want).norm().item() for x in (one, two)]
    assert max(off) <= 1.05 * bare + 2.0 ** -17 * want.norm().item(), (off, bare)
