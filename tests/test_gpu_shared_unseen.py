"""What no row of a group sees of its prefix may hold anything: page rows and table entries beyond the longest length of the
group's rows, where `shared` exceeds it (include/ember.h: rows of a page that no query of the call sees, entries of pages that
hold no visible key).  Tolerances as in test_gpu_shared.py."""
import pytest
import torch

from test_gpu_paged import ints
from test_gpu_shared import Shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("NH,NKV,D,P", [(14, 2, 64, 16), (8, 8, 128, 64), (4, 2, 16, 128)])
@pytest.mark.parametrize("extra", [0, 20000])    # each row for itself; the prefixes by themselves
def test_shared_beyond_every_length(NH, NKV, D, P, extra, dtype):
    """`shared` of 0 to 700 keys more than any row has: the pages are NaN there or do not exist, and nothing is raised."""
    groups = [(37, [37, 5, 0, 36]), (130, [130] * 40 + [129, 1]), (1, [1, 1, 1]), (64, [63, 64, 64]), (90, [90, 91, 200])]
    p = Shared(groups, NKV, D, P, dtype, extra_width=extra + 60)
    lens, cu, shared, prefixes = p.args
    q = p.queries(NH)
    more = ints([37 + 1, 130 + 700, 1 + 15, 64 + 64, 90])
    want, wl = p.run(q, return_lse=True)
    p.check(q, want, wl)
    out, lse = p.cache.decode_shared(q, lens, cu, more, prefixes, seqs=p.seqs, return_lse=True)
    assert p.cache.sync_status() == 0
    p.check(q, out, lse)


def test_invalid_rows_see_nothing():
    """A row that is refused for its length brings nothing of the prefix into the others' outputs; rows of padding, and rows
    that are refused for their table row, count with their lengths."""
    p = Shared([(50, [50, 50, 50, 20, 50, 50])], 2, 64, 16, extra_width=6000)
    lens, cu, shared, prefixes = p.args
    q = p.queries(8)
    more = ints([900])
    lens = lens.clone()
    lens[1], lens[4] = 0, 10 ** 6                # 1: padding; 4: longer than the table has room
    seqs = p.seqs.clone()
    seqs[1] = -1
    out = torch.full_like(q, 3.0)
    p.cache.decode_shared(q, lens, cu, more, prefixes, seqs=seqs, out=out)
    assert p.cache.sync_status() == 2
    assert (out[[1, 4]] == 3).all()
    p.check(q, out, None, rows={0, 2, 3, 5})
    lens[1], lens[4], seqs[4] = 50, 49, 10 ** 6  # a table row that does not exist
    out.fill_(3.0)
    p.cache.decode_shared(q, lens, cu, more, prefixes, seqs=seqs, out=out)
    assert p.cache.sync_status() == 1
    assert (out[[1, 4]] == 3).all()
    p.check(q, out, None, rows={0, 2, 3, 5})
