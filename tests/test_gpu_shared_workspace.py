"""What decode_shared's workspace takes: room for the rows that there are, however many groups they stand in.  A partial of a row
of NH heads is NH (D + 2) f32; a row has one of its prefix's and one of its own keys, and a CTA may leave one of a pair of row tiles
(256 rows of heads) and one of 16 heads for each of its warps beside them."""
import pytest
import torch

from test_gpu_shared import Shared

pytestmark = pytest.mark.gpu


def bound(B, NH, D, n_groups):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ctas = sms * 256 + 3 * sms * 4 * 16
    return 4 * ((2 * B * NH + ctas) * (D + 2) + 4 * B * NH + 2 * n_groups + 64)


@pytest.mark.parametrize("NH,NKV,D", [(32, 8, 128), (14, 2, 64), (8, 8, 128), (16, 1, 64), (4, 2, 16)])
@pytest.mark.parametrize("B,n_groups", [(64, 1), (64, 21), (4096, 1), (4096, 1365), (65535, 21845)])
def test_it_goes_by_the_rows(B, n_groups, NH, NKV, D):
    from gqa_transformer_decode_gb300 import runtime
    pages = torch.zeros(2, NKV, 16, D, dtype=torch.bfloat16, device="cuda")
    width = max(1, min(20000, 2 ** 30 // (B * NKV)))
    cache = runtime.PagedKV(pages, pages.clone(), torch.zeros(1, width, dtype=torch.int32, device="cuda"))
    got = cache.shared_workspace_bytes(B, NH, n_groups)
    # (calls that read each row's keys for itself have decode's workspace, also for scales that are not positive)
    assert 0 <= got <= max(bound(B, NH, D, n_groups), cache.workspace_bytes(B, NH))


@pytest.mark.parametrize("NH,NKV,D,n_groups,extra", [(32, 8, 128, 341, 400), (14, 2, 64, 100, 3000), (6, 2, 32, 70, 3000), (16, 1, 64, 40, 6000)])
def test_partials_of_many_groups_stand_apart(NH, NKV, D, n_groups, extra):
    """Groups of three rows and some of none, one and hundreds, each on a prefix of its own, in a workspace of exactly what is
    asked for; what lies behind it stays as it is."""
    groups = [(40 + 7 * (i % 50), [60 + 7 * (i % 50) + j for j in range((3, 3, 3, 1, 0, 12)[i % 6])]) for i in range(n_groups)]
    groups[n_groups // 2] = (1500, [1500 + j % 40 for j in range(300)])
    p = Shared(groups, NKV, D, 16, extra_width=extra)
    n = len(p.lens)
    assert len(groups) <= n // 3
    q = p.queries(NH)
    size = p.cache.shared_workspace_bytes(n, NH, len(groups))
    ws = torch.full((size + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    out, lse = p.run(q, return_lse=True, workspace=ws[:size])
    p.check(q, out, lse, rows=set(range(0, n, max(1, n // 120))) | {n - 1})
    assert (ws[size:] == 0x5a).all()
    again, lse2 = p.run(q, return_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
