"""The operators of a serving step together: projection with each request's adapter, append, attention under shared
prefixes, projection back, logits, log probabilities; against the same step in 64 bits.

Tolerance: every stage of the reference starts from the previous stage's own output, as the library gave it, so each
comparison has its operator's tolerance alone (test_gpu_adapters.py, test_gpu_shared.py, test_gpu_logprobs.py); the
rotated rows that append stores are compared bit for bit with what the kernel before returned as q."""
import numpy as np
import pytest
import torch

from oracle import paged as OP
from oracle import rows as OR
from test_gpu_logprobs import check as check_logprobs
from test_gpu_paged import U, check_rows, ints

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def check_project(y, x, w, a, b, s, ids):
    want, size, low, _ = OR.project(f64(x), f64(w), f64(a), f64(b), f64(s), ids.cpu().numpy())
    K, R = x.shape[1], a.shape[1]
    tol = (K / 16 + R / 8 + 9) * 2.0 ** -22 * (size + 2 * low) + (2.0 ** -23 + 2.0 ** -16) * low
    tol += (np.abs(want) + tol) * (2.0 ** -24 + (0.0 if y.dtype == torch.float32 else 2.0 ** -8))
    assert (np.abs(f64(y) - want) <= tol).all()


@pytest.mark.parametrize("B,shared,graph", [(5, 70, False), (40, 1037, False), (40, 1037, True)])
def test_a_step_of_many_requests(B, shared, graph):
    from gqa_transformer_decode_gb300 import runtime
    NH, NKV, D, H, V, P, R, A = 8, 2, 64, 512, 4099, 16, 16, 6
    g = torch.Generator(device="cuda").manual_seed(B)

    def rand(*s, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*s, generator=g, device="cuda") * scale).to(dtype)
    N = (NH + 2 * NKV) * D
    wqkv, wo, head = rand(N, H, scale=0.05), rand(H, NH * D, scale=0.05), rand(V, H, scale=0.1)
    ad = [(rand(A, R, k, scale=k ** -0.5), rand(A, n, R, scale=0.1), torch.rand(A, generator=g, device="cuda") * 2)
          for n, k in ((N, H), (H, NH * D))]
    qkv_ad, o_ad = (runtime.Adapters(*t) for t in ad)
    ids = torch.randint(-1, A, (B,), generator=g, device="cuda").int()

    # one prefix, held by table row 0; the requests' own rows follow, each a few tokens on
    tails = [(i * 37) % 200 for i in range(B)]
    own = [(shared // P, -(-(shared + t + 1) // P)) for t in tails]
    pages = -(-shared // P) + sum(b - a for a, b in own) + 1
    table = torch.full((B + 1, max(b for _, b in own)), -1, dtype=torch.int32)
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int()
    table[0, :-(-shared // P)] = perm[:-(-shared // P)]
    at = -(-shared // P)
    for i, (a, b) in enumerate(own):
        table[i + 1, a:b] = perm[at:at + b - a]
        at += b - a
    k, v = rand(pages, NKV, P, D), rand(pages, NKV, P, D)
    cache = runtime.PagedKV(k, v, table.cuda())
    pos = [shared + t for t in tails]
    seqs, positions = ints(list(range(1, B + 1))), ints(pos)
    lens, groups, sh, pre = ints([p + 1 for p in pos]), ints([0, B]), ints([shared]), ints([0])
    angle = torch.arange(max(pos) + 1, device="cuda", dtype=torch.float64)[:, None] * 1e4 ** (
        -torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    cos, sin = angle.cos().float(), angle.sin().float()
    given = torch.randint(V, (B,), generator=g, device="cuda").int()
    x = rand(B, H)

    def step():
        qkv = qkv_ad.project(x, wqkv, ids).view(B, NH + 2 * NKV, D)
        q, kk, vv = qkv.split((NH, NKV, NKV), 1)
        q = cache.append(kk, vv, seqs, positions, cos, sin, q=q)
        att = cache.decode_shared(q, lens, groups, sh, pre, seqs=seqs)
        y = o_ad.project(att.view(B, NH * D), wo, ids)
        logits = qkv_ad_free.project(y, head, none, out_dtype=torch.float32)
        return qkv, q, att, y, logits, runtime.logprobs(logits, given, top=7, temperature=0.8)
    # the head has no adapters: a projection whose rows name none
    V8 = -(-V // 8) * 8
    head = torch.cat((head, torch.zeros(V8 - V, H, dtype=torch.bfloat16, device="cuda")))
    qkv_ad_free = runtime.Adapters(rand(1, 8, H), rand(1, V8, 8))
    none = torch.full((B,), -1, dtype=torch.int32, device="cuda")

    out = step()
    if graph:
        x2 = rand(B, H)
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            out = step()
        x.copy_(x2)
        cg.replay()
    qkv, q, att, y, logits, lp = out
    assert qkv_ad.sync_status() == 0 and o_ad.sync_status() == 0 and cache.sync_status() == 0
    check_project(qkv.reshape(B, N), x, wqkv, *ad[0], ids)
    check_project(y, att.reshape(B, NH * D), wo, *ad[1], ids)
    check_project(logits, y, head, rand(1, 8, H), rand(1, V8, 8), torch.ones(1), none)
    for i in range(B):
        row = np.concatenate((table[0, :-(-shared // P)].numpy(), np.zeros(table.shape[1], np.int32)))[:table.shape[1]]
        own_row = table[i + 1].numpy()
        j = torch.arange(pos[i] + 1)
        page = torch.from_numpy(np.where(j.numpy() < shared, row[j // P], own_row[j // P])).long().cuda()
        kv = [t[page, :, (j % P).cuda()].double() for t in (k, v)]
        w = [t.cpu().numpy() for t in OP.attend_all(q[i:i + 1].double(), *kv, torch.tensor([pos[i]], device="cuda"))]
        check_rows(att[i:i + 1], None, w[:3] + [w[3].max()], U["bf16"], U["bf16"], D, pos[i] + 1)
        # the row that append stored: the key as rotated by the oracle in f32, the value as it was
        want = OP.norm_rope(f64(qkv[i:i + 1, NH:NH + NKV]), None, 0.0, cos[pos[i]].cpu().numpy()[None], sin[pos[i]].cpu().numpy()[None],
                            dtype=np.float32)
        assert torch.equal(k[page[-1], :, pos[i] % P], torch.from_numpy(want[0]).to(torch.bfloat16).cuda())
        assert torch.equal(v[page[-1], :, pos[i] % P], qkv[i, NH + NKV:])
    # the padded vocabulary's zeros count as tokens too, as the logits say
    check_logprobs(logits, given, 7, 0.8, lp)
