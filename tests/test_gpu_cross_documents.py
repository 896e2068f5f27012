"""Documents of the attention to other states over thousands of calls and long
lists: operands arrive in any order, searches take as long as they take."""
import pytest
import torch

import block_reference as ref
import neighborhood_attention_video_gb300 as na
from packed_reference import check

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def make(shape, S, NKV, seed):
    gen = torch.Generator().manual_seed(seed)
    q = (torch.randn(shape, generator=gen) * shape[5] ** -0.5).to(BF16)
    return q, torch.randn((shape[0], S, 2, NKV, shape[5]), generator=gen).to(BF16), torch.randn(shape, generator=gen).to(BF16)


@pytest.mark.parametrize("HD", [16, 64, 128])
@pytest.mark.parametrize("B,L,S,NKV", [
    (5, 300, 1300, 16),    # pairs of row tiles of which every second has one alone: the other's steps come late
    (3, 700, 90, 16),      # one column tile a document
    (200, 5, 40, 1),       # one row tile, units of one column tile and of several in turn
    (40, 7, 700, 5),
], ids=str)
def test_columns_of_other_documents_stay_out_over_many_calls(B, L, S, NKV, HD):
    """Every step has columns of other documents and of padding, which hold NaN: over
    thousands of calls the results of the others keep their bits."""
    q, kv, _ = make((B, 1, 1, L, NKV, HD), S, NKV, 1)
    gen = torch.Generator().manual_seed(2)
    doc = (torch.arange(L) * 3 // L).expand(B, 1, 1, L).to(torch.int32).contiguous()
    kv_doc = torch.randint(-1, 4, (B, S), generator=gen).sort(1).values.to(torch.int32)
    kv_doc[:, ::7] = -1
    kv_doc[1::2, 3 * S // 8:] = 1
    kv[(kv_doc < 0) | (kv_doc > 2)] = float("nan")
    q, kv, doc, kv_doc = (x.cuda() for x in (q, kv, doc, kv_doc))
    k, v = kv.unbind(2)
    first, lse = na.na3d_cross_attention(q, k, v, doc=doc, kv_doc=kv_doc, return_lse=True)
    n = min(B, 2)
    want = ref.cross(q[:n], k[:n], v[:n], doc[:n], kv_doc[:n])
    check("out", first[:n], want["out"])
    check("lse", lse[:n], want["lse"])
    assert torch.isfinite(first).all()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(1500):
        out, other = na.na3d_cross_attention(q, k, v, doc=doc, kv_doc=kv_doc, return_lse=True)
        differ += (out.view(torch.int16) != first.view(torch.int16)).sum() + (other.view(torch.int32) != lse.view(torch.int32)).sum()
    assert int(differ) == 0 and na.na3d_device_status() == 0


def test_a_search_may_take_its_time():
    """256 documents a row tile, most of them without states, in a list of 2^24 states of
    which no part can be left out by its smallest and largest document: the search tells
    nothing for longer than a wait's limit of two seconds, and the call is right."""
    S, L, HD, n = 1 << 24, 77 * 256, 16, 5
    q, end, _ = make((1, 1, 1, L, 1, HD), n, 1, 3)
    kv = torch.zeros((1, S, 2, 1, HD), dtype=BF16, device="cuda")
    kv[:, -n:] = end.cuda()
    kv_doc = ((torch.arange(S // 128, device="cuda", dtype=torch.int32) & 1) << 30).repeat_interleave(128).view(1, S)
    kv_doc[:, -n:] = 256
    doc = (1 + torch.arange(L) % 256).to(torch.int32).view(1, 1, 1, L)
    k, v = kv.unbind(2)
    out, lse = na.na3d_cross_attention(q.cuda(), k, v, doc=doc.cuda(), kv_doc=kv_doc, return_lse=True)
    torch.cuda.synchronize()
    assert na.na3d_device_status() == 0
    want = ref.cross(q, end[:, :, 0], end[:, :, 1], (doc != 256).to(torch.int32))
    check("out", out, want["out"])
    check("lse", lse, want["lse"])


@pytest.mark.parametrize("order", ["sorted", "shuffled", "mixed"])
@pytest.mark.parametrize("B,L,S,NKV,docs", [
    (1, 600, 20000, 2, 300),     # the states split over blocks
    (1, 600, 9300, 20, 300),     # ... in two
    (1, 600, 9000, 26, 300),     # not split
    (2, 5000, 300, 2, 200),      # many tokens to a state's tile
    (1, 257, 70000, 1, 257),
], ids=str)
def test_hundreds_of_documents(B, L, S, NKV, docs, order):
    """Documents one behind another, scattered, and in runs that come in any order; some
    without states, some without tokens."""
    HD = 16
    q, kv, g = make((B, 1, 1, L, NKV, HD), S, NKV, 4)
    gen = torch.Generator().manual_seed(5)
    doc, kv_doc = torch.arange(L) * docs // L, torch.arange(S) * docs // S
    if order == "mixed":
        doc, kv_doc = torch.randperm(docs, generator=gen)[doc], torch.randperm(docs, generator=gen)[kv_doc]
    doc, kv_doc = doc.expand(B, L).clone(), kv_doc.expand(B, S).clone()
    if order == "shuffled":
        doc, kv_doc = (torch.stack([x[b, torch.randperm(x.shape[1], generator=gen)] for b in range(B)]) for x in (doc, kv_doc))
    doc[doc % 17 == 3] = -1
    kv_doc[kv_doc % 13 == 5] = -2 ** 31
    doc, kv_doc = doc.to(torch.int32).view(B, 1, 1, L), kv_doc.to(torch.int32)
    want = ref.cross(q, kv[:, :, 0], kv[:, :, 1], doc, kv_doc, g)
    q, kv, g, doc, kv_doc = (x.cuda() for x in (q, kv, g, doc, kv_doc))
    k, v = kv.unbind(2)
    out, lse = na.na3d_cross_attention(q, k, v, doc=doc, kv_doc=kv_doc, return_lse=True)
    dq, dkv = torch.full_like(q, float("nan")), torch.full_like(kv, float("nan"))
    na.na3d_cross_bwd(q, k, v, out, lse, g, dq, *dkv.unbind(2), doc=doc, kv_doc=kv_doc)
    torch.cuda.synchronize()
    assert na.na3d_device_status() == 0
    got = dict(out=out, lse=lse, dq=dq, dk=dkv[:, :, 0], dv=dkv[:, :, 1])
    for name in want:
        check(name, got[name], want[name])
