"""Gradients of the attention to other states where their value is known, or
known better than the bounds that hold for every token: one state to a token, and
documents whose states lie in one aligned run of 64."""
import pytest
import torch

import block_reference as ref
import neighborhood_attention_video_gb300 as na

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64


def make(shape, S, NKV, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    q = (torch.randn(shape, generator=gen) * scale * shape[5] ** -0.5).to(BF16)
    kv = torch.randn((shape[0], S, 2, NKV, shape[5]), generator=gen).to(BF16)
    return q, kv, torch.randn(shape, generator=gen).to(BF16)


def run(q, kv, g, doc=None, kv_doc=None):
    q, kv, g, doc, kv_doc = (None if x is None else x.cuda() for x in (q, kv, g, doc, kv_doc))
    k, v = kv.unbind(2)
    out, lse = na.na3d_cross_attention(q, k, v, doc=doc, kv_doc=kv_doc, return_lse=True)
    dq, dkv = torch.full_like(q, float("nan")), torch.full_like(kv, float("nan"))
    na.na3d_cross_bwd(q, k, v, out, lse, g, dq, *dkv.unbind(2), doc=doc, kv_doc=kv_doc)
    torch.cuda.synchronize()
    assert na.na3d_device_status() == 0
    return dict(out=out, lse=lse, dq=dq, dk=dkv[:, :, 0], dv=dkv[:, :, 1])


@pytest.mark.parametrize("scale", [1.0, 10.0, 100.0])
@pytest.mark.parametrize("shape,NKV", [((1, 1, 1, 1, 1, 16), 1), ((2, 3, 7, 11, 6, 32), 3), ((1, 4, 12, 13, 4, 64), 4),
                                       ((3, 2, 5, 29, 4, 128), 2), ((1, 1, 8, 40, 5, 128), 1)], ids=str)
def test_one_state_has_no_slope(shape, NKV, scale):
    """p is 1 whatever q and k are: dq and dk are 0, out is the state's value."""
    q, kv, g = make(shape, 1, NKV, 1, scale)
    got = run(q, kv, g)
    assert not got["dq"].any() and not got["dk"].any()
    want = kv[:, 0, 1].repeat_interleave(shape[4] // NKV, 1)[:, None, None, None]
    assert torch.equal(got["out"].cpu(), want.expand(shape))


@pytest.mark.parametrize("HD", [16, 32, 64, 128])
@pytest.mark.parametrize("B,L,S,NH,NKV", [
    (1, 700, 600, 4, 4),       # the pass of dq with few row tiles: the states split over blocks
    (2, 9, 512, 6, 2),
    (1, 1, 1, 3, 1),
    (4, 1280, 300, 10, 10),    # ... and with many: not split
], ids=str)
@pytest.mark.parametrize("scale", [1.0, 100.0])
def test_one_state_a_document_has_no_slope(B, L, S, NH, NKV, HD, scale):
    """The same where each document has one state among other documents' and padding,
    anywhere in the list, and other documents have several."""
    q, kv, g = make((B, 1, 1, L, NH, HD), S, NKV, 2, scale)
    docs = min(5, S)
    gen = torch.Generator().manual_seed(3)
    doc = torch.randint(0, docs + 1, (B, 1, 1, L), generator=gen).to(torch.int32)
    kv_doc = torch.where(torch.arange(S).expand(B, S) % 3 == 0, -1, docs).to(torch.int32)   # document `docs`: many states
    for b in range(B):
        kv_doc[b, torch.randperm(S, generator=gen)[:docs]] = torch.arange(docs, dtype=torch.int32)
    got = run(q, kv, g, doc, kv_doc)
    one = (doc < docs).cuda()
    own = ((kv_doc >= 0) & (kv_doc < docs)).cuda()
    assert not got["dq"][one].any() and not got["dk"][own].any()
    if S > 2 * docs and L > 1:
        assert got["dq"][~one].any() and got["dk"][~own].any()


@pytest.mark.parametrize("n", [2, 7, 40, 64])
@pytest.mark.parametrize("HD", [16, 64, 128])
@pytest.mark.parametrize("B,L,NH,pad", [
    (1, 300, 2, 448),     # the states split over blocks
    (2, 1500, 10, 448),   # not split
    (1, 260, 2, 0),       # one tile of states
], ids=str)
def test_short_documents_take_delta_from_the_sum(B, L, NH, HD, n, pad):
    """States within one run of 64: dq is off by its own rounding and little else.
    Its one rounding has some variance; ds in one bf16 part, or a delta from the rounded
    out, would each bring about as much again (a factor of 1.41): 1.2 leaves 0.44 of it
    for everything else."""
    S = pad + 64
    q, kv, g = make((B, 1, 1, L, NH, HD), S, NH, n)
    kv_doc = torch.full((B, S), -1, dtype=torch.int32)
    at = pad // 2 // 64 * 64
    kv_doc[:, at:at + n] = 0
    got = run(q, kv, g, None, kv_doc)
    k, v = (x[:, at:at + n] for x in kv.unbind(2))
    want = ref.cross(q, k, v, dout=g)["dq"][0]
    once = (want.to(BF16).to(F64) - want).norm()
    assert (got["dq"].cpu().to(F64) - want).norm() <= 1.2 * once


@pytest.mark.parametrize("B,L,S,NH,NKV,HD,docs", [(3, 120, 130, 4, 2, 64, 2), (2, 700, 300, 3, 3, 32, 3), (3, 1300, 520, 16, 16, 16, 2),
                                                  (2, 5, 2000, 8, 1, 128, 1)], ids=str)
def test_an_entry_is_the_entry_by_itself(B, L, S, NH, NKV, HD, docs):
    """All five results of an entry of a batch and of the entry alone, which may be shared
    out over blocks otherwise: each within its bound of the same value, so within two of
    one another; of a row that sees nothing, the same."""
    q, kv, g = make((B, 1, 1, L, NH, HD), S, NKV, 16)
    gen = torch.Generator().manual_seed(17)
    doc = torch.randint(-1, docs, (B, 1, 1, L), generator=gen).to(torch.int32)
    kv_doc = torch.randint(-1, docs + 1, (B, S), generator=gen).sort(1).values.to(torch.int32)
    both = run(q, kv, g, doc, kv_doc)
    want = ref.cross(q, kv[:, :, 0], kv[:, :, 1], doc, kv_doc, g)
    for b in range(B):
        one = run(*(x[b:b + 1].contiguous() for x in (q, kv, g, doc, kv_doc)))
        for name, (value, bound) in want.items():
            x, y, off = one[name][0].cpu().to(F64), both[name][b].cpu().to(F64), bound[b]
            unseen = torch.isinf(value[b])
            assert torch.equal(torch.isinf(x), unseen) and torch.equal(torch.isinf(y), unseen), name
            assert ((x - y).abs() <= 2 * off)[~unseen].all(), name


@pytest.mark.parametrize("S", [1, 40, 600])
def test_scores_past_the_range_of_fp32_have_no_gradient(S):
    """Rows whose scores are all -infinity (products past fp32): lse is that, out and the
    gradients are 0, beside rows that are as ever."""
    q, kv, g = make((1, 1, 1, 30, 2, 64), S, 2, 5)
    kv[:, :, 0].abs_().neg_()
    q[:, :, :, ::3] = 2.0 ** 126
    got = run(q, kv, g)
    far = torch.zeros(30, dtype=torch.bool)
    far[::3] = True
    assert torch.isneginf(got["lse"][0, 0, 0, far]).all() and torch.isfinite(got["lse"][0, 0, 0, ~far]).all()
    assert not got["out"][0, 0, 0, far].any() and not got["dq"][0, 0, 0, far].any()
    assert all(torch.isfinite(got[n]).all() for n in ("out", "dq", "dk", "dv"))
