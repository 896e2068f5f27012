"""A block of a video model as it is used: projection, norm and rotation, windowed
attention, norm of q and attention to a prompt, and the gradients back through them."""
import pytest
import torch

import block_reference as ref
import neighborhood_attention_video_gb300 as na
import packed_reference as packed

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64


@pytest.mark.parametrize("HD,dims,inter", [(32, (8, 12, 12), True), (64, (16, 24, 24), False), (128, (44, 42, 42), True)])
def test_forward_and_backward(HD, dims, inter):
    B, T, H, W, NH, C, S, kernel = 1, 4, 6, 9, 2, 64, 45, (3, 3, 5)
    shape = (B, T, H, W, NH, HD)
    gen = torch.Generator().manual_seed(HD)
    rand = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, w = rand(B, T, H, W, C).to(BF16).cuda(), (rand(3 * NH * HD, C) * C ** -0.5).to(BF16).cuda()
    kv = rand(B, S, 2, NH, HD).to(BF16).cuda()
    wq, wk, wc = ((1 + 0.2 * rand(HD)).to(BF16).cuda() for _ in range(3))
    g = rand(*shape).to(BF16).cuda()
    doc = (torch.arange(T) // 2).view(1, T, 1, 1).expand(shape[:4]).to(torch.int32).contiguous().cuda()
    kv_doc = torch.where(torch.arange(S) < 20, 0, torch.where(torch.arange(S) < 40, 1, -1)).to(torch.int32).view(1, S).cuda()

    # forward
    qkv = torch.empty((B, T, H, W, 3, NH, HD), dtype=BF16, device="cuda")
    na.na3d_qkv_proj(x, w, None, qkv, NH, HD)
    q0, k0, v = na.qkv_views(qkv)
    how = dict(q_weight=wq, k_weight=wk, table=na.na3d_rope_table((T, H, W), dims), rope_dims=dims, q_eps=1e-6 / HD,
               q_scale=HD ** -0.5, interleaved=inter)
    q, k = torch.empty(shape, dtype=BF16, device="cuda"), torch.empty(shape, dtype=BF16, device="cuda")
    na.na3d_norm_rope(q0, k0, q, k, **how)
    mid, lse = na.na3d_scored_attention(q, k, v, kernel, doc=doc, return_lse=True)
    qc = torch.empty_like(mid)
    na.na3d_norm_rope(mid, None, qc, None, q_weight=wc, q_scale=HD ** -0.5)
    out, lse_c = na.na3d_cross_attention(qc, kv[:, :, 0], kv[:, :, 1], doc=doc, kv_doc=kv_doc, return_lse=True)

    # backward
    dqc, dkv, dmid, dqkv = torch.empty_like(qc), torch.empty_like(kv), torch.empty_like(mid), torch.empty_like(qkv)
    dwc, dwq, dwk = (torch.empty(HD, device="cuda") for _ in range(3))
    na.na3d_cross_bwd(qc, kv[:, :, 0], kv[:, :, 1], out, lse_c, g, dqc, dkv[:, :, 0], dkv[:, :, 1], doc=doc, kv_doc=kv_doc)
    na.na3d_norm_rope_bwd(mid, None, dqc, None, dmid, None, dq_weight=dwc, q_weight=wc, q_scale=HD ** -0.5)
    dq0, dk0, dv = na.qkv_views(dqkv)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    na.na3d_scored_bwd(q, k, v, mid, lse, dmid, dq, dk, dv, kernel, doc=doc)
    na.na3d_norm_rope_bwd(q0, k0, dq, dk, dq0, dk0, dq_weight=dwq, dk_weight=dwk, **how)
    torch.cuda.synchronize()
    assert na.na3d_device_status() == 0

    # every step against its reference on what the step before it gave
    ang, none = ref.angles((T, H, W), dims), ref.angles((T, H, W), (0, 0, 0))
    wants = {}
    for name, a, wt, eps, sc, d in (("q", q0, wq, 1e-6 / HD, HD ** -0.5, dq), ("k", k0, wk, 1e-6, 1.0, dk)):
        r = ref.norm_rope(a, ang, wt, eps=eps, scale=sc, interleaved=inter, dout=d)
        wants.update({name: r["out"], "d" + name + "0": r["dx"], "dw" + name: r["dw"]})
    r = ref.norm_rope(mid, none, wc, scale=HD ** -0.5, dout=dqc)
    wants.update(qc=r["out"], dmid=r["dx"], dwc=r["dw"])
    r = ref.cross(qc, kv[:, :, 0], kv[:, :, 1], doc, kv_doc, g)
    wants.update(out=r["out"], lse_c=r["lse"], dqc=r["dq"], dkc=r["dk"], dvc=r["dv"])
    r = packed.scored(q, k, v, kernel, doc=doc, dout=dmid)
    wants.update(mid=r["out"], dq=r["dq"], dk=r["dk"], dv=r["dv"])
    got = dict(q=q, k=k, mid=mid, qc=qc, out=out, lse_c=lse_c, dqc=dqc, dkc=dkv[:, :, 0], dvc=dkv[:, :, 1], dmid=dmid, dwc=dwc,
               dq=dq, dk=dk, dv=dv, dq0=dq0, dk0=dk0, dwq=dwq, dwk=dwk)
    assert set(got) == set(wants)
    for name in got:
        packed.check(name, got[name], wants[name])
