"""Failure detection of the attention to other states, without a fault: a wait that
runs out is reported through na3d_device_status, and the device stays usable.

na3d_cross_selftest_withhold loads one token less of each tile of rows than the
wait for the tile counts: the blocks give up after ~2 s, drain their copies and
products, free their tensor memory and exit. Nothing faults or hangs."""
import ctypes

import pytest
import torch

import block_reference as ref
import neighborhood_attention_video_gb300 as na
from packed_reference import check

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("B,L,S,NH,NKV,HD,docs", [
    (2, 300, 200, 4, 2, 64, 0),       # two row tiles to a block and one
    (2, 300, 200, 4, 2, 64, 2),
    (1, 1, 3000, 16, 4, 128, 0),      # states split over blocks, one row tile in turns
    (2, 1400, 300, 16, 16, 128, 0),   # not split
    (1, 700, 90, 3, 1, 16, 2),
], ids=str)
def test_withheld_token_is_reported_and_the_device_stays_usable(B, L, S, NH, NKV, HD, docs):
    gen = torch.Generator().manual_seed(1)
    q = (torch.randn((B, 1, 1, L, NH, HD), generator=gen) * HD ** -0.5).to(BF16)
    k, v = (torch.randn((B, S, NKV, HD), generator=gen).to(BF16) for _ in range(2))
    g = torch.randn(q.shape, generator=gen).to(BF16)
    doc = (torch.arange(L) * docs // L).expand(B, 1, 1, L).to(torch.int32).contiguous() if docs else None
    kv_doc = (torch.arange(S) * docs // S).expand(B, S).to(torch.int32).contiguous() if docs else None
    want = ref.cross(q, k, v, doc, kv_doc, g)
    q, k, v, g = (x.cuda() for x in (q, k, v, g))
    doc, kv_doc = (x.cuda() if docs else None for x in (doc, kv_doc))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:5], device="cuda")
    grads = [torch.empty_like(x) for x in (q, k, v)]
    need = max(na.na3d_cross_workspace(B, L, S, NH, NKV, HD, b) for b in (False, True))
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    lib, stream = na.load_library(), torch.cuda.current_stream().cuda_stream
    at = lambda x: ctypes.c_void_p(x.data_ptr() if x is not None else None)  # noqa: E731

    def withheld(dout):
        return lib.na3d_cross_selftest_withhold(*(at(x) for x in (q, k, v, out, lse, dout, *grads, work)), B, L, S, NH, NKV, HD,
                                                at(doc), at(kv_doc), ctypes.c_void_p(stream))

    def right():
        na.na3d_cross_fwd(q, k, v, out, lse, doc, kv_doc, work=work)
        na.na3d_cross_bwd(q, k, v, out, lse, g, *grads, doc, kv_doc, work=work)
        assert na.na3d_device_status() == 0
        for name, x in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
            check(name, x, want[name])

    assert na.na3d_device_status() == 0
    assert withheld(None) == 0
    assert na.na3d_device_status() == 10          # NA3D_ERR_DEVICE_TIMEOUT, flag cleared
    assert na.na3d_device_status() == 0
    right()
    assert withheld(g) == 0
    assert na.na3d_device_status() == 10
    assert na.na3d_device_status() == 0
    right()
