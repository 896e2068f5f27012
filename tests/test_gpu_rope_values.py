"""The norm and rotation on values that are not finite."""
import pytest
import torch

import neighborhood_attention_video_gb300 as na

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("shape,dims,inter", [
    ((1, 2, 3, 5, 3, 16), (2, 2, 6), True),
    ((2, 3, 4, 5, 4, 64), (4, 4, 10), True),
    ((2, 3, 4, 5, 4, 64), (6, 10, 16), True),
    ((2, 3, 4, 5, 40, 64), (6, 10, 44), True),
    ((1, 2, 5, 6, 3, 128), (32, 32, 50), True),
    ((1, 2, 3, 4, 2, 512), (0, 0, 2), True),
    ((2, 3, 4, 5, 4, 64), (4, 4, 8), False),
    ((2, 3, 4, 5, 40, 64), (6, 10, 32), False),
    ((1, 2, 5, 6, 3, 128), (32, 32, 48), False),
    ((1, 2, 3, 4, 2, 512), (0, 0, 16), False),
], ids=str)
@pytest.mark.parametrize("fill", [float("inf"), -float("inf"), float("nan")])
def test_values_that_do_not_turn_stay_by_themselves(shape, dims, inter, fill):
    """Without the norm a value behind those that turn reaches no other, forward and
    backward: all but the filled ones keep their bits, and those stay as they are."""
    HD, turned = shape[5], sum(dims)
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(shape, generator=gen).to(BF16).cuda()
    table = na.na3d_rope_table(shape[1:4], dims)
    how = dict(table=table, rope_dims=dims, norm=False, interleaved=inter)

    def both(x):
        out, dx = torch.empty_like(x), torch.empty_like(x)
        out_k, dk = torch.empty_like(x), torch.empty_like(x)
        na.na3d_norm_rope(x, x.clone(), out, out_k, **how)
        na.na3d_norm_rope_bwd(x, x, x, x.clone(), dx, dk, **how)
        return out, dx, out_k, dk

    want = both(x)
    assert torch.equal(want[0][..., turned:], x[..., turned:])
    for step in (1, 2, 3):
        sick = torch.zeros(HD, dtype=torch.bool, device="cuda")
        sick[turned::step] = True
        y = torch.where(sick, torch.tensor(fill, dtype=BF16, device="cuda"), x)
        for got, clean in zip(both(y), want):
            assert torch.equal(got[..., ~sick], clean[..., ~sick])
            assert torch.equal(got[..., sick].view(torch.int16), y[..., sick].view(torch.int16)) or torch.isnan(got[..., sick]).all()


def test_squares_past_the_range_of_their_sum():
    """As documented: a head whose mean square is past fp32 is normed to 0, others are as ever."""
    x = torch.ones((1, 1, 1, 2, 2, 64), dtype=BF16, device="cuda")
    x[..., 0, 0, :] = 2.0 ** 70
    x[..., 0, 1, :] = 2.0 ** 60
    out = torch.empty_like(x)
    na.na3d_norm_rope(x, None, out, None)
    assert not out[0, 0, 0, 0, 0].any() and (out[0, 0, 0, 0, 1] == 1).all() and (out[0, 0, 0, 1] == 1).all()
