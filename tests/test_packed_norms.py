"""The norm bounds of wide windows: the same values as the elementwise reference,
and narrow enough to tell a gradient that lacks a term."""
import pytest
import torch

import packed_norms as norms
import packed_reference as ref


def make(shape, seed, scale):
    gen = torch.Generator().manual_seed(seed)
    q, k, v, g = (torch.randn(shape, generator=gen) for _ in range(4))
    return [(x * s).to(torch.bfloat16) for x, s in ((q, scale * shape[-1] ** -0.5), (k, 1), (v, 1), (g, 1))]


# (shape, window, scale of the scores, cap, slopes): scores large enough that few keys
# carry a row, so that delta and the cap's derivative weigh in its gradients
WIDE = [
    ((1, 1, 80, 64, 1, 64), (1, 61, 55), 3.0, 0.0, False),
    ((1, 12, 13, 13, 1, 64), (11, 11, 11), 4.0, 4.0, False),
    ((1, 2, 40, 40, 1, 128), (1, 31, 33), 4.0, 3.0, True),
    ((1, 3, 30, 32, 2, 32), (3, 21, 25), 4.0, 5.0, True),
]


def slopes_of(shape, on):
    return 0.05 * torch.tensor([[1.0, 2.0, 3.0]] * shape[4]) if on else None


def test_values_of_the_elementwise_reference():
    shape, kernel = (2, 4, 6, 7, 2, 16), (3, 5, 5)
    q, k, v, g = make(shape, 3, 3.0)
    doc = torch.zeros(shape[:4], dtype=torch.int32)
    doc[:, 2:], doc[..., 6] = 1, -1
    o = dict(softcap=4.0, slopes=slopes_of(shape, True), doc=doc, prefix=torch.tensor([0, 2], dtype=torch.int32))
    want = ref.scored(q, k, v, kernel, dout=g, **o)
    got = norms.scored(q, k, v, g, kernel, **o)
    for name, (value, sq) in got.items():
        assert torch.allclose(value, want[name][0], rtol=1e-12, atol=1e-12), name
        assert bool((sq.sqrt() <= want[name][1] * 1.5 + 1e-12).all()), name


@pytest.mark.parametrize("shape,kernel,scale,softcap,slopes", [WIDE[1], WIDE[3], ((1, 1, 40, 40, 1, 64), (1, 31, 33), 3.0, 0.0, False)],
                         ids=lambda v: str(v).replace(" ", ""))
def test_a_missing_term_does_not_pass(shape, kernel, scale, softcap, slopes):
    q, k, v, g = make(shape, sum(shape), scale)
    o = dict(softcap=softcap, slopes=slopes_of(shape, slopes))
    want = norms.scored(q, k, v, g, kernel, **o)
    for spoilt in (dict(delta_by=0.0), dict(delta_by=0.5)) + ((dict(cap_slope=False),) if softcap else ()):
        got = norms.scored(q, k, v, g, kernel, **o, **spoilt)
        for name in ("dq", "dk"):
            assert norms.excess(got[name][0], want[name]) > 1, (spoilt, name)   # passes up to 1
    # what rounding alone does to the results passes
    for name in want:
        assert norms.excess(want[name][0].to(torch.bfloat16), want[name]) < 0.5, name
