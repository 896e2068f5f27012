"""The 64-bit references that the GPU tests hold the packed-batch kernels to:
against the NA3D oracle, against central differences and against cases that
can be said in closed form."""
import numpy as np
import pytest
import torch

import na3d_inputs
import oracle
import packed_reference as ref

F64 = torch.float64


def make(shape, seed=0):
    gen = torch.Generator().manual_seed(seed)
    q, k, v, g = (torch.randn(shape, generator=gen, dtype=F64) for _ in range(4))
    return q * shape[-1] ** -0.5, k, v, g


def options(shape, seed=1, pad=True):
    B, T, H, W, NH, _ = shape
    gen = torch.Generator().manual_seed(seed)
    doc = torch.randint(0, 2, (B, T, 1, 1), generator=gen).expand(B, T, H, W).contiguous().to(torch.int32)
    if pad:
        doc[..., W - 1] = -1
    return dict(softcap=3.0, slopes=torch.rand((NH, 3), generator=gen), doc=doc,
                prefix=torch.arange(B, dtype=torch.int32))


def test_without_options_it_is_the_oracle():
    shape, kernel = (1, 3, 5, 6, 2, 16), (3, 3, 5)
    q, k, v = na3d_inputs.make_qkv(*shape, seed=3)
    want = oracle.na3d_fwd(q, k, v, kernel)
    tq, tk, tv = (torch.from_numpy(na3d_inputs.bf16_bits_to_f64(x)) for x in (q, k, v))
    got = ref.scored(tq, tk, tv, kernel)["out"][0].numpy()
    assert np.abs(got - want).max() < 1e-12


def test_padding_and_masked_rows():
    """Padding's out is 0 and its lse -inf, and neither what it holds nor what
    another document holds reaches a row."""
    shape, kernel = (2, 4, 3, 5, 2, 16), (3, 3, 3)
    q, k, v, g = make(shape)
    opts = options(shape)
    want = ref.scored(q, k, v, kernel, dout=g, **opts)
    pad = opts["doc"] < 0
    assert bool((want["out"][0][pad] == 0).all()) and bool(torch.isneginf(want["lse"][0][pad]).all())
    for x in (q, k, v, g):
        x[pad] = float("nan")
    again = ref.scored(q, k, v, kernel, dout=g, **opts)
    for name in want:
        assert torch.equal(want[name][0], again[name][0]), name


@pytest.mark.parametrize("drop", [None, "softcap", "slopes", "doc", "prefix"])
def test_gradients_are_those_of_differences(drop):
    shape, kernel = (1, 3, 3, 4, 2, 16), (3, 3, 3)
    q, k, v, g = make(shape, 5)
    opts = options(shape)
    if drop:
        opts[drop] = 0.0 if drop == "softcap" else None
    grads = ref.scored(q, k, v, kernel, dout=g, **opts)
    loss = lambda: float((ref.scored(q, k, v, kernel, **opts)["out"][0] * g).sum())  # noqa: E731
    gen, eps = torch.Generator().manual_seed(7), 1e-5
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        for _ in range(6):
            i = tuple(int(torch.randint(0, n, (1,), generator=gen)) for n in shape)
            x[i] += eps
            up = loss()
            x[i] -= 2 * eps
            diff = (up - loss()) / (2 * eps)
            x[i] += eps
            assert abs(diff - float(grads[name][0][i])) < 1e-7, (name, i)


def test_adapter_gradients_are_those_of_differences():
    gen = torch.Generator().manual_seed(2)
    rand = lambda *s: torch.randn(s, generator=gen, dtype=F64)  # noqa: E731
    M, C, N, R, HD = 11, 8, 48, 8, 16
    x, w, b, A, Bm, g = rand(M, C), rand(N, C), rand(N), rand(3, R, C), rand(3, N, R), rand(M, N)
    scaling = torch.tensor([0.5, 2.0, 1.0])
    offsets, adapter = torch.tensor([1, 4, 4, 8, 10]), torch.tensor([1, 0, -1, 1])
    grads = ref.lora(x, w, b, A, Bm, scaling, offsets, adapter, HD, g)
    loss = lambda: float((ref.lora(x, w, b, A, Bm, scaling, offsets, adapter, HD)["qkv"][0] * g).sum())  # noqa: E731
    assert bool((grads["da"][0][2] == 0).all()) and bool((grads["da"][0][0] == 0).all())
    for name, t in (("dx", x), ("da", A), ("db", Bm)):
        for _ in range(8):
            i = tuple(int(torch.randint(0, n, (1,), generator=gen)) for n in t.shape)
            t[i] += 1e-5
            up = loss()
            t[i] -= 2e-5
            diff = (up - loss()) / 2e-5
            t[i] += 1e-5
            assert abs(diff - float(grads[name][0][i])) < 1e-6, (name, i)
