"""The convolution up to the largest numbers: pre-activations of 2.3e38 to 3.3e38, which fp32 and bf16 still
hold, in the forward, from the 8-bit checkpoint, in the gradient, in packed prompts and single tokens.

The last tap is one and the others zero, so that the pre-activation is the input itself.  SiLU is then the
identity above zero and nothing below: sigmoid is one or zero to the bit, its argument at most overflows,
and y = v (one product) in fp32 and in bf16.  dx = dy, dbias = sum dy and dw[:, -1] = sum dy x, where dy is
of the order of 2^-30: sums of n terms, off by n half steps of fp32 of the sum of magnitudes (and
again as much for the order of the sums)."""

import pytest
import torch

from test_conv_gpu import DT, S, U  # noqa: F401

pytestmark = pytest.mark.gpu


def rows(B, L, D, io, seed):
    g = torch.Generator().manual_seed(seed)
    x = (2.3e38 + 1.0e38 * torch.rand(B, L, D, generator=g)).to(DT[io]).cuda()
    assert bool(x.isfinite().all()) and float(x.float().max()) > 3e38
    return x, (torch.randn(B, L, D, generator=g) * 2.0 ** -30).to(DT[io]).cuda()


def last_tap(D, W):
    w = torch.zeros(D, W, device="cuda")
    w[:, -1] = 1
    return w


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L,D,W", [(5, 40, 2), (37, 72, 4), (300, 520, 3)])
@pytest.mark.parametrize("sign", [1, -1])
def test_conv_at_the_largest_preactivations(S, L, D, W, io, sign):  # noqa: F811
    x, dy = rows(2, L, D, io, L)
    x, w = sign * x, last_tap(D, W)
    y, _, q8 = S.ssm_conv_fwd(x, w, want_q8=True)
    assert torch.equal(y, x if sign > 0 else torch.zeros_like(x))
    r = S.ssm_conv_restore(q8, w, dtype=x.dtype)
    back = S.ssm_conv_restore(q8, w, silu=False, dtype=x.dtype)
    assert bool(back.isfinite().all())
    assert torch.equal(r, back if sign > 0 else torch.zeros_like(x))
    bias = torch.zeros(D, device="cuda")
    for src, q in ((x, None), (None, q8)):
        g = S.ssm_conv_bwd(src, w, bias, dy, q8=q)
        if sign < 0:
            assert not any(bool(g[k].any()) for k in ("dx", "dw", "dbias"))
            continue
        xs = (x if q is None else back).double()
        assert torch.equal(g["dx"], dy)
        d = dy.double()
        n = 2 * L
        assert bool(((g["dbias"].double() - d.sum((0, 1))).abs() <= 2 * n * U * d.abs().sum((0, 1))).all())
        for j in range(W):
            sh = W - 1 - j
            p = d[:, sh:] * xs[:, :L - sh]
            assert bool(((g["dw"][:, j].double() - p.sum((0, 1))).abs() <= 2 * n * U * p.abs().sum((0, 1))).all()), j


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_taps(S, io, sign):  # noqa: F811
    """The size in the tap, not in the input."""
    B, L, D = 1, 9, 24
    w = torch.zeros(D, 2, device="cuda")
    w[:, 1] = sign * torch.linspace(2.3e38, 3.3e38, D, device="cuda")
    x = torch.ones(B, L, D, dtype=DT[io], device="cuda")
    dy = torch.full_like(x, 2.0 ** -30)
    y = S.ssm_conv_fwd(x, w)[0]
    g = S.ssm_conv_bwd(x, w, None, dy)
    if sign > 0:
        assert torch.equal(y, w[:, 1].to(DT[io]).expand(B, L, D))
        assert torch.equal(g["dx"], (2.0 ** -30 * w[:, 1]).to(DT[io]).expand(B, L, D))
        assert torch.equal(g["dw"][:, 1], torch.full((D,), L * 2.0 ** -30, device="cuda"))
    else:
        assert not y.any() and not g["dx"].any() and not g["dw"].any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
def test_serving_at_the_largest_preactivations(S, io, sign):  # noqa: F811
    D, W = 72, 4
    x = sign * rows(1, 40, D, io, 3)[0][0]
    w, want = last_tap(D, W), x if sign > 0 else torch.zeros_like(x)
    off = torch.tensor([0, 3, 40], dtype=torch.int32, device="cuda")
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    pool = torch.zeros(2, W - 1, D, dtype=DT[io], device="cuda")
    assert torch.equal(S.ssm_conv_prompt(x, w, None, off, slots, pool), want)
    assert torch.equal(S.ssm_conv_step(x[:2].contiguous(), w, None, slots, pool), want[:2])
