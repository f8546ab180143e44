"""The short causal convolution where its pieces of rows are long: the rings of row copies wrap many times and the
gradient spends most rows on its inner path.  Against the formula in float64 (torch, a slice of the channels at
a time), element by element; from the 8-bit checkpoint bit by bit against the plain path on the restored input.

Bounds as in test_conv_gpu.py, but for dw and dbias, whose sums are chains of additions in fp32: a thread adds
the rows of its piece (512 at most), a CTA its pieces (64 at most), and the last kernel an eighth of the CTAs'
sums and then eight: each addition is off by half a step, 2^-24, of the sum of magnitudes so far."""

import pytest
import torch

from test_conv_gpu import DT, S, U  # noqa: F401

pytestmark = pytest.mark.gpu


def make(B, L, D, W, io, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda")
    dt = DT[io]
    return dict(x=rnd(B, L, D + 8).to(dt)[..., :D], dy=rnd(B, L, D).to(dt), w=rnd(D, W) / 2, bias=rnd(D) / 2,
                s0=rnd(B, W - 1, D).to(dt), dsL=rnd(B, W - 1, D).to(dt))


def inside(got, ref, tol, what):
    d = (got.double() - ref).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((d - tol).max()), bad.nonzero()[:4].tolist())


def check_slice(t, y, g, c, W, io, silu, chain):
    """Channels c of the forward and the gradient."""
    x, s0, dy, dsL = (t[k][..., c].double() for k in ("x", "s0", "dy", "dsL"))
    w, bias = t["w"][c].double(), t["bias"][c].double()
    L = x.shape[1]
    h = 2.0 ** -8 if io == "bf16" else U
    xp = torch.cat([s0, x], 1)
    v, size = bias.expand_as(x).clone(), bias.abs().expand_as(x).clone()
    for j in range(W):
        v += w[:, j] * xp[:, j:j + L]
        size += (w[:, j] * xp[:, j:j + L]).abs()
    dv = (W + 1) * U * size
    del size
    s = torch.sigmoid(v)
    ref = v * s if silu else v
    inside(y[..., c], ref, 2 * (1.1 * dv + ref.abs() * (10 + 2 * v.abs()) * U) + h * ref.abs(), "y")
    del ref
    if silu:
        gv = dy * s * (1 + v * (1 - s))
        dg = dy.abs() * (0.5 * dv + (14 + 2 * v.abs()) * (1 + v.abs()) * U) + U * gv.abs()
    else:
        gv, dg = dy, torch.zeros_like(dy)
    del s, v, dv
    for j in range(W):
        xs = xp[:, j:j + L]
        r = (gv * xs).sum((0, 1))
        tol = 2 * ((dg * xs.abs()).sum((0, 1)) + chain * U * (gv * xs).abs().sum((0, 1))) + U * r.abs()
        inside(g["dw"][c][:, j], r, tol, ("dw", j))
    r = gv.sum((0, 1))
    inside(g["dbias"][c], r, 2 * (dg.sum((0, 1)) + chain * U * gv.abs().sum((0, 1))) + U * r.abs(), "dbias")
    dxp, mag, err = (torch.zeros_like(xp) for _ in range(3))
    dxp[:, L:], mag[:, L:] = dsL, dsL.abs()
    for j in range(W):
        dxp[:, j:j + L] += w[:, j] * gv
        mag[:, j:j + L] += (w[:, j] * gv).abs()
        err[:, j:j + L] += w[:, j].abs() * dg
    tol = 2 * (err + (W + 1) * U * mag) + h * dxp.abs()
    inside(g["dx"][..., c], dxp[:, W - 1:], tol[:, W - 1:], "dx")
    inside(g["ds0"][..., c], dxp[:, :W - 1], tol[:, :W - 1], "ds0")


def eight_bits(x):
    """The values of the 8-bit checkpoint of x [B,L,D], from its definition, in x's type."""
    out = torch.empty(x.shape, dtype=x.dtype, device="cuda")
    for k in range(0, x.shape[-1], 32):
        g = x[..., k:k + 32].double()
        top = g.abs().amax(-1, keepdim=True)
        step = torch.exp2(torch.floor(torch.log2(top)) - 6)
        step = torch.where(top >= 127.5 * step, 2 * step, step)
        out[..., k:k + 32] = torch.where(top > 0, torch.round(g / step) * step, 0)
    return out


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D,W,silu", [(2, 2051, 4096, 4, True), (16, 1021, 1536, 3, True),
                                          (40, 517, 1544, 2, False), (9000, 301, 24, 4, True),
                                          (18, 2051, 4096, 4, True)])
def test_conv_of_long_pieces(S, B, L, D, W, silu, io):  # noqa: F811
    t = make(B, L, D, W, io, seed=L + D)
    parts = (S.conv_workspace_bytes(S.conv_shape(B, L, D, W, io=S.SSM_F32 if io == "f32" else S.SSM_BF16)) - 256) // (
        (W + 1) * D * 4)
    assert parts <= 1250
    chain = min(L, 512) + 64 + parts // 8 + 9
    kw = dict(silu=silu, s0=t["s0"])
    y, sL, q8 = S.ssm_conv_fwd(t["x"], t["w"], t["bias"], want_sL=True, want_q8=True, **kw)
    assert torch.equal(sL, t["x"][:, L - (W - 1):])
    assert torch.equal(S.ssm_conv_fwd(t["x"], t["w"], t["bias"], **kw)[0], y)
    g = S.ssm_conv_bwd(t["x"], t["w"], t["bias"], t["dy"], dsL=t["dsL"], **kw)
    wide = max(8, (1 << 25) // (B * L) // 8 * 8)
    for c0 in range(0, D, wide):
        check_slice(t, y, g, slice(c0, min(D, c0 + wide)), W, io, silu, chain)
    del y, g
    xr = eight_bits(t["x"])
    yr = S.ssm_conv_fwd(xr, t["w"], t["bias"], **kw)[0]
    assert torch.equal(S.ssm_conv_restore(q8, t["w"], t["bias"], dtype=DT[io], **kw), yr)
    g = S.ssm_conv_bwd(xr, t["w"], t["bias"], t["dy"], dsL=t["dsL"], **kw)
    g8 = S.ssm_conv_bwd(None, t["w"], t["bias"], t["dy"], q8=q8, dsL=t["dsL"], **kw)
    for k in g:
        assert torch.equal(g[k], g8[k]), k


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W,silu", [(2, True), (3, False), (4, True)])
def test_conv_prompts_of_long_pieces(S, W, silu, io):  # noqa: F811
    """Packed documents on 4096 channels: bit for bit each one's own forward, whose values the test above holds."""
    D = 4096
    lens = [3001, 0, 5003, 1, 2500, 2, 1777]
    t = make(1, sum(lens) + 5, D, W, io, seed=W)
    x = t["x"][0]
    off = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int().cuda()
    slots = torch.tensor([6, 0, 3, 8, -1, 2, 5], dtype=torch.int32, device="cuda")
    carry = torch.tensor([1, 1, 0, 1, 1, 1, 0], dtype=torch.uint8, device="cuda")
    pool = torch.randn(9, W - 1, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(DT[io])
    before, want = pool.clone(), pool.clone()
    y = torch.full((x.shape[0], D), 7, dtype=DT[io], device="cuda")
    S.ssm_conv_prompt(x, t["w"], t["bias"], off, slots, pool, carry=carry, silu=silu, y=y)
    lo = 0
    for s, n in enumerate(lens):
        k = int(slots[s])
        s0 = before[k][None].clone() if carry[s] and k >= 0 else torch.zeros(1, W - 1, D, dtype=DT[io], device="cuda")
        yr, sL, _ = S.ssm_conv_fwd(x[None, lo:lo + n], t["w"], t["bias"], silu=silu, s0=s0, want_sL=True)
        assert torch.equal(y[lo:lo + n], yr[0]), s
        if k >= 0:
            want[k] = sL[0]
        lo += n
    assert torch.equal(pool, want) and bool((y[lo:] == 7).all())
