"""GPU parity of the short causal convolution (forward, 8-bit checkpoint, restore, gradient) against the
float64 oracle, element by element.

Tolerances are counted in fp32 half steps, u = 2^-24, from the formula.  v is a sum of W + 1 terms:
|dv| <= (W + 1) u S with S the sum of the terms' magnitudes.  sigmoid comes from exp2 (4 u relative), an
argument v log2 e rounded twice (2 |v| u on its exponential), one addition and a quotient (1 u + 4 u),
so SiLU, whose slope is at most 1.1, is off by 1.1 |dv| + |y| (10 + 2 |v|) u.  dSiLU/dv = s (1 + v (1 -
s)) has a slope of at most 0.5 and, from the same sigmoid and four operations, is off by at most
0.5 |dv| + (14 + 2 |v|) (1 + |v|) u.  Sums over n terms add n u of the sum of magnitudes.  What is
stored in bf16 is off by half a bf16 step more, 2^-8 of the value.  Each bound is doubled once for the
products of these small terms and the intermediate roundings left out.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def S():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from selective_state_space_bwd_b200 import build, ssm_scan
    build.build()
    ssm_scan.lib()
    return ssm_scan


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().double().cpu().numpy()


def make(B, L, D, W, io, seed, state=True, pad=0):
    """x and dy with row stride D + pad."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[io]

    def rnd(*s):
        return torch.randn(*s, generator=g)
    t = dict(x=rnd(B, L, D + pad).to(dt).cuda()[..., :D], dy=rnd(B, L, D + pad).to(dt).cuda()[..., pad:],
             w=(rnd(D, W) / 2).cuda(), bias=rnd(D).cuda() / 2)
    if state:
        t.update(s0=rnd(B, W - 1, D).to(dt).cuda(), dsL=rnd(B, W - 1, D).to(dt).cuda())
    return t


def check(got, ref, tol, what):
    d = np.abs(f64(got) - ref)
    assert got.shape == ref.shape and np.all(np.isfinite(d)), what
    bad = d > tol
    assert not bad.any(), (what, float((d - tol).max()), np.argwhere(bad)[:4].tolist())


def steps(qe, L):
    """The checkpoint's bytes as [B, L, groups]; those past L are zero."""
    qe = qe.cpu().numpy()
    assert not qe[..., L:].any()
    return qe[..., :L].transpose(0, 2, 1)


def half(io, ref):
    return 2.0 ** -8 * np.abs(ref) if io == "bf16" else U * np.abs(ref)


def reference(oracle_mod, n, W, io, silu, dy=None, dsL=None):
    """Oracle results and tolerances for float64 arrays n (x, w, bias, s0)."""
    o = oracle_mod.conv
    a = {k: None if v is None else np.abs(v) for k, v in n.items()}
    v = o(n["x"], n["w"], n["bias"], False, n["s0"])["y"]
    Sv = o(a["x"], a["w"], a["bias"], False, a["s0"])["y"]
    dv = (W + 1) * U * Sv
    r = o(n["x"], n["w"], n["bias"], silu, n["s0"], dy, dsL)
    tol = {"y": 2 * (1.1 * dv + np.abs(r["y"]) * (10 + 2 * np.abs(v)) * U) + half(io, r["y"])}
    if dy is not None:
        ad = np.abs(dy)
        if silu:
            s = 1 / (1 + np.exp(-v))
            g = ad * np.abs(s * (1 + v * (1 - s)))
            dg = ad * (0.5 * dv + (14 + 2 * np.abs(v)) * (1 + np.abs(v)) * U) + U * g
        else:
            g, dg = ad, 0 * ad
        err = o(a["x"], a["w"], a["bias"], False, a["s0"], dg)
        mag = o(a["x"], a["w"], a["bias"], False, a["s0"], g, None if dsL is None else np.abs(dsL))
        rows = dy.shape[0] * dy.shape[1]
        for k in ("dx", "ds0"):
            tol[k] = 2 * (err[k] + (W + 1) * U * mag[k]) + half(io, r[k])
        for k in ("dw", "dbias"):
            tol[k] = 2 * (err[k] + min(rows, 64 + 32 + rows / 64 + 8) * U * mag[k]) + U * np.abs(r[k])
    return r, tol


CASES = [(1, 1, 8, 4, 0), (2, 2, 40, 4, 8), (3, 3, 8, 2, 0), (1, 5, 520, 3, 24), (2, 63, 264, 4, 0),
         (1, 64, 128, 2, 0), (5, 65, 1544, 4, 8), (2, 300, 768, 4, 768), (1, 4099, 104, 4, 0),
         (7, 130, 72, 3, 8), (1, 33, 4096, 4, 0), (300, 3, 16, 4, 0), (1, 9, 1000, 2, 0)]


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D,W,pad", CASES)
def test_conv_forward_and_gradient(S, oracle_mod, B, L, D, W, pad, io, silu):
    t = make(B, L, D, W, io, seed=B + 7 * L + D + W, pad=pad)
    kw = dict(silu=silu, s0=t["s0"])
    y, sL, _ = S.ssm_conv_fwd(t["x"], t["w"], t["bias"], want_sL=True, **kw)
    g = S.ssm_conv_bwd(t["x"], t["w"], t["bias"], t["dy"], dsL=t["dsL"], **kw)
    torch.cuda.synchronize()
    n = {k: f64(t[k]) for k in ("x", "w", "bias", "s0")}
    ref, tol = reference(oracle_mod, n, W, io, silu, f64(t["dy"]), f64(t["dsL"]))
    assert np.array_equal(f64(sL), ref["sL"])
    check(y, ref["y"], tol["y"], "y")
    for k in ("dx", "dw", "dbias", "ds0"):
        check(g[k], ref[k], tol[k], k)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_conv_without_optional_arrays(S, oracle_mod, io):
    B, L, D, W = 2, 77, 136, 4
    t = make(B, L, D, W, io, seed=5, state=False)
    y, sL, q8 = S.ssm_conv_fwd(t["x"], t["w"])
    g = S.ssm_conv_bwd(t["x"], t["w"], None, t["dy"])
    torch.cuda.synchronize()
    assert sL is None and q8 is None and g["dbias"] is None and g["ds0"] is None
    n = dict(x=f64(t["x"]), w=f64(t["w"]), bias=None, s0=None)
    ref, tol = reference(oracle_mod, n, W, io, True, f64(t["dy"]))
    check(y, ref["y"], tol["y"], "y")
    for k in ("dx", "dw"):
        check(g[k], ref[k], tol[k], k)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,L", [(2, 0), (0, 5)])
def test_conv_empty(S, B, L, io):
    D, W = 24, 4
    t = make(B, L, D, W, io, seed=1)
    y, sL, q8 = S.ssm_conv_fwd(t["x"], t["w"], t["bias"], s0=t["s0"], want_sL=True, want_q8=True)
    g = S.ssm_conv_bwd(t["x"], t["w"], t["bias"], t["dy"], s0=t["s0"], dsL=t["dsL"])
    S.ssm_conv_restore(q8, t["w"], t["bias"], s0=t["s0"], dtype=DT[io])
    torch.cuda.synchronize()
    assert y.shape == (B, L, D) and torch.equal(sL, t["s0"]) and torch.equal(g["ds0"], t["dsL"])
    assert not g["dw"].any() and not g["dbias"].any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D,W", [(2, 65, 520, 4), (1, 1, 8, 3), (3, 40, 32, 2), (1, 300, 1544, 4)])
def test_conv_from_the_8_bit_checkpoint(S, oracle_mod, B, L, D, W, io):
    t = make(B, L, D, W, io, seed=L + D, pad=8)
    x = t["x"]
    x[..., :32] *= torch.logspace(-30, 30, L, device="cuda").view(1, L, 1).to(x.dtype)  # every scale
    x[:, L // 2, :8] = 0
    kw = dict(s0=t["s0"])
    y, _, q8 = S.ssm_conv_fwd(x, t["w"], t["bias"], want_q8=True, **kw)
    plain = S.ssm_conv_fwd(x, t["w"], t["bias"], **kw)[0]
    q, qe, val = oracle_mod.ckpt8(f64(x))
    assert torch.equal(y, plain)
    assert np.array_equal(q8[0].cpu().numpy(), q) and np.array_equal(steps(q8[1], L), qe)
    # values of 7 bits times a power of two are bf16 and fp32 numbers: the restored path is the
    # plain path on them, bit for bit
    xr = torch.from_numpy(val).to(DT[io]).cuda()
    assert np.array_equal(f64(xr), val)
    r = S.ssm_conv_restore(q8, t["w"], t["bias"], dtype=DT[io], **kw)
    assert torch.equal(r, S.ssm_conv_fwd(xr, t["w"], t["bias"], **kw)[0])
    g = S.ssm_conv_bwd(None, t["w"], t["bias"], t["dy"], q8=q8, dsL=t["dsL"], **kw)
    h = S.ssm_conv_bwd(xr, t["w"], t["bias"], t["dy"], dsL=t["dsL"], **kw)
    for k in g:
        assert torch.equal(g[k], h[k]), k


def test_8_bit_checkpoint_borders(S, oracle_mod):
    """Groups of zeros, of one subnormal, at the rounding border between 127 and 128 steps, at the
    largest numbers, with an infinity and with a NaN."""
    D = 32 * 8
    x = torch.zeros(1, 1, D)
    x[0, 0, 32] = 2.0 ** -130
    x[0, 0, 64:67] = torch.tensor([127.49, -1.0, 0.5])
    x[0, 0, 96:99] = torch.tensor([127.5, -1.0, 0.5])
    x[0, 0, 128:130] = torch.tensor([3.4e38, -1e30])
    x[0, 0, 160:162] = torch.tensor([float("inf"), 1.0])
    x[0, 0, 192:194] = torch.tensor([1.0, float("nan")])
    x[0, 0, 224:228] = torch.tensor([64.0, 0.5, 1.5, -2.5])
    x = x.cuda()
    w = torch.zeros(D, 2, device="cuda")
    w[:, 1] = 1
    _, _, q8 = S.ssm_conv_fwd(x, w, silu=False, want_q8=True)
    q, qe, val = oracle_mod.ckpt8(f64(x))
    assert np.array_equal(q8[0].cpu().numpy(), q) and np.array_equal(steps(q8[1], 1), qe)
    back = f64(S.ssm_conv_restore(q8, w, silu=False, dtype=torch.float32))
    assert np.array_equal(back, val, equal_nan=True)


def test_conv_gradient_against_differences(S):
    """Central differences of the forward itself, in fp32, along random directions: the loss is
    summed in float64.  With step e the difference quotient is off by e^2 / 6 times a third
    derivative of order one and by the forward's rounding over e."""
    B, L, D, W = 2, 37, 64, 4
    t = make(B, L, D, W, "f32", seed=3)
    g = S.ssm_conv_bwd(t["x"], t["w"], t["bias"], t["dy"], s0=t["s0"], dsL=t["dsL"])

    def loss(d):
        y, sL, _ = S.ssm_conv_fwd(d["x"], d["w"], d["bias"], s0=d["s0"], want_sL=True)
        return float((y.double() * t["dy"].double()).sum() + (sL.double() * t["dsL"].double()).sum())
    gen = torch.Generator(device="cuda").manual_seed(9)
    for k, dk in (("x", "dx"), ("w", "dw"), ("bias", "dbias"), ("s0", "ds0")):
        dirn = torch.randn(t[k].shape, generator=gen, device="cuda")
        dirn /= dirn.norm()
        e = 2.0 ** -4
        base = {n: t[n] for n in ("x", "w", "bias", "s0")}
        num = (loss({**base, k: t[k] + e * dirn}) - loss({**base, k: t[k] - e * dirn})) / (2 * e)
        ana = float((g[dk].double() * dirn.double()).sum())
        # y is off by about 8 u of its size (about 1): over 5000 independent outputs times dy, / e
        noise = 2 * 8 * U * np.sqrt(B * L * D) * 4 / e
        assert abs(num - ana) <= noise + e * e / 6 * 20, (k, num, ana)


def test_conv_is_deterministic_and_stays_inside_its_workspace(S):
    B, L, D, W = 3, 1000, 520, 4
    t = make(B, L, D, W, "bf16", seed=11)
    need = S.conv_workspace_bytes(S.conv_shape(B, L, D, W))
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    a = S.ssm_conv_bwd(t["x"], t["w"], t["bias"], t["dy"], s0=t["s0"], ws=ws)
    assert bool((ws[need:] == 0xA5).all()) and S.ssm_scan_status(ws) == S.SSM_OK
    ws.fill_(0xFF)  # NaN in every float: nothing left by an earlier call may be read
    b = S.ssm_conv_bwd(t["x"], t["w"], t["bias"], t["dy"], s0=t["s0"], ws=ws)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_conv_infinities_stay_where_they_are(S):
    """A NaN reaches the W outputs from its step on and the W gradients up to it, of its channel."""
    B, L, D, W = 1, 40, 16, 4
    t = make(B, L, D, W, "f32", seed=2, state=False)
    t["x"][0, 20, 3] = float("nan")
    y = S.ssm_conv_fwd(t["x"], t["w"], t["bias"])[0]
    g = S.ssm_conv_bwd(t["x"], t["w"], t["bias"], t["dy"])
    bad = torch.zeros(B, L, D, dtype=torch.bool, device="cuda")
    bad[0, 20:20 + W, 3] = True
    assert torch.equal(y.isnan(), bad)
    bad[0, 20 - (W - 1):20 + W, 3] = True
    assert torch.equal(g["dx"].isnan(), bad)
    only = torch.zeros(D, dtype=torch.bool, device="cuda")
    only[3] = True
    assert torch.equal(g["dbias"].isnan(), only) and torch.equal(g["dw"].isnan().any(1), only)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e2, 1e4, 1e7, 1e12])
def test_conv_of_large_preactivations(S, size, io):
    """SiLU far from zero is the identity, or nothing: so are its values and gradients, at any size.  From v =
    100 on 1 - sigmoid is below 1e-40.  A value is W + 1 products with rounded taps, and SiLU's exp2 and
    quotient (2 u), two constants and two products; a gradient W products, the same and dy's own."""
    B, L, D, W = 2, 37, 72, 4
    g = torch.Generator().manual_seed(5)
    x = (size * (1 + torch.rand(B, L, D, generator=g))).to(DT[io]).cuda()
    dy = torch.randn(B, L, D, generator=g).to(DT[io]).cuda()
    w = (0.5 + torch.rand(D, W, generator=g)).cuda() * 2
    s0 = x[:, :W - 1].contiguous()
    xs = torch.cat([s0, x], 1).double()
    y = S.ssm_conv_fwd(x, w, s0=s0)[0]
    v = sum(w[:, j].double() * xs[:, j:j + L] for j in range(W))
    h = 2.0 ** -8 if io == "bf16" else 0.0
    assert bool(((y.double() - v).abs() <= (2 * (W + 1 + 8) * U + h) * v).all())
    r = S.ssm_conv_bwd(x, w, None, dy, s0=s0)
    gp = torch.cat([dy.double(), torch.zeros(B, W - 1, D, dtype=torch.float64, device="cuda")], 1)
    dx = sum(w[:, W - 1 - k].double() * gp[:, k:k + L] for k in range(W))
    mag = sum(w[:, W - 1 - k].double() * gp[:, k:k + L].abs() for k in range(W))
    assert bool(((r["dx"].double() - dx).abs() <= 2 * (W + 8) * U * mag + h * dx.abs()).all())
    for j in range(W):
        d = (dy.double() * xs[:, j:j + L])
        assert bool(((r["dw"][:, j].double() - d.sum((0, 1))).abs() <= 2 * (B * L + 8) * U * d.abs().sum((0, 1))).all())
    q8 = S.ssm_conv_fwd(x, w, s0=s0, want_q8=True)[2]
    assert torch.equal(S.ssm_conv_bwd(None, w, None, dy, s0=s0, q8=q8)["dx"], r["dx"])  # dx does not depend on x here
    down = S.ssm_conv_bwd(-x, w, None, dy, s0=-s0)
    assert not S.ssm_conv_fwd(-x, w, s0=-s0)[0].any() and not down["dx"].any() and not down["dw"].any()


def test_conv_past_two_to_the_31_elements(S):
    B, L, D, W = 1, 2 ** 31 // 4096 + 100, 4096, 4
    x = torch.empty(B, L, D, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    w = torch.randn(D, W, device="cuda") / 2
    y, sL, q8 = S.ssm_conv_fwd(x, w, want_sL=True, want_q8=True)
    tail = S.ssm_conv_fwd(x[:, -50:].contiguous(), w, s0=x[:, -53:-50].contiguous(), want_q8=True)
    assert torch.equal(y[:, -50:], tail[0]) and torch.equal(sL, x[:, -3:])
    assert torch.equal(q8[0][:, -50:], tail[2][0]) and np.array_equal(steps(q8[1], L)[:, -50:], steps(tail[2][1], 50))
    g = S.ssm_conv_bwd(x, w, None, y)
    h = S.ssm_conv_bwd(x[:, -50:].contiguous(), w, None, y[:, -50:].contiguous(),
                       s0=x[:, -53:-50].contiguous())
    assert torch.equal(g["dx"][:, -50:], h["dx"])


def test_conv_on_another_stream(S):
    t = make(2, 500, 512, 4, "bf16", seed=4)
    want = S.ssm_conv_bwd(t["x"], t["w"], t["bias"], t["dy"], s0=t["s0"])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = [S.ssm_conv_bwd(t["x"], t["w"], t["bias"], t["dy"], s0=t["s0"], stream=st) for _ in range(3)]
    st.synchronize()
    for g in got:
        for k in want:
            assert torch.equal(want[k], g[k]), k


def test_conv_captured_and_replayed(S):
    t = make(2, 130, 264, 4, "bf16", seed=6)
    need = S.conv_workspace_bytes(S.conv_shape(2, 130, 264, 4))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step():
        y, sL, q8 = S.ssm_conv_fwd(t["x"], t["w"], t["bias"], s0=t["s0"], want_sL=True, want_q8=True)
        r = S.ssm_conv_restore(q8, t["w"], t["bias"], s0=t["s0"])
        g = S.ssm_conv_bwd(None, t["w"], t["bias"], t["dy"], q8=q8, s0=t["s0"], dsL=t["dsL"], ws=ws)
        return [y, sL, *q8, r, *g.values()]
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (7, 8):
        n = make(2, 130, 264, 4, "bf16", seed=seed)
        for k in t:
            t[k].copy_(n[k])
        graph.replay()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)


def test_conv_binding_refusals(S):
    t = make(2, 10, 64, 4, "bf16", seed=1)
    x, w, b, dy = t["x"], t["w"], t["bias"], t["dy"]
    for args, kw in [((x.float()[0], w, b), {}), ((x, w.bfloat16(), b), {}), ((x, w[:, :3], b), {}),
                     ((x, w, b[:60]), {}), ((x.cpu(), w, b), {}), ((x, w.cpu(), b), {}),
                     ((x.half(), w, b), {}), ((x, w, b), dict(s0=x[:, :2])),
                     ((x.transpose(0, 1), w, b), dict(y=torch.empty_like(x))),
                     ((x[:, :1].expand(2, 10, 64), w, b), {}), ((x[:1, :1].expand(1, 10, 64), w, b), {}),
                     ((x, w, b), dict(q8=(x[0], x[0]))),
                     ((x, w, b), dict(y=torch.empty(2, 10, 64, device="cuda")))]:
        with pytest.raises(ValueError):
            S.ssm_conv_fwd(*args, **kw)
    with pytest.raises(ValueError):
        S.ssm_conv_bwd(None, w, b, dy)
    for args, code in [((x[..., :60].contiguous(), w[:60].contiguous(), None), 3),
                       ((x, torch.zeros(64, 5, device="cuda"), None), 2)]:
        with pytest.raises(S.SsmError) as e:
            S.ssm_conv_fwd(*args)
        assert e.value.code == code
    with pytest.raises(S.SsmError) as e:
        S.ssm_conv_fwd(x, w, b, y=x)
    assert e.value.code == 1
    with pytest.raises(S.SsmError) as e:
        S.ssm_conv_bwd(x, w, b, dy, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 4
