"""Host-side checks of the short convolution and the serving calls: the oracle against independent
arithmetic, the C ABI's refusals (before anything reaches the device), and host models of the kernels'
index arithmetic: the item numbering of a packed batch, its search, and the pieces of the gradient's
walk."""

import ctypes
import os
import shutil

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ---------------------------------------------------------------- oracle
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("B,L,D,W", [(2, 9, 3, 4), (1, 2, 4, 4), (1, 1, 2, 2), (3, 5, 1, 3)])
def test_oracle_conv_against_torch(oracle_mod, B, L, D, W, silu):
    import torch
    rng = np.random.default_rng(L + W)
    a = {k: torch.from_numpy(rng.standard_normal(s)).requires_grad_() for k, s in
         (("x", (B, L, D)), ("w", (D, W)), ("bias", (D,)), ("s0", (B, W - 1, D)))}
    dy, dsL = rng.standard_normal((B, L, D)), rng.standard_normal((B, W - 1, D))
    xp = torch.cat([a["s0"], a["x"]], 1)
    v = torch.nn.functional.conv1d(xp.transpose(1, 2), a["w"][:, None], a["bias"], groups=D).transpose(1, 2)
    y = torch.nn.functional.silu(v) if silu else v
    ((y * torch.from_numpy(dy)).sum() + (xp[:, L:] * torch.from_numpy(dsL)).sum()).backward()
    r = oracle_mod.conv(*[a[k].detach().numpy() for k in ("x", "w", "bias")], silu, a["s0"].detach().numpy(), dy, dsL)
    np.testing.assert_allclose(r["y"], y.detach().numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_array_equal(r["sL"], xp[:, L:].detach().numpy())
    for k in a:
        np.testing.assert_allclose(r["d" + k], a[k].grad.numpy(), rtol=1e-11, atol=1e-12)


def test_oracle_ckpt8_is_within_half_a_step_and_uses_the_range(oracle_mod):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 72)) * np.exp2(rng.integers(-100, 100, (50, 1)))
    x[7] = 0
    q, qe, val = oracle_mod.ckpt8(x)
    for m in range(50):
        for k in range(3):
            g = slice(32 * k, min(72, 32 * k + 32))
            top = np.abs(x[m, g]).max()
            if top == 0:
                assert qe[m, k] == 0 and not val[m, g].any()
                continue
            step = 2.0 ** (int(qe[m, k]) - 127)
            assert np.abs(val[m, g] - x[m, g]).max() <= step / 2
            assert 63 < np.abs(q[m, g].astype(int)).max() <= 127
            np.testing.assert_array_equal(val[m, g], q[m, g] * step)


def test_oracle_serving_splits_a_sequence(oracle_mod):
    """A sequence cut in two, the second part carrying on from the pool, is the whole sequence; a
    repeated entry is left out."""
    rng = np.random.default_rng(1)
    D, N, W = 3, 4, 4
    x, dr, z = (rng.standard_normal((12, D)) for _ in range(3))
    Bm, Cm = rng.standard_normal((2, 12, N))
    A, Ds, w = rng.standard_normal((D, N)) * 0.1, rng.standard_normal(D), rng.standard_normal((D, W))
    pool, cpool = np.zeros((2, D, N)), np.zeros((2, W - 1, D))
    y, p = oracle_mod.scan_serve(x, dr, A, Bm, Cm, Ds, [0, 12], [1], pool, z=z)
    c, cp = oracle_mod.conv_serve(x, w, None, [0, 12], [1], cpool)
    y1, p1 = oracle_mod.scan_serve(x, dr, A, Bm, Cm, Ds, [0, 5], [1], pool, z=z)
    y2, p2 = oracle_mod.scan_serve(x, dr, A, Bm, Cm, Ds, [5, 12, 12], [1, 1], p1, [1, 0], z=z)
    np.testing.assert_allclose(np.r_[y1[:5], y2[5:]], y, rtol=1e-12)
    np.testing.assert_allclose(p2, p, rtol=1e-12)
    c1, cp1 = oracle_mod.conv_serve(x, w, None, [0, 2], [1], cpool)
    c2, cp2 = oracle_mod.conv_serve(x, w, None, [2, 12], [1], cp1, [1])
    np.testing.assert_allclose(np.r_[c1[:2], c2[2:]], c, rtol=1e-12)
    np.testing.assert_array_equal(cp2, cp)


# ---------------------------------------------------------------- the C ABI's refusals
@pytest.fixture(scope="module")
def S():
    if shutil.which("nvcc") is None and not os.path.exists(
            os.path.join(ROOT, "selective_state_space_bwd_b200", "libssm_scan.so")):
        pytest.skip("needs nvcc or a prebuilt libssm_scan.so")
    from selective_state_space_bwd_b200 import build, ssm_scan
    build.build()
    ssm_scan.lib()
    return ssm_scan


P = 1 << 20  # stands for an aligned device address; no call here may get as far as using it


def conv_shape(S, **kw):
    d = dict(batch=2, seqlen=10, dim=64, ldx=0, ldy=0, lddy=0, lddx=0, width=4, io=S.SSM_BF16, flags=1, reserved=0)
    return S.SsmConvShape(**{**d, **kw})


BAD_CONV = [(dict(batch=-1), 1), (dict(seqlen=-1), 1), (dict(dim=0), 1), (dict(reserved=1), 1), (dict(flags=2), 1),
            (dict(width=1), 2), (dict(width=5), 2), (dict(io=2), 2), (dict(batch=65536), 2),
            (dict(seqlen=(1 << 30) + 1), 2), (dict(dim=(1 << 22) + 8), 2), (dict(batch=65535, seqlen=1 << 30), 2),
            (dict(dim=60), 3), (dict(ldx=32), 1), (dict(ldy=68), 3), (dict(lddy=-64), 1), (dict(lddx=1 << 40), 2)]


@pytest.mark.parametrize("change,code", BAD_CONV)
def test_conv_shapes_refused(S, change, code):
    L, s = S.lib(), conv_shape(S, **change)
    assert L.ssm_conv_fwd(s, P, P, P, P, 2 * P, None, None, None, None) == code
    assert L.ssm_conv_restore(s, P, P, P, P, None, 2 * P, None) == code
    assert L.ssm_conv_bwd(s, P, None, None, P, P, None, P, None, 2 * P, P, P, None, P, 1 << 40, None) == code
    assert L.ssm_conv_workspace_bytes(s) == 0


def test_conv_pointers_refused(S):
    L, s = S.lib(), conv_shape(S)
    assert L.ssm_conv_fwd(None, P, P, P, P, P, None, None, None, None) == 1
    base = [P, P, P, P, 2 * P, None, None, None]
    for i, v, code in [(0, None, 1), (0, P + 8, 3), (1, None, 1), (2, P + 4, 3), (3, P + 2, 3), (4, None, 1),
                       (4, P, 1), (5, P + 8, 3), (5, P, 1), (6, P, 1), (7, P, 1)]:
        a = list(base)
        a[i] = v
        assert L.ssm_conv_fwd(s, *a, None) == code, (i, v)
    need = L.ssm_conv_workspace_bytes(s)
    assert need >= 256 and need % 256 == 0
    #       x  q     qe    w  b  s0    dy dsL   dx     dw db ds0   ws n
    base = [P, None, None, P, P, None, P, None, 2 * P, P, P, None, P, need]
    for i, v, code in [(0, None, 1), (1, P, 1), (2, P, 1), (3, None, 1), (6, None, 1), (6, P + 8, 3), (7, P + 8, 3),
                       (8, None, 1), (8, P, 1), (9, None, 1), (10, P + 4, 3), (11, P + 2, 3), (12, None, 1),
                       (12, P + 8, 3), (13, need - 1, 4)]:
        a = list(base)
        a[i] = v
        assert L.ssm_conv_bwd(s, *a, None) == code, (i, v)
    assert L.ssm_conv_restore(s, None, P, P, P, None, P, None) == 1
    assert L.ssm_conv_restore(s, P, P + 4, P, P, None, P, None) == 3


def scan_serve(S, **kw):
    d = dict(rows=10, seqs=2, dim=64, dstate=16, slots=4, max_len=0, ldx=0, lddelta=0, ldz=0, ldb=0, ldc=0, ldy=0,
             io=S.SSM_BF16, discretization=0)
    return S.SsmScanServe(**{**d, **kw})


def conv_serve(S, **kw):
    d = dict(rows=10, seqs=2, dim=64, slots=4, ldx=0, ldy=0, width=4, io=S.SSM_BF16, flags=0, reserved=0)
    return S.SsmConvServe(**{**d, **kw})


COMMON = [(dict(rows=-1), 1), (dict(seqs=-1), 1), (dict(slots=-1), 1), (dict(dim=0), 1), (dict(seqs=65536), 2),
          (dict(rows=(1 << 30) + 1), 2), (dict(slots=(1 << 30) + 1), 2), (dict(io=7), 2), (dict(dim=60), 3),
          (dict(ldx=56), 1), (dict(ldy=68), 3)]


@pytest.mark.parametrize("change,code", COMMON + [(dict(max_len=-1), 1), (dict(discretization=2), 1),
                                                  (dict(dstate=5), 2), (dict(dim=(1 << 20) + 8), 2),
                                                  (dict(ldb=8), 1), (dict(ldc=18), 3), (dict(lddelta=1), 1)])
def test_scan_serve_shapes_refused(S, change, code):
    L, s = S.lib(), scan_serve(S, **change)
    assert L.ssm_scan_prompt(s, *[P] * 7, P, P, P, P, 2 * P, 3 * P, 1 << 40, None) == code
    s = scan_serve(S, **{"seqs": 0, **change})
    assert L.ssm_scan_step(s, *[P] * 7, P, P, 2 * P, None, 0, None) == (1 if change.get("seqs") else code)


@pytest.mark.parametrize("change,code", COMMON + [(dict(width=5), 2), (dict(flags=4), 1), (dict(reserved=1), 1),
                                                  (dict(dim=(1 << 22) + 8), 2)])
def test_conv_serve_shapes_refused(S, change, code):
    L, s = S.lib(), conv_serve(S, **change)
    assert L.ssm_conv_prompt(s, P, P, P, P, P, P, P, 2 * P, None, 0, None) == code
    s = conv_serve(S, **{"seqs": 0, **change})
    assert L.ssm_conv_step(s, P, P, P, P, P, 2 * P, None, 0, None) == (1 if change.get("seqs") else code)


def test_serving_pointers_refused(S):
    L = S.lib()
    s = scan_serve(S)
    need = 256
    #       x  dr A  B  C  D  z  off slot carry pool y      ws     n
    base = [P, P, P, P, P, P, P, P, P, P, P, 2 * P, 3 * P, need]
    for i, v, code in [(0, None, 1), (1, P + 8, 3), (2, None, 1), (3, P + 4, 3), (4, None, 1), (5, P + 8, 3),
                       (6, P + 2, 3), (7, None, 1), (7, P + 2, 3), (8, None, 1), (8, P + 1, 3), (10, None, 1),
                       (11, P, 1), (11, None, 1), (12, None, 1), (12, 3 * P + 8, 3), (13, need - 1, 4)]:
        a = list(base)
        a[i] = v
        assert L.ssm_scan_prompt(s, *a, None) == code, (i, v)
    s = scan_serve(S, seqs=0)
    assert L.ssm_scan_step(s, *[P] * 6, None, None, P, 2 * P, None, 0, None) == 1  # more rows than entries
    assert L.ssm_scan_step(s, *[P] * 6, None, P, P, 2 * P, 3 * P, 255, None) == 4
    assert L.ssm_scan_step(s, *[P] * 6, None, P, P, 2 * P, None, 256, None) == 1
    assert L.ssm_scan_step(scan_serve(S, seqs=0, max_len=3), *[P] * 6, None, P, P, 2 * P, None, 0, None) == 1
    assert L.ssm_scan_step(scan_serve(S, seqs=0, rows=4097, slots=9999), *[P] * 6, None, P, P, 2 * P, None, 0, None) == 2
    assert L.ssm_conv_step(conv_serve(S, seqs=0, rows=4097), P, P, P, P, P, 2 * P, None, 0, None) == 2
    assert L.ssm_scan_prompt(scan_serve(S, seqs=4097), *base, None) == 2
    assert L.ssm_scan_step(scan_serve(S, seqs=0, rows=65536), *[P] * 6, None, P, P, 2 * P, None, 0, None) == 2
    s = conv_serve(S, seqs=0)
    assert L.ssm_conv_step(s, P, P, P, None, P, 2 * P, None, 0, None) == 1
    assert L.ssm_conv_step(s, P, P, P, P, P, P, None, 0, None) == 1  # y on x
    assert L.ssm_conv_prompt(conv_serve(S), P, P, P, None, P, P, P, 2 * P, None, 0, None) == 1


# ---------------------------------------------------------------- host models
def base(off, s, G):
    return off[s] // G + s


def find_seq(off, S, G, item):
    """The device's 32-way search (layer_common.cuh)."""
    lo, hi = 0, S
    while hi - lo > 1:
        step = (hi - lo + 31) // 32
        n = sum(1 for k in range(32) if lo + k * step < hi and base(off, lo + k * step, G) <= item)
        if n == 0:
            break
        lo += (n - 1) * step
        hi = min(hi, lo + step)
    return lo


@pytest.mark.parametrize("seed", range(12))
def test_items_cover_every_row_of_every_sequence_once(seed):
    rng = np.random.default_rng(seed)
    S = int(rng.choice([1, 2, 5, 33, 64, 100, 1100]))
    G = int(rng.choice([8, 13, 32, 64]))
    lens = rng.integers(0, [2, 40, 300][seed % 3], S)
    off = np.concatenate([[int(rng.integers(0, 50))], lens]).cumsum().tolist()
    rows = off[-1] + 5
    seen, first = np.zeros(rows, int), np.zeros(S, int)
    for item in range(rows // G + S):
        s = find_seq(off, S, G, item)
        k = item - base(off, s, G)
        n = off[s + 1] - off[s]
        if k < 0 or not (k == 0 or k * G < n):
            continue
        lo = off[s] + k * G
        seen[lo:min(off[s + 1], lo + G)] += 1
        first[s] += k == 0
    assert (first == 1).all()  # the piece that holds the state, for empty sequences too
    assert (seen[off[0]:off[-1]] == 1).all() and seen.sum() == off[-1] - off[0]


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("L,G", [(1, 1), (2, 2), (3, 2), (16, 16), (17, 9), (70, 16), (64, 64)])
def test_backward_pieces_write_every_gradient_once(L, G, W):
    """The gradient's walk: rows of dx and ds0 written once, every g summed once, and each dx row's W
    gradients inside what its piece has computed."""
    U = 4
    wrote, summed = {}, np.zeros(L, int)
    for t0 in range(0, L, G):
        t1 = min(L, t0 + G)
        tend, lo = min(L, t1 + W - 1), t0 if t0 > 0 else -(W - 1)
        for t in range(t0, t1 + W - 1, U):
            for u in range(U):
                if t + u < t1:
                    summed[t + u] += 1
                r = t + u - (W - 1)
                if r < lo or r >= t1:
                    continue
                wrote[r] = wrote.get(r, 0) + 1
                for k in range(W):  # g of rows r..r+W-1: zero before the start and past the end
                    assert r + k < 0 or r + k >= L or t0 <= r + k < tend
    assert (summed == 1).all() and wrote == {r: 1 for r in range(-(W - 1), L)}


@pytest.mark.parametrize("turns", list(range(0, 20)) + [64, 100])
@pytest.mark.parametrize("W", [4, 8])
@pytest.mark.parametrize("seed", range(3))
def test_warps_hand_the_state_over_without_a_deadlock(turns, W, seed):
    """The prompt scan's ring of warps under random scheduling: one barrier per receiving warp,
    a hand-over is complete when one arrival and one wait have met on it.  Every turn runs once and in
    order, no arrival meets another arrival on its barrier, no slot is written before it was read, and all
    warps come to their end."""
    rng = np.random.default_rng(seed)
    arrived, slot, order = [False] * W, [None] * W, []

    def warp(w):
        for i in range(w, turns, W):
            yield "work"
            if i > 0:
                while not arrived[w]:
                    yield "wait"
                arrived[w] = False
                assert slot[w] == i - 1
                slot[w] = None
            order.append(i)
            yield "chain"
            if i + 1 < turns:
                to = (w + 1) % W
                assert slot[to] is None and not arrived[to]
                slot[to] = i
                yield "stored"
                arrived[to] = True
            yield "output"
    live = {w: warp(w) for w in range(W)}
    idle = 0
    while live:
        w = int(rng.choice(list(live)))
        try:
            idle = idle + 1 if next(live[w]) == "wait" else 0
        except StopIteration:
            del live[w]
            idle = 0
        assert idle < 10000
    assert order == list(range(turns)) and not any(arrived)


def test_ctypes_structs_have_the_header_sizes(S):
    assert ctypes.sizeof(S.SsmConvShape) == 7 * 8 + 4 * 4
    assert ctypes.sizeof(S.SsmConvServe) == 6 * 8 + 4 * 4
    assert ctypes.sizeof(S.SsmScanServe) == 12 * 8 + 2 * 4
