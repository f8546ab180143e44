"""GPU parity of the serving calls (packed prompts and single tokens, convolution and scan) against
the float64 oracle, sequence by sequence.

Tolerances.  The convolution's are those of a sum of W + 1 products and a SiLU, about 30 half steps
of fp32 (30 * 2^-24 = 1.8e-6) of the terms' size, here taken against the largest output: 4e-6; bf16
outputs add half a bf16 step, 2^-8, of each value.  The convolution's states are copies: equal.  The
scan's transition exp(delta A) is off by about 2^-21 relative and a state remembers 1 / (1 - a) steps of
it, tens to hundreds here, but at random signs: 1e-5 of the sequence's norm, the bound the training
scan is held to; bf16 outputs add 2^-8."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


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


def host(t):
    return t.detach().cpu().numpy()


def batch(lens, D, N, W, io, seed, slots, pool_slots, pad=3):
    g = torch.Generator().manual_seed(seed)
    dt = DT[io]
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    R = int(off[-1]) + pad

    def rnd(*s):
        return torch.randn(*s, generator=g)
    bc = rnd(R, 2 * N + 8).to(dt).cuda()
    xz = rnd(R, 2 * D).to(dt).cuda()
    return dict(
        x=xz[:, :D], z=xz[:, D:], Bm=bc[:, :N], Cm=bc[:, N:2 * N],
        delta_raw=(torch.rand(R, D, generator=g) * 6 - 7).to(dt).cuda(),
        A_log=torch.log(torch.arange(1, N + 1).float()).repeat(D, 1).cuda() + 0.1 * rnd(D, N).cuda(),
        Dskip=rnd(D).cuda(), w=rnd(D, W).cuda() / 2, bias=rnd(D).cuda() / 2,
        offsets=torch.from_numpy(off).cuda(), slots=torch.tensor(slots, dtype=torch.int32).cuda(),
        carry=(torch.rand(len(lens), generator=g) < 0.5).cuda(),
        cpool=rnd(pool_slots, W - 1, D).to(dt).cuda(), spool=rnd(pool_slots, D, N).cuda())


def close(got, ref, io, what, rel):
    """Norm and largest difference of one sequence."""
    got, ref = f64(got) if torch.is_tensor(got) else got, np.asarray(ref)
    if ref.size == 0:
        return
    h = 2.0 ** -8 if io == "bf16" else 0.0
    n = np.linalg.norm(ref)
    assert np.linalg.norm(got - ref) <= (rel + h) * n + 1e-30, (what, np.linalg.norm(got - ref) / n)
    assert np.all(np.abs(got - ref) <= h * np.abs(ref) + 20 * rel * np.abs(ref).max()), what


def check_prompt(y, pool, ry, rpool, t, io, rel, rel_pool):
    off = host(t["offsets"])
    for s in range(len(off) - 1):
        close(f64(y)[off[s]:off[s + 1]], ry[off[s]:off[s + 1]], io, ("y", s), rel)
    for k in range(len(rpool)):
        close(f64(pool)[k], rpool[k], "f32", ("pool", k), rel_pool)
    assert bool((y[int(off[-1]):] == 7).all())  # rows behind the last sequence


LENS = [([1], 8), ([1, 1, 1, 1, 1], 40), ([0, 2, 0, 3, 0], 24), ([4, 0, 7, 1, 64, 65, 9, 2], 520),
        ([300], 96), ([33, 1000, 5], 136), ([2500], 32), ([128] * 3 + [1], 1544), ([0, 0], 16)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W,silu", [(2, True), (3, False), (4, True)])
@pytest.mark.parametrize("lens,D", LENS)
def test_conv_prompt(S, oracle_mod, lens, D, W, silu, io):
    n = len(lens)
    slots = [(5 * i + 2) % (n + 2) if i % 4 != 3 else -1 for i in range(n)] if (n + 2) % 5 else list(range(n))
    t = batch(lens, D, 4, W, io, n + D, slots, n + 2)
    y = torch.full((t["x"].shape[0], D), 7, dtype=DT[io], device="cuda")
    pool = t["cpool"].clone()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    S.ssm_conv_prompt(t["x"], t["w"], t["bias"], t["offsets"], t["slots"], pool, carry=t["carry"], silu=silu,
                      y=y, ws=ws)
    assert S.ssm_scan_status(ws) == S.SSM_OK
    ry, rpool = oracle_mod.conv_serve(f64(t["x"]), f64(t["w"]), f64(t["bias"]), host(t["offsets"]), slots,
                                      f64(t["cpool"]), host(t["carry"]), silu, y=7.0)
    check_prompt(y, pool, ry, rpool, t, io, 4e-6, 0.0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N", [4, 8, 16])
@pytest.mark.parametrize("gate,zoh", [(True, False), (False, True)])
@pytest.mark.parametrize("lens,D", LENS)
def test_scan_prompt(S, oracle_mod, lens, D, N, gate, zoh, io):
    n = len(lens)
    slots = [n - i if i % 4 != 3 else -1 for i in range(n)]
    t = batch(lens, D, N, 4, io, n + D + N, slots, n + 2)
    y = torch.full((t["x"].shape[0], D), 7, dtype=DT[io], device="cuda")
    z = t["z"] if gate else None
    args = [t[k] for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip", "offsets", "slots")]
    ry, rpool = oracle_mod.scan_serve(*[f64(t[k]) for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")],
                                      host(t["offsets"]), slots, f64(t["spool"]), host(t["carry"]),
                                      None if z is None else f64(z), zoh, y=7.0)
    for max_len in (0, max(max(lens), 1)):
        y.fill_(7)
        pool = t["spool"].clone()
        S.ssm_scan_prompt(*args, pool, carry=t["carry"], z=z, zoh=zoh, max_len=max_len, y=y)
        check_prompt(y, pool, ry, rpool, t, io, 1e-5, 1e-5)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("zoh", [False, True])
@pytest.mark.parametrize("N,D,kind", [(16, 520, "even"), (8, 520, "even"), (4, 520, "even"), (16, 1544, "uneven")])
def test_scan_prompt_on_a_full_gpu(S, oracle_mod, N, D, kind, zoh, io):
    """Batches with many more CTAs than run at once (the form whose SMs are shared), and one of them with
    lengths uneven enough for the longest sequences to be started first."""
    g = torch.Generator().manual_seed(N)
    if kind == "even":
        lens = (torch.randint(1, 65, (110,), generator=g)).tolist()
    else:
        lens = [3, 600, 250] + torch.randint(0, 300, (14,), generator=g).tolist()
    n = len(lens)
    slots = [n - 1 - i if i % 5 else -1 for i in range(n)]
    t = batch(lens, D, N, 4, io, N + D, slots, n)
    y = torch.full((t["x"].shape[0], D), 7, dtype=DT[io], device="cuda")
    args = [t[k] for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip", "offsets", "slots")]
    pool = t["spool"].clone()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    S.ssm_scan_prompt(*args, pool, carry=t["carry"], z=t["z"], zoh=zoh, max_len=max(lens), y=y, ws=ws)
    assert S.ssm_scan_status(ws) == S.SSM_OK
    ry, rpool = oracle_mod.scan_serve(*[f64(t[k]) for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")],
                                      host(t["offsets"]), slots, f64(t["spool"]), host(t["carry"]), f64(t["z"]),
                                      zoh, y=7.0)
    check_prompt(y, pool, ry, rpool, t, io, 1e-5, 1e-5)


@pytest.mark.parametrize("n", [300, 1500, 4096])
def test_prompts_of_many_sequences(S, oracle_mod, n):
    D, N, W = 24, 4, 3
    lens = torch.randint(0, 6, (n,), generator=torch.Generator().manual_seed(n)).tolist()
    slots = torch.randperm(n + 5, generator=torch.Generator().manual_seed(n))[:n].tolist()
    t = batch(lens, D, N, W, "f32", n, slots, n + 5)
    off, cry = host(t["offsets"]), host(t["carry"])
    y = torch.full((t["x"].shape[0], D), 7.0, device="cuda")
    pool = t["cpool"].clone()
    S.ssm_conv_prompt(t["x"], t["w"], t["bias"], t["offsets"], t["slots"], pool, carry=t["carry"], y=y)
    ry, rp = oracle_mod.conv_serve(f64(t["x"]), f64(t["w"]), f64(t["bias"]), off, slots, f64(t["cpool"]), cry, y=7.0)
    assert np.array_equal(f64(pool), rp) and np.abs(f64(y) - ry).max() <= 4e-6 * np.abs(ry).max()
    args = [t[k] for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")]
    y = torch.full_like(y, 7.0)
    pool = t["spool"].clone()
    S.ssm_scan_prompt(*args, t["offsets"], t["slots"], pool, carry=t["carry"], y=y)
    ry, rp = oracle_mod.scan_serve(*[f64(a) for a in args], off, slots, f64(t["spool"]), cry, y=7.0)
    assert np.abs(f64(y) - ry).max() <= 2e-5 * np.abs(ry).max()
    assert np.abs(f64(pool) - rp).max() <= 2e-5 * np.abs(rp).max()


def test_largest_batch_of_single_tokens_that_name_entries(S):
    """4096 rows, entry 17 named by three of them: the first has it."""
    B, D, N = 4096, 64, 16
    slots = torch.randperm(B, generator=torch.Generator().manual_seed(1)).int()
    at = int((slots == 17).nonzero())
    for b in (at + 1, B - 1) if at < B - 2 else (at - 2, at - 1):
        slots[b] = 17
    first = int((slots == 17).nonzero()[0])
    t = batch([1] * B, D, N, 4, "bf16", 2, slots.tolist(), B, pad=0)
    args = [t[k] for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")]
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    for name in ("spool", "cpool"):
        def run(rows, sl, pool, y):
            if name == "spool":
                return S.ssm_scan_step(*rows, sl, pool, y=y, ws=ws)
            return S.ssm_conv_step(rows[0], t["w"], t["bias"], sl, pool, y=y, ws=ws)
        a, b = t[name].clone(), t[name].clone()
        y = torch.full((B, D), 7, dtype=torch.bfloat16, device="cuda")
        run(args, t["slots"], a, y)
        assert S.ssm_scan_status(ws) == 1
        good = [i for i in range(B) if slots[i] != 17 or i == first]
        rows = [x[good] if x.shape[0] == B and x.dim() == 2 and x.shape[1] != N or x is args[3] or x is args[4] else x
                for x in args]
        want = run(rows, t["slots"][good].contiguous(), b, torch.empty(len(good), D, dtype=torch.bfloat16, device="cuda"))
        assert S.ssm_scan_status(ws) == 0
        assert torch.equal(a, b) and torch.equal(y[good], want)
        bad = [i for i in range(B) if i not in set(good)]
        assert len(bad) == 2 and bool((y[bad] == 7).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,W", [(1, 8, 4), (3, 1544, 2), (70, 264, 3), (300, 32, 4), (5, 4096, 4)])
def test_conv_step(S, oracle_mod, B, D, W, io):
    perm = torch.randperm(B + 4, generator=torch.Generator().manual_seed(B)).int()
    slots = perm[:B].tolist()
    if B > 2:
        slots[1] = -1
    t = batch([1] * B, D, 4, W, io, B + D, slots, B + 4, pad=0)
    y = torch.full((B, D), 7, dtype=DT[io], device="cuda")
    pool = t["cpool"].clone()
    S.ssm_conv_step(t["x"], t["w"], t["bias"], t["slots"], pool, y=y)
    live = [b for b in range(B) if slots[b] >= 0]
    ry, rpool = oracle_mod.conv_serve(f64(t["x"])[live], f64(t["w"]), f64(t["bias"]), range(len(live) + 1),
                                      [slots[b] for b in live], f64(t["cpool"]), [1] * B)
    assert np.array_equal(f64(pool), rpool)
    for i, b in enumerate(live):
        close(f64(y)[b], ry[i], io, b, 4e-6)
    if B > 2:
        assert bool((y[1] == 7).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate,zoh", [(True, False), (False, True)])
@pytest.mark.parametrize("B,D,N", [(1, 8, 16), (3, 1544, 4), (70, 264, 8), (300, 32, 16), (37, 4096, 16),
                                   (1201, 16, 4)])
def test_scan_step(S, oracle_mod, B, D, N, gate, zoh, io):
    perm = torch.randperm(B + 4, generator=torch.Generator().manual_seed(B)).int()
    slots = perm[:B].tolist()
    if B > 2:
        slots[1] = -1
    t = batch([1] * B, D, N, 4, io, B + D, slots, B + 4, pad=0)
    y = torch.full((B, D), 7, dtype=DT[io], device="cuda")
    pool = t["spool"].clone()
    z = t["z"] if gate else None
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    args = [t[k] for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")]
    S.ssm_scan_step(*args, t["slots"], pool, z=z, zoh=zoh, y=y, ws=ws)
    assert S.ssm_scan_status(ws) == S.SSM_OK
    live = [b for b in range(B) if slots[b] >= 0]
    rows = [f64(t[k])[live] if t[k].shape[0] == B and k not in ("A_log", "Dskip") else f64(t[k])
            for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")]
    ry, rpool = oracle_mod.scan_serve(*rows, range(len(live) + 1), [slots[b] for b in live], f64(t["spool"]),
                                      [1] * B, None if z is None else f64(z)[live], zoh)
    for i, b in enumerate(live):
        close(f64(y)[b], ry[i], io, b, 1e-5)
        close(f64(pool)[slots[b]], rpool[slots[b]], "f32", b, 1e-5)
    rest = [k for k in range(B + 4) if k not in [slots[b] for b in live]]
    assert torch.equal(pool[rest], t["spool"][rest])
    if B > 2:
        assert bool((y[1] == 7).all())


def test_steps_without_slots_use_the_rows_entry(S):
    t = batch([1] * 5, 64, 16, 4, "f32", 1, list(range(5)), 6, pad=0)
    args = [t[k] for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")]
    a, b = t["spool"].clone(), t["spool"].clone()
    assert torch.equal(S.ssm_scan_step(*args, None, a), S.ssm_scan_step(*args, t["slots"], b))
    assert torch.equal(a, b)
    a, b = t["cpool"].clone(), t["cpool"].clone()
    assert torch.equal(S.ssm_conv_step(t["x"], t["w"], t["bias"], None, a),
                       S.ssm_conv_step(t["x"], t["w"], t["bias"], t["slots"], b))
    assert torch.equal(a, b)
    with pytest.raises(S.SsmError):
        S.ssm_scan_step(*args, None, t["spool"][:4].clone())


def test_bad_slots_and_offsets_are_left_out_and_reported(S, oracle_mod):
    """A repeated entry, an entry past the pool and offsets that run backwards or past the rows: the
    other sequences come out as without them, the bad ones' rows and entries stay, and the status
    word says so."""
    D, N, W = 72, 8, 4
    lens = [5, 40, 3, 200, 7]
    for slots, fix in (([2, 0, 2, 1, 4], None), ([3, 0, 9, 1, 3], None), ([0, 1, 2, 3, 4], 3),
                       ([0, 1, 2, 3, 4], 5)):
        t = batch(lens, D, N, W, "f32", 3, slots, 6)
        off = host(t["offsets"]).copy()
        if fix is not None:
            off[fix] = off[fix - 1] - 2 if fix == 3 else t["x"].shape[0] + 1
            t["offsets"] = torch.from_numpy(off).cuda()
        for conv in (True, False):
            name = "cpool" if conv else "spool"
            pool = t[name].clone()
            y = torch.full((t["x"].shape[0], D), 7.0, device="cuda")
            ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
            if conv:
                S.ssm_conv_prompt(t["x"], t["w"], t["bias"], t["offsets"], t["slots"], pool, y=y, ws=ws)
                ry, rp = oracle_mod.conv_serve(f64(t["x"]), f64(t["w"]), f64(t["bias"]), off, slots, f64(t[name]),
                                               y=7.0)
            else:
                args = [t[k] for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")]
                S.ssm_scan_prompt(*args, t["offsets"], t["slots"], pool, y=y, ws=ws)
                ry, rp = oracle_mod.scan_serve(*[f64(a) for a in args], off, slots, f64(t[name]), y=7.0)
            assert S.ssm_scan_status(ws) == 1
            if fix is None:
                assert np.abs(f64(y) - ry).max() <= 1e-4 and np.abs(f64(pool) - rp).max() <= 1e-4
                assert np.array_equal(f64(y) == 7, ry == 7)
            else:  # the sequences before the first bad offset are whole
                hi = min(off[fix], off[fix - 1])
                assert np.abs(f64(y)[:hi] - ry[:hi]).max() <= 1e-4
                bad = slots[fix - 1]
                assert torch.equal(pool[bad], t[name][bad])


def test_bad_slots_of_single_tokens(S):
    D, N = 520, 16
    slots = [4, 1, 4, 6, -3, 0, 1]
    t = batch([1] * 7, D, N, 4, "bf16", 3, slots, 6, pad=0)
    good = [0, 1, 5]
    args = [t[k] for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")]
    rows = [t[k][good] if k in ("x", "delta_raw", "Bm", "Cm") else t[k]
            for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")]
    gs = t["slots"][good].contiguous()
    for name in ("spool", "cpool"):
        def run(r, sl, pool, **k):
            if name == "spool":
                return S.ssm_scan_step(*r, sl, pool, **k)
            return S.ssm_conv_step(r[0], t["w"], t["bias"], sl, pool, **k)
        a, b = t[name].clone(), t[name].clone()
        ws = torch.empty(256, dtype=torch.uint8, device="cuda")
        y = torch.full((7, D), 7, dtype=torch.bfloat16, device="cuda")
        run(args, t["slots"], a, y=y, ws=ws)
        assert S.ssm_scan_status(ws) == 1
        want = run(rows, gs, b, ws=ws)
        assert S.ssm_scan_status(ws) == 0
        assert torch.equal(a, b) and torch.equal(y[good], want)
        assert bool((y[[2, 3, 4, 6]] == 7).all())


def test_sequences_longer_than_max_len_are_left_out(S):
    t = batch([10, 300, 20], 64, 16, 4, "f32", 3, [0, 1, 2], 3)
    args = [t[k] for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip", "offsets", "slots")]
    a, b = t["spool"].clone(), t["spool"].clone()
    y = torch.full((t["x"].shape[0], 64), 7.0, device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    S.ssm_scan_prompt(*args, a, max_len=100, y=y, ws=ws)
    assert S.ssm_scan_status(ws) == 1
    full = S.ssm_scan_prompt(*args, b, max_len=300, ws=ws)
    assert S.ssm_scan_status(ws) == 0
    assert bool((y[10:310] == 7).all()) and torch.equal(a[1], t["spool"][1])
    assert torch.allclose(y[:10], full[:10], atol=1e-5) and torch.allclose(y[310:330], full[310:330], atol=1e-5)


def test_nonfinite_state_is_reported(S):
    t = batch([5, 6], 64, 16, 4, "f32", 3, [0, 1], 3)
    t["spool"][1, 3, 2] = float("nan")
    args = [t[k] for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    on = torch.ones(2, dtype=torch.bool, device="cuda")
    y = S.ssm_scan_prompt(*args, t["offsets"], t["slots"], t["spool"].clone(), carry=on, ws=ws)
    assert S.ssm_scan_status(ws) == 7
    assert bool(y[5:11, 3].isnan().all()) and int(y[:11].isnan().sum()) == 6
    S.ssm_scan_prompt(*args, t["offsets"], t["slots"], t["spool"].clone(), ws=ws)  # from zero
    assert S.ssm_scan_status(ws) == 0


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("zoh", [False, True])
@pytest.mark.parametrize("N", [4, 8, 16])
def test_decay_rates_past_the_largest_number(S, oracle_mod, N, zoh, io):
    """exp(A_log) past fp32's range: such a state keeps nothing of the step before, in turns that the
    sequence's end leaves partly empty as well, and in single tokens."""
    lens, D = [1, 13, 30, 3], 40
    t = batch(lens, D, N, 4, io, N, [3, 0, 1, 2], 4)
    t["A_log"][3, 2], t["A_log"][8, 0], t["A_log"][39] = 100.0, 89.0, 200.0
    on = torch.ones(4, dtype=torch.bool, device="cuda")
    args = [t[k] for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")]
    n = [f64(a) for a in args]
    for max_len in (0, 30):
        pool, ws = t["spool"].clone(), torch.empty(256, dtype=torch.uint8, device="cuda")
        y = torch.full((t["x"].shape[0], D), 7, dtype=DT[io], device="cuda")
        S.ssm_scan_prompt(*args, t["offsets"], t["slots"], pool, carry=on, zoh=zoh, max_len=max_len, y=y, ws=ws)
        assert S.ssm_scan_status(ws) == S.SSM_OK
        ry, rp = oracle_mod.scan_serve(*n, host(t["offsets"]), [3, 0, 1, 2], f64(t["spool"]), host(on), None, zoh,
                                       y=7.0)
        check_prompt(y, pool, ry, rp, t, io, 1e-5, 1e-5)
    pool = t["spool"].clone()
    rows = [a[:4] if a.shape[0] == t["x"].shape[0] else a for a in args]
    y = S.ssm_scan_step(*rows, t["slots"], pool, zoh=zoh)
    ry, rp = oracle_mod.scan_serve(*[f64(a) for a in rows], np.arange(5, dtype=np.int32), [3, 0, 1, 2],
                                   f64(t["spool"]), np.ones(4, bool), None, zoh)
    close(y, ry, io, "y", 1e-5)
    close(pool, rp, "f32", "pool", 1e-5)


def test_prompt_then_tokens_equal_the_dense_forward(S):
    """A prompt split over three calls and then single tokens, through convolution and scan, give what
    the dense training forward gives for the whole sequence."""
    D, N, W, L = 264, 16, 4, 700
    t = batch([L], D, N, W, "bf16", 9, [2], 4, pad=0)
    xc, _, _ = S.ssm_conv_fwd(t["x"][None], t["w"], t["bias"])
    dr = t["delta_raw"]
    y, _, hL = S.ssm_scan_fwd_ex(xc, dr[None], t["A_log"], t["Bm"][None].contiguous(), t["Cm"][None].contiguous(),
                                 t["Dskip"])
    cpool, spool = t["cpool"].clone(), t["spool"].clone()
    got = []
    for lo, hi in ((0, 2), (2, 600), (600, 690)):
        off = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        carry = torch.tensor([lo > 0], device="cuda")
        r = slice(lo, hi)
        xs = S.ssm_conv_prompt(t["x"][r], t["w"], t["bias"], off, t["slots"], cpool, carry=carry)
        assert torch.equal(xs, xc[0, r])
        got.append(S.ssm_scan_prompt(xs, dr[r], t["A_log"], t["Bm"][r], t["Cm"][r], t["Dskip"], off, t["slots"],
                                     spool, carry=carry))
    for i in range(690, L):
        r = slice(i, i + 1)
        xs = S.ssm_conv_step(t["x"][r], t["w"], t["bias"], t["slots"], cpool)
        assert torch.equal(xs, xc[0, r])
        got.append(S.ssm_scan_step(xs, dr[r], t["A_log"], t["Bm"][r], t["Cm"][r], t["Dskip"], t["slots"], spool))
    got = f64(torch.cat(got))
    close(got, f64(y[0]), "bf16", "y", 2.0 ** -8)  # both are rounded to bf16
    close(f64(spool[2]), f64(hL[0]), "f32", "state", 1e-5)
    keep = [0, 1, 3]
    assert torch.equal(spool[keep], t["spool"][keep]) and torch.equal(cpool[keep], t["cpool"][keep])


def test_training_layer_from_the_8_bit_checkpoint(S, oracle_mod):
    """Convolution, step-size projection, scan and back: only the 8-bit input, the projection's input
    and the scan's checkpoints are kept, the scan's input is restored.  Held to the oracle on the
    restored input at the bf16 pipeline tolerance 2e-2 (three bf16 roundings of 2^-8 in a row)."""
    B, L, D, N, W, R = 2, 200, 128, 16, 4, 16
    g = torch.Generator().manual_seed(12)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    xz = torch.randn(B, L, 2 * D, generator=g).to(**bf)
    x, u = xz[..., :D], torch.randn(B, L, R, generator=g).to(**bf)
    w, bias = torch.randn(D, W, generator=g).cuda() / 2, torch.randn(D, generator=g).cuda() / 2
    pw = (torch.randn(D, R, generator=g) / 8).to(**bf)
    pb = torch.full((D,), -3.0).cuda()
    Bm, Cm, dy = (torch.randn(B, L, k, generator=g).to(**bf) for k in (N, N, D))
    A_log = torch.log(torch.arange(1, N + 1).float()).repeat(D, 1).cuda()
    Dskip = torch.randn(D, generator=g).cuda()
    xc, _, q8 = S.ssm_conv_fwd(x, w, bias, want_q8=True)
    dr = S.ssm_dtproj_fwd(u, pw, pb)
    y, ck = S.ssm_scan_fwd(xc, dr, A_log, Bm, Cm, Dskip)
    del xc
    xr = S.ssm_conv_restore(q8, w, bias)
    gs = S.ssm_scan_bwd(xr, dr, A_log, Bm, Cm, Dskip, ck, dy)
    gp = S.ssm_dtproj_bwd(u, pw, gs["ddelta_raw"])
    dxz = torch.zeros_like(xz)
    gc = S.ssm_conv_bwd(None, w, bias, gs["dx"], q8=q8, out=dict(dx=dxz[..., :D]))
    torch.cuda.synchronize()
    val = oracle_mod.ckpt8(f64(x))[2]
    c = oracle_mod.conv(val, f64(w), f64(bias))
    p = oracle_mod.dtproj(f64(u), f64(pw), f64(pb))
    s = oracle_mod.real(c["y"], p["delta_raw"], f64(A_log), f64(Bm), f64(Cm), f64(Dskip), f64(dy))
    c = oracle_mod.conv(val, f64(w), f64(bias), dy=s["dx"])
    p = oracle_mod.dtproj(f64(u), f64(pw), f64(pb), s["ddelta_raw"])

    def rel(a, b):
        return np.linalg.norm(f64(a) - b) / np.linalg.norm(b)
    assert rel(gc["dx"], c["dx"]) <= 2e-2 and rel(gc["dw"], c["dw"]) <= 2e-2
    assert rel(gc["dbias"], c["dbias"]) <= 2e-2
    assert rel(gs["dA_log"], s["dA_log"]) <= 2e-2 and rel(gp["dw"], p["dw"]) <= 2e-2
    assert not dxz[..., D:].any() and gc["dx"].data_ptr() == dxz.data_ptr()


def test_serving_captured_and_replayed(S):
    """A captured prompt and a captured token, two graphs on two workspaces, replayed on new inputs,
    offsets, slots and padding."""
    D, N, W = 264, 16, 4
    t = batch([40, 1, 200, 7], D, N, W, "bf16", 1, [3, 0, 1, 2], 6)
    names = ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")

    def prompt(p, q):
        xs = S.ssm_conv_prompt(t["x"], t["w"], t["bias"], t["offsets"], t["slots"], q, carry=t["carry"],
                               y=torch.zeros(t["x"].shape[0], D, dtype=torch.bfloat16, device="cuda"))
        return S.ssm_scan_prompt(xs, *[t[k] for k in names[1:]], t["offsets"], t["slots"], p, carry=t["carry"],
                                 z=t["z"], y=torch.zeros_like(xs))

    def token(p, q):
        xs = S.ssm_conv_step(t["x"][:4], t["w"], t["bias"], t["slots"], q, y=t["z"][:4].clone())
        return S.ssm_scan_step(xs, t["delta_raw"][:4], t["A_log"], t["Bm"][:4], t["Cm"][:4], t["Dskip"], t["slots"],
                               p, z=t["z"][:4], y=torch.zeros_like(xs))
    for fn in (prompt, token):
        p, q = t["spool"].clone(), t["cpool"].clone()
        fn(p, q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fn(p, q)
        for lens, slots in (([10, 0, 230, 8], [5, 1, 0, -1]), ([100, 100, 1, 47], [0, 1, 2, 3])):
            n = batch(lens, D, N, W, "bf16", sum(slots), slots, 6)
            for k in ("x", "z", "delta_raw", "Bm", "Cm", "offsets", "slots", "carry"):
                t[k].copy_(n[k])
            p.copy_(n["spool"]), q.copy_(n["cpool"])
            graph.replay()
            p2, q2 = n["spool"].clone(), n["cpool"].clone()
            want = fn(p2, q2)
            assert torch.equal(out, want) and torch.equal(p, p2) and torch.equal(q, q2)


def test_scan_prompt_stays_inside_its_workspace(S):
    t = batch([3000, 17, 0, 900], 64, 16, 4, "f32", 1, [3, 0, 1, 2], 4)
    need = 256
    args = [t[k] for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip", "offsets", "slots")]
    res = []
    for fill in (0x00, 0xFF):
        ws = torch.full((need + 256,), fill, dtype=torch.uint8, device="cuda")
        p = t["spool"].clone()
        y = S.ssm_scan_prompt(*args, p, max_len=3000, ws=ws[:need], y=torch.zeros(t["x"].shape[0], 64, device="cuda"))
        assert bool((ws[need:] == fill).all())
        res.append((y, p))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    with pytest.raises(S.SsmError) as e:
        S.ssm_scan_prompt(*args, t["spool"], max_len=3000, ws=ws[:need - 1])
    assert e.value.code == 4


def test_pool_past_two_to_the_31_elements(S):
    D, N, k = 4096, 16, 2 ** 31 // (4096 * 16) + 5
    big = torch.zeros(k + 1, D, N, device="cuda")
    t = batch([70, 3], D, N, 4, "bf16", 2, [k, 0], 2)
    args = [t[n] for n in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip")]
    small = torch.zeros(2, D, N, device="cuda")
    sl = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    a = S.ssm_scan_prompt(*args, t["offsets"], t["slots"], big)
    b = S.ssm_scan_prompt(*args, t["offsets"], sl, small)
    assert torch.equal(a[:73], b[:73]) and torch.equal(big[k], small[1]) and torch.equal(big[0], small[0])
    row = [x[:2] if x.shape[0] == t["x"].shape[0] else x for x in args]
    a, b = S.ssm_scan_step(*row, t["slots"], big), S.ssm_scan_step(*row, sl, small)
    assert torch.equal(a, b) and torch.equal(big[k], small[1])
    assert not big[1:k].any()


def test_serving_on_another_stream(S):
    t = batch([2000, 5], 128, 16, 4, "bf16", 2, [1, 0], 2)
    args = [t[n] for n in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip", "offsets", "slots")]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    pools = [t["spool"].clone() for _ in range(4)]
    torch.cuda.synchronize()
    ys = [S.ssm_scan_prompt(*args, p, stream=st) for p in pools[:3]]
    st.synchronize()
    want = S.ssm_scan_prompt(*args, pools[3])
    for y, p in zip(ys, pools):
        assert torch.equal(y[:2005], want[:2005]) and torch.equal(p, pools[3])


def test_serving_binding_refusals(S):
    t = batch([3, 2], 64, 16, 4, "bf16", 2, [1, 0], 2)
    a = {k: t[k] for k in ("x", "delta_raw", "A_log", "Bm", "Cm", "Dskip", "offsets", "slots")}
    a["pool"] = t["spool"]
    for change in (dict(pool=t["spool"].bfloat16()), dict(slots=t["slots"].long()), dict(offsets=t["offsets"].cpu()),
                   dict(delta_raw=t["delta_raw"].float()), dict(Bm=t["Bm"][:, :8]), dict(A_log=t["A_log"][:32]),
                   dict(offsets=None), dict(slots=t["slots"][:1]), dict(carry=t["slots"]), dict(z=t["z"][:4]),
                   dict(Dskip=t["Dskip"][:8]), dict(y=torch.empty(8, 128, device="cuda")[:, ::2])):
        with pytest.raises(ValueError):
            S.ssm_scan_prompt(**{**a, **change})
    with pytest.raises(S.SsmError) as e:  # B's columns start off the four-element grid
        S.ssm_scan_prompt(**{**a, "Bm": torch.zeros(8, 18, dtype=torch.bfloat16, device="cuda")[:, 2:]})
    assert e.value.code == 3
    with pytest.raises(ValueError):
        S.ssm_conv_prompt(t["x"], t["w"], t["bias"], t["offsets"], t["slots"], t["cpool"].float())
    with pytest.raises(ValueError):
        S.ssm_conv_step(t["x"], t["w"], t["bias"], t["slots"], t["cpool"])  # a slot a row
