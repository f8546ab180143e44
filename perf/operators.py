"""Cases and plain forms of the operators around the selective scan: the short causal convolution
(training, with its gradient, from the input itself or from an 8-bit checkpoint of it), the
convolution and the scan over packed prompts with a pool of states, and both for single tokens.

``run`` computes a case in elementary torch operations, or, with ``own`` set, through the library's
calls; ``exact`` computes the same in float64 from the definitions.
"""

import math
import random

import torch
import torch.nn.functional as F

own = False

KINDS = ("conv_train", "conv_prompt", "scan_prompt", "conv_step", "scan_step")
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _ops():
    from selective_state_space_bwd_b200 import ssm_scan
    return ssm_scan


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # A piece of a sequence whose convolution state is carried from piece to piece, fp32.
        dict(name="conv_train_piece", kind="conv_train", batch=1, seqlen=300, dim=768, width=4,
             io="f32", silu=True, state=True, q8=False),
        # The convolution of a 130M-parameter model's layer: batch 8 of 2048 tokens.
        dict(name="conv_train_130m", kind="conv_train", batch=8, seqlen=2048, dim=1536, width=4,
             io="bf16", silu=True, state=False, q8=False),
        # An odd length and width, a width of three taps, from the 8-bit checkpoint.
        dict(name="conv_train8_odd", kind="conv_train", batch=3, seqlen=777, dim=520, width=3,
             io="bf16", silu=True, state=True, q8=True),
        # The convolution of a 1.4B-parameter model's layer on long sequences, where the kept
        # activations are what fills the memory: from the 8-bit checkpoint.
        dict(name="conv_train8_1p4b", kind="conv_train", batch=4, seqlen=8192, dim=4096, width=4,
             io="bf16", silu=True, state=False, q8=True),
        # Many short questions packed in one batch.
        dict(name="conv_prompt_short", kind="conv_prompt", seqs=48, longest=96, lens=1, pad=5,
             dim=1536, width=4, io="bf16", silu=True),
        # A few long documents, some continuing from a kept state.
        dict(name="conv_prompt_long", kind="conv_prompt", seqs=9, longest=6000, lens=2, pad=0,
             dim=4096, width=4, io="bf16", silu=True),
        # One document alone: few channels, all the work along time.
        dict(name="scan_prompt_one", kind="scan_prompt", seqs=1, longest=4096, lens=3, pad=0,
             dim=1536, dstate=16, io="bf16", gate=True, zoh=False),
        # A ragged batch of documents of a 1.4B-parameter model's layer.
        dict(name="scan_prompt_ragged", kind="scan_prompt", seqs=24, longest=3000, lens=4, pad=7,
             dim=4096, dstate=16, io="bf16", gate=True, zoh=False),
        # One user's next token: what counts is the latency.
        dict(name="conv_step_one", kind="conv_step", batch=1, slots=4, dim=1536, width=4,
             io="bf16", silu=True),
        # The next tokens of a large batch.
        dict(name="conv_step_batch", kind="conv_step", batch=512, slots=700, dim=4096, width=4,
             io="bf16", silu=True),
        # One user's next token.
        dict(name="scan_step_one", kind="scan_step", batch=1, slots=4, dim=1536, dstate=16,
             io="bf16", gate=True, zoh=False),
        # The next tokens of a large batch: what counts is the states' traffic.
        dict(name="scan_step_batch", kind="scan_step", batch=256, slots=300, dim=4096, dstate=16,
             io="bf16", gate=True, zoh=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(KINDS)
    io = rng.choice(("bf16", "bf16", "f32"))
    vec = 8 if io == "bf16" else 4
    dim = vec * _log_int(rng, 16, 4096 // vec)
    c = dict(kind=kind, dim=dim, io=io)
    if kind == "conv_train":
        rows = _log_int(rng, 64, max(65, min(1 << 15, (1 << 26) // dim)))
        batch = _log_int(rng, 1, min(16, rows))
        c.update(batch=batch, seqlen=max(1, rows // batch), width=rng.choice((2, 3, 4)),
                 silu=rng.random() < 0.8, state=rng.random() < 0.5, q8=rng.random() < 0.5)
    elif kind in ("conv_prompt", "scan_prompt"):
        c.update(seqs=_log_int(rng, 1, 64), longest=_log_int(rng, 16, 3000),
                 lens=rng.randrange(1 << 20), pad=rng.choice((0, 0, 1, 13)))
    else:
        batch = _log_int(rng, 1, 300)
        c.update(batch=batch, slots=batch + rng.randrange(0, 40))
    if kind in ("conv_prompt", "conv_step"):
        c.update(width=rng.choice((2, 3, 4)), silu=rng.random() < 0.8)
    if kind in ("scan_prompt", "scan_step"):
        c.update(dstate=rng.choice((4, 8, 16, 16)), gate=rng.random() < 0.7, zoh=rng.random() < 0.25)
    if kind == "scan_prompt":  # as much work as the largest listed case at most
        while sum(_lengths(c)) * dim > (1 << 26):
            c["seqs"] = max(1, c["seqs"] // 2)
            c["longest"] = max(16, c["longest"] // 2)
    return c


def _lengths(c):
    """The sequences' lengths: one of the longest, the others spread over all lengths below."""
    rng = random.Random(c["lens"])
    out = [c["longest"]] + [_log_int(rng, 1, c["longest"]) for _ in range(c["seqs"] - 1)]
    if len(out) > 4 and rng.random() < 0.5:
        out[1] = 0  # a request without new tokens
    rng.shuffle(out)
    return out


def _carries(c):
    rng = random.Random(c["lens"] + 1)
    return [rng.random() < 0.4 for _ in range(c["seqs"])]


def work(c):
    e, D = (2 if c["io"] == "bf16" else 4), c["dim"]
    if c["kind"] == "conv_train":
        M, W, B = c["batch"] * c["seqlen"], c["width"], c["batch"]
        act = 10 if c["silu"] else 0
        b = M * D * (2 * e + 3 * e)  # forward: x, y; backward: x, dy, dx
        f = M * D * (2 * W + act + 6 * W + act)
        if c["q8"]:  # the forward writes the checkpoint; restoring reads it and writes y, the
            # backward reads it in place of x
            q = M * (D + -(-D // 32))
            b += 3 * q + M * D * e - M * D * e
            f += M * D * (2 * W + act + 4)
        if c["state"]:
            b += 6 * B * (W - 1) * D * e
        return {"bytes": b + 2 * D * (W + 1) * 4, "flops": f}
    if c["kind"] == "conv_step":
        M, W = c["batch"], c["width"]
        return {"bytes": M * D * e * (2 + 2 * (W - 1)) + D * (W + 1) * 4, "flops": M * D * (2 * W + 5)}
    if c["kind"] == "conv_prompt":
        M, W = sum(_lengths(c)), c["width"]
        states = c["seqs"] + sum(_carries(c))
        return {"bytes": 2 * M * D * e + states * (W - 1) * D * e + D * (W + 1) * 4,
                "flops": M * D * (2 * W + 5)}
    N = c["dstate"]
    if c["kind"] == "scan_step":
        M, states = c["batch"], 2 * c["batch"]
    else:
        M, states = sum(_lengths(c)), c["seqs"] + sum(_carries(c))
    rows = M * (D * e * (4 if c["gate"] else 3) + 2 * N * e)
    return {"bytes": rows + states * D * N * 4 + D * (N + 1) * 4,
            "flops": M * D * (N * (10 if c["zoh"] else 7) + (16 if c["gate"] else 10))}


# ------------------------------------------------------------------------------------ inputs
def _raw(v):
    return math.log(math.expm1(v))  # softplus(_raw(v)) = v


def prepare(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, D = DTYPES[c["io"]], c["dim"]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

    st = dict(case=c)
    if c["kind"] in ("conv_train", "conv_prompt", "conv_step"):
        W = c["width"]
        st["w"] = (torch.rand(D, W, generator=gen, device=dev) * 2 - 1) / math.sqrt(W)
        st["bias"] = (torch.rand(D, generator=gen, device=dev) * 2 - 1) / math.sqrt(W)
    else:
        N = c["dstate"]
        st["A_log"] = torch.log(torch.arange(1, N + 1, device=dev, dtype=torch.float32)).repeat(D, 1)
        st["Dskip"] = normal(D, dtype=torch.float32)
    if c["kind"] == "conv_train":
        B, L = c["batch"], c["seqlen"]
        # the input is one half of the rows of the projection before it, as in a layer
        st["xz"] = normal(B, L, 2 * D)
        st["dy"] = normal(B, L, D)
        if c["state"]:
            st["s0"] = normal(B, W - 1, D)
            st["dsL"] = normal(B, W - 1, D)
        return st
    if c["kind"] in ("conv_prompt", "scan_prompt"):
        ls = _lengths(c)
        off = [0]
        for n in ls:
            off.append(off[-1] + n)
        rows, slots = off[-1] + c["pad"], c["seqs"] + 3
        st["offsets_host"], st["rows"] = off, rows
        st["offsets"] = torch.tensor(off, dtype=torch.int32, device=dev)
        st["carry_host"] = _carries(c)
        st["carry"] = torch.tensor(st["carry_host"], dtype=torch.uint8, device=dev)
        st["slots"] = torch.randperm(slots, generator=gen, device=dev)[: c["seqs"]].to(torch.int32)
    else:
        rows, slots = c["batch"], c["slots"]
        st["slots"] = torch.randperm(slots, generator=gen, device=dev)[:rows].to(torch.int32)
    st["slots64"] = st["slots"].long()
    if c["kind"] in ("conv_prompt", "conv_step"):
        st["x"] = normal(rows, 2 * D)[:, :D]
        st["pool"] = normal(slots, W - 1, D)
    else:
        st["x"] = normal(rows, D)
        lo, hi = _raw(1e-3), _raw(1e-1)
        st["delta_raw"] = (torch.rand(rows, D, generator=gen, device=dev) * (hi - lo) + lo).to(dt)
        # B and C are columns of one projection's rows
        st["bc"] = normal(rows, 2 * N + (8 if dt == torch.bfloat16 else 4))
        st["z"] = normal(rows, 2 * D)[:, D:] if c["gate"] else None
        st["pool"] = normal(slots, D, N, dtype=torch.float32)
    st["y"] = torch.zeros(rows, D, dtype=dt, device=dev)
    return st


# ------------------------------------------------------------------------------------ plain forms
def _silu(v):
    return v / (1 + torch.exp(-v))


def _taps(x, w, bias, s0, silu):
    """x [B,L,D], s0 [B,W-1,D] in 32 bits -> (x with its past, pre-activation, output)."""
    L, W = x.shape[1], w.shape[1]
    xp = torch.cat([s0, x], 1)
    v = bias + sum(w[:, j] * xp[:, j:j + L] for j in range(W))
    return xp, v, _silu(v) if silu else v


def _eight_bits(x):
    """The values that the 8-bit checkpoint of x holds: in each row, groups of 32 channels share a
    power of two 2^(e-6), e = floor(log2(largest magnitude)), one more where rounding would pass
    127; the values are whole multiples, ties to even."""
    B, L, D = x.shape
    g = F.pad(x, (0, -D % 32)).view(B, L, -1, 32)
    top = g.abs().amax(-1, keepdim=True)
    e = torch.frexp(top)[1] - 1
    e = e + (torch.ldexp(top, 6 - e) >= 127.5).int()
    q = torch.round(torch.ldexp(g, 6 - e))
    return torch.ldexp(q, e - 6).view(B, L, -1)[..., :D]


def _plain_conv_train(st):
    c = st["case"]
    dt, L, D, W, B = DTYPES[c["io"]], c["seqlen"], c["dim"], c["width"], c["batch"]
    x, dy = st["xz"][..., :D].float(), st["dy"].float()
    zero = torch.zeros(B, W - 1, D, device=x.device)
    s0 = st["s0"].float() if c["state"] else zero
    w, bias = st["w"], st["bias"]
    out = {}
    xp, v, y = _taps(x, w, bias, s0, c["silu"])
    out["y"] = y.to(dt)
    if c["state"]:
        out["sL"] = xp[:, L:].to(dt)
    if c["q8"]:
        xp, v, y = _taps(_eight_bits(x), w, bias, s0, c["silu"])
        out["restored"] = y.to(dt)
    if c["silu"]:
        s = 1 / (1 + torch.exp(-v))
        g = dy * s * (1 + v * (1 - s))
    else:
        g = dy
    out["dbias"] = g.sum((0, 1))
    out["dw"] = torch.stack([(g * xp[:, j:j + L]).sum((0, 1)) for j in range(W)], 1)
    dxp = torch.zeros_like(xp)
    for j in range(W):
        dxp[:, j:j + L] += w[:, j] * g
    if c["state"]:
        dxp[:, L:] += st["dsL"].float()
        out["ds0"] = dxp[:, :W - 1].to(dt)
    out["dx"] = dxp[:, W - 1:].to(dt)
    return out


def _plain_conv_prompt(st):
    c = st["case"]
    w, bias, W, dt = st["w"], st["bias"], c["width"], DTYPES[c["io"]]
    off = st["offsets_host"]
    past = st["pool"][st["slots64"]].float() * st["carry"].float()[:, None, None]
    for s in range(c["seqs"]):
        x = st["x"][off[s]:off[s + 1]].float()
        xp, _, y = _taps(x[None], w, bias, past[s:s + 1], c["silu"])
        st["y"][off[s]:off[s + 1]] = y[0].to(dt)
        past[s] = xp[0, xp.shape[1] - (W - 1):]
    st["pool"].index_copy_(0, st["slots64"], past.to(dt))
    return st["y"], st["pool"]


def _plain_conv_step(st):
    c = st["case"]
    past = st["pool"][st["slots64"]].float()
    xp, _, y = _taps(st["x"].float()[:, None], st["w"], st["bias"], past, c["silu"])
    st["y"].copy_(y[:, 0])
    st["pool"].index_copy_(0, st["slots64"], xp[:, 1:].to(st["pool"].dtype))
    return st["y"], st["pool"]


def _update(h, A, x, delta, Bm, Cm, Dskip, z, zoh):
    """One step of the scan: h [S,D,N], x, delta, z [S,D], Bm, Cm [S,N] -> (h, y)."""
    e = delta[:, :, None] * A
    b = torch.expm1(e) / A if zoh else delta[:, :, None]
    h = torch.exp(e) * h + b * x[:, :, None] * Bm[:, None, :]
    y = (h * Cm[:, None, :]).sum(-1) + Dskip * x
    return h, y if z is None else y * _silu(z)


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _scan_inputs(st):
    c = st["case"]
    N = c["dstate"]
    return (-torch.exp(st["A_log"]), st["x"].float(), _softplus(st["delta_raw"].float()),
            st["bc"][:, :N].float(), st["bc"][:, N:2 * N].float(),
            st["z"].float() if c["gate"] else None)


def _plain_scan_prompt(st):
    c = st["case"]
    A, x, delta, Bm, Cm, z = _scan_inputs(st)
    off, y = st["offsets_host"], torch.zeros_like(x)
    order = sorted(range(c["seqs"]), key=lambda s: off[s] - off[s + 1])  # the longest first
    lens = [off[s + 1] - off[s] for s in order]
    perm = torch.tensor(order, device=x.device)
    first, slots = st["offsets"].long()[perm], st["slots64"][perm]
    h = st["pool"][slots] * st["carry"][perm].float()[:, None, None]
    n = len(order)
    for t in range(c["longest"]):
        while n and lens[n - 1] <= t:
            n -= 1
        r = first[:n] + t
        h[:n], y[r] = _update(h[:n], A, x[r], delta[r], Bm[r], Cm[r], st["Dskip"],
                              z[r] if c["gate"] else None, c["zoh"])
    st["y"].copy_(y)
    st["pool"].index_copy_(0, slots, h)
    return st["y"], st["pool"]


def _plain_scan_step(st):
    c = st["case"]
    A, x, delta, Bm, Cm, z = _scan_inputs(st)
    h, y = _update(st["pool"][st["slots64"]], A, x, delta, Bm, Cm, st["Dskip"], z, c["zoh"])
    st["y"].copy_(y)
    st["pool"].index_copy_(0, st["slots64"], h)
    return st["y"], st["pool"]


# ------------------------------------------------------------------------------------ the library's calls
def _own_conv_train(st):
    S, c = _ops(), st["case"]
    x, s0, dsL = st["xz"][..., : c["dim"]], st.get("s0"), st.get("dsL")
    kw = dict(silu=c["silu"], s0=s0)
    y, sL, q8 = S.ssm_conv_fwd(x, st["w"], st["bias"], want_sL=c["state"], want_q8=c["q8"], **kw)
    out = {"y": y}
    if c["state"]:
        out["sL"] = sL
    if c["q8"]:
        out["restored"] = S.ssm_conv_restore(q8, st["w"], st["bias"], dtype=x.dtype, **kw)
        x = None
    g = S.ssm_conv_bwd(x, st["w"], st["bias"], st["dy"], q8=q8, dsL=dsL, **kw)
    out.update(dbias=g["dbias"], dw=g["dw"])
    if c["state"]:
        out["ds0"] = g["ds0"]
    out["dx"] = g["dx"]
    return out


def _own_conv_prompt(st):
    c = st["case"]
    y = _ops().ssm_conv_prompt(st["x"], st["w"], st["bias"], st["offsets"], st["slots"], st["pool"],
                               carry=st["carry"], silu=c["silu"], y=st["y"])
    return y, st["pool"]


def _own_conv_step(st):
    y = _ops().ssm_conv_step(st["x"], st["w"], st["bias"], st["slots"], st["pool"],
                             silu=st["case"]["silu"], y=st["y"])
    return y, st["pool"]


def _own_scan_prompt(st):
    c = st["case"]
    N = c["dstate"]
    y = _ops().ssm_scan_prompt(st["x"], st["delta_raw"], st["A_log"], st["bc"][:, :N],
                               st["bc"][:, N:2 * N], st["Dskip"], st["offsets"], st["slots"],
                               st["pool"], carry=st["carry"], z=st["z"], zoh=c["zoh"],
                               max_len=c["longest"], y=st["y"])
    return y, st["pool"]


def _own_scan_step(st):
    c = st["case"]
    N = c["dstate"]
    y = _ops().ssm_scan_step(st["x"], st["delta_raw"], st["A_log"], st["bc"][:, :N],
                             st["bc"][:, N:2 * N], st["Dskip"], st["slots"], st["pool"], z=st["z"],
                             zoh=c["zoh"], y=st["y"])
    return y, st["pool"]


def run(st):
    return globals()[("_own_" if own else "_plain_") + st["case"]["kind"]](st)


# ------------------------------------------------------------------------------------ float64
def _exact_conv(x, w, bias, past, silu):
    """One sequence: x [L,D], past [W-1,D], all float64; differentiable."""
    v = torch.einsum("ldw,dw->ld", torch.cat([past, x]).unfold(0, w.shape[1], 1), w) + bias
    return v * torch.sigmoid(v) if silu else v


def _exact_eight_bits(x):
    out = x.clone()
    for k in range(0, x.shape[-1], 32):
        g = x[..., k:k + 32]
        top = g.abs().amax(-1, keepdim=True)
        step = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))) - 6)
        step = torch.where(top / step >= 127.5, 2 * step, step)
        out[..., k:k + 32] = torch.round(g / step) * step
    return out


def _exact_conv_train(st):
    c = st["case"]
    D, W, B, L = c["dim"], c["width"], c["batch"], c["seqlen"]
    w, bias = (st[k].double().requires_grad_() for k in ("w", "bias"))
    rows, dw, db = [], 0, 0
    for b in range(B):  # a sequence at a time: the float64 graph of all would not fit
        x, dy = st["xz"][b, :, :D].double(), st["dy"][b].double()
        s0 = st["s0"][b].double() if c["state"] else torch.zeros(W - 1, D, dtype=x.dtype, device=x.device)
        r = {}
        with torch.no_grad():
            r["y"] = _exact_conv(x, w, bias, s0, c["silu"])
            if c["state"]:
                r["sL"] = torch.cat([s0, x])[L:]
            if c["q8"]:
                x = _exact_eight_bits(x)
        x.requires_grad_(), s0.requires_grad_()
        y = _exact_conv(x, w, bias, s0, c["silu"])
        if c["q8"]:
            r["restored"] = y.detach()
        loss = (y * dy).sum()
        if c["state"]:
            loss = loss + (torch.cat([s0, x])[L:] * st["dsL"][b].double()).sum()
        dx, ds0, gw, gb = torch.autograd.grad(loss, (x, s0, w, bias))
        r["dx"], r["ds0"] = dx, ds0
        dw, db = dw + gw, db + gb
        rows.append(r)
        del y, loss
    out = {}
    for k in ("y", "sL", "restored", "dbias", "dw", "ds0", "dx"):
        if k in ("dbias", "dw"):
            out[k] = db if k == "dbias" else dw
        elif k in rows[0] and (k != "ds0" or c["state"]):
            out[k] = torch.stack([r.pop(k) for r in rows])
    return out


def _exact_conv_serve(st, off, carry):
    c = st["case"]
    W = c["width"]
    w, bias = st["w"].double(), st["bias"].double()
    y, pool = st["y"].double(), st["pool"].double()
    for s, k in enumerate(st["slots"].tolist()):
        x = st["x"][off[s]:off[s + 1]].double()
        past = pool[k].clone() if carry[s] else torch.zeros_like(pool[k])
        if x.shape[0]:
            y[off[s]:off[s + 1]] = _exact_conv(x, w, bias, past, c["silu"])
        pool[k] = torch.cat([past, x])[x.shape[0]:]
    return y, pool


def _exact_scan_serve(st, off, carry):
    c = st["case"]
    N = c["dstate"]
    A, Dskip = -torch.exp(st["A_log"].double()), st["Dskip"].double()
    y, pool = st["y"].double(), st["pool"].double()
    for s, k in enumerate(st["slots"].tolist()):
        h = pool[k].clone() if carry[s] else torch.zeros_like(pool[k])
        for lo in range(off[s], off[s + 1], 256):  # the transitions of 256 steps at a time
            sl = slice(lo, min(off[s + 1], lo + 256))
            x, Bm, Cm = st["x"][sl].double(), st["bc"][sl, :N].double(), st["bc"][sl, N:2 * N].double()
            delta = F.softplus(st["delta_raw"][sl].double(), threshold=1e9)
            a = torch.exp(delta[..., None] * A)
            b = (torch.expm1(delta[..., None] * A) / A if c["zoh"] else delta[..., None])
            b = b * torch.einsum("td,tn->tdn", x, Bm)
            for t in range(a.shape[0]):  # b becomes the trajectory of the state
                h = b[t].addcmul_(a[t], h)
            yt = torch.einsum("tdn,tn->td", b, Cm) + Dskip * x
            if c["gate"]:
                yt = yt * F.silu(st["z"][sl].double())
            y[sl] = yt
            h = h.clone()
        pool[k] = h
    return y, pool


def exact(c, seed):
    st = prepare(c, seed)
    if c["kind"] == "conv_train":
        return _exact_conv_train(st)
    serve = _exact_conv_serve if c["kind"].startswith("conv") else _exact_scan_serve
    if c["kind"].endswith("prompt"):
        return serve(st, st["offsets_host"], st["carry_host"])
    return serve(st, list(range(c["batch"] + 1)), [True] * c["batch"])
