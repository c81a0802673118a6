"""Cases of the gated delta rule and the group norm: what they are, their plain forms, and their
values in 64 bits.

The gated delta rule keeps a matrix S [d, dv] for each head.  Token t with key k, value v, query q,
log decay g and write strength beta does

    S <- exp(g) S;   S <- S + beta k (v - S^T k)^T;   o = scale S^T q

``prefill`` takes a whole prompt through it, ``train`` a forward and its gradients, ``step`` one
token of every sequence.  The group norm normalises each group of channels of every row of a
channels-last tensor (what a linear-attention layer does to its heads' outputs), ``norm`` forward
and ``norm_grad`` backward.

Layouts: "bhtd" is [B, H, T, d], "bthd" is [B, T, H, d].  ``hk`` query/key heads serve ``h`` value
heads, h/hk each.
"""
import math

import torch

own = False
DEV = "cuda"
CHUNK = 64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _delta(name, kind, dtype, b, hk, h, t, d, dv, layout="bhtd", state=False, ragged=False):
    return {"name": name, "kind": kind, "dtype": dtype, "b": b, "hk": hk, "h": h, "t": t, "d": d, "dv": dv,
            "layout": layout, "state": state, "ragged": ragged}


def _norm(name, kind, dtype, rows, groups, width, gate, silu, center, affine):
    return {"name": name, "kind": kind, "dtype": dtype, "rows": rows, "groups": groups, "width": width,
            "gate": gate, "silu": silu, "center": center, "affine": affine}


def listed():
    return [
        # one user, one token: latency of a single decode step
        _delta("step_bf16_1x16x64", "step", "bf16", 1, 16, 16, 1, 64, 64),
        # a full serving batch of an odd number of sequences, two value heads to each key head
        _delta("step_bf16_193x8x16x128", "step", "bf16", 193, 8, 16, 1, 128, 128),
        # the smallest prompt: two short heads in fp32
        _delta("prefill_f32_1x2x256x32", "prefill", "f32", 1, 2, 2, 256, 32, 32),
        # a batch of prompts over many heads
        _delta("prefill_bf16_4x16x4096x64", "prefill", "bf16", 4, 16, 16, 4096, 64, 64),
        # one long document over few heads, in the layout that projections write
        _delta("prefill_bf16_1x4x16384x64", "prefill", "bf16", 1, 4, 4, 16384, 64, 64, layout="bthd"),
        # a padded batch of prompts of different lengths that continue a cached state
        _delta("prefill_bf16_3x4x8x1999x128", "prefill", "bf16", 3, 4, 8, 1999, 128, 128, layout="bthd",
               state=True, ragged=True),
        # a training step's forward and backward
        _delta("train_bf16_4x16x4096x64", "train", "bf16", 4, 16, 16, 4096, 64, 64),
        # the same in fp32 with narrow heads
        _delta("train_f32_2x8x4096x32", "train", "f32", 2, 8, 8, 4096, 32, 32),
        # output norm of a decode batch, gated: latency
        _norm("norm_bf16_64x16x64", "norm", "bf16", 64, 16, 64, True, True, False, True),
        # output norm of a prefill, gated
        _norm("norm_bf16_16384x16x64", "norm", "bf16", 16384, 16, 64, True, True, False, True),
        # its gradients
        _norm("norm_grad_bf16_16384x16x64", "norm_grad", "bf16", 16384, 16, 64, True, True, False, True),
        # odd rows and groups in fp32, mean subtracted, activation on the result
        _norm("norm_grad_f32_1023x7x96", "norm_grad", "f32", 1023, 7, 96, False, True, True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["step", "step", "prefill", "prefill", "prefill", "train", "train", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("norm", "norm_grad"):
        groups, width = _log(rng, 1, 33), rng.choice([32, 33, 64, 96, 100, 128, 256])
        rows = _log(rng, 1, min(16384, (1 << 24) // (groups * width)))
        return {"kind": kind, "dtype": dtype, "rows": rows, "groups": groups, "width": width,
                "gate": rng.random() < 0.5, "silu": rng.random() < 0.7, "center": rng.random() < 0.5,
                "affine": rng.random() < 0.8}
    d = rng.choice([32, 64, 64, 128])
    dv = d if rng.random() < 0.7 else rng.choice([32, 64, 128])
    hk, share = _log(rng, 1, 16), rng.choice([1, 1, 2, 3])
    h = hk * share
    case = {"kind": kind, "dtype": dtype, "hk": hk, "h": h, "d": d, "dv": dv,
            "layout": rng.choice(["bhtd", "bthd"]), "state": rng.random() < 0.4, "ragged": rng.random() < 0.3}
    if kind == "step":
        most = max(1, (193 * 16 * 128 * 128) // (h * d * dv))
        return {**case, "b": _log(rng, 1, min(193, most)), "t": 1, "state": False, "ragged": False}
    # half of the largest listed case's elements in bf16, a quarter of that in fp32
    most = (4 * 16 * 4096 * 64) // (2 if dtype == "bf16" else 8) // (h * max(d, dv))
    t = _log(rng, 1, max(1, min(16384, most)))
    return {**case, "t": t, "b": _log(rng, 1, max(1, min(8, most // t)))}


def _shape(case, heads, *last):
    b, t = case["b"], case["t"]
    return (b, heads, t, *last) if case["layout"] == "bhtd" else (b, t, heads, *last)


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    s = {"case": case}
    if case["kind"] in ("norm", "norm_grad"):
        n, c = case["rows"], case["groups"] * case["width"]
        s["x"] = (randn(n, c) * 0.5 + 0.1).to(dt)
        s["gate"] = randn(n, c).to(dt) if case["gate"] else None
        s["weight"] = 1 + 0.2 * randn(c) if case["affine"] else None
        s["bias"] = 0.1 * randn(c) if case["affine"] else None
        s["dy"] = randn(n, c).to(dt) if case["kind"] == "norm_grad" else None
        return s
    step = case["kind"] == "step"
    hk, h, d, dv = case["hk"], case["h"], case["d"], case["dv"]

    def shape(heads, *last):
        return (case["b"], heads, *last) if step else _shape(case, heads, *last)

    def unit(x):  # keys and queries come out of an activation and are normalised
        x = torch.nn.functional.silu(x)
        return x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()

    s["q"], s["k"] = unit(randn(*shape(hk, d))).to(dt), unit(randn(*shape(hk, d))).to(dt)
    s["v"] = randn(*shape(h, dv)).to(dt)
    # decays between slow and fast heads, write strengths in (0, 1)
    s["g"] = -torch.nn.functional.softplus(randn(*shape(h)) - 2.0)
    s["beta"] = torch.sigmoid(randn(*shape(h)))
    s["scale"] = d ** -0.5
    s["state"] = randn(case["b"], h, d, dv) * 0.1 if step or case["state"] else None
    if case["ragged"]:
        u = torch.rand(case["b"], generator=gen, device=DEV)
        s["lengths"] = (u * (case["t"] + 1)).to(torch.int32)
    else:
        s["lengths"] = None
    if case["kind"] == "train":
        s["dout"] = randn(*shape(h, dv)).to(dt)
        s["dstate"] = randn(case["b"], h, d, dv) * 0.1 if case["state"] else None
    return s


# ---------------------------------------------------------------- plain forms, 32 bits

def _heads_first(x, layout):
    return x if layout == "bhtd" else x.transpose(1, 2)


def _plain_rule(q, k, v, g, beta, state, lengths, scale):
    """All [B, H, T, ...] fp32; the chunk form, one loop over the chunks that carry the state."""
    b, h, t, d = q.shape
    dv = v.shape[-1]
    if lengths is not None:  # tokens behind a sequence's end leave the state and answer nothing
        live = torch.arange(t, device=q.device)[None, None, :] < lengths[:, None, None]
        q, k, v = (torch.where(live[..., None], x, torch.zeros_like(x)) for x in (q, k, v))
        g, beta = (torch.where(live, x, torch.zeros_like(x)) for x in (g, beta))
    n = -(-t // CHUNK)
    more = n * CHUNK - t

    def chunks(x, *last):
        pad = torch.zeros(b, h, more, *last, dtype=x.dtype, device=x.device)
        return torch.cat([x, pad], 2).reshape(b, h, n, CHUNK, *last)

    q, k, v, g, beta = chunks(q, d), chunks(k, d), chunks(v, dv), chunks(g), chunks(beta)
    cum = g.double().cumsum(-1)
    gap = cum[..., :, None] - cum[..., None, :]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = torch.where(low, gap, torch.full_like(gap, -math.inf)).exp().float()
    since, left = cum.exp().float(), (cum[..., -1:] - cum).exp().float()
    eye = torch.eye(CHUNK, device=q.device)
    m = (k @ k.transpose(-1, -2)) * decay * (1 - eye)
    a = m * beta[..., None, :] + eye
    both = torch.linalg.solve_triangular(a, torch.cat([v, since[..., None] * k], -1), upper=False, unitriangular=True)
    r0, w = both[..., :dv], both[..., dv:]
    key = left[..., None] * k
    s = torch.zeros(b, h, d, dv, device=q.device) if state is None else state
    starts, us = [], []
    for i in range(n):
        starts.append(s)
        u = beta[:, :, i, :, None] * (r0[:, :, i] - w[:, :, i] @ s)
        us.append(u)
        s = since[:, :, i, -1, None, None] * s + key[:, :, i].transpose(-1, -2) @ u
    p = (q @ k.transpose(-1, -2)) * decay
    o = scale * (since[..., None] * (q @ torch.stack(starts, 2)) + p @ torch.stack(us, 2))
    return o.reshape(b, h, n * CHUNK, dv)[:, :, :t], s


def _plain_delta(s):
    case = s["case"]
    dt, layout, share = DTYPES[case["dtype"]], case["layout"], case["h"] // case["hk"]
    train = case["kind"] == "train"
    leaves = [s[n].float() for n in ("q", "k", "v", "g", "beta")]
    state = s["state"]
    if train:
        leaves = [x.detach().clone().requires_grad_() for x in leaves]
        state = state.clone().requires_grad_() if state is not None else None
    with torch.set_grad_enabled(train):
        q, k, v, g, beta = (_heads_first(x, layout) for x in leaves)
        q, k = q.repeat_interleave(share, 1), k.repeat_interleave(share, 1)
        o, last = _plain_rule(q, k, v, g, beta, state, s["lengths"], s["scale"])
        o = _heads_first(o, layout)
    out = {"o": o.detach().to(dt).contiguous(), "state": last.detach()}
    if not train:
        return out
    wrt = leaves + ([state] if state is not None else [])
    back = [s["dout"].float()] + ([s["dstate"]] if s["dstate"] is not None else [])
    grads = torch.autograd.grad([o] + ([last] if s["dstate"] is not None else []), wrt, back)
    for name, x in zip(("dq", "dk", "dv", "dg", "dbeta", "dstate"), grads):
        out[name] = x.to(dt) if name in ("dq", "dk", "dv") else x
    return out


def _plain_step(s):
    case = s["case"]
    share = case["h"] // case["hk"]
    q, k = (s[n].float().repeat_interleave(share, 1) for n in ("q", "k"))
    old = s["g"].exp()[..., None, None] * s["state"]
    u = s["beta"][..., None] * (s["v"].float() - (old * k[..., None]).sum(-2))
    new = old + k[..., None] * u[..., None, :]
    o = s["scale"] * (new * q[..., None]).sum(-2)
    s["state"].copy_(new)
    return {"o": o.to(DTYPES[case["dtype"]]), "state": s["state"]}


def _normal(x, case, eps):
    n, groups, width = case["rows"], case["groups"], case["width"]
    x = x.reshape(n, groups, width)
    if case["center"]:
        x = x - x.mean(-1, keepdim=True)
    rstd = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    return (x * rstd).reshape(n, -1), rstd


EPS = 1e-5


def _plain_norm(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    groups, width = case["groups"], case["width"]
    xhat, rstd = _normal(s["x"].float(), case, EPS)
    z = xhat * s["weight"] + s["bias"] if case["affine"] else xhat
    # the activation is on the gate where there is one, and on the result where there is none
    a = s["gate"].float() if case["gate"] else z
    sig = torch.sigmoid(a)
    act = a * sig if case["silu"] else a
    if case["kind"] == "norm":
        return {"y": (z * act if case["gate"] else act).to(dt)}
    dy = s["dy"].float()
    slope = sig * (1 + a * (1 - sig)) if case["silu"] else torch.ones_like(a)
    out = {}
    if case["gate"]:
        dz, out["dgate"] = dy * act, (dy * z * slope).to(dt)
    else:
        dz = dy * slope
    dxhat = dz
    if case["affine"]:
        out["dweight"], out["dbias"] = (dz * xhat).double().sum(0).float(), dz.double().sum(0).float()
        dxhat = dz * s["weight"]
    grp = (case["rows"], groups, width)
    dxhat, xg = dxhat.reshape(grp), xhat.reshape(grp)
    dx = dxhat - xg * (dxhat * xg).mean(-1, keepdim=True)
    if case["center"]:
        dx = dx - dxhat.mean(-1, keepdim=True)
    out["dx"] = (dx * rstd).reshape(case["rows"], -1).to(dt)
    return out


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import higher_order_linear_chunked_b200 as hla
    case = s["case"]
    kind = case["kind"]
    if kind in ("norm", "norm_grad"):
        how = {"weight": s["weight"], "bias": s["bias"], "gate": s["gate"], "eps": EPS, "center": case["center"],
               "activation": "silu" if case["silu"] else "none"}
        if kind == "norm":
            return {"y": hla.group_norm(s["x"], case["groups"], **how)}
        dx, dgate, dweight, dbias = hla.group_norm_backward(s["x"], s["dy"], case["groups"], **how)
        got = {"dx": dx, "dgate": dgate, "dweight": dweight, "dbias": dbias}
        return {n: x for n, x in got.items() if x is not None}
    leaves = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    if kind == "step":
        return {"o": hla.gated_delta_step(s["state"], *leaves, scale=s["scale"]), "state": s["state"]}
    how = {"scale": s["scale"], "initial_state": s["state"], "lengths": s["lengths"], "layout": case["layout"]}
    o, last = hla.gated_delta(*leaves, return_state=True, **how)
    out = {"o": o, "state": last}
    if kind == "train":
        grads = hla.gated_delta_backward(*leaves, s["dout"], dstate=s["dstate"], **how)
        out.update({n: x for n, x in zip(("dq", "dk", "dv", "dg", "dbeta", "dstate"), grads) if x is not None})
    return out


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind in ("norm", "norm_grad"):
        return _plain_norm(state)
    return _plain_step(state) if kind == "step" else _plain_delta(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] in ("norm", "norm_grad"):
        n = case["rows"] * case["groups"] * case["width"]
        planes = 2 + case["gate"] if case["kind"] == "norm" else 3 + 2 * case["gate"]
        return {"bytes": planes * n * size, "flops": (10 if case["kind"] == "norm" else 25) * n}
    b, hk, h, t, d, dv = (case[n] for n in ("b", "hk", "h", "t", "d", "dv"))
    leaves = b * t * ((2 * hk * d + h * dv) * size + 8 * h)
    out = b * t * h * dv * size
    state = 4 * b * h * d * dv
    # a token reads S^T k, writes k u^T and reads S^T q: six d dv, and the decay
    rule = 7 * b * h * t * d * dv
    if case["kind"] == "train":  # forward and backward each read the leaves; the gradients leave once
        return {"bytes": 3 * leaves + 2 * out + state * (4 if case["state"] else 1), "flops": 3.5 * rule}
    return {"bytes": leaves + out + state * (2 if case["kind"] == "step" or case["state"] else 1), "flops": rule}


# ---------------------------------------------------------------- the definitions, 64 bits

def _exact_norm(case, s):
    x = s["x"].double().view(case["rows"], case["groups"], case["width"])
    mean = x.mean(2, keepdim=True) if case["center"] else torch.zeros_like(x[..., :1])
    sd = torch.sqrt(((x - mean) ** 2).mean(2, keepdim=True) + EPS)
    one = torch.ones(x.shape[1] * x.shape[2], dtype=torch.float64, device=x.device)
    w = (s["weight"].double() if case["affine"] else one).requires_grad_()
    c = (s["bias"].double() if case["affine"] else one * 0).requires_grad_()
    leaf = ((x - mean) / sd).reshape(case["rows"], -1).requires_grad_()
    gate = s["gate"].double().requires_grad_() if case["gate"] else None
    with torch.enable_grad():
        z = leaf * w + c
        hot = gate if case["gate"] else z
        act = hot / (1 + torch.exp(-hot)) if case["silu"] else hot
        y = z * act if case["gate"] else act
    if case["kind"] == "norm":
        return {"y": y.detach()}
    wrt = [leaf, w, c] + ([gate] if case["gate"] else [])
    got = torch.autograd.grad(y, wrt, s["dy"].double())
    out = {"dgate": got[3]} if case["gate"] else {}
    if case["affine"]:
        out["dweight"], out["dbias"] = got[1], got[2]
    # through sd = sqrt(mean((x - mean)^2) + eps)
    dn = got[0].view_as(x)
    dsd = -(dn * (x - mean)).sum(2, keepdim=True) / sd ** 2
    dx = dn / sd + dsd * (x - mean) / (sd * case["width"])
    out["dx"] = (dx - dx.mean(2, keepdim=True) if case["center"] else dx).reshape(case["rows"], -1)
    return out


def _exact_tokens(case, s):
    """The leaves in 64 bits, time first: [T, B*H, ...], with every value head's own query and key."""
    share, b, h = case["h"] // case["hk"], case["b"], case["h"]

    def flat(x, wide):
        x = x.double()
        if case["kind"] == "step":
            x = x.unsqueeze(2)
        elif case["layout"] == "bthd":
            x = x.transpose(1, 2)
        x = x.repeat_interleave(share, 1) if wide else x
        return x.transpose(0, 2).transpose(1, 2).reshape(x.shape[2], b * h, *x.shape[3:])

    return [flat(s[n], n in "qk") for n in ("q", "k", "v", "g", "beta")]


def _token(S, k, v, a, beta):
    S = a[:, None, None] * S
    e = v - torch.einsum("nij,ni->nj", S, k)
    return S + torch.einsum("ni,nj->nij", beta[:, None] * k, e), e


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return _exact_norm(case, s) if case["kind"] in ("norm", "norm_grad") else _exact_delta(case, s)


def _exact_delta(case, s):
    b, hk, h, t, d, dv = (case[n] for n in ("b", "hk", "h", "t", "d", "dv"))
    train = case["kind"] == "train"
    if t * (4 if train else 1) > 70000:
        return None
    q, k, v, g, beta = _exact_tokens(case, s)
    a, scale = g.exp(), s["scale"]
    n = b * h
    S = s["state"].double().reshape(n, d, dv).clone() if s["state"] is not None else \
        torch.zeros(n, d, dv, dtype=torch.float64, device=q.device)
    live = torch.ones(t, n, dtype=torch.bool, device=q.device)
    if s["lengths"] is not None:
        live = (torch.arange(t, device=q.device)[:, None] < s["lengths"][None, :]).repeat_interleave(h, 1)
        a = torch.where(live, a, torch.ones_like(a))
        beta = beta * live
    o = torch.empty(t, n, dv, dtype=torch.float64, device=q.device)
    kept = {}
    for i in range(t):
        if i % CHUNK == 0 and train:
            kept[i] = S
        S, _ = _token(S, k[i], v[i], a[i], beta[i])
        o[i] = scale * torch.einsum("nij,ni->nj", S, q[i])
    o *= live[..., None]

    def back(x):  # [T, B*H, ...] to the case's layout
        x = x.reshape(t, b, h, *x.shape[2:]).transpose(0, 1)
        return x if case["layout"] == "bthd" else x.transpose(1, 2)

    last = S.reshape(b, h, d, dv)
    if case["kind"] == "step":
        return {"o": o[0].reshape(b, h, dv), "state": last}
    out = {"o": back(o), "state": last}
    if not train:
        return out
    dout = s["dout"].double()
    dout = dout if case["layout"] == "bthd" else dout.transpose(1, 2)
    dout = dout.transpose(0, 1).reshape(t, n, dv) * live[..., None]
    dq, dk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(g), torch.zeros_like(g)
    dS = s["dstate"].double().reshape(n, d, dv).clone() if s["dstate"] is not None else torch.zeros_like(S)
    for start in sorted(kept, reverse=True):
        states, errs = [kept[start]], []
        for i in range(start, min(t, start + CHUNK)):
            S, e = _token(states[-1], k[i], v[i], a[i], beta[i])
            states.append(S)
            errs.append(e)
        for i in range(min(t, start + CHUNK) - 1, start - 1, -1):
            before, after, e = states[i - start], states[i - start + 1], errs[i - start]
            dq[i] = scale * torch.einsum("nij,nj->ni", after, dout[i])
            dS = dS + scale * q[i][:, :, None] * dout[i][:, None, :]
            # after = a S + beta k e^T, e = v - a S^T k
            dSk = torch.einsum("nij,ni->nj", dS, k[i])
            de = beta[i][:, None] * dSk
            db[i] = (dSk * e).sum(-1)
            dvv[i] = de
            faded = a[i][:, None, None] * before
            dk[i] = beta[i][:, None] * torch.einsum("nij,nj->ni", dS, e) - torch.einsum("nij,nj->ni", faded, de)
            dfaded = dS - k[i][:, :, None] * de[:, None, :]
            dg[i] = (dfaded * faded).sum((1, 2))
            dS = a[i][:, None, None] * dfaded
    keep = live.double()
    dq, dk, dvv = dq * keep[..., None], dk * keep[..., None], dvv * keep[..., None]
    head = 2 if case["layout"] == "bthd" else 1

    def shared(x):
        return back(x).unflatten(head, (hk, h // hk)).sum(head + 1)

    out.update({"dq": shared(dq), "dk": shared(dk), "dv": back(dvv), "dg": back(dg * keep), "dbeta": back(db * keep)})
    if s["state"] is not None:
        out["dstate"] = dS.reshape(b, h, d, dv)
    return out
