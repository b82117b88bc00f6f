"""The cases of the training operators that sit next to the halo path: a gated projection, a group
norm with an activation, and an AdamW step over many tensors, each in its plain form (elementary
torch operations in float32, float64 where a value decides a branch or a code) and as the calls
that a program makes of libqha's binding.

Gated projection   H = act(A Wg^T) * (A Wu^T), and its gradients dA, dWg, dWu.
Group norm         y = act(w * (x - mean) * rstd + b), statistics per sample and group of channels,
                   channels last, and its gradients dx, dw, db.
AdamW              one step over a list of tensors, with moments in float32 or in 8-bit codes.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 256            # elements that share one scale of an 8-bit moment
EPS_NORM = 1e-5
BETA1, BETA2, EPS_ADAM, DECAY, LR = 0.9, 0.999, 1e-8, 0.01, 1e-3
STEP = 10              # steps taken before the timed one


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one token (or one queried node) through a gated block whose weights stream from memory
        dict(name="gated token bf16", op="gated", way="infer", type="bf16", act="silu", m=1, n=4096, k=2048),
        # the node-wise transform of the 300k-node partition, width 128, outputs kept for the backward
        dict(name="gated fwd nodes f32", op="gated", way="fwd", type="f32", act="silu", m=300000, n=128, k=128),
        # a training batch of tokens through a wide block
        dict(name="gated fwd tokens bf16", op="gated", way="fwd", type="bf16", act="silu", m=16384, n=8192, k=2048),
        # the gradients of the node-wise transform on the dense-degree partition (30k nodes, width 256)
        dict(name="gated bwd nodes f32", op="gated", way="bwd", type="f32", act="relu", m=30000, n=256, k=256),
        # the gradients of a token batch with a ragged row count
        dict(name="gated bwd tokens bf16", op="gated", way="bwd", type="bf16", act="gelu", m=8191, n=4096, k=1024),
        # every node of the 300k partition normalised on its own, 8 groups of 16 channels
        dict(name="norm fwd nodes f32", op="norm", way="fwd", type="f32", act="relu", samples=300000, positions=1,
             c=128, groups=8),
        # gradients of the same at width 256 with one group (the whole row), odd node count
        dict(name="norm bwd nodes f32", op="norm", way="bwd", type="f32", act="relu", samples=300001, positions=1,
             c=256, groups=1),
        # feature maps: 16 samples of 64 x 64 positions, 512 channels in 32 groups
        dict(name="norm fwd maps bf16", op="norm", way="fwd", type="bf16", act="silu", samples=16, positions=4096,
             c=512, groups=32),
        # a small ragged batch's gradients, where launches count
        dict(name="norm bwd small f16", op="norm", way="bwd", type="f16", act="silu", samples=3, positions=97, c=64,
             groups=8),
        # the weights of a 4-layer node model at width 128: the smallest step
        dict(name="adamw nodes 32", op="adamw", bits=32, grad="f32", copy=False, layers=4, width=128, odd=1),
        # a model of 24 blocks at width 1024, float32 moments
        dict(name="adamw model 32", op="adamw", bits=32, grad="f32", copy=False, layers=24, width=1024, odd=0),
        # the same kind of model with 8-bit moments, bf16 gradients and a bf16 copy of the weights
        dict(name="adamw model 8", op="adamw", bits=8, grad="bf16", copy=True, layers=16, width=1024, odd=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "norm", "norm", "adamw"])
    act = rng.choice(["none", "relu", "silu", "gelu"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op == "gated":
        way = rng.choice(["infer", "fwd", "bwd"])
        limit = 4 * 30000 * 300 * 300 if kind == "f32" else 4 * 16384 * 8192 * 2048 // (2 if way == "bwd" else 1)
        while True:
            m, n, k = _log(rng, 1, 300000), 8 * _log(rng, 2, 1024), 8 * _log(rng, 2, 512)
            if 1 << 16 <= 4 * m * n * k <= limit and m * max(n, k) <= 1 << 27:
                return dict(op=op, way=way, type=kind, act=act, m=m, n=n, k=k)
    if op == "norm":
        while True:
            positions = 1 if rng.random() < 0.4 else _log(rng, 2, 8192)
            samples = _log(rng, 1, 300000)
            groups = rng.choice([1, 2, 4, 5, 8, 16, 32])
            c = 8 * groups * _log(rng, 1, 64)
            if c <= 4096 and 1 << 10 <= samples * positions * c <= 300001 * 256:
                return dict(op=op, way=rng.choice(["fwd", "bwd"]), type=kind, act=act, samples=samples,
                            positions=positions, c=c, groups=groups)
    bits = rng.choice([8, 32])
    width = 4 * _log(rng, 4, 255)
    return dict(op=op, bits=bits, grad=rng.choice(["f32", "bf16", "f16"]), copy=rng.random() < 0.5,
                layers=_log(rng, 1, 16), width=width, odd=rng.randrange(0, 64))


def _shapes(case):
    """Sizes of the tensors of a model: per layer a gated pair, a projection, and two norm vectors;
    a last tensor of `odd` elements more than a multiple of the width."""
    d = case["width"]
    wide = 4 * d if d >= 512 else d
    return [s for _ in range(case["layers"]) for s in (wide * d, wide * d, d * wide, d, d)] + [d + case["odd"]]


def work(case):
    if case["op"] == "gated":
        m, n, k, b = case["m"], case["n"], case["k"], BYTES[case["type"]]
        if case["way"] == "bwd":
            return {"bytes": b * (3 * m * n + 2 * m * k + 2 * n * k) + 8 * n * k, "flops": 8 * m * n * k}
        kept = 2 if case["way"] == "fwd" else 0
        return {"bytes": b * (m * k + 2 * n * k + (1 + kept) * m * n), "flops": 4 * m * n * k}
    if case["op"] == "norm":
        e, b = case["samples"] * case["positions"] * case["c"], BYTES[case["type"]]
        stats = 8 * case["samples"] * case["groups"]
        if case["way"] == "bwd":
            return {"bytes": 3 * b * e + stats + 16 * case["c"], "flops": 20 * e}
        return {"bytes": 2 * b * e + stats + 8 * case["c"], "flops": 10 * e}
    e = sum(_shapes(case))
    moments = 16 if case["bits"] == 32 else 4 + 8 + 16.0 / BLOCK   # codes in and out, and read back as values
    return {"bytes": e * (8 + BYTES[case["grad"]] + (2 if case["copy"] else 0) + moments), "flops": 20 * e}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _act64(z, act):
    """act(z) in the type of z."""
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    st = {"case": case}
    if case["op"] == "gated":
        m, n, k, t = case["m"], case["n"], case["k"], TYPES[case["type"]]
        st["a"] = _randn(g, m, k).to(t)
        st["wg"] = (_randn(g, n, k) / math.sqrt(k)).to(t)
        st["wu"] = (_randn(g, n, k) / math.sqrt(k)).to(t)
        if case["way"] == "bwd":
            st["gate"] = (st["a"].float() @ st["wg"].float().T).to(t)       # what the forward kept
            st["up"] = (st["a"].float() @ st["wu"].float().T).to(t)
            st["dh"] = _randn(g, m, n).to(t)
    elif case["op"] == "norm":
        s, p, c, t = case["samples"], case["positions"], case["c"], TYPES[case["type"]]
        st["x"] = (_randn(g, s * p, c) * 1.5 + 0.5 * _randn(g, c) + 0.25).to(t)
        st["w"] = 1 + 0.2 * _randn(g, c)
        st["b"] = 0.2 * _randn(g, c)
        if case["way"] == "bwd":
            x = st["x"].view(s, p, case["groups"], -1).double()             # what the forward kept
            mean = x.mean((1, 3), keepdim=True)
            st["mean"] = mean.reshape(s, -1).float()
            st["rstd"] = ((x - mean).square().mean((1, 3)) + EPS_NORM).rsqrt().float()
            st["dy"] = _randn(g, s * p, c).to(t)
    else:
        sizes = _shapes(case)
        starts, at = [], 0
        for n in sizes:                                     # every tensor starts at a block
            starts.append(at)
            at += -(-n // BLOCK) * BLOCK
        live = torch.zeros(at, dtype=torch.bool, device=DEV)
        size = torch.ones(at, device=DEV)
        for n, s in zip(sizes, starts):
            live[s:s + n] = True
            size[s:s + n] = 1.0 / math.sqrt(n)              # larger tensors have smaller gradients
        st["p"] = _randn(g, at) * 0.05 * live
        st["g"] = (_randn(g, at) * size * live).to(TYPES[case["grad"]])
        m = _randn(g, at) * 0.3 * size * live
        v = (0.7 * size * live).square() * torch.exp(0.7 * _randn(g, at))
        st["t"] = STEP
        if case["bits"] == 32:
            st["m"], st["v"] = m, v
        else:
            st["m"], st["m_scale"] = _code(m.double(), 127, 2)
            st["v"], st["v_scale"] = _code(v.double(), 255, 4)
        st["views"] = [(s, n) for n, s in zip(sizes, starts)]
        if case["copy"]:
            st["copy"] = torch.zeros(at, dtype=torch.bfloat16, device=DEV)
    if own:
        _handles(st)
    return st


def _handles(st):
    """The output buffers, workspaces and the optimiser that a program keeps between steps."""
    from quantized_halo_aggregation_amd import binding as B
    case = st["case"]
    if case["op"] == "adamw":
        cut = lambda x: [x[s:s + n] for s, n in st["views"]]
        opt = B.AdamW(cut(st["p"]), bits=case["bits"], betas=(BETA1, BETA2), eps=EPS_ADAM, weight_decay=DECAY,
                      copies=cut(st["copy"]) if case["copy"] else None)
        for name in ("m", "v") + (("m_scale", "v_scale") if case["bits"] == 8 else ()):
            getattr(opt, name).copy_(st[name])
        opt.t = st["t"]
        st["opt"], st["grads"] = opt, cut(st["g"])
        if case["bits"] == 8:
            st["mv"] = (torch.empty(st["p"].numel(), device=DEV), torch.empty(st["p"].numel(), device=DEV))
        return
    t = TYPES[case["type"]]
    st["act"] = {"none": B.ACT_NONE, "relu": B.ACT_RELU, "silu": B.ACT_SILU, "gelu": B.ACT_GELU}[case["act"]]
    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device=DEV)
    if case["op"] == "gated":
        m, n, k = case["m"], case["n"], case["k"]
        if case["way"] == "bwd":
            st["out"] = (new(m, k, dtype=t), new(n, k), new(n, k))
            need = B.gated_backward_workspace(t, m, n, k)
        else:
            kept = [new(m, n, dtype=t) for _ in range(2)] if case["way"] == "fwd" else [None, None]
            st["out"] = (new(m, n, dtype=t), *kept)
            need = B.gated_project_workspace(t, m, n, k)
    else:
        rows, c, way = case["samples"] * case["positions"], case["c"], case["way"]
        stats = (case["samples"], case["groups"])
        st["out"] = (new(rows, c, dtype=t), *((new(*stats), new(*stats)) if way == "fwd" else (new(c), new(c))))
        need = B.group_norm_workspace(rows, case["positions"], c, case["groups"], way == "bwd")
    st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "gated":
        return _gated_bwd(state) if case["way"] == "bwd" else _gated_fwd(state)
    if case["op"] == "norm":
        return _norm_bwd(state) if case["way"] == "bwd" else _norm_fwd(state)
    return _adamw(state)


def _run_own(st):
    from quantized_halo_aggregation_amd import binding as B
    case = st["case"]
    if case["op"] == "gated":
        if case["way"] == "bwd":
            da, dwg, dwu = st["out"]
            B.gated_backward(st["dh"], st["gate"], st["up"], st["a"], st["wg"], st["wu"], da, dwg, dwu,
                             act=st["act"], workspace=st["ws"])
            return {"da": da, "dwg": dwg, "dwu": dwu}
        h, gate, up = st["out"]
        B.gated_project(st["a"], st["wg"], st["wu"], h, gate=gate, up=up, act=st["act"], workspace=st["ws"])
        return {"h": h, "gate": gate, "up": up} if case["way"] == "fwd" else {"h": h}
    if case["op"] == "norm":
        if case["way"] == "bwd":
            dx, dw, db = st["out"]
            B.group_norm_bwd(st["dy"], st["x"], st["mean"], st["rstd"], dx, case["groups"], weight=st["w"],
                             bias=st["b"], dweight=dw, dbias=db, act=st["act"], positions=case["positions"],
                             workspace=st["ws"])
            return {"dx": dx, "dw": dw, "db": db}
        y, mean, rstd = st["out"]
        B.group_norm_fwd(st["x"], y, case["groups"], weight=st["w"], bias=st["b"], mean=mean, rstd=rstd,
                         eps=EPS_NORM, act=st["act"], positions=case["positions"], workspace=st["ws"])
        return {"y": y, "mean": mean, "rstd": rstd}
    opt = st["opt"]
    opt.step(st["grads"], LR)
    out = {"p": st["p"], "m": opt.m, "v": opt.v}
    if case["bits"] == 8:
        out["m"], out["v"] = opt.values(*st["mv"])
    if case["copy"]:
        out["copy"] = st["copy"]
    return out


def _slope(z, act):
    """act'(z)."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _gated_fwd(st):
    case = st["case"]
    a = st["a"].float()
    gate = a @ st["wg"].float().T
    up = a @ st["wu"].float().T
    h = _act64(gate, case["act"]) * up
    t = TYPES[case["type"]]
    return {"h": h.to(t), "gate": gate.to(t), "up": up.to(t)} if case["way"] == "fwd" else {"h": h.to(t)}


def _gated_bwd(st):
    act = st["case"]["act"]
    a, dh, gate, up = st["a"].float(), st["dh"].float(), st["gate"].float(), st["up"].float()
    dg = dh * up * _slope(gate, act)
    du = dh * _act64(gate, act)
    da = dg @ st["wg"].float() + du @ st["wu"].float()
    return {"da": da.to(st["a"].dtype), "dwg": dg.T @ a, "dwu": du.T @ a}


def _norm_fwd(st):
    case = st["case"]
    x = st["x"].float().view(case["samples"], case["positions"], case["groups"], -1)
    mean = x.mean((1, 3), keepdim=True)
    rstd = ((x - mean).square().mean((1, 3), keepdim=True) + EPS_NORM).rsqrt()
    z = ((x - mean) * rstd).view(-1, case["c"]) * st["w"] + st["b"]
    stats = (case["samples"], case["groups"])
    return {"y": _act64(z, case["act"]).to(st["x"].dtype), "mean": mean.view(stats), "rstd": rstd.view(stats)}


def _norm_bwd(st):
    case = st["case"]
    s, p, c, gr = case["samples"], case["positions"], case["c"], case["groups"]
    wide = torch.float64 if case["act"] == "relu" else torch.float32       # the sign of z decides
    mean, rstd = st["mean"].view(s, 1, gr, 1), st["rstd"].view(s, 1, gr, 1)
    x = st["x"].float().view(s, p, gr, -1)
    xhat = ((x.to(wide) - mean) * rstd).view(-1, c)
    dz = st["dy"].float() * _slope(xhat * st["w"] + st["b"], case["act"]).float()
    xhat = xhat.float()
    dw, db = (dz * xhat).sum(0), dz.sum(0)
    q = (dz * st["w"]).view(s, p, gr, -1)
    xhat = xhat.view(s, p, gr, -1)
    dx = rstd * (q - q.mean((1, 3), keepdim=True) - xhat * (q * xhat).mean((1, 3), keepdim=True))
    return {"dx": dx.view(-1, c).to(st["x"].dtype), "dw": dw, "db": db}


def _code(x, top, power):
    """8-bit codes of x (float64): |x| = scale * (|code| / top)^power with the block's largest value
    as its scale (kept in float32), to the nearest code, the smaller one at half-way points (which equal
    ratios of 16-bit gradients hit exactly); a positive second moment keeps a code of at least 1."""
    x = x.view(-1, BLOCK)
    scale = x.abs().amax(1, keepdim=True)
    c = torch.ceil(top * (x.abs() / scale.clamp_min(1e-300)) ** (1.0 / power) - (0.5 + 1e-10)).clamp_max(top)
    if power == 4:
        c = torch.where(x > 0, c.clamp_min(1), c)
        return c.to(torch.uint8).view(-1), scale.float().view(-1)
    return (c * x.sign()).to(torch.int8).view(-1), scale.float().view(-1)


def _value(code, scale, top, power):
    c = code.view(-1, BLOCK).double()
    c = c * c.abs() if power == 2 else (c * c) * (c * c)
    return (scale.view(-1, 1).double() * c * (1.0 / top ** power)).view(-1)


def _keep(st, name, x, top, power):
    """Stores x as codes and gives the values that they stand for."""
    code, scale = _code(x, top, power)
    st[name].copy_(code)
    st[name + "_scale"].copy_(scale)
    return _value(code, scale, top, power).float()


def _adamw(st):
    case = st["case"]
    st["t"] += 1
    small = case["bits"] == 8
    if small:        # codes are decided in float64
        g = st["g"].double()
        m, v = _value(st["m"], st["m_scale"], 127, 2), _value(st["v"], st["v_scale"], 255, 4)
    else:
        g, m, v = st["g"].float(), st["m"], st["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    out = {}
    if small:
        out["m"], out["v"] = _keep(st, "m", m, 127, 2), _keep(st, "v", v, 255, 4)
        m, v = m.float(), v.float()
    else:
        out["m"], out["v"] = st["m"].copy_(m), st["v"].copy_(v)
    c1, c2 = 1 - BETA1 ** st["t"], 1 - BETA2 ** st["t"]
    step = (m / c1) / (torch.sqrt(v / c2) + EPS_ADAM)
    out["p"] = st["p"].copy_(st["p"] * (1 - LR * DECAY) - LR * step)
    if case["copy"]:
        out["copy"] = st["copy"].copy_(st["p"].to(torch.bfloat16))
    return out


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    d = {k: v.double() for k, v in st.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    act = case.get("act", "none")
    normal = torch.distributions.normal.Normal(torch.zeros((), dtype=torch.float64, device=DEV), 1.0)
    if act == "relu":
        f, df = (lambda z: z.clamp_min(0)), (lambda z: torch.heaviside(z, torch.zeros_like(z)))
    elif act == "silu":
        f, df = (lambda z: z * torch.sigmoid(z)), (lambda z: torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z))
    elif act == "gelu":
        f = lambda z: z * normal.cdf(z)
        df = lambda z: normal.cdf(z) + z * torch.exp(normal.log_prob(z))
    else:
        f, df = (lambda z: z), (lambda z: torch.ones_like(z))
    if case["op"] == "gated":
        if case["way"] != "bwd":
            both = torch.mm(torch.cat([d["wg"], d["wu"]]), d["a"].T.contiguous()).T
            gate, up = both[:, :case["n"]], both[:, case["n"]:]
            h = f(gate) * up
            return {"h": h, "gate": gate, "up": up} if case["way"] == "fwd" else {"h": h}
        grads = torch.cat([df(d["gate"]).mul_(d["dh"]).mul_(d["up"]), f(d["gate"]).mul_(d["dh"])], 1)
        dw = torch.mm(grads.T.contiguous(), d["a"])
        return {"da": torch.mm(grads, torch.cat([d["wg"], d["wu"]])), "dwg": dw[:case["n"]], "dwu": dw[case["n"]:]}
    if case["op"] == "norm":
        s, p, c, gr = case["samples"], case["positions"], case["c"], case["groups"]
        per = p * (c // gr)
        flat = lambda x: x.view(s, p, gr, c // gr).transpose(1, 2).reshape(s, gr, per)
        back = lambda x: x.view(s, gr, p, c // gr).transpose(1, 2).reshape(s * p, c)
        x = flat(d["x"])
        if case["way"] == "fwd":
            var, mean = torch.var_mean(x, 2, correction=0)
            rstd = 1 / torch.sqrt(var + EPS_NORM)
            y = f(torch.addcmul(d["b"], back((x - mean[..., None]) * rstd[..., None]), d["w"]))
            return {"y": y, "mean": mean, "rstd": rstd}
        xhat = (x - d["mean"][..., None]) * d["rstd"][..., None]
        dz = d["dy"] * df(torch.addcmul(d["b"], back(xhat), d["w"]))
        q = flat(dz * d["w"])
        dx = (q - q.sum(2, keepdim=True) / per - xhat * (q * xhat).sum(2, keepdim=True) / per) * d["rstd"][..., None]
        return {"dx": back(dx), "dw": (dz * back(xhat)).sum(0), "db": dz.sum(0)}
    t = st["t"] + 1
    if case["bits"] == 8:
        c = st["m"].view(-1, BLOCK).double()
        m = (c.sign() * (c / 127).square() * d["m_scale"][:, None]).view(-1)
        v = ((st["v"].view(-1, BLOCK).double() / 255).pow(4) * d["v_scale"][:, None]).view(-1)
    else:
        m, v = d["m"], d["v"]
    m = torch.lerp(d["g"], m, BETA1)
    v = torch.lerp(d["g"].square(), v, BETA2)
    update = m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)).sqrt() + EPS_ADAM)
    out = {"p": d["p"] - LR * DECAY * d["p"] - LR * update, "m": m, "v": v}
    if case["copy"]:
        out["copy"] = out["p"]
    if case["bits"] == 8:
        # the nearest code is the one between whose neighbours' half-way points the root falls
        def nearest(x, top, power):
            x = x.view(-1, BLOCK)
            scale = x.abs().max(1, keepdim=True).values
            unit = torch.where(scale > 0, x.abs() / scale, torch.zeros_like(x))
            edges = ((torch.arange(top, device=DEV, dtype=torch.float64) + 0.5) / top) ** power * (1 + 2.0 ** -40)
            level = torch.bucketize(unit, edges, right=True)
            level = torch.maximum(level, (x > 0).long()) if power == 4 else level
            return (scale * (level.double() / top) ** power * x.sign()).view(-1)
        out["m"], out["v"] = nearest(m, 127, 2), nearest(v, 255, 4)
    return out
