"""The cases of the operators that train deep stacks of the gated node layers: the norms around a block
fused with its gate and the residual stream, and updates orthogonalised by Newton-Schulz products,
each in its plain form (elementary torch operations in float32, float64 for the sum of a norm) and as the
calls that a program makes of libqha's binding.

Residual norm   x' = skip x + branch gate * post(h),  u = pre(x'), with post and pre an RMS or a layer norm of
                every row, and its gradients dx, dh, dgate and those of both norms' weights and biases.
Newton-Schulz   X = G / |G|, then five times X = a X + (b A + c A^2) X with A = X X^T.
Muon            the optimiser's step: momentum, Newton-Schulz, weight decay and update of many matrices.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS_ROW = 1e-6
SKIP, BRANCH = 1.0, 0.7
STEPS, COEF, EPS_NS = 5, (3.4445, -4.7750, 2.0315), 1e-7
MU, LR, DECAY = 0.95, 0.02, 0.1


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _norm(name, way, stream, type, post, pre, samples, positions, c, gate, bias):
    d = dict(op="norm", way=way, stream=stream, type=type, post=post, pre=pre, samples=samples, positions=positions, c=c,
             gate=gate, bias=bias)
    return dict(name=name, **d) if name else d


def listed():
    return [
        # one token (or one queried node) between two blocks of a 4096-wide stack: a call's latency
        _norm("norm fwd token bf16", "fwd", "f32", "bf16", "rms", "rms", 1, 1, 4096, False, False),
        # every node of the 300k-node partition between two layers of width 128
        _norm("norm fwd nodes f32", "fwd", "f32", "f32", "layer", "layer", 300000, 1, 128, False, True),
        # four sequences of 4096 tokens with one gate row each, on a float32 stream
        _norm("norm fwd tokens bf16", "fwd", "f32", "bf16", "rms", "layer", 4, 4096, 2048, True, False),
        # gradients of the node rows at width 256, odd node count
        _norm("norm bwd nodes f32", "bwd", "f32", "f32", "layer", "layer", 300001, 1, 256, False, True),
        # gradients of a ragged token batch with a gate for every token, all in bf16
        _norm("norm bwd tokens bf16", "bwd", "bf16", "bf16", "rms", "rms", 8191, 1, 2048, True, False),
        # a small ragged batch's gradients with a shared gate, where launches count
        _norm("norm bwd small f16", "bwd", "f16", "f16", "layer", "rms", 3, 97, 64, True, True),
        # one square update of a wide model
        dict(name="orthogonal square f32", op="ns", type="f32", out="f32", groups="1x4096x4096"),
        # a few ragged updates in half precision, wide and tall
        dict(name="orthogonal ragged f16", op="ns", type="f16", out="f16", groups="5x1000x520,3x333x777"),
        # the weights of a 4-layer node model of width 128: the smallest step
        dict(name="muon nodes f32", op="muon", type="f32", copy=False, nesterov=True, groups="8x128x128"),
        # the dense-degree partition's 4 layers of width 256
        dict(name="muon dense nodes f32", op="muon", type="f32", copy=False, nesterov=True, groups="8x256x256"),
        # a model of 8 blocks of width 1024, bf16 gradients and a bf16 copy of the weights
        dict(name="muon model bf16", op="muon", type="bf16", copy=True, nesterov=True, groups="16x4096x1024,8x1024x4096"),
    ]


def _groups(case):
    """(count, rows, cols) of the case's equal matrices."""
    return [tuple(int(v) for v in g.split("x")) for g in case["groups"].split(",")]


def _products(case):
    """Floating-point operations of the products, those of symmetric results counted once."""
    total = 0
    for count, rows, cols in _groups(case):
        m, n = min(rows, cols), max(rows, cols)
        total += count * STEPS * (3 * m * m * n + m * m * m)
    return total


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "ns", "muon"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op == "norm":
        way, gate = rng.choice(["fwd", "bwd"]), rng.random() < 0.6
        stream = rng.choice(["f32", kind])
        post, pre = rng.choice(["none", "rms", "layer"]), rng.choice(["rms", "layer", "none"])
        while True:
            c = (4 if kind == "f32" else 8) * _log(rng, 2, 1024)
            positions = 1 if rng.random() < 0.5 else _log(rng, 2, 8192)
            samples = _log(rng, 1, 300000)
            if c <= 8192 and 1 << 10 <= samples * positions * c <= 8191 * 2048 * (4 if kind == "f32" else 1):
                return _norm(None, way, stream, kind, post, pre, samples, positions, c, gate, rng.random() < 0.5)
    while True:
        sizes = [(rng.choice([1, 1, 2, 3, 4, 8, 12]), _log(rng, 8, 4096), _log(rng, 8, 4096))
                 for _ in range(rng.choice([1, 2]))]
        case = dict(op=op, type=kind, groups=",".join("%dx%dx%d" % s for s in sizes))
        if 1 << 20 <= _products(case) <= 8e11 and sum(k * r * c for k, r, c in sizes) <= 1 << 26:
            more = dict(out=rng.choice(["f32", kind])) if op == "ns" else dict(copy=rng.random() < 0.5,
                                                                              nesterov=rng.random() < 0.7)
            return dict(case, **more)


def work(case):
    if case["op"] == "norm":
        rows, c, b, s = case["samples"] * case["positions"], case["c"], BYTES[case["type"]], BYTES[case["stream"]]
        pre, gates = case["pre"] != "none", case["samples"] * c if case["gate"] else 0
        stats = 8 * rows * ((case["post"] != "none") + pre)
        vectors = 4 * c * (((case["post"] != "none") + pre) * (2 if case["bias"] else 1))
        if case["way"] == "fwd":       # x, h, gate -> x', u, statistics
            return {"bytes": rows * c * (2 * s + b + b * pre) + gates * b + stats + vectors, "flops": 14 * rows * c}
        # dy, x', h, du, gate, statistics -> dx, dh, dgate and the vectors' gradients
        return {"bytes": rows * c * (3 * s - s * (not pre) + 2 * b + b * pre) + 2 * gates * b + stats + 2 * vectors,
                "flops": 30 * rows * c}
    e, b = sum(k * r * c for k, r, c in _groups(case)), BYTES[case["type"]]
    if case["op"] == "ns":
        return {"bytes": e * (b + BYTES[case["out"]]), "flops": _products(case)}
    return {"bytes": e * (b + 16 + (2 if case["copy"] else 0)), "flops": _products(case)}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _gradients(g, count, rows, cols):
    """Gradients of matrices: noise and a few directions that stand out of it."""
    top = 3 * (rows ** 0.5 + cols ** 0.5) / (rows * cols) ** 0.5
    return (_randn(g, count, rows, cols) + top * (_randn(g, count, rows, 4) @ _randn(g, count, 4, cols))) * 1e-3


def _row_stats(x, kind):
    """(mean, 1 / deviation) of every row as a forward keeps them: float32 [rows, 2]."""
    x = x.double()
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    return torch.cat([mean, ((x - mean).square().mean(1, keepdim=True) + EPS_ROW).rsqrt()], 1).float()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    st = {"case": case}
    if case["op"] == "norm":
        rows, c, t, s = case["samples"] * case["positions"], case["c"], TYPES[case["type"]], TYPES[case["stream"]]
        x = _randn(g, rows, c) * 1.5 + 0.5 * _randn(g, c)               # the stream, before or after the block
        st["h"] = (_randn(g, rows, c) * 0.8 + 0.3 * _randn(g, c)).to(t)
        st["gate"] = (0.5 + 0.5 * _randn(g, case["samples"], c)).to(t) if case["gate"] else None
        for side in ("post", "pre"):
            normed = case[side] != "none"
            st[side + "_w"] = 1 + 0.2 * _randn(g, c) if normed else None
            st[side + "_b"] = 0.2 * _randn(g, c) if normed and case["bias"] else None
        if case["way"] == "fwd":
            st["x"] = x.to(s)
        else:
            st["y"] = x.to(s)                                           # what the forward kept
            st["post_stats"] = _row_stats(st["h"], case["post"]) if case["post"] != "none" else None
            st["pre_stats"] = _row_stats(st["y"], case["pre"]) if case["pre"] != "none" else None
            st["dy"] = _randn(g, rows, c).to(s)
            st["du"] = _randn(g, rows, c).to(t) if case["pre"] != "none" else None
    else:
        t = TYPES[case["type"]]
        st["g"] = [_gradients(g, *k).to(t) for k in _groups(case)]
        if case["op"] == "muon":
            st["p"] = [_randn(g, k, r, c) * c ** -0.5 for k, r, c in _groups(case)]
            st["m"] = [4 * _gradients(g, *k) for k in _groups(case)]
            st["copy"] = [torch.zeros_like(p, dtype=torch.bfloat16) for p in st["p"]] if case["copy"] else None
    if own:
        _handles(st)
    return st


def _handles(st):
    """The output buffers, workspaces and the optimiser that a program keeps between steps."""
    from quantized_halo_aggregation_amd import binding as B
    case = st["case"]
    if case["op"] == "norm":
        rows, c, t, s = case["samples"] * case["positions"], case["c"], TYPES[case["type"]], TYPES[case["stream"]]
        new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device=DEV)
        post, pre = case["post"] != "none", case["pre"] != "none"
        st["kind"] = {"none": B.ROW_NONE, "rms": B.ROW_RMS, "layer": B.ROW_LAYER}
        if case["way"] == "fwd":
            st["out"] = {"y": new(rows, c, dtype=s), "u": new(rows, c, dtype=t) if pre else None,
                         "post_stats": new(rows, 2) if post else None, "pre_stats": new(rows, 2) if pre else None}
            return
        st["out"] = {"dx": new(rows, c, dtype=s), "dh": new(rows, c, dtype=t),
                     "dgate": new(case["samples"], c, dtype=t) if case["gate"] else None,
                     **{"d%s_%s" % (side, v): new(c) if st["%s_%s" % (side, v)] is not None else None
                        for side in ("post", "pre") for v in ("w", "b")}}
        need = B.residual_norm_workspace(rows, c, case["positions"])
        st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        return
    cut = lambda stacks: [x for stack in stacks for x in stack.unbind(0)]
    if case["op"] == "ns":
        st["out"] = [torch.empty_like(x, dtype=TYPES[case["out"]]) for x in st["g"]]
        st["lists"] = cut(st["g"]), cut(st["out"])
        need = B.newton_schulz_workspace([tuple(x.shape) for x in st["lists"][0]], STEPS)
        st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        return
    st["opt"] = B.Muon(cut(st["p"]), momentum=MU, nesterov=case["nesterov"], weight_decay=DECAY, scale="spectral",
                       steps=STEPS, coefficients=COEF, eps=EPS_NS, momenta=cut(st["m"]),
                       copies=cut(st["copy"]) if case["copy"] else None)
    st["grads"] = cut(st["g"])


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    if state["case"]["op"] == "norm":
        return _norm_fwd(state) if state["case"]["way"] == "fwd" else _norm_bwd(state)
    if state["case"]["op"] == "ns":
        return {"o": [_newton_schulz(x.float()).to(TYPES[state["case"]["out"]]) for x in state["g"]]}
    return _muon(state)


def _given(d):
    return {k: v for k, v in d.items() if v is not None}


def _run_own(st):
    from quantized_halo_aggregation_amd import binding as B
    case = st["case"]
    if case["op"] == "ns":
        B.newton_schulz(*st["lists"], steps=STEPS, coefficients=COEF, eps=EPS_NS, workspace=st["ws"])
        return {"o": st["out"]}
    if case["op"] == "muon":
        st["opt"].step(st["grads"], LR)
        return _given({"p": st["p"], "m": st["m"], "copy": st["copy"]})
    o, kind = st["out"], st["kind"]
    both = dict(post=kind[case["post"]], pre=kind[case["pre"]], post_weight=st["post_w"], post_bias=st["post_b"],
                pre_weight=st["pre_w"], pre_bias=st["pre_b"], gate=st["gate"], positions=case["positions"], skip=SKIP,
                branch=BRANCH)
    if case["way"] == "fwd":
        B.residual_norm_fwd(st["x"], st["h"], o["y"], o["u"], post_stats=o["post_stats"], pre_stats=o["pre_stats"],
                            eps=EPS_ROW, **both)
    else:
        B.residual_norm_bwd(st["dy"], st["du"], st["y"], st["h"], o["dx"], o["dh"], post_stats=st["post_stats"],
                            pre_stats=st["pre_stats"], dgate=o["dgate"], dpost_weight=o["dpost_w"],
                            dpost_bias=o["dpost_b"], dpre_weight=o["dpre_w"], dpre_bias=o["dpre_b"],
                            workspace=st["ws"], **both)
    return _given(o)


def _normed(x, kind, w, b):
    """The norm of every row of x (float32), and its statistics."""
    if kind == "none":
        return x, None
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    rstd = ((x - mean).square().mean(1, keepdim=True) + EPS_ROW).rsqrt()
    y = (x - mean) * rstd * w
    return (y if b is None else y + b), torch.cat([mean, rstd], 1)


def _over_samples(gate, case):
    """A sample's gate row for each of its positions (rows, c)."""
    return gate.float().repeat_interleave(case["positions"], 0)


def _norm_fwd(st):
    case = st["case"]
    r, post_stats = _normed(st["h"].float(), case["post"], st["post_w"], st["post_b"])
    if case["gate"]:
        r = r * _over_samples(st["gate"], case)
    y = SKIP * st["x"].float() + BRANCH * r
    u, pre_stats = _normed(y, case["pre"], st["pre_w"], st["pre_b"])
    return _given({"y": y.to(st["x"].dtype), "u": u.to(st["h"].dtype) if case["pre"] != "none" else None,
                   "post_stats": post_stats, "pre_stats": pre_stats})


def _normed_bwd(dz, x, kind, stats, w, b):
    """Gradients of _normed from its result's: dx, dw, db."""
    if kind == "none":
        return dz, None, None
    mean, rstd = stats[:, :1], stats[:, 1:]
    xhat = (x - mean) * rstd
    q = dz * w
    dx = q - xhat * (q * xhat).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - q.mean(1, keepdim=True)
    return rstd * dx, (dz * xhat).sum(0), dz.sum(0) if b is not None else None


def _norm_bwd(st):
    case, out = st["case"], {}
    t = st["dy"].float()
    if case["pre"] != "none":
        dx, out["dpre_w"], out["dpre_b"] = _normed_bwd(st["du"].float(), st["y"].float(), case["pre"], st["pre_stats"],
                                                       st["pre_w"], st["pre_b"])
        t = t + dx
    e = dp = BRANCH * t
    h = st["h"].float()
    if case["gate"]:
        z = h
        if case["post"] != "none":
            z = (h - st["post_stats"][:, :1]) * st["post_stats"][:, 1:] * st["post_w"]
            z = z if st["post_b"] is None else z + st["post_b"]
        out["dgate"] = (e * z).view(case["samples"], case["positions"], -1).sum(1).to(st["h"].dtype)
        dp = e * _over_samples(st["gate"], case)
    dh, out["dpost_w"], out["dpost_b"] = _normed_bwd(dp, h, case["post"], st["post_stats"], st["post_w"], st["post_b"])
    out = {"dx": (SKIP * t).to(st["dy"].dtype), "dh": dh.to(st["h"].dtype), **out}
    return _given({k: out.get(k) for k in ("dx", "dh", "dgate", "dpost_w", "dpost_b", "dpre_w", "dpre_b")})


def _newton_schulz(x):
    """Newton-Schulz of a stack of equal matrices in float32."""
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2).contiguous() if tall else x
    x = x / (x.double().square().sum((1, 2), keepdim=True).sqrt() + EPS_NS).float()
    a, b, c = COEF
    for _ in range(STEPS):
        s = x @ x.transpose(1, 2).contiguous()
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.transpose(1, 2) if tall else x


def _muon(st):
    case = st["case"]
    for i, (_, rows, cols) in enumerate(_groups(case)):
        g = st["g"][i].float()
        m = st["m"][i].mul_(MU).add_(g)
        o = _newton_schulz(g + MU * m if case["nesterov"] else m)
        p = st["p"][i].mul_(1 - LR * DECAY).sub_(LR * max(1.0, rows / cols) ** 0.5 * o)
        if case["copy"]:
            st["copy"][i].copy_(p)
    return _given({"p": st["p"], "m": st["m"], "copy": st["copy"]})


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _polar(u):
    """Newton-Schulz in float64, by products on the shorter side: X (a I + b S + c S^2) with S = X^T X, or the same
    from the left."""
    a, b, c = COEF
    u = u / (torch.linalg.matrix_norm(u, keepdim=True) + EPS_NS)
    short = min(u.shape[1:])
    eye = torch.eye(short, dtype=torch.float64, device=DEV).expand(u.shape[0], -1, -1)
    left = u.shape[1] <= u.shape[2]
    for _ in range(STEPS):
        ut = u.mT.contiguous()
        s = torch.bmm(u, ut) if left else torch.bmm(ut, u)
        w = torch.baddbmm(a * eye, s, b * eye + c * s)
        u = torch.bmm(w, u) if left else torch.bmm(u, w)
    return u


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] != "norm":
        u = [x.double() for x in st["g"]]
        if case["op"] == "ns":
            return {"o": [_polar(x) for x in u]}
        m = [MU * x.double() + y for x, y in zip(st["m"], u)]
        o = [_polar(MU * x + y if case["nesterov"] else x) for x, y in zip(m, u)]
        size = [math.sqrt(max(1.0, r / c)) for _, r, c in _groups(case)]
        p = [x.double() - LR * DECAY * x.double() - LR * s * y for x, s, y in zip(st["p"], size, o)]
        return _given({"p": p, "m": m, "copy": p if case["copy"] else None})
    d = {k: v.double() for k, v in st.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    n, c = case["samples"], case["c"]
    apart = lambda x: x.view(n, -1, c)                                    # samples, positions, channels
    gate = d["gate"][:, None] if case["gate"] else torch.ones(n, 1, c, dtype=torch.float64, device=DEV)

    def norm(x, side):
        w = d.get(side + "_w", torch.ones(c, dtype=torch.float64, device=DEV))
        b = d.get(side + "_b", torch.zeros(c, dtype=torch.float64, device=DEV))
        if case[side] == "none":
            return x, None
        mean = x.sum(2, keepdim=True) / c if case[side] == "layer" else 0 * x[..., :1]
        rstd = 1 / torch.sqrt(((x - mean) ** 2).sum(2, keepdim=True) / c + EPS_ROW)
        return torch.addcmul(b, (x - mean) * rstd, w), torch.cat([mean, rstd], 2).view(-1, 2)

    if case["way"] == "fwd":
        z, post_stats = norm(apart(d["h"]), "post")
        y = SKIP * apart(d["x"]) + BRANCH * gate * z
        u, pre_stats = norm(y, "pre")
        return _given({"y": y.view(-1, c), "u": u.view(-1, c) if case["pre"] != "none" else None,
                       "post_stats": post_stats, "pre_stats": pre_stats})
    out = {}

    def back(dz, x, side):
        """The gradient through the norm's Jacobian: rstd (P q), P taking out xhat and, for layer norms, the ones."""
        if case[side] == "none":
            return dz
        s = apart(d[side + "_stats"].repeat_interleave(c, 1).view(-1, 2 * c)[:, :c]), apart(
            d[side + "_stats"].repeat_interleave(c, 1).view(-1, 2 * c)[:, c:])
        hat = (x - s[0]) * s[1]
        out["d%s_w" % side] = torch.einsum("npc,npc->c", dz, hat)
        out["d%s_b" % side] = dz.sum((0, 1)) if side + "_b" in d else None
        q = dz * d[side + "_w"]
        along = (q * hat).sum(2, keepdim=True) / c
        level = q.sum(2, keepdim=True) / c if case[side] == "layer" else 0
        return (q - level - hat * along) * s[1]

    t = apart(d["dy"])
    if case["pre"] != "none":
        t = t + back(apart(d["du"]), apart(d["y"]), "pre")
    h = apart(d["h"])
    if case["gate"]:
        z = h
        if case["post"] != "none":
            z = (h - apart(d["post_stats"][:, :1].expand(-1, c).contiguous())) * apart(
                d["post_stats"][:, 1:].expand(-1, c).contiguous()) * d["post_w"]
            z = z + d["post_b"] if "post_b" in d else z
        out["dgate"] = BRANCH * (t * z).sum(1)
    dh = back(BRANCH * t * gate, h, "post")
    out["dx"], out["dh"] = (SKIP * t).reshape(-1, c), dh.reshape(-1, c)
    return _given({k: out.get(k) for k in ("dx", "dh", "dgate", "dpost_w", "dpost_b", "dpre_w", "dpre_b")})
