"""The dense operators that stand between a table's looked-up rows and its loss, as measured cases.

Layer norm's forward and backward pass, the Newton-Schulz orthogonalisation of a gradient matrix, and the
Muon step that applies it to a weight.  A case is one call of one of them.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
COEF = (3.4445, -4.7750, 2.0315)  # x -> a x + b x^3 + c x^5 on every singular value
STEPS, NS_EPS, LN_EPS = 5, 1e-7, 1e-5
LR, MOMENTUM, DECAY = 3e-4, 0.95, 0.1


def listed():
    return [
        # four tokens of one decoding step
        {"name": "ln forward 4x1024 bf16", "op": "ln_forward", "rows": 4, "cols": 1024, "dtype": "bf16", "wdtype": "bf16"},
        # one batch of lookups out of the 128-column table, normalised before the dense layers
        {"name": "ln forward 65536x128 f32", "op": "ln_forward", "rows": 65536, "cols": 128, "dtype": "f32", "wdtype": "f32"},
        # a ragged batch at an odd width
        {"name": "ln forward 4099x1001 f16", "op": "ln_forward", "rows": 4099, "cols": 1001, "dtype": "f16", "wdtype": "f32"},
        # that batch's gradient on its way back to the table
        {"name": "ln backward 65536x128 f32", "op": "ln_backward", "rows": 65536, "cols": 128, "dtype": "f32", "wdtype": "f32"},
        # a training batch of a wide model, weights kept in 32 bits
        {"name": "ln backward 16384x4096 bf16", "op": "ln_backward", "rows": 16384, "cols": 4096, "dtype": "bf16", "wdtype": "f32"},
        # few rows at a width that is no multiple of a vector
        {"name": "ln backward 777x5003 bf16", "op": "ln_backward", "rows": 777, "cols": 5003, "dtype": "bf16", "wdtype": "bf16"},
        # one small projection: latency
        {"name": "orthogonalise 128x128 bf16", "op": "newton_schulz", "batch": 1, "m": 128, "n": 128, "dtype": "bf16"},
        # the up-projections of 16 experts at once
        {"name": "orthogonalise 16x1024x512 bf16", "op": "newton_schulz", "batch": 16, "m": 1024, "n": 512, "dtype": "bf16"},
        # one square projection of a wide model, gradient accumulated in 32 bits
        {"name": "orthogonalise 4096x4096 f32", "op": "newton_schulz", "batch": 1, "m": 4096, "n": 4096, "dtype": "f32"},
        # the projection that takes 128-column rows to an odd number of classes
        {"name": "muon step 1001x128 f32", "op": "muon_step", "batch": 1, "m": 1001, "n": 128, "dtype": "f32", "pdtype": "f32"},
        # a square projection, 32-bit weights and 16-bit gradients
        {"name": "muon step 1024x1024 bf16", "op": "muon_step", "batch": 1, "m": 1024, "n": 1024, "dtype": "bf16", "pdtype": "f32"},
        # a wide model's down-projection, all in 16 bits but the momentum
        {"name": "muon step 2048x8192 bf16", "op": "muon_step", "batch": 1, "m": 2048, "n": 8192, "dtype": "bf16", "pdtype": "bf16"},
    ]


def _between(rng, low, high):
    """A whole number, its logarithm uniform over [low, high]."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["ln_forward", "ln_backward", "newton_schulz", "muon_step"])
    if op in ("ln_forward", "ln_backward"):
        cols = _between(rng, 16, 16384)
        rows = _between(rng, 1, min(131072, (16384 * 4096) // cols))
        dtype = rng.choice(["f32", "bf16", "f16"])
        if dtype == "f32":
            rows = max(1, rows // 2)
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "wdtype": rng.choice(["f32", dtype])}
    m, n = _between(rng, 16, 4096), _between(rng, 16, 4096)
    most = max(1, min(32, 4096 ** 2 // (m * n)))
    case = {"op": op, "batch": _between(rng, 1, most), "m": m, "n": n, "dtype": rng.choice(["f32", "bf16"])}
    if op == "muon_step":
        case["pdtype"] = rng.choice(["f32", "bf16"])
    return case


def _gradient(case, gen):
    """Gradients of weights: a few strong directions (the batch's) over noise."""
    b, m, n = case["batch"], case["m"], case["n"]
    k = max(1, min(16, m // 4, n // 4))
    fall = torch.logspace(0, -1, k, device="cuda")[:, None]
    left = torch.randn(b, m, k, device="cuda", generator=gen)
    right = torch.randn(b, k, n, device="cuda", generator=gen) * fall
    g = torch.matmul(left, right) + 0.3 * torch.randn(b, m, n, device="cuda", generator=gen)
    return (g * 1e-3).to(DTYPES[case["dtype"]])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] in ("ln_forward", "ln_backward"):
        t, w = DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
        shape, cols = (case["rows"], case["cols"]), case["cols"]
        # activations: a mean that is not zero and a few columns much larger than the others
        x = torch.randn(shape, device="cuda", generator=gen) + 0.5
        x = x * (1 + 9 * (torch.rand(cols, device="cuda", generator=gen) < 0.02))
        s["x"] = x.to(t)
        s["weight"] = (1 + 0.1 * torch.randn(cols, device="cuda", generator=gen)).to(w)
        s["bias"] = (0.1 * torch.randn(cols, device="cuda", generator=gen)).to(w)
        if case["op"] == "ln_backward":
            s["dy"] = torch.randn(shape, device="cuda", generator=gen).to(t)
            xd = s["x"].double()  # what the forward pass kept
            s["mean"] = xd.mean(1).float()
            s["rstd"] = (1 / torch.sqrt(xd.var(1, unbiased=False) + LN_EPS)).float()
        return s
    s["grad"] = _gradient(case, gen)
    if case["op"] == "muon_step":
        shape = s["grad"].shape
        s["params"] = (torch.randn(shape, device="cuda", generator=gen) / math.sqrt(case["n"])).to(DTYPES[case["pdtype"]])
        s["momentum_buf"] = 8 * _gradient(dict(case, dtype="f32"), gen)  # a mean over the steps before
        s["scale"] = 0.2 * math.sqrt(max(case["m"], case["n"]))  # updates of root mean square near 0.2
    return s


def _orthogonal(g):
    """The Newton-Schulz iteration in 32 bits."""
    flip = g.shape[-2] > g.shape[-1]
    x = g.mT if flip else g
    x = x / (torch.sqrt((x * x).sum((-2, -1), keepdim=True)) + NS_EPS)
    for _ in range(STEPS):
        a = x @ x.mT
        x = COEF[0] * x + (COEF[1] * a + COEF[2] * (a @ a)) @ x
    return x.mT if flip else x


def run(state):
    op = state["op"]
    if own:
        import lazy_optimizer_step_amd as L
        if op == "ln_forward":
            y, mean, rstd = L.layer_norm_forward(state["x"], state["weight"], state["bias"], eps=LN_EPS)
            return {"y": y, "mean": mean, "rstd": rstd}
        if op == "ln_backward":
            dx, dw, db = L.layer_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"], state["weight"])
            return {"dx": dx, "dweight": dw, "dbias": db}
        if op == "newton_schulz":
            return {"out": L.newton_schulz(state["grad"], steps=STEPS, coefficients=COEF, eps=NS_EPS)}
        L.muon_step(state["params"], state["grad"], state["momentum_buf"], lr=LR, momentum=MOMENTUM, nesterov=True, weight_decay=DECAY,
                    scale=state["scale"], steps=STEPS, coefficients=COEF, eps=NS_EPS)
        return {"params": state["params"], "momentum_buf": state["momentum_buf"]}
    if op == "ln_forward":
        x = state["x"].float()
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = 1 / torch.sqrt((c * c).mean(1) + LN_EPS)
        y = c * rstd[:, None] * state["weight"].float() + state["bias"].float()
        return {"y": y.to(state["x"].dtype), "mean": mean, "rstd": rstd}
    if op == "ln_backward":
        dy, x, rstd = state["dy"].float(), state["x"].float(), state["rstd"][:, None]
        xhat = (x - state["mean"][:, None]) * rstd
        wdy = dy * state["weight"].float()
        dx = rstd * (wdy - wdy.mean(1, keepdim=True) - xhat * (wdy * xhat).mean(1, keepdim=True))
        w = state["weight"].dtype
        return {"dx": dx.to(state["x"].dtype), "dweight": (dy * xhat).sum(0).to(w), "dbias": dy.sum(0).to(w)}
    g = state["grad"].float()
    if op == "newton_schulz":
        return {"out": _orthogonal(g).to(torch.bfloat16)}
    p, buf = state["params"], state["momentum_buf"]
    buf.mul_(MOMENTUM).add_(g)
    o = _orthogonal(g + MOMENTUM * buf)
    p.copy_((1 - LR * DECAY) * p.float() - (LR * state["scale"]) * o)
    return {"params": p, "momentum_buf": buf}


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if case["op"] in ("ln_forward", "ln_backward"):
        rows, cols, e, w = case["rows"], case["cols"], size[case["dtype"]], size[case["wdtype"]]
        if case["op"] == "ln_forward":
            return {"bytes": 2 * rows * cols * e + 2 * cols * w + 8 * rows, "flops": 8 * rows * cols}
        return {"bytes": 3 * rows * cols * e + 3 * cols * w + 8 * rows, "flops": 15 * rows * cols}
    b, r, c = case["batch"], min(case["m"], case["n"]), max(case["m"], case["n"])
    # both products with a symmetric result need half of it
    flops = STEPS * b * (r * r * c + r * r * r + 2 * r * r * c)
    values = b * r * c
    if case["op"] == "newton_schulz":
        return {"bytes": values * (size[case["dtype"]] + 2), "flops": flops}
    return {"bytes": values * (size[case["dtype"]] + 2 * size[case["pdtype"]] + 8), "flops": flops}


def _polynomial64(u):
    """The same iteration of a stack of matrices in 64 bits, on the side of the Gram matrix that is smaller."""
    a, b, c = COEF
    u = u / (u.flatten(1).norm(dim=1)[:, None, None] + NS_EPS)
    tall = u.shape[1] > u.shape[2]
    eye = torch.eye(min(u.shape[1:]), dtype=torch.float64, device=u.device)
    for _ in range(STEPS):
        gram = torch.matmul(u.mT.contiguous(), u) if tall else torch.matmul(u, u.mT.contiguous())
        p = a * eye + torch.matmul(gram, b * eye + c * gram)
        u = torch.matmul(u, p) if tall else torch.matmul(p, u)
    return u


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("ln_forward", "ln_backward"):
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=-1, unbiased=False, keepdim=True)
        sigma = torch.sqrt(var + LN_EPS)
        z = (x - mean) / sigma
        if case["op"] == "ln_forward":
            return {"y": torch.addcmul(s["bias"].double(), z, s["weight"].double()), "mean": mean[:, 0], "rstd": 1 / sigma[:, 0]}
        dy = s["dy"].double()
        dz = dy * s["weight"].double()
        # the gradient with respect to x: dz with its parts along 1 and along z taken out, over sigma
        n = case["cols"]
        dx = (dz - (dz.sum(1, keepdim=True) + z * (dz * z).sum(1, keepdim=True)) / n) / sigma
        return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, z), "dbias": dy.sum(0)}
    g = s["grad"].double()
    if case["op"] == "newton_schulz":
        return {"out": _polynomial64(g)}
    buf = s["momentum_buf"].double() * MOMENTUM + g
    p = s["params"].double() * (1 - LR * DECAY)
    return {"params": p - LR * s["scale"] * _polynomial64(g + MOMENTUM * buf), "momentum_buf": buf}
