"""Plain 64-bit forms of the dense operators, and the error bounds of 32-bit kernels.

U is float32's half step.  The bounds are first-order: every operation of the kernel's formula
is off by at most U relative, a sum by at most U times its longest chain of additions times the
sum of magnitudes, and the result's rounding by half a step of its type."""
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}  # below its normals


def d(t):
    return None if t is None else t.detach().cpu().double()


def chain(cols):
    """Longest chain of additions over a row: 64 lanes at least share it, then join."""
    return cols / 64 + 16


def ln_forward(x, w, b, eps):
    x = d(x)
    mu = x.mean(-1, keepdim=True)
    rs = 1 / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    h = (x - mu) * rs
    y = h * (1 if w is None else d(w)) + (0 if b is None else d(b))
    return y, mu[..., 0], rs[..., 0]


def ln_forward_bounds(x, w, b, eps):
    y, mu, rs = ln_forward(x, w, b, eps)
    x64 = d(x)
    k = chain(x.shape[-1]) * U
    m, r = mu[..., None], rs[..., None]
    e_mu = k * x64.abs().mean(-1, keepdim=True) + U * m.abs()
    e_rs = r * (k + 6 * U + (r * e_mu) ** 2 / 2)       # the variance is taken about the rounded mean
    h = (x64 - m) * r
    e_h = r * (e_mu + U * (x64.abs() + m.abs())) + h.abs() * (e_rs / r + 2 * U)
    aw = 1.0 if w is None else d(w).abs()
    ab = 0.0 if b is None else d(b).abs()
    e_y = HALF[x.dtype] * y.abs() + TINY[x.dtype] + 2 * (aw * e_h + 3 * U * (aw * h.abs() + ab))
    return e_y, (2 * e_mu)[..., 0], (2 * e_rs)[..., 0]


def ln_backward(dy, x, mu, rs, w):
    dy, x, m, r = d(dy), d(x), d(mu)[..., None], d(rs)[..., None]
    h = (x - m) * r
    z = dy * (1 if w is None else d(w))
    dx = r * (z - z.mean(-1, keepdim=True) - h * (z * h).mean(-1, keepdim=True))
    axes = tuple(range(x.dim() - 1))
    return dx, (dy * h).sum(axes), dy.sum(axes)


def ln_backward_bounds(dy, x, mu, rs, w, wdtype):
    dx, dw, db = ln_backward(dy, x, mu, rs, w)
    dy64, x64, m, r = d(dy), d(x), d(mu)[..., None], d(rs)[..., None]
    h = ((x64 - m) * r).abs()
    e_h = U * (3 * h + r * (x64.abs() + m.abs()))
    z = (dy64 * (1 if w is None else d(w))).abs()
    k = chain(x.shape[-1]) * U
    m1 = z.mean(-1, keepdim=True)
    m2 = (z * h).mean(-1, keepdim=True)
    e_m2 = k * m2 + (z * e_h).mean(-1, keepdim=True) + 3 * U * m2
    e_dx = r * (4 * U * (z + m1 + h * m2) + (k + 2 * U) * m1 + h * e_m2 + e_h * m2)
    e_dx = HALF[x.dtype] * dx.abs() + TINY[x.dtype] + 2 * e_dx
    axes = tuple(range(x.dim() - 1))
    rows = max(1, x.numel() // x.shape[-1])
    kr = min(rows, 256 + rows / 128) * U               # rows one partial sum takes, at most
    a = dy64.abs()
    e_dw = HALF[wdtype] * dw.abs() + 2 * ((kr + 4 * U) * (a * h).sum(axes) + (a * e_h).sum(axes))
    e_db = HALF[wdtype] * db.abs() + 2 * (kr + 2 * U) * a.sum(axes)
    t = TINY[wdtype]
    return e_dx, e_dw + t, e_db + t


def newton_schulz(g, steps=5, coef=(3.4445, -4.7750, 2.0315), eps=1e-7, rounded=False,
                  on="cpu"):
    """The iteration in 64 bits; `rounded` puts in the kernels' roundings of the operands to
    float16 (X * 2^6, A * 2^12, B but for its diagonal) and nothing else."""
    def r16(t, s):
        return (t * s).half().double() / s if rounded else t
    x = g.detach().to(on).double()
    flip = x.shape[-2] > x.shape[-1]
    x = x.mT.contiguous() if flip else x
    x = x / (x.flatten(-2).norm(dim=-1)[..., None, None] + eps)
    a, b, c = coef
    for _ in range(steps):
        xh = r16(x, 64.0)
        gram = r16(xh @ xh.mT.contiguous(), 4096.0)
        poly = b * gram + c * (gram @ gram.mT.contiguous())
        diag = poly.diagonal(dim1=-2, dim2=-1)[..., None]
        x = (a + diag) * x + r16(poly - torch.diag_embed(diag[..., 0]), 1.0) @ xh
    return x.mT if flip else x


def ns_error_bound(g, **kw):
    """How far (norm) a result may be from the iteration in 64 bits: twice what the operands'
    roundings alone do on these inputs (the kernel's are other samples of the same roundings:
    sums in another order move some by a step), and float32 sums."""
    ref = newton_schulz(g, **kw)
    em = newton_schulz(g, rounded=True, **kw)
    steps = kw.get("steps", 5)
    rel = 2 * (em - ref).flatten(-2).norm(dim=-1) + \
        steps * (16 + max(g.shape[-2:]) / 32) * U * ref.flatten(-2).norm(dim=-1)
    return ref, rel


def within(got, ref, bound, what):
    got = d(got)
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)} vs {tuple(ref.shape)}"
    bad = ~((got - ref).abs() <= bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        b = bound[i] if torch.is_tensor(bound) else bound
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; first "
                             f"at {i}: got {float(got[i])!r}, 64 bits {float(ref[i])!r}, bound "
                             f"{float(b):.3g}")
