"""Newton-Schulz with the kernels' roundings of the operands, and inputs that are hard on them.

The bounds are fixed numbers, not taken from the kernels' form: on matrices of low rank, or with
few rows that are not zero, rounding that reaches directions the matrix lacks grows by the first
coefficient in every later step.  They are one and a half to two times the largest error that the
form below has over these inputs."""
import torch

MUON = (3.4445, -4.7750, 2.0315)
LOW = 4e-3    # shorter side of 8 and more: low rank, few rows, gradients of few samples
ANY = 1e-2    # any input: also matrices of 2 or 3 rows, and constant ones, whose values round alike
MORE = 5e-3   # LOW's inputs by 8 steps


def r16(t, scale):
    return (t * scale).half().double() / scale


def kernel_form(g, steps=5, coef=MUON, eps=1e-7):
    """X * 2^6, A * 2^12 and B in float16, what that leaves of B's diagonal beside a X in float32;
    in the last two steps and for a single row the whole diagonal is beside a X."""
    x = g.detach().cpu().double()
    flip = x.shape[-2] > x.shape[-1]
    x = x.mT.contiguous() if flip else x
    x = (x / (x.flatten(-2).norm(dim=-1)[..., None, None] + eps)).float().double()
    a, b, c = coef
    for k in range(steps):
        xh = r16(x, 64.0)
        gram = r16(xh @ xh.mT.contiguous(), 4096.0)
        poly = b * gram + c * (gram @ gram.mT.contiguous())
        diag = poly.diagonal(dim1=-2, dim2=-1)[..., None]
        whole = steps - 1 - k < 2 or x.shape[-2] == 1
        beside = diag if whole else diag - r16(diag, 1.0)
        inside = r16(poly - torch.diag_embed(beside[..., 0]), 1.0)
        x = ((a + beside) * x + inside @ xh).float().double()
    return x.mT if flip else x


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def rank(m, n, k, seed=0):
    return rand(m, k, seed=seed) @ rand(k, n, seed=seed + 1)


def rows(m, n, k, seed=0):
    """k rows of one direction, the others zero."""
    g = torch.zeros(m, n)
    g[torch.randperm(m, generator=torch.Generator().manual_seed(seed))[:k]] = rank(k, n, 1, seed)
    return g


def softmax_gradient(batch, classes, dim, seed=0):
    """A classifier's weight gradient from `batch` samples: of that rank at most."""
    z = rand(batch, classes, seed=seed).softmax(1)
    z[torch.arange(batch), torch.arange(batch) * 7 % classes] -= 1
    return z.t() @ rand(batch, dim, seed=seed + 5) / batch


def low_inputs(m, n):
    """Matrices of m x n (8 and more) that lack directions."""
    r = min(m, n)
    yield "rank 1", rank(m, n, 1)
    yield "rank 2", rank(m, n, 2, seed=3)
    yield "rank r/2", rank(m, n, r // 2, seed=6)
    yield "3 rows", rows(m, n, 3, seed=9)
    yield "4 rows", rows(m, n, 4, seed=12)
    yield "1 sample", softmax_gradient(1, m, n, seed=15)
    yield "4 samples", softmax_gradient(4, m, n, seed=18)


def other_inputs(m, n):
    yield "gauss", rand(m, n, seed=21)
    yield "constant", torch.ones(m, n)
    yield "identity", torch.eye(m, n)
    yield "rank 1", rank(m, n, 1, seed=24)
