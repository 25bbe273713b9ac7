"""Plain 64-bit forms of the loss over a table of classes and of dropout, and the error bounds of
32-bit kernels.

U is float32's half step.  Bounds are first-order, and count for every output: the sum of K products
(K additions, each off by at most a step, 2 U, of the sum of magnitudes so far: the matrix cores may
cut instead of rounding), the operands' own rounding where float32 is taken as two float16, the
exponential (its argument's two roundings and its own), and the result's rounding."""
import numpy as np
import torch

from tests.dense_ref import HALF, TINY, U

IGNORED = -100


def d(t):
    return None if t is None else t.detach().double()


def product_bound(a, b, k, split):
    """How far a product of matrices a (m x k) and b (k x n) may be off, from magnitudes."""
    a, b = a.abs(), b.abs()
    m = a @ b
    # below 2^-126 a step is 2^-149 whatever the value: one for each product and each addition
    e = 2 * U * (k + 8) * m + 2 * (k + 8) * 2.0 ** -149
    if split:
        # a = hi + lo + r: |r| <= 2^-22 |a|, or half of float16's smallest step at a scale that
        # brings the largest value to 2^14 at least; lo lo, left out, is 2^-22 |a b| at most
        e = e + 3 * 2.0 ** -22 * m
        ea = 2.0 ** -39 * (a.max() if a.numel() else 0.0)
        eb = 2.0 ** -39 * (b.max() if b.numel() else 0.0)
        e = e + ea * b.sum(0, keepdim=True) + eb * a.sum(1, keepdim=True)
    return e


def clean(x, targets):
    """x in 64 bits with the rows that are ignored as zeros."""
    return torch.where((targets != IGNORED)[:, None], d(x), 0.0)


def forward(x, w, targets, reduction, e):
    """(loss, lse, bound of loss, bound of lse)."""
    valid = targets != IGNORED
    xc, wd = clean(x, targets), d(w)
    z = xc @ wd.T
    ez = product_bound(xc, wd.T.contiguous(), x.shape[1], x.dtype == torch.float32)
    lse = torch.logsumexp(z, 1)
    top = z.max(1, keepdim=True).values
    p = torch.exp(z - lse[:, None])
    # sums of exponentials: a tile's additions (64 in a lane, then joins), in 64 bits from there
    e_lse = (p * (ez + 3 * U * (top - z))).sum(1) + 100 * U + U * lse.abs()
    at = targets.clamp(min=0)[:, None]
    loss = lse - (1 - e) * z.gather(1, at)[:, 0] - e * z.mean(1)
    e_loss = e_lse + ez.gather(1, at)[:, 0] + U * loss.abs() + U * e
    if e:
        e_loss = e_loss + e * (ez.mean(1) + 100 * U * z.abs().mean(1))
    loss, e_loss = torch.where(valid, loss, 0.0), torch.where(valid, e_loss, 0.0)
    lse, e_lse = torch.where(valid, lse, 0.0), torch.where(valid, e_lse, 0.0)
    if reduction != "none":
        n = valid.sum().clamp(min=1) if reduction == "mean" else 1
        loss, e_loss = loss.sum() / n, e_loss.sum() / n
        e_loss = e_loss + U * loss.abs()
    return loss, lse, 2 * e_loss, 2 * e_lse


def factors(dloss, targets, reduction):
    valid = targets != IGNORED
    c = d(dloss).expand(len(targets))
    if reduction == "mean":
        c = c / valid.sum().clamp(min=1)
    return torch.where(valid, c, 0.0)


def backward(dloss, x, w, targets, lse, reduction, e):
    """(dx, dweight, bound of dx, bound of dweight)."""
    split = x.dtype == torch.float32
    xc, wd = clean(x, targets), d(w)
    c = factors(dloss, targets, reduction)
    z = xc @ wd.T
    ez = product_bound(xc, wd.T.contiguous(), x.shape[1], split)
    p = torch.exp(z - d(lse)[:, None])
    y = torch.full_like(z, e / w.shape[0])
    y.scatter_add_(1, targets.clamp(min=0)[:, None], torch.full_like(z[:, :1], 1 - e))
    valid = (targets != IGNORED)[:, None]
    g = torch.where(valid, c[:, None] * (p - y), 0.0)
    # an exponential below float32's smallest normal value, 2^-126, may come out as zero
    eg = c[:, None].abs() * (p * (ez + 3 * U * (z - d(lse)[:, None]).abs() + 6 * U) + 6 * U * y
                             + 2 * U * (p - y).abs() + 2.0 ** -126)
    top = c.abs().max() if c.numel() else 0.0
    # g's own rounding; float16 holds it times a power of two that brings the largest factor to
    # 2^13 at least
    if split:
        eg = eg + 2.0 ** -22 * g.abs() + top * 2.0 ** -38
    else:
        eg = eg + HALF[x.dtype] * g.abs() + (top * 2.0 ** -38 if x.dtype == torch.float16 else 0.0)
    eg = torch.where(valid, eg, 0.0)
    dx, dw = g @ wd, g.T @ xc
    e_dx = eg @ wd.abs() + product_bound(g, wd, w.shape[0], split)
    e_dw = eg.T @ xc.abs() + product_bound(g.T.contiguous(), xc, len(targets), split)
    t = x.dtype
    return (dx, dw, HALF[t] * dx.abs() + TINY[t] + 2 * e_dx,
            HALF[t] * dw.abs() + TINY[t] + 2 * e_dw)


def within(got, ref, bound, what):
    got = got.detach().double().cpu()
    ref, bound = ref.cpu(), torch.as_tensor(bound).cpu()
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)} vs {tuple(ref.shape)}"
    bad = ~((got - ref).abs() <= bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; first at "
                             f"{i}: got {float(got[i])!r}, 64 bits {float(ref[i])!r}, bound "
                             f"{float(bound.expand_as(ref)[i]):.3g}")


# ---- dropout --------------------------------------------------------------------------------

def philox(counter, key):
    """Philox4x32-10 of counters [n, 4] under a key of two words, in Python's own integers' stead
    unsigned 64-bit ones: [n, 4] of 32 bits."""
    u = np.uint64
    c = [np.asarray(counter)[:, k].astype(u) for k in range(4)]
    low, by = u(0xFFFFFFFF), u(32)
    k = [int(key[0]), int(key[1])]
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> by) ^ c[1] ^ u(k[0]), b & low, (a >> by) ^ c[3] ^ u(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1)


def bits16(first, count, seed, offset):
    """The 16 bits of values first .. first + count - 1."""
    chunks = np.arange(first // 8, (first + count + 7) // 8, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    ctr = np.stack([chunks & low, chunks >> np.uint64(32), np.full_like(chunks, offset & 0xFFFFFFFF),
                    np.full_like(chunks, offset >> 32)], 1)
    words = philox(ctr, (seed & 0xFFFFFFFF, seed >> 32)).astype("<u4")
    return words.view("<u2").reshape(-1)[first % 8:first % 8 + count]


def kept(shape, p, seed, offset=0):
    n = int(np.prod(shape))
    return torch.from_numpy(bits16(0, n, seed, offset) >= round(p * 65536)).view(shape)


def dropout(x, p, seed, offset=0, residual=None):
    """(y in 64 bits, its bound): the factor, the product and the sum are rounded once each, and
    then the result."""
    q = round(p * 65536)
    x64 = x.detach().cpu().double()
    keep = kept(x.shape, p, seed, offset)
    y = torch.where(keep, x64 * (65536 / (65536 - q) if q < 65536 else 0.0), 0.0)
    e = 2 * U * y.abs()
    if residual is not None:
        y = y + residual.detach().cpu().double()
        e = e + U * y.abs()
    return y, e + HALF[x.dtype] * y.abs() + TINY[x.dtype]
