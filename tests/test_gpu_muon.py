"""The Newton-Schulz iteration and the Muon step against their formulas in 64 bits."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from tests import dense_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def matrix(*shape, kind="low", seed=0):
    g = torch.Generator().manual_seed(seed + sum((k + 1) * s for k, s in enumerate(shape)))
    m, n = shape[-2:]
    noise = torch.randn(*shape, generator=g)
    if kind == "gauss":
        return noise
    k = max(1, min(8, m // 4, n // 4))
    fall = torch.logspace(0, -1, k)[:, None]
    return torch.randn(*shape[:-1], k, generator=g) @ \
        (torch.randn(*shape[:-2], k, n, generator=g) * fall) + 0.3 * noise


def check_ns(g, **kw):
    out = L.newton_schulz(g, **kw)
    assert out.dtype == BF16 and out.shape == g.shape
    ref, bound = R.ns_error_bound(g, **kw)
    norm = ref.flatten(-2).norm(dim=-1)
    off = (R.d(out) - ref).flatten(-2).norm(dim=-1)
    assert (off <= bound + R.HALF[BF16] * norm).all(), (off / norm, bound / norm)
    return out


SHAPES = [(1, 1), (1, 9), (9, 1), (2, 3), (16, 16), (17, 16), (31, 100), (63, 64), (64, 64),
          (65, 64), (64, 65), (100, 300), (300, 100), (127, 128), (128, 128), (129, 128),
          (128, 257), (256, 256), (257, 255), (200, 1000), (1001, 128), (385, 511), (512, 640)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_shapes(shape, dtype):
    check_ns(matrix(*shape).to(dtype).cuda())


@pytest.mark.parametrize("shape", [(3, 40, 70), (2, 3, 130, 64), (5, 257, 200), (70, 17, 33),
                                   (16, 128, 128), (9, 300, 520)],
                         ids=lambda s: "x".join(map(str, s)))
def test_batches(shape):
    g = matrix(*shape).cuda()
    out = check_ns(g)
    one = g.reshape(-1, *shape[-2:])[-1].contiguous()
    # a batch may take other tiles than one matrix: the same values within their bounds
    ref, bound = R.ns_error_bound(one)
    off = (R.d(out.reshape(-1, *shape[-2:])[-1]) - ref).norm()
    assert off <= bound + R.HALF[BF16] * ref.norm()


@pytest.mark.parametrize("shape", [(1100, 1100), (700, 2100), (2048, 300), (1536, 1024)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_large(shape):
    check_ns(matrix(*shape).to(BF16).cuda())


@pytest.mark.parametrize("shape", [(2048, 2048), (4096, 4096), (4100, 4160), (5700, 5700),
                                   (3, 2000, 2500)], ids=lambda s: "x".join(map(str, s)))
def test_largest_tiles(shape):
    """Sizes that take the 96, 192 and 256 tiles; the 64-bit iteration runs on the GPU."""
    g = matrix(*shape).to(BF16).cuda()
    out = L.newton_schulz(g)
    ref, bound = R.ns_error_bound(g, on="cuda")
    off = (out.double() - ref).flatten(-2).norm(dim=-1)
    assert (off <= bound + R.HALF[BF16] * ref.flatten(-2).norm(dim=-1)).all()


@pytest.mark.parametrize("steps,coefficients", [
    (1, (3.4445, -4.7750, 2.0315)), (10, (2.0, -1.5, 0.5)), (6, (1.5, -0.5, 0.0)),
    (2, (1.875, -1.25, 0.375)), (7, (3.4445, -4.7750, 2.0315))])
@pytest.mark.parametrize("shape", [(48, 80), (200, 300)])
def test_steps_and_coefficients(steps, coefficients, shape):
    g = matrix(*shape, kind="gauss").cuda()
    out = L.newton_schulz(g, steps=steps, coefficients=coefficients)
    ref, bound = R.ns_error_bound(g, steps=steps, coef=coefficients)
    assert (R.d(out) - ref).norm() <= bound + R.HALF[BF16] * ref.norm()


@pytest.mark.parametrize("shape", [(60, 90), (300, 200)])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 1.0, 1e30])
def test_any_size_of_gradient(shape, size):
    """The norm is summed in 64 bits: nothing overflows, and small ones are held by eps alone."""
    g = (matrix(*shape).double() * size).float().cuda()
    check_ns(g)


@pytest.mark.parametrize("shape", [(4, 50, 60), (4, 260, 300)])
def test_zero_and_spoilt_matrices(shape):
    g = matrix(*shape).cuda()
    g[1] = 0
    clean = check_ns(g)
    assert not clean[1].any()
    g[2, 5, 5] = float("nan")
    out = L.newton_schulz(g)
    for k in (0, 1, 3):
        assert torch.equal(out[k], clean[k])


@pytest.mark.parametrize("shape", [(3, 100, 60), (500, 520)])
def test_repeats_streams_and_workspace(shape):
    """The same bits again, on another stream and from a workspace full of NaN."""
    g = matrix(*shape).to(BF16).cuda()
    first = check_ns(g)
    b = g.numel() // (shape[-1] * shape[-2])
    ws = torch.full((L.newton_schulz_workspace_size(b, *shape[-2:]),), 255, dtype=torch.uint8,
                    device="cuda")
    keep = g.clone()
    assert torch.equal(L.newton_schulz(g, workspace=ws), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = L.newton_schulz(g, stream=s)
    s.synchronize()
    assert torch.equal(out, first)
    assert torch.equal(g, keep)


def check_muon(p, g, buf, *, lr, momentum, nesterov, weight_decay, scale, steps=3):
    for _ in range(steps):
        b0 = buf.clone() if buf is not None else None
        before = R.d(p)
        L.muon_step(p, g, buf, lr=lr, momentum=momentum, nesterov=nesterov,
                    weight_decay=weight_decay, scale=scale)
        if momentum:
            b64 = momentum * R.d(b0) + R.d(g)
            R.within(buf, b64, 3 * R.U * ((momentum * R.d(b0)).abs() + R.d(g).abs()), "momentum")
            u = R.d(g) + momentum * R.d(buf) if nesterov else R.d(buf)
        else:
            u = R.d(g)
        ref, bound = R.ns_error_bound(u)
        p64 = (1 - lr * weight_decay) * before - lr * scale * ref
        off = (R.d(p) - p64).flatten(-2).norm(dim=-1)
        half = 3 * R.U + (R.HALF[p.dtype] if p.dtype != F32 else 0)
        most = lr * scale * bound + half * (before.flatten(-2).norm(dim=-1) +
                                            p64.flatten(-2).norm(dim=-1))
        assert (off <= most).all(), (off, most)


@pytest.mark.parametrize("shape", [(1, 5), (40, 64), (130, 70), (3, 65, 129), (256, 512),
                                   (520, 300)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("pd,gd", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)],
                         ids=["f32-f32", "f32-bf16", "bf16-bf16", "bf16-f32"])
def test_muon_types(shape, pd, gd):
    p = (matrix(*shape, kind="gauss", seed=5) * 0.05).to(pd).cuda()
    g = matrix(*shape).to(gd).cuda()
    check_muon(p, g, torch.zeros(shape, device="cuda"), lr=0.02, momentum=0.95, nesterov=True,
               weight_decay=0.1, scale=1.5)


@pytest.mark.parametrize("momentum,nesterov", [(0.0, True), (0.0, False), (0.9, False),
                                               (0.9, True)])
@pytest.mark.parametrize("shape", [(70, 40), (300, 400)])
def test_muon_momentum(momentum, nesterov, shape):
    p, g = matrix(*shape, kind="gauss", seed=3).cuda(), matrix(*shape).cuda()
    buf = matrix(*shape, seed=9).cuda() if momentum else None
    check_muon(p, g, buf, lr=0.1, momentum=momentum, nesterov=nesterov, weight_decay=0.0,
               scale=0.7)


def test_muon_without_a_step():
    """lr 0 leaves the weight as it was and still moves the momentum."""
    p, g = matrix(90, 50, seed=1).cuda(), matrix(90, 50).cuda()
    keep, buf = p.clone(), torch.zeros(90, 50, device="cuda")
    L.muon_step(p, g, buf, lr=0.0, weight_decay=0.1)
    assert torch.equal(p, keep) and torch.equal(buf, g)
    e = torch.empty(0, 4, 4, device="cuda")
    L.muon_step(e, e, e, lr=0.1)
    assert L.newton_schulz(e).shape == (0, 4, 4)


@pytest.mark.parametrize("shape", [(64, 96), (260, 300)])
def test_muon_class_and_graph(shape):
    """The optimizer object's steps, and the same steps replayed from a graph, bit for bit."""
    p0 = matrix(*shape, kind="gauss", seed=2).cuda()
    grads = [matrix(*shape, seed=k).cuda() for k in range(4)]
    a, b, c = (p0.clone() for _ in range(3))
    buf = torch.zeros(shape, device="cuda")
    opt = L.Muon(a, lr=0.02, weight_decay=0.01, adjust="rms")
    for g in grads:
        opt.step(g)
        L.muon_step(b, g, buf, lr=0.02, weight_decay=0.01, scale=0.2 * max(shape) ** 0.5)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(opt.momentum_buf, buf)
    gopt = L.Muon(c, lr=0.02, weight_decay=0.01, adjust="rms")
    g_in = torch.zeros(shape, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gopt.step(g_in)
    for g in grads:
        g_in.copy_(g)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
    assert torch.equal(c, a) and torch.equal(gopt.momentum_buf, buf)


def test_more_matrices_than_a_grid_axis_and_32_bit_offsets():
    m, n = 48, 64
    batch = (1 << 31) // (m * n) + 70
    g = torch.empty(batch, m, n, dtype=BF16, device="cuda").normal_()
    out = L.newton_schulz(g)
    for at in (0, 65534, 65535, 65536, batch - 1):
        ref, bound = R.ns_error_bound(g[at])
        assert (R.d(out[at]) - ref).norm() <= bound + R.HALF[BF16] * ref.norm()


def test_more_large_matrices_than_one_grid_takes():
    """Matrices beyond the one-launch kernel's sizes, with 32-bit offsets passed in the workspace."""
    m, n, batch = 130, 260, 40000
    g = torch.empty(batch, m, n, dtype=BF16, device="cuda").normal_()
    out = L.newton_schulz(g)
    for at in (0, 32767, 32768, 34953, batch - 1):
        ref, bound = R.ns_error_bound(g[at])
        assert (R.d(out[at]) - ref).norm() <= bound + R.HALF[BF16] * ref.norm()


@pytest.mark.parametrize("shape", [(64, 1024), (1023, 63), (128, 512), (511, 127), (2, 64, 1000),
                                   (64, 1025), (128, 513), (120, 130), (128, 256), (6, 128, 512),
                                   (6, 400, 100), (3, 520, 128), (33, 2100)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_around_the_one_launch_sizes(shape, dtype):
    check_ns(matrix(*shape).to(dtype).cuda())


@pytest.mark.parametrize("shape", [(1, 3000), (40, 5001), (5000, 64), (100, 1028), (2, 1500, 100),
                                   (128, 4096), (3, 65, 700)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("pd,gd,momentum,nesterov", [(F32, F32, 0.95, True), (BF16, BF16, 0.9, False),
                                                     (F32, BF16, 0.0, True)],
                         ids=["f32", "bf16", "plain"])
def test_muon_on_wide_matrices(shape, pd, gd, momentum, nesterov):
    """Up to 128 rows or columns and more than one block holds."""
    p = (matrix(*shape, kind="gauss", seed=5) * 0.05).to(pd).cuda()
    buf = matrix(*shape, seed=8).cuda() if momentum else None
    check_muon(p, matrix(*shape).to(gd).cuda(), buf, lr=0.02, momentum=momentum,
               nesterov=nesterov, weight_decay=0.1, scale=1.5, steps=2)


@pytest.mark.parametrize("shape", [(1, 1 << 20), ((1 << 20) - 3, 2), (130, 50001), (70000, 131)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_longest_sides(shape):
    check_ns(matrix(*shape).to(BF16).cuda())


def test_more_wide_matrices_than_one_grid_takes():
    batch, m, n = 4100, 64, 1025
    g = torch.empty(batch, m, n, dtype=BF16, device="cuda").normal_()
    out = L.newton_schulz(g)
    for at in (0, 4095, 4096, batch - 1):
        ref, bound = R.ns_error_bound(g[at])
        assert (R.d(out[at]) - ref).norm() <= bound + R.HALF[BF16] * ref.norm()


@pytest.mark.parametrize("shape", [(128, 200), (100, 900), (1500, 1500), (2048, 2100), (4100, 4096),
                                   (5, 700, 800)], ids=lambda s: "x".join(map(str, s)))
def test_graph_of_every_form(shape):
    """Captured steps replay the eager ones bit for bit, also with LDS beyond the default size."""
    p0, grad = torch.randn(shape, device="cuda"), torch.randn(shape, device="cuda")
    a, b = p0.clone(), p0.clone()
    bufs = [torch.zeros(shape, device="cuda") for _ in range(2)]
    ws = torch.empty(L.newton_schulz_workspace_size(shape[0] if len(shape) > 2 else 1,
                                                    *shape[-2:]), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    g_in = torch.zeros_like(grad)
    with torch.cuda.graph(graph):
        L.muon_step(b, g_in, bufs[1], lr=0.1, workspace=ws)
    for k in range(3):
        g = torch.roll(grad, k, -1)
        L.muon_step(a, g, bufs[0], lr=0.1)
        g_in.copy_(g)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(*bufs)


def test_validate_refuses_and_writes_nothing():
    p, g, buf = (matrix(70, 30, seed=k).cuda() for k in range(3))
    L.muon_step(p, g, buf, lr=0.1, validate=True)
    keep = p.clone(), buf.clone()
    g[69, 29] = float("nan")
    out = torch.full((70, 30), 5.0, dtype=BF16, device="cuda")
    for call in (lambda: L.muon_step(p, g, buf, lr=0.1, validate=True),
                 lambda: L.newton_schulz(g, out=out, validate=True)):
        with pytest.raises(L.SparseOptError) as e:
            call()
        assert e.value.code == -5
    torch.cuda.synchronize()
    assert torch.equal(p, keep[0]) and torch.equal(buf, keep[1]) and (out == 5.0).all()


def test_python_refusals():
    g = matrix(6, 8).cuda()
    for bad, kind in ((g.double(), TypeError), (g.half(), TypeError), (g.t(), ValueError),
                      (g[0], ValueError), (g.cpu(), ValueError), (g[:0], ValueError)):
        with pytest.raises(kind):
            L.newton_schulz(bad)
    with pytest.raises(TypeError):
        L.newton_schulz(g, out=torch.empty_like(g))
    with pytest.raises(ValueError):
        L.muon_step(g, g[:5].contiguous(), torch.zeros_like(g), lr=0.1)
    with pytest.raises(L.SparseOptError):
        L.muon_step(g, g, None, lr=0.1)
    with pytest.raises(ValueError):
        L.Muon(g, lr=0.1, adjust="other")
