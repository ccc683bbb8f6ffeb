"""Newton-Schulz orthogonalisation against the definition in 64 bits.

Tolerance. `emulate` repeats the iteration in 64 bits with the roundings that
the kernel's header states (X as hi + lo of fp16, the products on hi, A and B
rounded once to fp16 off their diagonals, the result to bf16); its distance
from the exact iteration is what the scheme itself costs on that input. The
kernels add fp32 sums: n terms, off by at most n 2^-24 of the sum of absolute
values, which moves a result by far less than its fp16 rounding except where it
flips one. So the kernels have to lie within 1.25 times the emulation's
distance, in the Frobenius norm, plus 2^-20. For matrices of at least 64 rows
and columns, where elements' roundings average out, also within 2^-8.97 of the
exact result's norm: rounding to bf16 alone is off by 1.7e-3 of it (uniform in
half a step, 2^-9 to 2^-8 of a value), and the scheme's own error, independent
of that, is below 1e-3 there (in 64-bit emulation, 2.5e-4 at 64 x 1000 to
9.6e-4 at 64 x 64): sqrt(1.7^2 + 1^2) 1e-3 < 2^-8.97.
"""
import ctypes

import pytest
import torch

from mxfp8_quantization_moe_device_b200 import binding as mxq

DEV = "cuda"
COEF = (3.4445, -4.7750, 2.0315)


def exact(g, coefs, eps=1e-7):
    x = g.double()
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + eps)
    t = x.shape[-2] > x.shape[-1]
    x = x.mT if t else x
    for a, b, c in coefs:
        A = x @ x.mT
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.mT if t else x


def emulate(g, coefs, eps=1e-7):
    def half(v, scale):
        return (v * scale).half().double() / scale

    x = g.double()
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + eps)
    t = x.shape[-2] > x.shape[-1]
    x = x.mT if t else x
    for a, b, c in coefs:
        hi = half(x, 256.0)
        x = hi + half(x - hi, 256.0 * 2048.0)
        A = hi @ hi.mT
        alpha = torch.diagonal(A, dim1=-2, dim2=-1)
        A = half(A - torch.diag_embed(alpha), 1024.0)
        D = A @ A
        beta = b * alpha + c * alpha * alpha + c * torch.diagonal(D, dim1=-2, dim2=-1)
        B = c * D + (b + c * (alpha[..., :, None] + alpha[..., None, :])) * A
        B = half(B - torch.diag_embed(torch.diagonal(B, dim1=-2, dim2=-1)), 1024.0)
        x = (a + beta)[..., None] * x + B @ hi
    x = x.mT if t else x
    return x.bfloat16().double()


def norm(x):
    return torch.linalg.vector_norm(x, dim=(-2, -1))


def matrices(E, N, K, dtype, seed, kind="gradient"):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(E, N, K, generator=g, device=DEV)
    if kind == "gradient":
        r = max(1, min(N, K) // 16)
        x = x + torch.randn(E, N, r, generator=g, device=DEV) @ torch.randn(E, r, K, generator=g, device=DEV) \
            * (2.0 / r ** 0.5)
        x = x * torch.exp(0.5 * torch.randn(E, N, 1, generator=g, device=DEV)) * 1e-3
    elif kind == "decay":  # singular values from 1 down to 1e-4
        u, s, v = torch.linalg.svd(x.double(), full_matrices=False)
        x = (u * torch.logspace(0, -4, s.shape[-1], dtype=torch.float64, device=DEV)) @ v
    return x.to(dtype)


def check(got, g, coefs, eps=1e-7):
    want = exact(g, coefs, eps)
    assert got.shape == g.shape and got.dtype == torch.bfloat16
    off, scheme, size = norm(got.double() - want), norm(emulate(g, coefs, eps) - want), norm(want)
    assert bool((off <= 1.25 * scheme + 2.0 ** -20 * size).all()), (off / size, scheme / size)
    if min(g.shape[-2:]) >= 64:
        assert bool((off <= 2.0 ** -8.97 * size).all()), off / size


# ------------------------------------------------------------ refusals (CPU)
def test_host_checks():
    L = mxq.lib()
    p = 256
    co = (ctypes.c_float * 3)(*COEF)
    bad = (ctypes.c_float * 3)(3.0, -17.0, 2.0)
    nan = (ctypes.c_float * 3)(3.0, float("nan"), 2.0)
    big = 1 << 40
    assert L.newton_schulz(p, 0, -1, 8, 8, 1, co, 1e-7, p, p, big, None) == mxq.ERR_SHAPE
    assert L.newton_schulz(p, 0, 1, 8, 8, 0, co, 1e-7, p, p, big, None) == mxq.ERR_SHAPE
    assert L.newton_schulz(p, 0, 1, 8, 8, 65, co, 1e-7, p, p, big, None) == mxq.ERR_UNSUPPORTED
    assert L.newton_schulz(p, 0, 1, 65537, 8, 1, co, 1e-7, p, p, big, None) == mxq.ERR_UNSUPPORTED
    assert L.newton_schulz(p, 3, 1, 8, 8, 1, co, 1e-7, p, p, big, None) == mxq.ERR_UNSUPPORTED
    assert L.newton_schulz(p, 0, 1, 8, 8, 1, bad, 1e-7, p, p, big, None) == mxq.ERR_UNSUPPORTED
    assert L.newton_schulz(p, 0, 1, 8, 8, 1, nan, 1e-7, p, p, big, None) == mxq.ERR_UNSUPPORTED
    assert L.newton_schulz(p, 0, 1, 8, 8, 1, co, -1.0, p, p, big, None) == mxq.ERR_UNSUPPORTED
    assert L.newton_schulz(p, 0, 1, 8, 8, 1, None, 1e-7, p, p, big, None) == mxq.ERR_NULL
    assert L.newton_schulz(None, 0, 1, 8, 8, 1, co, 1e-7, p, p, big, None) == mxq.ERR_NULL
    assert L.newton_schulz(p, 0, 1, 8, 8, 1, co, 1e-7, p + 1, p, big, None) == mxq.ERR_ALIGN
    assert L.newton_schulz(p, 0, 1, 200, 300, 1, co, 1e-7, p, p + 16, big, None) == mxq.ERR_ALIGN
    assert L.newton_schulz(p, 0, 1, 200, 300, 1, co, 1e-7, p, p, 100, None) == mxq.ERR_WORKSPACE
    assert L.newton_schulz(p, 0, 0, 8, 8, 1, co, 1e-7, None, None, 0, None) == mxq.OK
    assert L.newton_schulz(None, 0, 3, 0, 8, 1, co, 1e-7, None, None, 0, None) == mxq.OK
    assert L.newton_schulz_workspace_bytes(0, 8, 8, 5) == 0
    assert L.newton_schulz_workspace_bytes(2, 128, 2048, 5) == 0
    assert L.newton_schulz_workspace_bytes(2, 129, 2048, 5) > 0
    assert L.newton_schulz_workspace_bytes(2, 4097, 8, 5) > 0


def test_refusals_of_the_binding_and_fake_shape():
    import mxfp8_quantization_moe_device_b200.ops  # noqa: F401
    with pytest.raises(TypeError):
        mxq.newton_schulz(torch.zeros(4, 4))
    m = torch.empty(3, 20, 40, device="meta")
    out = torch.ops.mxq.newton_schulz(m, 5, list(COEF), 1e-7)
    assert out.shape == m.shape and out.dtype == torch.bfloat16


# ------------------------------------------------------------ values
SHAPES = [(1, 1, 1), (1, 1, 9), (2, 7, 1), (3, 16, 16), (2, 33, 65), (4, 96, 224), (2, 128, 128), (1, 129, 127),
          (2, 256, 64), (3, 300, 260), (2, 257, 520), (1, 513, 511), (5, 64, 1000), (1, 1409, 577), (2, 768, 1280),
          (2, 17, 255), (3, 100, 257), (1, 128, 513), (2, 900, 30), (2, 48, 1300), (1, 2048, 128), (2, 128, 2049),
          (40, 65, 300), (3, 90, 4000), (1, 4096, 128), (1, 20, 4097)]


@pytest.mark.gpu
@pytest.mark.parametrize("E,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_newton_schulz(E, N, K, dtype):
    g = matrices(E, N, K, dtype, E + N + K)
    check(mxq.newton_schulz(g), g, [COEF] * 5)
    for tile in (64, 128, 256):
        mxq.testing_set(mxq.TESTING_NS_TILE, tile)
        try:
            check(mxq.newton_schulz(g), g, [COEF] * 5)
        finally:
            mxq.testing_set(mxq.TESTING_NS_TILE, 0)
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("E,N,K", [(2, 2500, 5001), (1, 9000, 3300), (300, 130, 140)])
def test_larger(E, N, K):
    g = matrices(E, N, K, torch.bfloat16, 6)
    check(mxq.newton_schulz(g), g, [COEF] * 5)
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_more_than_2_31_elements():
    E, N, K = 260, 2050, 4100
    g = torch.randn(E, N, K, device=DEV, dtype=torch.bfloat16)
    assert g.numel() > 2 ** 31
    out = mxq.newton_schulz(g, steps=3)
    for i in (0, E // 2, E - 1):  # a matrix alone goes through the same products in other tiles
        check(out[i:i + 1], g[i:i + 1], [COEF] * 3)
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["noise", "decay"])
@pytest.mark.parametrize("N,K", [(200, 500), (384, 256)])
def test_spectra(kind, N, K):
    g = matrices(2, N, K, torch.float32, 5, kind)
    check(mxq.newton_schulz(g), g, [COEF] * 5)


@pytest.mark.gpu
def test_steps_coefficients_scale_and_shapes():
    g = matrices(2, 130, 300, torch.float32, 9)
    for steps in (1, 2, 7):
        check(mxq.newton_schulz(g, steps=steps), g, [COEF] * steps)
    co = [(4.0, -8.0, 5.0), (3.5, -5.0, 2.2), (1.875, -1.25, 0.375)]
    check(mxq.newton_schulz(g, steps=3, coefficients=co), g, co)
    # the norm is taken in 64 bits: scales whose squares leave fp32's range
    for s in (1e-18, 1e-25, 1e25):
        check(mxq.newton_schulz(g * s, eps=0.0), g * s, [COEF] * 5, eps=0.0)
    two = matrices(1, 64, 96, torch.bfloat16, 2)
    assert torch.equal(mxq.newton_schulz(two[0]), mxq.newton_schulz(two)[0])
    out = torch.empty(1, 64, 96, dtype=torch.bfloat16, device=DEV)
    assert mxq.newton_schulz(two, out=out) is out and torch.equal(out, mxq.newton_schulz(two))
    assert mxq.newton_schulz(torch.empty(0, 4, 8, device=DEV)).shape == (0, 4, 8)
    # an output that starts on a 2-byte boundary
    buf = torch.empty(64 * 96 + 1, dtype=torch.bfloat16, device=DEV)
    odd = buf[1:].view(1, 64, 96)
    assert torch.equal(mxq.newton_schulz(two, out=odd), out)


@pytest.mark.gpu
def test_zeros_nan_and_neighbours():
    g = matrices(5, 150, 270, torch.float32, 4)
    want = mxq.newton_schulz(g)
    g[1] = 0.0
    g[2, 3, 4] = float("nan")
    g[3, 149, 269] = float("inf")
    got = mxq.newton_schulz(g)
    assert torch.equal(got[0], want[0]) and torch.equal(got[4], want[4])
    assert bool((got[1] == 0).all()) and bool(got[2].isnan().all()) and bool(got[3].isnan().all())
    assert bool((mxq.newton_schulz(g[1:2], eps=0.0) == 0).all())
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_gpu_refusals():
    g = matrices(2, 64, 96, torch.float32, 4)
    for call in (lambda: mxq.newton_schulz(g.half()), lambda: mxq.newton_schulz(g.mT), lambda: mxq.newton_schulz(g[0, 0]),
                 lambda: mxq.newton_schulz(g, out=torch.empty_like(g))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: mxq.newton_schulz(g, steps=0), lambda: mxq.newton_schulz(g, steps=65),
                 lambda: mxq.newton_schulz(g, coefficients=[COEF] * 4), lambda: mxq.newton_schulz(g, coefficients=(1, 2))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mxq.newton_schulz(g, coefficients=(20.0, 0.0, 0.0)), lambda: mxq.newton_schulz(g, eps=-1.0)):
        with pytest.raises(mxq.MXQError):
            call()
    import mxfp8_quantization_moe_device_b200.ops  # noqa: F401
    torch.library.opcheck(torch.ops.mxq.newton_schulz, (g, 5, list(COEF), 1e-7),
                          test_utils=("test_schema", "test_faketensor"))
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("tile", [0, 64, 128, 256])
@pytest.mark.parametrize("E,N,K", [(2, 130, 135), (1, 700, 300), (1, 513, 1030), (2, 1100, 1030)])
def test_a_workspace_of_nans(E, N, K, tile):
    # what a call did not write itself it does not read: half of A and B, edges
    g = matrices(E, N, K, torch.bfloat16, 9)
    mxq.testing_set(mxq.TESTING_NS_TILE, tile)
    try:
        want = mxq.newton_schulz(g)
        L = mxq.lib()
        nbytes = L.newton_schulz_workspace_bytes(E, N, K, 5)
        assert nbytes > 0
        ws = torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)
        out = torch.empty_like(g)
        co = (ctypes.c_float * 15)(*(COEF * 5))
        torch.cuda.synchronize()
        assert L.newton_schulz(g.data_ptr(), 0, E, N, K, 5, co, 1e-7, out.data_ptr(), ws.data_ptr(), nbytes, None) == 0
        torch.cuda.synchronize()
    finally:
        mxq.testing_set(mxq.TESTING_NS_TILE, 0)
    assert torch.equal(out, want)


@pytest.mark.gpu
def test_out_over_its_input_is_refused():
    b = torch.randn(4, 64, 96, device=DEV).bfloat16()
    f = torch.randn(2, 64, 96, device=DEV)
    for call in (lambda: mxq.newton_schulz(b, out=b), lambda: mxq.newton_schulz(b[:2], out=b[1:3]),
                 lambda: mxq.newton_schulz(f, out=f.view(torch.bfloat16).reshape(4, 64, 96)[2:])):
        with pytest.raises(ValueError, match="overlap"):
            call()
    assert torch.equal(mxq.newton_schulz(b[:2], out=b[2:]), mxq.newton_schulz(b[:2]))


@pytest.mark.gpu
def test_streams_graph_and_repeat():
    g = matrices(3, 400, 700, torch.bfloat16, 8)
    want = mxq.newton_schulz(g)
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(mxq.newton_schulz(g))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            graphs.append((gr, mxq.newton_schulz(g)))
    g.copy_(matrices(3, 400, 700, torch.bfloat16, 18))
    torch.cuda.synchronize()
    for gr, _ in graphs:
        with torch.cuda.stream(torch.cuda.Stream()):
            gr.replay()
    torch.cuda.synchronize()
    want = mxq.newton_schulz(g)
    assert all(torch.equal(o, want) for _, o in graphs)
    check(want, g, [COEF] * 5)
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_update_from_the_weight_gradient():
    """The expert weight gradient of the FP8 grouped product, orthogonalised:
    the singular values of the update lie where the polynomial takes those of
    the normalised gradient."""
    from mxfp8_quantization_moe_device_b200.autograd import fp8_grouped_mm
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(512, 256, generator=gen, device=DEV).bfloat16()
    w = (torch.randn(3, 128, 256, generator=gen, device=DEV) * 0.05).bfloat16().requires_grad_(True)
    offs = torch.tensor([160, 160, 512], dtype=torch.int32, device=DEV)
    out = fp8_grouped_mm(x, w, offs)
    (dw,) = torch.autograd.grad(out, w, torch.randn(512, 128, generator=gen, device=DEV).bfloat16())
    up = mxq.newton_schulz(dw)
    assert bool((up[1] == 0).all())  # the expert without tokens
    check(up[[0, 2]], dw[[0, 2]], [COEF] * 5)


# ------------------------------------------------------------ large values on the way
def emulate_wide(g, coefs, b_scales, eps=1e-7):
    """`emulate` with a scale of B of its own in every step, so that B' stays
    within fp16 where singular values come near to 4."""
    def half(v, scale):
        return (v * scale).half().double() / scale

    x = g.double()
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + eps)
    t = x.shape[-2] > x.shape[-1]
    x = x.mT if t else x
    for (a, b, c), scale in zip(coefs, b_scales):
        hi = half(x, 256.0)
        x = hi + half(x - hi, 256.0 * 2048.0)
        A = hi @ hi.mT
        alpha = torch.diagonal(A, dim1=-2, dim2=-1)
        A = half(A - torch.diag_embed(alpha), 1024.0)
        D = A @ A
        beta = b * alpha + c * alpha * alpha + c * torch.diagonal(D, dim1=-2, dim2=-1)
        B = c * D + (b + c * (alpha[..., :, None] + alpha[..., None, :])) * A
        B = half(B - torch.diag_embed(torch.diagonal(B, dim1=-2, dim2=-1)), scale)
        x = (a + beta)[..., None] * x + B @ hi
    x = x.mT if t else x
    return x.bfloat16().double()


WIDE = [(2, 96, 224), (2, 224, 96), (2, 100, 257), (1, 17, 1300), (2, 300, 260), (1, 513, 1030), (1, 700, 300)]


@pytest.mark.gpu
@pytest.mark.parametrize("E,N,K", WIDE)
@pytest.mark.parametrize("second,scale", [(COEF, 64.0), ((16.0, 16.0, 16.0), 4.0), ((0.5, -15.0, 0.0), 64.0)])
def test_singular_values_near_four(E, N, K, second, scale):
    """Two like rows (or columns) hold nearly all of G, so its singular value
    after the first step is nearly 3.9 and B has 198, 1972 and -114 off its
    diagonal: times 2^10, what A is stored in, the first two are past fp16."""
    x = matrices(E, N, K, torch.float32, N + K, "noise") * 1e-3
    if N <= K:
        x[:, 0] += torch.randn(E, K, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
        x[:, 1] = x[:, 0] + x[:, 1]
    else:
        x[:, :, 0] += torch.randn(E, N, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
        x[:, :, 1] = x[:, :, 0] + x[:, :, 1]
    co = [(3.9, 0.0, 0.0), second]
    want, scheme = exact(x, co), emulate_wide(x, co, (1024.0, scale))
    assert bool(scheme.isfinite().all()) and bool((norm(scheme - want) <= 2.0 ** -7 * norm(want)).all())
    for tile in (0, 64, 128, 256):
        mxq.testing_set(mxq.TESTING_NS_TILE, tile)
        try:
            got = mxq.newton_schulz(x, steps=2, coefficients=co)
        finally:
            mxq.testing_set(mxq.TESTING_NS_TILE, 0)
        assert bool(got.isfinite().all())
        assert bool((norm(got.double() - want) <= 1.25 * norm(scheme - want) + 2.0 ** -20 * norm(want)).all())
    assert mxq.device_status() == 0


@pytest.mark.gpu
def test_singular_value_near_four_of_two_by_two():
    """ones(2, 2): s = 3.9 after the first step, A = 7.6 everywhere, B off its
    diagonal 198.6, and a + b s^2 + c s^4 = 400.7 in every element's factor.
    Roundings, at most half a step of 2^-10 each: of X in A (2 b s^2 + 4 c s^4
    of 2^-11: 0.99), of A' (198.6 2^-11 in B', 2 c A'^2 2^-11 in beta: 0.21), of
    B' (0.1) and of X in B' X (0.1): 1.4 of 400.7, 3.5e-3, and bf16's 2^-8:
    below 2^-7."""
    g = torch.ones(2, 2, device=DEV)
    co = [(3.9, 0.0, 0.0), COEF]
    want = exact(g, co)
    for tile in (0, 64, 128, 256):
        mxq.testing_set(mxq.TESTING_NS_TILE, tile)
        try:
            got = mxq.newton_schulz(g, steps=2, coefficients=co).double()
        finally:
            mxq.testing_set(mxq.TESTING_NS_TILE, 0)
        assert bool(((got - want).abs() <= 2.0 ** -7 * want.abs()).all()), got


@pytest.mark.gpu
@pytest.mark.parametrize("E,N,K", [(2, 96, 224), (2, 100, 257), (2, 300, 260)])
def test_a_loose_bound_costs_no_accuracy(E, N, K):
    """Coefficients whose bound on the singular values is far above what these
    matrices reach: B is stored at a scale 2^-7 of what it could be, which stays
    below what the scheme costs anyway."""
    g = matrices(E, N, K, torch.float32, 3, "noise")
    for co in ([(1.0, 16.0, -16.0), (2.0, -4.0, 16.0), (1.0, 0.5, -2.0)], [(2.0, 16.0, 16.0), (1.5, -1.0, 16.0), (1.5, -0.5, 0.0)]):
        s = torch.linalg.svdvals(g.double() / norm(g.double())[:, None, None]).max()
        for a, b, c in co[:-1]:
            s = max(s, abs(a * s + b * s ** 3 + c * s ** 5))
        assert s < 4
        check(mxq.newton_schulz(g, steps=3, coefficients=co), g, co)


# ------------------------------------------------------------ schedules with large first steps
# a schedule of five steps that takes every singular value from 1e-3 to 1 near
# one, scaled so that none passes 2 (1.02 per power)
SCHEDULE = [(a / 1.02, b / 1.02 ** 3, c / 1.02 ** 5) for a, b, c in
            ((8.287, -23.596, 17.3), (4.107, -2.948, 0.545), (3.949, -2.909, 0.552), (3.318, -2.488, 0.51),
             (2.301, -1.669, 0.419))]


def test_larger_coefficients_where_the_bound_holds():
    L = mxq.lib()

    def status(*co):
        flat = [v for c in co for v in c]
        return L.newton_schulz(None, 0, 3, 0, 8, len(co), (ctypes.c_float * len(flat))(*flat), 1e-7, None, None, 0, None)

    assert status(*SCHEDULE) == mxq.OK
    assert status((8.3, -23.6, 17.3)) == mxq.OK          # 2.0 at s = 1, 2.1 at 1 + 2^-8
    assert status((20.0, 0.0, 0.0)) == mxq.ERR_UNSUPPORTED
    assert status((3.0, -17.0, 2.0)) == mxq.ERR_UNSUPPORTED   # -12 at s = 1
    assert status((2.0, -20.0, 21.0)) == mxq.OK          # 3 at s = 1
    assert status((2.0, -20.0, 21.98)) == mxq.ERR_UNSUPPORTED  # 3.98 there, 4.3 at 1 + 2^-8
    # the bound is carried on: the same step behind one that may reach 4
    assert status((4.0, 0.0, 0.0), (2.0, -20.0, 21.0)) == mxq.ERR_UNSUPPORTED
    assert status((0.9, 0.0, 0.0), (2.0, -20.0, 21.0)) == mxq.OK
    # inner maximum alone: 27 s - 27 s^3 is 10.4 at s^2 = 1/3, 0 at 1
    assert status((27.0, -27.0, 0.0)) == mxq.ERR_UNSUPPORTED
    assert status((10.0, -18.0, 8.0)) == mxq.OK          # 3 at s = 0.5, 0 at 1
    assert status((-8.3, 23.6, -17.3)) == mxq.OK
    assert status((1.0, -256.5, 256.5)) == mxq.ERR_UNSUPPORTED
    for bad in (float("nan"), float("inf"), -float("inf")):
        for i in range(3):
            assert status(tuple(bad if j == i else 1.0 for j in range(3))) == mxq.ERR_UNSUPPORTED
    # up to 16 the caller's word counts
    assert status(*[(16.0, -16.0, 16.0)] * 5) == mxq.OK


@pytest.mark.gpu
@pytest.mark.parametrize("E,N,K", [(2, 96, 224), (2, 257, 100), (2, 300, 260), (1, 256, 512)])
@pytest.mark.parametrize("kind", ["gradient", "noise", "decay"])
def test_schedule(E, N, K, kind):
    g = matrices(E, N, K, torch.float32, 7, kind)
    want, scheme = exact(g, SCHEDULE), emulate(g, SCHEDULE)
    for tile in (0, 64, 128, 256):
        mxq.testing_set(mxq.TESTING_NS_TILE, tile)
        try:
            got = mxq.newton_schulz(g, coefficients=SCHEDULE).double()
        finally:
            mxq.testing_set(mxq.TESTING_NS_TILE, 0)
        assert bool((norm(got - want) <= 1.25 * norm(scheme - want) + 2.0 ** -20 * norm(want)).all())
    assert mxq.device_status() == 0


# ------------------------------------------------------------ the one-launch path alone
SMALL = [(2, 96, 224), (2, 224, 96), (2, 100, 257), (2, 1030, 37)]  # one CTA a matrix, then clusters


@pytest.mark.gpu
@pytest.mark.parametrize("E,N,K", SMALL)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_small_steps_coefficients_and_scale(E, N, K, dtype):
    assert mxq.lib().newton_schulz_workspace_bytes(E, N, K, 5) == 0
    g = matrices(E, N, K, dtype, 9)
    for steps in (1, 2, 7):
        check(mxq.newton_schulz(g, steps=steps), g, [COEF] * steps)
    co = [(4.0, -8.0, 5.0), (3.5, -5.0, 2.2), (1.875, -1.25, 0.375)]
    check(mxq.newton_schulz(g, steps=3, coefficients=co), g, co)
    check(mxq.newton_schulz(g, steps=3, coefficients=co[::-1]), g, co[::-1])
    for s in (1e-18, 1e-25, 1e25):
        check(mxq.newton_schulz(g * s, eps=0.0), g * s, [COEF] * 5, eps=0.0)
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(96, 224), (224, 96), (100, 257), (1030, 37)])
def test_small_zeros_nan_and_neighbours(N, K):
    g = matrices(5, N, K, torch.float32, 4)
    want = mxq.newton_schulz(g)
    g[1] = 0.0
    g[2, 3, 4] = float("nan")
    g[3, N - 1, K - 1] = float("inf")
    got = mxq.newton_schulz(g)
    assert torch.equal(got[0], want[0]) and torch.equal(got[4], want[4])
    assert bool((got[1] == 0).all()) and bool(got[2].isnan().all()) and bool(got[3].isnan().all())
    assert bool((mxq.newton_schulz(g[1:2], eps=0.0) == 0).all())
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(17, 30), (33, 65), (1, 9), (100, 250), (97, 301), (50, 1290), (1000, 75), (3, 4000)])
def test_small_behind_nans(N, K):
    """What a matrix finds on its SMs, rows and columns behind its own in shared
    and tensor memory, it does not read: NaN matrices on every SM come first."""
    g = matrices(3, N, K, torch.float32, 2)
    want = mxq.newton_schulz(g)
    if min(N, K) >= 16:  # of fewer rows, single roundings would decide
        check(want, g, [COEF] * 5)
    for shape in ((600, 128, 256), (64, 128, 2048)):
        poison = torch.full(shape, float("nan"), device=DEV)
        got = []
        for _ in range(3):
            assert bool(mxq.newton_schulz(poison, steps=1).isnan().all())
            got.append(mxq.newton_schulz(g))
        assert all(torch.equal(x, want) for x in got)
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("E,N,K", [(40, 96, 224), (30, 100, 257), (20, 90, 4000)])
def test_small_streams_graphs_and_calls_at_once(E, N, K):
    g, h = matrices(E, N, K, torch.bfloat16, 8), matrices(3, 400, 700, torch.bfloat16, 8)
    want, other = mxq.newton_schulz(g), mxq.newton_schulz(h)
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append((mxq.newton_schulz(g), mxq.newton_schulz(h), mxq.newton_schulz(g)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, other) and torch.equal(c, want) for a, b, c in outs)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            graphs.append((gr, mxq.newton_schulz(g)))
    g.copy_(matrices(E, N, K, torch.bfloat16, 18))
    torch.cuda.synchronize()
    for gr, _ in graphs:
        with torch.cuda.stream(torch.cuda.Stream()):
            gr.replay()
    torch.cuda.synchronize()
    want = mxq.newton_schulz(g)
    assert all(torch.equal(o, want) for _, o in graphs)
    check(want, g, [COEF] * 5)
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("E,N,K", [(3, 140, 150), (1, 700, 1100)])
def test_calls_back_to_back(E, N, K):
    """The kernel that scales G starts while the one that sums its squares still
    runs, and their workspace is the one of the call before: the norm of another
    call's matrices must not show."""
    L = mxq.lib()
    base = matrices(E, N, K, torch.float32, 5)
    batches = [base * s for s in (1.0, 1e6, 1e-6, 3.0)]
    want = [mxq.newton_schulz(b) for b in batches]
    for b, w in zip(batches, want):
        check(w, b, [COEF] * 5)
    nbytes = L.newton_schulz_workspace_bytes(E, N, K, 1)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    want = [mxq.newton_schulz(b, steps=1) for b in batches]
    outs = torch.empty(60, E, N, K, dtype=torch.bfloat16, device=DEV)
    co = (ctypes.c_float * 3)(*COEF)
    stream = torch.cuda.current_stream().cuda_stream
    for i in range(60):
        assert L.newton_schulz(batches[i % 4].data_ptr(), 1, E, N, K, 1, co, 1e-7, outs[i].data_ptr(), ws.data_ptr(),
                               nbytes, stream) == mxq.OK
    for i in range(60):
        assert torch.equal(outs[i], want[i % 4])
    assert mxq.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(65536, 32760), (32760, 65536), (65536, 1000), (65536, 9)])
def test_the_largest_matrices(N, K):
    """Sides of 65536 and just below 2^31 elements, one step, 2 + 66 rows of X^T
    against 64 bits: a X + (b A + c A A) X with A summed in parts. The scheme's
    error stays below 1e-3 of the norm and the result's rounding is 1.7e-3."""
    gen = torch.Generator(device=DEV).manual_seed(4)
    g = torch.randn(N, K, generator=gen, device=DEV, dtype=torch.bfloat16)
    out = mxq.newton_schulz(g, steps=1)
    gt, ot = (g, out) if N >= K else (g.t(), out.t())  # X^T and its update
    n, m = gt.shape
    A = torch.zeros(m, m, dtype=torch.float64, device=DEV)
    for part in gt.split(4096):
        p = part.double()
        A += p.t() @ p
    f = 1.0 / (A.diagonal().sum().sqrt() + 1e-7)
    A *= f * f
    rows = torch.cat([torch.tensor([0, n - 1]), torch.randint(0, n, (64,), generator=torch.Generator().manual_seed(2)),
                      torch.tensor([n // 2, n - 2])]).to(DEV)
    X = gt[rows].double() * f
    a, b, c = COEF
    XA = X @ A
    want = a * X + b * XA + c * (XA @ A)
    off = ot[rows].double() - want
    size = norm(want)
    assert bool(norm(off) <= 2.0 ** -8.97 * size), float(norm(off) / size)
    # no row and no column of them off by more than rounding makes it
    assert bool((off.abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -7 * size / want.numel() ** 0.5).all())
    assert bool(out.isfinite().all()) and mxq.device_status() == 0
