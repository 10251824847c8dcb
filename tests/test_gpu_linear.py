"""moe_linear_fwd and moe_linear_bwd through the C ABI, every buffer guarded.

Most cases take small whole numbers: every product and sum is then exact in fp32 (K 4 + bias stays
below 2^24), so the outputs must equal the exact results rounded once to their type, element for
element, in every tile shape, slice count and layout.  With random inputs the tolerances follow the
arithmetic (u = 2^-24, half: 2^-8 for bf16, u for fp32): a sum of K products in any order is off by at
most K u sum |x w|, fp32's dropped part products by 4 u sum |x w| more, and as errors of either sign
mostly cancel, by 2e-6 in the 2-norm for K <= 4096 in fp32 (about 0.6 u sqrt(6 K / 32) of the partial
sums' size); the activations (their slope is at most 1.13) pass that on and add at most 16 u of
their own value and argument each; dz is one rounding of at most 2^-8 |dz| on each term of dx and
dw; dbias sums at most 64 + 64 + 128 values in a row."""
import numpy as np
import pytest
import torch

from harness import Guards

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("ty", [BF, F32], ids=["bf16", "f32"])


def _half(ty):
    return torch.finfo(ty).eps / 2


def _code(ty):
    import grouped_gemm_top_amd as G
    return G.MOE_BF16 if ty == BF else G.MOE_F32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import grouped_gemm_top_amd as G
    G.lib()


def _ints(shape, lo, hi, seed):
    return torch.randint(lo, hi + 1, shape, generator=torch.Generator().manual_seed(seed)).float()


def _rand(shape, seed, scale=1.0, ty=BF):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(ty)


def _up(g, name, t):
    if t is None:
        return None
    v = g.alloc(name, t.shape, t.dtype)
    v.copy_(t)
    return v


def _mm(a, b):
    """The exact product of whole-number matrices (fp32 on the CPU is exact at these sizes)."""
    return a @ b


SHAPES = [  # N, K, O
    (1, 8, 8), (1, 4096, 16), (2, 64, 4104), (16, 520, 72), (17, 64, 24), (33, 136, 40), (64, 2880, 128), (65, 64, 64),
    (70, 8, 8), (100, 72, 200), (129, 1000, 136), (333, 288, 264), (300, 2880, 512), (257, 520, 264), (513, 1032, 520),
    (1000, 200, 1000), (2050, 264, 1544), (4097, 136, 2056), (8200, 72, 4104), (3000, 4096, 64),
]


@TYPES
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("N,K,O", SHAPES)
def test_forward_exact(N, K, O, act, ty):
    import grouped_gemm_top_amd as G
    x, w = _ints((N, K), -2, 2, 1), _ints((O, K), -2, 2, 2)
    b, r = _ints((O,), -50, 50, 3), _ints((N, O), -9, 9, 4)
    g = Guards()
    dx, dw, db, dr = _up(g, "x", x.to(ty)), _up(g, "w", w.to(ty)), _up(g, "b", b), _up(g, "r", r.to(ty))
    out, z = g.alloc("out", (N, O), ty), g.alloc("z", (N, O), ty)
    ws = g.alloc("ws", (G.workspace_bytes(G.OP_LINEAR_FWD, _code(ty), N, 1, 1, K, O),), torch.uint8)
    G.linear_fwd(dx, dw, bias=db, act=act, residual=dr, out=out, z=z, ws=ws)
    g.check("linear_fwd")
    zr = _mm(x, w.t()) + b
    f = (lambda v: v.clamp(min=0)) if act == "relu" else (lambda v: v)
    assert torch.equal(z.cpu(), zr.to(ty)) and torch.equal(out.cpu(), (f(zr) + r).to(ty))
    # no bias, no residual, no z; then in place over the residual
    o2, z2 = G.linear_fwd(dx, dw, act=act)
    assert z2 is None and torch.equal(o2.cpu(), f(_mm(x, w.t())).to(ty))
    o3, _ = G.linear_fwd(dx, dw, bias=db, act=act, residual=dr, out=dr, ws=ws)
    g.check("linear_fwd in place")
    assert o3.data_ptr() == dr.data_ptr() and torch.equal(o3, out)


@TYPES
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("N,K,O", SHAPES)
def test_backward_exact(N, K, O, act, ty):
    import grouped_gemm_top_amd as G
    x, w = _ints((N, K), -2, 2, 5), _ints((O, K), -2, 2, 6)
    d, z = _ints((N, O), -3, 3, 7), _ints((N, O), -1, 1, 8)
    g = Guards()
    D = {n: _up(g, n, t.to(ty)) for n, t in (("d", d), ("x", x), ("w", w), ("z", z))}
    dx, dw, db = g.alloc("dx", (N, K), ty), g.alloc("dw", (O, K), ty), g.alloc("db", (O,), torch.float32)
    ws = g.alloc("ws", (G.workspace_bytes(G.OP_LINEAR_BWD, _code(ty), N, 1, 1, K, O),), torch.uint8)
    zz = D["z"] if act == "relu" else None
    G.linear_bwd(D["d"], D["x"], D["w"], z=zz, act=act, dx=dx, dw=dw, dbias=db, ws=ws)
    g.check("linear_bwd")
    dz = d * (z > 0) if act == "relu" else d
    assert torch.equal(dx.cpu(), _mm(dz, w).to(ty)), "dx"
    assert torch.equal(dw.cpu(), _mm(dz.t(), x).to(ty)), "dw"
    assert torch.equal(db.cpu(), dz.sum(0)), "dbias"
    # each alone
    for n, ref in (("dx", dx), ("dw", dw), ("dbias", db)):
        r = G.linear_bwd(D["d"], D["x"], D["w"], z=zz, act=act, **{f"want_{m}": m == n for m in ("dx", "dw", "dbias")})
        torch.cuda.synchronize()
        assert torch.equal(r[n], ref) and all(r[m] is None for m in r if m != n)


def _act64(v, act):
    return {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu,
            "gelu": torch.nn.functional.gelu,
            "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act](v)


@TYPES
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("N,K,O", [(5, 264, 136), (30, 200, 72), (200, 520, 328), (1030, 256, 1032), (300, 4096, 264)])
def test_forward_activations(N, K, O, act, ty):
    import grouped_gemm_top_amd as G
    x, w, b, r = _rand((N, K), 9, ty=ty), _rand((O, K), 10, K ** -0.5, ty), _rand((O,), 11).float(), \
        _rand((N, O), 12, ty=ty)
    H = _half(ty)
    x[0] *= 30  # saturated activations too
    out, z = G.linear_fwd(x.cuda(), w.cuda(), bias=b.cuda(), act=act, residual=r.cuda(), want_z=True)
    z64 = x.double() @ w.double().t() + b.double()
    ez = (K + 4) * U * (x.double().abs() @ w.double().abs().t()) + U * z64.abs()
    assert bool(((z.cpu().double() - z64).abs() <= ez + H * z64.abs()).all())
    if ty == F32:
        assert float((z.cpu().double() - z64).norm()) <= 2e-6 * float(z64.norm())
    ref = _act64(z64, act) + r.double()
    tol = 1.13 * ez + 16 * U * (z64.abs() + 1) + U * ref.abs() + H * ref.abs()
    assert bool(((out.cpu().double() - ref).abs() <= tol).all())


@TYPES
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("N,K,O", [(1, 264, 136), (200, 520, 328), (1030, 256, 1032), (3000, 136, 264)])
def test_backward_activations(N, K, O, act, ty):
    import grouped_gemm_top_amd as G
    x, w, d, z = _rand((N, K), 13, ty=ty), _rand((O, K), 14, K ** -0.5, ty), _rand((N, O), 15, ty=ty), \
        _rand((N, O), 16, 1.5, ty)
    H = _half(ty)
    z[0, :4] = torch.tensor([40.0, -40.0, 0.0, 3e4])
    r = G.linear_bwd(d.cuda(), x.cuda(), w.cuda(), z=z.cuda(), act=act)
    z64 = z.double().requires_grad_(True)
    slope = torch.autograd.grad(_act64(z64, act).sum(), z64)[0]
    dz = d.double() * slope
    e = 32 * U * d.double().abs()  # the slope's own error (it is at most 1.13)
    each = H * dz.abs() + e * (1 + H)
    x64, w64 = x.double(), w.double()
    for n, ref, err in (("dx", dz @ w64, each @ w64.abs() + (O + 4) * U * (dz.abs() @ w64.abs())),
                        ("dw", dz.t() @ x64, each.t() @ x64.abs() + (N + 4) * U * (dz.abs().t() @ x64.abs()))):
        got = r[n].cpu().double()
        assert bool(((got - ref).abs() <= err * 1.01 + H * ref.abs() + 2.0 ** -126).all()), n
        if ty == F32:  # (and the slopes' few u, of either sign)
            assert float((got - ref).norm()) <= 2e-6 * float(ref.norm()), n
    tol = e.sum(0) + 256 * U * dz.abs().sum(0)
    assert bool(((r["dbias"].cpu().double() - dz.sum(0)).abs() <= tol).all())


def test_gradient_against_differences():
    """dx, dw and dbias along random directions against central differences of the fp64 formula.
    Beside the differences' own error (below 1e-5 of the size with steps of 2^-8) stand the two bf16
    roundings, of dz and of the gradient: each term at most 2^-8, so at most 2^-7 of the sum of
    the terms' magnitudes; they do not line up, so a tenth of that is asked for."""
    import grouped_gemm_top_amd as G
    N, K, O, act = 24, 64, 40, "gelu_tanh"
    x, w, b, d = _rand((N, K), 17), _rand((O, K), 18, K ** -0.5), _rand((O,), 19).float(), _rand((N, O), 20)
    _, z = G.linear_fwd(x.cuda(), w.cuda(), bias=b.cuda(), act=act, want_z=True)
    r = {n: v.cpu().double() for n, v in G.linear_bwd(d.cuda(), x.cuda(), w.cuda(), z=z, act=act).items()}
    off = z.cpu().double() - (x.double() @ w.double().t() + b.double())  # the stored z is the point
    f = lambda xx, ww, bb: float((_act64(xx @ ww.t() + bb + off, act) * d.double()).sum())  # noqa: E731
    st = 2.0 ** -8
    base = [x.double(), w.double(), b.double()]
    for i, n in enumerate(("dx", "dw", "dbias")):
        for seed in range(3):
            e = torch.randn(base[i].shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
            hi, lo = list(base), list(base)
            hi[i], lo[i] = base[i] + st * e, base[i] - st * e
            num = (f(*hi) - f(*lo)) / (2 * st)
            terms = (r[n] * e).abs().sum()
            assert abs(float((r[n] * e).sum()) - num) <= 0.1 * 2.0 ** -7 * float(terms), n


@TYPES
def test_bad_rows_stay_alone(ty):
    """A NaN or infinity in one token's x reaches that token's outputs only, in every path."""
    import grouped_gemm_top_amd as G
    for N, K, O in ((5, 136, 72), (90, 200, 264), (700, 136, 520)):
        x, w = _rand((N, K), 21, ty=ty), _rand((O, K), 22, ty=ty)
        clean, _ = G.linear_fwd(x.cuda(), w.cuda())
        x[2, K - 1] = float("nan")
        x[4, 0] = float("inf")
        got, _ = G.linear_fwd(x.cuda(), w.cuda())
        keep = [t for t in range(N) if t not in (2, 4)]
        assert torch.equal(got[keep], clean[keep]) and bool(got[2].isnan().all())


@TYPES
def test_empty_input(ty):
    import grouped_gemm_top_amd as G
    x, w = torch.empty((0, 64), dtype=ty, device="cuda"), _rand((24, 64), 23, ty=ty).cuda()
    out, z = G.linear_fwd(x, w, want_z=True)
    assert out.shape == (0, 24) and z.shape == (0, 24)
    dw, db = torch.full((24, 64), 7.0, dtype=ty, device="cuda"), torch.full((24,), 7.0, device="cuda")
    r = G.linear_bwd(out, x, w, dw=dw, dbias=db)
    torch.cuda.synchronize()
    assert r["dx"].shape == (0, 64) and float(dw.abs().max()) == 0.0 and float(db.abs().max()) == 0.0


@TYPES
@pytest.mark.parametrize("N,K,O", [(3, 512, 264), (300, 2880, 512), (2050, 264, 1544)])
def test_stream_and_graph(N, K, O, ty):
    import grouped_gemm_top_amd as G
    x, w, b, d = _rand((N, K), 24, ty=ty).cuda(), _rand((O, K), 25, K ** -0.5, ty).cuda(), \
        _rand((O,), 26).float().cuda(), _rand((N, O), 27, ty=ty).cuda()

    def both(**s):
        out, z = G.linear_fwd(x, w, bias=b, act="gelu_tanh", residual=d, want_z=True, **s)
        return dict(G.linear_bwd(d, x, w, z=z, act="gelu_tanh", **s), out=out, z=z)

    eager = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = both(stream=s)
    s.synchronize()
    assert all(torch.equal(eager[n], other[n]) for n in eager)
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    with torch.cuda.graph(graph2):
        got2 = both()
    for seed in range(3):
        x.copy_(_rand((N, K), 60 + seed, ty=ty))
        graph.replay()
        graph2.replay()
        torch.cuda.synchronize()
        eager = both()
        torch.cuda.synchronize()
        assert all(torch.equal(eager[n], got[n]) and torch.equal(eager[n], got2[n]) for n in eager)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slope_far_from_zero(act, dt):
    """Far out the slope is 1 or 0, also where z^2 or z^3 overflow fp32: dbias is the sum of dout or 0, exactly
    (small integers; silu's slope is within e^-100 of its limit from |z| = 128 on)."""
    import grouped_gemm_top_amd as G
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    z = torch.tensor([128.0, -128.0, 1e6, -1e6, 1e20, -1e20, 3e38, -3e38], dtype=t, device="cuda").repeat(5, 1)
    dout = torch.arange(1, 41, device="cuda").reshape(5, 8).to(t)
    x, w = torch.ones(5, 8, dtype=t, device="cuda"), torch.eye(8, dtype=t, device="cuda")
    r = G.linear_bwd(dout, x, w, z, act=act)
    want = dout.float() * (z > 0)
    assert torch.equal(r["dbias"], want.sum(0))
    assert torch.equal(r["dx"].float(), want)
    assert torch.equal(r["dw"].float(), want.sum(0)[:, None].expand(8, 8))


@TYPES
@pytest.mark.parametrize("N", [10, 60])
def test_gelu_in_its_tail(N, ty):
    """The erf GELU and its slope keep their relative accuracy down to z = -12.5, where 1 + erf would be
    a difference of nearly equal numbers (few tokens and tiles).  Phi(z) for z < 0 is e^(-z^2 / 2) times a
    function of size 1 / |z|: the exponent carries three roundings of z^2 / 2 (the square, the constant, the
    product), 1.5 z^2 u of the result, the function and the products at most 40 u: (2 z^2 + 40) u of
    Phi.  The slope's second term z phi(z) has the same exponent and six more operations: (1.5 z^2 + 12) u
    of it; the sum and the store 2 u.  W is the identity, so z is x exactly."""
    import grouped_gemm_top_amd as G
    H = _half(ty)
    z = torch.linspace(-12.5, 6.0, 8 * N).reshape(N, 8).to(ty)
    out, zz = G.linear_fwd(z.cuda(), torch.eye(8, dtype=ty, device="cuda"), act="gelu", want_z=True)
    assert torch.equal(zz.cpu(), z)
    z64 = z.double()
    phi_c = 0.5 * torch.special.erfc(-z64 * 0.5 ** 0.5)
    tol = (2 * z64 ** 2 + 40) * U * (z64 * phi_c).abs() + H * (z64 * phi_c).abs() + 2.0 ** -125
    err = (out.cpu().double() - z64 * phi_c).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    # the slope: dbias of one row of ones
    zr = z.reshape(1, -1)
    O = zr.shape[1]
    one = torch.ones(1, O, dtype=ty, device="cuda")
    r = G.linear_bwd(one, torch.ones(1, 8, dtype=ty, device="cuda"), torch.ones(O, 8, dtype=ty, device="cuda"),
                     z=zr.cuda(), act="gelu", want_dx=False, want_dw=False)
    z64, phi_c = z64.reshape(-1), phi_c.reshape(-1)
    zpdf = z64 * torch.exp(-0.5 * z64 ** 2) * (2 * np.pi) ** -0.5
    ref = phi_c + zpdf
    tol = (2 * z64 ** 2 + 40) * U * phi_c + (1.5 * z64 ** 2 + 12) * U * zpdf.abs() + 2 * U * ref.abs() + 2.0 ** -122
    err = (r["dbias"].cpu().double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_slope_where_the_sigmoid_is_near_one(act):
    """fp32 slopes s (1 + v q c) with s = 1 / (1 + E), q = E / (1 + E), c the inner derivative (1 for silu): q
    must come from E, not from 1 - s, whose error of 1 u counts v c times.  Relative errors in u: E from its
    exponent g (silu g = |v|, two roundings and the constant's; tanh gelu g = 2 u(v), four) and the
    instruction: a = 1.25 g + 2 and 4 g + 2; s: (1 - s) a + 3 (an addition, the reciprocal's 2); q: that
    and a and 1, at most 2 a + 4; c and the products 10.  So s ((1 - s) a + 3) + |v s q c| (3 a + 17)
    and 2 for the sum and the store.  A sigmoid below 2^-126 is flushed to 0, which costs 2^-126 (1 + |v c|)
    (|v c| is 230 at z = -10, where the tanh gelu's gets there), and so may be the sum.  dbias of a single
    row of ones is the slope itself."""
    import grouped_gemm_top_amd as G
    z = torch.linspace(-12.0, 60.0, 20000)[None]
    O = z.shape[1]
    r = G.linear_bwd(torch.ones(1, O, device="cuda"), torch.ones(1, 8, device="cuda"), torch.ones(O, 8, device="cuda"),
                     z=z.cuda(), act=act, want_dx=False, want_dw=False)
    v = z[0].double()
    kg, k3 = (2 / np.pi) ** 0.5, 0.044715
    if act == "silu":
        t, c, a = v, torch.ones_like(v), 1.25 * v.abs() + 2
    else:
        t, c = 2 * kg * (v + k3 * v ** 3), 2 * kg * (1 + 3 * k3 * v ** 2)
        a = 4 * t.abs() + 2
    s, q = torch.sigmoid(t), torch.sigmoid(-t)
    ref = s + v * s * q * c
    tol = U * (s * (q * a + 3) + (v * s * q * c).abs() * (3 * a + 17) + 2 * ref.abs()) + 2.0 ** -126 * (2 + (v * c).abs())
    err = (r["dbias"].cpu().double() - ref).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), float(v[(err / tol).argmax()]))


@pytest.mark.parametrize("e", [-100, -116, -126])
def test_fp32_parts_of_tiny_values(e):
    """Where the third bf16 part of an fp32 value falls below bf16's smallest step, 2^-133, it is rounded to
    that step: the value is off by at most 2^-134 (nothing from 2^-109 on), which the product passes on."""
    import grouped_gemm_top_amd as G
    N, s = 64, 60
    x = (1 + torch.rand(N, 8, generator=torch.Generator().manual_seed(27))) * 2.0 ** e
    w = torch.eye(8) * 2.0 ** s
    out, _ = G.linear_fwd(x.cuda(), w.cuda())
    r = G.linear_bwd(x.cuda(), w.repeat(8, 1).cuda(), w.cuda(), want_dbias=False)
    ref = x.double() * 2.0 ** s
    tol = (2.0 ** (s - 134) if e < -109 else 0.0) + U * ref
    assert bool(((out.cpu().double() - ref).abs() <= tol).all())
    assert bool(((r["dx"].cpu().double() - ref).abs() <= tol).all())
    # dw[o, i] = sum_t x[t, o] 2^s [t mod 8 == i]: eight terms
    ref = ref.reshape(8, 8, 8).sum(0).t()
    tol = (8 * 2.0 ** (s - 134) if e < -109 else 0.0) + 16 * U * ref
    assert bool(((r["dw"].cpu().double() - ref).abs() <= tol).all())
