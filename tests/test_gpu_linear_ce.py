"""moe_linear_ce_fwd and moe_linear_ce_bwd through the C ABI against the formulas in 64 bits.

Tolerances (u = 2^-24; half: 2^-8 for bf16, u for fp32).  A logit is a sum of H products, off by at most
ez = (H + 8) u sum |x w| in any order (fp32's dropped part products are within the 8).  lse: the largest ez of its
row, the sum of V exponentials (at most 32 in a lane, 2 + 2 joins, then V / (64 16) turns and 16 joins of two
roundings each, their arguments' rounding 1.5 |z - lse| u weighted by p: under (256 + V / 256) u in all for the sizes
here) and 4 u |lse| for the logarithm and the stored value.  dz = g (c p - [v = y]): p is off by (ez + dlse + (16 +
2 |z - lse|) u) p, the subtraction by u, and bf16 rounds dz by half of its value.  dx and dw pass that on as
sums of |error| |operand|, add V or N roundings of u of sum |dz operand|, and round once."""
import pytest
import torch

from harness import Guards

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("ty", [BF, F32], ids=["bf16", "f32"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import grouped_gemm_top_amd as G
    G.lib()


def _rand(shape, seed, scale=1.0, ty=BF):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(ty)


def _targets(N, V, seed, ign):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, V, (N,), generator=g)
    out = torch.tensor([-100, -1, V, V + 7, -2 ** 31, 2 ** 31 - 1])
    t = torch.where(torch.rand(N, generator=g) < ign, out[torch.randint(0, 6, (N,), generator=g)], t)
    if N > 3:
        t[0], t[-1] = V - 1, 0
    return t.int()


def _case(N, H, V, ty, ign, zc, seed=1):
    x, w = _rand((N, H), seed, ty=ty), _rand((V, H), seed + 1, 2.0 * H ** -0.5, ty)
    return dict(x=x, w=w, t=_targets(N, V, seed + 2, ign), g=_rand((N,), seed + 3, ty=F32), zc=zc)


def _exact(c):
    """The formulas in 64 bits (on the GPU, row block by row block) with each output's bound."""
    x, w, t, g = (c[n].cuda() for n in ("x", "w", "t", "g"))
    ty, zc = x.dtype, c["zc"]
    half = torch.finfo(ty).eps / 2
    N, H = x.shape
    V = w.shape[0]
    live = ((t >= 0) & (t < V)).nonzero()[:, 0]
    w64, wa = w.double(), w.double().abs()
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
    o = dict(loss=zero(N), lse=zero(N), dx=zero(N, H), dw=zero(V, H))
    b = {n: torch.zeros_like(v) for n, v in o.items()}
    for r in live.split(max(1, 2 ** 26 // V)):
        x64 = x[r].double()
        z = x64 @ w64.t()
        ez = (H + 8) * U * (x64.abs() @ wa.t())
        lse = torch.logsumexp(z, dim=1)
        y = t[r].long()
        dl = ez.max(dim=1).values + (256 + V / 256) * U + 4 * U * lse.abs()
        o["lse"][r], b["lse"][r] = lse, dl
        o["loss"][r] = lse - z.gather(1, y[:, None])[:, 0] + zc * lse * lse
        b["loss"][r] = dl + ez.gather(1, y[:, None])[:, 0] + 2 * zc * lse.abs() * dl + 4 * U * (
            lse.abs() + z.gather(1, y[:, None])[:, 0].abs() + zc * lse * lse)
        p = torch.exp(z - lse[:, None])
        gr, cf = g[r].double()[:, None], (1 + 2 * zc * lse)[:, None]
        dz = gr * cf * p
        ed = gr.abs() * (cf.abs() * p * (ez + dl[:, None] + (16 + 2 * (z - lse[:, None]).abs()) * U +
                                         2 * abs(zc) * dl[:, None]) + U)
        dz.scatter_add_(1, y[:, None], -gr)
        ed += (half if ty == BF else 4 * U) * dz.abs()
        o["dx"][r] = dz @ w64
        b["dx"][r] = ed @ wa + (V + 8) * U * (dz.abs() @ wa)
        o["dw"] += dz.t() @ x64
        b["dw"] += ed.t() @ x64.abs() + (live.numel() + 8) * U * (dz.abs().t() @ x64.abs())
    for n in ("dx", "dw"):
        b[n] += half * (o[n].abs() + b[n])
    return o, b


def _run(c, guarded=True, **kw):
    import grouped_gemm_top_amd as G
    g = Guards()
    N, H = c["x"].shape
    V = c["w"].shape[0]
    up = {}
    for n in ("x", "w", "t", "g"):
        up[n] = g.alloc(n, c[n].shape, c[n].dtype)
        up[n].copy_(c[n])
    dt = G.MOE_BF16 if c["x"].dtype == BF else G.MOE_F32
    o = {n: g.alloc(n, (N,), F32) for n in ("loss", "lse")}
    o["dx"], o["dw"] = g.alloc("dx", (N, H), c["x"].dtype), g.alloc("dw", (V, H), c["x"].dtype)
    wf, wb = (g.alloc(f"ws{op}", (G.workspace_bytes(op, dt, N, 1, 1, H, V),), torch.uint8)
              for op in (G.OP_LINEAR_CE_FWD, G.OP_LINEAR_CE_BWD))
    G.linear_ce_fwd(up["x"], up["w"], up["t"], z_coef=c["zc"], loss=o["loss"], lse=o["lse"], ws=wf)
    g.check("linear_ce_fwd")
    G.linear_ce_bwd(up["g"], up["x"], up["w"], up["t"], o["lse"], z_coef=c["zc"], dx=o["dx"], dw=o["dw"], ws=wb)
    g.check("linear_ce_bwd")
    return o, up


def _check(o, ref, bound, norms=True):
    ty = o["dx"].dtype
    for n in ("loss", "lse", "dx", "dw"):
        d = (o[n].double() - ref[n]).abs()
        bad = ~(d <= bound[n])
        assert not bool(bad.any()), f"{n}: {int(bad.sum())} of {bad.numel()} off, worst {float((d - bound[n]).max())}"
        if norms and float(ref[n].norm()):
            # one rounding of the output and one of dz, each uniform in half a step at most: 2^-8 / sqrt 3 each, together
            # 0.0032.  Where few tokens or columns count, few roundings of dz make up the error and it need not
            # average: with one token dw is the outer product of dz and x, off by 2^-8 of each value, twice.
            tol = 5e-6
            if ty == BF and n in ("dx", "dw"):
                tol = 4e-3 if min(int((ref["lse"] != 0).sum()), ref["dw"].shape[0]) >= 16 else 2 ** -7
            assert float(d.norm()) <= tol * float(ref[n].norm()), (n, float(d.norm() / ref[n].norm()))


SHAPES = [  # N, H, V, share of tokens that take no part
    (1, 8, 1, 0.0), (2, 8, 2, 0.0), (1, 64, 50, 0.0), (3, 72, 257, 0.0), (16, 136, 63, 0.3), (65, 264, 1000, 0.2),
    (130, 1032, 511, 0.5), (300, 520, 4099, 0.4), (513, 128, 8200, 0.0), (257, 2880, 640, 0.1), (1000, 64, 12345, 0.9),
    (4100, 256, 2050, 0.1),
]


@TYPES
@pytest.mark.parametrize("zc", [0.0, 0.01])
@pytest.mark.parametrize("N,H,V,ign", SHAPES)
def test_against_formulas(N, H, V, ign, zc, ty):
    c = _case(N, H, V, ty, ign, zc)
    ref, bound = _exact(c)
    o, _ = _run(c)
    _check(o, ref, bound)
    dead = ~((c["t"] >= 0) & (c["t"] < V))
    for n in ("loss", "lse", "dx"):
        assert bool((o[n].cpu()[dead] == 0).all()), n


@TYPES
def test_pieces_of_the_vocabulary(ty):
    """Several backward pieces, the last one ragged: dx is summed over them."""
    N, H, V = 20000, 64, 8001
    c = _case(N, H, V, ty, 0.05, 1e-3, seed=11)
    ref, bound = _exact(c)
    o, _ = _run(c)
    _check(o, ref, bound)


@TYPES
@pytest.mark.parametrize("N,H,V,ign", [(1, 96, 60011, 0.0), (33, 328, 50021, 0.2), (64, 200, 33001, 0.0)])
def test_few_tokens_large_vocabulary(N, H, V, ign, ty):
    c = _case(N, H, V, ty, ign, 1e-3)
    ref, bound = _exact(c)
    o, _ = _run(c)
    _check(o, ref, bound)


@pytest.mark.parametrize("ty,N,H,V", [(BF, 8192, 2048, 9001), (F32, 8192, 4096, 8100)], ids=["bf16", "f32"])
def test_pieces_that_share_launches(ty, N, H, V):
    """Pieces large enough that dx and dW of one run beside dz of the next; on two streams at once and from a graph.
    In the 2-norm: bf16 rounds dz and the result, sqrt 2 2^-8 / sqrt 3 = 0.0032; fp32 rounds 6 K / 32 running sums, which
    for K = 8100 at random is 39 2^-24 = 2.3e-6 of the sum, and dz carries that of z, K = 4096, 1.7e-6."""
    import grouped_gemm_top_amd as G
    gen = torch.Generator(device="cuda").manual_seed(91)
    x = torch.randn(N, H, generator=gen, device="cuda").to(ty)
    w = (H ** -0.5 * torch.randn(V, H, generator=gen, device="cuda")).to(ty)
    t = torch.randint(-V // 9, V, (N,), generator=gen, device="cuda").int()
    g = torch.rand(N, generator=gen, device="cuda")

    def step(stream=None):
        f = G.linear_ce_fwd(x, w, t, z_coef=1e-3, stream=stream)
        return dict(f, **G.linear_ce_bwd(g, x, w, t, f["lse"], z_coef=1e-3, stream=stream))
    o = step()
    live = t >= 0
    xl, wd, tl = x[live].double(), w.double(), t[live].long()[:, None]
    z = xl @ wd.t()
    lse = torch.logsumexp(z, dim=1)
    rel = lambda p, q: float((p.double() - q).norm() / q.norm())  # noqa: E731
    assert rel(o["loss"][live], lse - z.gather(1, tl)[:, 0] + 1e-3 * lse ** 2) <= 1e-6
    gl = g[live].double()
    dz = torch.exp(z - lse[:, None]) * (gl * (1 + 2e-3 * lse))[:, None]
    dz.scatter_add_(1, tl, -gl[:, None])
    tol = 4e-3 if ty is BF else 1e-5
    assert rel(o["dx"][live], dz @ wd) <= tol and bool((o["dx"][~live] == 0).all())
    assert rel(o["dw"], dz.t().contiguous() @ xl) <= tol
    st = [torch.cuda.Stream() for _ in range(2)]
    for s in st:
        s.wait_stream(torch.cuda.current_stream())
    p, q = step(st[0]), step(st[1])
    torch.cuda.synchronize()
    assert all(torch.equal(o[n], p[n]) and torch.equal(o[n], q[n]) for n in o)
    with torch.cuda.stream(st[0]):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st[0]):
            r = step()
    for i in range(2):
        x.copy_(torch.randn(N, H, generator=gen, device="cuda"))
        t.copy_(torch.randint(-V * (2 - i), V, (N,), generator=gen, device="cuda"))
        e = step()
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(e[n], r[n]) for n in e), i


@TYPES
def test_many_tokens(ty):
    """More tokens than one group a workgroup lists: 140003 of them, a third without a target."""
    N, H, V = 140003, 16, 40
    c = _case(N, H, V, ty, 0.33, 1e-3, seed=12)
    ref, bound = _exact(c)
    o, _ = _run(c)
    _check(o, ref, bound)


def test_past_32_bits():
    """W of more than 2^31 elements and 2 GiB: forward pieces, offsets of W and dW past 32 bits.  The first
    and last rows alone are checked in full."""
    import grouped_gemm_top_amd as G
    N, H, V = 40, 8192, 270001
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(N, H, generator=gen, device="cuda").to(BF)
    w = (0.02 * torch.randn(V, H, generator=gen, device="cuda")).to(BF)
    t = torch.randint(0, V, (N,), generator=gen, device="cuda").int()
    t[0], t[1] = V - 1, 0
    r = G.linear_ce_fwd(x, w, t)
    b = G.linear_ce_bwd(torch.ones(N, device="cuda"), x, w, t, r["lse"])
    z = torch.cat([x.double() @ p.double().t() for p in w.split(50000)], dim=1)
    lse = torch.logsumexp(z, dim=1)
    # |z| is about 1.8: an error of 8200 u sum |x w| = 8200 u 8192 0.013 at the very most, typically 1e-6
    assert float((r["lse"].double() - lse).abs().max()) <= 1e-4
    assert float((r["loss"].double() - (lse - z.gather(1, t.long()[:, None])[:, 0])).abs().max()) <= 1e-4
    dz = torch.exp(z - lse[:, None])
    dz.scatter_add_(1, t.long()[:, None], -torch.ones(N, 1, dtype=torch.float64, device="cuda"))
    dx = sum(dz[:, i * 50000:(i + 1) * 50000] @ p.double() for i, p in enumerate(w.split(50000)))
    assert float((b["dx"].double() - dx).norm()) <= 4e-3 * float(dx.norm())
    for rows in (slice(0, 300), slice(131000, 131300), slice(V - 300, V)):
        dw = dz[:, rows].t() @ x.double()
        assert float((b["dw"][rows].double() - dw).norm()) <= 4e-3 * float(dw.norm())


@TYPES
def test_masked_rows_hold_anything(ty):
    """NaN and infinities in the rows of tokens that take no part reach nothing."""
    c = _case(200, 136, 777, ty, 0.4, 1e-3, seed=21)
    o, _ = _run(c)
    dead = ~((c["t"] >= 0) & (c["t"] < 777))
    assert bool(dead.any())
    d = dict(c, x=c["x"].clone(), g=c["g"].clone())
    d["x"][dead] = float("nan")
    d["x"][dead.nonzero()[0]] = float("inf")
    d["g"][dead] = float("nan")
    p, _ = _run(d)
    for n in o:
        assert torch.equal(o[n], p[n]), n


def test_spoilt_token():
    """A counted token with a NaN spoils its own loss, lse and dx (and dw), no other row."""
    c = _case(70, 64, 300, BF, 0.0, 0.0, seed=31)
    o, _ = _run(c)
    d = dict(c, x=c["x"].clone())
    d["x"][17, 5] = float("nan")
    p, _ = _run(d)
    keep = torch.arange(70) != 17
    for n in ("loss", "lse", "dx"):
        assert bool(torch.isnan(p[n][17]).all()) and torch.equal(o[n].cpu()[keep], p[n].cpu()[keep]), n


@TYPES
def test_no_token_counts(ty):
    c = _case(33, 64, 100, ty, 0.0, 0.0)
    c["t"][:] = -100
    o, _ = _run(c)
    assert all(bool((v == 0).all()) for v in o.values())


@TYPES
def test_empty(ty):
    import grouped_gemm_top_amd as G
    x, w = torch.empty(0, 64, dtype=ty, device="cuda"), torch.ones(100, 64, dtype=ty, device="cuda")
    t, f = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    r = G.linear_ce_fwd(x, w, t)
    b = G.linear_ce_bwd(f, x, w, t, r["lse"], dw=torch.ones_like(w))
    assert r["loss"].shape == (0,) and b["dx"].shape == (0, 64) and bool((b["dw"] == 0).all())


@TYPES
def test_far_logits(ty):
    """Logits of thousands: the running maximum keeps the sums finite, the target's own probability is 0 or 1."""
    c = _case(40, 64, 500, ty, 0.0, 0.0, seed=41)
    c["x"] = c["x"] * 1000
    ref, bound = _exact(c)
    o, _ = _run(c)
    _check(o, ref, bound, norms=False)


def test_each_gradient_alone_and_reproducible():
    import grouped_gemm_top_amd as G
    c = _case(300, 264, 5003, BF, 0.2, 1e-3, seed=51)
    o, up = _run(c)
    a = (up["g"], up["x"], up["w"], up["t"], o["lse"])
    for _ in range(2):
        b = G.linear_ce_bwd(*a, z_coef=c["zc"], want_dw=False)
        assert b["dw"] is None and torch.equal(b["dx"], o["dx"])
        b = G.linear_ce_bwd(*a, z_coef=c["zc"], want_dx=False)
        assert b["dx"] is None and torch.equal(b["dw"], o["dw"])
        f = G.linear_ce_fwd(*a[1:4], z_coef=c["zc"])
        assert torch.equal(f["loss"], o["loss"]) and torch.equal(f["lse"], o["lse"])


def test_ones_for_no_dloss():
    import grouped_gemm_top_amd as G
    c = _case(50, 64, 300, BF, 0.0, 0.0, seed=61)
    c["g"][:] = 1.0
    o, up = _run(c)
    dx = torch.empty_like(up["x"])
    nb = G.workspace_bytes(G.OP_LINEAR_CE_BWD, G.MOE_BF16, 50, 1, 1, 64, 300)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    st = G.lib().moe_linear_ce_bwd(G.MOE_BF16, None, up["x"].data_ptr(), up["w"].data_ptr(), up["t"].data_ptr(),
                                   o["lse"].data_ptr(), 50, 64, 300, 0.0, dx.data_ptr(), None, ws.data_ptr(), nb,
                                   torch.cuda.current_stream().cuda_stream)
    assert st == G.MOE_OK and torch.equal(dx, o["dx"])


def test_differences():
    """dx and dw along random directions against central differences of the loss in 64 bits."""
    c = _case(60, 64, 211, F32, 0.2, 0.01, seed=71)
    o, _ = _run(c)
    live = (c["t"] >= 0) & (c["t"] < 211)

    def total(x, w):
        z = x[live] @ w.t()
        lse = torch.logsumexp(z, dim=1)
        each = lse - z.gather(1, c["t"][live].long()[:, None])[:, 0] + c["zc"] * lse ** 2
        return float((each * c["g"][live].double()).sum())
    x, w, e = c["x"].double(), c["w"].double(), 1e-5
    for n, (a, b) in dict(dx=(1, 0), dw=(0, 1)).items():
        dirn = torch.randn(o[n].shape, generator=torch.Generator().manual_seed(72), dtype=torch.float64)
        num = (total(x + a * e * dirn if a else x, w + b * e * dirn if b else w) -
               total(x - a * e * dirn if a else x, w - b * e * dirn if b else w)) / (2 * e)
        ana = float((o[n].cpu().double() * dirn).sum())
        assert abs(num - ana) <= 1e-4 * max(1.0, abs(num)), n


def test_streams_and_graph():
    import grouped_gemm_top_amd as G
    c = _case(150, 136, 1001, BF, 0.2, 1e-3, seed=81)
    o, up = _run(c)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    f = G.linear_ce_fwd(up["x"], up["w"], up["t"], z_coef=c["zc"], stream=st)
    b = G.linear_ce_bwd(up["g"], up["x"], up["w"], up["t"], f["lse"], z_coef=c["zc"], stream=st)
    st.synchronize()
    assert all(torch.equal(v, o[n]) for n, v in {**f, **b}.items())
    x = up["x"].clone()
    with torch.cuda.stream(st):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            f = G.linear_ce_fwd(x, up["w"], up["t"], z_coef=c["zc"])
            b = G.linear_ce_bwd(up["g"], x, up["w"], up["t"], f["lse"], z_coef=c["zc"])
    for i in range(4):
        d = _case(150, 136, 1001, BF, 0.2, 1e-3, seed=81 + 10 * i)
        e, u2 = _run(dict(c, x=d["x"]))
        x.copy_(u2["x"])
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        for n, v in {**f, **b}.items():
            assert torch.equal(v, e[n]), (i, n)


def test_no_dloss_in_python():
    import grouped_gemm_top_amd as G
    c = _case(50, 64, 300, BF, 0.1, 1e-3, seed=63)
    c["g"][:] = 1.0
    o, up = _run(c)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for kw in ({}, dict(stream=st)):
        b = G.linear_ce_bwd(None, up["x"], up["w"], up["t"], o["lse"], z_coef=1e-3, **kw)
        torch.cuda.synchronize()
        assert torch.equal(b["dx"], o["dx"]) and torch.equal(b["dw"], o["dw"])


@pytest.mark.parametrize("N,H,V", [(37, 4096, 45007), (300, 2048, 43617)])
def test_fp32_pieces_of_a_large_projection(N, H, V):
    """V H above 512 MB / 6: W's three parts are made and read piece by piece in the forward as well, in one buffer, the last
    piece ragged (three pieces, and a second one of 97 columns), and the pairs of all pieces meet in each token's sum."""
    c = _case(N, H, V, F32, 0.2, 1e-3, seed=95)
    most = (512 << 20) // (6 * H) // 256 * 256
    assert V > most and (V % most < 256 or V > 2 * most)
    c["t"][2:6] = torch.tensor([most - 1, most, V // most * most, V // most * most - 1], dtype=torch.int32)
    ref, bound = _exact(c)
    o, _ = _run(c)
    _check(o, ref, bound)


@pytest.mark.parametrize("ty,N,H,V", [(BF, 8192, 2048, 9001), (F32, 8192, 4096, 8100), (BF, 3000, 264, 700), (F32, 3000, 264, 700),
                                      (BF, 20000, 64, 8001)], ids=str)
def test_few_of_many_tokens_count(ty, N, H, V):
    """The host sees N, the device's count is 0, 1 or 5: pieces that share launches and slices of sums over (almost) nothing.
    Rows that take no part hold NaN.  In the 2-norm: bf16 rounds dz and the result, 2^-8 each at most; fp32 as above."""
    import grouped_gemm_top_amd as G
    gen = torch.Generator(device="cuda").manual_seed(97)
    w = (H ** -0.5 * torch.randn(V, H, generator=gen, device="cuda")).to(ty)
    g = torch.rand(N, generator=gen, device="cuda") + 0.5
    rel = lambda p, q: float((p.double() - q).norm() / q.norm())  # noqa: E731
    for rows in ([], [N - 1], [0, 17, N // 2, N // 2 + 1, N - 2]):
        x = torch.full((N, H), float("nan"), device="cuda").to(ty)
        t = torch.full((N,), -100, device="cuda", dtype=torch.int32)
        dead = torch.ones(N, dtype=torch.bool, device="cuda")
        for i, r in enumerate(rows):
            x[r] = torch.randn(H, generator=gen, device="cuda")
            t[r] = (V - 1, 0, V // 2, 255 % V, 256 % V)[i]
            dead[r] = False
        f = G.linear_ce_fwd(x, w, t, z_coef=1e-3)
        b = G.linear_ce_bwd(g, x, w, t, f["lse"], z_coef=1e-3)
        assert all(bool((v[dead] == 0).all()) for v in (f["loss"], f["lse"], b["dx"])), rows
        if not rows:
            assert bool((b["dw"] == 0).all())
            continue
        xl, wd, tl = x[rows].double(), w.double(), t[rows].long()[:, None]
        z = xl @ wd.t().contiguous()
        lse = torch.logsumexp(z, dim=1)
        assert rel(f["loss"][rows], lse - z.gather(1, tl)[:, 0] + 1e-3 * lse ** 2) <= 1e-6
        dz = torch.exp(z - lse[:, None]) * (g[rows].double() * (1 + 2e-3 * lse))[:, None]
        dz.scatter_add_(1, tl, -g[rows].double()[:, None])
        tol = 2 ** -7 if ty is BF else 1e-5
        assert rel(b["dx"][rows], dz @ wd) <= tol and rel(b["dw"], dz.t().contiguous() @ xl) <= tol
