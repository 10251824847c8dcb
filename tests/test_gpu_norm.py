"""moe_add_rmsnorm and moe_add_rmsnorm_bwd against fp64 references, through the C ABI, every
buffer guarded.

Tolerances, element by element, from the arithmetic (u = 2^-24, half a step of fp32; half(t) half
a step of the stored type, 2^-8 for bf16):
* h = x + res: one fp32 addition and one store: u + half(t), relative;
* y = s r w: s, two products and r.  r comes from a sum of H <= 16384 squares, each lane adding at
  most 32 of them in a row, then 6 + 16 steps: its relative error is below (32 + 22 + 4) / 2 u (the
  square root halves it) plus a few u for the mean, the root and the division.  64 u covers all;
* codes: half a step of e4m3 (2^-4 relative, 2^-10 of the scale below its normal range) on top;
* dh = r a - r (r^2 m) h + dh_in with m = sum a h / H: 64 u of |r a| and, the sum's terms having any
  sign, 64 u of |r^3 h| sum |a h| / H for its own error plus as much for r^3's, plus the last
  additions' 2 u of each term, then the store;
* dw = sum_t dy h r: a workgroup adds its rows one after another (at most 64 in these cases), then
  at most 32 + 16 partial sums: 128 u of sum |dy h r|, which leaves 16 u for each term's own error."""
import numpy as np
import pytest

from harness import Guards

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import grouped_gemm_top_amd as G
    G.lib()


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _half(t):
    import torch
    return torch.finfo(t).eps / 2


def _guarded(g, name, t):
    """A guarded device copy of host tensor t."""
    v = g.alloc(name, t.shape, t.dtype)
    v.copy_(t)
    return v


def _make(shape, dt, seed, scale=1.0):
    import torch
    gen = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=gen)).to(dt)


def _ref_fwd(x, res, w, eps):
    s = x.double() + (res.double() if res is not None else 0)
    r = 1 / (s.square().mean(1, keepdim=True) + eps).sqrt()
    return s, s * r * (w.double() if w is not None else 1)


def _check_close(got, ref, tol, what):
    err = (got.double().cpu() - ref).abs()
    bad = err > tol + TINY
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst " \
                                f"{float((err / (tol + TINY)).max()):.3g} of it"


def _check_codes(q, sc, y, H):
    """Scales are the smallest powers of two that hold each block, codes within half a step."""
    import torch
    KS = 4 * ((H + 127) // 128)
    sc = sc.cpu()
    assert bool((sc[:, H // 32:] == 0).all()) and sc.shape[1] == KS
    X = torch.exp2(sc[:, :H // 32].double() - 127)
    v = q.cpu().view(torch.float8_e4m3fn).double().view(-1, H // 32, 32)
    yb = y.view(-1, H // 32, 32)
    top = yb.abs().amax(2)
    assert bool((top <= 448 * X * (1 + 64 * U)).all()), "a block clips"
    assert bool(((top * (1 + 64 * U) > 224 * X) | (sc[:, :H // 32] == 0)).all()), "a scale is larger than needed"
    tol = torch.maximum(2.0 ** -4 * yb.abs(), 2.0 ** -10 * X[:, :, None]) + 64 * U * yb.abs()
    assert bool(((v * X[:, :, None] - yb).abs() <= tol).all()), "a code is more than half a step off"


SHAPES = [(1, 8), (1, 2048), (3, 64), (5, 520), (7, 1016), (2, 1024), (9, 1056), (4, 2880), (2, 4096), (3, 5000),
          (2, 8192), (3, 8224), (2, 16384), (1023, 96)]


@pytest.mark.parametrize("dt,rdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("N,H", SHAPES)
def test_forward(N, H, dt, rdt):
    import torch
    import grouped_gemm_top_amd as G
    t, rt = _dt(dt), _dt(rdt)
    x, res, w = _make((N, H), t, 1), _make((N, H), rt, 2, 2.0), 1 + 0.1 * _make((H,), torch.float32, 3)
    g = Guards()
    dx, dr, dw = _guarded(g, "x", x), _guarded(g, "res", res), _guarded(g, "w", w)
    quant = H % 32 == 0
    h, y = g.alloc("h", (N, H), rt), g.alloc("y", (N, H), t)
    q = g.alloc("q", (N, H), torch.uint8) if quant else None
    sc = g.alloc("sc", (N, G.mx_scale_cols(H)), torch.uint8) if quant else None
    G.add_rmsnorm(dx, dw, residual=dr, eps=1e-5, h=h, y=y, q=q, scales=sc)
    g.check("add_rmsnorm")
    s, ref = _ref_fwd(x, res, w, 1e-5)
    _check_close(h, s, (U + _half(rt)) * s.abs(), "h")
    _check_close(y, ref, (64 * U + _half(t)) * ref.abs(), "y")
    if quant:
        _check_codes(q, sc, ref, H)
        if dt == "f32":  # the stored y is then the value the codes round
            q2, s2 = G.quantize_mxfp8(y)
            assert torch.equal(q2, q) and torch.equal(s2, sc)
    # fewer outputs give the same values; no residual, no weight
    r = G.add_rmsnorm(dx, dw, residual=dr, eps=1e-5, want_h=False, want_y=not quant, quantize=quant)
    torch.cuda.synchronize()
    assert r["h"] is None and (r["y"] is None) == quant
    assert torch.equal(r["q"], q) if quant else torch.equal(r["y"].view(torch.uint8), y.view(torch.uint8))
    r = G.add_rmsnorm(dx, eps=1e-5)
    s, ref = _ref_fwd(x, None, None, 1e-5)
    _check_close(r["h"], s, torch.zeros_like(s), "h without a residual")
    _check_close(r["y"], ref, (64 * U + _half(t)) * ref.abs(), "y without a residual")


@pytest.mark.parametrize("dt,rdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("N,H", SHAPES + [(600, 2048)])
def test_backward(N, H, dt, rdt):
    import torch
    import grouped_gemm_top_amd as G
    t, rt = _dt(dt), _dt(rdt)
    dy, h, din = _make((N, H), t, 4), _make((N, H), rt, 5, 2.0), _make((N, H), rt, 6)
    w = 1 + 0.1 * _make((H,), torch.float32, 7)
    g = Guards()
    D = {n: _guarded(g, n, v) for n, v in (("dy", dy), ("h", h), ("din", din), ("w", w))}
    dh, dx, dw = g.alloc("dh", (N, H), rt), g.alloc("dx", (N, H), t), g.alloc("dw", (H,), torch.float32)
    ws = g.alloc("ws", (G.workspace_bytes(G.OP_ADD_RMSNORM_BWD, G.MOE_BF16, N, 1, 1, H),), torch.uint8)
    G.add_rmsnorm_bwd(D["dy"], D["h"], D["w"], dh_in=D["din"], eps=1e-5, dh=dh, dx=dx, dw=dw, ws=ws)
    g.check("add_rmsnorm_bwd")
    h64, a, d64 = h.double(), dy.double() * w.double(), din.double()
    r = 1 / (h64.square().mean(1, keepdim=True) + 1e-5).sqrt()
    m, mabs = (a * h64).mean(1, keepdim=True), (a * h64).abs().mean(1, keepdim=True)
    ref = r * a - r ** 3 * m * h64 + d64
    tol = U * (66 * (r * a).abs() + 130 * (r ** 3 * h64).abs() * mabs + 2 * d64.abs())
    _check_close(dh, ref, tol + _half(rt) * ref.abs(), "dh")
    _check_close(dx, ref, tol + _half(t) * ref.abs(), "dx")
    terms = dy.double() * h64 * r
    _check_close(dw, terms.sum(0), 128 * U * terms.abs().sum(0), "dw")
    # bitwise reproducible; in place over dh_in; without dw, dh_in and w
    again = G.add_rmsnorm_bwd(D["dy"], D["h"], D["w"], dh_in=D["din"], eps=1e-5, dh=D["din"])
    torch.cuda.synchronize()
    assert torch.equal(again["dh"].view(torch.uint8), dh.view(torch.uint8)) and torch.equal(again["dw"], dw)
    plain = G.add_rmsnorm_bwd(D["dy"], D["h"], eps=1e-5, want_dw=False)
    assert plain["dw"] is None and plain["dx"] is None
    a = dy.double()
    m, mabs = (a * h64).mean(1, keepdim=True), (a * h64).abs().mean(1, keepdim=True)
    ref = r * a - r ** 3 * m * h64
    tol = U * (66 * (r * a).abs() + 130 * (r ** 3 * h64).abs() * mabs)
    _check_close(plain["dh"], ref, tol + _half(rt) * ref.abs(), "dh without a weight")


def test_gradient_against_differences():
    """The GPU's gradient along random directions against central differences of the fp64 norm.
    With a step of 2^-10 the differences' own error is the third derivative's, below 2^-20 times
    (h is of size 1, so each derivative of the norm is of the size of the first)."""
    import torch
    import grouped_gemm_top_amd as G
    N, H, eps = 3, 64, 1e-5
    h, dy, w = _make((N, H), torch.float32, 8), _make((N, H), torch.float32, 9), 1 + 0.1 * _make((H,), torch.float32, 10)
    r = G.add_rmsnorm_bwd(dy.cuda(), h.cuda(), w.cuda(), eps=eps)
    f = lambda hh, ww: float((_ref_fwd(hh, None, ww, eps)[1] * dy.double()).sum())  # noqa: E731
    st = 2.0 ** -10
    for seed in range(4):
        d, e = _make((N, H), torch.float64, 20 + seed), _make((H,), torch.float64, 30 + seed)
        num = (f(h.double() + st * d, w) - f(h.double() - st * d, w)) / (2 * st)
        size = float((r["dh"].cpu().double() * d).norm())
        assert abs(float((r["dh"].cpu().double() * d).sum()) - num) <= 1e-4 * size
        num = (f(h.double(), w.double() + st * e) - f(h.double(), w.double() - st * e)) / (2 * st)
        size = float((r["dw"].cpu().double() * e).norm())
        assert abs(float((r["dw"].cpu().double() * e).sum()) - num) <= 1e-4 * size


def test_rows_that_hold_zeros_infinities_and_nans_stay_alone():
    import torch
    import grouped_gemm_top_amd as G
    N, H = 9, 256
    x = _make((N, H), torch.bfloat16, 11)
    x[2] = 0
    x[4, 7] = float("inf")
    x[6, 200] = float("nan")
    x[8] *= 2.0 ** -60
    r = G.add_rmsnorm(x.cuda(), eps=1e-6, quantize=True)
    b = G.add_rmsnorm_bwd(torch.ones_like(x).cuda(), x.cuda(), eps=1e-6, want_dw=False)
    _, ref = _ref_fwd(x, None, None, 1e-6)
    y = r["y"].float().cpu()
    assert float(y[2].abs().max()) == 0.0 and int(r["q"][2].max()) == 0 and int(r["scales"][2].max()) == 0
    assert bool(y[6].isnan().all()) and bool(y[4, 7].isnan()) and float(y[4, :7].abs().max()) == 0.0
    for t in (0, 1, 3, 5, 7, 8):
        assert bool(((y[t].double() - ref[t]).abs() <= (2.0 ** -8 + 64 * U) * ref[t].abs() + TINY).all())
        assert bool(b["dh"][t].isfinite().all())
    assert bool(b["dh"][6].isnan().all()) and bool(b["dh"][2].isfinite().all())


def test_in_place_residual():
    import torch
    import grouped_gemm_top_amd as G
    x, res, w = _make((33, 2048), torch.bfloat16, 12).cuda(), _make((33, 2048), torch.float32, 13).cuda(), \
        _make((2048,), torch.float32, 14).cuda()
    a = G.add_rmsnorm(x, w, residual=res, quantize=True)
    mine = res.clone()
    b = G.add_rmsnorm(x, w, residual=mine, h=mine, quantize=True)
    torch.cuda.synchronize()
    assert b["h"].data_ptr() == mine.data_ptr() and torch.equal(a["h"], mine)
    assert all(torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)) for n in ("y", "q", "scales"))


def test_empty_input():
    import torch
    import grouped_gemm_top_amd as G
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    r = G.add_rmsnorm(e, quantize=True)
    assert r["y"].shape == (0, 64) and r["scales"].shape == (0, 4)
    dw = torch.full((64,), 7.0, device="cuda")
    r = G.add_rmsnorm_bwd(e, e, dw=dw)
    torch.cuda.synchronize()
    assert r["dh"].shape == (0, 64) and float(dw.abs().max()) == 0.0


def test_stream_and_graph():
    """On a stream of its own, and captured: every replay gives the eager result, with eager calls and
    new inputs in between."""
    import torch
    import grouped_gemm_top_amd as G
    N, H = 700, 2048
    x, res = _make((N, H), torch.bfloat16, 15).cuda(), _make((N, H), torch.bfloat16, 16).cuda()
    w = (1 + 0.1 * _make((H,), torch.float32, 17)).cuda()

    def both(**kw):
        f = G.add_rmsnorm(x, w, residual=res, quantize=True, **kw)
        return f, G.add_rmsnorm_bwd(f["y"], f["h"], w, dh_in=res, **kw)

    ef, eb = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sf, sb = both(stream=s)
    s.synchronize()
    assert torch.equal(sf["q"], ef["q"]) and torch.equal(sb["dw"], eb["dw"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gf, gb = both()
    for seed in range(4):
        x.copy_(_make((N, H), torch.bfloat16, 40 + seed))
        graph.replay()
        torch.cuda.synchronize()
        ef, eb = both()
        torch.cuda.synchronize()
        for a, b in ((gf, ef), (gb, eb)):
            for n in a:
                if a[n] is not None:
                    assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), n


def test_offsets_past_32_bits():
    """N H beyond 2^31 elements: the last rows are computed where they are."""
    import torch
    import grouped_gemm_top_amd as G
    H = 16384
    N = (1 << 31) // H + 5
    x = torch.zeros((N, H), dtype=torch.bfloat16, device="cuda")
    tail = _make((3, H), torch.bfloat16, 18)
    x[-3:] = tail.cuda()
    r = G.add_rmsnorm(x, eps=1e-5, want_h=False, quantize=True)
    b = G.add_rmsnorm_bwd(x, x, eps=1e-5)
    torch.cuda.synchronize()
    _, ref = _ref_fwd(tail, None, None, 1e-5)
    _check_close(r["y"][-3:], ref, (64 * U + 2.0 ** -8) * ref.abs(), "y")
    _check_codes(r["q"][-3:], r["scales"][-3:], ref, H)
    assert float(r["y"][0].abs().max()) == 0.0 and float(b["dh"][0].abs().max()) == 0.0
    h64 = tail.double()
    rr = 1 / (h64.square().mean(1, keepdim=True) + 1e-5).sqrt()
    terms = h64 * h64 * rr
    # (rows of zeros add nothing, but the tail's rows may meet in one workgroup's sum)
    _check_close(b["dw"], terms.sum(0), 128 * U * terms.abs().sum(0), "dw")


@pytest.mark.parametrize("N,H,quant", [((1 << 21) + 3, 32, True), ((1 << 22) + 1, 8, False), ((1 << 26) + 5, 8, False)])
def test_more_rows_than_one_launch_takes(N, H, quant):
    """Rows are independent: the rows around 2^21, 2^22 and at the end equal those of a call of their own."""
    import torch
    import grouped_gemm_top_amd as G
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(N, H, device="cuda", generator=gen, dtype=torch.bfloat16)
    w = torch.rand(H, device="cuda", generator=gen) + 0.5
    r = G.add_rmsnorm(x, w, residual=x, want_h=quant, quantize=quant)
    for lo in (0, (1 << 21) - 5, (1 << 22) - 5, N - 9):
        hi = min(N, lo + 9)
        if lo >= N:
            continue
        one = G.add_rmsnorm(x[lo:hi].contiguous(), w, residual=x[lo:hi].contiguous(), want_h=quant, quantize=quant)
        for key, v in one.items():
            assert (v is None) == (r[key] is None)
            if v is not None:
                assert torch.equal(v, r[key][lo:hi]), (key, lo)


@pytest.mark.parametrize("dt,rdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("N,H", [(4099, 96), (4099, 1024), (2051, 2048), (1101, 2880), (1101, 8192), (1101, 8224)])
def test_backward_of_many_rows(N, H, dt, rdt):
    """More rows than one turn of the backward's 512 workgroups takes, with a ragged last turn, at each of its
    six widths: every row of dh and dx, and dw across the turns."""
    test_backward(N, H, dt, rdt)
