"""The layer with [G | U] kept as MX-FP8 codes (moe_grouped_gemm_fwd_ckpt8, moe_layer_bwd_ckpt8) and
moe_dequantize_mxfp8, through the C ABI, every buffer guarded.

A code's value is exact in bf16, so the backward at codes is held bit for bit to moe_layer_bwd at the
dequantized [G | U], which the oracle tests pin, and to the formulas in 64 bits.  Tolerances (u = 2^-24): a G or U is a sum of H
products, off by at most ez = (H + 8) u sum |x w|; its code by half an e4m3 step of the value, 2^-4 |v|, or 2^-10 of the
block's scale where that is more.  Backward, 2-norm: every rounding to bf16 is off by at most 2^-8 of its
value, uniformly, 2^-8 / sqrt 3 = 0.00226 in the norm: dW has two (dH or A', and its own), dx three (dH, the expert rows, its
own), ds none (fp32 sums of H and I products and the exponential, 1e-5)."""
import numpy as np
import pytest
import torch

from harness import Guards

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import grouped_gemm_top_amd as G
    G.lib()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _case(N, H, I, E, k, routing="topk", seed=1, ints=False, drop=0):
    """Inputs and a plan; the last `drop` experts get no token."""
    import grouped_gemm_top_amd as G
    g, gen = Guards(), _gen(seed)

    def make(name, *shape, scale=1.0):
        t = g.alloc(name, shape, BF)
        t.copy_(torch.randint(-2, 3, shape, generator=gen, device="cuda") if ints else
                scale * torch.randn(shape, generator=gen, device="cuda"))
        return t
    c = dict(g=g, N=N, H=H, I=I, E=E, k=k, x=make("x", N, H), dout=make("dout", N, H),
             wg=make("wg", E, I, H, scale=H ** -0.5), wu=make("wu", E, I, H, scale=H ** -0.5),
             wd=make("wd", E, H, I, scale=I ** -0.5))
    logits = torch.randn(N, E, generator=gen, device="cuda")
    if drop:
        logits[:, E - drop:] -= 100
    alloc = lambda name, n, dt: g.alloc("plan." + name, (n,), dt)  # noqa: E731
    if routing == "tr":
        c["plan"] = G.route_token_rounding(logits, k, 16, plan=G.Plan(N, E, k, G.PLAN_TR, 16, alloc=alloc))[0]
    elif routing == "cap":
        cap = max(1, N * k // E)
        c["plan"] = G.route_capacity(logits, k, cap, plan=G.Plan(N, E, k, G.PLAN_CAP, cap, alloc=alloc))[0]
    else:
        idx, w, _ = G.route_topk(logits, k)
        c["plan"] = G.permute(idx, w, E, plan=G.Plan(N, E, k, alloc=alloc))
    return c


def _fwd(c):
    import grouped_gemm_top_amd as G
    g, p, I, H = c["g"], c["plan"], c["I"], c["H"]
    mc = max(p.M_cap, 1)
    hq, hs = g.alloc("hq", (mc, 2 * I), U8), g.alloc("hs", (mc, 2 * G.mx_scale_cols(I)), U8)
    y = g.alloc("y", (mc, H), BF)
    ws = g.alloc("ws", (G.workspace_bytes(G.OP_GEMM_FWD, G.MOE_BF16, p.N, p.E, p.k, H, I, p.M_cap),), U8)
    G.grouped_gemm_fwd_ckpt8(c["x"], c["wg"], c["wu"], c["wd"], p, hq=hq, hs=hs, y=y, ws=ws)
    g.check("grouped_gemm_fwd_ckpt8")
    return hq, hs, y


def _bwd(c, hq, hs, x=None):
    import grouped_gemm_top_amd as G
    g, p, I, H, E, N = c["g"], c["plan"], c["I"], c["H"], c["E"], c["N"]
    o = dict(dx=g.alloc("dx", (N, H), BF), dw_gate=g.alloc("dwg", (E, I, H), BF), dw_up=g.alloc("dwu", (E, I, H), BF),
             dw_down=g.alloc("dwd", (E, H, I), BF),
             ds=g.alloc("ds", (N, c["k"]) if p.kind == G.PLAN_TOPK else (max(p.M_cap, 1),), F32))
    ws = g.alloc("wsb", (G.workspace_bytes(G.OP_LAYER_BWD_CKPT8, G.MOE_BF16, p.N, p.E, p.k, H, I, p.M_cap),), U8)
    G.layer_bwd_ckpt8(c["dout"], c["x"] if x is None else x, c["wg"], c["wu"], c["wd"], p, (hq, hs), ws=ws, **o)
    g.check("layer_bwd_ckpt8")
    return o


def _value(hq, hs, I):
    """[G | U] of codes, exactly, in fp64."""
    M = hq.shape[0]
    v = hq.view(torch.float8_e4m3fn).double().view(M, 2, I // 32, 32)
    s = hs.view(M, 2, -1)[:, :, :I // 32].double()
    return (v * torch.exp2(s - 127)[..., None]).view(M, 2, I)


def _rows(c):
    """The plan's rows on the host: token, expert, weight."""
    h = c["plan"].host()
    e = np.repeat(np.arange(c["E"]), h["counts"])
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (h["row_token"].astype(np.int64), e.astype(np.int64),
                                                                       h["row_w"])], h


def _gu(c, tok, exp):
    """G and U of every row in fp64 and the bound of their sums."""
    x, M = c["x"].double(), tok.numel()
    v, b = (torch.zeros(M, 2, c["I"], dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(c["E"]):
        r = (exp == e).nonzero()[:, 0]
        for h, n in enumerate(("wg", "wu")):
            w = c[n][e].double()
            v[r, h] = x[tok[r]] @ w.t()
            b[r, h] = (c["H"] + 8) * U * (x[tok[r]].abs() @ w.abs().t())
    return v, b


def _formulas(c, gu, x, tok, exp, w):
    """The backward's outputs in fp64, dS per row."""
    N, H, I, E = (c[n] for n in "NHIE")
    d64 = dict(dtype=torch.float64, device="cuda")
    o = dict(dx=torch.zeros(N, H, **d64), dw_gate=torch.zeros(E, I, H, **d64), dw_up=torch.zeros(E, I, H, **d64),
             dw_down=torch.zeros(E, H, I, **d64), ds=torch.zeros(tok.numel(), **d64))
    dout, w = c["dout"].double(), w.double()
    for e in range(E):
        r = (exp == e).nonzero()[:, 0]
        if not r.numel():
            continue
        t, g, u = tok[r], gu[r, 0], gu[r, 1]
        s = torch.sigmoid(g)
        a, da = g * s * u, dout[t] @ c["wd"][e].double()
        o["ds"][r] = (da * a).sum(1)
        da = da * w[r][:, None]
        dg, du = da * u * s * (1 + g * (1 - s)), da * g * s
        o["dx"].index_add_(0, t, dg @ c["wg"][e].double() + du @ c["wu"][e].double())
        o["dw_gate"][e], o["dw_up"][e] = dg.t() @ x[t], du.t() @ x[t]
        o["dw_down"][e] = dout[t].t() @ (a * w[r][:, None])
    return o


SHAPES = [  # N, H, I, E, k, routing, experts without tokens
    (1, 64, 32, 4, 1, "topk", 0), (64, 64, 32, 8, 2, "topk", 3), (100, 136, 96, 5, 3, "topk", 0),
    (333, 264, 736, 7, 4, "topk", 2), (700, 512, 160, 3, 1, "topk", 0), (250, 96, 224, 6, 6, "topk", 0),
    (777, 1440, 256, 16, 4, "topk", 1), (300, 200, 96, 8, 2, "tr", 0), (300, 200, 288, 8, 2, "cap", 2),
]


@pytest.mark.parametrize("N,H,I,E,k,routing,drop", SHAPES)
def test_layer(N, H, I, E, k, routing, drop):
    import grouped_gemm_top_amd as G
    c = _case(N, H, I, E, k, routing, drop=drop)
    hq, hs, y = _fwd(c)
    (tok, exp, w), h = _rows(c)
    M = tok.numel()
    # the forward: y as without codes, the codes nearest to the sums
    hc, y0 = G.grouped_gemm_fwd(c["x"], c["wg"], c["wu"], c["wd"], c["plan"])
    assert torch.equal(y[:M], y0[:M])
    v, ez = _gu(c, tok, exp)
    KS = G.mx_scale_cols(I)
    got = _value(hq[:M], hs[:M], I)
    X = torch.exp2(hs[:M].view(M, 2, KS)[:, :, :I // 32].double() - 127)
    step = torch.maximum(2.0 ** -4 * (v.abs() + ez), (2.0 ** -10 * X).repeat_interleave(32, dim=2))
    assert bool(((got - v).abs() <= step + ez).all())
    top = v.abs().view(M, 2, I // 32, 32).amax(3)
    et = ez.view(M, 2, I // 32, 32).amax(3)
    assert bool((top - et <= 448 * X).all()) and bool((top + et > 224 * X).all())
    assert bool((hs[:M].view(M, 2, KS)[:, :, I // 32:] == 0).all())
    # the backward: bit for bit the one at the bf16 values, and the formulas
    o = _bwd(c, hq, hs)
    mc = hq.shape[0]
    gu = G.dequantize_mxfp8(hq.view(mc, 2, I), hs.view(mc, 2, KS)).view(mc, 2 * I)
    assert torch.equal(gu[:M].double().view(M, 2, I), got)
    p = G.layer_bwd(c["dout"], c["x"], c["wg"], c["wu"], c["wd"], c["plan"], gu)
    used = slice(0, M) if routing != "topk" else slice(None)
    for n in o:
        a, b = (o[n][used], p[n][used]) if n == "ds" else (o[n], p[n])
        assert torch.equal(a, b), n
    ref = _formulas(c, got, c["x"].double(), tok, exp, w)
    ds = o["ds"][:M] if routing != "topk" else o["ds"].view(-1)[torch.from_numpy(h["row_pair"].astype(np.int64)).cuda()]
    for n, tol in dict(dx=0.0039 * 1.2, dw_gate=0.0032 * 1.2, dw_up=0.0032 * 1.2, dw_down=0.0032 * 1.2, ds=1e-5).items():
        d = (ds if n == "ds" else o[n]).double() - ref[n]
        # (few values need not average: one rounding may be all of 2^-8)
        tol = tol if M * I >= 4096 or n == "ds" else 3 * 2 ** -8
        assert float(d.norm()) <= tol * float(ref[n].norm()), (n, float(d.norm() / ref[n].norm()))
    # x as codes: the weights' gradients at the values these stand for, all else unchanged
    if H % 32:
        return
    xq, xs = G.quantize_mxfp8(c["x"])
    xv = G.dequantize_mxfp8(xq, xs)
    q = _bwd(c, hq, hs, x=(xq, xs))
    p = G.layer_bwd(c["dout"], xv, c["wg"], c["wu"], c["wd"], c["plan"], gu)
    for n in o:
        a, b = (q[n][used], p[n][used]) if n == "ds" else (q[n], p[n])
        assert torch.equal(a, b), n
    assert torch.equal(q["dx"], o["dx"]) and torch.equal(q["dw_down"], o["dw_down"])


@pytest.mark.parametrize("N,H,I,E,k", [(50, 64, 32, 4, 2), (200, 136, 416, 3, 2), (600, 64, 128, 2, 1)])
def test_codes_exact(N, H, I, E, k):
    """Whole-number inputs: G and U are exact, so every code and scale is the one moe_quantize_mxfp8 gives."""
    import grouped_gemm_top_amd as G
    c = _case(N, H, I, E, k, ints=True, seed=5)
    hq, hs, _ = _fwd(c)
    (tok, exp, _), _ = _rows(c)
    v, _ = _gu(c, tok, exp)
    q, s = G.quantize_mxfp8(v.float())
    M = N * k
    assert torch.equal(hs.view(M, 2, -1), s) and torch.equal(hq.view(M, 2, I), q)


def test_differences():
    """dx, dw_gate and dw_down against central differences of the layer around the codes' [G | U], in 64 bits."""
    c = _case(40, 64, 96, 4, 2, seed=9)
    hq, hs, _ = _fwd(c)
    (tok, exp, w), _ = _rows(c)
    o = _bwd(c, hq, hs)
    gu0, x0 = _value(hq, hs, 96), c["x"].double()
    W = {n: c[n].double() for n in ("wg", "wu", "wd")}

    def total(dx=None, dwg=None, dwd=None):
        g, u = gu0[:, 0].clone(), gu0[:, 1].clone()
        out = torch.zeros_like(x0)
        for e in range(4):
            r = (exp == e).nonzero()[:, 0]
            if dx is not None:
                g[r] += dx[tok[r]] @ W["wg"][e].t()
                u[r] += dx[tok[r]] @ W["wu"][e].t()
            if dwg is not None:
                g[r] += x0[tok[r]] @ dwg[e].t()
            a = torch.nn.functional.silu(g[r]) * u[r]
            out.index_add_(0, tok[r], w[r].double()[:, None] * (a @ (W["wd"][e] + (0 if dwd is None else dwd[e])).t()))
        return float((out * c["dout"].double()).sum())
    for n, kw, shape in (("dx", "dx", x0.shape), ("dw_gate", "dwg", W["wg"].shape), ("dw_down", "dwd", W["wd"].shape)):
        d = torch.randn(shape, generator=_gen(10), device="cuda", dtype=torch.float64)
        num = (total(**{kw: 1e-5 * d}) - total(**{kw: -1e-5 * d})) / 2e-5
        ana = float((o[n].double() * d).sum())
        # the outputs' rounding: 2^-8 of each of sum d_i o_i's terms, of random signs
        assert abs(num - ana) <= 4 * 0.0039 * float((o[n].double() * d).norm()) + 1e-6 * abs(num), n


def test_empty():
    import grouped_gemm_top_amd as G
    plan = G.Plan(0, 4, 2)
    for t in (plan.counts, plan.offsets, plan.tok_ptr):
        t.zero_()
    z = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")  # noqa: E731
    (hq, hs), y = G.grouped_gemm_fwd_ckpt8(z(0, 64), z(4, 32, 64), z(4, 32, 64), z(4, 64, 32), plan)
    r = G.layer_bwd_ckpt8(z(0, 64), z(0, 64), z(4, 32, 64), z(4, 32, 64), z(4, 64, 32), plan, (hq, hs),
                          dw_gate=torch.ones(4, 32, 64, dtype=BF, device="cuda"))
    assert r["dx"].shape == (0, 64) and all(bool((r[n] == 0).all()) for n in ("dw_gate", "dw_up", "dw_down"))
    assert G.dequantize_mxfp8(torch.zeros(0, 64, dtype=U8, device="cuda"), torch.zeros(0, 4, dtype=U8, device="cuda")).shape == (0, 64)


def test_nan_stays_in_its_rows():
    c = _case(60, 64, 64, 4, 2, seed=13)
    hq, hs, y = _fwd(c)
    o = _bwd(c, hq, hs)
    c["x"][7, 3] = float("nan")
    q2, s2, y2 = _fwd(c)
    (tok, _, _), _ = _rows(c)
    keep = tok != 7
    assert torch.equal(hq[keep], q2[keep]) and torch.equal(hs[keep], s2[keep]) and torch.equal(y[keep], y2[keep])
    assert bool(torch.isnan(_value(q2, s2, 64)[~keep]).all())
    p = _bwd(c, q2, s2)
    rest = torch.arange(60, device="cuda") != 7
    assert torch.equal(o["dx"][rest], p["dx"][rest]) and bool(torch.isnan(p["dx"][7]).all())


@pytest.mark.parametrize("ty", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (37, 2880), (513, 128)])
def test_dequantize(rows, K, ty):
    """Every code at every scale, exactly; NaN codes stay NaN."""
    import grouped_gemm_top_amd as G
    g, gen = Guards(), _gen(17)
    q, s = g.alloc("q", (rows, K), U8), g.alloc("s", (rows, G.mx_scale_cols(K)), U8)
    q.copy_(torch.randint(0, 256, (rows, K), generator=gen, device="cuda"))
    s.copy_(torch.randint(0, 240, s.shape, generator=gen, device="cuda"))
    out = g.alloc("out", (rows, K), ty)
    G.dequantize_mxfp8(q, s, out=out)
    g.check("dequantize_mxfp8")
    v = q.view(torch.float8_e4m3fn).double().view(rows, K // 32, 32)
    ref = (v * torch.exp2(s[:, :K // 32].double() - 127)[..., None]).view(rows, K).to(ty)
    assert torch.equal(torch.nan_to_num(out.float(), nan=12345.0), torch.nan_to_num(ref.float(), nan=12345.0))


def test_streams_graph_and_repeats():
    import grouped_gemm_top_amd as G
    c = _case(200, 128, 96, 6, 2, seed=21)
    a = (c["wg"], c["wu"], c["wd"], c["plan"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    xq = G.quantize_mxfp8(c["x"])
    torch.cuda.synchronize()
    x, (q, s) = c["x"].clone(), xq

    def step(stream=None):
        h, y = G.grouped_gemm_fwd_ckpt8(x, *a, stream=stream)
        return dict(y=y, hq=h[0], hs=h[1], **G.layer_bwd_ckpt8(c["dout"], (q, s), *a, h, stream=stream))
    o = step()
    torch.cuda.synchronize()
    p = step(st)
    st.synchronize()
    assert all(torch.equal(o[n], p[n]) for n in o)
    with torch.cuda.stream(st):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            r = step()
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=_gen(30 + i), device="cuda"))
        e = step()
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(e[n], r[n]) for n in e), i
