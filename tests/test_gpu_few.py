"""moe_layer_few and moe_layer_few_mxfp8 through the C ABI, every buffer guarded, against the formulas in 64 bits.

Tolerances (u = 2^-24; half: 2^-8 for bf16, u for fp32).  A sum of n products is off by at most (n + 8) u sum |x w|.
Router weights: twice the largest error of a token's logits and 32 u.  a' = w silu(g) u is off by what its factors
are (silu's slope is at most 1.1; its exponential and reciprocal 16 u) and by its rounding, half |a'|; out sums those
through |W_down|, adds (k I + 8) u sum |a' W_down| and rounds once."""
import pytest
import torch

from harness import Guards

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
KINDS = pytest.mark.parametrize("kind", ["bf16", "f32", "mxfp8"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import grouped_gemm_top_amd as G
    G.lib()


def _case(N, H, I, E, k, kind, seed=1, bias=False, same=False):
    """same: every token names the same experts."""
    import grouped_gemm_top_amd as G
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ty = F32 if kind == "f32" else BF
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    c = dict(N=N, H=H, I=I, E=E, k=k, kind=kind, x=rnd(N, H).to(ty), wr=1.5 * H ** -0.5 * rnd(H, E),
             b=rnd(E) if bias else None)
    if same:
        c["b"] = 40.0 * torch.arange(E, device="cuda").float().roll(3)
    for n, s in (("wg", (E, I, H)), ("wu", (E, I, H)), ("wd", (E, H, I))):
        w = rnd(*s) * s[2] ** -0.5
        c[n] = G.quantize_mxfp8(w) if kind == "mxfp8" else w.to(ty)
    return c


def _val(w):
    import grouped_gemm_top_amd as G
    return G.dequantize_mxfp8(*w, dtype=F32).double() if isinstance(w, tuple) else w.double()


def _run(c, guarded=True):
    import grouped_gemm_top_amd as G
    g = Guards()

    def up(name, t):
        if t is None:
            return None
        if isinstance(t, tuple):
            return tuple(up(name + str(i), v) for i, v in enumerate(t))
        v = g.alloc(name, t.shape, t.dtype)
        v.copy_(t)
        return v
    a = {n: up(n, c[n]) for n in ("x", "wr", "b", "wg", "wu", "wd")}
    N, H, I, E, k = (c[n] for n in "NHIEk")
    ty = c["x"].dtype
    o = dict(out=g.alloc("out", (N, H), ty), topk_idx=g.alloc("idx", (N, k), I32), topk_w=g.alloc("w", (N, k), F32))
    nb = G.workspace_bytes(G.OP_LAYER_FEW, G.MOE_BF16 if ty == BF else G.MOE_F32, N, E, k, H, I)
    ws = g.alloc("ws", (nb,), U8)
    ws.fill_(0xFF)  # (as fp32: NaN)
    G.layer_few(a["x"], a["wr"], a["wg"], a["wu"], a["wd"], k, bias=a["b"], ws=ws, **o)
    g.check("layer_few")
    return o, a


def _check(c, o, tokens=None):
    N, H, I, E, k = (c[n] for n in "NHIEk")
    ty = c["x"].dtype
    half = torch.finfo(ty).eps / 2
    x, wr = c["x"].double(), c["wr"].double()
    z = x @ wr
    ez = (H + 8) * U * (x.abs() @ wr.abs())
    if c["b"] is not None:
        z = z + c["b"].double()
        ez = ez + U * z.abs()
    idx, w = o["topk_idx"].long(), o["topk_w"].double()
    # the choice: each slot's logit at least the next one's and every other expert's, within the errors
    zi = z.gather(1, idx)
    worst = ez.max(dim=1, keepdim=True).values
    assert bool((idx >= 0).all() and (idx < E).all())
    assert bool((zi[:, 1:] <= zi[:, :-1] + 2 * worst).all())
    rest = z.scatter(1, idx, -float("inf"))
    assert bool((rest <= zi[:, -1:] + 2 * worst).all())
    assert all(len(set(r)) == k for r in idx.tolist())
    we = torch.softmax(zi, dim=1)
    assert bool(((w - we).abs() <= (2 * worst + 32 * U) * we + 1e-38).all())
    # the experts at the call's own choice
    out, bound = torch.zeros(N, H, dtype=torch.float64, device="cuda"), torch.zeros(N, H, dtype=torch.float64, device="cuda")
    for e in sorted(set(idx.flatten().tolist())):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        pair = lambda n: _val(tuple(v[e] for v in c[n]) if isinstance(c[n], tuple) else c[n][e])  # noqa: E731
        wg, wu, wd = pair("wg"), pair("wu"), pair("wd")
        g, u = x[t] @ wg.t(), x[t] @ wu.t()
        eg, eu = ((H + 8) * U * (x[t].abs() @ v.abs().t()) for v in (wg, wu))
        wt = w[t, j][:, None]
        s = torch.nn.functional.silu(g)
        a = wt * s * u
        ea = wt * (1.1 * eg * u.abs() + (s.abs() + 1.1 * eg) * eu) + 16 * U * a.abs()
        ea = ea + half * (a.abs() + ea)
        out.index_add_(0, t, a @ wd.t())
        bound.index_add_(0, t, (ea + (k * I + 8) * U * a.abs()) @ wd.abs().t())
    bound = bound + half * (out.abs() + bound)
    rows = slice(None) if tokens is None else tokens
    d = (o["out"].double() - out).abs()[rows]
    assert bool((d <= bound[rows]).all()), float((d - bound[rows]).max())
    if N * H >= 512:  # two roundings, uniform in half a step: 2^-8 / sqrt 3 each, together 0.0032
        assert float(d.norm()) <= (4e-3 if ty == BF else 5e-6) * float(out[rows].norm())


SHAPES = [  # N, H, I, E, k
    (1, 32, 32, 1, 1), (1, 64, 96, 4, 2), (2, 96, 32, 4, 4), (1, 2048, 512, 128, 8), (3, 160, 224, 65, 5),
    (15, 288, 64, 16, 3), (16, 512, 128, 200, 8), (17, 128, 160, 64, 4), (31, 96, 96, 8, 8), (33, 416, 96, 256, 2),
    (64, 256, 64, 32, 8), (64, 64, 32, 1000, 32), (61, 1440, 544, 24, 4), (5, 4096, 32, 300, 1), (7, 32, 2080, 3, 2),
]


@KINDS
@pytest.mark.parametrize("N,H,I,E,k", SHAPES)
def test_against_formulas(N, H, I, E, k, kind):
    c = _case(N, H, I, E, k, kind, bias=N % 2 == 0)
    o, _ = _run(c)
    _check(c, o)


@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("N,H,I,E,k", [(1, 8, 8, 2, 1), (9, 24, 40, 5, 2), (40, 72, 8, 7, 3), (64, 1000, 104, 12, 5)])
def test_multiples_of_eight(N, H, I, E, k, ty):
    c = _case(N, H, I, E, k, ty, seed=3)
    o, _ = _run(c)
    _check(c, o)


@KINDS
@pytest.mark.parametrize("N,H,I,E,k", [(2, 96, 2080, 32, 8), (10, 128, 1024, 128, 8), (24, 160, 544, 80, 6),
                                       (61, 224, 544, 64, 5), (40, 32, 800, 100, 2)])
def test_narrow_rows_and_many_tasks(N, H, I, E, k, kind):
    """Where a few of a workgroup's wavefronts share a task, and it has several at a time."""
    c = _case(N, H, I, E, k, kind, seed=6)
    o, _ = _run(c)
    _check(c, o)


@KINDS
@pytest.mark.parametrize("N", [1, 16, 48, 64])
def test_all_tokens_name_the_same_experts(N, kind):
    c = _case(N, 128, 96, 6, 2, kind, seed=5, same=True)
    o, _ = _run(c)
    assert len(set(map(tuple, o["topk_idx"].tolist()))) == 1
    _check(c, o)


def test_choice_is_exact_on_ties():
    """Whole-number logits with many ties, -0 among them: z descending, expert ascending."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    c = _case(50, 64, 32, 77, 9, "bf16", seed=7)
    c["x"] = torch.randint(-1, 2, (50, 64), generator=gen, device="cuda").to(BF)
    c["wr"] = torch.randint(-1, 2, (64, 77), generator=gen, device="cuda").float()
    c["b"] = torch.where(torch.rand(77, generator=gen, device="cuda") < 0.5, -0.0, 0.0)
    o, _ = _run(c)
    z = c["x"].float().cpu() @ c["wr"].cpu()
    ref = torch.sort(z + 0.0, dim=1, descending=True, stable=True)
    assert torch.equal(o["topk_idx"].cpu(), ref.indices[:, :9].int())
    _check(c, o)


def test_router_agrees_with_route_topk():
    import grouped_gemm_top_amd as G
    c = _case(60, 256, 32, 128, 8, "bf16", seed=9, bias=True)
    o, _ = _run(c)
    idx, w, _ = G.route_topk(G.router_logits(c["x"], c["wr"]), 8, bias=c["b"])
    assert torch.equal(idx, o["topk_idx"]) and float((w - o["topk_w"]).abs().max()) <= 1e-5


@KINDS
def test_a_token_alone(kind):
    """A token of a batch gets what it gets alone, but for the order of fp32 sums (its roundings may then differ)."""
    c = _case(40, 128, 96, 20, 3, kind, seed=11)
    o, _ = _run(c)
    for t in (0, 17, 39):
        p, _ = _run(dict(c, N=1, x=c["x"][t:t + 1].contiguous()))
        assert torch.equal(p["topk_idx"][0], o["topk_idx"][t])
        d = (p["out"][0].double() - o["out"][t].double()).norm()
        assert float(d) <= (4e-3 if kind != "f32" else 2e-6) * float(o["out"][t].double().norm())


def test_experts_left_out():
    """-inf leaves an expert out; with fewer than k others the rest weigh nothing; with none, out is 0."""
    c = _case(20, 64, 32, 10, 4, "bf16", seed=13)
    c["b"] = torch.zeros(10, device="cuda")
    c["b"][[1, 2, 5, 7]] = -float("inf")
    o, _ = _run(c)
    assert not bool(torch.isin(o["topk_idx"], torch.tensor([1, 2, 5, 7], device="cuda")).any())
    _check(c, o)
    c["b"][:] = -float("inf")
    c["b"][[3, 8]] = 0.0
    o, _ = _run(c)
    assert bool((o["topk_idx"][:, :2].sort(dim=1).values == torch.tensor([3, 8], device="cuda")).all())
    assert o["topk_idx"][0, 2:].tolist() == [0, 1] and bool((o["topk_w"][:, 2:] == 0).all())
    assert bool(((o["topk_w"].sum(1) - 1).abs() <= 4 * U).all())
    c["b"][:] = -float("inf")
    o, _ = _run(c)
    assert bool((o["topk_w"] == 0).all() and (o["out"] == 0).all() and (o["topk_idx"] == torch.arange(4, device="cuda")).all())


@KINDS
def test_a_spoilt_token_and_a_spoilt_expert(kind):
    c = _case(30, 96, 64, 12, 3, kind, seed=17)
    o, _ = _run(c)
    d = dict(c, x=c["x"].clone())
    d["x"][4] = float("nan")
    d["x"][5, 7] = float("inf")
    p, _ = _run(d)
    keep = torch.ones(30, dtype=torch.bool, device="cuda")
    keep[[4, 5]] = False
    # (the experts that token 4 and 5 named before may have left the batch: sums in another order)
    _check(c, dict(out=torch.where(keep[:, None], p["out"], o["out"]), topk_idx=torch.where(keep[:, None], p["topk_idx"], o["topk_idx"]),
                   topk_w=torch.where(keep[:, None], p["topk_w"], o["topk_w"])))
    assert bool(torch.isnan(p["out"][4]).all()) and bool(((p["topk_idx"] >= 0) & (p["topk_idx"] < 12)).all())
    if kind == "mxfp8":
        return
    e = int(o["topk_idx"][0, 0])
    d = dict(c, wd=c["wd"].clone(), wg=c["wg"].clone())
    d["wd"][e] = float("inf")
    d["wg"][e, 3] = float("nan")
    p, _ = _run(d)
    names = (o["topk_idx"] == e).any(dim=1)
    assert bool(names.any()) and not bool(names.all())
    assert torch.equal(p["out"][~names], o["out"][~names])
    assert bool(torch.isnan(p["out"][names]).all())


@pytest.mark.parametrize("code", [0, 1, 2, 9, 253])
def test_smallest_and_largest_scales(code):
    """W_down at the ends of the scale codes' range: its values are exact in bf16 down to 2^-133, out's in bf16 and fp32 too
    (subnormals: half of 2^-133 is allowed for every rounding)."""
    c = _case(9, 64, 64, 4, 2, "mxfp8", seed=29)
    q, s = c["wd"]
    q = (q & 0x87) | 0x08 if code == 253 else q  # (magnitudes below 2^-5: out stays finite)
    c["wd"] = (q, torch.full_like(s, code))
    c["wd"][1][:, :, 2:] = 0
    o, _ = _run(c)
    idx, w = o["topk_idx"].long(), o["topk_w"].double()
    ref, size = torch.zeros(9, 64, dtype=torch.float64, device="cuda"), torch.zeros(9, 64, dtype=torch.float64, device="cuda")
    x, wg, wu, wd = c["x"].double(), _val(c["wg"]), _val(c["wu"]), q.view(torch.float8_e4m3fn).double() * 2.0 ** (code - 127)
    for t in range(9):
        for j in range(2):
            e = idx[t, j]
            a = w[t, j] * torch.nn.functional.silu(wg[e] @ x[t]) * (wu[e] @ x[t])
            ref[t] += wd[e] @ a
            size[t] += wd[e].abs() @ a.abs()
    # a' is off by 2^-8 and what its own factors are (below 2^-12 here), out by 2^-8 and the subnormals' steps of 64 * 2 terms
    assert bool(((o["out"].double() - ref).abs() <= 2 ** -8 * ref.abs() + 1.07 * 2 ** -8 * size + 130 * 2.0 ** -134).all())


def test_empty():
    import grouped_gemm_top_amd as G
    c = _case(1, 64, 32, 4, 2, "bf16")
    r = G.layer_few(c["x"][:0], c["wr"], c["wg"], c["wu"], c["wd"], 2)
    assert r["out"].shape == (0, 64) and r["topk_idx"].shape == (0, 2)


def test_offsets_past_32_bits():
    """Weights of more than 4 GiB a matrix: the last experts."""
    gen = torch.Generator(device="cuda").manual_seed(19)
    N, H, I, E, k = 5, 4096, 2048, 300, 2
    c = dict(N=N, H=H, I=I, E=E, k=k, kind="bf16", x=torch.randn(N, H, generator=gen, device="cuda").to(BF),
             wr=torch.randn(H, E, generator=gen, device="cuda") / 64, b=torch.zeros(E, device="cuda"))
    c["b"][-6:] = 20.0
    for n, s in (("wg", (E, I, H)), ("wu", (E, I, H)), ("wd", (E, H, I))):
        c[n] = torch.empty(s, dtype=BF, device="cuda")
        for e in range(E):
            c[n][e] = torch.randn(s[1:], generator=gen, device="cuda") * s[2] ** -0.5
    import grouped_gemm_top_amd as G
    o = G.layer_few(c["x"], c["wr"], c["wg"], c["wu"], c["wd"], k, bias=c["b"])
    assert int(o["topk_idx"].min()) >= E - 6
    _check(c, o)


@KINDS
def test_streams_graph_and_repeats(kind):
    import grouped_gemm_top_amd as G
    c = _case(20, 128, 96, 30, 4, kind, seed=23, bias=True)
    o, a = _run(c)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    call = lambda x, **kw: G.layer_few(x, a["wr"], a["wg"], a["wu"], a["wd"], 4, bias=a["b"], **kw)  # noqa: E731
    for _ in range(3):
        r = call(a["x"], stream=st)
        st.synchronize()
        assert all(torch.equal(r[n], o[n]) for n in o)
    # two calls at once, on two streams, with workspaces of their own
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        r, q = call(a["x"], stream=st), call(a["x"], stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(r[n], o[n]) and torch.equal(q[n], o[n]) for n in o)
    x = a["x"].clone()
    with torch.cuda.stream(st):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            r = call(x)
    for i in range(5):
        x.copy_(torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(40 + i), device="cuda"))
        e = call(x)
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(e[n], r[n]) for n in e), i


# ------------------------------------------------------------------ a single token: a choice of its own, by counting ranks
# (a kernel of its own each for E <= 128, E <= 256 and beyond)

@KINDS
@pytest.mark.parametrize("H,I,E,k", [(64, 32, 128, 32), (96, 64, 129, 8), (128, 32, 200, 5), (64, 64, 256, 32), (160, 32, 257, 9),
                                     (64, 32, 1000, 32), (64, 32, 1024, 1), (2048, 64, 256, 8), (4096, 32, 513, 8)])
def test_one_token(H, I, E, k, kind):
    c = _case(1, H, I, E, k, kind, seed=101 + E, bias=E % 2 == 0)
    o, _ = _run(c)
    _check(c, o)


ONE = pytest.mark.parametrize("E,k", [(7, 7), (77, 9), (128, 32), (129, 17), (200, 32), (256, 8), (257, 32), (1000, 32), (1024, 20)])


def _sorted_choice(z, k):
    """Stable, -0 and +0 equal, NaN behind everything beside -inf."""
    z = torch.where(torch.isnan(z), torch.full_like(z, -float("inf")), z) + 0.0
    return torch.sort(z, dim=-1, descending=True, stable=True).indices[..., :k].int()


@ONE
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_one_token_choice_is_exact_on_ties(E, k, seed):
    """Whole-number logits with many ties (sums of 64 products of -1, 0 and 1 are exact in any order), -0 among the biases."""
    gen = torch.Generator(device="cuda").manual_seed(1000 * seed + E)
    c = _case(1, 64, 32, E, k, "bf16", seed=seed)
    c["x"] = torch.randint(-1, 2, (1, 64), generator=gen, device="cuda").to(BF)
    c["wr"] = torch.randint(-1, 2, (64, E), generator=gen, device="cuda").float()
    c["b"] = torch.where(torch.rand(E, generator=gen, device="cuda") < 0.5, -0.0, 0.0)
    o, _ = _run(c)
    assert torch.equal(o["topk_idx"].cpu(), _sorted_choice(c["x"].float().cpu() @ c["wr"].cpu(), k))
    _check(c, o)
    c["wr"][:] = 0.0  # one tie of all
    o, _ = _run(c)
    assert o["topk_idx"][0].tolist() == list(range(k))
    assert bool(((o["topk_w"] - 1 / k).abs() <= 40 * U / k).all())


@ONE
def test_one_token_experts_left_out(E, k):
    """As for several tokens: -inf (and NaN) leave an expert out, too few others leave the rest without weight."""
    gen = torch.Generator(device="cuda").manual_seed(E)
    c = _case(1, 64, 32, E, k, "bf16", seed=13)
    c["x"] = torch.randint(-1, 2, (1, 64), generator=gen, device="cuda").to(BF)
    c["wr"] = torch.randint(-1, 2, (64, E), generator=gen, device="cuda").float()
    z = c["x"].float().cpu() @ c["wr"].cpu()
    for share in (0.3, 0.9, 1.0):
        out = torch.rand(E, generator=gen, device="cuda") < share
        c["b"] = torch.where(out, -float("inf"), 0.0)
        c["b"][out & (torch.rand(E, generator=gen, device="cuda") < 0.2)] = float("nan")
        o, _ = _run(c)
        zb = z + c["b"].cpu()
        zb = torch.where(torch.isnan(zb), torch.full_like(zb, -float("inf")), zb)
        idx = _sorted_choice(zb, k)
        assert torch.equal(o["topk_idx"].cpu(), idx)
        zi = zb.gather(1, idx.long()).double()
        w = torch.softmax(zi, dim=1) if bool((zi > -float("inf")).any()) else torch.zeros_like(zi)
        # (exponentials of whole numbers, k of them added, one division)
        assert bool(((o["topk_w"].cpu().double() - w).abs() <= 32 * U * w).all())
        if not bool((w > 0).any()):
            assert bool((o["out"] == 0).all())


@KINDS
@pytest.mark.parametrize("E", [12, 200, 300])
def test_one_spoilt_token(E, kind):
    for value in (float("nan"), float("inf")):
        c = _case(1, 96, 64, E, 3, kind, seed=17)
        c["x"][0, 7] = value
        o, _ = _run(c)
        idx = o["topk_idx"][0].tolist()
        assert len(set(idx)) == 3 and all(0 <= e < E for e in idx)
        assert bool(torch.isnan(o["out"]).all())


@KINDS
@pytest.mark.parametrize("E", [200, 300])
def test_one_token_streams_graph_and_repeats(E, kind):
    import grouped_gemm_top_amd as G
    c = _case(1, 128, 96, E, 4, kind, seed=23, bias=True)
    o, a = _run(c)
    st = [torch.cuda.Stream() for _ in range(2)]
    for s in st:
        s.wait_stream(torch.cuda.current_stream())
    call = lambda x, **kw: G.layer_few(x, a["wr"], a["wg"], a["wu"], a["wd"], 4, bias=a["b"], **kw)  # noqa: E731
    for _ in range(10):
        r, q = call(a["x"], stream=st[0]), call(a["x"], stream=st[1])
    torch.cuda.synchronize()
    assert all(torch.equal(r[n], o[n]) and torch.equal(q[n], o[n]) for n in o)
    x = a["x"].clone()
    with torch.cuda.stream(st[0]):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st[0]):
            r = call(x)
    for i in range(5):
        x.copy_(torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(40 + i), device="cuda"))
        e = call(x)
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(e[n], r[n]) for n in e), i
