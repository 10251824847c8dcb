"""The operators in a row, as an MoE transformer block uses them: projection with residual, add + RMS
norm (with the MX-FP8 codes), router, top-k, plan, balance loss, expert MLP, combine; and back.

The reference is one fp64 autograd graph of the whole block on the CPU from the same bf16 inputs,
with the GPU's expert selection (a decision, not a value).  The chain stores about a dozen tensors in
bf16 between input and gradient; each rounding is off by at most 2^-8 relative per element, spread
evenly about 2^-8 / sqrt(3) in the 2-norm, independent from tensor to tensor: sqrt(12) of them make
0.8 %, and the norm's and the gates' slopes pass errors on with a factor of about one.  Asked for: 3 %
in the 2-norm of every output and gradient (MX-FP8: codes carry 3 bits, 2^-4 / sqrt(3) = 3.6 % an
operand, two operands twice over: 10 %)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
N, A, H, I, E, K = 600, 192, 256, 128, 16, 4
ALPHA, BETA, EPS = 0.05, 0.01, 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import grouped_gemm_top_amd as G
    G.lib()


def _inputs(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: std * torch.randn(*s, generator=g)  # noqa: E731
    t = dict(a=r(N, A).to(BF), wo=r(H, A, std=A ** -0.5).to(BF), bo=r(H, std=0.1), res=r(N, H).to(BF),
             wn=1 + r(H, std=0.1), wr=r(H, E, std=H ** -0.5), br=r(E, std=0.2),
             wg=r(E, I, H, std=H ** -0.5).to(BF), wu=r(E, I, H, std=H ** -0.5).to(BF),
             wd=r(E, H, I, std=I ** -0.5).to(BF), dout=r(N, H).to(BF))
    t["mask"] = (torch.rand(N, generator=g) < 0.9).to(torch.uint8)
    t["ptr"] = torch.tensor([0, 150, 150, 420, 590], dtype=torch.int32)
    return t


def _forward(G, D):
    """The block's forward on the GPU; everything its backward needs."""
    s = {}
    s["p"], _ = G.linear_fwd(D["a"], D["wo"], bias=D["bo"], residual=D["res"])
    n = G.add_rmsnorm(s["p"], D["wn"], eps=EPS, quantize=True)
    s["h"], s["x"], s["xq"] = n["h"], n["y"], (n["q"], n["scales"])
    s["logits"] = G.router_logits(s["x"], D["wr"])
    s["idx"], w, _ = G.route_topk(s["logits"], K, bias=D["br"])
    s["plan"] = G.permute(s["idx"], w, E)
    s["bal"] = G.balance_loss(s["logits"], s["idx"], ALPHA, BETA, bias=D["br"], mask=D["mask"], seq_ptr=D["ptr"])
    s["hc"], y = G.grouped_gemm_fwd(s["x"], D["wg"], D["wu"], D["wd"], s["plan"])
    s["out"] = G.unpermute_combine(y, s["plan"])
    return s


def _backward(G, D, s):
    b = G.layer_bwd(D["dout"], s["x"], D["wg"], D["wu"], D["wd"], s["plan"], s["hc"])
    aux = G.balance_loss_bwd(s["logits"], s["bal"]["saved"], bias=D["br"], mask=D["mask"], seq_ptr=D["ptr"])
    r = G.router_bwd(s["logits"], s["idx"], s["plan"], b["ds"], s["x"], D["wr"], bias=D["br"], dx_in=b["dx"],
                     dlogits_in=aux)
    # the block's output is added to the stream: dout reaches h itself
    n = G.add_rmsnorm_bwd(r["dx"], s["h"], D["wn"], dh_in=D["dout"], eps=EPS)
    p = G.linear_bwd(n["dh"], D["a"], D["wo"])
    return dict(wg=b["dw_gate"], wu=b["dw_up"], wd=b["dw_down"], wr=r["dw_r"], br=r["dbias"], wn=n["dw"],
                res=n["dh"], a=p["dx"], wo=p["dw"], bo=p["dbias"])


def _reference(t, idx):
    """Output, balance losses and gradients of sum(dout * (h + experts)) + losses, in fp64."""
    v = {n: x.double().requires_grad_(n not in ("dout",)) for n, x in t.items() if x.is_floating_point()}
    h = v["a"] @ v["wo"].t() + v["bo"] + v["res"]
    x = h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * v["wn"]
    z = x @ v["wr"] + v["br"]
    sel = z.gather(1, idx.long())
    w = torch.softmax(sel, 1)
    out = torch.zeros_like(h)
    for e in range(E):
        tok, slot = torch.nonzero(idx == e, as_tuple=True)
        if tok.numel():
            xe = x[tok]
            ye = (torch.nn.functional.silu(xe @ v["wg"][e].t()) * (xe @ v["wu"][e].t())) @ v["wd"][e].t()
            out = out.index_add(0, tok, ye * w[tok, slot][:, None])
    p, lse = torch.softmax(z, 1), torch.logsumexp(z, 1)
    ptr, l0, live = t["ptr"].tolist(), 0.0, []
    B = len(ptr) - 1
    for b in range(B):
        ts = [i for i in range(ptr[b], ptr[b + 1]) if t["mask"][i]]
        live += ts
        if ts:
            c = torch.bincount(idx[ts].reshape(-1), minlength=E).double()
            l0 = l0 + ALPHA / B * E / (K * len(ts) ** 2) * (c * p[ts].sum(0)).sum()
    l1 = BETA * lse[live].square().mean()
    loss = (v["dout"] * (h + out)).sum() + l0 + l1
    names = [n for n in v if n != "dout"]
    grads = dict(zip(names, torch.autograd.grad(loss, [v[n] for n in names])))
    return out.detach(), (float(l0.detach()), float(l1.detach())), grads, x.detach()


def _rel(got, ref):
    return float((got.double().cpu() - ref).norm() / ref.norm())


def test_block_forward_and_backward():
    import grouped_gemm_top_amd as G
    t = _inputs(1)
    D = {n: x.cuda() for n, x in t.items()}
    s = _forward(G, D)
    g = _backward(G, D, s)
    torch.cuda.synchronize()
    out, losses, grads, x = _reference(t, s["idx"].cpu())
    assert _rel(s["out"], out) <= 0.03
    for i in range(2):
        assert abs(float(s["bal"]["loss"][i]) - losses[i]) <= 0.03 * losses[i]
    errs = {n: _rel(g[n], grads[n]) for n in g}
    bad = {n: e for n, e in errs.items() if not e <= 0.03}
    assert not bad, bad


def test_balance_loss_moves_the_router_gradient():
    """Without the balance loss's gradient the router's is another one: the path carries it."""
    import grouped_gemm_top_amd as G
    t = _inputs(2)
    D = {n: x.cuda() for n, x in t.items()}
    s = _forward(G, D)
    b = G.layer_bwd(D["dout"], s["x"], D["wg"], D["wu"], D["wd"], s["plan"], s["hc"])
    aux = G.balance_loss_bwd(s["logits"], s["bal"]["saved"], bias=D["br"], mask=D["mask"], seq_ptr=D["ptr"],
                             dloss=torch.tensor([1e4, 0.0], device="cuda"))
    args = (s["logits"], s["idx"], s["plan"], b["ds"], s["x"], D["wr"])
    with_, without = (G.router_bwd(*args, bias=D["br"], dlogits_in=v, want_dx=False) for v in (aux, None))
    torch.cuda.synchronize()
    want = s["x"].double().t() @ aux.double()
    got = with_["dw_r"].double() - without["dw_r"].double()
    assert float((got - want).norm() / want.norm()) <= 1e-4


def test_quantized_forward_from_the_norm():
    """The norm's own codes drive the MX-FP8 layer: the output of the bf16 path within the codes' precision,
    and nearly that of codes made from the stored y (they differ where two roundings differ)."""
    import grouped_gemm_top_amd as G
    t = _inputs(3)
    D = {n: x.cuda() for n, x in t.items()}
    s = _forward(G, D)
    w = [G.quantize_mxfp8(D[n]) for n in ("wg", "wu", "wd")]
    _, y = G.grouped_gemm_fwd_mxfp8(s["xq"], *w, s["plan"])
    out = G.unpermute_combine(y, s["plan"])
    _, y2 = G.grouped_gemm_fwd_mxfp8(G.quantize_mxfp8(s["x"]), *w, s["plan"])
    out2 = G.unpermute_combine(y2, s["plan"])
    torch.cuda.synchronize()
    ref, _, _, _ = _reference(t, s["idx"].cpu())
    assert _rel(out, ref) <= 0.10 and _rel(out2, ref) <= 0.10


def test_block_in_a_graph():
    """Forward and backward captured once; every replay on new inputs gives the eager result, with eager
    work in between (the permute and the products are the library's own launches too)."""
    import grouped_gemm_top_amd as G
    D = {n: x.cuda() for n, x in _inputs(4).items()}

    def block():
        s = _forward(G, D)
        return dict(_backward(G, D, s), out=s["out"], loss=s["bal"]["loss"], counts=s["bal"]["counts"])

    block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block()
    for seed in range(5, 9):
        for n, x in _inputs(seed).items():
            D[n].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        eager = block()
        torch.cuda.synchronize()
        for n in eager:
            assert torch.equal(eager[n].view(torch.uint8) if eager[n].dtype == BF else eager[n],
                               got[n].view(torch.uint8) if got[n].dtype == BF else got[n]), (seed, n)


def test_stream_handles():
    """`stream` may be any object with a cuda_stream handle, as the layer's own calls take it, a torch external
    stream among them; the results are those of the current stream."""
    import grouped_gemm_top_amd as G
    t = _inputs(4)
    D = {n: x.cuda() for n, x in t.items()}
    lg = torch.randn(N, E, device="cuda")
    idx = lg.topk(K, dim=1).indices.int()

    def calls(**kw):
        n = G.add_rmsnorm(D["res"], D["wn"], quantize=True, **kw)
        b = G.add_rmsnorm_bwd(D["dout"], D["res"], D["wn"], **kw)
        r = G.balance_loss(lg, idx, ALPHA, BETA, **kw)
        p, z = G.linear_fwd(D["a"], D["wo"], bias=D["bo"], act="silu", want_z=True, **kw)
        q = G.linear_bwd(D["dout"], D["a"], D["wo"], z=z, act="silu", **kw)
        return [n["y"], n["q"].float(), b["dh"], b["dw"], r["loss"], G.balance_loss_bwd(lg, r["saved"], **kw), p, q["dx"],
                q["dw"], q["dbias"]]

    want = calls()
    side = torch.cuda.Stream()

    class Handle:
        cuda_stream = side.cuda_stream

    class Default:
        cuda_stream = torch.cuda.default_stream().cuda_stream

    for stream in (side, Handle, Handle(), torch.cuda.ExternalStream(side.cuda_stream), Default()):
        torch.cuda.synchronize()
        got = calls(stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), stream


def test_codes_of_the_norm_and_of_the_stored_output_drive_nearly_the_same_layer():
    """The norm's codes round the fp32 y, quantize_mxfp8(x) the stored bf16 y, which is off by up to 2^-8 of it
    (2^-9.5 in the mean).  A code's step is 2^-3.5 of its value in the mean, so about one code in 64 falls
    on the other side of a border, a step away: 2^-3.5 sqrt(1 / 64) = 1 % in the 2-norm.  The gate's slope
    and the up factor make 2 % of it; the activations are then quantized again, where 2 % move one code
    in five by a step: 2^-3.5 sqrt(1 / 5) = 4 %, which the down product keeps.  Asked for: 6 %."""
    import grouped_gemm_top_amd as G
    t = _inputs(3)
    D = {n: x.cuda() for n, x in t.items()}
    s = _forward(G, D)
    w = [G.quantize_mxfp8(D[n]) for n in ("wg", "wu", "wd")]
    out, out2 = (G.unpermute_combine(G.grouped_gemm_fwd_mxfp8(q, *w, s["plan"])[1], s["plan"])
                 for q in (s["xq"], G.quantize_mxfp8(s["x"])))
    torch.cuda.synchronize()
    assert _rel(out, out2.double().cpu()) <= 0.06
