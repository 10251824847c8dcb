"""The newer operators in a row, as a model with routed experts uses them.

Training: norm (its codes kept as the layer's x) -> router -> top-k and plan -> experts, [G | U] kept in 8 bits
-> combine -> cross entropy over the vocabulary, and back through all of it, in bf16, against 64 bits.  The codes'
rounding stands in for the activations in the backward: e4m3 is off by at most 2^-4 of a value, 2^-4 / sqrt 3 = 0.036 in
the 2-norm, for each of x, G and U; dG and dU hold all three factors' errors, so weight gradients and dx may
be off by sqrt 3 0.036 = 0.063, and by the bf16 roundings beside it (0.01 in all).  What does not pass through codes
(loss, lse, the gradient of the projection) is held to its own roundings.

Serving: a token's output from the whole-layer call equals the prefill's (route, permute, grouped GEMMs, combine) to
the roundings of both."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import grouped_gemm_top_amd as G
    G.lib()


def _params(H, I, E, V, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, dt=BF, sc=None: ((s[-1] ** -0.5 if sc is None else sc) * torch.randn(  # noqa: E731
        s, generator=gen, device="cuda")).to(dt)
    return dict(wr=rnd(H, E, dt=F32, sc=1.5 * H ** -0.5), b=rnd(E, dt=F32, sc=0.3), wg=rnd(E, I, H), wu=rnd(E, I, H),
                wd=rnd(E, H, I), wn=1 + rnd(H, dt=F32, sc=0.1), wv=rnd(V, H, sc=2.0 * H ** -0.5)), rnd


def _step(G, p, res, t, g, k, zc):
    """One forward and backward; everything that comes back."""
    n = G.add_rmsnorm(res, p["wn"], want_h=False, quantize=True)
    x, xq = n["y"], (n["q"], n["scales"])
    logits = G.router_logits(x, p["wr"])
    idx, w, _ = G.route_topk(logits, k, bias=p["b"])
    plan = G.permute(idx, w, p["wg"].shape[0])
    h, y = G.grouped_gemm_fwd_ckpt8(x, p["wg"], p["wu"], p["wd"], plan)
    out = G.unpermute_combine(y, plan)
    f = G.linear_ce_fwd(out, p["wv"], t, z_coef=zc)
    c = G.linear_ce_bwd(g, out, p["wv"], t, f["lse"], z_coef=zc)
    b = G.layer_bwd_ckpt8(c["dx"], xq, p["wg"], p["wu"], p["wd"], plan, h)
    return dict(loss=f["loss"], lse=f["lse"], dwv=c["dw"], out=out, idx=idx, w=w,
                **{n: b[n] for n in ("dx", "dw_gate", "dw_up", "dw_down", "ds")})


@pytest.mark.parametrize("N,H,I,E,k,V", [(300, 256, 96, 12, 3, 1003), (64, 96, 160, 4, 2, 77)])
def test_training_step(N, H, I, E, k, V):
    import grouped_gemm_top_amd as G
    p, rnd = _params(H, I, E, V, 1)
    res = rnd(N, H, sc=2.0)
    gen = torch.Generator(device="cuda").manual_seed(2)
    t = torch.randint(0, V, (N,), generator=gen, device="cuda").int()
    t[::7] = -100
    g = torch.full((N,), 1.0 / N, device="cuda")
    zc = 1e-3
    o = _step(G, p, res, t, g, k, zc)
    # the same in 64 bits, at the GPU's choice of experts; the norm's stored y is the layer's input on both sides
    x = G.add_rmsnorm(res, p["wn"], want_h=False)["y"].double().requires_grad_(True)
    P = {n: v.double().requires_grad_(n[0] == "w") for n, v in p.items()}
    idx, w = o["idx"].long(), o["w"].double().requires_grad_(True)
    out = torch.zeros(N, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        r, j = torch.nonzero(idx == e, as_tuple=True)
        a = torch.nn.functional.silu(x[r] @ P["wg"][e].t()) * (x[r] @ P["wu"][e].t())
        out = out.index_add(0, r, w[r, j][:, None] * (a @ P["wd"][e].t()))
    live = t >= 0
    z = out[live] @ P["wv"].t()
    lse = torch.logsumexp(z, dim=1)
    each = lse - z.gather(1, t[live].long()[:, None])[:, 0] + zc * lse ** 2
    grads = torch.autograd.grad((each * g[live]).sum(), (x, w, P["wg"], P["wu"], P["wd"], P["wv"]))
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    # out passes three roundings (a, the expert rows, itself) into the logits: 0.0039 of their spread
    assert rel(o["loss"][live], each.detach()) <= 5e-3 and bool((o["loss"][~live] == 0).all())
    assert rel(o["out"], out.detach()) <= 5e-3
    assert rel(o["dwv"], grads[5]) <= 0.02
    for n, ref in zip(("dx", "ds", "dw_gate", "dw_up", "dw_down"), grads):
        assert rel(o[n], ref) <= 0.08, (n, rel(o[n], ref))
    assert bool((o["dx"][~live] == 0).all())
    # twice the same, bit for bit
    q = _step(G, p, res, t, g, k, zc)
    assert all(torch.equal(o[n], q[n]) for n in o)


def test_training_step_captured():
    """The step in a graph, replayed on new inputs between eager steps."""
    import grouped_gemm_top_amd as G
    N, H, I, E, k, V = 200, 128, 64, 8, 2, 501
    p, rnd = _params(H, I, E, V, 5)
    res, t, g = rnd(N, H, sc=2.0), torch.zeros(N, dtype=torch.int32, device="cuda"), torch.full((N,), 1.0 / N, device="cuda")
    _step(G, p, res, t, g, k, 0.0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            r = _step(G, p, res, t, g, k, 0.0)
    for i in range(4):
        gen = torch.Generator(device="cuda").manual_seed(20 + i)
        res.copy_(2 * torch.randn(N, H, generator=gen, device="cuda"))
        t.copy_(torch.randint(-20, V, (N,), generator=gen, device="cuda"))
        e = _step(G, p, res, t, g, k, 0.0)
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(e[n], r[n]) for n in e), i


@pytest.mark.parametrize("N,H,I,E,k", [(1, 256, 128, 16, 4), (48, 512, 160, 24, 3)])
@pytest.mark.parametrize("kind", ["bf16", "mxfp8"])
def test_prefill_and_decode_agree(N, H, I, E, k, kind):
    import grouped_gemm_top_amd as G
    p, rnd = _params(H, I, E, 8, 9)
    x = rnd(N, H, sc=1.0)
    w3 = [p[n] for n in ("wg", "wu", "wd")]
    q3 = [G.quantize_mxfp8(w) for w in w3]
    if kind == "mxfp8":  # prefill on the values that the codes stand for
        w3 = [G.dequantize_mxfp8(*q) for q in q3]
    logits = G.router_logits(x, p["wr"])
    idx, w, _ = G.route_topk(logits, k, bias=p["b"])
    plan = G.permute(idx, w, E)
    _, y = G.grouped_gemm_fwd(x, *w3, plan)
    out = G.unpermute_combine(y, plan)
    r = G.layer_few(x, p["wr"], *(q3 if kind == "mxfp8" else w3), k, bias=p["b"])
    assert torch.equal(r["topk_idx"], idx) and float((r["topk_w"] - w).abs().max()) <= 1e-5
    # each side rounds twice or three times: 2^-8 / sqrt 3 each, sqrt 5 of it together
    assert float((r["out"].double() - out.double()).norm()) <= 6e-3 * float(out.double().norm())
