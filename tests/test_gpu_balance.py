"""moe_balance_loss, moe_balance_loss_bwd and moe_router_bwd_acc against fp64 references, through the
C ABI, every buffer guarded.

Counts are equal.  Tolerances of the rest, from the arithmetic (u = 2^-24, zm the largest |z|):
* p: z = logits + bias is off by u zm, which e^z takes as a relative error, numerator and sum; so is
  x = z - max (at most 2 zm in size) with u |x|, rounded itself and in its product with log2 e; the
  exponential, at most 16 + 6 additions, the reciprocal and the product add less than 40 u:
  (4 zm + 40) u relative;
* loss[0], a sum of positive terms: p's error, then at most 128 additions in a row (tokens of one
  slot, lane exchanges, slots, experts): (4 zm + 168) u relative, below (2 zm + 256) u for zm <= 44;
* lse = max + log(sum): (zm + 40) u absolute; loss[1] takes it times 2 |lse|, and 256 u for its sum;
* saved: three divisions and a product from a rounded constant: 8 u relative;
* dlogits: the two errors above on each of its terms p g, p sum(g p) and p lse, at most 64 u for the
  dot product, and one rounding of the addition."""
import numpy as np
import pytest
import torch

from harness import Guards

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ALPHA, BETA = 0.02, 0.003


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import grouped_gemm_top_amd as G
    G.lib()


def _ref(lg, bias, idx, mask, ptr, alpha=ALPHA, beta=BETA, d=(1.0, 1.0)):
    """fp64: loss, counts, saved, dlogits and the size of dlogits' terms, one sequence at a time."""
    N, E = lg.shape
    k = idx.shape[1]
    ptr = [0, N] if ptr is None else ptr.tolist()
    B = len(ptr) - 1
    z = lg.double() + (bias.double() if bias is not None else 0)
    toks = [[t for t in range(ptr[b], ptr[b + 1]) if mask is None or mask[t]] for b in range(B)]
    n = sum(len(t) for t in toks)
    counts = torch.zeros(B, E, dtype=torch.int32)
    saved = torch.zeros(B * E + 1, dtype=torch.float64)
    saved[-1] = 2 * beta / n if n else 0.0
    dz, size = torch.zeros(N, E, dtype=torch.float64), torch.zeros(N, E, dtype=torch.float64)
    l0 = l1 = l1size = 0.0
    zm = 0.0
    for b, ts in enumerate(toks):
        if not ts:
            continue
        for t in ts:
            for e in set(idx[t].tolist()):
                if 0 <= e < E:
                    counts[b, e] += 1
        zz = z[ts]
        top = zz.amax(1, keepdim=True)
        dead = top == -np.inf
        ez = torch.where(dead, 0.0, torch.exp(zz - torch.where(dead, 0.0, top)))
        s = ez.sum(1, keepdim=True)
        p = torch.where(dead, 0.0, ez / torch.where(dead, 1.0, s))
        lse = torch.where(dead, 0.0, top + torch.log(torch.where(dead, 1.0, s)))
        g = alpha * E * counts[b].double() / (B * k * len(ts) ** 2)
        saved[b * E:(b + 1) * E] = g
        l0 += float((g * p.sum(0)).sum())
        l1 += float(beta / n * lse.square().sum())
        fin = zz[torch.isfinite(zz)].abs()
        zm = max(zm, float(fin.max()) if fin.numel() else 0.0)
        l1size += float(beta / n * 2 * lse.abs().sum())
        dot = (g * p).sum(1, keepdim=True)
        dz[ts] = p * (d[0] * (g - dot) + d[1] * 2 * beta / n * lse)
        size[ts] = p * (abs(d[0]) * (g + dot) + abs(d[1]) * 2 * beta / n * (lse.abs() + 1))
    return dict(loss=(l0, l1), l1size=l1size, counts=counts, saved=saved, dz=dz, size=size, zm=zm)


def _check(r, dl, ref, din=None):
    zm = ref["zm"]
    assert torch.equal(r["counts"].cpu(), ref["counts"])
    l0, l1 = (float(v) for v in r["loss"].cpu().double())
    assert abs(l0 - ref["loss"][0]) <= (2 * zm + 256) * U * ref["loss"][0], (l0, ref["loss"][0])
    assert abs(l1 - ref["loss"][1]) <= 256 * U * ref["loss"][1] + (zm + 40) * U * ref["l1size"], (l1, ref["loss"][1])
    assert bool(((r["saved"].cpu().double() - ref["saved"]).abs() <= 8 * U * ref["saved"]).all())
    want = ref["dz"] + (din.double() if din is not None else 0)
    tol = (4 * zm + 200) * U * ref["size"] + U * want.abs() + 2.0 ** -126
    err = (dl.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def _inputs(N, E, k, B, mask, bias, seed, ragged=True):
    gen = torch.Generator().manual_seed(seed)
    lg = 2.0 * torch.randn(N, E, generator=gen)
    bs = torch.randn(E, generator=gen) if bias else None
    z = lg if bs is None else lg + bs
    idx = z.topk(k, dim=1).indices.int()
    mk = (torch.rand(N, generator=gen) < 0.8).to(torch.uint8) if mask else None
    ptr = None
    if B > 1:
        ptr = torch.randint(0, N + 1, (B + 1,), generator=gen).sort().values.int()
    return lg, bs, idx, mk, ptr


CASES = [  # N, E, k, B, mask, bias
    (1, 1, 1, 1, False, False), (1, 8, 2, 1, False, True), (64, 8, 2, 1, False, False), (64, 8, 2, 3, True, True),
    (3, 5, 5, 2, False, False), (37, 12, 3, 4, True, False), (200, 16, 1, 1, False, False), (130, 32, 4, 7, True, True),
    (300, 33, 6, 5, False, True), (257, 64, 8, 1, True, False), (1000, 100, 8, 9, True, True),
    (1025, 128, 8, 4, False, False), (777, 160, 7, 30, True, False), (513, 256, 8, 2, False, True),
    (300, 255, 8, 3, True, True), (129, 512, 10, 3, False, False), (65, 511, 65, 2, True, False),
    (70, 1024, 128, 2, True, True), (33, 1023, 8, 1, False, True), (90, 128, 100, 40, False, False),
    (20000, 16, 2, 11, True, True), (40000, 4, 1, 300, True, False),
]


@pytest.mark.parametrize("N,E,k,B,mask,bias", CASES)
def test_against_fp64(N, E, k, B, mask, bias):
    import grouped_gemm_top_amd as G
    lg, bs, idx, mk, ptr = _inputs(N, E, k, B, mask, bias, seed=N + E)
    hostile = lg.clone()
    if mk is not None:  # what a token left out holds must not matter
        hostile[mk == 0] = float("nan")
        if int((mk == 0).sum()) > 2:
            hostile[torch.nonzero(mk == 0)[0]] = float("inf")
            hostile[torch.nonzero(mk == 0)[1]] = torch.finfo(torch.float32).min
    g = Guards()
    up = lambda n, t: None if t is None else g.upload(n, t.numpy())  # noqa: E731
    D = dict(lg=up("lg", hostile), bias=up("bias", bs), idx=up("idx", idx), mask=up("mask", mk), ptr=up("ptr", ptr))
    loss, counts = g.alloc("loss", (2,), torch.float32), g.alloc("counts", (B, E), torch.int32)
    saved, dl = g.alloc("saved", (B * E + 1,), torch.float32), g.alloc("dl", (N, E), torch.float32)
    ws = g.alloc("ws", (G.workspace_bytes(G.OP_BALANCE_LOSS, G.MOE_F32, N, E, k, 0, B),), torch.uint8)
    kw = dict(bias=D["bias"], mask=D["mask"], seq_ptr=D["ptr"])
    r = G.balance_loss(D["lg"], D["idx"], ALPHA, BETA, loss=loss, counts=counts, saved=saved, ws=ws, **kw)
    g.check("balance_loss")
    G.balance_loss_bwd(D["lg"], saved, dlogits=dl, **kw)
    g.check("balance_loss_bwd")
    ref = _ref(lg, bs, idx, mk, ptr)
    _check(r, dl, ref)
    # two runs are bitwise equal; upstream gradients and a gradient to add, in place
    r2 = G.balance_loss(D["lg"], D["idx"], ALPHA, BETA, **kw)
    torch.cuda.synchronize()
    assert torch.equal(r2["loss"], loss) and torch.equal(r2["saved"], saved) and torch.equal(r2["counts"], counts)
    din = torch.randn(N, E, generator=torch.Generator().manual_seed(5)) * 1e-3
    mine, up2 = din.cuda(), torch.tensor([-0.7, 3.0], device="cuda")
    out = G.balance_loss_bwd(D["lg"], saved, dloss=up2, dlogits_in=mine, dlogits=mine, **kw)
    assert out.data_ptr() == mine.data_ptr()
    _check(r, out, _ref(lg, bs, idx, mk, ptr, d=(-0.7, 3.0)), din)


def test_unaligned_logits():
    """Logits at an address that is no multiple of 16 take the scalar path and the same tolerance."""
    import grouped_gemm_top_amd as G
    N, E, k = 300, 64, 4
    lg, _, idx, _, _ = _inputs(N, E, k, 1, False, False, seed=3)
    buf = torch.empty(N * E + 1, device="cuda")
    view = buf[1:].view(N, E)
    view.copy_(lg)
    r = G.balance_loss(view, idx.cuda(), ALPHA, BETA)
    out = torch.empty(N * E + 3, device="cuda")[3:].view(N, E)
    _check(r, G.balance_loss_bwd(view, r["saved"], dlogits=out), _ref(lg, None, idx, None, None))


def test_indices_that_make_no_pair():
    """Out-of-range indices and repeated experts count as moe_permute counts them."""
    import grouped_gemm_top_amd as G
    N, E, k = 50, 12, 4
    lg, _, idx, _, _ = _inputs(N, E, k, 1, False, False, seed=4)
    idx[0] = torch.tensor([3, 3, 3, 3])
    idx[1] = torch.tensor([-1, 12, 5, 1 << 30])
    idx[2] = torch.tensor([7, -5, 7, 0])
    r = G.balance_loss(lg.cuda(), idx.cuda(), ALPHA, BETA)
    _check(r, G.balance_loss_bwd(lg.cuda(), r["saved"]), _ref(lg, None, idx, None, None))
    plan = G.permute(idx.cuda(), torch.ones(N, k, device="cuda"), E)
    torch.cuda.synchronize()
    assert torch.equal(plan.counts, r["counts"][0])


def test_everything_masked_and_no_tokens():
    import grouped_gemm_top_amd as G
    N, E, k = 40, 24, 2
    lg, _, idx, _, _ = _inputs(N, E, k, 1, False, False, seed=6)
    lg[:] = float("nan")
    zero = torch.zeros(N, dtype=torch.bool, device="cuda")
    for ptr in (None, torch.tensor([0, 0, 20, 20, 40, 40], dtype=torch.int32, device="cuda"),
                torch.tensor([40, 40], dtype=torch.int32, device="cuda")):
        r = G.balance_loss(lg.cuda(), idx.cuda(), ALPHA, BETA, mask=zero, seq_ptr=ptr)
        d = G.balance_loss_bwd(lg.cuda(), r["saved"], mask=zero, seq_ptr=ptr)
        torch.cuda.synchronize()
        assert all(float(r[n].abs().max()) == 0.0 for n in ("loss", "counts", "saved")) and float(d.abs().max()) == 0.0
    e = torch.empty((0, E), device="cuda")
    r = G.balance_loss(e, torch.empty((0, k), dtype=torch.int32, device="cuda"), ALPHA, BETA,
                       loss=torch.full((2,), 7.0, device="cuda"), counts=torch.full((1, E), 7, dtype=torch.int32, device="cuda"))
    d = G.balance_loss_bwd(e, r["saved"])
    torch.cuda.synchronize()
    assert d.shape == (0, E) and all(float(r[n].abs().max()) == 0.0 for n in ("loss", "counts", "saved"))


def test_experts_switched_off():
    """-inf logits and biases, and rows at the type's lowest value: no NaN anywhere."""
    import grouped_gemm_top_amd as G
    N, E, k = 65, 40, 2
    lg, bs, idx, _, _ = _inputs(N, E, k, 1, False, True, seed=7)
    bs[3] = float("-inf")
    bs[39] = torch.finfo(torch.float32).min
    lg[5] = float("-inf")
    lg[6, 1:] = torch.finfo(torch.float32).min
    idx = (lg + bs).topk(k, dim=1).indices.int()
    r = G.balance_loss(lg.cuda(), idx.cuda(), ALPHA, BETA, bias=bs.cuda())
    d = G.balance_loss_bwd(lg.cuda(), r["saved"], bias=bs.cuda())
    torch.cuda.synchronize()
    assert bool(d.isfinite().all()) and bool(r["loss"].isfinite().all())
    ref = _ref(lg, bs, idx, None, None)
    assert bool((d[:, 3] == 0).all()) and bool((d[5] == 0).all())
    zm = 12.0  # the largest |z| of an expert that is on
    tol = (4 * zm + 200) * U * ref["size"] + 2.0 ** -126
    assert bool(((d.cpu().double() - ref["dz"]).abs() <= tol).all())


def test_gradient_against_differences():
    """The GPU's gradient against central differences of the fp64 loss with the counts held fixed.
    Steps of 2^-10 leave a third-order error below 2^-20 of the first derivative's size times a
    small constant."""
    import grouped_gemm_top_amd as G
    N, E, k = 9, 6, 2
    lg, bs, idx, mk, _ = _inputs(N, E, k, 1, True, True, seed=8)
    ptr = torch.tensor([1, 4, 4, 8], dtype=torch.int32)
    kw = dict(bias=bs.cuda(), mask=mk.cuda(), seq_ptr=ptr.cuda())
    r = G.balance_loss(lg.cuda(), idx.cuda(), ALPHA, BETA, **kw)
    d = G.balance_loss_bwd(lg.cuda(), r["saved"], **kw).cpu().double()
    f = lambda v: sum(_ref(v, bs, idx, mk, ptr)["loss"])  # noqa: E731
    st = 2.0 ** -10
    for seed in range(4):
        e = torch.randn(N, E, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
        num = (f(lg.double() + st * e) - f(lg.double() - st * e)) / (2 * st)
        assert abs(float((d * e).sum()) - num) <= 1e-4 * float((d * e).norm())


def test_graph_and_stream():
    import grouped_gemm_top_amd as G
    N, E, k, B = 3000, 128, 8, 5
    lg, bs, idx, mk, ptr = _inputs(N, E, k, B, True, True, seed=9)
    lg, idx = lg.cuda(), idx.cuda()
    kw = dict(bias=bs.cuda(), mask=mk.cuda(), seq_ptr=ptr.cuda())

    def both(**s):
        r = G.balance_loss(lg, idx, ALPHA, BETA, **kw, **s)
        return dict(r, d=G.balance_loss_bwd(lg, r["saved"], **kw, **s))

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
    for seed in range(4):
        lg.copy_(torch.randn(N, E, generator=torch.Generator().manual_seed(50 + seed)))
        graph.replay()
        graph2.replay()
        torch.cuda.synchronize()
        eager = both()
        torch.cuda.synchronize()
        assert all(torch.equal(eager[n], got[n]) and torch.equal(eager[n], got2[n]) for n in eager)


def test_router_backward_takes_the_gradient():
    """moe_router_bwd_acc: dlogits is the sum, and dx, dW_r and dbias are the products of that sum;
    without a further gradient it is moe_router_bwd, bit for bit."""
    import grouped_gemm_top_amd as G
    N, H, E, k = 300, 320, 12, 3
    gen = torch.Generator().manual_seed(10)
    x, wr = torch.randn(N, H, generator=gen).cuda(), (0.05 * torch.randn(H, E, generator=gen)).cuda()
    bias, ds = torch.randn(E, generator=gen).cuda(), torch.randn(N, k, generator=gen).cuda()
    lg = G.router_logits(x, wr)
    idx, w, _ = G.route_topk(lg, k, bias=bias)
    plan = G.permute(idx, w, E)
    r = G.balance_loss(lg, idx, 1.0, 0.1, bias=bias)
    aux = G.balance_loss_bwd(lg, r["saved"], bias=bias)
    a = G.router_bwd(lg, idx, plan, ds, x, wr, bias=bias)
    b = G.router_bwd(lg, idx, plan, ds, x, wr, bias=bias, dlogits_in=aux)
    torch.cuda.synchronize()
    assert torch.equal(b["dlogits"], a["dlogits"] + aux)
    dz = b["dlogits"].cpu().double()
    x64, w64 = x.cpu().double(), wr.cpu().double()
    for got, ref in ((b["dx"], dz @ w64.t()), (b["dw_r"], x64.t() @ dz), (b["dbias"], dz.sum(0))):
        assert float((got.cpu().double() - ref).abs().max()) <= 1e-5 * float(ref.abs().max())
    mine = aux.clone()
    c = G.router_bwd(lg, idx, plan, ds, x, wr, bias=bias, dlogits_in=mine, dlogits=mine)
    torch.cuda.synchronize()
    assert all(torch.equal(b[n], c[n]) for n in b)


@pytest.mark.parametrize("E,k", [(8, 2), (9, 1)])
def test_gradient_of_more_tokens_than_one_launch_takes(E, k):
    """With `saved` given a token's gradient depends on its own row and sequence alone: the rows around
    2^22 and at the end equal those of a call with these tokens only."""
    import grouped_gemm_top_amd as G
    N = (1 << 22) + 37
    gen = torch.Generator(device="cuda").manual_seed(11)
    lg = torch.randn(N, E, device="cuda", generator=gen)
    mask = (torch.rand(N, device="cuda", generator=gen) > 0.2).to(torch.uint8)
    ptr = torch.tensor([3, 1000, 1 << 21, (1 << 22) - 7, (1 << 22) + 11, N - 2], dtype=torch.int32, device="cuda")
    saved = torch.rand(5 * E + 1, device="cuda", generator=gen)
    dz = G.balance_loss_bwd(lg, saved, mask=mask, seq_ptr=ptr)
    for lo in (0, (1 << 22) - 40, N - 30):
        hi = min(N, lo + 70)
        sub = (ptr - lo).clamp(0, hi - lo).int()
        one = G.balance_loss_bwd(lg[lo:hi].clone(), saved, mask=mask[lo:hi].clone(), seq_ptr=sub)
        assert torch.equal(one, dz[lo:hi]), lo


@pytest.mark.parametrize("E,hot", [(32, 0), (33, 32), (200, 77)])
def test_small_probabilities(E, hot):
    """A probability far below the largest keeps its relative accuracy.  Every token chooses expert
    `hot`, whose logit is 0; the others' are between -64 and -44, so x = z - max is exact, the sum of the
    exponentials is 1 within 1 u and, with beta 0, dlogits[t,m] = -p_m g p_hot for m != hot.  Of that,
    relative: the exponential 2 u from the instruction and 3 u from its argument's and its
    correction's roundings; 1 / sum 4 u, twice (in p_m and in the dot product); products and the
    addition 6 u: 20 u covers the 19.  (x log2 e rounded once would alone be off by up to 44 u.)"""
    import grouped_gemm_top_amd as G
    N = 500
    lg = -44 - 20 * torch.rand(N, E, generator=torch.Generator().manual_seed(12))
    lg[:, hot] = 0.0
    idx = torch.full((N, 1), hot, dtype=torch.int32, device="cuda")
    r = G.balance_loss(lg.cuda(), idx, 0.5)
    d = G.balance_loss_bwd(lg.cuda(), r["saved"]).cpu().double()
    p, g = torch.softmax(lg.double(), 1), float(r["saved"][hot])
    ref = -p * g * p[:, hot:hot + 1]
    err = (d - ref).abs() / (20 * U * ref.abs())
    err[:, hot] = 0.0
    assert float(err.max()) <= 1, float(err.max())


def test_offsets_past_32_bits():
    """N E beyond 2^31 elements: counts and loss of the whole batch, and the last sequence's gradient is that of
    its tokens alone."""
    import grouped_gemm_top_amd as G
    N, E, k = (1 << 21) + 37, 1024, 2
    gen = torch.Generator(device="cuda").manual_seed(13)
    lg = torch.empty(N, E, device="cuda")
    idx = torch.empty(N, k, dtype=torch.int32, device="cuda")
    ptr = torch.tensor([5, 1 << 20, N - 30, N], dtype=torch.int32, device="cuda")
    psum = torch.zeros(3, E, dtype=torch.float64, device="cuda")
    lse2, zm, rows = 0.0, 0.0, 1 << 16
    for lo in range(0, N, rows):
        z = torch.randn(min(rows, N - lo), E, generator=gen, device="cuda")
        lg[lo:lo + rows], idx[lo:lo + rows] = z, z.topk(k, dim=1).indices.int()
        z64, zm = z.double(), max(zm, float(z.abs().max()))
        lse = torch.logsumexp(z64, 1, keepdim=True)
        p = torch.exp(z64 - lse)
        for b in range(3):
            a, e = max(int(ptr[b]) - lo, 0), min(int(ptr[b + 1]) - lo, len(z))
            if a < e:
                psum[b] += p[a:e].sum(0)
                lse2 += float(lse[a:e].square().sum())
    r = G.balance_loss(lg, idx, ALPHA, BETA, seq_ptr=ptr)
    d = G.balance_loss_bwd(lg, r["saved"], seq_ptr=ptr)
    l0 = 0.0
    for b in range(3):
        a, e = int(ptr[b]), int(ptr[b + 1])
        counts = torch.bincount(idx[a:e].reshape(-1).long(), minlength=E)
        assert torch.equal(r["counts"][b].long(), counts)
        l0 += float(ALPHA / 3 * E / (k * (e - a) ** 2) * (counts * psum[b]).sum())
    l1 = BETA * lse2 / (N - 5)
    # a slot adds up to T / SL = 2064 / 4 tokens in a row, then lane exchanges and at most 1024 / 16 + 16 partial rows
    assert abs(float(r["loss"][0]) - l0) <= (4 * zm + 40 + 516 + 16 + 80) * U * l0
    assert abs(float(r["loss"][1]) - l1) <= (2 * zm + 80 + 516 + 16 + 80) * U * l1
    one = G.balance_loss_bwd(lg[-30:].clone(), torch.cat([r["saved"][2 * E:3 * E], r["saved"][-1:]]))
    assert torch.equal(one, d[-30:]) and float(d[:5].abs().max()) == 0.0


@pytest.mark.parametrize("E", [8, 32, 33, 200])
def test_a_bad_token_spoils_the_losses_and_its_own_gradient_alone(E):
    """A counted token with a NaN or +inf logit: NaN losses and a NaN row; other tokens' gradients, which depend on
    the counts alone, are those of the clean call, bit for bit."""
    import grouped_gemm_top_amd as G
    N, k = 70, 2
    lg, _, idx, _, _ = _inputs(N, E, k, 1, False, False, seed=14)
    bad = {3: float("nan"), 7: float("inf"), 64: -float("nan")}
    hurt = lg.clone()
    for t, v in bad.items():
        hurt[t, (5 * t) % E] = v
    a = G.balance_loss(lg.cuda(), idx.cuda(), ALPHA, BETA)
    b = G.balance_loss(hurt.cuda(), idx.cuda(), ALPHA, BETA)
    da, db = (G.balance_loss_bwd(x.cuda(), a["saved"]).cpu() for x in (lg, hurt))
    assert torch.equal(a["counts"], b["counts"]) and torch.equal(a["saved"], b["saved"])
    assert bool(b["loss"].isnan().all())
    keep = [t for t in range(N) if t not in bad]
    assert torch.equal(da[keep], db[keep]) and bool(db[list(bad)].isnan().all())
