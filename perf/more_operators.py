"""Cases, plain forms and 64-bit definitions of three further operators of a model with routed experts.

* ``few`` / ``few8``: the whole expert layer for a few tokens (router product, top-k, gate / up with
  SwiGLU, down, weighted sum), on bf16 or fp32 weights and on MX-FP8 weights;
* ``ckpt_fwd`` / ``ckpt_bwd``: the layer's forward that keeps [G | U] for its backward as MX-FP8
  codes, and the backward that reads them (and, where asked, x too as codes);
* ``ce_fwd`` / ``ce_step``: softmax cross entropy with a z-loss over a large vocabulary whose logits
  x W^T are never kept: the losses alone, or the losses and the gradients of x and W.

``run`` computes a case with elementary torch operations in fp32, rounded once at the end; with
``own`` set it makes the library's calls.  ``exact`` is the definition in fp64, written apart.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token through the microbenchmark's layer: latency
        dict(name="few-1", op="few", N=1, H=2048, I=512, E=128, k=8, dt="bf16", bias=False),
        # sixteen decoding sequences, twice the experts, a skewed router
        dict(name="few-16", op="few", N=16, H=2048, I=512, E=256, k=8, dt="bf16", bias=True),
        # a verification batch of odd size in fp32
        dict(name="few-61-f32", op="few", N=61, H=1432, I=520, E=64, k=4, dt="f32", bias=False),
        # one decoded token on MX-FP8 weights
        dict(name="few8-1", op="few8", N=1, H=2048, I=512, E=128, k=8, bias=False),
        # a small batch on MX-FP8 weights, wide rows and narrow experts
        dict(name="few8-24", op="few8", N=24, H=4096, I=256, E=256, k=8, bias=True),
        # the training forward of the usual micro-batch
        dict(name="ckpt-fwd-4k", op="ckpt_fwd", N=4096, H=2048, I=512, E=128, k=8, skew=0.0),
        # a small ragged forward: odd row counts, scale rows that end inside a word
        dict(name="ckpt-fwd-ragged", op="ckpt_fwd", N=777, H=1440, I=736, E=32, k=4, skew=0.5),
        # the training backward of the usual micro-batch
        dict(name="ckpt-bwd-4k", op="ckpt_bwd", N=4096, H=2048, I=512, E=128, k=8, skew=0.0, x8=False),
        # a coarse layer's large micro-batch, x kept as the norm's codes
        dict(name="ckpt-bwd-coarse", op="ckpt_bwd", N=8192, H=2880, I=2880, E=128, k=4, skew=0.5, x8=True),
        # evaluation of a packed batch: losses only
        dict(name="ce-eval", op="ce_fwd", N=4096, H=2048, V=32000, dt="bf16", ign=0.0, z=0.0),
        # a short fine-tuning batch whose prompt tokens take no part; odd vocabulary
        dict(name="ce-step-300", op="ce_step", N=300, H=1024, V=50021, dt="bf16", ign=0.4, z=0.0),
        # the training step of a large micro-batch, with z-loss and padding
        dict(name="ce-step-8k", op="ce_step", N=8192, H=2048, V=50021, dt="bf16", ign=0.1, z=1e-4),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("few", "few8", "ckpt_fwd", "ckpt_bwd", "ce_fwd", "ce_step"))
    if op in ("few", "few8"):
        E = _log(rng, 4, 256)
        k = rng.randint(1, min(8, E))
        g = 32 if op == "few8" else 8
        H, I = g * _log(rng, 128 // g, 4096 // g), g * _log(rng, 64 // g, 2048 // g)
        while E * H * I > 256 * 2048 * 1024:
            E = max(k, E // 2)
            if E == k:
                I = max(g, 256 * 2048 * 1024 // (E * H) // g * g)
        c = dict(op=op, N=_log(rng, 1, 64), H=H, I=I, E=E, k=k, bias=rng.random() < 0.5)
        if op == "few":
            c["dt"] = rng.choice(("bf16", "bf16", "f32"))
        return c
    if op in ("ckpt_fwd", "ckpt_bwd"):
        E = _log(rng, 2, 256)
        k = rng.randint(1, min(8, E))
        H, I = 32 * _log(rng, 2, 90), 32 * _log(rng, 1, 90)
        E = max(k, min(E, 128 * 2880 * 2880 // (H * I)))
        N = _log(rng, 1, max(1, min(8192, 8192 * 4 * 2880 * 2880 // (k * H * I))))
        c = dict(op=op, N=N, H=H, I=I, E=E, k=k, skew=rng.choice((0.0, 0.5)))
        if op == "ckpt_bwd":
            c["x8"] = rng.random() < 0.5
        return c
    dt = rng.choice(("bf16", "bf16", "f32"))
    top = 8192 * 2048 * 50021 // (8 if dt == "f32" else 1)
    H, V = 8 * _log(rng, 8, 512), _log(rng, 50, 131072)
    V = min(V, 2048 * 50021 // H)
    N = _log(rng, 1, max(1, min(16384, top // (H * V))))
    return dict(op=op, N=N, H=H, V=V, dt=dt, ign=rng.choice((0.0, 0.1, 0.5)), z=rng.choice((0.0, 1e-4)))


def work(case):
    op, N, H = case["op"], case["N"], case["H"]
    if op in ("few", "few8"):
        I, E, k = case["I"], case["E"], case["k"]
        # the experts that N tokens are expected to name, each read once
        named = E * (1.0 - (1.0 - k / E) ** N)
        es = {"bf16": 2, "f32": 4}[case.get("dt", "bf16")]
        ws = 1 + 1 / 32 if op == "few8" else es
        return {"bytes": named * 3 * H * I * ws + 4 * H * E + 2 * N * H * es + 8 * N * k,
                "flops": 2 * N * H * E + 6 * N * k * H * I}
    if op in ("ckpt_fwd", "ckpt_bwd"):
        I, E, M = case["I"], case["E"], N * case["k"]
        q = 1 + 1 / 32  # bytes of a value held as a code with its share of the scale
        if op == "ckpt_fwd":
            return {"bytes": 2 * N * H + 6 * E * H * I + 2 * M * I * q + 2 * M * H, "flops": 6 * M * H * I}
        return {"bytes": N * H * (4 + (q if case["x8"] else 2)) + 12 * E * H * I + 2 * M * I * q + 4 * M,
                "flops": 12 * M * H * I}
    V, es, n = case["V"], {"bf16": 2, "f32": 4}[case["dt"]], N * (1 - case["ign"])
    if op == "ce_fwd":
        return {"bytes": es * (n * H + V * H) + 12 * N, "flops": 2 * n * H * V}
    # without keeping the logits, the gradient forms them again: four products of n x H x V
    return {"bytes": 2 * es * (N * H + V * H) + 16 * N, "flops": 8 * n * H * V}


# ------------------------------------------------------------------ inputs

def _mx(v):
    """v [..., K] as MX-FP8 -> (codes uint8 [..., K], scale codes uint8 [..., 4 ceil(K / 128)])."""
    K = v.shape[-1]
    b = v.float().view(*v.shape[:-1], K // 32, 32)
    # the smallest power of two X with max |v| <= 448 X, 448 = 0.875 * 2^9
    m, e = torch.frexp(b.abs().amax(dim=-1))
    x8 = (e - 9 + (m > 0.875)).clamp(-127, 127)
    q = torch.ldexp(b, -x8[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(v.shape)
    s = torch.zeros(*v.shape[:-1], 4 * ((K + 127) // 128), dtype=torch.uint8, device=v.device)
    s[..., :K // 32] = (x8 + 127).to(torch.uint8)
    return q, s


def _unmx(q, s, dt=torch.float32):
    """The values that codes and scale codes stand for."""
    K = q.shape[-1]
    v = q.view(torch.float8_e4m3fn).to(dt).view(*q.shape[:-1], K // 32, 32)
    x = torch.exp2(s[..., :K // 32].to(dt) - 127)
    return (v * x[..., None]).view(q.shape)


def _plan(N, E, k, logits):
    """The expert-sorted plan of a top-k routing, and each expert's rows on the host."""
    idx = logits.topk(k, dim=1).indices
    z = logits.gather(1, idx)
    w = torch.softmax(z, dim=1).float()
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=flat.device), counts.cumsum(0)])
    rows = torch.empty_like(order)
    rows[order] = torch.arange(N * k, device=flat.device)
    i32 = torch.int32
    return dict(counts=counts.to(i32), offsets=offsets.to(i32), row_token=(order // k).to(i32),
                row_w=w.reshape(-1)[order].contiguous(), row_pair=order.to(i32),
                tok_ptr=(torch.arange(N + 1, device=flat.device) * k).to(i32),
                tok_rows=rows.view(N, k).sort(dim=1).values.reshape(-1).to(i32)), counts.tolist()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s, op, bf = dict(case), case["op"], torch.bfloat16
    N, H = case["N"], case["H"]
    if op in ("few", "few8"):
        I, E, k = case["I"], case["E"], case["k"]
        dt = DT[case.get("dt", "bf16")]
        s["w_r"] = 1.5 / math.sqrt(H) * rnd(H, E)
        s["b"] = None
        if case["bias"]:  # a skewed router: half the logarithm of a Zipf law over a random order of the experts
            s["b"] = (-0.5 * torch.log(torch.randperm(E, generator=cpu).float() + 1.0)).cuda()
        x = rnd(N, H).to(dt)
        while True:  # tokens whose choice of experts hangs on the last digits of a logit are drawn again
            z = x.double() @ s["w_r"].double() + (0.0 if s["b"] is None else s["b"].double())
            t = z.sort(dim=1, descending=True).values[:, :k + 1]
            near = (t[:, :-1] - t[:, 1:] < 2e-4).any(dim=1) if t.shape[1] > 1 else torch.zeros(N, dtype=torch.bool)
            if not bool(near.any()):
                break
            x[near] = rnd(int(near.sum()), H).to(dt)
        s["x"] = x
        for n, shape in (("wg", (E, I, H)), ("wu", (E, I, H)), ("wd", (E, H, I))):
            w = rnd(*shape).mul_(1.0 / math.sqrt(shape[2]))
            s[n] = _mx(w) if op == "few8" else w.to(dt)
        return s
    if op in ("ckpt_fwd", "ckpt_bwd"):
        I, E, k = case["I"], case["E"], case["k"]
        s["plan"], s["rows"] = _plan(N, E, k, rnd(N, E) + case["skew"] * rnd(E))
        x = rnd(N, H).to(bf)
        s["x"] = _mx(x) if case.get("x8") else x
        for n, shape in (("wg", (E, I, H)), ("wu", (E, I, H)), ("wd", (E, H, I))):
            s[n] = rnd(*shape).mul_(1.0 / math.sqrt(shape[2])).to(bf)
        if op == "ckpt_bwd":
            s["dout"] = rnd(N, H).to(bf)
            hq, hs = _mx(0.9 * rnd(N * k, 2, I))
            s["hq"], s["hs"] = hq.view(N * k, 2 * I), hs.view(N * k, -1)
        return s
    V, dt = case["V"], DT[case["dt"]]
    s["x"], s["w"] = rnd(N, H).to(dt), (2.0 / math.sqrt(H) * rnd(V, H)).to(dt)
    # targets by a Zipf law; a token without one has -100
    t = torch.exp(torch.rand(N, generator=g, device="cuda") * math.log(V)).long().clamp(max=V) - 1
    s["t"] = torch.where(torch.rand(N, generator=g, device="cuda") < case["ign"], -100, t).int()
    s["dloss"] = (1.0 + 0.1 * rnd(N)) / N
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        import grouped_gemm_top_amd as G
        return _RUN_OWN[s["op"]](G, s)
    return _RUN[s["op"]](s)


def _own_few(G, s):
    r = G.layer_few(s["x"], s["w_r"], s["wg"], s["wu"], s["wd"], s["k"], bias=s["b"])
    return dict(out=r["out"], idx=r["topk_idx"], w=r["topk_w"])


def _own_plan(G, s):
    return G.Plan(s["N"], s["E"], s["k"], alloc=lambda name, n, dt: s["plan"][name])


def _own_ckpt_fwd(G, s):
    (hq, hs), y = G.grouped_gemm_fwd_ckpt8(s["x"], s["wg"], s["wu"], s["wd"], _own_plan(G, s))
    return dict(y=y, hq=hq.view(torch.float8_e4m3fn), hs=hs.view(torch.float8_e8m0fnu))


def _own_ckpt_bwd(G, s):
    r = G.layer_bwd_ckpt8(s["dout"], s["x"], s["wg"], s["wu"], s["wd"], _own_plan(G, s), (s["hq"], s["hs"]))
    return {n: r[n] for n in ("dx", "dw_gate", "dw_up", "dw_down", "ds")}


def _own_ce_fwd(G, s):
    r = G.linear_ce_fwd(s["x"], s["w"], s["t"], z_coef=s["z"])
    return dict(loss=r["loss"], lse=r["lse"])


def _own_ce_step(G, s):
    f = G.linear_ce_fwd(s["x"], s["w"], s["t"], z_coef=s["z"])
    b = G.linear_ce_bwd(s["dloss"], s["x"], s["w"], s["t"], f["lse"], z_coef=s["z"])
    return dict(loss=f["loss"], lse=f["lse"], dx=b["dx"], dw=b["dw"])


_RUN_OWN = dict(few=_own_few, few8=_own_few, ckpt_fwd=_own_ckpt_fwd, ckpt_bwd=_own_ckpt_bwd, ce_fwd=_own_ce_fwd,
                ce_step=_own_ce_step)


def _plain_few(s):
    N, k = s["N"], s["k"]
    # (the choice of experts compares logits: 64 bits)
    z = s["x"].double() @ s["w_r"].double()
    if s["b"] is not None:
        z = z + s["b"]
    z, idx = z.sort(dim=1, descending=True, stable=True)
    z, idx = z[:, :k].float(), idx[:, :k]
    e = torch.exp(z - z[:, :1])
    w = e / e.sum(dim=1, keepdim=True)
    p = idx.reshape(-1)
    take = (lambda t: _unmx(t[0][p], t[1][p])) if s["op"] == "few8" else (lambda t: t[p].float())
    xp = s["x"].float().repeat_interleave(k, dim=0)[:, :, None]
    gate, up = take(s["wg"]) @ xp, take(s["wu"]) @ xp
    a = gate / (1 + torch.exp(-gate)) * up
    y = (take(s["wd"]) @ a).view(N, k, -1)
    return dict(out=(w[:, :, None] * y).sum(dim=1).to(s["x"].dtype), idx=idx.int(), w=w)


def _padded(s):
    """Each expert's rows as [E, C] with C the fullest one's count: the row, and whether there is one."""
    c = torch.arange(max(s["rows"]), device=s["plan"]["counts"].device)
    live = c[None, :] < s["plan"]["counts"][:, None]
    row = torch.where(live, s["plan"]["offsets"][:-1, None] + c, 0).long()
    return row, live


def _plain_ckpt_fwd(s):
    row, live = _padded(s)
    x = s["x"].float()[s["plan"]["row_token"][row].long()]  # [E, C, H]
    gate, up = (torch.bmm(x, s[n].float().transpose(1, 2).contiguous()) for n in ("wg", "wu"))
    a = gate / (1 + torch.exp(-gate)) * up
    y = torch.bmm(a, s["wd"].float().transpose(1, 2).contiguous())
    # back to the rows' order: the live entries of [E, C], expert by expert
    hq, hs = _mx(torch.stack([gate[live], up[live]], dim=1))
    M = hq.shape[0]
    return dict(y=y[live].to(torch.bfloat16), hq=hq.view(M, -1).view(torch.float8_e4m3fn),
                hs=hs.view(M, -1).view(torch.float8_e8m0fnu))


def _plain_ckpt_bwd(s):
    N, I, k = s["N"], s["I"], s["k"]
    row, live = _padded(s)
    M, p, bf = N * k, s["plan"], torch.bfloat16
    tok = p["row_token"][row].long()
    h = _unmx(s["hq"].view(M, 2, I), s["hs"].view(M, 2, -1))[row] * live[:, :, None, None]
    gate, up = h[:, :, 0], h[:, :, 1]
    x = (_unmx(*s["x"]) if s["x8"] else s["x"].float())[tok]
    dout = s["dout"].float()[tok] * live[:, :, None]
    w = (p["row_w"][row] * live)[:, :, None]
    da = torch.bmm(dout, s["wd"].float())
    sg = 1 / (1 + torch.exp(-gate))
    a = gate * sg * up
    dsr = (da * a).sum(dim=2)[live]
    da = da * w
    dg, du = da * up * sg * (1 + gate * (1 - sg)), da * gate * sg
    dxe = torch.bmm(dg, s["wg"].float()) + torch.bmm(du, s["wu"].float())
    dx = torch.zeros(N, s["H"], device=x.device).index_add_(0, p["row_token"].long(), dxe[live])
    ds = torch.empty(M, device=x.device)
    ds[p["row_pair"].long()] = dsr
    return dict(dx=dx.to(bf), dw_gate=torch.bmm(dg.transpose(1, 2).contiguous(), x).to(bf),
                dw_up=torch.bmm(du.transpose(1, 2).contiguous(), x).to(bf),
                dw_down=torch.bmm(dout.transpose(1, 2).contiguous(), a * w).to(bf), ds=ds.view(N, k))


def _plain_ce(s):
    x, w, t = s["x"].float(), s["w"].float(), s["t"].long()
    live = (t >= 0) & (t < s["V"])
    z = x @ w.t().contiguous()
    m = z.max(dim=1, keepdim=True).values
    lse = (m + torch.log(torch.exp(z - m).sum(dim=1, keepdim=True)))[:, 0]
    tt = torch.where(live, t, 0)
    loss = lse - z.gather(1, tt[:, None])[:, 0] + s["z"] * lse * lse
    return x, w, z, lse, tt, live, loss


def _plain_ce_fwd(s):
    _, _, _, lse, _, live, loss = _plain_ce(s)
    return dict(loss=torch.where(live, loss, 0.0), lse=torch.where(live, lse, 0.0))


def _plain_ce_step(s):
    x, w, z, lse, tt, live, loss = _plain_ce(s)
    g = torch.where(live, s["dloss"], 0.0)[:, None]
    dz = torch.exp(z - lse[:, None]) * (g * (1 + 2 * s["z"] * lse[:, None]))
    dz.scatter_add_(1, tt[:, None], -g)
    ty = s["x"].dtype
    return dict(loss=torch.where(live, loss, 0.0), lse=torch.where(live, lse, 0.0), dx=(dz @ w).to(ty),
                dw=(dz.t().contiguous() @ x).to(ty))


_RUN = dict(few=_plain_few, few8=_plain_few, ckpt_fwd=_plain_ckpt_fwd, ckpt_bwd=_plain_ckpt_bwd, ce_fwd=_plain_ce_fwd,
            ce_step=_plain_ce_step)


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _values(t):
    """A tensor, or what a pair of codes and scale codes stands for, in 64 bits."""
    if not isinstance(t, tuple):
        return t.double()
    q, s = t
    v = q.view(torch.float8_e4m3fn).double()
    return v * torch.pow(2.0, s.double() - 127).repeat_interleave(32, dim=-1)[..., :q.shape[-1]]


def _at(t, e):
    return _values((t[0][e], t[1][e]) if isinstance(t, tuple) else t[e])


def _exact_few(case, s):
    x = s["x"].double()
    z = x @ s["w_r"].double()
    if s["b"] is not None:
        z = z + s["b"].double()
    top, idx = torch.topk(z, case["k"], dim=1)
    w = torch.softmax(top, dim=1)
    out = torch.zeros_like(x)
    for e in sorted(set(idx.flatten().tolist())):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        h = torch.nn.functional.silu(x[t] @ _at(s["wg"], e).t()) * (x[t] @ _at(s["wu"], e).t())
        out.index_add_(0, t, w[t, j][:, None] * (h @ _at(s["wd"], e).t()))
    return dict(out=out, idx=None, w=w)


def _exact_ckpt_fwd(case, s):
    tok, M = s["plan"]["row_token"].long(), case["N"] * case["k"]
    x = s["x"].double()
    y, gu, o = [], [], 0
    for e, n in enumerate(s["rows"]):
        xe = x[tok[o:o + n]]
        o += n
        g, u = xe @ s["wg"][e].double().t(), xe @ s["wu"][e].double().t()
        y.append((torch.nn.functional.silu(g) * u) @ s["wd"][e].double().t())
        gu.append(torch.stack([g, u], dim=1))
    # the values that the codes round (their rounding is a code's own); the scales are whole powers
    b = torch.cat(gu).view(M, 2, case["I"] // 32, 32)
    x8 = torch.ceil(torch.log2(b.abs().amax(dim=3).clamp(min=2.0 ** -126) / 448.0)).clamp(-127, 127)
    return dict(y=torch.cat(y), hq=(b * torch.exp2(-x8)[..., None]).view(M, 2 * case["I"]), hs=None)


def _exact_ckpt_bwd(case, s):
    N, I, E, k, p = case["N"], case["I"], case["E"], case["k"], s["plan"]
    M = N * k
    tok, rw = p["row_token"].long(), p["row_w"].double()
    h = _values((s["hq"].view(M, 2, I), s["hs"].view(M, 2, -1)))
    x, dout = _values(s["x"]), s["dout"].double()
    dx = torch.zeros_like(x)
    dw = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=x.device) for n in ("wg", "wu", "wd")}
    ds, o = torch.zeros(M, dtype=torch.float64, device=x.device), 0
    for e, n in enumerate(s["rows"]):
        if n == 0:
            continue
        r = slice(o, o + n)
        o += n
        t = tok[r]
        g, u, w = h[r, 0].requires_grad_(True), h[r, 1].requires_grad_(True), rw[r].requires_grad_(True)
        wd = s["wd"][e].double().requires_grad_(True)
        y = w[:, None] * torch.nn.functional.linear(torch.nn.functional.silu(g) * u, wd)
        dg, du, dw_, dwd = torch.autograd.grad(y, (g, u, w, wd), dout[t])
        dx.index_add_(0, t, dg @ s["wg"][e].double() + du @ s["wu"][e].double())
        dw["wg"][e], dw["wu"][e], dw["wd"][e] = dg.t() @ x[t], du.t() @ x[t], dwd
        ds[p["row_pair"][r].long()] = dw_
    return dict(dx=dx, dw_gate=dw["wg"], dw_up=dw["wu"], dw_down=dw["wd"], ds=ds.view(N, k))


def _exact_ce(case, s, grads):
    t = s["t"].long()
    live = torch.nonzero((t >= 0) & (t < case["V"]))[:, 0]
    x, w = s["x"][live].double().requires_grad_(grads), s["w"].double().requires_grad_(grads)
    z = torch.nn.functional.linear(x, w)
    lse = torch.logsumexp(z, dim=1)
    each = torch.nn.functional.cross_entropy(z, t[live], reduction="none") + case["z"] * lse.square()
    full = lambda v, *n: torch.zeros(case["N"], *n, dtype=torch.float64, device=v.device).index_copy_(0, live, v)  # noqa: E731
    o = dict(loss=full(each.detach()), lse=full(lse.detach()))
    if grads:
        dx, o["dw"] = torch.autograd.grad(each, (x, w), s["dloss"][live].double())
        o["dx"] = full(dx, case["H"])
    return {n: o[n] for n in ("loss", "lse", "dx", "dw") if n in o}


_EXACT = dict(few=_exact_few, few8=_exact_few, ckpt_fwd=_exact_ckpt_fwd, ckpt_bwd=_exact_ckpt_bwd,
              ce_fwd=lambda c, s: _exact_ce(c, s, False), ce_step=lambda c, s: _exact_ce(c, s, True))
