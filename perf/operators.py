"""Cases, plain forms and 64-bit definitions of three operators around the routed expert layer.

* ``balance``: the router's balance loss and z-loss with per-expert counts, and their gradient with
  respect to the logits (one training pass: forward and gradient);
* ``norm`` / ``norm_bwd``: residual addition + RMS norm, optionally with an MX-FP8 output (e4m3
  codes, one power-of-two scale per 32 values), and its backward pass;
* ``linear`` / ``linear_bwd``: x W^T with bias, activation and residual in the epilogue (bf16),
  and its backward pass.

``run`` computes a case with elementary torch operations in fp32, rounded once at the end; with
``own`` set it makes the library's calls.  ``exact`` is the definition in fp64, written apart.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one small micro-batch of a tiny model (64 tokens, 8 experts): launch latency
        dict(name="balance-tiny", op="balance", N=64, E=8, k=2, B=1, mask=False, bias=False, z=True),
        # the layer's usual micro-batch, four equal sequences
        dict(name="balance-4k", op="balance", N=4096, E=128, k=8, B=4, mask=False, bias=False, z=True),
        # a long packed batch: ragged sequences, padding tokens masked, a skewed router with bias
        dict(name="balance-packed-64k", op="balance", N=65536, E=256, k=8, B=37, mask=True, bias=True, z=True),
        # one decoded token in front of an MX-FP8 layer
        dict(name="norm-token", op="norm", N=1, H=2048, dt="bf16", rdt="bf16", y=True, quant=True),
        # the layer's usual micro-batch: bf16 for the router and the backward, codes for the experts
        dict(name="norm-quant-4k", op="norm", N=4096, H=2048, dt="bf16", rdt="bf16", y=True, quant=True),
        # a long prefill on an fp32 residual stream, codes only, rows that fill no whole number of wavefronts
        dict(name="norm-quant-f32-stream", op="norm", N=16383, H=2880, dt="bf16", rdt="f32", y=False, quant=True),
        # training, the usual micro-batch
        dict(name="norm-bwd-4k", op="norm_bwd", N=4096, H=2048, dt="bf16", rdt="bf16", dh=True),
        # training, a wide model's large micro-batch on an fp32 residual stream
        dict(name="norm-bwd-wide", op="norm_bwd", N=16384, H=4096, dt="bf16", rdt="f32", dh=True),
        # one decoded token through a projection with its residual
        dict(name="linear-token", op="linear", N=1, K=4096, O=4096, act="silu", bias=True, res=True, z=False),
        # a ragged batch of odd sizes
        dict(name="linear-ragged", op="linear", N=333, K=2880, O=2056, act="gelu", bias=True, res=True, z=False),
        # a large prefill or training forward; z is kept for the backward
        dict(name="linear-prefill", op="linear", N=8192, K=4096, O=4096, act="gelu_tanh", bias=True, res=True, z=True),
        # the training backward of a dense MLP's first product
        dict(name="linear-bwd", op="linear_bwd", N=8192, K=2048, O=4096, act="gelu_tanh", bias=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("balance", "norm", "norm_bwd", "linear", "linear_bwd"))
    if op == "balance":
        N, E = _log(rng, 1, 65536), _log(rng, 4, 256)
        return dict(op=op, N=N, E=E, k=rng.randint(1, min(8, E)), B=_log(rng, 1, 64), mask=rng.random() < 0.5,
                    bias=rng.random() < 0.5, z=rng.random() < 0.7)
    if op in ("norm", "norm_bwd"):
        H = 32 * _log(rng, 2, 256)
        N = _log(rng, 1, min(32768, 16384 * 4096 // H))
        dt = rng.choice(("bf16", "bf16", "f32"))
        rdt = "f32" if dt == "f32" else rng.choice(("bf16", "f32"))
        if op == "norm_bwd":
            return dict(op=op, N=N, H=H, dt=dt, rdt=rdt, dh=rng.random() < 0.8)
        quant = rng.random() < 0.6
        if not quant:
            H += 8 * rng.randint(0, 3)
        return dict(op=op, N=N, H=H, dt=dt, rdt=rdt, y=not quant or rng.random() < 0.6, quant=quant)
    K, O = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 512)
    act, bias = rng.choice(ACTS), rng.random() < 0.7
    if op == "linear":
        return dict(op=op, N=_log(rng, 1, 8192), K=K, O=O, act=act, bias=bias, res=rng.random() < 0.6,
                    z=rng.random() < 0.3)
    return dict(op=op, N=_log(rng, 1, 8192), K=K, O=min(O, 4096 * 2048 // K) // 8 * 8, act=act, bias=bias)


def work(case):
    op = case["op"]
    if op == "balance":
        N, E, k, B = case["N"], case["E"], case["k"], case["B"]
        # forward and gradient each read the logits; the gradient and the counts are written
        return {"bytes": 12 * N * E + 4 * N * k + 4 * B * E + 2 * N * case["mask"], "flops": 12 * N * E}
    es = {"bf16": 2, "f32": 4}
    if op == "norm":
        N, H, d, r = case["N"], case["H"], es[case["dt"]], es[case["rdt"]]
        out = d * case["y"] + (1 + 1 / 32) * case["quant"]
        return {"bytes": N * H * (d + 2 * r + out) + 4 * H, "flops": 8 * N * H}
    if op == "norm_bwd":
        N, H, d, r = case["N"], case["H"], es[case["dt"]], es[case["rdt"]]
        return {"bytes": N * H * (d + r * (2 + case["dh"])) + 8 * H, "flops": 12 * N * H}
    N, K, O = case["N"], case["K"], case["O"]
    if op == "linear":
        return {"bytes": 2 * (N * K + O * K + N * O * (1 + case["res"] + case["z"])) + 4 * O * case["bias"],
                "flops": 2 * N * K * O}
    z = case["act"] != "none"
    return {"bytes": 2 * (2 * N * K + 2 * O * K + N * O * (1 + z)) + 4 * O * case["bias"], "flops": 4 * N * K * O}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s, op = dict(case), case["op"]
    if op == "balance":
        N, E, k, B = case["N"], case["E"], case["k"], case["B"]
        s["logits"] = 1.5 * rnd(N, E)
        # a skewed router: the logarithm of a Zipf law over a random order of the experts
        s["bias"] = None
        if case["bias"]:
            s["bias"] = (-torch.log(torch.randperm(E, generator=cpu).float() + 1.0)).cuda()
        z = s["logits"] if s["bias"] is None else s["logits"] + s["bias"]
        s["idx"] = z.topk(k, dim=1).indices.int()
        # ragged sequences (some may be empty); with a mask, a tenth of the tokens is padding
        # and the batch's last tokens belong to no sequence
        if case["mask"]:
            s["mask"] = (torch.rand(N, generator=g, device="cuda") < 0.9).to(torch.uint8)
            cuts = torch.randint(0, N + 1, (B,), generator=cpu).sort().values.int()
            s["seq_ptr"] = torch.cat([torch.zeros(1, dtype=torch.int32), cuts]).cuda()
        else:
            s["mask"] = None
            s["seq_ptr"] = (torch.arange(B + 1, dtype=torch.int64) * N // B).int().cuda()
        s["alpha"], s["beta"] = 1e-2, 1e-3 if case["z"] else 0.0
        return s
    if op in ("norm", "norm_bwd"):
        N, H, dt, rdt = case["N"], case["H"], DT[case["dt"]], DT[case["rdt"]]
        s["w"] = 1.0 + 0.1 * rnd(H)
        if op == "norm":
            s["x"], s["res"] = rnd(N, H).to(dt), (2.0 * rnd(N, H)).to(rdt)
        else:
            s["dy"], s["h"] = (0.01 * rnd(N, H)).to(dt), (2.0 * rnd(N, H)).to(rdt)
            s["dh_in"] = (0.01 * rnd(N, H)).to(rdt) if case["dh"] else None
        return s
    N, K, O = case["N"], case["K"], case["O"]
    bf = torch.bfloat16
    s["x"], s["w"] = rnd(N, K).to(bf), (rnd(O, K) / math.sqrt(K)).to(bf)
    if op == "linear":
        s["b"] = 0.5 * rnd(O) if case["bias"] else None
        s["r"] = rnd(N, O).to(bf) if case["res"] else None
    else:
        s["dout"] = (0.1 * rnd(N, O)).to(bf)
        s["zin"] = (1.2 * rnd(N, O)).to(bf) if case["act"] != "none" else None
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        import grouped_gemm_top_amd as G
        return _RUN_OWN[s["op"]](G, s)
    return _RUN[s["op"]](s)


def _own_balance(G, s):
    f = G.balance_loss(s["logits"], s["idx"], s["alpha"], s["beta"], bias=s["bias"], mask=s["mask"],
                       seq_ptr=s["seq_ptr"])
    d = G.balance_loss_bwd(s["logits"], f["saved"], bias=s["bias"], mask=s["mask"], seq_ptr=s["seq_ptr"])
    return dict(loss=f["loss"], counts=f["counts"], dlogits=d)


def _own_norm(G, s):
    r = G.add_rmsnorm(s["x"], s["w"], residual=s["res"], eps=EPS, want_y=s["y"], quantize=s["quant"])
    return _norm_out(s, r["h"], r["y"], r["q"], r["scales"])


def _own_norm_bwd(G, s):
    r = G.add_rmsnorm_bwd(s["dy"], s["h"], s["w"], dh_in=s["dh_in"], eps=EPS)
    return dict(dh=r["dh"], dw=r["dw"])


def _own_linear(G, s):
    out, z = G.linear_fwd(s["x"], s["w"], bias=s["b"], act=s["act"], residual=s["r"], want_z=s["z"])
    return dict(out=out, z=z) if s["z"] else dict(out=out)


def _own_linear_bwd(G, s):
    r = G.linear_bwd(s["dout"], s["x"], s["w"], z=s["zin"], act=s["act"], want_dbias=s["bias"])
    return {n: r[n] for n in ("dx", "dw", "dbias") if r[n] is not None}


_RUN_OWN = dict(balance=_own_balance, norm=_own_norm, norm_bwd=_own_norm_bwd, linear=_own_linear,
                linear_bwd=_own_linear_bwd)


def _norm_out(s, h, y, q, scales):
    """The outputs asked for; codes and scale codes as the 8-bit floating-point values they are."""
    o = dict(h=h)
    if s["y"]:
        o["y"] = y
    if s["quant"]:
        o["q"], o["scales"] = q.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)
    return o


def _seq_of(s):
    """Each token's sequence and whether it counts."""
    N, ptr = s["N"], s["seq_ptr"]
    t = torch.arange(N, device=ptr.device, dtype=torch.int32)
    seq = torch.searchsorted(ptr, t, right=True) - 1
    live = (seq >= 0) & (seq < s["B"])
    if s["mask"] is not None:
        live = live & (s["mask"] != 0)
    return torch.where(live, seq, 0), live


def _plain_balance(s):
    N, E, k, B = s["N"], s["E"], s["k"], s["B"]
    seq, live = _seq_of(s)
    z = s["logits"] if s["bias"] is None else s["logits"] + s["bias"]
    zmax = z.max(dim=1, keepdim=True).values
    ez = torch.exp(z - zmax)
    sum_e = ez.sum(dim=1, keepdim=True)
    p = ez / sum_e * live[:, None]
    lse = (zmax + torch.log(sum_e))[:, 0] * live
    slot = (seq[:, None] * E + s["idx"]).reshape(-1)
    counts = torch.bincount(slot, weights=live[:, None].expand(N, k).reshape(-1).double(), minlength=B * E)
    counts = counts.view(B, E).int()
    # whole-number sums in fp64; the sums of probabilities per sequence as a product with the
    # sequences' indicator matrix
    nb = torch.bincount(seq, weights=live.double(), minlength=B).float()
    member = (seq[None, :] == torch.arange(B, device=seq.device)[:, None]).float()
    psum = member @ p
    n = nb.sum()
    coef = torch.where(nb > 0, s["alpha"] * E / (B * k * nb.clamp(min=1) ** 2), 0.0)
    g = coef[:, None] * counts
    loss = torch.stack([(g * psum).sum(), s["beta"] * (lse * lse).sum() / n.clamp(min=1)])
    gt = g[seq]
    dz = p * (gt - (gt * p).sum(dim=1, keepdim=True)) + (2 * s["beta"] / n.clamp(min=1)) * lse[:, None] * p
    return dict(loss=loss, counts=counts, dlogits=dz)


def _plain_norm(s):
    x = s["x"].float() + s["res"].float()
    r = torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS)
    y = x * r * s["w"]
    q = scales = None
    if s["quant"]:
        N, H = y.shape
        blocks = y.view(N, H // 32, 32)
        # the smallest power of two X with max |v| <= 448 X, 448 = 0.875 * 2^9
        m, e = torch.frexp(blocks.abs().amax(dim=2))
        x8 = (e - 9 + (m > 0.875)).clamp(-127, 127)
        q = torch.ldexp(blocks, -x8[:, :, None]).to(torch.float8_e4m3fn).view(N, H)
        scales = torch.zeros(N, 4 * ((H + 127) // 128), dtype=torch.uint8, device=y.device)
        scales[:, :H // 32] = (x8 + 127).to(torch.uint8)
    return _norm_out(s, x.to(s["res"].dtype), y.to(s["x"].dtype), q, scales)


def _plain_norm_bwd(s):
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    a = dy * s["w"]
    dh = r * (a - h * (r * r * (a * h).mean(dim=1, keepdim=True)))
    if s["dh_in"] is not None:
        dh = dh + s["dh_in"].float()
    return dict(dh=dh.to(s["h"].dtype), dw=(dy * h * r).sum(dim=0))


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _dact(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().t().contiguous()
    if s["b"] is not None:
        z = z + s["b"]
    out = _act(z, s["act"])
    if s["r"] is not None:
        out = out + s["r"].float()
    out = out.to(torch.bfloat16)
    return dict(out=out, z=z.to(torch.bfloat16)) if s["z"] else dict(out=out)


def _plain_linear_bwd(s):
    dz = s["dout"].float()
    if s["zin"] is not None:
        dz = dz * _dact(s["zin"].float(), s["act"])
    bf = torch.bfloat16
    o = dict(dx=(dz @ s["w"].float()).to(bf), dw=(dz.t().contiguous() @ s["x"].float()).to(bf))
    if s["bias"]:
        o["dbias"] = dz.sum(dim=0)
    return o


_RUN = dict(balance=_plain_balance, norm=_plain_norm, norm_bwd=_plain_norm_bwd, linear=_plain_linear,
            linear_bwd=_plain_linear_bwd)


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = {n: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for n, v in prepare(case, seed).items()}
    return _EXACT[case["op"]](case, s)


def _exact_balance(case, s):
    N, E, k, B = (case[n] for n in ("N", "E", "k", "B"))
    z = s["logits"] + (s["bias"] if s["bias"] is not None else 0.0)
    z.requires_grad_(True)
    lsm = torch.log_softmax(z, dim=1)
    lse = torch.logsumexp(z, dim=1)
    keep = torch.ones(N, dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"].bool()
    ptr = s["seq_ptr"].tolist()
    l0, l1, n = 0.0, 0.0, 0
    for b in range(B):
        t = torch.nonzero(keep[ptr[b]:ptr[b + 1]])[:, 0] + ptr[b]
        nb = t.numel()
        if nb == 0:
            continue
        hot = torch.zeros(nb, E, dtype=torch.float64, device=z.device).scatter_(1, s["idx"][t].long(), 1.0)
        f = hot.sum(dim=0) * (E / (k * nb))
        l0 = l0 + s["alpha"] / B * (f * lsm[t].exp().mean(dim=0)).sum()
        l1, n = l1 + lse[t].square().sum(), n + nb
    if n == 0:
        return dict(loss=torch.zeros(2, dtype=torch.float64), counts=None, dlogits=torch.zeros_like(z))
    l1 = s["beta"] * l1 / n
    grad = torch.autograd.grad(l0 + l1, z)[0]
    return dict(loss=torch.stack([l0.detach(), l1.detach()]), counts=None, dlogits=grad)


def _exact_norm(case, s):
    h = s["x"] + s["res"]
    y = h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + EPS) * s["w"]
    o = dict(h=h)
    if case["y"]:
        o["y"] = y
    if case["quant"]:
        # the values that the codes round (their rounding is a code's own); the scales are whole powers
        N, H = y.shape
        top = y.view(N, H // 32, 32).abs().amax(dim=2).clamp(min=2.0 ** -126)
        x8 = torch.ceil(torch.log2(top / 448.0)).clamp(-127, 127)
        o["q"] = (y.view(N, H // 32, 32) * torch.exp2(-x8)[:, :, None]).view(N, H)
        o["scales"] = None
    return o


def _exact_norm_bwd(case, s):
    h, w = s["h"].requires_grad_(True), s["w"].requires_grad_(True)
    y = h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + EPS) * w
    dh, dw = torch.autograd.grad(y, (h, w), s["dy"])
    return dict(dh=dh if s["dh_in"] is None else dh + s["dh_in"], dw=dw)


_TORCH_ACT = dict(none=lambda z: z, relu=torch.relu, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu,
                  gelu_tanh=lambda z: torch.nn.functional.gelu(z, approximate="tanh"))


def _exact_linear(case, s):
    z = torch.nn.functional.linear(s["x"], s["w"], s["b"])
    out = _TORCH_ACT[case["act"]](z) + (s["r"] if s["r"] is not None else 0.0)
    return dict(out=out, z=z) if case["z"] else dict(out=out)


def _exact_linear_bwd(case, s):
    dz = s["dout"]
    if s["zin"] is not None:
        z = s["zin"].requires_grad_(True)
        dz = torch.autograd.grad(_TORCH_ACT[case["act"]](z), z, dz)[0]
    o = dict(dx=torch.matmul(dz, s["w"]), dw=torch.matmul(dz.t(), s["x"]))
    if case["bias"]:
        o["dbias"] = dz.sum(dim=0)
    return o


_EXACT = dict(balance=_exact_balance, norm=_exact_norm, norm_bwd=_exact_norm_bwd, linear=_exact_linear,
              linear_bwd=_exact_linear_bwd)
