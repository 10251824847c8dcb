"""Refusals of the layer's few-token and 8-bit checkpoint forms and of the cross entropy, on the host: the C entry
points return the documented status before anything is queued, and the Python bindings check every tensor
they are given.  No test here launches a kernel."""
import ctypes
import os

import pytest
import torch

import grouped_gemm_top_amd as G

FAKE = 0x10000  # a non-NULL, 16-byte aligned address; never dereferenced by these calls
ODD = ctypes.c_void_p(FAKE + 8)


def ptr(k):
    return ctypes.c_void_p(FAKE + 4096 * k)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(G.lib_path()):
        import grouped_gemm_top_amd.build as B
        B.build()
    return G.lib()


def test_linear_ce_fwd_errors(L):
    need = L.moe_workspace_bytes(G.OP_LINEAR_CE_FWD, G.MOE_BF16, 40, 1, 1, 64, 101, 0)
    assert need > 0

    def call(dt=G.MOE_BF16, x=ptr(1), w=ptr(2), t=ptr(3), N=40, H=64, V=101, zc=0.0, loss=ptr(4), lse=ptr(5), ws=ptr(6),
             nb=need):
        return L.moe_linear_ce_fwd(dt, x, w, t, N, H, V, zc, loss, lse, ws, nb, None)
    assert call(dt=3) == G.MOE_EUNSUPPORTED
    assert call(N=-1) == G.MOE_EINVAL
    assert call(H=0) == G.MOE_EINVAL
    assert call(V=0) == G.MOE_EINVAL
    assert call(H=12) == G.MOE_EUNSUPPORTED
    assert call(zc=float("nan")) == G.MOE_EINVAL
    assert call(zc=float("inf")) == G.MOE_EINVAL
    for n in ("x", "w", "t", "loss", "lse", "ws"):
        assert call(**{n: None}) == G.MOE_EINVAL, n
    for n in ("x", "w", "ws"):
        assert call(**{n: ODD}) == G.MOE_EUNSUPPORTED, n
    for n in ("t", "loss", "lse"):
        assert call(**{n: ctypes.c_void_p(FAKE + 2)}) == G.MOE_EUNSUPPORTED, n
    assert call(lse=ptr(4)) == G.MOE_EINVAL             # lse over loss
    assert call(loss=ptr(3)) == G.MOE_EINVAL            # loss over targets
    assert call(nb=need - 1) == G.MOE_EWORKSPACE
    assert call(N=1 << 23) == G.MOE_EUNSUPPORTED        # 256 columns of dz past 2 GiB
    assert call(dt=G.MOE_F32, N=1 << 21) == G.MOE_EUNSUPPORTED
    assert call(N=1 << 20, V=1 << 17) == G.MOE_EUNSUPPORTED
    assert call(H=1 << 23, V=8) == G.MOE_EUNSUPPORTED
    assert call(N=0, x=None, t=None, loss=None, lse=None) == G.MOE_OK


def test_linear_ce_bwd_errors(L):
    need = L.moe_workspace_bytes(G.OP_LINEAR_CE_BWD, G.MOE_BF16, 40, 1, 1, 64, 101, 0)
    assert need > 0
    assert L.moe_workspace_bytes(G.OP_LINEAR_CE_BWD, G.MOE_BF16, 40, 1, 1, 60, 101, 0) == 0
    assert L.moe_workspace_bytes(G.OP_LINEAR_CE_BWD, 9, 40, 1, 1, 64, 101, 0) == 0

    def call(dt=G.MOE_BF16, g=ptr(0), x=ptr(1), w=ptr(2), t=ptr(3), lse=ptr(4), N=40, H=64, V=101, zc=0.0, dx=ptr(5),
             dw=ptr(6), ws=ptr(7), nb=need):
        return L.moe_linear_ce_bwd(dt, g, x, w, t, lse, N, H, V, zc, dx, dw, ws, nb, None)
    assert call(dt=3) == G.MOE_EUNSUPPORTED
    assert call(N=-1) == G.MOE_EINVAL
    assert call(V=0) == G.MOE_EINVAL
    assert call(H=20) == G.MOE_EUNSUPPORTED
    assert call(zc=float("nan")) == G.MOE_EINVAL
    assert call(dx=None, dw=None) == G.MOE_EINVAL
    for n in ("x", "w", "t", "lse", "ws"):
        assert call(**{n: None}) == G.MOE_EINVAL, n
    for n in ("x", "w", "dx", "dw", "ws"):
        assert call(**{n: ODD}) == G.MOE_EUNSUPPORTED, n
    for n in ("t", "lse", "g"):
        assert call(**{n: ctypes.c_void_p(FAKE + 2)}) == G.MOE_EUNSUPPORTED, n
    assert call(dx=ptr(1)) == G.MOE_EINVAL              # dx over x
    assert call(dw=ptr(2)) == G.MOE_EINVAL              # dw over w
    assert call(dw=ptr(5)) == G.MOE_EINVAL              # dw over dx
    assert call(nb=need - 1) == G.MOE_EWORKSPACE
    assert call(N=1 << 23) == G.MOE_EUNSUPPORTED


def test_linear_ce_bindings():
    b, f, i = torch.bfloat16, torch.float32, torch.int32
    x, w, t, g = torch.zeros(4, 64, dtype=b), torch.zeros(9, 64, dtype=b), torch.zeros(4, dtype=i), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        G.linear_ce_fwd(x, w, t)
    with pytest.raises(ValueError, match="GPU"):
        G.linear_ce_bwd(g, x, w, t, g)
    with pytest.raises(TypeError):
        G.linear_ce_fwd(x, w, t.long())
    with pytest.raises(TypeError):
        G.linear_ce_fwd(x, w.float(), t)
    with pytest.raises(TypeError):
        G.linear_ce_fwd(x.half(), w.half(), t)
    with pytest.raises(ValueError):
        G.linear_ce_fwd(x, w[:, :32].contiguous(), t)
    with pytest.raises(ValueError):
        G.linear_ce_fwd(x, w, t[:3])
    with pytest.raises(ValueError, match="contiguous"):
        G.linear_ce_fwd(torch.zeros(4, 128, dtype=b)[:, ::2], w, t)
    with pytest.raises(ValueError):
        G.linear_ce_fwd(x[0], w, t)
    with pytest.raises(ValueError):
        G.linear_ce_bwd(g[:2], x, w, t, g)
    with pytest.raises(TypeError):
        G.linear_ce_bwd(g.to(b), x, w, t, g)
    with pytest.raises(TypeError):
        G.linear_ce_bwd(g, x, w, t, g.to(b))


def _plan(N=16, E=4, k=2, kind=G.PLAN_TOPK, mtile=0, **null):
    cap = G.plan_rows_cap(kind, N, E, k, mtile)
    f = dict(counts=FAKE, offsets=FAKE, row_token=FAKE, row_w=FAKE, row_pair=FAKE, tok_ptr=FAKE, tok_rows=FAKE)
    f.update(null)
    return G.CPlan(kind, N, E, k, cap, mtile, *f.values())


def test_fwd_ckpt8_errors(L):
    p = _plan()
    need = L.moe_workspace_bytes(G.OP_GEMM_FWD, G.MOE_BF16, 16, 4, 2, 64, 96, p.M_cap)

    def call(x=ptr(1), wg=ptr(2), wu=ptr(3), wd=ptr(4), H=64, I=96, plan=p, hq=ptr(5), hs=ptr(6), y=ptr(7), ws=ptr(8),
             nb=need):
        return L.moe_grouped_gemm_fwd_ckpt8(x, wg, wu, wd, H, I, None if plan is None else ctypes.byref(plan), hq, hs, y,
                                            ws, nb, None)
    assert call(I=0) == G.MOE_EINVAL
    assert call(H=12) == G.MOE_EUNSUPPORTED
    assert call(I=72) == G.MOE_EUNSUPPORTED             # blocks of 32
    assert call(plan=None) == G.MOE_EINVAL
    assert call(plan=_plan(counts=0)) == G.MOE_EINVAL
    for n in ("x", "wg", "wu", "wd", "hq", "hs", "y", "ws"):
        assert call(**{n: None}) == G.MOE_EINVAL, n
    for n in ("x", "wg", "wu", "wd", "hq", "y", "ws"):
        assert call(**{n: ODD}) == G.MOE_EUNSUPPORTED, n
    assert call(hs=ctypes.c_void_p(FAKE + 2)) == G.MOE_EUNSUPPORTED
    assert call(nb=need - 1) == G.MOE_EWORKSPACE
    big = _plan(N=1 << 20)
    assert call(plan=big, H=1024) == G.MOE_EUNSUPPORTED  # x of 2 GiB


def test_bwd_ckpt8_errors(L):
    p = _plan()
    need = L.moe_workspace_bytes(G.OP_LAYER_BWD_CKPT8, G.MOE_BF16, 16, 4, 2, 64, 96, p.M_cap)
    assert need > L.moe_workspace_bytes(G.OP_LAYER_BWD, G.MOE_BF16, 16, 4, 2, 64, 96, p.M_cap)
    assert L.moe_workspace_bytes(G.OP_LAYER_BWD_CKPT8, G.MOE_BF16, 16, 4, 2, 64, 72, p.M_cap) == 0
    assert L.moe_workspace_bytes(G.OP_LAYER_BWD_CKPT8, G.MOE_BF16, 16, 4, 2, 60, 96, p.M_cap) == 0

    def call(dout=ptr(0), x=ptr(1), xs=None, wg=ptr(2), wu=ptr(3), wd=ptr(4), H=64, I=96, plan=p, hq=ptr(5), hs=ptr(6),
             dx=ptr(7), dwg=ptr(8), dwu=ptr(9), dwd=ptr(10), ds=ptr(11), ws=ptr(12), nb=need):
        return L.moe_layer_bwd_ckpt8(dout, x, xs, wg, wu, wd, H, I, None if plan is None else ctypes.byref(plan), hq, hs,
                                     dx, dwg, dwu, dwd, ds, ws, nb, None)
    assert call(I=72) == G.MOE_EUNSUPPORTED
    assert call(H=72, xs=ptr(13)) == G.MOE_EUNSUPPORTED  # x as codes needs H % 32
    assert call(plan=None) == G.MOE_EINVAL
    for n in ("dout", "x", "wg", "wu", "wd", "hq", "hs", "dx", "dwg", "dwu", "dwd", "ds", "ws"):
        assert call(**{n: None}) == G.MOE_EINVAL, n
    for n in ("dout", "x", "wg", "wu", "wd", "hq", "dx", "dwg", "dwu", "dwd", "ws"):
        assert call(**{n: ODD}) == G.MOE_EUNSUPPORTED, n
    assert call(nb=need - 1) == G.MOE_EWORKSPACE


def test_dequantize_errors(L):
    def call(dt=G.MOE_BF16, q=ptr(1), s=ptr(2), rows=4, K=64, out=ptr(3)):
        return L.moe_dequantize_mxfp8(dt, q, s, rows, K, out, None)
    assert call(dt=5) == G.MOE_EUNSUPPORTED
    assert call(rows=-1) == G.MOE_EINVAL
    assert call(K=48) == G.MOE_EUNSUPPORTED
    assert call(K=0) == G.MOE_EUNSUPPORTED
    for n in ("q", "s", "out"):
        assert call(**{n: None}) == G.MOE_EINVAL, n
    assert call(q=ODD) == G.MOE_EUNSUPPORTED
    assert call(out=ODD) == G.MOE_EUNSUPPORTED
    assert call(rows=1 << 40) == G.MOE_EINVAL
    assert call(rows=0, q=None, s=None, out=None) == G.MOE_OK


def test_ckpt8_bindings():
    b, u = torch.bfloat16, torch.uint8
    plan = G.Plan(4, 3, 2, device="cpu")
    x, wg, wd = torch.zeros(4, 64, dtype=b), torch.zeros(3, 32, 64, dtype=b), torch.zeros(3, 64, 32, dtype=b)
    hq, hs = torch.zeros(8, 64, dtype=u), torch.zeros(8, 8, dtype=u)
    xq, xs = torch.zeros(4, 64, dtype=u), torch.zeros(4, 4, dtype=u)

    def fwd(x=x, wg=wg, wu=wg, wd=wd, plan=plan, **kw):
        return G.grouped_gemm_fwd_ckpt8(x, wg, wu, wd, plan, **kw)

    def bwd(dout=x, x=x, wg=wg, wu=wg, wd=wd, plan=plan, h=(hq, hs), **kw):
        return G.layer_bwd_ckpt8(dout, x, wg, wu, wd, plan, h, **kw)
    for f in (fwd, bwd):
        with pytest.raises(ValueError, match="GPU"):
            f()
        with pytest.raises(TypeError):
            f(x=x.float())
        with pytest.raises(TypeError):
            f(wd=wd.float())
        with pytest.raises(ValueError):
            f(x=x[:3])
        with pytest.raises(ValueError):
            f(wu=wg[:2])
        with pytest.raises(ValueError):
            f(wg=wg[0])
        with pytest.raises(ValueError, match="experts"):
            f(plan=G.Plan(4, 4, 2, device="cpu"))
        with pytest.raises(ValueError, match="contiguous"):
            f(x=torch.zeros(4, 128, dtype=b)[:, ::2])
    with pytest.raises(ValueError, match="GPU"):
        bwd(x=(xq, xs))
    with pytest.raises(TypeError):
        bwd(x=(x, xs))
    with pytest.raises(ValueError):
        bwd(x=(xq, xs[:, :2]))
    with pytest.raises(ValueError):
        bwd(h=(hq[:7], hs))
    with pytest.raises(ValueError):
        bwd(h=(hq, hs[:, :4].contiguous()))
    with pytest.raises(TypeError):
        bwd(h=(hq.to(b), hs))
    with pytest.raises(ValueError, match="GPU"):
        G.dequantize_mxfp8(xq, xs)
    with pytest.raises(TypeError):
        G.dequantize_mxfp8(x, xs)
    with pytest.raises(ValueError):
        G.dequantize_mxfp8(xq, xs[:, :3].contiguous())


def test_layer_few_errors(L):
    need = L.moe_workspace_bytes(G.OP_LAYER_FEW, G.MOE_BF16, 16, 8, 2, 64, 96, 0)
    assert need > 0 and L.moe_workspace_bytes(G.OP_LAYER_FEW, G.MOE_BF16, 0, 8, 2, 64, 96, 0) > 0
    assert L.moe_workspace_bytes(G.OP_LAYER_FEW, G.MOE_BF16, 65, 8, 2, 64, 96, 0) == 0

    def call(dt=G.MOE_BF16, x=ptr(1), wr=ptr(2), b=None, wg=ptr(3), wu=ptr(4), wd=ptr(5), N=16, H=64, I=96, E=8, k=2,
             out=ptr(6), idx=ptr(7), w=ptr(8), ws=ptr(9), nb=need, sc=None):
        if sc is None:
            return L.moe_layer_few(dt, x, wr, b, wg, wu, wd, N, H, I, E, k, out, idx, w, ws, nb, None)
        return L.moe_layer_few_mxfp8(x, wr, b, wg, sc, wu, sc, wd, sc, N, H, I, E, k, out, idx, w, ws, nb, None)
    assert call(dt=4) == G.MOE_EUNSUPPORTED
    for sc in (None, ptr(10)):
        f = lambda **kw: call(sc=sc, **kw)  # noqa: E731,B023
        assert f(N=-1) == G.MOE_EINVAL
        assert f(N=65) == G.MOE_EUNSUPPORTED
        assert f(E=0) == G.MOE_EINVAL
        assert f(E=1025) == G.MOE_EINVAL
        assert f(k=0) == G.MOE_EINVAL
        assert f(k=9) == G.MOE_EINVAL
        assert f(E=64, k=33) == G.MOE_EUNSUPPORTED
        assert f(H=0) == G.MOE_EINVAL
        assert f(I=100) == G.MOE_EUNSUPPORTED
        assert f(H=1 << 21) == G.MOE_EUNSUPPORTED
        for n in ("x", "wr", "wg", "wu", "wd", "out", "idx", "w", "ws"):
            assert f(**{n: None}) == G.MOE_EINVAL, n
        for n in ("x", "wg", "wu", "wd", "out", "ws"):
            assert f(**{n: ODD}) == G.MOE_EUNSUPPORTED, n
        for n in ("wr", "b", "idx", "w"):
            assert f(**{n: ctypes.c_void_p(FAKE + 2)}) == G.MOE_EUNSUPPORTED, n
        assert f(out=ptr(1)) == G.MOE_EINVAL        # out over x
        assert f(idx=ptr(8)) == G.MOE_EINVAL        # topk_idx over topk_w
        assert f(nb=need - 1) == G.MOE_EWORKSPACE
        assert f(N=0, x=None, out=None, idx=None, w=None) == G.MOE_OK
    assert call(sc=ptr(10), I=104, H=64) == G.MOE_EUNSUPPORTED    # codes: multiples of 32
    assert call(sc=ctypes.c_void_p(FAKE + 2)) == G.MOE_EUNSUPPORTED
    assert L.moe_layer_few_mxfp8(ptr(1), ptr(2), None, ptr(3), None, ptr(4), ptr(10), ptr(5), ptr(10), 16, 64, 96, 8, 2,
                                 ptr(6), ptr(7), ptr(8), ptr(9), need, None) == G.MOE_EINVAL


def test_layer_few_bindings():
    b, u = torch.bfloat16, torch.uint8
    x, wr = torch.zeros(4, 64, dtype=b), torch.zeros(64, 3)
    wg, wd = torch.zeros(3, 32, 64, dtype=b), torch.zeros(3, 64, 32, dtype=b)
    gq, dq = (torch.zeros(3, 32, 64, dtype=u), torch.zeros(3, 32, 4, dtype=u)), (torch.zeros(3, 64, 32, dtype=u),
                                                                              torch.zeros(3, 64, 4, dtype=u))

    def call(x=x, wr=wr, wg=wg, wu=wg, wd=wd, k=2, **kw):
        return G.layer_few(x, wr, wg, wu, wd, k, **kw)
    with pytest.raises(ValueError, match="GPU"):
        call()
    with pytest.raises(ValueError, match="GPU"):
        call(wg=gq, wu=gq, wd=dq)
    with pytest.raises(ValueError, match="all"):
        call(wg=gq)
    with pytest.raises(TypeError):
        call(x=x.float(), wg=gq, wu=gq, wd=dq)
    with pytest.raises(TypeError):
        call(x=x.float())
    with pytest.raises(TypeError):
        call(wr=wr.to(b))
    with pytest.raises(ValueError):
        call(wr=wr[:, :2].contiguous())
    with pytest.raises(ValueError):
        call(bias=torch.zeros(4))
    with pytest.raises(ValueError):
        call(wd=wg)
    with pytest.raises(ValueError):
        call(wg=gq, wu=gq, wd=(dq[0], dq[1][:, :, :2].contiguous()))
    with pytest.raises(ValueError):
        call(x=x[0])
    with pytest.raises(ValueError, match="contiguous"):
        call(x=torch.zeros(4, 128, dtype=b)[:, ::2])


def test_linear_ce_largest_vocabulary(L):
    """Columns are counted in 32 bits: V up to 2^30, whatever memory there is."""
    for op in (G.OP_LINEAR_CE_FWD, G.OP_LINEAR_CE_BWD):
        assert L.moe_workspace_bytes(op, G.MOE_BF16, 1, 1, 1, 8, 1 << 30, 0) > 0
        assert L.moe_workspace_bytes(op, G.MOE_BF16, 1, 1, 1, 8, (1 << 30) + 1, 0) == 0
    big = 1 << 62
    assert L.moe_linear_ce_fwd(G.MOE_BF16, ptr(1), ptr(2), ptr(3), 1, 8, (1 << 31) - 1, 0.0, ptr(4), ptr(5), ptr(6), big,
                               None) == G.MOE_EUNSUPPORTED
    assert L.moe_linear_ce_bwd(G.MOE_BF16, None, ptr(1), ptr(2), ptr(3), ptr(4), 1, 8, (1 << 31) - 1, 0.0, ptr(5), ptr(7),
                               ptr(6), big, None) == G.MOE_EUNSUPPORTED


def test_layer_few_codes_come_in_pairs():
    """MX-FP8 weights are (codes, scale codes): anything longer or shorter is refused, not passed on argument by argument."""
    b, u = torch.bfloat16, torch.uint8
    x, wr = torch.zeros(4, 64, dtype=b), torch.zeros(64, 3)
    gq, dq = [torch.zeros(3, 32, 64, dtype=u), torch.zeros(3, 32, 4, dtype=u)], [torch.zeros(3, 64, 32, dtype=u),
                                                                              torch.zeros(3, 64, 4, dtype=u)]
    for n in range(3):
        for m in ([], [0], [0, 1, 1]):
            w = [gq, gq, dq]
            w[n] = tuple(w[n][i] for i in m)
            with pytest.raises(ValueError, match=r"\(codes, scale codes\)"):
                G.layer_few(x, wr, *w, 2)
    with pytest.raises(ValueError, match="GPU"):  # a list is a pair too
        G.layer_few(x, wr, gq, gq, dq, 2)


def test_outputs_are_no_other_argument(L):
    """Every output of the calls that say so, over every other argument (an output written early would be read as input)."""
    q = G.workspace_bytes

    def few(a, sc):
        nb = q(G.OP_LAYER_FEW, G.MOE_BF16, 16, 8, 2, 64, 96)
        size = (16, 64, 96, 8, 2)
        if sc:
            return L.moe_layer_few_mxfp8(a["x"], a["wr"], a["b"], a["wg"], a["gs"], a["wu"], a["us"], a["wd"], a["ds"], *size,
                                         a["out"], a["idx"], a["w"], a["ws"], nb, None)
        return L.moe_layer_few(G.MOE_BF16, a["x"], a["wr"], a["b"], a["wg"], a["wu"], a["wd"], *size, a["out"], a["idx"],
                               a["w"], a["ws"], nb, None)

    def fwd(a):
        nb = q(G.OP_LINEAR_CE_FWD, G.MOE_F32, 40, 1, 1, 64, 101)
        return L.moe_linear_ce_fwd(G.MOE_F32, a["x"], a["w"], a["t"], 40, 64, 101, 0.0, a["loss"], a["lse"], a["ws"], nb, None)

    def bwd(a):
        nb = q(G.OP_LINEAR_CE_BWD, G.MOE_F32, 40, 1, 1, 64, 101)
        return L.moe_linear_ce_bwd(G.MOE_F32, a["g"], a["x"], a["w"], a["t"], a["lse"], 40, 64, 101, 0.0, a["dx"], a["dw"],
                                   a["ws"], nb, None)
    for call, ins, outs in ((lambda a: few(a, False), ("x", "wr", "b", "wg", "wu", "wd", "ws"), ("out", "idx", "w")),
                            (lambda a: few(a, True), ("x", "wr", "b", "wg", "gs", "wu", "us", "wd", "ds", "ws"), ("out", "idx", "w")),
                            (fwd, ("x", "w", "t", "ws"), ("loss", "lse")), (bwd, ("g", "x", "w", "t", "lse", "ws"), ("dx", "dw"))):
        every = {n: ptr(i + 1) for i, n in enumerate(ins + outs)}
        for o in outs:
            for n in every:
                if n != o:
                    assert call(dict(every, **{o: every[n]})) == G.MOE_EINVAL, (o, n)
    # no token: dw is still written
    nb = q(G.OP_LINEAR_CE_BWD, G.MOE_F32, 0, 1, 1, 64, 101)
    assert L.moe_linear_ce_bwd(G.MOE_F32, None, None, ptr(1), None, None, 0, 64, 101, 0.0, None, ptr(1), ptr(2), nb,
                               None) == G.MOE_EINVAL


def test_linear_ce_bwd_without_dloss():
    """None stands for ones, as NULL does in C; the tensors' device is x's."""
    x, w, t, l = torch.zeros(4, 64), torch.zeros(9, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        G.linear_ce_bwd(None, x, w, t, l)
    with pytest.raises(ValueError, match="GPU"):
        G.linear_ce_bwd(dloss=None, x=x, w=w, targets=t, lse=l)
    with pytest.raises(TypeError, match="needs x"):
        G.linear_ce_bwd(l, None, w, t, l)
