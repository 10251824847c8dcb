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
