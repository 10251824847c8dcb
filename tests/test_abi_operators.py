"""Refusals of the operators around the layer, on the host: the C entry points return the documented
status before anything is queued, and the Python bindings check every tensor they are given.  No
test here launches a kernel."""
import ctypes
import os

import pytest
import torch

import grouped_gemm_top_amd as G

FAKE = 0x10000  # a non-NULL, 16-byte aligned address; never dereferenced by these calls
F = ctypes.c_void_p(FAKE)
ODD = ctypes.c_void_p(FAKE + 8)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(G.lib_path()):
        import grouped_gemm_top_amd.build as B
        B.build()
    return G.lib()


def test_add_rmsnorm_errors(L):
    def call(dt=G.MOE_BF16, rdt=G.MOE_BF16, x=F, res=F, w=F, eps=1e-6, N=4, H=64, h=F, y=ctypes.c_void_p(FAKE + 4096),
             q=None, sc=None):
        return L.moe_add_rmsnorm(dt, rdt, x, res, w, eps, N, H, h, y, q, sc, None)
    assert call(dt=7) == G.MOE_EUNSUPPORTED
    assert call(rdt=7) == G.MOE_EUNSUPPORTED
    assert call(dt=G.MOE_F32, rdt=G.MOE_BF16) == G.MOE_EUNSUPPORTED       # bf16 stream under fp32 activations
    assert call(N=-1) == G.MOE_EINVAL
    assert call(H=0) == G.MOE_EINVAL
    assert call(H=12) == G.MOE_EUNSUPPORTED
    assert call(H=16392) == G.MOE_EUNSUPPORTED
    assert call(H=40, q=F, sc=F) == G.MOE_EUNSUPPORTED                     # codes need H % 32
    assert call(q=F) == G.MOE_EINVAL                                       # codes without scales
    assert call(h=None, y=None) == G.MOE_EINVAL                            # no output
    assert call(x=None) == G.MOE_EINVAL
    assert call(eps=-1e-6) == G.MOE_EINVAL
    assert call(eps=float("nan")) == G.MOE_EINVAL
    assert call(eps=float("inf")) == G.MOE_EINVAL
    assert call(x=ODD) == G.MOE_EUNSUPPORTED
    assert call(w=ODD) == G.MOE_EUNSUPPORTED
    assert call(y=F) == G.MOE_EINVAL                                       # y over h
    assert call(rdt=G.MOE_F32) == G.MOE_EINVAL                             # h over an x of another type
    assert call(N=1 << 30, H=2048) == G.MOE_EUNSUPPORTED
    assert call(N=0, x=None) == G.MOE_OK                                   # nothing to do


def test_add_rmsnorm_bwd_errors(L):
    ptr = lambda k: ctypes.c_void_p(FAKE + 4096 * k)  # noqa: E731
    need = L.moe_workspace_bytes(G.OP_ADD_RMSNORM_BWD, G.MOE_BF16, 40, 1, 1, 64, 0, 0)
    assert need >= 64 * 4
    assert L.moe_workspace_bytes(G.OP_ADD_RMSNORM_BWD, G.MOE_BF16, 40, 1, 1, 60, 0, 0) == 0
    assert L.moe_workspace_bytes(G.OP_ADD_RMSNORM_BWD, 5, 40, 1, 1, 64, 0, 0) == 0

    def call(dt=G.MOE_BF16, rdt=G.MOE_BF16, dy=ptr(0), h=ptr(1), din=ptr(2), N=40, H=64, dh=ptr(3), dx=ptr(4),
             dw=ptr(5), ws=ptr(6), nb=need, eps=1e-6):
        return L.moe_add_rmsnorm_bwd(dt, rdt, dy, h, din, F, eps, N, H, dh, dx, dw, ws, nb, None)
    assert call(nb=need - 1) == G.MOE_EWORKSPACE
    assert call(ws=None) == G.MOE_EINVAL
    assert call(dy=None) == G.MOE_EINVAL
    assert call(dh=None) == G.MOE_EINVAL
    assert call(dh=ptr(1)) == G.MOE_EINVAL      # dh over h
    assert call(dx=ptr(3)) == G.MOE_EINVAL      # dx over dh
    assert call(dx=ptr(2)) == G.MOE_EINVAL      # dx over dh_in
    assert call(H=20) == G.MOE_EUNSUPPORTED
    assert call(dt=G.MOE_F32, rdt=G.MOE_BF16) == G.MOE_EUNSUPPORTED
    assert call(eps=float("nan")) == G.MOE_EINVAL
    assert call(dw=ODD) == G.MOE_EUNSUPPORTED


def test_add_rmsnorm_bindings():
    b, f = torch.bfloat16, torch.float32
    x, r, w = torch.zeros(4, 64, dtype=b), torch.zeros(4, 64, dtype=b), torch.zeros(64)
    with pytest.raises(ValueError, match="GPU"):
        G.add_rmsnorm(x, w, residual=r)
    with pytest.raises(TypeError):
        G.add_rmsnorm(x.half(), w)
    with pytest.raises(TypeError):
        G.add_rmsnorm(x, w.to(b))
    with pytest.raises(ValueError, match="shape"):
        G.add_rmsnorm(x, w, residual=r[:3])
    with pytest.raises(ValueError, match="shape"):
        G.add_rmsnorm(x, w[:8])
    with pytest.raises(ValueError, match="contiguous"):
        G.add_rmsnorm(torch.zeros(64, 4, dtype=b).t())
    with pytest.raises(ValueError, match="contiguous"):
        G.add_rmsnorm(x, w, residual=torch.zeros(4, 128, dtype=b)[:, ::2])
    with pytest.raises(ValueError):
        G.add_rmsnorm(x[0])
    with pytest.raises(ValueError, match="GPU"):
        G.add_rmsnorm_bwd(x, r, w)
    with pytest.raises(ValueError, match="shape"):
        G.add_rmsnorm_bwd(x, r, w, dh_in=r[:1])
    with pytest.raises(TypeError):
        G.add_rmsnorm_bwd(x, r.to(f), w, dh_in=r)


def test_balance_loss_errors(L):
    need = L.moe_workspace_bytes(G.OP_BALANCE_LOSS, G.MOE_F32, 64, 8, 2, 0, 3, 0)
    assert need > 0
    assert L.moe_workspace_bytes(G.OP_BALANCE_LOSS, G.MOE_F32, 64, 8, 2, 0, 0, 0) == 0
    assert L.moe_workspace_bytes(G.OP_BALANCE_LOSS, G.MOE_F32, 64, 8, 9, 0, 1, 0) == 0
    assert L.moe_workspace_bytes(G.OP_BALANCE_LOSS, G.MOE_F32, 0, 8, 2, 0, 1, 0) > 0

    def call(lg=F, idx=F, ptr=F, B=3, N=64, E=8, k=2, al=0.1, be=0.1, loss=F, cnt=F, sv=F, ws=F, nb=need):
        return L.moe_balance_loss(lg, None, idx, None, ptr, B, N, E, k, al, be, loss, cnt, sv, ws, nb, None)
    assert call(nb=need - 1) == G.MOE_EWORKSPACE
    assert call(ws=None) == G.MOE_EINVAL
    assert call(ws=ODD) == G.MOE_EUNSUPPORTED
    assert call(k=9) == G.MOE_EINVAL
    assert call(E=1025) == G.MOE_EINVAL
    assert call(N=-1) == G.MOE_EINVAL
    assert call(B=0) == G.MOE_EINVAL
    assert call(B=(1 << 20) + 1) == G.MOE_EINVAL
    assert call(ptr=None) == G.MOE_EINVAL       # three sequences without their ends
    assert call(lg=None) == G.MOE_EINVAL
    assert call(idx=None) == G.MOE_EINVAL
    assert call(loss=None) == G.MOE_EINVAL
    assert call(sv=None) == G.MOE_EINVAL
    assert call(al=float("nan")) == G.MOE_EINVAL
    assert call(be=float("inf")) == G.MOE_EINVAL

    def bwd(lg=F, ptr=F, B=3, N=64, E=8, sv=ctypes.c_void_p(FAKE + 4096), dl=ctypes.c_void_p(FAKE + 8192)):
        return L.moe_balance_loss_bwd(lg, None, None, ptr, B, N, E, sv, None, None, dl, None)
    assert bwd(lg=None) == G.MOE_EINVAL
    assert bwd(dl=None) == G.MOE_EINVAL
    assert bwd(dl=F) == G.MOE_EINVAL            # over the logits
    assert bwd(sv=None) == G.MOE_EINVAL
    assert bwd(B=0) == G.MOE_EINVAL
    assert bwd(ptr=None) == G.MOE_EINVAL
    assert bwd(E=0) == G.MOE_EINVAL
    assert bwd(N=0, lg=None, sv=None, dl=None) == G.MOE_OK


def test_balance_loss_bindings():
    lg, idx = torch.zeros(6, 8), torch.zeros(6, 2, dtype=torch.int32)
    ptr = torch.tensor([0, 6], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        G.balance_loss(lg, idx, 0.1, seq_ptr=ptr, mask=torch.ones(6, dtype=torch.bool))
    with pytest.raises(TypeError):
        G.balance_loss(lg.bfloat16(), idx, 0.1)
    with pytest.raises(TypeError):
        G.balance_loss(lg, idx.long(), 0.1)
    with pytest.raises(ValueError, match="shape"):
        G.balance_loss(lg, idx[:5], 0.1)
    with pytest.raises(ValueError, match="contiguous"):
        G.balance_loss(torch.zeros(8, 6).t(), idx, 0.1)
    with pytest.raises(TypeError):
        G.balance_loss(lg, idx, 0.1, mask=torch.ones(6))
    with pytest.raises(ValueError, match="shape"):
        G.balance_loss(lg, idx, 0.1, mask=torch.ones(5, dtype=torch.bool))
    with pytest.raises(TypeError):
        G.balance_loss(lg, idx, 0.1, seq_ptr=ptr.long())
    with pytest.raises(ValueError):
        G.balance_loss(lg, idx, 0.1, seq_ptr=ptr[:1])
    with pytest.raises(ValueError, match="shape"):
        G.balance_loss_bwd(lg, torch.zeros(8))
    with pytest.raises(TypeError):
        G.balance_loss_bwd(lg, torch.zeros(9), dloss=torch.ones(2, dtype=torch.float64))
    with pytest.raises(ValueError, match="GPU"):
        G.balance_loss_bwd(lg, torch.zeros(9))


def test_linear_errors(L):
    ptr = lambda k: ctypes.c_void_p(FAKE + 4096 * k)  # noqa: E731
    N, K, O = 100, 64, 72
    for op in (G.OP_LINEAR_FWD, G.OP_LINEAR_BWD):
        assert L.moe_workspace_bytes(op, G.MOE_F32, N, 1, 1, K, O, 0) > 6 * K * (N + O)   # the operands' parts
        assert L.moe_workspace_bytes(op, 7, N, 1, 1, K, O, 0) == 0
        assert L.moe_workspace_bytes(op, G.MOE_BF16, N, 1, 1, K, O, 0) > 0
        assert L.moe_workspace_bytes(op, G.MOE_BF16, 0, 1, 1, K, O, 0) > 0
        assert L.moe_workspace_bytes(op, G.MOE_BF16, N, 1, 1, 60, O, 0) == 0
        assert L.moe_workspace_bytes(op, G.MOE_BF16, N, 1, 1, K, 0, 0) == 0
    need = L.moe_workspace_bytes(G.OP_LINEAR_FWD, G.MOE_BF16, N, 1, 1, K, O, 0)

    def fwd(dt=G.MOE_BF16, x=ptr(0), w=ptr(1), b=ptr(2), act=0, res=ptr(3), N=N, K=K, O=O, out=ptr(4), z=ptr(5), ws=ptr(6), nb=need):
        return L.moe_linear_fwd(dt, x, w, b, act, res, N, K, O, out, z, ws, nb, None)
    assert fwd(nb=need - 1) == G.MOE_EWORKSPACE
    assert fwd(ws=None) == G.MOE_EINVAL
    assert fwd(dt=2) == G.MOE_EUNSUPPORTED
    assert fwd(dt=G.MOE_F32) == G.MOE_EWORKSPACE              # bf16's workspace is too small
    assert fwd(dt=G.MOE_F32, N=1 << 19, K=1024) == G.MOE_EUNSUPPORTED   # x's parts of more than 2 GiB
    assert fwd(act=5) == G.MOE_EINVAL
    assert fwd(act=-1) == G.MOE_EINVAL
    assert fwd(K=60) == G.MOE_EUNSUPPORTED
    assert fwd(O=4) == G.MOE_EINVAL
    assert fwd(O=76) == G.MOE_EUNSUPPORTED
    assert fwd(N=-1) == G.MOE_EINVAL
    assert fwd(N=1 << 20, K=1024) == G.MOE_EUNSUPPORTED       # x of 2 GiB
    assert fwd(N=1 << 20, O=1024) == G.MOE_EUNSUPPORTED       # out of 2 GiB
    assert fwd(K=1 << 15, O=1 << 15) == G.MOE_EUNSUPPORTED    # w of 2 GiB
    assert fwd(x=None) == G.MOE_EINVAL
    assert fwd(w=None) == G.MOE_EINVAL
    assert fwd(out=None) == G.MOE_EINVAL
    assert fwd(out=ptr(0)) == G.MOE_EINVAL                    # out over x
    assert fwd(z=ptr(4)) == G.MOE_EINVAL                      # z over out
    assert fwd(z=ptr(3)) == G.MOE_EINVAL                      # z over the residual
    assert fwd(b=ODD) == G.MOE_EUNSUPPORTED
    assert fwd(x=None, out=None, N=0) == G.MOE_OK
    need = L.moe_workspace_bytes(G.OP_LINEAR_BWD, G.MOE_BF16, N, 1, 1, K, O, 0)

    def bwd(dt=G.MOE_BF16, d=ptr(0), x=ptr(1), w=ptr(2), z=ptr(3), act=2, N=N, K=K, O=O, dx=ptr(4), dw=ptr(5), db=ptr(6), ws=ptr(7),
            nb=need):
        return L.moe_linear_bwd(dt, d, x, w, z, act, N, K, O, dx, dw, db, ws, nb, None)
    assert bwd(nb=need - 1) == G.MOE_EWORKSPACE
    assert bwd(z=None) == G.MOE_EINVAL
    assert bwd(dx=None, dw=None, db=None) == G.MOE_EINVAL
    assert bwd(d=None) == G.MOE_EINVAL
    assert bwd(w=None) == G.MOE_EINVAL
    assert bwd(x=None) == G.MOE_EINVAL
    assert bwd(dx=ptr(0)) == G.MOE_EINVAL                     # dx over dout
    assert bwd(dw=ptr(4)) == G.MOE_EINVAL                     # dw over dx
    assert bwd(act=9) == G.MOE_EINVAL
    assert bwd(db=ODD) == G.MOE_EUNSUPPORTED


def test_linear_bindings():
    b = torch.bfloat16
    x, w, d = torch.zeros(4, 64, dtype=b), torch.zeros(24, 64, dtype=b), torch.zeros(4, 24, dtype=b)
    with pytest.raises(ValueError, match="GPU"):
        G.linear_fwd(x, w, bias=torch.zeros(24), residual=d, act="silu")
    with pytest.raises(TypeError):
        G.linear_fwd(x.float(), w)
    with pytest.raises(TypeError):
        G.linear_fwd(x.half(), w.half())
    with pytest.raises(TypeError):
        G.linear_fwd(x, w, bias=torch.zeros(24, dtype=b))
    with pytest.raises(ValueError, match="shape"):
        G.linear_fwd(x, w[:, :32])
    with pytest.raises(ValueError, match="shape"):
        G.linear_fwd(x, w, residual=x)
    with pytest.raises(ValueError, match="contiguous"):
        G.linear_fwd(x, torch.zeros(64, 24, dtype=b).t())
    with pytest.raises(ValueError, match="act"):
        G.linear_fwd(x, w, act="tanh")
    with pytest.raises(ValueError, match="needs z"):
        G.linear_bwd(d, x, w, act="gelu")
    with pytest.raises(ValueError, match="shape"):
        G.linear_bwd(d[:3], x, w)
    with pytest.raises(ValueError, match="GPU"):
        G.linear_bwd(d, x, w)


def test_bindings_take_every_argument_by_name():
    """The documented names work for the first argument too (a host tensor reaches the binding's own refusal)."""
    b, f = torch.bfloat16, torch.float32
    x, w = torch.zeros(4, 64, dtype=b), torch.zeros(32, 64, dtype=b)
    lg, ix, sv = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(9, dtype=f)
    for call in (lambda: G.add_rmsnorm(x=x), lambda: G.add_rmsnorm_bwd(dy=x, h=x), lambda: G.linear_fwd(w=w, x=x),
                 lambda: G.linear_bwd(dout=torch.zeros(4, 32, dtype=b), x=x, w=w),
                 lambda: G.balance_loss(logits=lg, topk_idx=ix, alpha=0.1), lambda: G.balance_loss_bwd(logits=lg, saved=sv)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        G.linear_fwd()


def test_balance_loss_sequences_times_experts(L):
    """B ceil(E / 64) workgroups of 1024 threads are one launch: refused from 2^32 threads on."""
    big = 1 << 20
    ok = L.moe_workspace_bytes(G.OP_BALANCE_LOSS, G.MOE_F32, 64, 192, 2, 0, big, 0)
    assert ok > 0
    assert L.moe_workspace_bytes(G.OP_BALANCE_LOSS, G.MOE_F32, 64, 193, 2, 0, big, 0) == 0
    assert L.moe_balance_loss(F, None, F, None, F, big, 64, 256, 2, 0.1, 0.1, F, F, F, F, 1 << 62, None) == G.MOE_EUNSUPPORTED
    assert L.moe_balance_loss_bwd(F, None, None, F, big, 64, 256, F, None, None, F, None) == G.MOE_EUNSUPPORTED


def test_linear_widest_output(L):
    """ceil(O / 16) workgroups of 512 threads are one launch: an O near 2^27 is refused, for both directions."""
    for op in (G.OP_LINEAR_FWD, G.OP_LINEAR_BWD):
        assert L.moe_workspace_bytes(op, G.MOE_BF16, 1, 1, 1, 8, 1 << 26, 0) > 0
        assert L.moe_workspace_bytes(op, G.MOE_BF16, 1, 1, 1, 8, (1 << 27) - 8, 0) == 0
    assert L.moe_linear_fwd(G.MOE_BF16, F, F, None, 0, None, 1, 8, (1 << 27) - 8, ctypes.c_void_p(FAKE + 4096), None, F,
                            1 << 62, None) == G.MOE_EUNSUPPORTED


def test_norm_backward_workspace_for_as_many_rows_as_the_call_takes(L):
    """N H below 2^40 is what bounds the norm: the workspace query answers wherever the call accepts the sizes."""
    for N, H in ((1 << 30, 8), ((1 << 31) - 1, 8), ((1 << 31) - 1, 504), (1 << 26, 16376)):
        need = L.moe_workspace_bytes(G.OP_ADD_RMSNORM_BWD, G.MOE_BF16, N, 1, 1, H, 0, 0)
        assert need >= H * 4, (N, H)
        st = L.moe_add_rmsnorm_bwd(G.MOE_BF16, G.MOE_BF16, F, ctypes.c_void_p(FAKE + 4096), None, None, 1e-6, N, H,
                                   ctypes.c_void_p(FAKE + 8192), None, F, F, need - 1, None)
        assert st == G.MOE_EWORKSPACE
    assert L.moe_workspace_bytes(G.OP_ADD_RMSNORM_BWD, G.MOE_BF16, 1 << 27, 1, 1, 8192, 0, 0) == 0   # N H = 2^40
    assert L.moe_workspace_bytes(G.OP_ADD_RMSNORM_BWD, G.MOE_BF16, -1, 1, 1, 64, 0, 0) == 0
