"""Which kernels the dense products run on, and whole-number parity on each of them.

`choose` below restates the library's choice of tile and K slices (linear.hip); the host test holds
it against the library's own workspace sizes, which contain the partial sums of that choice.  With
it the GPU cases here and in test_gpu_linear.py are shown to reach every kernel: three products,
each tile, with and without K slices, in both types.  Whole numbers make every sum exact, so outputs
must equal the exact results rounded once."""
import os
import random

import pytest
import torch

import grouped_gemm_top_amd as G
import test_gpu_linear as TL

BF, F32 = TL.BF, TL.F32


def choose(kind, M, N, K, f32):
    """(tile, slices): tile 2 is 256 x 256, 1 128 x 128, 0 64 x 64 (64 x 128 for dx)."""
    steps = (6 if f32 else 1) * ((K + 63) // 64)
    tiles = [(64, 64, 3, 3.0, 0.23, 0.26) if kind == "fwd" else (64, 128, 2, 3.0, 0.32, 0.47),
             (128, 128, 2, 3.1, 0.75, 0.49), (256, 256, 1, 6.4, 0.40, 1.20)]
    best, least = (1, 1), 1e30
    for b in range(1 if kind == "dw" else 0, 3):
        bm, bn, occ, fix, lat, thr = tiles[b]
        n = -(-M // bm) * -(-N // bn)
        for S in (1, 2, 4, 8, 16):
            if S > steps or (S > 1 and S * M * N > 64e6):
                break
            per_cu = (n * S + 255) // 256
            t = 2.5 + -(-per_cu // occ) * fix + (steps + S - 1) // S * max(thr * per_cu, lat)
            if S > 1:
                t += 2.2 + 2.3e-6 * (S * M * N)
            if t < least:
                best, least = (b, S), t
    return best


def few(f32, N, K):
    return N <= 16 or (N <= 32 and (f32 or K <= 2048))


def kernels(N, K, O, f32):
    """The kernels of a forward and a backward: (product, tile, sliced)."""
    r = set()
    if few(f32, N, K):
        r.add(("fwd", "few", N > 16))
    else:
        b, S = choose("fwd", N, O, K, f32)
        r.add(("fwd", b, S > 1))
    for kind, dims in (("dx", (N, K, O)), ("dw", (O, K, N))):
        b, S = choose(kind, *dims, f32)
        r.add((kind, b, S > 1))
    return r


# N, K, O: what test_gpu_linear.py's shapes leave out (bf16, fp32, both)
MORE = {BF: [(8475, 136, 72), (7485, 152, 4968), (9061, 152, 3304), (2175, 4440, 72), (9187, 5272, 136)],
        F32: [(139, 1672, 4344), (8475, 136, 72)]}
BOTH = [(5, 1096, 7448)]


def _up(n):
    return (n + 255) // 256 * 256


def test_choice_is_the_librarys():
    """Workspace sizes over random shapes: they hold the partial sums of the choice restated above."""
    if not os.path.exists(G.lib_path()):
        import grouped_gemm_top_amd.build as B
        B.build()
    rng = random.Random(3)
    for _ in range(400):
        N, K, O = int(10 ** rng.uniform(0, 4.2)), 8 * int(10 ** rng.uniform(0, 3)), 8 * int(10 ** rng.uniform(0, 3))
        f32 = rng.random() < 0.5
        dt = G.MOE_F32 if f32 else G.MOE_BF16
        part = {}
        for kind, (m, n, k) in (("fwd", (N, O, K)), ("dx", (N, K, O)), ("dw", (O, K, N))):
            S = choose(kind, m, n, k, f32)[1]
            part[kind] = _up(S * m * n * 4) if S > 1 else 0
        ops = _up(N * K * 6) + _up(O * K * 6) if f32 else 0
        want = 256 if few(f32, N, K) else 256 + ops + part["fwd"]
        assert G.workspace_bytes(G.OP_LINEAR_FWD, dt, N, 1, 1, K, O) == want, (N, K, O, f32)
        groups = 1 if N <= 64 else (128 if N >= 2048 else (N + 15) // 16)
        want = 256 + _up(N * O * (6 if f32 else 2)) + _up(groups * O * 4) + ops + max(part["dx"], part["dw"])
        assert G.workspace_bytes(G.OP_LINEAR_BWD, dt, N, 1, 1, K, O) == want, (N, K, O, f32)


@pytest.mark.parametrize("ty", [BF, F32], ids=["bf16", "f32"])
def test_every_kernel_has_a_case(ty):
    every = {(k, b, s) for k in ("fwd", "dx", "dw") for b in (0, 1, 2) for s in (False, True) if (k, b) != ("dw", 0)}
    every |= {("fwd", "few", False), ("fwd", "few", True)}
    have = set().union(*(kernels(*s, ty == F32) for s in TL.SHAPES + MORE[ty] + BOTH))
    assert every - have == set()
    # the large tiles with rows and columns that fill none of them
    assert all(K % 256 and O % 256 for _, K, O in MORE[ty] + BOTH)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,O,ty", [(*s, t) for t in (BF, F32) for s in MORE[t] + BOTH],
                         ids=lambda v: {BF: "bf16", F32: "f32"}.get(v, str(v)))
def test_exact_on_the_other_kernels(N, K, O, ty):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    TL.test_forward_exact(N, K, O, "relu", ty)
    TL.test_backward_exact(N, K, O, "relu", ty)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,O,ty", [
    (131071, 8184, 72, BF), (131071, 72, 8184, BF), (40, 8184, 131064, BF), (3, 8184, 131064, BF),
    (43733, 8184, 72, F32), (43733, 72, 8184, F32), (40, 8184, 43728, F32), (3, 8184, 43728, F32)],
    ids=lambda v: {BF: "bf16", F32: "f32"}.get(v, str(v)))
def test_exact_just_below_the_limit(N, K, O, ty):
    """x, out or w (in fp32 its three parts) a few bytes below 2 GiB: the farthest offsets of every operand layout,
    both directions.  The references are fp32 products on the GPU, exact for these whole numbers."""
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gen = torch.Generator(device="cuda").manual_seed(31)
    ints = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=gen, device="cuda", dtype=torch.int8).to(ty)  # noqa: E731
    x, w, d = ints(-2, 2, N, K), ints(-2, 2, O, K), ints(-3, 3, N, O)
    out, _ = G.linear_fwd(x, w)
    g = G.linear_bwd(d, x, w)
    torch.cuda.synchronize()
    rows = 1 << 14
    wf, dw, db = w.float(), torch.zeros(O, K, device="cuda"), torch.zeros(O, device="cuda")
    wt = wf.t().contiguous()
    for lo in range(0, N, rows):
        xs, ds = x[lo:lo + rows].float(), d[lo:lo + rows].float()
        assert torch.equal(out[lo:lo + rows], (xs @ wt).to(ty)), ("out", lo)
        assert torch.equal(g["dx"][lo:lo + rows], (ds @ wf).to(ty)), ("dx", lo)
        dw += ds.t().contiguous() @ xs
        db += ds.sum(0)
    assert torch.equal(g["dw"], dw.to(ty)) and torch.equal(g["dbias"], db)
