"""The routing calls without a GPU: the references' gradients against
differences, the C ABI's argument checks (every call fails validation or has
nothing to do, so nothing is launched) and the binding's refusals."""
import ctypes
import re

import numpy as np
import pytest
import torch

import moe_grouped_gemm_act_amd as fg
from moe_grouped_gemm_act_amd import routed
import routed_ref as ref

OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3
P = ctypes.c_void_p(0x10000)       # aligned non-null stand-in; never dereferenced
Q = ctypes.c_void_p(0x20000)
P_ODD = ctypes.c_void_p(0x10004)   # 4-byte but not 16-byte aligned
P_BAD = ctypes.c_void_p(0x10002)
NUL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    return routed._load()


def test_exports_every_declared_function(lib):
    text = re.sub(r"/\*.*?\*/", "", open(routed.ROUTED_HEADER).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|long long)\s+(\w+)\s*\(", text, flags=re.M)
    assert len(names) >= 12
    for n in names:
        assert hasattr(lib, n), n


def test_the_package_has_the_binding():
    for n in routed.__all__:
        assert getattr(fg, n) is getattr(routed, n) and n in fg.__all__


@pytest.mark.parametrize("renorm", [0, 1])
def test_topk_gradient_against_differences(renorm):
    rng = np.random.default_rng(4100 + renorm)
    x = rng.normal(size=(5, 9)) * 1.5
    x[1, ::2] = -np.inf
    x[2, :] = -np.inf
    x[3, 4] = np.nan
    dw = rng.normal(size=(5, 4))
    ids, _ = ref.topk(x, 4, renorm, 2.5)
    g = ref.topk_backward(x, ids, dw, renorm, 2.5)
    h = 1e-6
    for t in range(5):
        for e in range(9):
            if not np.isfinite(x[t, e]):
                assert g[t, e] == 0
                continue
            hi, lo = x.copy(), x.copy()
            hi[t, e] += h
            lo[t, e] -= h
            d = ((ref.topk(hi, 4, renorm, 2.5)[1] - ref.topk(lo, 4, renorm, 2.5)[1]) * dw).sum() / (2 * h)
            assert abs(d - g[t, e]) < 1e-8


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(4110)
    Y, w = rng.normal(size=(8, 5)), rng.normal(size=(3, 3))
    row = np.array([[0, 5, -1], [7, 2, 3], [-1, 99, -1]])
    dout = rng.normal(size=(3, 5))
    dY, dw, _ = ref.combine_backward(dout, Y, row, w, np.zeros_like(Y))

    def loss(Y, w):
        return (ref.combine(Y, row, w)[0] * dout).sum()
    for a, g in ((Y, dY), (w, dw)):
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + 1e-3
            up = loss(Y, w)
            a[i] = old - 1e-3
            down = loss(Y, w)
            a[i] = old
            assert abs((up - down) / 2e-3 - g[i]) < 1e-10  # the loss is linear in each


def test_dispatch_gradient_is_the_adjoint():
    rng = np.random.default_rng(4120)
    X, dA = rng.normal(size=(3, 5)), rng.normal(size=(8, 5))
    row = np.array([[0, 5, -1], [7, 2, 3], [-1, 99, -1]])
    A = ref.dispatch(X, row, np.zeros((8, 5)))
    dX, _ = ref.combine(dA, row, None)
    assert abs((A * dA).sum() - (X * dX).sum()) < 1e-12


def test_topk_validation(lib):
    for f in (lib.moe_topk_f32, lib.moe_topk_bf16):
        def call(x=P, ids=P, w=P, T=4, E=16, k=2, scale=1.0):
            return f(x, ids, w, T, E, k, 1, scale, NUL)
        assert call(T=-1) == call(E=0, k=0) == call(k=0) == call(k=17) == INVALID
        assert call(x=NUL) == call(ids=NUL) == call(w=NUL) == INVALID
        assert call(scale=0.0) == call(scale=-1.0) == call(scale=float("nan")) == call(scale=float("inf")) == INVALID
        assert call(E=1025) == call(E=128, k=65) == SHAPE
        assert call(T=1 << 22, E=1024) == SHAPE
        assert call(x=P_ODD) == call(ids=P_BAD) == call(w=P_BAD) == MISALIGNED
        assert call(x=NUL, ids=NUL, w=NUL, T=0) == OK
    for f in (lib.moe_topk_backward_f32, lib.moe_topk_backward_bf16):
        def call(x=P, ids=P, w=P, dw=P, dx=P, T=4, E=16, k=2, scale=1.0):
            return f(x, ids, w, dw, dx, T, E, k, 1, scale, NUL)
        assert call(dw=NUL) == call(dx=NUL) == call(k=17) == call(scale=0.0) == INVALID
        assert call(dx=P_ODD) == call(dw=P_BAD) == MISALIGNED
        assert call(x=NUL, ids=NUL, w=NUL, dw=NUL, dx=NUL, T=0) == OK


def test_sort_sizes(lib):
    assert lib.moe_contiguous_rows(0, 4) == 0
    assert lib.moe_contiguous_rows(1, 4) == 128
    assert lib.moe_contiguous_rows(129, 1) == 256
    assert lib.moe_contiguous_rows(3, 8) == 384
    assert lib.moe_contiguous_rows(-1, 8) == lib.moe_contiguous_rows(3, 0) == 0
    assert lib.moe_contiguous_rows((1 << 31) - 1, 1024) == 0  # more than fit
    # the largest layout that any ids need is reached and never passed
    for S in range(0, 700, 37):
        for G in (1, 2, 5):
            worst = max(sum(-(-c // 128) * 128 for c in split) for split in _splits(S, G))
            assert worst <= lib.moe_contiguous_rows(S, G)
    assert lib.moe_sort_workspace(16, 8) == 0
    assert lib.moe_sort_workspace(131072, 256) > 0


def _splits(S, G):
    """some ways to split S choices over G experts, the costliest among them"""
    if G == 1:
        return [[S]]
    out = []
    for small in (0, 1, 129):
        c = [min(small, S // G)] * (G - 1)
        out.append(c + [S - sum(c)])
    return out


def test_sort_validation(lib):
    def contig(ids=P, row=P, mi=P, cnt=P, ws=P, S=100, G=4, M=512):
        return lib.moe_sort_contiguous(ids, row, mi, cnt, ws, S, G, M, NUL)

    def masked(ids=P, row=P, mm=P, ws=P, S=100, G=4, M=40):
        return lib.moe_sort_masked(ids, row, mm, ws, S, G, M, NUL)
    for call in (contig, masked):
        assert call(S=-1) == call(G=0) == call(M=-128) == INVALID
        assert call(ids=NUL) == call(row=NUL) == INVALID
        assert call(ws=NUL, S=100000) == INVALID
        assert call(G=1025) == SHAPE
        assert call(S=(1 << 31) - 1) == SHAPE
        assert call(ids=P_BAD) == call(row=P_BAD) == call(ws=P_BAD) == MISALIGNED
    assert contig(cnt=NUL) == contig(mi=NUL) == masked(mm=NUL) == INVALID
    assert contig(M=500) == SHAPE
    assert masked(G=1024, M=1 << 21) == SHAPE
    assert contig(mi=P_BAD) == masked(mm=P_BAD) == MISALIGNED


def test_dispatch_validation(lib):
    def bf16(X=P, row=P, A=P, T=4, H=64, k=2, M=128, G=1):
        return lib.moe_dispatch_bf16(X, row, A, T, H, k, M, G, NUL)

    def fp8(X=P, row=P, A=P, sa=P, T=4, H=128, k=2, M=128, G=1):
        return lib.moe_dispatch_fp8(X, row, A, sa, T, H, k, M, G, NUL)
    for call in (bf16, fp8):
        assert call(T=-1) == call(H=-1) == call(k=0) == call(M=-1) == call(G=0) == INVALID
        assert call(X=NUL) == call(row=NUL) == call(A=NUL) == INVALID
        assert call(T=1 << 30, k=2) == call(M=1 << 20, G=1 << 11) == SHAPE
        assert call(X=P_ODD) == call(A=P_ODD) == call(row=P_BAD) == MISALIGNED
        assert call(X=NUL, row=NUL, A=NUL, T=0) == call(X=NUL, row=NUL, A=NUL, H=0) == OK
    assert fp8(sa=NUL) == INVALID
    assert fp8(H=64) == SHAPE
    assert fp8(sa=P_BAD) == MISALIGNED


def test_combine_validation(lib):
    def fwd(Y=P, row=P, w=P, out=Q, T=4, H=64, k=2, M=128):
        return lib.moe_combine_bf16(Y, row, w, out, T, H, k, M, NUL)

    def bwd(dout=P, Y=P, row=P, w=P, dY=Q, dw=P, T=4, H=64, k=2, M=128):
        return lib.moe_combine_backward_bf16(dout, Y, row, w, dY, dw, T, H, k, M, NUL)
    for call in (fwd, bwd):
        assert call(T=-1) == call(H=-1) == call(k=0) == call(M=-1) == INVALID
        assert call(Y=NUL) == call(row=NUL) == INVALID
        assert call(T=1 << 30, k=2) == SHAPE
        assert call(Y=P_ODD) == call(row=P_BAD) == call(w=P_BAD) == MISALIGNED
    assert fwd(out=NUL) == bwd(dout=NUL) == bwd(w=NUL) == bwd(dY=NUL) == bwd(dw=NUL) == INVALID
    assert bwd(dY=P) == INVALID  # dY must not be Y
    assert fwd(out=P_ODD) == bwd(dout=P_ODD) == bwd(dY=P_ODD) == bwd(dw=P_BAD) == MISALIGNED
    assert fwd(Y=NUL, row=NUL, w=NUL, out=NUL, T=0) == fwd(Y=NUL, row=NUL, w=NUL, out=NUL, H=0) == OK
    assert bwd(NUL, NUL, NUL, NUL, NUL, NUL, T=0) == OK


def test_lora_validation(lib):
    def bf16(A=P, B=P, La=P, Lb=P, ids=P, scale=P, D=Q, ws=P, M=4, N=64, K=128, R=16, G=2):
        return lib.gemm_bf16_nt_lora(A, B, La, Lb, ids, scale, D, ws, M, N, K, R, G, NUL)

    def fp8(A=P, sa=P, B=P, sb=P, X=P, La=P, Lb=P, ids=P, scale=P, D=Q, ws=P, M=4, N=64, K=128, R=16, G=2):
        return lib.gemm_fp8_1x128_128x128_bf16_lora(A, sa, B, sb, X, La, Lb, ids, scale, D, ws, M, N, K, R, G, NUL)
    for call in (bf16, fp8):
        assert call(M=-1) == call(N=-1) == call(K=-128) == call(R=-8) == call(G=-1) == INVALID
        for name in ("A", "B", "La", "Lb", "ids", "scale", "D", "ws"):
            assert call(**{name: NUL}) == INVALID, name
        assert call(K=100) == call(R=12) == call(R=4104) == call(G=4097) == SHAPE
        assert call(M=1 << 23, K=128, R=128) == call(N=1 << 20, G=4096) == SHAPE
        for name in ("A", "B", "La", "Lb", "D", "ws"):
            assert call(**{name: P_ODD}) == MISALIGNED, name
        assert call(ids=P_BAD) == call(scale=P_BAD) == MISALIGNED
        assert call(M=0, A=NUL, B=NUL, La=NUL, Lb=NUL, ids=NUL, scale=NUL, D=NUL, ws=NUL) == OK
        assert call(R=0, Lb=NUL, A=NUL) == INVALID  # the base call's own check
    assert bf16(K=1 << 23, M=1, N=1, R=8) == SHAPE
    assert fp8(sa=NUL) == fp8(X=NUL) == INVALID
    assert fp8(X=P_ODD) == MISALIGNED
    assert fp8(K=20608) == SHAPE
    for fp8 in (0, 1):
        assert lib.lora_workspace(0, 64, 128, 16, fp8) == lib.lora_workspace(4, 64, 128, 0, fp8) == 0
        assert lib.lora_workspace(4, 64, 128, 16, fp8) >= 4 * 16 * 4 + 4 * 64 * 4
        assert lib.lora_workspace(4096, 64, 7168, 64, fp8) > 4096 * 64 * 2


def test_lora_reference_is_the_dense_sum():
    rng = np.random.default_rng(4200)
    base, X, La, Lb = rng.normal(size=(3, 4)), rng.normal(size=(3, 6)), rng.normal(size=(2, 5, 6)), rng.normal(size=(2, 4, 5))
    D, _, h = ref.lora(base, X, La, Lb, [1, -1, 0], [0.5, 2.0])
    assert np.allclose(D[0], base[0] + 2.0 * X[0] @ (Lb[1] @ La[1]).T)
    assert (D[1] == base[1]).all() and (h[1] == 0).all()
    assert np.allclose(D[2], base[2] + 0.5 * X[2] @ (Lb[0] @ La[0]).T)


def test_binding_refusals():
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    row = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(TypeError):
        fg.moe_topk(x.half(), 2)
    with pytest.raises(ValueError):  # CPU tensors
        fg.moe_topk(x, 2)
    with pytest.raises(TypeError):
        fg.moe_sort_contiguous(row.long(), 4, 128)
    with pytest.raises(TypeError):
        fg.moe_dispatch_bf16(x, row.long(), 128)
    with pytest.raises(ValueError):
        fg.moe_dispatch_bf16(x, row[:3], 128)
    with pytest.raises(ValueError):
        fg.moe_dispatch_fp8(x, row, 128, A=torch.zeros((64, 128), dtype=torch.uint8))
    with pytest.raises(TypeError):
        fg.moe_combine(x.float(), row)
    with pytest.raises(ValueError):
        fg.moe_combine(x, row, w=torch.zeros((4, 3)))
    with pytest.raises(ValueError):
        fg.moe_combine_backward(x[:3], x, row, torch.zeros((4, 2)))
    La, Lb = torch.zeros((2, 8, 128), dtype=torch.bfloat16), torch.zeros((2, 16, 8), dtype=torch.bfloat16)
    W, ids, scale = torch.zeros((16, 128), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), torch.ones(2)
    for bad in ((x, W, La, Lb, ids, scale), (x, W, La, Lb[:1], ids, scale), (x, W, La, Lb, ids[:3], scale)):
        with pytest.raises(ValueError):
            fg.gemm_bf16_nt_lora(*bad)
    with pytest.raises(TypeError):
        fg.gemm_bf16_nt_lora(x, W, La.float(), Lb, ids, scale)
