"""The routing calls on the GPU against plain references in 64 bits.

Choices, rows, indices, counts and codes are whole numbers and must be equal.
Bounds for the others, from the arithmetic: a bf16 result is one rounding
(relative 2^-8 at most, half the smallest subnormal below) of an fp32 sum of
n terms, whose error is at most (n + 1) 2^-24 sum |terms|; a softmax weight is
an exponential of a rounded difference, over a sum of such."""
import sys

import numpy as np
import pytest
import torch

import moe_grouped_gemm_act_amd as fg
import routed_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
TINY = 2.0 ** -133  # the smallest bf16 subnormal


def announce(msg):
    print(f"[gpu] {msg}", file=sys.stderr, flush=True)


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def bf16_values(rng, *shape):
    """normal draws that bf16 holds exactly, as float64"""
    return torch.from_numpy(rng.normal(size=shape)).to(torch.bfloat16).double().numpy()


def within(got, want, bound, what):
    bad = np.abs(got - want) > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {want[bad][0]}, bound {np.broadcast_to(bound, bad.shape)[bad][0]}"


def bf16_bound(want, mag, n):
    return 2.0 ** -8 * np.abs(want) + (n + 2) * U * mag + TINY


# ---- route -----------------------------------------------------------------

def logits_for(rng, T, E, bf16):
    x = rng.normal(size=(T, E)) * 2
    x = (torch.from_numpy(x).to(torch.bfloat16 if bf16 else torch.float32)).double().numpy()
    if T > 3:
        x[1, rng.random(E) < 0.5] = -np.inf    # part of the experts masked
        x[2] = -np.inf                         # no expert at all
        x[3] = np.where(rng.random(E) < 0.9, np.nan, x[3])
    if T > 6:
        x[4] = 1.0                             # all equal: the lowest indices
        x[5] = np.where(np.arange(E) % 3 == 0, -3.3895313892515355e38, 0.5)  # the type's lowest values
        x[6] = np.where(np.arange(E) % 2 == 0, 0.0, -0.0)  # zeros of both signs are equal
    return x


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (7, 64, 6), (9, 65, 3), (33, 128, 8), (5, 160, 6),
                                   (8, 256, 8), (11, 384, 9), (8, 511, 1), (7, 1000, 64), (8, 1024, 10),
                                   (4096, 64, 6), (4099, 128, 8), (4102, 200, 16), (4097, 511, 3), (4099, 33, 5), (4100, 256, 17)])
def test_topk(T, E, k, bf16):
    rng = np.random.default_rng(5000 + T * E + k)
    x = logits_for(rng, T, E, bf16)
    xt = gpu(x, torch.bfloat16 if bf16 else torch.float32)
    dw = torch.from_numpy(rng.normal(size=(T, k))).float()
    for renorm in (True, False):
        announce(f"topk T={T} E={E} k={k} bf16={bf16} renorm={renorm}")
        scale = 2.5 if renorm else 1.0
        ids, w = fg.moe_topk(xt, k, renormalize=renorm, scale=scale)
        want_ids, want_w = ref.topk(x, k, renorm, scale)
        assert (ids.cpu().numpy() == want_ids).all()
        # |x - m| roundings in the exponent, a few ulp of exp and of the
        # quotient, E terms in the sum
        span = np.nan_to_num(np.where(np.isfinite(x), np.nanmax(np.where(np.isfinite(x), x, -np.inf), axis=1,
                                                                keepdims=True, initial=-1e30) - x, 0.0))
        rel = (np.minimum(span.max(1), 100) + 24 + E / 32)[:, None] * 2 * U
        within(f64(w), want_w, rel * want_w + 1e-37, "weights")
        g = fg.moe_topk_backward(xt, ids, w, dw.to(DEV), renormalize=renorm, scale=scale)
        assert g.dtype == xt.dtype
        want = ref.topk_backward(x, want_ids, dw.double().numpy(), renorm, scale)
        mag = (want_w * np.abs(dw.double().numpy())).sum(1, keepdims=True)  # no term of a row is larger
        bound = (rel + (k + 4) * U) * 2 * mag + (2.0 ** -8 * np.abs(want) + TINY if bf16 else 0)
        within(f64(g), want, bound + 1e-37, "dlogits")


def test_topk_infinities_share():
    x = torch.zeros((2, 70), device=DEV)
    x[0, 3] = x[0, 40] = float("inf")
    x[1, 69] = float("inf")
    ids, w = fg.moe_topk(x, 3, renormalize=False)
    assert ids.tolist() == [[3, 40, 0], [69, 0, 1]]
    assert w.tolist() == [[0.5, 0.5, 0.0], [1.0, 0.0, 0.0]]


def test_topk_backward_ignores_ids_out_of_range():
    x = torch.randn((3, 16), generator=torch.Generator().manual_seed(1)).to(DEV)
    ids = torch.tensor([[0, -1], [16, 3], [-5, 99]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[1.0, float("nan")], [float("inf"), 0.5], [1.0, 1.0]], device=DEV)
    dw = torch.full((3, 2), 2.0, device=DEV)
    g = fg.moe_topk_backward(x, ids, w, dw, renormalize=True)
    assert torch.isfinite(g).all()
    want = torch.zeros((3, 16))
    want[0, 0] = 1.0 * (2.0 - 2.0)
    want[1, 3] = 0.5 * (2.0 - 1.0)
    assert torch.equal(g.cpu(), want)


# ---- sort ------------------------------------------------------------------

def choices(rng, S, G, skew):
    if skew == "one":
        return np.full(S, G - 1)
    if skew == "none":
        return rng.choice([-1, G, G + 7, -2147483648, 2147483647], size=S)
    if skew == "popular":
        return np.where(rng.random(S) < 0.7, G // 2, rng.integers(-1, G, size=S))
    return rng.integers(-1, G + 1, size=S)


@pytest.mark.parametrize("skew", ["even", "popular", "one", "none"])
@pytest.mark.parametrize("S,G", [(1, 1), (8, 256), (63, 5), (64, 2), (129, 3), (1000, 16), (4096, 1024), (4097, 7), (5000, 1000),
                                 (9000, 129), (70001, 384)])
def test_sort(S, G, skew):
    announce(f"sort S={S} G={G} {skew}")
    rng = np.random.default_rng(6000 + S + G)
    ids = choices(rng, S, G, skew).astype(np.int32)
    t = gpu(ids).view(S, 1)
    full = fg.moe_contiguous_rows(S, G)
    for M in (full, full + 256, max(0, full // 256 * 128)):  # exact, roomy, too small
        sent = dict(row=torch.full((S, 1), 7777, dtype=torch.int32, device=DEV),
                    m_indices=torch.full((M,), 7777, dtype=torch.int32, device=DEV),
                    counts=torch.full((G,), 7777, dtype=torch.int32, device=DEV))
        got = fg.moe_sort_contiguous(t, G, M, **sent)
        for a, b, n in zip(got, ref.sort(ids, G, M, False), ("row", "m_indices", "counts")):
            assert (a.cpu().numpy().ravel() == b).all(), (n, M)
    for M in (0, 1, S // G + 3, S):
        if G * M + S >= 2 ** 31 - 65536:
            continue
        got = fg.moe_sort_masked(t, G, M)
        for a, b, n in zip(got, ref.sort(ids, G, M, True), ("row", "masked_m")):
            assert (a.cpu().numpy().ravel() == b).all(), (n, M)


def test_sort_of_nothing():
    ids = torch.empty((0, 4), dtype=torch.int32, device=DEV)
    row, m_indices, counts = fg.moe_sort_contiguous(ids, 3, 256)
    assert row.shape == (0, 4) and (m_indices == -1).all() and counts.tolist() == [0, 0, 0]
    assert fg.moe_sort_masked(ids, 3, 8)[1].tolist() == [0, 0, 0]


# ---- dispatch and combine --------------------------------------------------

def rows_for(rng, T, k, R, dead):
    """distinct rows of R, some choices dropped, one token without any"""
    row = np.full(T * k, -1, np.int64)
    take = rng.permutation(R)[:T * k]
    row[:take.size] = take
    row = rng.permutation(row).reshape(T, k)
    row[rng.random((T, k)) < dead] = rng.choice([-1, R, R + 1000, -2147483648])
    if T > 2:
        row[1] = -1
    return row.astype(np.int32)


SIZES = [(1, 8, 1), (1, 7168, 8), (3, 1, 2), (5, 7, 3), (4, 136, 9), (17, 2048, 4), (6, 2056, 8), (9, 4099, 17), (64, 640, 6)]


@pytest.mark.parametrize("T,H,k", SIZES)
@pytest.mark.parametrize("G", [1, 3])
def test_dispatch_bf16_and_back(T, H, k, G):
    announce(f"dispatch bf16 T={T} H={H} k={k} G={G}")
    rng = np.random.default_rng(7000 + T + H + k + G)
    M = -(-(T * k + 5) // G)
    R = G * M
    row = rows_for(rng, T, k, R, 0.1)
    X, before = bf16_values(rng, T, H), bf16_values(rng, R, H)
    A = gpu(before, torch.bfloat16).view((G, M, H) if G > 1 else (M, H))
    got = fg.moe_dispatch_bf16(gpu(X, torch.bfloat16), gpu(row), (G, M) if G > 1 else M, A=A)
    assert got is A
    assert (f64(A).reshape(R, H) == ref.dispatch(X, row, before)).all()
    dA = bf16_values(rng, R, H)
    dA[~np.isin(np.arange(R), row)] = np.nan  # rows that no choice names are not read
    dX = fg.moe_dispatch_backward(gpu(dA, torch.bfloat16).view(A.shape), gpu(row))
    want, mag = ref.combine(np.nan_to_num(dA), row, None)
    within(f64(dX), want, bf16_bound(want, mag, k), "dX")


@pytest.mark.parametrize("T,H,k", [(1, 128, 1), (1, 7168, 8), (5, 384, 3), (7, 4096, 9), (3, 4224, 2), (130, 256, 4)])
@pytest.mark.parametrize("G", [1, 3])
def test_dispatch_fp8_equals_quantise_then_copy(T, H, k, G):
    announce(f"dispatch fp8 T={T} H={H} k={k} G={G}")
    rng = np.random.default_rng(7500 + T + H + k + G)
    M = -(-(T * k + 5) // G)
    R = G * M
    row = rows_for(rng, T, k, R, 0.1)
    X = rng.normal(size=(T, H)) * np.exp(rng.normal(size=(T, 1)) * 3)
    X[0, :5] = [np.nan, -0.0, 0.0, 1e-30, -1e-30]
    X[-1, 0] = np.inf
    X[T // 2, :128] = 0.0
    Xt = gpu(X, torch.bfloat16)
    before = rng.integers(0, 255, size=(R, H)).astype(np.uint8)
    sbefore = rng.normal(size=(R, H // 128)).astype(np.float32)
    A = gpu(before).view((G, M, H) if G > 1 else (M, H))
    sa = gpu(sbefore).view(G, M, H // 128).transpose(1, 2).contiguous()
    sa = sa if G > 1 else sa[0]
    fg.moe_dispatch_fp8(Xt, gpu(row), (G, M) if G > 1 else M, A=A, sa=sa)
    q, s = fg.quantize_fp8_1x128(Xt)
    assert (A.cpu().numpy().reshape(R, H) == ref.dispatch(q.cpu().numpy(), row, before)).all()
    want = ref.dispatch(s.t().contiguous().cpu().numpy().view(np.uint32), row, sbefore.view(np.uint32))
    got = sa.view(G, H // 128, M).transpose(1, 2).contiguous().cpu().numpy().view(np.uint32).reshape(R, H // 128)
    assert (got == want).all()


@pytest.mark.parametrize("T,H,k", SIZES)
def test_combine_and_gradients(T, H, k):
    announce(f"combine T={T} H={H} k={k}")
    rng = np.random.default_rng(8000 + T + H + k)
    R = T * k + 5
    row = rows_for(rng, T, k, R, 0.15)
    named = np.isin(np.arange(R), row)
    Y = bf16_values(rng, R, H)
    Yn = np.where(named[:, None], Y, np.nan)  # what no choice names is not read
    w = rng.random((T, k)).astype(np.float32)
    w[row < 0] = np.nan                       # nor the weight of a choice without a row
    w[(row >= R)] = np.inf
    if T > 3:
        w[3] = 0.0
    out = fg.moe_combine(gpu(Yn, torch.bfloat16), gpu(row), gpu(w))
    want, mag = ref.combine(Y, row, w)
    within(f64(out), want, bf16_bound(want, mag, k), "out")
    if T > 2:
        assert (out[1] == 0).all()
    dout, before = bf16_values(rng, T, H), bf16_values(rng, R, H)
    dY = gpu(before, torch.bfloat16)
    _, dw = fg.moe_combine_backward(gpu(dout, torch.bfloat16), gpu(Yn, torch.bfloat16), gpu(row), gpu(w), dY=dY)
    want_dY, want_dw, mag = ref.combine_backward(dout, Y, row, w, before)
    b = np.where(named[:, None], bf16_bound(want_dY, np.abs(want_dY), 1), 0.0)
    within(f64(dY), want_dY, b, "dY")
    within(f64(dw), want_dw, (H / 64 + 16) * U * mag, "dw")


def test_empty_operands():
    e = torch.empty
    row = e((0, 2), dtype=torch.int32, device=DEV)
    assert fg.moe_dispatch_bf16(e((0, 8), dtype=torch.bfloat16, device=DEV), row, 4).shape == (4, 8)
    assert fg.moe_combine(e((4, 8), dtype=torch.bfloat16, device=DEV), row).shape == (0, 8)
    # tokens, but no rows at all: zeros
    row = torch.zeros((3, 2), dtype=torch.int32, device=DEV)
    none = e((0, 8), dtype=torch.bfloat16, device=DEV)
    assert (fg.moe_combine(none, row) == 0).all()
    x = torch.ones((3, 8), dtype=torch.bfloat16, device=DEV)
    dY, dw = fg.moe_combine_backward(x, none, row, torch.ones((3, 2), device=DEV))
    assert dY.shape == (0, 8) and (dw == 0).all()
    fg.moe_dispatch_bf16(x, row, 0)
    a, sa = fg.moe_dispatch_fp8(torch.ones((3, 128), dtype=torch.bfloat16, device=DEV), row, 0)
    assert a.shape == (0, 128) and sa.shape == (1, 0)
    ids, w = fg.moe_topk(e((0, 8), device=DEV), 2)
    assert ids.shape == w.shape == (0, 2)


def test_operand_past_2_31_bytes():
    """rows whose byte offset passes 32 bits"""
    H, M = 8192, 270000  # 4.4 GB of bf16 rows
    announce(f"dispatch into {M} x {H}")
    A = torch.zeros((M, H), dtype=torch.bfloat16, device=DEV)
    x = torch.randn((2, H), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    row = torch.tensor([[0, M - 1], [131072, 262144]], dtype=torch.int32, device=DEV)
    fg.moe_dispatch_bf16(x, row, M, A=A)
    assert torch.equal(A[M - 1], x[0]) and torch.equal(A[0], x[0])
    assert torch.equal(A[131072], x[1]) and torch.equal(A[262144], x[1])
    back = fg.moe_combine(A, row)
    assert torch.equal(back, (x.float() * 2).to(torch.bfloat16))


# ---- streams, graphs, the chain --------------------------------------------

def chain(x, logits, k, E, rows, A, sa):
    ids, w = fg.moe_topk(logits, k)
    row, m_indices, counts = fg.moe_sort_contiguous(ids, E, rows)
    fg.moe_dispatch_fp8(x, row, rows, A=A, sa=sa)
    A2 = fg.moe_dispatch_bf16(x, row, rows, A=torch.zeros((rows, x.shape[1]), dtype=torch.bfloat16, device=DEV))
    out = fg.moe_combine(A2, row, w)
    dY, dw = fg.moe_combine_backward(x, A2, row, w, dY=torch.zeros_like(A2))
    dl = fg.moe_topk_backward(logits, ids, w, dw)
    return ids, w, row, m_indices, counts, A, sa, out, dY, dw, dl


def test_graph_replays_and_other_stream_equal_eager():
    T, H, k, E = 700, 512, 8, 32
    gen = torch.Generator().manual_seed(11)
    x = torch.randn((T, H), generator=gen).to(torch.bfloat16).to(DEV)
    logits = torch.randn((T, E), generator=gen).to(DEV)
    rows = fg.moe_contiguous_rows(T * k, E)
    assert fg.routed._load().moe_sort_workspace(T * k, E) > 0  # the two-launch sort is captured too
    A = torch.zeros((rows, H), dtype=torch.uint8, device=DEV)
    sa = torch.zeros((H // 128, rows), device=DEV)
    eager = [t.clone() for t in chain(x, logits, k, E, rows, A, sa)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain(x, logits, k, E, rows, A, sa)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = chain(x, logits, k, E, rows, A, sa)
    for r in range(3):
        announce(f"replay {r}")
        A.zero_()
        sa.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b)
        again = chain(x, logits, k, E, rows, A, sa)  # eager work between the replays
        torch.cuda.synchronize()
        for a, b in zip(again, eager):
            assert torch.equal(a, b)


def test_stream_argument():
    """the calls run on the stream they are given, temporary workspace included"""
    s = torch.cuda.Stream()
    ids = torch.randint(0, 9, (3000, 4), dtype=torch.int32, generator=torch.Generator().manual_seed(5)).to(DEV)
    want = fg.moe_sort_contiguous(ids, 9)
    torch.cuda.synchronize()
    for _ in range(20):
        got = fg.moe_sort_contiguous(ids, 9, stream=s)
        junk = torch.full((64,), 12345, dtype=torch.int32, device=DEV)  # would reuse a workspace freed too early
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk
