"""The products with low-rank adapters on the GPU against 64-bit references.

Bound of an element: one rounding to bf16 of the result (2^-8 of it), one of
each h (2^-8 of the sum of |h||Lb|), and fp32 sums of n terms, n 2^-24 of the
sum of their magnitudes; the FP8 matrix instruction's own sum of 128 products
is off by up to 2^-12 of theirs."""
import ctypes
import sys

import numpy as np
import pytest
import torch

import moe_grouped_gemm_act_amd as fg
import routed_ref as ref
import synth
from parity_util import sentinel_out, to_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def announce(msg):
    print(f"[gpu] {msg}", file=sys.stderr, flush=True)


def bf(rng, *shape, scale=1.0):
    return torch.from_numpy(rng.normal(size=shape) * scale).to(torch.bfloat16)


def ids_for(rng, M, G, how):
    if how == "none":
        return np.full(M, -1)
    if how == "one":
        return np.full(M, G - 1)
    if how == "runs":  # requests one after the other, some without an adapter
        ends = np.sort(rng.integers(0, M + 1, size=4))
        return rng.integers(-1, G, size=5)[np.searchsorted(ends, np.arange(M), side="right")]
    odd = rng.choice([-1, -2, G, G + 5, -2147483648, 2147483647], size=M)
    return np.where(rng.random(M) < 0.2, odd, rng.integers(0, G, size=M))


class Case:
    def __init__(self, seed, M, N, K, R, G, how, fp8):
        rng = np.random.default_rng(seed)
        self.M, self.N, self.K, self.R, self.G, self.fp8 = M, N, K, R, G, fp8
        self.X = bf(rng, M, K)
        self.La, self.Lb = bf(rng, G, R, K, scale=K ** -0.5), bf(rng, G, N, R, scale=R ** -0.5)
        self.scale = rng.uniform(0.25, 2.0, size=G).astype(np.float32)
        self.ids = ids_for(rng, M, G, how).astype(np.int32)
        if fp8:
            A, sa = synth.act(seed, M, K)
            B, sb = synth.weight(seed + 1, N, K)
            self.ops = [to_gpu(t) for t in (A, sa, B, sb)]
            a = torch.from_numpy(A).view(torch.float8_e4m3fn).double().numpy() * np.repeat(sa.T.astype(float), 128, 1)
            b = torch.from_numpy(B).view(torch.float8_e4m3fn).double().numpy()
            b = b * np.repeat(np.repeat(sb.astype(float), 128, 0)[:N], 128, 1)
        else:
            W = bf(rng, N, K, scale=K ** -0.5)
            self.ops = [W.to(DEV)]
            a, b = self.X.double().numpy(), W.double().numpy()
        self.base, self.base_mag = a @ b.T, np.abs(a) @ np.abs(b).T

    def run(self, La=None, Lb=None, **kw):
        La = self.La if La is None else La
        Lb = self.Lb if Lb is None else Lb
        X, t = self.X.to(DEV), torch.from_numpy
        rest = (La.to(DEV), Lb.to(DEV), t(self.ids).to(DEV), t(self.scale).to(DEV))
        D = sentinel_out((self.M, self.N))
        kw = {"D": D, **kw}
        if self.fp8:
            out = fg.gemm_fp8_1x128_128x128_bf16_lora(*self.ops, X, *rest, **kw)
        else:
            out = fg.gemm_bf16_nt_lora(X, *self.ops, *rest, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, D, Lb=None):
        Lb = self.Lb if Lb is None else Lb
        with np.errstate(invalid="ignore", over="ignore"):
            want, mag, _ = ref.lora(self.base, self.X.double().numpy(), self.La.double().numpy(), Lb.double().numpy(),
                                    self.ids, self.scale)
            got = D.double().cpu().numpy()
            n = self.K + self.R + 16
            bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -8 * mag + n * U * (2 * mag + self.base_mag)
            # h itself: its sum's error, seen through Lb
            xm = np.abs(self.X.double().numpy()) @ np.abs(self.La.double().numpy()).reshape(-1, self.K).T
            xm = xm.reshape(self.M, self.G, self.R)
            for m, a in enumerate(self.ids):
                if 0 <= a < self.G:
                    he = self.K * U * self.scale[a] * xm[m, a]
                    bound[m] += np.abs(Lb[a].double().numpy()) @ he
            if self.fp8:
                bound += 2.0 ** -12 * self.base_mag
            fine = np.isfinite(want)
            assert (np.isnan(got) == np.isnan(want)).all()
            assert (got[~fine & ~np.isnan(want)] == want[~fine & ~np.isnan(want)]).all()
            bad = fine & ~(np.abs(got - want) <= bound)
        assert not bad.any(), f"{bad.sum()} of {bad.size} outside; first {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


SHAPES = [  # M, N, K, R, G
    (1, 64, 128, 8, 1), (1, 2112, 1024, 16, 4), (3, 97, 256, 24, 2), (17, 130, 128, 8, 40), (63, 576, 384, 64, 64),
    (64, 4096, 2048, 16, 64), (64, 24576, 256, 8, 5), (65, 1000, 640, 72, 9), (128, 4096, 1024, 32, 128),
    (128, 24600, 128, 16, 33), (129, 257, 256, 16, 7), (300, 1030, 512, 40, 3), (515, 2112, 384, 128, 12),
    (200, 150, 960, 64, 3), (257, 300, 7168, 48, 2), (600, 70, 2048, 16, 300), (150, 64, 1024, 200, 5),
    (16, 300, 512, 128, 5), (2, 4099, 256, 1024, 3), (30, 1000, 128, 64, 7), (9, 500, 256, 40, 4), (33, 2112, 640, 32, 33),
    (1030, 64, 512, 16, 3), (1500, 72, 1024, 64, 5), (1027, 48, 1984, 40, 30), (2100, 33, 320, 32, 9),
    (1100, 3700, 256, 64, 4096),
]


@pytest.mark.parametrize("how", ["random", "runs", "one", "none"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("M,N,K,R,G", SHAPES)
def test_product_with_adapters(M, N, K, R, G, fp8, how):
    if G == 4096 and how != "random":
        pytest.skip("the largest adapter count is run once")
    if G == 4096:
        N, R = 61, 8
    if fp8:
        K = K // 128 * 128
    announce(f"lora M={M} N={N} K={K} R={R} G={G} fp8={fp8} {how}")
    c = Case(9000 + M + N + K + R, M, N, K, R, G, how, fp8)
    c.check(c.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("K", [128, 192, 64])
def test_few_base_blocks(K, fp8):
    """fewer blocks of the base product than loads in flight"""
    if fp8 and K % 128:
        pytest.skip("FP8 takes multiples of 128")
    for M in (5, 100, 200):
        announce(f"lora few blocks M={M} K={K} fp8={fp8}")
        c = Case(9100 + M + K, M, 200, K, 16, 30, "random", fp8)
        c.check(c.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("M,N,R", [(40, 320, 24), (64, 4096, 24), (100, 320, 48), (300, 520, 24)])
def test_an_adapter_with_nan_and_inf_reaches_its_own_rows_alone(M, N, R, fp8):
    announce(f"lora wild adapter M={M} N={N} R={R} fp8={fp8}")
    c = Case(9200 + M, M, N, 1024, R, 6, "random", fp8)
    Lb = c.Lb.clone()
    Lb[2, ::7, 3] = float("nan")
    Lb[2, 1::7, 20] = float("inf")
    Lb[4, 5, 0] = -float("inf")
    D = c.run(Lb=Lb)
    assert D.isnan().any() and D.isinf().any()
    c.check(D, Lb)
    clean = c.run()
    La = c.La.clone()
    La[3, 7, 100] = float("nan")
    La[3, R - 1, 1000] = float("inf")
    D = c.run(La=La)
    mine = torch.from_numpy(c.ids == 3)
    assert D.cpu()[mine].isnan().all() and not D.cpu()[~mine].isnan().any()
    c.check(torch.where(mine.to(DEV)[:, None], clean, D))


def test_a_row_with_nan_and_inf_reaches_itself_alone():
    c = Case(9300, 70, 200, 256, 16, 5, "random", False)
    c.ids[[7, 33]] = 1
    clean = c.run()
    c.X[7, 5] = float("nan")
    c.X[33, 9] = float("inf")
    D = c.run()
    other = [m for m in range(70) if m not in (7, 33)]
    assert torch.equal(D[other], clean[other])
    assert D[7].isnan().all() and not D[33].isfinite().any()


@pytest.mark.parametrize("fp8", [False, True])
def test_without_adapters_it_is_the_base_product(fp8):
    for M, N, K in ((64, 2112, 1024), (300, 700, 512)):
        c = Case(9400 + M, M, N, K, 16, 4, "none", fp8)
        D = c.run()
        base = fg.gemm_fp8_1x128_128x128_bf16(*c.ops) if fp8 else fg.gemm_bf16_nt(c.X.to(DEV), *c.ops)
        assert torch.equal(D, base)
        # R = 0 and G = 0 are the base call
        none = torch.empty((4, 0, K), dtype=torch.bfloat16), torch.empty((4, N, 0), dtype=torch.bfloat16)
        c.R = 0
        assert torch.equal(c.run(*none), base)
        c.R, c.G, c.scale = 16, 0, c.scale[:0]
        none = torch.empty((0, 16, K), dtype=torch.bfloat16), torch.empty((0, N, 16), dtype=torch.bfloat16)
        assert torch.equal(c.run(*none), base)


def test_zero_sizes():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    ids, sc = torch.zeros(3, dtype=torch.int32, device=DEV), torch.ones(2, device=DEV)
    assert fg.gemm_bf16_nt_lora(z(0, 64), z(8, 64), z(2, 8, 64), z(2, 8, 8), ids[:0], sc).shape == (0, 8)
    assert fg.gemm_bf16_nt_lora(z(3, 64), z(0, 64), z(2, 8, 64), z(2, 0, 8), ids, sc).shape == (3, 0)
    D = sentinel_out((3, 8))
    fg.gemm_bf16_nt_lora(z(3, 0), z(8, 0), z(2, 8, 0), z(2, 8, 8), ids, sc, D=D)
    assert (D == 0).all()


def test_deterministic_and_independent_of_the_batch():
    """the same bits every time; and a row's bits do not depend on which other
    adapters its tile holds (decode, one K split plan)"""
    c = Case(9500, 64, 4096, 2048, 16, 64, "random", False)
    a, b = c.run().clone(), c.run()
    assert torch.equal(a, b)


def test_streams_and_graph_replay():
    # few rows; a K split in the library's workspace; the matrix form, with and without planes to join
    for M, N, K, R, fp8 in ((64, 4096, 7168, 16, False), (64, 2112, 7168, 16, True), (128, 2112, 2048, 128, True),
                            (128, 2112, 2048, 128, False), (300, 1030, 1024, 40, True), (400, 520, 7168, 64, False)):
        announce(f"lora graph {M}x{N}x{K} rank {R} fp8={fp8}")
        c = Case(9600 + M, M, N, K, R, 8, "random", fp8)
        X, t = c.X.to(DEV), torch.from_numpy
        rest = [c.La.to(DEV), c.Lb.to(DEV), t(c.ids).to(DEV), t(c.scale).to(DEV)]
        D = sentinel_out((M, N))

        def call(**kw):
            if fp8:
                return fg.gemm_fp8_1x128_128x128_bf16_lora(*c.ops, X, *rest, D=D, **kw)
            return fg.gemm_bf16_nt_lora(X, *c.ops, *rest, D=D, **kw)
        call()
        torch.cuda.synchronize()
        eager = D.clone()
        s = torch.cuda.Stream()
        D.zero_()
        torch.cuda.synchronize()
        call(stream=s)  # a temporary workspace, used on a stream that is not the current one
        junk = torch.full((M, 16), float("nan"), dtype=torch.bfloat16, device=DEV)
        s.synchronize()
        assert torch.equal(D, eager)
        del junk
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
        for r in range(3):
            D.zero_()
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                g.replay()
            s.synchronize()
            assert torch.equal(D, eager), r
            call()
            torch.cuda.synchronize()


def test_earlier_hip_error_is_not_reported():
    torch.zeros(1, device=DEV)
    with open("/proc/self/maps") as f:
        paths = {line.split()[-1] for line in f if "libamdhip64.so" in line}
    if len(paths) != 1:
        pytest.skip(f"HIP runtimes loaded: {sorted(paths)}")
    hip = ctypes.CDLL(paths.pop())
    c = Case(9700, 20, 256, 256, 16, 4, "random", False)
    want = c.run().clone()
    X, t = c.X.to(DEV), torch.from_numpy
    args = (X, *c.ops, c.La.to(DEV), c.Lb.to(DEV), t(c.ids).to(DEV), t(c.scale).to(DEV))
    D = sentinel_out((20, 256))
    torch.cuda.synchronize()
    p = ctypes.c_void_p()
    assert hip.hipMalloc(ctypes.byref(p), ctypes.c_size_t(1 << 62)) != 0
    try:
        fg.gemm_bf16_nt_lora(*args, D=D)
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    assert torch.equal(D, want)
