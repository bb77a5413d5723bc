"""The 8-bit operators on the GPU against their float64 oracle.

Bounds, derived from the arithmetic (u = 2^-24, float32 half step):

* norm: h is one addition (u).  The sum of squares adds at most 32 products
  in a thread, 6 + 16 partial sums over lanes and waves, and the squares and
  h itself 3 more, 57 u in all, halved by the root; the division by D, eps,
  the root, the reciprocal and two products are under 16 u together (the
  hardware root, reciprocal and quotient are within 2.5 ulp = 5 u each).
  64 u = 2^-18 bounds y relative to itself.
* gated activation: exp(-g) carries |g| u / ln 2 + 4 u, but enters as
  1 + exp(-g), so only up to the share exp(-g) / (1 + exp(-g)); with
  |g| <= 16 that is under 32 u, division and products 10 u: 64 u again.
* codes: v off by a relative 2^-18 (and the scale by as much, the division
  by 2 u) gives a code between those of v (1 - d) and v (1 + d) with
  d = 2^-16.  Scales: 2^-17.
* product: the terms of a run are exact in float32 and each of at most 128
  additions is off by at most a whole step 2u of the sum of magnitudes (the
  matrix cores' rounding is not specified), 256 u; its two scales and the
  fused multiply-add 3 u; the ceil(K/128) + 32 additions over runs and
  partial sums u each.  All relative to the sum of the terms' magnitudes.
* bf16 products: the FP8 matrix instruction truncates seven of each eight
  products at 2^-13 of the power of two of the largest, 7 * 2^-13 of the sum
  of magnitudes, and the output adds half a step, 2^-8 relative.
"""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
VALUE_TOL = 2.0 ** -18
CODE_TOL = 2.0 ** -16
SCALE_TOL = 2.0 ** -17
E4 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rotated_bit_amd  # noqa: F401
    yield


@pytest.fixture(autouse=True)
def _named(request):
    print(f"[{request.node.name}]", flush=True)
    yield
    torch.cuda.synchronize()


def lib():
    import rotated_bit_amd as H
    return H


def rounded(a, dt):
    """A float64 array as a GPU tensor of dt, and the values it holds."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DT[dt])
    return t.cuda(), t.double().numpy()


def codes(q):
    return torch.from_numpy(np.ascontiguousarray(q)).cuda().view(E4)


def f64(t):
    return t.double().cpu().numpy()


def check_codes(q, s, v):
    """Codes q and scales s of the float64 rows v."""
    got, sc = q.view(torch.uint8).cpu().numpy(), f64(s)
    ref = F.row_scales(v)
    assert np.all(np.abs(sc - ref) <= SCALE_TOL * ref)
    full = F.spread(sc, v.shape[1])
    ends = [F.decode(F.encode(v / full * (1 + d))) for d in (-CODE_TOL, CODE_TOL)]
    val = F.decode(got)
    assert np.all((val >= np.minimum(*ends)) & (val <= np.maximum(*ends)))


def check_product(y, ref, mag, K, dt):
    drop = 7 * 2.0 ** -13 if dt == "bf16" else 0.0
    tol = ((259 + F.runs(K) + 32) * U + drop) * mag * (1 + HALF[dt]) + HALF[dt] * np.abs(ref)
    off = np.abs(f64(y) - ref)
    assert np.all(off <= tol), (off / np.maximum(tol, 1e-300)).max()
    norm = np.linalg.norm(ref)
    print(f"    rel_l2 {np.linalg.norm(f64(y) - ref) / max(norm, 1e-300):.2e}", flush=True)


# ---- norm and gated activation ----------------------------------------------

NORM_SHAPES = [(1, 16), (3, 48), (2, 128), (5, 144), (333, 272), (7, 4096), (4, 5120),
               (2, 8192), (3, 8208), (1, 11008), (2, 16400), (1, 32768), (1100, 1024)]


@pytest.mark.parametrize("x_dt,w_dt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"),
                                       ("f32", "bf16")])
@pytest.mark.parametrize("M,D", NORM_SHAPES)
def test_norm_fp8(M, D, x_dt, w_dt):
    rng = np.random.default_rng(M * 100003 + D)
    x, x64 = rounded(rng.standard_normal((M, D)), x_dt)
    r, r64 = rounded(4 * rng.standard_normal((M, D)), x_dt)
    w, w64 = rounded(1 + 0.2 * rng.standard_normal(D), w_dt)
    for res in (None, r):
        q = torch.empty((M, D), dtype=E4, device="cuda")
        s = torch.empty((M, F.runs(D)), device="cuda")
        out = None if res is None else torch.empty_like(x)
        lib().harp_rmsnorm_fp8(x, w, q, s, eps=1e-5, residual=res, residual_out=out)
        h, y = F.rmsnorm(x64, None if res is None else r64, w64, 1e-5)
        check_codes(q, s, y)
        if out is not None:
            assert np.all(np.abs(f64(out) - h) <= (U + HALF[x_dt]) * (1 + U) * np.abs(h))


@pytest.mark.parametrize("y_dt", ["f32", "bf16"])
@pytest.mark.parametrize("x_dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,D", NORM_SHAPES + [(3, 1), (2, 7), (4, 129), (2, 5121), (1, 32767),
                                               (1, 9001)])
def test_norm(M, D, x_dt, y_dt):
    rng = np.random.default_rng(M * 100003 + D + 1)
    x, x64 = rounded(rng.standard_normal((M, D)), x_dt)
    r, r64 = rounded(4 * rng.standard_normal((M, D)), x_dt)
    w, w64 = rounded(1 + 0.2 * rng.standard_normal(D), x_dt)
    y = torch.empty((M, D), dtype=DT[y_dt], device="cuda")
    lib().harp_rmsnorm(x, w, y, eps=1e-5, residual=r, residual_out=r)      # in place
    h, ref = F.rmsnorm(x64, r64, w64, 1e-5)
    assert np.all(np.abs(f64(y) - ref) <= (VALUE_TOL * (1 + HALF[y_dt]) + HALF[y_dt]) *
                  np.abs(ref))
    assert np.all(np.abs(f64(r) - h) <= (U + HALF[x_dt]) * (1 + U) * np.abs(h))
    # without the sum stored: the same y, the residual left alone
    before = r.clone()
    y2 = torch.empty_like(y)
    lib().harp_rmsnorm(x, w, y2, eps=1e-5, residual=r)
    assert torch.equal(r, before)
    h2, ref2 = F.rmsnorm(x64, f64(before), w64, 1e-5)
    assert np.all(np.abs(f64(y2) - ref2) <= (VALUE_TOL * (1 + HALF[y_dt]) + HALF[y_dt]) *
                  np.abs(ref2))


def test_norm_special_rows():
    D = 272
    x = torch.zeros((5, D), device="cuda")
    x[1] = torch.arange(D) - 100.0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 1e-30
    w = torch.ones(D, device="cuda")
    y = torch.empty_like(x)
    lib().harp_rmsnorm(x, w, y, eps=1e-6)
    assert torch.equal(y[0], torch.zeros_like(y[0])) and torch.isfinite(y[1]).all()
    assert torch.isnan(y[2]).all()
    assert torch.isnan(y[3, 7]) and not torch.isfinite(x[3] * 0 + y[3, 7]).any()
    assert torch.all((y[4] - 1e-27).abs() <= 2.0 ** -17 * 1e-27)
    lib().harp_rmsnorm(x, w, y, eps=0.0)
    assert torch.isnan(y[0]).all()                     # documented: 0 / 0
    q = torch.empty((5, D), dtype=E4, device="cuda")
    s = torch.empty((5, 3), device="cuda")
    lib().harp_rmsnorm_fp8(x, w, q, s, eps=1e-6)
    assert torch.equal(q[0].float(), torch.zeros(D, device="cuda"))
    assert torch.all(s[0] == 2.0 ** -126)
    assert torch.isnan(q[2].float()).all()
    check_codes(q[1:2], s[1:2], F.rmsnorm(f64(x[1:2]), None, f64(w), 1e-6)[1])
    check_codes(q[4:5], s[4:5], F.rmsnorm(f64(x[4:5]), None, f64(w), 1e-6)[1])


# Rows whose squares leave float32's range, either way.  h is scaled by a power
# of two there (exact), so the bounds above hold; eps next to h decides how
# much of the mean it is.  y below 2^-126 is a subnormal number: its two
# products are off by half a subnormal step each, 2^-150, the first times w.
FAR_EPS = [0.0, 1e-44, 1e-38, 1e-30, 1e-6, 1e30, 3e38]
FAR_MAG = [1e-44, 1e-41, 1e-36, 1e-30, 1e-24, 1e-18, 1e-12, 1.0, 1e16, 1e18, 1e19, 1e20, 1e30,
           5e37]


def far_rows(rng, D, dt):
    """Rows of each magnitude, then rows in which one value stands out."""
    a = np.clip(rng.standard_normal((2 * len(FAR_MAG), D)), -3, 3)
    a[:, 0] = 2.0                                        # a row is never all zeros
    mag = np.array(FAR_MAG)[:, None]
    if dt == "bf16":                                     # whose least value is 2^-133
        mag = np.maximum(mag, 1e-39)
    a[:len(FAR_MAG)] *= mag
    a[len(FAR_MAG):, D // 2:] *= mag
    return rounded(a, dt)


@pytest.mark.parametrize("y_dt", ["f32", "bf16"])
@pytest.mark.parametrize("x_dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 16, 272, 5121, 9008, 16400, 32768])
def test_norm_far_from_one(D, x_dt, y_dt):
    rng = np.random.default_rng(D + 40)
    x, x64 = far_rows(rng, D, x_dt)
    w, w64 = rounded(np.clip(1 + 0.2 * rng.standard_normal(D), 0.25, 2), "f32")
    y = torch.empty(x.shape, dtype=DT[y_dt], device="cuda")
    r = torch.empty_like(x)
    for eps in FAR_EPS:
        eps64 = float(np.float32(eps))
        lib().harp_rmsnorm(x, w, y, eps=eps, residual=torch.zeros_like(x), residual_out=r)
        assert torch.equal(r, x)                         # stored as it is, not scaled
        ref = F.rmsnorm(x64, None, w64, eps64)[1]
        tol = (VALUE_TOL * (1 + HALF[y_dt]) + HALF[y_dt]) * np.abs(ref) + 3 * 2.0 ** -150
        if y_dt == "bf16":
            tol += 2.0 ** -134                           # half a subnormal bf16 step
        off = np.abs(f64(y) - ref)
        assert np.all(off <= tol), (eps, np.argwhere(~(off <= tol))[0])


@pytest.mark.parametrize("x_dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [16, 272, 9008, 32768])
def test_norm_fp8_far_from_one(D, x_dt):
    rng = np.random.default_rng(D + 41)
    x, x64 = far_rows(rng, D, x_dt)
    x, x64 = x[:len(FAR_MAG)], x64[:len(FAR_MAG)]
    w, w64 = rounded(np.clip(1 + 0.2 * rng.standard_normal(D), 0.25, 2), "f32")
    q = torch.empty(x.shape, dtype=E4, device="cuda")
    s = torch.empty((x.shape[0], F.runs(D)), device="cuda")
    lib().harp_rmsnorm_fp8(x, w, q, s, eps=0.0)          # y is about 1 in every row
    check_codes(q, s, F.rmsnorm(x64, None, w64, 0.0)[1])


@pytest.mark.parametrize("x_dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [272, 9008])
def test_norm_infinity_and_nan_in_a_row(D, x_dt):
    # an infinity: NaN in its place, zero elsewhere; a NaN: the whole row; a
    # sum of x and residual beyond float32 is an infinity
    x = torch.ones((4, D), dtype=DT[x_dt], device="cuda")
    x[0, 7] = float("inf")
    x[1, 7] = float("-inf")
    x[1, 200] = float("nan")
    x[2, 7] = 3e38
    r = torch.zeros_like(x)
    r[2, 7] = 3e38
    w = torch.ones(D, device="cuda")
    other = torch.arange(D, device="cuda") != 7
    for eps in (0.0, 1e-6):
        for y_dt in ("f32", "bf16"):
            y = torch.empty(x.shape, dtype=DT[y_dt], device="cuda")
            lib().harp_rmsnorm(x, w, y, eps=eps, residual=r)
            for row in (0, 2):
                assert torch.isnan(y[row, 7]) and torch.all(y[row][other] == 0)
            assert torch.isnan(y[1]).all()
            assert torch.all((y[3].float() - 1).abs() <= 2.0 ** -8)
        q = torch.empty(x.shape, dtype=E4, device="cuda")
        s = torch.empty((4, F.runs(D)), device="cuda")
        lib().harp_rmsnorm_fp8(x, w, q, s, eps=eps, residual=r)
        for row in (0, 2):
            assert torch.isnan(q[row, 7].float()) and torch.all(q[row].float()[other] == 0)
            assert torch.all(s[row] == 2.0 ** -126)
        assert torch.isnan(q[1].float()).all() and torch.all(s[1] == 2.0 ** -126)


@pytest.mark.parametrize("x_dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,D", [(1, 16), (3, 144), (16, 11008), (130, 2064), (5, 128),
                                 (1, 262144), (700, 272)])
def test_silu_mul(M, D, x_dt):
    rng = np.random.default_rng(M * 100003 + D + 2)
    x, x64 = rounded(np.clip(3 * rng.standard_normal((M, 2 * D)), -16, 16), x_dt)
    q = torch.empty((M, D), dtype=E4, device="cuda")
    s = torch.empty((M, F.runs(D)), device="cuda")
    lib().harp_silu_mul_fp8(x, q, s)
    check_codes(q, s, F.silu_mul(x64))


def test_silu_mul_special_values():
    D = 400
    x = torch.ones((1, 2 * D), device="cuda")
    x[0, 3] = -200.0                       # exp overflows, silu is -0
    x[0, 4] = 200.0                        # silu(g) = g
    x[0, 130] = float("nan")
    x[0, D + 260] = float("inf")           # u of the third run
    q = torch.empty((1, D), dtype=E4, device="cuda")
    s = torch.empty((1, 4), device="cuda")
    lib().harp_silu_mul_fp8(x, q, s)
    v = q.float()[0]
    assert v[3] == 0 and v[4] == 448 and abs(float(s[0, 0]) - 200 / 448) < 1e-6
    assert torch.isnan(v[130]) and torch.isfinite(v[:130]).all()
    assert torch.isfinite(v[131:256]).all() and torch.isfinite(s[0, 1])
    assert torch.isinf(s[0, 2]) and torch.isnan(v[256:384] * s[0, 2]).all()
    assert torch.isfinite(v[384:]).all() and torch.isfinite(s[0, 3])


@pytest.mark.parametrize("x_dt", ["f32", "bf16"])
def test_silu_mul_gates_past_the_exponential(x_dt):
    # one gate per run, u = 1: the run's scale is that gate's |v| / 448
    gates = [-80.0, -88.0, -89.0, -1000.0, -3e38, float("-inf"), 88.0, 1000.0, 3e38]
    D = 128 * len(gates)
    x = torch.zeros((1, 2 * D), dtype=DT[x_dt], device="cuda")
    x[0, D:] = 1.0
    x[0, 0:D:128] = torch.tensor(gates, dtype=DT[x_dt], device="cuda")
    g = f64(x[0, 0:D:128])
    q = torch.empty((1, D), dtype=E4, device="cuda")
    s = torch.empty((1, len(gates)), device="cuda")
    lib().harp_silu_mul_fp8(x, q, s)
    code, s = q.float()[0, ::128], f64(s)[0]
    # at -80 and -88 the exponential is off by |g| u / ln 2 + 4 u, all else by
    # 10 u: under 2^-16; v / 448 lies below the least scale at -88
    v = g[:2] * np.exp(g[:2]) / (1 + np.exp(g[:2]))
    assert code[0] == -448 and abs(s[0] * 448 / -v[0] - 1) <= 2.0 ** -16
    ends = [F.decode(F.encode(v[1] * 2.0 ** 126 * (1 + d))) for d in (-2.0 ** -16, 2.0 ** -16)]
    assert min(ends) <= float(code[1]) <= max(ends)
    assert torch.isnan(code[5]) and torch.all(code[2:5] == 0)
    assert np.all(s[1:6] == 2.0 ** -126)
    assert torch.all(code[6:] == 448) and np.all(np.abs(s[6:] * 448 / g[6:] - 1) <= 2.0 ** -17)
    assert torch.all(q.float()[0].reshape(-1, 128)[:, 1:] == 0)


# ---- product ------------------------------------------------------------------

def weight(rng, N, K, experts=None):
    """A coded weight (some outlier columns), as the handle and as numpy."""
    shape = (experts or 1, N, K)
    w = 0.02 * rng.standard_normal(shape) * np.where(rng.random(K) < 0.02, 20, 1)
    qs = [F.code_weight(w[e]) for e in range(shape[0])]
    q, s = np.stack([a for a, _ in qs]), np.stack([b for _, b in qs])
    if experts is None:
        return lib().FP8Weight(codes(q[0]), torch.from_numpy(s[0]).cuda()), q, s
    return lib().FP8Weight(codes(q), torch.from_numpy(s).cuda()), q, s


def rows_of(rng, M, K):
    a = rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.02, 20, 1)
    q, s = F.code_rows(a)
    return codes(q), torch.from_numpy(s).cuda(), q, s


SHAPES = [(1, 1, 16), (1, 16, 128), (1, 4096, 4096), (2, 17, 144), (3, 100, 112), (16, 128, 256),
          (16, 1030, 4096), (17, 130, 400), (33, 96, 1040), (48, 2048, 2048), (64, 257, 1024),
          (65, 384, 1040), (100, 1000, 272), (128, 256, 2048), (129, 511, 144), (200, 1100, 1536),
          (256, 512, 512), (257, 640, 656), (300, 512, 4096), (513, 1153, 640),
          (1024, 2304, 1152), (1500, 900, 16), (2100, 2050, 400), (33, 5458, 400),
          (17, 4162, 1040), (65, 5455, 272), (257, 3587, 656), (1000, 4001, 1040),
          (1000, 4635, 144), (1500, 5391, 272), (700, 16400, 144), (50, 30000, 144)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, dt):
    rng = np.random.default_rng((M * 1009 + N) * 1009 + K)
    W, wq, ws = weight(rng, N, K)
    a, sa, aq, as_ = rows_of(rng, M, K)
    y = torch.full((M + 2, N), 7.0, dtype=DT[dt], device="cuda")[:M]
    guard = y.as_strided((2, N), (N, 1), M * N)
    lib().harp_fp8_gemm(W, a, sa, y)
    ref, mag = F.product(aq, as_, wq[0], ws[0])
    check_product(y, ref, mag, K, dt)
    assert torch.all(guard == 7.0)
    again = torch.empty_like(y)
    lib().harp_fp8_gemm(W, a, sa, again)
    assert torch.equal(again, y)


@pytest.mark.parametrize("M", [1, 20, 150, 700])
def test_product_keeps_nan_in_its_row_and_column(M):
    rng = np.random.default_rng(M)
    N, K = 300, 272
    W, wq, ws = weight(rng, N, K)
    a, sa, aq, as_ = rows_of(rng, M, K)
    W.w.view(torch.uint8)[200, 270] = 0x7f
    a.view(torch.uint8)[M // 2, 3] = 0xff
    y = torch.empty((M, N), device="cuda")
    lib().harp_fp8_gemm(W, a, sa, y)
    bad = torch.isnan(y).cpu().numpy()
    want = np.zeros((M, N), dtype=bool)
    want[M // 2] = True
    want[:, 200] = True
    assert np.array_equal(bad, want)


def sizes_to_offsets(sizes, start=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]) + start, dtype=torch.int32,
                        device="cuda")


GROUPS = [
    ([1], 16, 128, False), ([0, 0, 5], 40, 144, True), ([3, 0, 17, 1], 130, 272, True),
    ([1] * 8, 256, 1024, True), ([64, 0, 65, 1, 0], 200, 400, False),
    ([0, 300, 0, 1, 129, 0, 0], 384, 656, True), ([128, 128, 257], 300, 512, False),
    ([5] * 70, 48, 160, True), ([0] * 130 + [3] + [0] * 70 + [9], 33, 144, True),
    ([700, 1, 2, 900], 260, 256, True), ([256] * 4, 512, 384, False),
    ([700, 0, 900, 500], 5001, 272, True), ([100, 300, 0, 20] * 3, 2100, 144, False),
    ([2500, 2, 3000], 4100, 144, True), ([5, 0, 20], 4832, 400, True),
    ([0, 200, 5, 60, 20, 1, 20, 1, 20], 3330, 144, True),
    ([200, 5, 0, 100, 20, 1, 5, 0, 130], 3398, 272, True),
    ([100, 5, 5, 0, 0, 100, 1, 0], 3734, 656, True), ([0, 0, 5, 0, 1], 3274, 272, True),
    ([1, 1, 1, 1, 5], 862, 400, True), ([1, 130, 5, 1, 20, 5], 4936, 144, True),
    ([0, 0, 1, 1, 60, 5], 4535, 272, True),
    ([5, 60, 100, 5, 20, 60, 0, 300, 0, 0, 20], 4887, 144, False),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("sizes,N,K,gather", GROUPS)
def test_grouped(sizes, N, K, gather, dt):
    rng = np.random.default_rng(sum(sizes) * 31 + N)
    E, live = len(sizes), sum(sizes)
    M = live + 5                       # two rows before the first expert, three behind the last
    W, wq, ws = weight(rng, N, K, E)
    a_rows = max(4, live // 3) if gather else M
    a, sa, aq, as_ = rows_of(rng, a_rows, K)
    rows = rng.integers(0, a_rows, M) if gather else np.arange(M)
    rows[:min(M, 4)] = rows[0] if gather else rows[:min(M, 4)]      # the same row again
    off = sizes_to_offsets(sizes, 2)
    y = torch.full((M, N), 7.0, dtype=DT[dt], device="cuda")
    lib().harp_fp8_gemm_grouped(
        W, a, sa, off, y, rows=torch.tensor(rows, dtype=torch.int32, device="cuda")
        if gather else None)
    assert torch.all(y[:2] == 7.0) and torch.all(y[2 + live:] == 7.0)
    at = 2
    ref, mag = np.zeros((live, N)), np.zeros((live, N))
    for e, n in enumerate(sizes):
        i = rows[at:at + n]
        ref[at - 2:at - 2 + n], mag[at - 2:at - 2 + n] = F.product(aq[i], as_[i], wq[e], ws[e])
        at += n
    check_product(y[2:2 + live], ref, mag, K, dt)


# Many runs of K, with a ragged last one: large tiles and split runs.
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [
    (2361, 1686, 2480), (1239, 1561, 2064), (714, 1399, 1264), (260, 980, 4400),
    (1237, 1642, 2208), (2675, 891, 2208), (1306, 391, 1456), (670, 885, 1616),
    (591, 425, 3600), (456, 578, 4368), (33, 1100, 8336)])
def test_product_long(M, N, K, dt):
    test_product(M, N, K, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("sizes,N,K,gather", [
    ([1500, 3, 1098], 1737, 2576, True),
    ([400, 0, 300, 1, 500, 200, 366, 250, 250], 824, 2736, False),
    ([300, 0, 0, 1, 200, 100, 257, 100, 100], 787, 1136, True),
    ([1000, 320, 1000], 849, 2384, False), ([5, 60, 0, 100, 100, 1, 39, 0, 0], 1746, 400, True),
    ([3, 0, 60], 1864, 480, False), ([470, 0, 300], 352, 4272, True)])
def test_grouped_long(sizes, N, K, gather, dt):
    test_grouped(sizes, N, K, gather, dt)


# Large products, with waves that have no row or no output in the last tiles of
# a row or an expert (test_gpu_fp8_tiles.py: each tile by name).
@pytest.mark.parametrize("M,N,K", [(3900, 4240, 912), (4000, 4001, 1168)])
def test_product_large(M, N, K):
    test_product(M, N, K, "bf16")


@pytest.mark.parametrize("sizes,N,K,gather", [([2000, 3, 1900, 90], 5000, 1040, True),
                                              ([1, 2600, 2399], 3400, 912, False)])
def test_grouped_large(sizes, N, K, gather):
    test_grouped(sizes, N, K, gather, "bf16")


@pytest.mark.parametrize("sizes", [[2, 3], [40, 90], [300, 500]])
def test_grouped_rows_out_of_range_are_zero(sizes):
    rng = np.random.default_rng(8)
    M, N, K = sum(sizes), 140, 272
    W, wq, ws = weight(rng, N, K, 2)
    a, sa, aq, as_ = rows_of(rng, 9, K)
    rows = torch.from_numpy(rng.integers(0, 9, M)).int().cuda()
    bad = torch.tensor([0, M // 2, M - 1], device="cuda")
    rows[bad] = torch.tensor([-1, 9, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    y = torch.full((M, N), 7.0, device="cuda")
    lib().harp_fp8_gemm_grouped(W, a, sa, sizes_to_offsets(sizes), y, rows=rows)
    assert torch.all(y[bad] == 0)
    fine = torch.ones(M, dtype=torch.bool, device="cuda")
    fine[bad] = False
    assert torch.all((y[fine] != 0).any(1)) and torch.isfinite(y).all()


@pytest.mark.parametrize("sizes,N", [([3, 2, 4], 40), ([30, 70, 90], 500), ([300, 1, 400], 2100)])
def test_grouped_nan_stays_where_it_is(sizes, N):
    # NaN codes and scales in rows nobody asks for, in one row of one expert
    # and in another expert's weights
    rng = np.random.default_rng(12)
    M, K, a_rows = sum(sizes), 272, 50
    W, wq, ws = weight(rng, N, K, 3)
    a, sa, aq, as_ = rows_of(rng, a_rows, K)
    rows = rng.integers(0, 40, M)
    off = np.concatenate([[0], np.cumsum(sizes)])
    rows[0] = 60                                          # no such row: zeros, of a NaN weight too
    rows[off[1]] = 45
    a.view(torch.uint8)[40:] = 0x7f
    sa[40:] = float("nan")
    W.w.view(torch.uint8)[0, N // 2, 7] = 0xff
    y = torch.empty((M, N), device="cuda")
    lib().harp_fp8_gemm_grouped(W, a, sa, sizes_to_offsets(sizes), y,
                                rows=torch.tensor(rows, dtype=torch.int32, device="cuda"))
    want = np.zeros((M, N), dtype=bool)
    want[1:off[1], N // 2] = True
    want[off[1]] = True
    assert np.array_equal(torch.isnan(y).cpu().numpy(), want)
    assert torch.all(y[0] == 0)


@pytest.mark.parametrize("M", [6, 90, 600])
def test_grouped_offsets_out_of_range_write_nothing_else(M):
    # offsets past M and below 0 are taken as the nearer end; decreasing ones
    # leave y undefined, but the rows around it stay as they were
    rng = np.random.default_rng(9)
    N, K = 70, 144
    W, wq, ws = weight(rng, N, K, 4)
    a, sa, aq, as_ = rows_of(rng, M, K)
    big = torch.full((M + 8, N), 7.0, device="cuda")
    y = big[4:4 + M]
    y = y if y.data_ptr() % 16 == 0 else None
    assert y is not None
    ends = torch.tensor([-5, M // 2, M // 2, M + 1000, 2 ** 31 - 1], dtype=torch.int32,
                        device="cuda")
    lib().harp_fp8_gemm_grouped(W, a, sa, ends, y)
    lo, mag_lo = F.product(aq[:M // 2], as_[:M // 2], wq[0], ws[0])
    hi, mag_hi = F.product(aq[M // 2:], as_[M // 2:], wq[2], ws[2])
    check_product(y, np.concatenate([lo, hi]), np.concatenate([mag_lo, mag_hi]), K, "f32")
    for wild in ([M, 0, M, 0, M], [3, 2, 1, 0, -7], [2 ** 31 - 1, -2 ** 31, 5, M, 1]):
        lib().harp_fp8_gemm_grouped(W, a, sa, torch.tensor(wild, dtype=torch.int32,
                                                           device="cuda"), y)
    assert torch.all(big[:4] == 7.0) and torch.all(big[4 + M:] == 7.0)


@pytest.mark.parametrize("M", [3, 100])
def test_grouped_rows_past_two_gigabytes(M):
    rng = np.random.default_rng(10)
    N, K, a_rows = 48, 65536, 40000                       # a of 2.6e9 bytes
    W, wq, ws = weight(rng, N, K, 1)
    a = torch.zeros((a_rows, K), dtype=torch.uint8, device="cuda").view(E4)
    sa = torch.zeros((a_rows, K // 128), device="cuda")
    used = [0, 5, 32767, 32768, 39998, 39999]
    u, su, uq, us = rows_of(rng, len(used), K)
    a.view(torch.uint8)[used] = u.view(torch.uint8)
    sa[used] = su
    pick = rng.integers(0, len(used), M)
    rows = torch.tensor(np.array(used)[pick], dtype=torch.int32, device="cuda")
    y = torch.empty((M, N), device="cuda")
    lib().harp_fp8_gemm_grouped(W, a, sa, sizes_to_offsets([M]), y, rows=rows)
    check_product(y, *F.product(uq[pick], us[pick], wq[0], ws[0]), K, "f32")


def test_product_output_past_four_gigabytes():
    rng = np.random.default_rng(13)
    M, N, K = 65536, 33001, 16                            # y of 4.3e9 bytes, rows not aligned
    W, wq, ws = weight(rng, N, K)
    a, sa, aq, as_ = rows_of(rng, M, K)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    lib().harp_fp8_gemm(W, a, sa, y)
    for i in (slice(0, 3), slice(65070, 65090), slice(65533, 65536)):
        ref, mag = F.product(aq[i], as_[i], wq[0], ws[0])
        check_product(y[i], ref, mag, K, "bf16")
    assert not torch.any(y[:, 0] == 7.0) and not torch.any(y[:, -1] == 7.0)


@pytest.mark.parametrize("rows", [3, 200])
def test_grouped_weights_past_four_gigabytes(rows):
    rng = np.random.default_rng(14)
    E, N, K = 70, 8192, 8192                              # w of 4.7e9 bytes
    w = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda")
    s = torch.zeros((E, 64, 64), device="cuda")
    used = (0, 63, 64, 69)
    small, wq, ws = weight(rng, N, 256, len(used))
    for i, e in enumerate(used):                          # inputs 7936 .. 8191 only
        w[e, :, 7936:] = small.w[i].view(torch.uint8)
        s[e, :, 62:] = small.scale[i]
    sizes = [rows if e in used else 0 for e in range(E)]
    a, sa, aq, as_ = rows_of(rng, 4 * rows, K)
    y = torch.empty((4 * rows, N), device="cuda")
    lib().harp_fp8_gemm_grouped(lib().FP8Weight(w.view(E4), s), a, sa, sizes_to_offsets(sizes), y)
    for i in range(4):
        r = slice(i * rows, (i + 1) * rows)
        ref, mag = F.product(np.ascontiguousarray(aq[r, 7936:]), as_[r, 62:], wq[i], ws[i])
        check_product(y[r], ref, mag, K, "f32")


def test_empty_calls():
    H = lib()
    rng = np.random.default_rng(1)
    W, _, _ = weight(rng, 32, 128)
    We, _, _ = weight(rng, 32, 128, 3)
    a, sa = torch.empty((0, 128), dtype=E4, device="cuda"), torch.empty((0, 1), device="cuda")
    y = torch.empty((0, 32), device="cuda")
    H.harp_fp8_gemm(W, a, sa, y)
    H.harp_fp8_gemm_grouped(We, a, sa, torch.zeros(4, dtype=torch.int32, device="cuda"), y)
    x = torch.empty((0, 128), device="cuda")
    H.harp_rmsnorm_fp8(x, torch.ones(128, device="cuda"), a, sa)
    H.harp_rmsnorm(x, torch.ones(128, device="cuda"), x.clone())
    H.harp_silu_mul_fp8(torch.empty((0, 256), device="cuda"), a, sa)
    # every expert empty: y stays
    y = torch.full((4, 32), 7.0, device="cuda")
    a, sa, _, _ = rows_of(rng, 4, 128)
    H.harp_fp8_gemm_grouped(We, a, sa, torch.zeros(4, dtype=torch.int32, device="cuda"), y)
    assert torch.all(y == 7.0)


# ---- together -------------------------------------------------------------------

def experts_layer(H, st, stream=None):
    """norm -> gate and up of each row's expert -> gated activation -> down."""
    H.harp_rmsnorm_fp8(st["x"], st["nw"], st["q"], st["qs"], eps=1e-5, residual=st["r"],
                       residual_out=st["r_out"], stream=stream)
    H.harp_fp8_gemm_grouped(st["Wgu"], st["q"], st["qs"], st["off"], st["gu"], rows=st["rows"],
                            stream=stream)
    H.harp_silu_mul_fp8(st["gu"], st["h"], st["hs"], stream=stream)
    H.harp_fp8_gemm_grouped(st["Wd"], st["h"], st["hs"], st["off"], st["y"], stream=stream)


def experts_state(seed, tokens, top, E, K, I, dt="bf16"):
    rng = np.random.default_rng(seed)
    M = tokens * top
    st = {"K": K, "I": I, "np": {}}
    for name, scale in (("x", 1), ("r", 4)):
        st[name], st["np"][name] = rounded(scale * rng.standard_normal((tokens, K)), dt)
    st["r_out"] = torch.empty_like(st["r"])
    st["nw"], st["np"]["nw"] = rounded(1 + 0.2 * rng.standard_normal(K), dt)
    st["Wgu"], *st["np"]["Wgu"] = weight(rng, 2 * I, K, E)
    st["Wd"], *st["np"]["Wd"] = weight(rng, K, I, E)
    reroute(st, rng, tokens, top, E)
    e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    st["q"], st["qs"] = e(tokens, K, dtype=E4), e(tokens, F.runs(K))
    st["gu"], st["y"] = e(M, 2 * I, dtype=DT[dt]), e(M, K, dtype=DT[dt])
    st["h"], st["hs"] = e(M, I, dtype=E4), e(M, F.runs(I))
    return st


def reroute(st, rng, tokens, top, E):
    expert = np.stack([rng.permutation(E)[:top] for _ in range(tokens)]).ravel()
    order = np.argsort(expert, kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(expert, minlength=E))])
    st["np"]["rows"], st["np"]["off"] = order // top, off
    for name in ("rows", "off"):
        t = torch.tensor(st["np"][name], dtype=torch.int32, device="cuda")
        if name in st:
            st[name].copy_(t)
        else:
            st[name] = t


def check_experts(st):
    """Every step against the oracle on the step's own stored inputs."""
    n = st["np"]
    h, y = F.rmsnorm(n["x"], n["r"], n["nw"], 1e-5)
    check_codes(st["q"], st["qs"], y)
    q, qs = st["q"].view(torch.uint8).cpu().numpy(), f64(st["qs"])
    hq, hs = st["h"].view(torch.uint8).cpu().numpy(), f64(st["hs"])
    check_codes(st["h"], st["hs"], F.silu_mul(f64(st["gu"])))
    off, rows = n["off"], n["rows"]
    for e in range(len(off) - 1):
        i = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        src = rows[i]
        check_product(st["gu"][i], *F.product(q[src], qs[src], n["Wgu"][0][e], n["Wgu"][1][e]),
                      st["K"], "bf16")
        check_product(st["y"][i], *F.product(hq[i], hs[i], n["Wd"][0][e], n["Wd"][1][e]),
                      st["I"], "bf16")


@pytest.mark.parametrize("tokens,top,E,K,I", [(1, 2, 4, 256, 144), (8, 4, 8, 512, 256),
                                              (150, 2, 5, 400, 272)])
def test_experts_layer(tokens, top, E, K, I):
    st = experts_state(tokens, tokens, top, E, K, I)
    experts_layer(lib(), st)
    torch.cuda.synchronize()
    check_experts(st)


def test_experts_layer_captured_with_other_routings():
    H = lib()
    tokens, top, E, K, I = 24, 2, 6, 256, 160
    st = experts_state(5, tokens, top, E, K, I)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        experts_layer(H, st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        experts_layer(H, st)
    rng = np.random.default_rng(11)
    for _ in range(4):
        reroute(st, rng, tokens, top, E)
        g.replay()
        torch.cuda.synchronize()
        check_experts(st)
        got = st["y"].clone()
        experts_layer(H, st)                          # the eager call between replays
        torch.cuda.synchronize()
        assert torch.equal(got, st["y"])


def test_two_streams_at_once():
    H = lib()
    sts = [experts_state(20 + i, 64, 2, 4, 512, 256) for i in range(2)]
    want = []
    for st in sts:
        experts_layer(H, st)
        torch.cuda.synchronize()
        want.append(st["y"].clone())
        st["y"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sts]
    for _ in range(10):
        for st, s in zip(sts, streams):
            experts_layer(H, st, stream=s)
    torch.cuda.synchronize()
    for st, w in zip(sts, want):
        assert torch.equal(st["y"], w)


@pytest.mark.parametrize("M", [1, 16])
def test_norm_feeds_both_linears(M):
    """One norm in front of a rotated 2-bit linear (bf16 y) and of an 8-bit one (codes)."""
    import devbuf as d
    from oracle import harp_oracle as O
    from synth import workloads as S
    H = lib()
    K, N = 4096, 4096
    li = S.layer_inputs(S.CONFIGS["l7b_decode"], 0, 2, M)
    V, U_, Wq = d.dev_rotation(li.V), d.dev_rotation(li.U), d.dev_qweight(li.W)
    rng = np.random.default_rng(M)
    x, x64 = rounded(rng.standard_normal((M, K)), "bf16")
    r, r64 = rounded(rng.standard_normal((M, K)), "bf16")
    w, w64 = rounded(1 + 0.2 * rng.standard_normal(K), "bf16")
    y = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((M, N), device="cuda")
    H.harp_rmsnorm(x, w, y, eps=1e-5, residual=r)
    H.harp_linear_fused(V, Wq, U_, y, out, d.workspace(M, N, K))
    ref = O.linear(f64(y), li.W.words, li.W.scale.view(np.float16), li.W.zero.view(np.float16),
                   2, li.V.cs, li.V.sign_bits, li.V.block, li.U.cs, li.U.sign_bits, li.U.block)
    assert O.rel_l2(f64(out), ref) <= 1e-3
    assert np.all(np.abs(f64(y) - F.rmsnorm(x64, r64, w64, 1e-5)[1]) <=
                  (VALUE_TOL * 2 + 2.0 ** -8) * np.abs(F.rmsnorm(x64, r64, w64, 1e-5)[1]))
    W8, wq, ws = weight(rng, 256, K)
    q, s = torch.empty((M, K), dtype=E4, device="cuda"), torch.empty((M, K // 128), device="cuda")
    y8 = torch.empty((M, 256), device="cuda")
    H.harp_rmsnorm_fp8(x, w, q, s, eps=1e-5, residual=r)
    H.harp_fp8_gemm(W8, q, s, y8)
    check_product(y8, *F.product(q.view(torch.uint8).cpu().numpy(), f64(s), wq[0], ws[0]), K,
                  "f32")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M", [3, 300])
def test_product_of_scales_below_the_normal_range(M, dt):
    # sa sw is float32: below 2^-126 it is off by half a subnormal step, 2^-150,
    # which enters y times the run's sum; all else as ever
    rng = np.random.default_rng(M + 70)
    N, K = 272, 400
    W, wq, ws = weight(rng, N, K)
    a, sa, aq, as_ = rows_of(rng, M, K)
    for down in (100, 109, 114, 117):
        s = np.ldexp(as_, -down).astype(np.float32)      # exact: scales from 2^-8 on
        assert np.array_equal(np.ldexp(s.astype(np.float64), down), as_)
        y = torch.empty((M, N), dtype=DT[dt], device="cuda")
        lib().harp_fp8_gemm(W, a, torch.from_numpy(s).cuda(), y)
        ref, mag = F.product(aq, s, wq[0], ws[0])
        ones = np.ones_like
        plain = F.product(aq, ones(s), wq[0], ones(ws[0]))[1]      # sums of |a w|
        drop = 7 * 2.0 ** -13 if dt == "bf16" else 0.0
        tol = ((259 + F.runs(K) + 32) * U + drop) * mag + HALF[dt] * np.abs(ref) * (1 + drop)
        tol = tol * (1 + HALF[dt]) + 2.0 ** -150 * plain * (1 + HALF[dt] + drop) + 2.0 ** -134
        assert np.all(np.abs(f64(y) - ref) <= tol)
