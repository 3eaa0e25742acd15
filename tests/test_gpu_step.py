"""A step's operators on the GPU against the 64-bit oracle (oracle/step.py).

norm: h, the scales and the codes are defined by float32 roundings: equal.  y in a 16-bit type is one rounding of a float32: equal to
torch's.

product: a term a w (8 bits of mantissa) is exact; a block's 128 terms are added by the tensor cores, at worst each addition truncating
at float32's 2^-23 of the magnitudes so far: 2^-16 of their sum A; the factor s_a s_w is rounded once, each block's sum times the factor and the addition
once: with B blocks
    |got - want| <= (2^-16 + (B + 3) 2^-24) A,   plus eps / 2 of the value in a 16-bit type (and fp16's smallest step).

rope: with a the exact angle, freqs[i] / 2 pi is off by three roundings of 2^-53, so the angle by pos f 2^-51 at most; the
fraction's cut (2^-32 turns) and its rounding to float32 (2^-27 half turns) by under 2^-25; cos and sin have two units in the last place
(2^-23), the factor one rounding (2^-24), products and sums of |u|, |v| <= |u| + |v| two (2^-23):
    |got - want| <= (|u| + |v|) |scale| (2^-21 + pos f 2^-51),   plus eps / 2 of the value in a 16-bit type.

logprobs: with d = z - max, exact to 2^-24 |d|: 2^(d log2 e) is off by a factor 1 + 2^-22 + |d| 2^-22; a sum's chain has at most L = vocab / 256 + 64
additions (a thread's, then the merges'), each 2^-24.  So log S is off by 2^-22 (1 + sum p |d|) + L 2^-24, the merges' factors by
2^-20 more, and
    |logprob| : 2^-20 + L 2^-24 + 2^-22 sum p |d| + 2^-23 (drop + |log p|)
    |entropy| : (2^-19 + L 2^-23) (1 + sum p |d|) + 2^-22 sum p d^2 <= (2^-19 + L 2^-23) (1 + sum p |d|) + 2^-22 * 128 sum p |d|
(p d^2 <= 128 p |d| where p is not 0 in float32).  Ranks and ids go by the logits as given: equal.
"""
import numpy as np
import pytest

from oracle import kv4, step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def B(cuda):
    from layer_range_stage_gb300 import binding
    return binding


def dev(x, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(x))
    return t.to("cuda", dtype) if dtype is not None else t.cuda()


def i32(x):
    return dev(np.asarray(x), torch.int32)


def given(x, dtype):
    """float64 of the numbers that a tensor of this type holds."""
    return torch.as_tensor(np.ascontiguousarray(x)).to(DT[dtype]).double().numpy()


def same(a, b):
    a, b = np.asarray(a), np.asarray(b)
    assert a.shape == b.shape
    assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f"), (np.argwhere(~((a == b) | ((a != a) & (b != b))))[:5], (a != b).mean())


def close(got, want, tol):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), np.argwhere(np.isnan(got) != nan)[:4]
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    ok = ~nan & ~inf
    err, tol = np.abs(got - np.where(ok, want, 0))[ok], np.broadcast_to(tol, want.shape)[ok]
    assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), np.argwhere(ok)[~(err <= tol)][:4])


def half_step(want, dtype):
    """eps / 2 of the value, and half of fp16's smallest step."""
    if dtype == "f32":
        return 0.0
    return np.abs(want) * torch.finfo(DT[dtype]).eps / 2 + (2.0 ** -25 if dtype == "f16" else 0.0)


def spaced(n, k, dtype, gap, fill=0):
    """[n, k] rows `gap` elements apart inside a larger tensor, and that tensor."""
    whole = torch.full((n, k + gap), fill, dtype=torch.float32, device="cuda").to(dtype)
    return whole[:, :k], whole


# ------------------------------------------------------------------------------------------- norm

def run_norm(B, x, resid, gamma, xt, rt, eps=1e-5, gap=0, plain=True, inplace=False):
    n_tok, n = x.shape
    xd, _ = spaced(n_tok, n, DT[xt], gap)
    xd.copy_(torch.as_tensor(x))
    rd = ro = None
    if resid is not None:
        rd, _ = spaced(n_tok, n, DT[rt], gap)
        rd.copy_(torch.as_tensor(resid))
        ro, whole = (rd, None) if inplace else spaced(n_tok, n, DT[rt], gap, 7)
    q, qw = spaced(n_tok, n, F8, gap + (-(n + gap)) % 16, 3)
    s = torch.zeros(-(-n // 128), n_tok, device="cuda")
    y = spaced(n_tok, n, DT[xt], gap, 5)[0] if plain else None
    B.stage_op_norm_f8(xd, q, s, None if gamma is None else dev(gamma), eps, rd, ro, y)
    torch.cuda.synchronize()
    if gap:
        assert (qw[:, n:].float() == 3).all()
    return ro, q, s, y


def check_norm(B, x, resid, gamma, xt="f32", rt="f32", **kw):
    x = given(x, xt)
    resid = None if resid is None else given(resid, rt)
    ro, q, s, y = run_norm(B, x, resid, gamma, xt, rt, **kw)
    store = lambda h: torch.as_tensor(h).to(DT[rt]).float().numpy()   # noqa: E731
    h, yy, codes, scales = step.norm_f8(x, resid, gamma, kw.get("eps", 1e-5), store)
    if resid is not None:
        same(ro.float().cpu().numpy(), h)
    table = step.e4m3_values()
    same(s.cpu().numpy(), scales)
    got = q.contiguous().view(torch.uint8).cpu().numpy()
    assert np.array_equal(np.signbit(table[got]), np.signbit(table[codes])) or np.isnan(table[codes]).any()
    same(table[got], table[codes])
    if y is not None:
        same(y.float().cpu().numpy(), torch.as_tensor(yy).to(DT[xt]).float().numpy())


@pytest.mark.parametrize("xt,rt", [("f32", None), ("f32", "f32"), ("bf16", None), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f16", None)])
@pytest.mark.parametrize("n_tok,n,gap", [(1, 128, 0), (3, 256, 0), (5, 688, 8), (7, 1000, 4), (2, 127, 1), (3, 1, 3), (9, 129, 7), (2, 4096, 0), (2, 8192, 16), (1, 28672, 0),
                                         (3, 32768, 0), (2, 14337, 1), (130, 512, 0)])
def test_norm_is_exact(B, xt, rt, n_tok, n, gap):
    rng = np.random.default_rng(n_tok * 100003 + n)
    x = rng.standard_normal((n_tok, n)) * 10.0 ** rng.uniform(-3, 3, (n_tok, 1))
    resid = None if rt is None else rng.standard_normal((n_tok, n)) * (1 + 50 * (rng.random(n) < 0.02))
    gamma = (1 + 0.3 * rng.standard_normal(n)).astype(np.float32)
    if n > 300:
        gamma[128:256] = 0                        # a block of zeros
        gamma[256] = 3e30
    check_norm(B, x, resid, gamma, xt, rt or "f32", gap=gap, plain=n % 2 == 0, inplace=n == 256)


@pytest.mark.parametrize("xt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n_tok,n", [(4, 256), (3, 1000), (2, 28672), (6, 77)])
def test_rows_quantised_as_they_are(B, xt, n_tok, n):
    rng = np.random.default_rng(n)
    x = rng.standard_normal((n_tok, n)) * 10.0 ** rng.integers(-7, 4, (n_tok, n))
    x[0, :64] = 0
    x[1] *= 1e-6
    check_norm(B, x, None, None, xt)
    check_norm(B, x, x[::-1], None, xt, xt)


def test_norm_of_zeros_tiny_huge_and_no_numbers(B):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((9, 384)).astype(np.float32)
    x[0] = 0
    x[1] *= 1e-30
    x[2, 5], x[3, 200], x[4, 0] = np.nan, np.inf, -np.inf
    x[5] *= 1e18                                  # sum of squares just below float32's end
    x[6] *= 1e25                                  # and beyond it
    x[7, 1:] = 0
    with np.errstate(all="ignore"):
        check_norm(B, x, None, np.ones(384, np.float32))
        check_norm(B, x, None, None)
        check_norm(B, x, None, np.ones(384, np.float32), eps=0.25)
    g = np.ones(384, np.float32)
    g[130] = np.nan
    check_norm(B, x[7:], None, g)


@pytest.mark.parametrize("xt,rt", [("f32", None), ("f32", "f32"), ("bf16", None), ("bf16", "f32")])
@pytest.mark.parametrize("n", [100, 384, 4096, 8191, 8192, 14336, 28672])
def test_norm_of_tiny_rows_and_huge_ones(B, xt, rt, n):
    """Means whose squares, roots or squared roots leave float32's range: no eps, or one as small."""
    rng = np.random.default_rng(n)
    sizes = 10.0 ** np.array([-12.0, -13.5, -14, -18, -19, -19.5, -20, -22, -24, -30, -37, -38.5, -40, -43, 13, 14, 15, 16.5])
    x = rng.standard_normal((len(sizes), n)) * sizes[:, None]
    x[5, 1:] = 0                                  # one number among zeros
    resid = None if rt is None else rng.standard_normal(x.shape) * sizes[:, None]
    gamma = (1 + 0.3 * rng.standard_normal(n)).astype(np.float32)
    for eps in (0.0, 1e-42, 3e-38, 1e-30, 2.0 ** -90, 1e-20):
        with np.errstate(all="ignore"):
            check_norm(B, x, resid, gamma, xt, rt or "f32", eps=eps)
    zero = np.zeros((5, n))
    with np.errstate(all="ignore"):
        check_norm(B, zero, None, gamma, xt)
        check_norm(B, zero, None, gamma, xt, eps=1e-42)
        check_norm(B, zero, None, gamma, xt, eps=0.0)      # 0 / 0


def test_norm_up_to_the_last_sum_of_squares(B):
    """Sums of squares on both sides of 2^128, and an eps that takes their mean beyond it."""
    n = 256
    x = np.zeros((5, n), np.float32)
    for i, at in enumerate((0.5, 0.999, 1.01, 0.97, 3.0)):
        x[i] = np.sqrt(at * 2.0 ** 128 / n)
        x[i, ::2] *= -1
    sums = (x.astype(np.float64) ** 2).sum(1)
    assert (sums[[0, 1, 3]] < 2.0 ** 128).all() and (sums[[2, 4]] > 2.0 ** 128).all()
    for eps in (1e-5, 1e38, 3.4e38):
        with np.errstate(all="ignore"):
            check_norm(B, x, None, np.ones(n, np.float32), eps=eps)
            y = run_norm(B, x, None, np.ones(n, np.float32), "f32", "f32", eps=eps)[3]
        assert torch.isnan(y).all(1).tolist() == [False, False, True, False, True]


def test_norm_ties_of_the_codes(B):
    """Every value halfway between two codes, at a scale of one."""
    v = step.e4m3_values()[:127]
    mids = np.concatenate([(v[1:] + v[:-1]) / 2, v])
    mids = np.concatenate([mids, -mids])
    x = np.zeros((1, 128 * 8), np.float32)
    for b in range(8):
        part = mids[b * 64: b * 64 + 64]
        x[0, 128 * b: 128 * b + len(part)] = part
        x[0, 128 * b + 100] = 448
    check_norm(B, x, None, None)


def test_norm_only_plain_and_only_codes_and_no_rows(B):
    x = torch.randn(3, 640, device="cuda")
    y = torch.zeros_like(x)
    B.stage_op_norm_f8(x, gamma=torch.ones(640, device="cuda"), y=y)
    want = step.norm_f8(x.cpu().numpy(), None, np.ones(640, np.float32))[1]
    same(y.cpu().numpy(), want)
    B.stage_op_norm_f8(x[:0], torch.zeros(0, 640, dtype=F8, device="cuda"), torch.zeros(5, 0, device="cuda"))


# ------------------------------------------------------------------------------------------- product

def random_f8(rng, n, k, wide=1.0):
    """Codes without NaN, their distribution that of quantised normal rows; a few rows are full-scale."""
    x = rng.standard_normal((n, k)) * 100 * wide
    x[:: 7] = rng.uniform(-448, 448, x[:: 7].shape)
    return step.e4m3_codes(x)


def put_f8(codes, gap=0):
    n, k = codes.shape
    whole = torch.full((n, k + (-k) % 16 + gap), 0x7F, dtype=torch.uint8, device="cuda")   # NaN beside the rows
    whole[:, :k] = torch.as_tensor(codes)
    return whole.view(F8)[:, :k]


def check_gemm(B, a, sa, w, sw, dtype="f32", gap=0, ygap=0, rows=None):
    M, N = a.shape[0], w.shape[0]
    y, whole = spaced(M, N, DT[dtype], ygap, 9)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.stage_op_f8_gemm(put_f8(a, gap), dev(sa), put_f8(w, gap), dev(sw), y, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    if ygap:
        assert (whole[:, N:] == 9).all()
    at = slice(None) if rows is None else rows
    want, mag = step.f8_gemm(a[at], sa[:, at], w, sw)
    close(y[at], want, (2.0 ** -16 + (len(sa) + 3) * 2.0 ** -24) * mag + half_step(want, dtype))
    return y


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (1, 1, 1), (2, 130, 300), (3, 256, 1000), (7, 1001, 688), (8, 4096, 256), (16, 512, 2048), (17, 300, 129), (33, 640, 4096), (64, 1024, 1024),
                                   (65, 257, 513), (100, 2000, 16), (127, 383, 900), (128, 256, 128), (129, 513, 640), (200, 1500, 1300), (256, 512, 4096), (333, 777, 2500), (700, 128, 96)])
def test_product(B, dtype, M, N, K):
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    nb, kb = -(-N // 128), -(-K // 128)
    sa = (10.0 ** rng.uniform(-4, 0, (kb, M))).astype(np.float32) * (1e-3 if dtype == "f16" else 1)
    sw = (10.0 ** rng.uniform(-4, -1, (nb, kb))).astype(np.float32)
    check_gemm(B, random_f8(rng, M, K), sa, random_f8(rng, N, K), sw, dtype, gap=16 * (M % 3), ygap=M % 4)


@pytest.mark.parametrize("M,N,K", [(513, 12801, 300), (1000, 10300, 512), (300, 30000, 100), (12, 9856, 700), (16, 9728, 300), (9, 9729, 300), (12, 39040, 300), (20, 39040, 140), (40, 39040, 300),
                                   (64, 38912, 200), (33, 38913, 200)])
def test_product_of_wide_weights(B, M, N, K):
    """Several tiles of 256 x 256 for each pair of SMs, with an odd and an even number of blocks; few rows by more weight tiles than SMs, and than two
    or three CTAs of each hold."""
    rng = np.random.default_rng(M + N + K)
    nb, kb = -(-N // 128), -(-K // 128)
    sa, sw = rng.uniform(0.1, 1, (kb, M)).astype(np.float32), rng.uniform(0.1, 1, (nb, kb)).astype(np.float32)
    a, w = random_f8(rng, M, K), random_f8(rng, N, K)
    check_gemm(B, a, sa, w, sw, "f32", ygap=M % 2)
    check_gemm(B, a, sa, w, sw, "bf16", gap=16)


@pytest.mark.parametrize("M,N", [(1, 512), (8, 300), (12, 512), (12, 9856), (30, 512), (60, 400), (100, 512), (200, 600), (1024, 700)])
def test_product_loses_no_bits_of_a_block(B, M, N):
    """Whole numbers whose sums over a block stay below 2^24 (128 * 240^2 < 2^23): float32 holds each of them, in any order."""
    t = step.e4m3_values()
    whole = np.array([c for c in range(256) if t[c] == t[c] and t[c] == int(t[c]) and abs(t[c]) <= 240], np.uint8)
    small = whole[np.abs(t[whole]) <= 3]
    rng = np.random.default_rng(M)
    for first in (False, True):
        a, w = rng.choice(whole, (M, 128)), rng.choice(whole, (N, 128))
        if first:                                    # one product of 240^2 beside small ones
            a[:, 1:], a[:, 0], w[:, 0] = rng.choice(small, (M, 127)), 0x77, 0x77
        y = torch.zeros(M, N, device="cuda")
        B.stage_op_f8_gemm(put_f8(a), torch.ones(1, M, device="cuda"), put_f8(w), torch.ones(-(-N // 128), 1, device="cuda"), y)
        want = t[a] @ t[w].T
        assert (want % 2 != 0).any() and np.abs(want).max() > 2.0 ** 15
        same(y.double().cpu().numpy(), want)


def test_product_of_exact_numbers(B):
    """Small whole numbers with powers of two as scales: every sum is exact, whatever its order, so the result is too."""
    rng = np.random.default_rng(5)
    for M, N, K in ((5, 300, 700), (70, 129, 1500), (300, 400, 640)):
        a, w = (step.e4m3_codes(rng.integers(-8, 9, (n, K))) for n in (M, N))
        sa, sw = (2.0 ** rng.integers(-3, 3, s).astype(np.float32) for s in ((-(-K // 128), M), (-(-N // 128), -(-K // 128))))
        y = torch.zeros(M, N, device="cuda")
        B.stage_op_f8_gemm(put_f8(a), dev(sa), put_f8(w), dev(sw), y)
        same(y.double().cpu().numpy(), step.f8_gemm(a, sa, w, sw)[0])


def test_product_every_tile_edge(B):
    """One row and one column of ones in turn: each output is one known element, so no tile, half or swizzled place is swapped."""
    rng = np.random.default_rng(6)
    K = 400
    for M, N in ((40, 300), (300, 600)):
        w = random_f8(rng, N, K)
        a = np.zeros((M, K), np.uint8)
        pick = rng.integers(0, K, M)
        a[np.arange(M), pick] = 0x38            # 1.0
        sa, sw = np.ones((4, M), np.float32), np.ones((-(-N // 128), 4), np.float32)
        y = torch.zeros(M, N, device="cuda")
        B.stage_op_f8_gemm(put_f8(a), dev(sa), put_f8(w), dev(sw), y)
        same(y.double().cpu().numpy(), step.e4m3_values()[w][:, pick].T)


@pytest.mark.parametrize("M,N", [(5, 300), (12, 9856), (40, 300), (100, 300), (300, 700)])
def test_product_of_scales_at_the_ends_of_float32(B, M, N):
    """The scales' product is one float32: 2^-140 is held, 2^130 is not."""
    rng = np.random.default_rng(M)
    a, w = (step.e4m3_codes(rng.integers(-8, 9, (n, 128))) for n in (M, N))
    sa, sw = np.full((1, M), 2.0 ** -100, np.float32), np.full((-(-N // 128), 1), 2.0 ** -40, np.float32)
    sa[0, 1], sa[0, 2] = 2.0 ** 100, 2.0 ** -20           # 2^60, and 2^-60
    sw[1] = 2.0 ** 30                                     # 2^-70; 2^130 in the first of these rows
    y = torch.zeros(M, N, device="cuda")
    B.stage_op_f8_gemm(put_f8(a), dev(sa), put_f8(w), dev(sw), y)
    got = y.double().cpu().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        factor = (sa.T * np.repeat(sw[:, 0], 128)[:N][None]).astype(np.float32).astype(np.float64)
        want = step.f8_gemm(a, np.ones_like(sa), w, np.ones_like(sw))[0] * factor
    assert np.isinf(factor[1, 128]) and 0 < factor[0, 0] < 2.0 ** -139
    same(got, want)


def test_product_keeps_rows_apart(B):
    """NaN in one row or weight row, infinite or zero scales: nothing else changes."""
    rng = np.random.default_rng(7)
    for M, N, K in ((9, 400, 500), (200, 600, 500)):
        a, w = random_f8(rng, M, K), random_f8(rng, N, K)
        a[3, 77], w[130, 400] = 0x7F, 0xFF
        sa, sw = np.full((4, M), 0.5, np.float32), np.full((-(-N // 128), 4), 0.25, np.float32)
        sa[2, 5], sa[:, 7], sw[2, 1] = np.inf, 0, np.nan
        y = torch.zeros(M, N, device="cuda")
        B.stage_op_f8_gemm(put_f8(a), dev(sa), put_f8(w), dev(sw), y)
        got = y.double().cpu().numpy()
        with np.errstate(all="ignore"):
            clean = step.f8_gemm(a, sa, w, sw)
        assert np.isnan(got[3]).all() and np.isnan(got[:, 130]).all() and np.isnan(got[:, 256:384]).all()
        rows = [m for m in range(M) if m not in (3, 5)]
        cols = [n for n in range(N) if n != 130 and not 256 <= n < 384]
        at = np.ix_(rows, cols)
        close(got[at], clean[0][at], (2.0 ** -16 + 7 * 2.0 ** -24) * clean[1][at])
        assert (got[7][cols] == 0).all() and not np.isfinite(got[5][cols]).any()


@pytest.mark.parametrize("M", [1, 50, 90, 300, 1111])
def test_product_is_repeatable_and_long(B, M):
    rng = np.random.default_rng(M)
    K, N = 14336, 1280
    a, w = random_f8(rng, M, K), random_f8(rng, N, K)
    sa, sw = rng.uniform(0.5, 1, (112, M)).astype(np.float32), rng.uniform(0.5, 1, (10, 112)).astype(np.float32)
    rows = np.unique(np.r_[0, M // 2, M - 1])
    first = check_gemm(B, a, sa, w, sw, "f32", rows=rows).clone()
    again = check_gemm(B, a, sa, w, sw, "f32", rows=rows)
    assert torch.equal(first, again)


@pytest.mark.parametrize("M,N,K", [(300, 1, 200), (17, 1, 50), (129, 100, 1100), (1, 5000, 16), (16, 17, 33), (256, 300, 2048), (512, 256, 1024)])
def test_product_of_narrow_weights_and_shared_k(B, M, N, K):
    rng = np.random.default_rng(M + N)
    sa, sw = rng.uniform(0.1, 1, (-(-K // 128), M)).astype(np.float32), rng.uniform(0.1, 1, (-(-N // 128), -(-K // 128))).astype(np.float32)
    for dtype, ygap in (("f32", 0), ("bf16", 3)):
        check_gemm(B, random_f8(rng, M, K), sa, random_f8(rng, N, K), sw, dtype, ygap=ygap)


def test_product_rows_do_not_depend_on_their_neighbours(B):
    """The same row in calls of other rows: within a kernel's range of M the same bits, and beside NaN rows too."""
    rng = np.random.default_rng(12)
    K, N = 1536, 640
    w, sw = put_f8(random_f8(rng, N, K)), dev(rng.uniform(0.1, 1, (5, 12)).astype(np.float32))
    for M in (7, 15, 50, 100, 400):
        a, sa = random_f8(rng, M, K), rng.uniform(0.1, 1, (12, M)).astype(np.float32)
        y, z = torch.zeros(M, N, device="cuda"), torch.zeros(M, N, device="cuda")
        B.stage_op_f8_gemm(put_f8(a), dev(sa), w, sw, y)
        b = a.copy()
        b[: M // 2] = 0x7F
        B.stage_op_f8_gemm(put_f8(b), dev(sa), w, sw, z)
        assert torch.isnan(z[: M // 2]).all() and torch.equal(y[M // 2:], z[M // 2:])


def test_product_that_runs_out_of_time(B):
    rng = np.random.default_rng(8)
    for M in (5, 300):
        a, w = random_f8(rng, M, 500), random_f8(rng, 700, 500)
        sa, sw = np.ones((4, M), np.float32), np.ones((6, 4), np.float32)
        y = torch.zeros(M, 700, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        B.stage_op_f8_debug_stall(1)
        B.stage_op_f8_gemm(put_f8(a), dev(sa), put_f8(w), dev(sw), y, err)
        torch.cuda.synchronize()
        assert err.item() == 1 and torch.isnan(y).all()
        check_gemm(B, a, sa, w, sw)                # the next one is as ever


@pytest.mark.parametrize("M,N,K", [(513, 12801, 300), (256, 512, 4096), (130, 300, 3200), (100, 700, 500), (40, 1300, 1500)])
def test_product_that_runs_out_of_time_with_many_tiles_or_a_shared_k(B, M, N, K):
    """(More tiles than pairs; K over two pairs, over a cluster's CTAs.)"""
    rng = np.random.default_rng(M)
    a, w = put_f8(random_f8(rng, M, K)), put_f8(random_f8(rng, N, K))
    sa, sw = torch.ones(-(-K // 128), M, device="cuda"), torch.ones(-(-N // 128), -(-K // 128), device="cuda")
    y, z = torch.zeros(M, N, device="cuda"), torch.zeros(M, N, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.stage_op_f8_debug_stall(1)
    B.stage_op_f8_gemm(a, sa, w, sw, y, err)
    torch.cuda.synchronize()
    assert err.item() == 1 and torch.isnan(y).all()
    err.zero_()
    B.stage_op_f8_gemm(a, sa, w, sw, y, err)
    B.stage_op_f8_gemm(a, sa, w, sw, z)
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(y, z)


@pytest.mark.parametrize("K", [200, 384])
def test_product_that_comes_too_late(B, K):
    """A product that completes after its readers have given up: it is not taken for the next tile's.  Three tiles or more for each pair."""
    rng = np.random.default_rng(K)
    M, N = 1000, 15360
    kb = -(-K // 128)
    ac, wc = random_f8(rng, M, K), random_f8(rng, N, K)
    sa, sw = rng.uniform(0.5, 1, (kb, M)).astype(np.float32), rng.uniform(0.5, 1, (120, kb)).astype(np.float32)
    a, w = put_f8(ac), put_f8(wc)
    y = torch.zeros(M, N, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.stage_op_f8_debug_late(1)
    B.stage_op_f8_gemm(a, dev(sa), w, dev(sw), y, err)
    torch.cuda.synchronize()
    assert err.item() == 1
    got = y.double().cpu().numpy()
    want, mag = step.f8_gemm(ac, sa, wc, sw)
    some = ~np.isnan(got)
    assert some.any() and not some.all()
    err = np.abs(got - want)[some] / ((2.0 ** -16 + (kb + 3) * 2.0 ** -24) * mag)[some]
    assert (err <= 1).all(), (err > 1).mean()
    check_gemm(B, ac, sa, wc, sw)              # the next one is as ever


# ------------------------------------------------------------------------------------------- rope

def check_rope(B, q, k, pos, freqs, dtype="f32", interleaved=False, scale=1.0, gap=0, inplace=False):
    n, hq, d = q.shape
    q, k = given(q, dtype), None if k is None else given(k, dtype)
    hk = 0 if k is None else k.shape[1]
    whole = torch.full((n, (hq + hk) * d + gap), 0, dtype=DT[dtype], device="cuda")
    qd = whole[:, : hq * d].unflatten(1, (hq, d))
    kd = whole[:, hq * d: (hq + hk) * d].unflatten(1, (hk, d)) if hk else None
    qd.copy_(torch.as_tensor(q))
    qo, ko = qd, kd
    if hk:
        kd.copy_(torch.as_tensor(k))
    if not inplace:
        qo, ko = (None if not h else torch.full((n, h, d), 7.0, dtype=DT[dtype], device="cuda") for h in (hq, hk))
    fd = dev(np.asarray(freqs, np.float64))
    if inplace:
        B.stage_op_rope(qd, kd, i32(pos), fd, interleaved=interleaved, scale=scale)
    else:
        B.stage_op_rope(qd, kd, i32(pos), fd, qo, ko, interleaved, scale)
    torch.cuda.synchronize()
    pos, live = np.asarray(pos), np.asarray(pos) >= 0
    r = 2 * len(freqs)
    for x, got in ((q, qo), (k, ko)):
        if x is None:
            continue
        got = got.double().cpu().numpy()
        same(got[~live], x[~live] if inplace else np.full_like(x[~live], 7.0))
        want = step.rope(x[live], pos[live], freqs, interleaved, scale)
        same(got[live][..., r:], x[live][..., r:])
        at = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
        size = np.abs(x[live][..., at[0]]) + np.abs(x[live][..., at[1]])
        tol = size * abs(scale) * (2.0 ** -21 + pos[live][:, None, None] * np.abs(freqs) * 2.0 ** -51)
        for part in at:
            close(got[live][..., part], want[..., part], tol + half_step(want[..., part], dtype))
    if gap:
        assert (whole[:, (hq + hk) * d:] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hk,d,rot,gap", [(1, 4, 2, 64, 64, 0), (3, 32, 8, 128, 128, 8), (70, 7, 1, 80, 80, 16), (5, 2, 2, 80, 20, 0), (17, 3, 1, 96, 48, 8), (4, 5, 0, 128, 32, 0),
                                               (2, 1, 1, 2, 2, 0), (6, 3, 2, 7, 6, 1), (9, 2, 1, 256, 64, 3), (2, 2, 1, 1024, 1024, 0), (1000, 2, 1, 64, 64, 0), (2500, 8, 2, 64, 32, 8),
                                               (1, 64, 8, 128, 128, 0), (33, 1, 1, 24, 8, 0)])
def test_rope(B, dtype, interleaved, n, hq, hk, d, rot, gap):
    rng = np.random.default_rng(n * 17 + d + rot)
    q, k = rng.standard_normal((n, hq, d)), rng.standard_normal((n, hk, d)) if hk else None
    pos = rng.integers(0, 5000, n)
    pos[:: 5] = rng.integers(0, 2 ** 31 - 1, len(pos[:: 5]))
    if n > 4:
        pos[[1, 3]] = [-1, -2 ** 31]
        pos[4] = 0
    f, s = step.rope_freqs(rot, 10000.0, "parts" if rot > 16 else "plain", 8.0, 4096.0)
    check_rope(B, q, k, pos, f, dtype, interleaved, s, gap, inplace=n % 2 == 0)


def test_rope_positions_from_zero_to_the_last(B):
    """Quadrants and their borders: turns of an exact eighth, and the far end."""
    rng = np.random.default_rng(3)
    f = 2 * np.pi / np.array([8.0, 16.0, 7.0, 1.0, 2.0 ** 31, 3.0, 64.0, 4.0])
    pos = np.concatenate([np.arange(80), 2 ** 31 - 1 - np.arange(20)])
    check_rope(B, rng.standard_normal((100, 2, 16)), rng.standard_normal((100, 1, 16)), pos, f)
    check_rope(B, rng.standard_normal((100, 2, 16)), None, pos, -f, interleaved=True, scale=-0.5)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,n,hq,hk,d,rot", [("f32", 6000, 2, 1, 64, 64), ("bf16", 6000, 2, 1, 64, 32), ("f16", 11003, 1, 0, 24, 8), ("f32", 5200, 1, 0, 1024, 1024), ("bf16", 5200, 1, 0, 1024, 512),
                                                 ("f32", 5200, 1, 0, 301, 150), ("f32", 15000, 1, 1, 6, 4)])
def test_rope_of_more_tokens_than_warps(B, dtype, interleaved, n, hq, hk, d, rot):
    """A warp goes from token to token, padding among them: each token has its own cos and sin, in heads of more than 32 vectors too."""
    rng = np.random.default_rng(n + d)
    q, k = rng.standard_normal((n, hq, d)), rng.standard_normal((n, hk, d)) if hk else None
    pos = rng.integers(0, 100000, n)
    pos[rng.random(n) < 0.2] = -1
    f, _ = step.rope_freqs(rot, 10000.0)
    check_rope(B, q, k, pos, f, dtype, interleaved, 1.25, inplace=n % 1000 != 0)


def test_rope_of_negative_frequencies_at_the_last_positions(B):
    """Turning backwards is as exact as turning forwards: small frequencies times positions next to 2^31."""
    rng = np.random.default_rng(5)
    f = -10.0 ** rng.uniform(-9, 0, 128)
    pos = 2 ** 31 - 1 - rng.integers(0, 1000, 50)
    q, k = rng.standard_normal((50, 4, 256)), rng.standard_normal((50, 2, 256))
    check_rope(B, q, k, pos, f)
    check_rope(B, q, k, pos, f, interleaved=True)
    check_rope(B, q, k, pos, -f)


def test_rope_of_no_numbers_and_padding_only(B):
    x = np.random.default_rng(1).standard_normal((3, 2, 64))
    x[1, 0, 3], x[2, 1, 40] = np.nan, np.inf
    f, _ = step.rope_freqs(64, 10000.0)
    q = dev(x, torch.float32)
    B.stage_op_rope(q, None, i32([4, 5, 6]), dev(f))
    with np.errstate(invalid="ignore"):
        want = step.rope(x, [4, 5, 6], f)
    assert np.array_equal(np.isfinite(q.cpu().numpy()), np.isfinite(want))
    before = q.clone()
    B.stage_op_rope(q, q, i32([-1, -1, -5]), dev(f))
    assert torch.equal(q.view(torch.int32), before.view(torch.int32))


# ------------------------------------------------------------------------------------------- log probabilities

def check_logprobs(B, z, tokens, top, dtype="f32", gap=0, shift=0):
    n, vocab = z.shape
    z = given(z, dtype)
    flat = torch.full((n * (vocab + gap) + shift + 64,), float("nan"), dtype=DT[dtype], device="cuda")   # what lies beside the rows is no logit
    zd = flat[shift: shift + n * (vocab + gap)].view(n, vocab + gap)[:, :vocab]
    zd.copy_(torch.as_tensor(z))
    lp, h = (torch.full((n,), 7.0, device="cuda") for _ in range(2))
    rank = torch.full((n,), 7, dtype=torch.int32, device="cuda")
    ids = torch.full((n, top), 7, dtype=torch.int32, device="cuda")
    best = torch.full((n, top), 7.0, device="cuda")
    B.stage_op_logprobs(zd, i32(tokens), lp, h, rank, ids if top else None, best if top else None)
    torch.cuda.synchronize()
    w = step.logprobs(z, tokens, top)
    same(rank.cpu().numpy(), w["rank"])
    same(ids.cpu().numpy(), w["ids"])
    L = vocab / 256 + 64
    base = 2.0 ** -20 + L * 2.0 ** -24 + 2.0 ** -22 * w["away"]
    with np.errstate(invalid="ignore"):
        close(lp, w["logprob"], base + 2.0 ** -23 * (w["drop"] + np.abs(w["logprob"])))
        close(best, w["best"], base[:, None] + 2.0 ** -23 * (w["fall"] + np.abs(w["best"])))
        close(h, w["entropy"], (2.0 ** -19 + L * 2.0 ** -23) * (1 + w["away"]) + 2.0 ** -15 * w["away"])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,vocab,top,gap,shift", [(1, 1, 1, 0, 0), (3, 2, 2, 1, 1), (5, 17, 17, 0, 3), (4, 33, 32, 5, 0), (2, 1000, 20, 0, 7), (7, 1024, 0, 0, 0), (3, 4099, 5, 1, 2), (2, 32000, 1, 0, 0),
                                                   (1, 50257, 20, 0, 0), (3, 50257, 8, 0, 5), (2, 151936, 32, 0, 0), (1, 262144, 3, 3, 1), (400, 700, 2, 0, 0), (20, 128256, 5, 0, 0),
                                                   (1, 524288, 32, 0, 0)])
def test_logprobs(B, dtype, n, vocab, top, gap, shift):
    rng = np.random.default_rng(vocab + n)
    z = rng.standard_normal((n, vocab)) * 3 + rng.uniform(-20, 20, (n, 1))
    z[:, rng.integers(0, vocab, 2)] += 12
    if vocab > 100:
        z[:, 3:: 11] = -np.inf
        z[:, 5:: 13] = float(torch.finfo(DT[dtype]).min)
    tokens = rng.integers(0, vocab, n)
    tokens[0] = z[0].argmax()
    if n > 2:
        tokens[1], tokens[2] = -1, vocab
    check_logprobs(B, z, tokens, top, dtype, gap, shift)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [40, 5000, 70001])
def test_logprobs_of_equal_logits(B, dtype, vocab):
    """Ties, through every chunk, thread and CTA: the lowest ids first."""
    rng = np.random.default_rng(vocab)
    low = float(torch.finfo(DT[dtype]).min)
    z = np.stack([np.zeros(vocab), np.full(vocab, -3.0), np.full(vocab, low), rng.integers(0, 3, vocab), rng.integers(-1, 1, vocab) * 1.0, np.where(np.arange(vocab) == vocab - 1, 1.0, -np.inf),
                  np.where(np.arange(vocab) % 9 == 4, -np.inf, low)])
    z[4][z[4] == 0] *= rng.choice([-1.0, 1.0], (z[4] == 0).sum())     # -0 and 0 are equal
    check_logprobs(B, z, rng.integers(0, vocab, len(z)), 32, dtype)


@pytest.mark.parametrize("vocab,top", [(300, 4), (40000, 20), (151936, 0)])
def test_rows_without_a_distribution(B, vocab, top):
    rng = np.random.default_rng(vocab)
    z = rng.standard_normal((8, vocab))
    z[0, vocab // 2], z[1, vocab - 1], z[2] = np.nan, np.inf, -np.inf
    z[3, 0], z[3, 7], z[4, 5] = np.nan, np.inf, -np.nan
    z[5, 1:], z[6, : vocab - 1] = -np.inf, -np.inf       # one token left: log p = 0
    check_logprobs(B, z, [1, 2, 3, 4, 5, 0, 0, 9], top)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_logprobs_rising_and_falling(B, dtype):
    """Every chunk raises the maximum, or none does."""
    vocab = 33000
    up = np.linspace(-60, 60, vocab)
    check_logprobs(B, np.stack([up, up[::-1], up * 100 if dtype == "f32" else up]), [vocab - 1, 5, 17], 32, dtype)


@pytest.mark.parametrize("rows,vocab,top", [(1, 5000, 32), (160, 20000, 20), (2, 100000, 32), (160, 100003, 5)])
def test_logprobs_with_the_best_in_few_places(B, rows, vocab, top):
    """The likeliest tokens all in one thread's chunks, all but one group's, or in one chunk: the first bound is too low, or its chunks many."""
    rng = np.random.default_rng(vocab)
    place = np.arange(vocab) // 8                    # 32 bytes of float32
    z = rng.standard_normal((rows, vocab))
    for i in range(rows):
        kind, nt = i % 5, 256 if i % 2 else 512
        if kind == 0:
            z[i] += 30 * (place % nt == 3)
        elif kind == 1:
            z[i] -= 200 * (place % nt < 8)
        elif kind == 2:
            z[i] += 50 * (place == vocab // 16) + 40 * (place == vocab // 9)
        elif kind == 3:
            z[i] = np.where(place % nt == 7, 5.0, -5.0)
        else:
            z[i] += 30 * (place % nt < 2) + 0.01 * np.arange(vocab)
    check_logprobs(B, z, rng.integers(0, vocab, rows), top)


def test_logprobs_without_tokens_or_some_outputs(B):
    z = torch.randn(5, 3000, device="cuda")
    w = step.logprobs(z.cpu().numpy(), None, 3)
    ids = torch.zeros(5, 3, dtype=torch.int32, device="cuda")
    B.stage_op_logprobs(z, top_ids=ids)
    same(ids.cpu().numpy(), w["ids"])
    h = torch.zeros(5, device="cuda")
    B.stage_op_logprobs(z, entropy=h)
    close(h, w["entropy"], 1e-4)
    best = torch.zeros(5, 3, device="cuda")
    B.stage_op_logprobs(z, top_logprobs=best)
    close(best, w["best"], 1e-5)
    B.stage_op_logprobs(z[:0])


# ------------------------------------------------------------------------------------------- streams, graphs, a step

def test_other_streams_and_graphs(B):
    """Captured calls replayed with other inputs, and calls of two streams at once, give what single ones give."""
    torch.manual_seed(0)
    M, K, N, V = 40, 1024, 768, 9000
    x, g = torch.randn(M, K, device="cuda"), torch.ones(K, device="cuda")
    w = put_f8(random_f8(np.random.default_rng(1), N, K))
    sw = torch.rand(6, 8, device="cuda")
    z = torch.randn(M, V, device="cuda")
    pos = torch.arange(M, dtype=torch.int32, device="cuda")
    f = dev(step.rope_freqs(128, 10000.0)[0])

    def buffers():
        return dict(q=torch.zeros(M, K, dtype=F8, device="cuda"), s=torch.zeros(8, M, device="cuda"), y=torch.zeros(M, N, device="cuda"), r=torch.zeros(M, 6, 128, device="cuda"),
                    lp=torch.zeros(M, device="cuda"), ids=torch.zeros(M, 9, dtype=torch.int32, device="cuda"))

    def go(b, stream=None):
        B.stage_op_norm_f8(x, b["q"], b["s"], g, stream=stream)
        B.stage_op_f8_gemm(b["q"], b["s"], w, sw, b["y"], stream=stream)
        B.stage_op_rope(b["y"].view(M, 6, 128), None, pos, f, b["r"], stream=stream)
        B.stage_op_logprobs(z, pos, b["lp"], top_ids=b["ids"], stream=stream)

    def equal(a, b):
        return all(torch.equal(a[k].view(torch.uint8) if a[k].dtype is F8 else a[k], b[k].view(torch.uint8) if b[k].dtype is F8 else b[k]) for k in a)

    want, got = buffers(), buffers()
    go(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(got)
    for _ in range(3):
        x.normal_()
        z.normal_()
        graph.replay()
        go(want)
        torch.cuda.synchronize()
        assert equal(want, got)
    streams, many = [torch.cuda.Stream() for _ in range(4)], [buffers() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, b in zip(streams, many):
            go(b, st)
    torch.cuda.synchronize()
    assert all(equal(want, b) for b in many)


@pytest.mark.parametrize("M", [3, 12, 30, 200, 600])
def test_products_of_every_kernel_captured_and_at_once(B, M):
    rng = np.random.default_rng(M)
    K, N = 2048, 768
    w, sw = put_f8(random_f8(rng, N, K)), dev(rng.uniform(0.1, 1, (6, 16)).astype(np.float32))
    inputs = [(put_f8(random_f8(rng, M, K)), dev(rng.uniform(0.1, 1, (16, M)).astype(np.float32))) for _ in range(3)]
    want = [torch.zeros(M, N, dtype=torch.bfloat16, device="cuda") for _ in inputs]
    for (a, s), y in zip(inputs, want):
        B.stage_op_f8_gemm(a, s, w, sw, y)
    a, s = inputs[0][0].clone(), inputs[0][1].clone()
    y = torch.zeros_like(want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.stage_op_f8_gemm(a, s, w, sw, y)
    for (b, r), expected in zip(inputs, want):
        a.view(torch.uint8).copy_(b.view(torch.uint8))
        s.copy_(r)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, expected)
    streams, outs = [torch.cuda.Stream() for _ in inputs], [torch.zeros_like(y) for _ in inputs]
    torch.cuda.synchronize()
    for _ in range(8):
        for st, (b, r), o in zip(streams, inputs, outs):
            B.stage_op_f8_gemm(b, r, w, sw, o, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, e) for o, e in zip(outs, want))


def test_products_right_behind_one_another(B):
    """CTAs of one call on SMs that others have just left: what these had in flight is done (the arrivals of a pair come to both its CTAs)."""
    rng = np.random.default_rng(3)
    calls = []
    for M, N, K in ((300, 700, 384), (40, 700, 384), (1024, 5120, 128), (256, 512, 3200), (100, 300, 640), (12, 9856, 256), (2, 600, 384), (129, 257, 64)):
        sa, sw = dev(rng.uniform(0.5, 1, (-(-K // 128), M)).astype(np.float32)), dev(rng.uniform(0.5, 1, (-(-N // 128), -(-K // 128))).astype(np.float32))
        calls.append((put_f8(random_f8(rng, M, K)), sa, put_f8(random_f8(rng, N, K)), sw, torch.zeros(M, N, device="cuda")))
    want = []
    for c in calls:
        B.stage_op_f8_gemm(*c)
        torch.cuda.synchronize()
        want.append(c[-1].clone())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in rng.integers(0, len(calls), 200):
            B.stage_op_f8_gemm(*calls[i], err)
        for c in calls:
            B.stage_op_f8_gemm(*c, err)
    for _ in range(5):
        for c in calls:
            c[-1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert err.item() == 0 and all(torch.equal(c[-1], w) for c, w in zip(calls, want))


def test_first_calls_inside_a_capture(B):
    """In a new process whose first calls are captured ones: nothing that a call does once may be what a capture forbids."""
    import subprocess
    import sys
    code = """
import torch
import layer_range_stage_gb300 as L
c = dict(device="cuda")
x = torch.randn(200, 1024, **c)
w, sw = torch.randint(0, 120, (512, 1024), dtype=torch.uint8, **c), torch.rand(4, 8, **c)
f = torch.rand(32, dtype=torch.float64, **c)
sizes = (3, 12, 40, 100, 200)
q = [torch.zeros(n, 1024, dtype=torch.uint8, **c) for n in sizes]
s = [torch.zeros(8, n, **c) for n in sizes]
def buffers():
    return [torch.zeros(n, 512, **c) for n in sizes], [torch.zeros(n, 2, dtype=torch.int32, **c) for n in sizes]
def go(y, ids):
    for n, a, b, z, i in zip(sizes, q, s, y, ids):
        L.stage_op_norm_f8(x[:n], a, b, gamma=x[0])
        L.stage_op_f8_gemm(a, b, w, sw, z)
        L.stage_op_rope(z.view(n, 8, 64), None, torch.arange(n, dtype=torch.int32, **c), f)
        L.stage_op_logprobs(z, top_ids=i)
got = buffers()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    go(*got)
graph.replay()
want = buffers()
go(*want)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for u, v in zip(got, want) for a, b in zip(u, v))
assert all(z.abs().max() > 0 for z in want[0])
print("same")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=240)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_refusals_of_the_binding_on_device_tensors(B):
    c = dict(device="cuda")
    x, q, s = torch.zeros(3, 256, **c), torch.zeros(3, 256, dtype=F8, **c), torch.zeros(2, 3, **c)
    i, f = torch.zeros(3, dtype=torch.int32, **c), torch.zeros(32, dtype=torch.float64, **c)
    h = x.view(3, 2, 128)
    bad = [
        lambda: B.stage_op_norm_f8(x, q, s.t()), lambda: B.stage_op_norm_f8(x, q, s[:1]), lambda: B.stage_op_norm_f8(x, q.float(), s), lambda: B.stage_op_norm_f8(x, q[:, :200], s),
        lambda: B.stage_op_norm_f8(x, q, s, gamma=torch.zeros(255, **c)), lambda: B.stage_op_norm_f8(x, q, s, gamma=torch.zeros(256)), lambda: B.stage_op_norm_f8(x.t(), q, s),
        lambda: B.stage_op_norm_f8(x, q, s, resid=x.half(), resid_out=x.half()), lambda: B.stage_op_norm_f8(x, q, s, y=x.half()), lambda: B.stage_op_norm_f8(x, q, s, eps=-1.0),
        lambda: B.stage_op_norm_f8(x), lambda: B.stage_op_norm_f8(x.double(), q, s),
        lambda: B.stage_op_f8_gemm(q, s, q[:, :250], torch.zeros(1, 2, **c), torch.zeros(3, 3, **c)), lambda: B.stage_op_f8_gemm(q, s, q, torch.zeros(1, 3, **c), torch.zeros(3, 3, **c)),
        lambda: B.stage_op_f8_gemm(q, s, q, torch.zeros(1, 2, **c), torch.zeros(3, 4, **c)), lambda: B.stage_op_f8_gemm(q, s, q, torch.zeros(1, 2), torch.zeros(3, 3, **c)),
        lambda: B.stage_op_f8_gemm(q[:, 1:], s, q[:, 1:], torch.zeros(1, 2, **c), torch.zeros(3, 3, **c)), lambda: B.stage_op_f8_gemm(x, s, q, torch.zeros(1, 2, **c), torch.zeros(3, 3, **c)),
        lambda: B.stage_op_f8_gemm(q, s, q, torch.zeros(1, 2, **c), torch.zeros(3, 3, **c), torch.zeros(2, dtype=torch.int32, **c)),
        lambda: B.stage_op_rope(h, None, i.long(), f), lambda: B.stage_op_rope(h, None, i, f.float()), lambda: B.stage_op_rope(h, None, i[:2], f), lambda: B.stage_op_rope(x, None, i, f),
        lambda: B.stage_op_rope(h, h.half(), i, f), lambda: B.stage_op_rope(h, h[:, :, :64], i, f), lambda: B.stage_op_rope(h, None, i, f, k_out=h),
        lambda: B.stage_op_rope(h, None, i, torch.zeros(65, dtype=torch.float64, **c)), lambda: B.stage_op_rope(h.transpose(1, 2), None, i, f), lambda: B.stage_op_rope(h, None, i, f, scale=float("nan")),
        lambda: B.stage_op_logprobs(x, i.long(), torch.zeros(3, **c)), lambda: B.stage_op_logprobs(x, None, torch.zeros(3, **c)), lambda: B.stage_op_logprobs(x, i, torch.zeros(4, **c)),
        lambda: B.stage_op_logprobs(x, i, top_ids=torch.zeros(3, 33, dtype=torch.int32, **c)), lambda: B.stage_op_logprobs(x, top_ids=i), lambda: B.stage_op_logprobs(x.t()[:, ::2], i),
        lambda: B.stage_op_logprobs(x, top_ids=torch.zeros(3, 2, dtype=torch.int32, **c), top_logprobs=torch.zeros(3, 3, **c)), lambda: B.stage_op_logprobs(x, i.cpu(), torch.zeros(3, **c)),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(B.StageError) as e:
            call()
        assert e.value.code == B.STAGE_E_INVALID, n


def test_a_decoding_step_of_single_ops(B):
    """Blocks of 8-bit projections on the paged 4-bit cache, as a program puts them together, captured and replayed while the sequences
    grow; every operator's result is held against the oracle's on the operator's own inputs."""
    rng = np.random.default_rng(11)
    H, hq, hk, d, F, V, page, n = 512, 8, 2, 64, 688, 1000, 16, 3
    qkv_w = (hq + 2 * hk) * d

    def weights(rows, cols):
        x = rng.standard_normal((rows, cols)).astype(np.float32) * 0.05
        codes, scale = np.zeros((rows, cols), np.uint8), np.zeros((-(-rows // 128), -(-cols // 128)), np.float32)
        for i in range(scale.shape[0]):
            for j in range(scale.shape[1]):
                at = (slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
                scale[i, j] = np.abs(x[at]).max() / 448
                codes[at] = step.e4m3_codes(x[at] / scale[i, j])
        return (codes, scale, put_f8(codes), dev(scale))

    Wqkv, Wo, Wup, Wdown, Whead = weights(qkv_w, H), weights(H, hq * d), weights(F, H), weights(H, F), weights(V, H)
    gammas = [(1 + 0.1 * rng.standard_normal(H)).astype(np.float32) for _ in range(3)]
    gd = [dev(g) for g in gammas]
    freqs = step.rope_freqs(d, 10000.0)[0]
    fd = dev(freqs)
    cap = n + 2                                                   # two rows of padding behind the step's tokens
    pages = 40
    cache = torch.zeros(B.stage_op_kv4_cache_shape(pages, page, hk, d), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(B.stage_op_kv4_attention_workspace_bytes(n, hq, hk, d, 1, 64), dtype=torch.uint8, device="cuda")
    length, new = i32([0] * n), i32([1] * n)
    table, ring, free = i32(np.full((n, 8), -1)), i32(rng.permutation(pages)), i32([0, pages])
    cu, slot, pos, seq, status = i32([0] * (n + 1)), i32([0] * cap), i32([0] * cap), i32([0] * cap), i32([0])
    stream_in = torch.zeros(cap, H, device="cuda")
    f32 = dict(device="cuda")

    def q8(k):
        return torch.zeros(cap, k + (-k) % 16, dtype=F8, **f32)[:, :k], torch.zeros(-(-k // 128), cap, **f32)

    b = dict(a1=q8(H), qkv=torch.zeros(cap, hq + 2 * hk, d, dtype=torch.bfloat16, **f32), att=torch.zeros(cap, hq, d, dtype=torch.bfloat16, **f32), a2=q8(hq * d),
             o=torch.zeros(cap, H, dtype=torch.bfloat16, **f32), a3=q8(H), h1=torch.zeros(cap, H, **f32), up=torch.zeros(cap, F, dtype=torch.bfloat16, **f32), a4=q8(F),
             down=torch.zeros(cap, H, dtype=torch.bfloat16, **f32), a5=q8(H), h2=torch.zeros(cap, H, **f32), z=torch.zeros(cap, V, **f32), ids=torch.zeros(cap, 4, dtype=torch.int32, **f32),
             best=torch.zeros(cap, 4, **f32), raw=torch.zeros(cap, hq + 2 * hk, d, dtype=torch.bfloat16, **f32))

    def go():
        B.stage_op_kv4_plan(page, length, new, table, ring, free, length, free, cu, slot, pos, seq, status)
        B.stage_op_norm_f8(stream_in, *b["a1"], gamma=gd[0])
        B.stage_op_f8_gemm(*b["a1"], *Wqkv[2:], b["qkv"].flatten(1))
        b["raw"].copy_(b["qkv"])
        B.stage_op_rope(b["qkv"][:, :hq], b["qkv"][:, hq:hq + hk], pos, fd)
        B.stage_op_kv4_append(cache, b["qkv"][:, hq:hq + hk], b["qkv"][:, hq + hk:], slot)
        B.stage_op_kv4_attention(cache, b["qkv"][:, :hq], cu, length, table, b["att"], 1, 64, ws)
        B.stage_op_norm_f8(b["att"].flatten(1), *b["a2"])
        B.stage_op_f8_gemm(*b["a2"], *Wo[2:], b["o"])
        B.stage_op_norm_f8(b["o"], *b["a3"], gamma=gd[1], resid=stream_in, resid_out=b["h1"])
        B.stage_op_f8_gemm(*b["a3"], *Wup[2:], b["up"])
        B.stage_op_norm_f8(b["up"], *b["a4"])
        B.stage_op_f8_gemm(*b["a4"], *Wdown[2:], b["down"])
        B.stage_op_norm_f8(b["down"], *b["a5"], gamma=gd[2], resid=b["h1"], resid_out=b["h2"])
        B.stage_op_f8_gemm(*b["a5"], *Whead[2:], b["z"])
        B.stage_op_logprobs(b["z"], top_ids=b["ids"], top_logprobs=b["best"])

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    oracle_cache = kv4.cache_array(pages, page, hk, d)

    def np_of(t):
        return t.double().cpu().numpy()

    def codes_of(a):
        return a[0].contiguous().view(torch.uint8).cpu().numpy(), a[1].cpu().numpy()

    def product(a, W, out, dtype):
        ac, s = codes_of(a)
        want, mag = step.f8_gemm(ac, s, W[0], W[1])
        close(out, want, (2.0 ** -16 + (len(s) + 3) * 2.0 ** -24) * mag + half_step(want, dtype))

    def rows8(a, x, resid, gamma):
        h, _, codes, scales = step.norm_f8(x, resid, gamma)
        got = codes_of(a)
        same(got[0], codes)
        same(got[1], scales)
        return h

    for t in range(20):
        stream_in.copy_(torch.as_tensor(rng.standard_normal((cap, H))))
        graph.replay()
        torch.cuda.synchronize()
        assert status.item() == 0 and pos.tolist() == [t] * n + [-1] * 2
        rows8(b["a1"], np_of(stream_in), None, gammas[0])
        product(b["a1"], Wqkv, b["raw"].flatten(1), "bf16")
        raw, got = np_of(b["raw"]), np_of(b["qkv"])
        want = step.rope(raw[:n, :hq + hk], [t] * n, freqs)
        size = np.abs(raw[:n, :hq + hk])
        size = np.tile(size[..., :d // 2] + size[..., d // 2:], 2)
        close(got[:n, :hq + hk], want, size * 2.0 ** -21 + half_step(want, "bf16"))
        same(got[n:], raw[n:])
        same(got[:, hq + hk:], raw[:, hq + hk:])
        kv4.append(oracle_cache, got[:, hq:hq + hk], got[:, hq + hk:], slot.cpu().numpy())
        same(cache.cpu().numpy(), oracle_cache)
        rows8(b["a2"], np_of(b["att"].flatten(1)), None, None)
        product(b["a2"], Wo, b["o"], "bf16")
        same(np_of(b["h1"]), rows8(b["a3"], np_of(b["o"]), np_of(stream_in), gammas[1]))
        product(b["a3"], Wup, b["up"], "bf16")
        rows8(b["a4"], np_of(b["up"]), None, None)
        product(b["a4"], Wdown, b["down"], "bf16")
        same(np_of(b["h2"]), rows8(b["a5"], np_of(b["down"]), np_of(b["h1"]), gammas[2]))
        product(b["a5"], Whead, b["z"], "f32")
        w = step.logprobs(np_of(b["z"]), None, 4)
        same(b["ids"].cpu().numpy(), w["ids"])
        close(b["best"], w["best"], 1e-5)
