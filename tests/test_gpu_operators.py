"""GPU tests of the operators around a quantised linear (woq_add_rmsnorm,
woq_qgemm_int8_a8, woq_lora_add) against their float64 definitions.

Tolerances count roundings: u = 2^-24 is half a step of fp32, 2^-11 of fp16,
and 2^-25 half the spacing of fp16's subnormals.

* sum_out: one fp32 addition, one rounding to fp16.
* y of the norm: at most 64 + 6 + 16 roundings in the sum of squares count half
  in the root; the mean, the root, the division, the gain and two products add
  fewer than 20: 64 u = 2^-18 together, taken as 2^-17.
* codes: |v / scale - q| <= 1/2 plus the same error of v and of the scale,
  127 * 2^-16.
* product: the integer sum is exact; its conversion and two scales cost 3 u.
* adapters: a sum of n terms in fp32, over the magnitudes of its terms, is off
  by at most n u; the matrix cores add 32 products a step (two roundings of
  the running sum), so K/16 for the inner products, as many as there are rank
  steps and partial sums (R + 32) for the outer ones, and 2^-20 for inner
  products carried as two fp16 halves of at least 22 bits.
"""
import numpy as np
import pytest

import oracle as O
from weight_only_quantized_quantize_amd import woq

pytestmark = pytest.mark.gpu

H, SUB, U = 2.0 ** -11, 2.0 ** -25, 2.0 ** -24


def case(*a):
    print("case:", *a, flush=True)


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    import torch
    torch.cuda.synchronize()
    return t.cpu().numpy()


def up(n, m):
    return -(-n // m) * m


def padded(a, ld, fill):
    """a's rows in a wider device buffer whose padding holds ``fill``."""
    out = np.full((a.shape[0], ld), fill, a.dtype)
    out[:, :a.shape[1]] = a
    return dev(out)


def full(b, ld, v, dtype):
    import torch
    return torch.full((b, ld), v, dtype=getattr(torch, dtype), device="cuda")


def within(y, ref, tol, what=""):
    y, err = y.astype(np.float64), np.abs(y.astype(np.float64) - ref)
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert np.all(err <= tol), (what, worst, y[worst], ref[worst], np.broadcast_to(tol, err.shape)[worst])


# -------------------------------------------------------------------- norm

def norm_case(b, K, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((b, K)) * spread).astype(np.float16)
    x[:, rng.choice(K, -(-K // 100), replace=False)] *= 20
    res = (rng.standard_normal((b, K)) * 2).astype(np.float16)
    w = (1 + 0.1 * rng.standard_normal(K)).astype(np.float16)
    return x, res, w


def check_norm(x, res, w, offset, eps, outs, pad=0, got=None):
    """Runs the norm with the outputs named in ``outs`` (s, y, q) and checks
    them; inputs are padded with NaN, outputs with 7 that has to stay."""
    b, K = x.shape
    ld, ldq = up(K, 8) + 8 * pad, up(K, 16) + 16 * pad
    s_ref, v_ref = O.add_rmsnorm(x, res, w, offset, eps)
    xd = padded(x, ld, np.float16(np.nan))
    rd = None if res is None else padded(res, ld, np.float16(np.nan))
    so = full(b, ld, 7, "float16") if "s" in outs else None
    y = full(b, ld, 7, "float16") if "y" in outs else None
    q = full(b, ldq, 7, "int8") if "q" in outs else None
    qs = full(1, b, 7, "float32")[0] if "q" in outs else None
    woq.woq_add_rmsnorm(xd, None if w is None else dev(w), eps, res=rd, sum_out=so, y=y, q=q, q_scale=qs,
                        offset=offset, K=K)
    if so is not None:
        g = host(so)
        within(g[:, :K], s_ref, np.abs(s_ref) * (H + 2 * U) + SUB, "sum")
        assert np.all(g[:, K:] == 7)
    if y is not None:
        g = host(y)
        within(g[:, :K], v_ref, np.abs(v_ref) * (H + 2.0 ** -17) + SUB, "y")
        assert np.all(g[:, K:] == 7)
    if q is not None:
        g, scale, ref = host(q), host(qs).astype(np.float64), O.rows_scale(v_ref)
        within(scale, ref, ref * 2.0 ** -17, "scale")
        live = ref > 0
        within(g[live, :K], v_ref[live] / ref[live, None], 0.5 + 127 * 2.0 ** -16, "codes")
        assert not g[~live, :K].any()
        assert np.all(np.abs(g[:, :K].astype(int)) <= 127)
        assert not g[:, K:up(K, 16)].any() and np.all(g[:, up(K, 16):] == 7)


@pytest.mark.parametrize("b,K", [(1, 1), (3, 7), (2, 8), (5, 9), (4, 16), (3, 511), (2, 513), (33, 1000), (7, 1024),
                                 (3, 2047), (5, 2049), (4, 4099), (2, 8192), (1, 8200), (2, 16392), (1, 32769),
                                 (2, 65536)])
def test_norm_widths_and_outputs(gpu_lib, b, K):
    x, res, w = norm_case(b, K, 100 + K)
    for outs in ("syq", "y", "q", "s"):
        case("norm", b, K, outs)
        check_norm(x, res, w, 0.0, 1e-6, outs)
    check_norm(x, None, w, 1.0, 1e-5, "yq", pad=1)
    check_norm(x, res, None, 0.0, 1e-6, "syq", pad=2)


@pytest.mark.parametrize("b,K", [(700, 96), (300, 3584), (70000, 24), (257, 640), (1025, 1536)])
def test_norm_many_rows(gpu_lib, b, K):
    case("norm rows", b, K)
    x, res, w = norm_case(b, K, b + K)
    check_norm(x, res, w, 0.0, 1e-6, "syq")
    check_norm(x, None, w, 0.0, 1e-6, "y")


def test_norm_small_and_large_magnitudes(gpu_lib):
    for spread, eps in ((1e-4, 1e-6), (1e-4, 1e-12), (300.0, 1e-6), (1.0, 1e30)):
        case("norm spread", spread, eps)
        x, res, w = norm_case(4, 1000, 5, spread)
        check_norm(x, None, w, 0.0, eps, "sy" if eps > 1 else "syq")
        check_norm(x, None, w, -1.0, eps, "sy")


@pytest.mark.parametrize("K", [5, 1000, 8192])
def test_rows_without_a_norm_are_encoded_as_the_weights_are(gpu_lib, K):
    """Codes and scales equal the INT8 encoder's on each row, bit for bit, ties
    included (K integers up to 127 times a power of two)."""
    import torch
    rng = np.random.default_rng(K)
    x = (rng.standard_normal((6, K)) * 3).astype(np.float16)
    x[1] = rng.integers(-254, 255, K) / 2
    x[1, 0] = 127                       # scale 1: halves are ties
    x[2] = 0
    x[3] = np.float16(2.0 ** -24) * rng.integers(-3, 4, K)
    xd, ld = padded(x, up(K, 8), np.float16(np.nan)), up(K, 16)
    q, qs = torch.empty(6, ld, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    woq.woq_add_rmsnorm(xd, None, 1e-6, q=q, q_scale=qs, K=K)
    q, qs = host(q), host(qs)
    for r in range(6):
        qr, s = O.quantize_int8(x[r:r + 1].astype(np.float32))
        assert np.float32(s) == qs[r], r
        np.testing.assert_array_equal(q[r, :K], qr[0], err_msg=str(r))


def test_norm_rows_of_zeros_nan_and_infinity(gpu_lib):
    import torch
    for K in (40, 5000):
        case("norm special rows", K)
        x, res, w = norm_case(6, K, 3)
        x[0], res[0] = 0, 0
        x[2, K - 1] = np.nan
        x[3, 0] = np.inf
        res[4, K // 2] = -np.inf
        so, y = full(6, K, 7, "float16"), full(6, K, 7, "float16")
        q, qs = full(6, up(K, 16), 7, "int8"), full(1, 6, 7, "float32")[0]
        for weight in (w, None):
            woq.woq_add_rmsnorm(dev(x), None if weight is None else dev(w), 1e-6, res=dev(res), sum_out=so, y=y,
                                q=q, q_scale=qs, K=K)
            s_ref, v_ref = O.add_rmsnorm(x, res, weight)
            gy, gq, gs = host(y), host(q), host(qs)
            assert not gy[0].any() and not gq[0].any() and gs[0] == 0
            assert np.all(np.isnan(gs[2:5])) and not gq[2:5].any()
            assert np.isnan(gy[2, K - 1])
            if weight is not None:
                assert np.all(np.isnan(gy[2])) and np.isnan(gy[3, 0]) and not gy[3, 1:].any()
            np.testing.assert_array_equal(np.isnan(host(so)), np.isnan(s_ref))
            for r in (1, 5):
                within(gy[r], v_ref[r], np.abs(v_ref[r]) * (H + 2.0 ** -17) + SUB)
                within(gq[r, :K], v_ref[r] / O.rows_scale(v_ref)[r], 0.5 + 127 * 2.0 ** -16)
    torch.cuda.synchronize()


@pytest.mark.parametrize("K", [100, 8192, 20000])
def test_norm_in_place(gpu_lib, K):
    """The sum over the residual, the output over the input."""
    x, res, w = norm_case(9, K, K)
    ld = up(K, 8)
    xd, rd = padded(x, ld, np.float16(3)), padded(res, ld, np.float16(3))
    woq.woq_add_rmsnorm(xd, dev(w), 1e-6, res=rd, sum_out=rd, y=xd, K=K)
    s_ref, v_ref = O.add_rmsnorm(x, res, w)
    within(host(rd)[:, :K], s_ref, np.abs(s_ref) * (H + 2 * U) + SUB)
    within(host(xd)[:, :K], v_ref, np.abs(v_ref) * (H + 2.0 ** -17) + SUB)
    assert np.all(host(rd)[:, K:] == 3) and np.all(host(xd)[:, K:] == 3)


# ----------------------------------------------------------------- product

def a8_weight(N, K, rng, ends=None, extreme=False):
    import torch
    ends = [N] if ends is None else ends
    codes = (np.full((N, K), 127, np.int8) if extreme else
             np.clip(np.rint(rng.standard_normal((N, K)) * 30), -127, 127).astype(np.int8))
    scales = [0.003 * (i + 1) for i in range(len(ends))]
    parts, lo = [], 0
    for e, s in zip(ends, scales):
        parts.append((codes[lo:e], np.float32(s)))
        lo = e
    w = woq.DeviceInt8([p for p in parts])
    torch.cuda.synchronize()
    return codes, [np.float32(s) for s in scales], w


def check_a8(N, K, b, seed, ends=None, ldy=None, pad=0):
    rng = np.random.default_rng(seed)
    codes, scales, w = a8_weight(N, K, rng, ends)
    xq = np.clip(np.rint(rng.standard_normal((b, K)) * 35), -128, 127).astype(np.int8)
    xs = (0.01 + rng.random(b)).astype(np.float32)
    ldy = N if ldy is None else ldy
    y = full(b, ldy, 7, "float16")
    # what follows a row's K codes is read against zero codes: garbage here
    woq.woq_qgemm_int8_a8(w.desc, padded(xq, up(K, 16) + 16 * pad, 77), dev(xs), y)
    ref = O.linear_int8_a8(codes, ends or [N], scales, xq, xs)
    g = host(y)
    with np.errstate(over="ignore"):
        big = np.abs(ref) > 65519          # past fp16: infinite
    assert np.all(np.isinf(g[:, :N][big]))
    within(np.where(big, 0, g[:, :N]), np.where(big, 0, ref), np.abs(ref) * (H + 4 * U) + SUB, (N, K, b))
    assert np.all(g[:, N:] == 7)


@pytest.mark.parametrize("b", [1, 2, 3, 8, 15, 16, 17, 31, 33, 64, 65, 100, 129, 257])
def test_product_batches(gpu_lib, b):
    for N, K in ((16, 64), (1, 1), (37, 100), (130, 1000), (515, 257), (256, 2048)):
        case("product", N, K, b)
        check_a8(N, K, b, b + N)


@pytest.mark.parametrize("N,K,b", [(1030, 3584, 4), (3584, 1100, 70), (777, 14336, 130), (200, 130000, 3),
                                   (4100, 640, 300), (300, 512, 1500), (64, 96, 5000)])
def test_product_sizes(gpu_lib, N, K, b):
    case("product", N, K, b)
    check_a8(N, K, b, N)


@pytest.mark.parametrize("b", [1, 5, 40, 200])
def test_product_segments_and_strides(gpu_lib, b):
    for N, ends, ldy, pad in ((100, [40, 60, 100], 100, 0), (1000, [1, 999, 1000], 1003, 3), (300, [0, 300, 300], 307, 1),
                              (520, [64, 128, 192, 256, 320, 384, 448, 520], 528, 2)):
        case("product segments", N, ends, ldy, pad, b)
        check_a8(N, 700, b, b, ends, ldy, pad)


# (N, K, b, tile): every tile of the product, with rows and outputs that end inside
# it, several rounds of workgroups on the largest, and K of one stage, of an odd and
# an even number of them, fewer and more than are read ahead
PRODUCT_TILES = [
    (100, 1100, 5, (16, 16)), (4100, 600, 13, (16, 32)), (9000, 300, 9, (16, 64)), (28600, 200, 3, (16, 128)),
    (28600, 50, 15, (16, 128)), (3900, 1000, 33, (32, 32)), (3901, 600, 40, (32, 32)), (8052, 700, 33, (32, 64)), (8053, 260, 40, (32, 64)),
    (1000, 700, 1000, (64, 64)), (1010, 200, 1001, (64, 64)), (28600, 200, 61, (64, 128)), (28606, 600, 33, (64, 128)),
    (28600, 100, 64, (64, 128)), (4100, 640, 300, (64, 128)), (4100, 130, 250, (64, 128)), (1000, 300, 3001, (128, 128)),
    (28670, 200, 70, (128, 128)), (8190, 300, 1021, (128, 256)), (8190, 128, 900, (128, 256)), (28670, 200, 1021, (256, 256)),
    (28670, 100, 400, (256, 256)), (16390, 400, 1300, (256, 256)), (2000, 333, 5003, (256, 256)),
]


def check_product_tile(N, K, b, ends, ldy, pad):
    rng = np.random.default_rng(N + K + b)
    codes, scales, w = a8_weight(N, K, rng, ends)
    xq = rng.integers(-128, 128, (b, K)).astype(np.int8)
    xs = (1e-4 + 1e-3 * rng.random(b)).astype(np.float32)
    y = full(b, ldy, 7, "float16")
    woq.woq_qgemm_int8_a8(w.desc, padded(xq, up(K, 16) + 16 * pad, 77), dev(xs), y)
    sums = xq.astype(np.float64) @ codes.T.astype(np.float64)      # integers below 2^53: exact
    col = np.repeat(np.array(scales, np.float64), np.diff([0] + ends))
    ref = sums * col[None, :] * xs.astype(np.float64)[:, None]
    g = host(y)
    within(g[:, :N], ref, np.abs(ref) * (H + 4 * U) + SUB, (N, K, b))
    assert np.all(g[:, N:] == 7)


@pytest.mark.parametrize("N,K,b,tile", PRODUCT_TILES)
def test_product_every_tile(gpu_lib, N, K, b, tile):
    import torch
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert woq.woq_qgemm_int8_a8_tile(N, b) == tile
    for ends, ldy, pad in (([N], N, 0), ([N // 3, N // 3, N - 7, N], N + 3, 1)):
        case("product tile", N, K, b, tile, ends, ldy)
        check_product_tile(N, K, b, ends, ldy, pad)


@pytest.mark.parametrize("N,K,b,rows", [(33000, 200, 1, 16), (66000, 90, 16, 16), (66010, 300, 17, 32), (33003, 140, 61, 64),
                                        (66000, 150, 100, 128)])
def test_product_of_wide_weights_and_few_rows(gpu_lib, N, K, b, rows):
    """More workgroups than compute units: several rounds of a tile no taller than the batch needs."""
    assert woq.woq_qgemm_int8_a8_tile(N, b)[0] == rows
    for ends, ldy, pad in (([N], N, 0), ([5, N - 1000, N], N + 5, 2)):
        case("product wide", N, K, b, rows, ends, ldy)
        check_product_tile(N, K, b, ends, ldy, pad)


@pytest.mark.parametrize("code", [127, -128])
def test_product_extreme_sums_stay_exact(gpu_lib, code):
    """Every product at its largest over the longest row: 127 * 128 * 131072 < 2^31."""
    for b in (1, 20, 150):
        case("product extreme", code, b)
        rng = np.random.default_rng(1)
        codes, scales, w = a8_weight(20, woq.A8_MAX_K, rng, extreme=True)
        xq = full(b, woq.A8_MAX_K, code, "int8")
        xs = np.full(b, 2.0 ** -17, np.float32)
        y = full(b, 20, 7, "float16")
        woq.woq_qgemm_int8_a8(w.desc, xq, dev(xs), y)
        ref = 127.0 * code * woq.A8_MAX_K * 2.0 ** -17 * float(scales[0])
        within(host(y), np.full((b, 20), ref), abs(ref) * (H + 4 * U))


def test_product_of_a_row_that_is_not_finite(gpu_lib):
    """A scale of NaN (a row the norm refused to encode) makes that row NaN and
    leaves the others."""
    for b in (3, 40, 200):
        rng = np.random.default_rng(b)
        codes, scales, w = a8_weight(50, 130, rng)
        xq = rng.integers(-127, 128, (b, 144)).astype(np.int8)
        xs = rng.random(b).astype(np.float32)
        xs[1] = np.nan
        y = full(b, 50, 7, "float16")
        woq.woq_qgemm_int8_a8(w.desc, dev(xq), dev(xs), y)
        ref, g = O.linear_int8_a8(codes, [50], scales, xq[:, :130], xs), host(y)
        assert np.all(np.isnan(g[1]))
        keep = np.arange(b) != 1
        within(g[keep], ref[keep], np.abs(ref[keep]) * (H + 4 * U) + SUB)


# ---------------------------------------------------------------- adapters

def lora_pool(count, N, K, R, S, rng, rank=None, junk=False):
    """A pool whose entries past each adapter's rank (and past K) are NaN where
    ``junk``: they count as absent."""
    ends = {1: [N], 2: [N // 3, N], 3: [N // 2, N // 2 + N // 4, N]}[S]
    A = (rng.standard_normal((count, S * R, up(K, 8))) / np.sqrt(K)).astype(np.float16)
    B = (rng.standard_normal((count, N, R)) * 0.3).astype(np.float16)
    scale = (0.5 + rng.random(count)).astype(np.float32)
    if junk:
        A[:, :, K:] = np.nan
        for a in range(count):
            k = R if rank is None else min(max(int(rank[a]), 0), R)
            for i in range(S):
                A[a, i * R + k:(i + 1) * R] = np.nan
            B[a, :, k:] = np.nan
    return A, B, scale, ends


def check_lora(b, N, K, R, S, count, ids, seed, rank=None, junk=False, base=True, place=False, pad=0, odd=0, x=None):
    import torch
    rng = np.random.default_rng(seed)
    A, B, scale, ends = lora_pool(count, N, K, R, S, rng, rank, junk)
    x = rng.standard_normal((b, K)).astype(np.float16) if x is None else x
    basev = rng.standard_normal((b, N)).astype(np.float16)
    ids = np.asarray(ids, np.int32)
    rank32 = None if rank is None else np.asarray(rank, np.int32)
    pool = woq.DeviceLora(dev(A), dev(B), dev(scale), None if rank is None else dev(rank32), K, ends)
    xd = padded(x, up(K, 8) + 8 * pad, np.float16(np.nan))
    bd = padded(basev, N + odd, np.float16(3))
    y = bd if place else full(b, N + odd, 7, "float16")
    ws = torch.full((woq.woq_lora_workspace(pool.desc, b) // 4 + 4,), float("nan"), device="cuda")
    woq.woq_lora_add(pool.desc, xd, dev(ids), bd if base else None, y, ws)
    zero = basev if base else np.zeros_like(basev)
    ref, spread = O.lora_add(zero, x, ids, A, B, scale, ends, rank)
    g = host(y)
    n = K / 16 + R + 32
    within(g[:, :N], ref, np.abs(ref) * (H + 2 * U) + SUB + spread * (n * U + 2.0 ** -20), (b, N, K, R, S, count))
    off = (ids < 0) | (ids >= count)
    np.testing.assert_array_equal(g[off, :N], zero[off])      # untouched rows, bit for bit
    assert np.all(g[:, N:] == (3 if place else 7))
    assert np.all(np.isnan(host(ws)[-4:]))                    # nothing past the workspace


@pytest.mark.parametrize("b,N,K,R,S,count", [
    (1, 1, 1, 8, 1, 1), (1, 16, 32, 16, 1, 2), (2, 40, 100, 8, 1, 3), (5, 100, 257, 16, 3, 4), (1, 8192, 1024, 16, 1, 8),
    (16, 515, 640, 24, 2, 5), (17, 300, 1000, 32, 3, 17), (64, 640, 512, 16, 3, 64), (64, 200, 3584, 64, 1, 3),
    (33, 130, 96, 256, 2, 2), (256, 130, 300, 16, 2, 200), (250, 96, 1100, 48, 1, 40), (3, 4097, 8192, 8, 2, 2), (50, 72, 2040, 40, 1, 1)])
def test_adapters_decode_batches(gpu_lib, b, N, K, R, S, count):
    case("adapters", b, N, K, R, S, count)
    rng = np.random.default_rng(b + N)
    check_lora(b, N, K, R, S, count, rng.integers(-1, count + 1, b), 1)
    check_lora(b, N, K, R, S, count, np.full(b, count - 1), 2, pad=1, odd=3)


@pytest.mark.parametrize("lens", [[65], [100, 1, 1, 30], [200, 7, 300, 0, 64, 64], [1] * 90, [1500, 3], [129, 255, 640]])
def test_adapters_packed_prompts(gpu_lib, lens):
    """Rows of one request side by side, requests of any length, one without an
    adapter; two requests may share one."""
    b = sum(lens)
    for N, K, R, S, count in ((130, 200, 16, 1, 3), (515, 640, 64, 2, 5), (72, 1000, 8, 3, 2)):
        case("adapters packed", lens[:6], N, K, R, S, count)
        ids = np.repeat([(3 * i + 1) % (count + 1) - 1 for i in range(len(lens))], lens)
        check_lora(b, N, K, R, S, count, ids, b)


@pytest.mark.parametrize("b,N,K,R,S,count", [
    (257, 40, 72, 8, 1, 17), (683, 130, 200, 16, 1, 7), (1021, 70, 96, 64, 2, 5), (1025, 66, 40, 24, 3, 1500), (4097, 24, 32, 16, 1, 2),
    (4500, 16, 24, 72, 1, 3), (9000, 8, 16, 8, 1, 2500), (120, 20011, 64, 16, 2, 4), (256, 8210, 48, 40, 1, 30), (200, 20000, 32, 8, 1, 26)])
def test_adapters_mixed_large_batches(gpu_lib, b, N, K, R, S, count):
    """Rows of one adapter anywhere in the batch, more adapters than the order
    has bins, rows without one among them, all of one adapter, none of any."""
    case("adapters mixed", b, N, K, R, S, count)
    rng = np.random.default_rng(b + N)
    check_lora(b, N, K, R, S, count, rng.integers(-1, count + 1, b), 1, pad=1, odd=3)
    check_lora(b, N, K, R, S, count, np.arange(b) % count, 2, rank=rng.integers(-1, R + 2, count), junk=True, place=True)
    check_lora(b, N, K, R, S, count, np.full(b, count - 1), 3)
    check_lora(b, N, K, R, S, count, np.full(b, -7), 4)
    if count > 1024:
        check_lora(b, N, K, R, S, count, (np.arange(b) % 2) * 1024 + 3, 5)


@pytest.mark.parametrize("b,N,R,count", [(30, 50, 16, 5), (150, 16000, 16, 8), (700, 75, 16, 9), (5000, 20, 72, 6)])
def test_adapters_bits_do_not_depend_on_the_order_of_rows(gpu_lib, b, N, R, count):
    """The rows shuffled, and again with those of one adapter side by side: the same bits."""
    import torch
    case("adapters shuffled", b, N, R, count)
    rng = np.random.default_rng(b)
    A, B, s, ends = lora_pool(count, N, 136, R, 1, rng)
    pool = woq.DeviceLora(dev(A), dev(B), dev(s))
    x, base = rng.standard_normal((b, 136)).astype(np.float16), rng.standard_normal((b, N)).astype(np.float16)
    ids = rng.integers(-1, count, b).astype(np.int32)
    ws = torch.empty(woq.woq_lora_workspace(pool.desc, b), dtype=torch.uint8, device="cuda")

    def run(at):
        y = full(b, N, 7, "float16")
        woq.woq_lora_add(pool.desc, dev(x[at]), dev(ids[at]), dev(base[at]), y, ws)
        out = np.empty((b, N), np.float16)
        out[at] = host(y)
        return out.view(np.uint16)

    first = run(np.arange(b))
    for at in (np.arange(b), rng.permutation(b), np.argsort(ids, kind="stable")):
        np.testing.assert_array_equal(run(at), first)


def test_adapters_of_a_mixed_batch_captured_and_replayed(gpu_lib):
    """Replays with other rows and ids than the captured ones, eager calls in between."""
    import torch
    case("adapters mixed, captured")
    rng = np.random.default_rng(12)
    b, N, K, R, count = 1100, 90, 136, 32, 6
    A, B, s, ends = lora_pool(count, N, K, R, 1, rng)
    pool = woq.DeviceLora(dev(A), dev(B), dev(s))
    inputs = [(dev(rng.standard_normal((b, K)).astype(np.float16)), dev(rng.integers(-1, count, b).astype(np.int32))) for _ in range(3)]
    x, ids, y = inputs[0][0].clone(), inputs[0][1].clone(), full(b, N, 7, "float16")
    ws, other = (torch.empty(woq.woq_lora_workspace(pool.desc, b), dtype=torch.uint8, device="cuda") for _ in range(2))
    woq.woq_lora_add(pool.desc, x, ids, None, y, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        woq.woq_lora_add(pool.desc, x, ids, None, y, ws)
    for i in (0, 1, 2, 1):
        x.copy_(inputs[i][0])
        ids.copy_(inputs[i][1])
        graph.replay()
        eager = full(b, N, 7, "float16")
        woq.woq_lora_add(pool.desc, *inputs[i], None, eager, other)
        np.testing.assert_array_equal(host(y).view(np.uint16), host(eager).view(np.uint16))


def by_adapter(base, x, ids, A, B, scale, ends, rank=None):
    """O.lora_add, all rows of an adapter at once."""
    y, spread = base.astype(np.float64), np.zeros(base.shape)
    count, N, R = B.shape
    for a in range(count):
        rows = np.flatnonzero(ids == a)
        k = R if rank is None else min(max(int(rank[a]), 0), R)
        if k == 0 or rows.size == 0:
            continue
        xr, lo = x[rows].astype(np.float64), 0
        for i, end in enumerate(ends):
            down = A[a, i * R:i * R + k, :x.shape[1]].astype(np.float64).T
            up_ = B[a, lo:end, :k].astype(np.float64).T
            y[rows, lo:end] += float(scale[a]) * (xr @ down @ up_)
            spread[rows, lo:end] = abs(float(scale[a])) * (np.abs(xr) @ np.abs(down) @ np.abs(up_))
            lo = end
    return y, spread


@pytest.mark.parametrize("R", [8, 24, 40, 72])
@pytest.mark.parametrize("b,N,S", [(2100, 4100, 1), (2100, 4103, 3), (4100, 4100, 2), (4099, 4201, 3)])
def test_adapters_of_wide_outputs_and_many_rows(gpu_lib, b, N, S, R):
    """Each workgroup goes through two (2100 rows) or four tiles of outputs, with
    segments that end inside its span: from a base, in place and without one,
    adapters' rows side by side (windows of one or several) and mixed, rows without one."""
    import torch
    rng = np.random.default_rng(b + N + R)
    K, count = 40, 5
    rank = rng.integers(0, R + 1, count)
    A, B, scale, ends = lora_pool(count, N, K, R, S, rng, rank, junk=True)
    pool = woq.DeviceLora(dev(A), dev(B), dev(scale), dev(rank.astype(np.int32)), K, ends)
    x, base = rng.standard_normal((b, K)).astype(np.float16), rng.standard_normal((b, N)).astype(np.float16)
    xd = padded(x, up(K, 8) + 8, np.float16(np.nan))
    ws = torch.full((woq.woq_lora_workspace(pool.desc, b) // 4 + 4,), float("nan"), device="cuda")
    mixed = rng.integers(-1, count + 1, b)
    for ids, odd, form in ((mixed, 0, "place"), (np.sort(mixed), 3, "base"), (np.sort(mixed), 4, "place"),
                           (np.where(mixed < 0, -1, 1), 1, "none"), (mixed, 1, "base")):
        case("adapters wide", b, N, K, R, S, odd, form)
        bd = padded(base, N + odd, np.float16(7))
        y = bd if form == "place" else full(b, N + odd, 7, "float16")
        woq.woq_lora_add(pool.desc, xd, dev(ids.astype(np.int32)), None if form == "none" else bd, y, ws)
        zero = np.zeros_like(base) if form == "none" else base
        ref, spread = by_adapter(zero, x, ids, A, B, scale, ends, rank)
        g = host(y)
        within(g[:, :N], ref, np.abs(ref) * (H + 2 * U) + SUB + spread * ((K / 16 + R + 32) * U + 2.0 ** -20), form)
        off = (ids < 0) | (ids >= count)
        np.testing.assert_array_equal(g[off, :N], zero[off])
        assert np.all(g[:, N:] == 7)
    assert np.all(np.isnan(host(ws)[-4:]))


@pytest.mark.parametrize("R", [8, 32, 64, 72])
@pytest.mark.parametrize("b", [5, 300])
def test_adapters_eight_segments_some_empty(gpu_lib, b, R):
    """Every kernel sees the same tiles of every segment: eight of them, empty
    ones at the start, inside and at the end, beside ends that are not tiles'."""
    import torch
    case("adapters eight segments", b, R)
    rng = np.random.default_rng(b + R)
    N, K, count, ends = 260, 72, 3, [0, 1, 66, 66, 130, 259, 260, 260]
    A = (rng.standard_normal((count, 8 * R, K)) / np.sqrt(K)).astype(np.float16)
    B = (rng.standard_normal((count, N, R)) * 0.3).astype(np.float16)
    s = (0.5 + rng.random(count)).astype(np.float32)
    x, base = rng.standard_normal((b, K)).astype(np.float16), rng.standard_normal((b, N)).astype(np.float16)
    ids = rng.integers(-1, count, b).astype(np.int32)
    pool = woq.DeviceLora(dev(A), dev(B), dev(s), segments=ends)
    ws = torch.empty(woq.woq_lora_workspace(pool.desc, b), dtype=torch.uint8, device="cuda")
    y = full(b, N + 4, 7, "float16")
    woq.woq_lora_add(pool.desc, dev(x), dev(ids), dev(base), y, ws)
    ref, spread = O.lora_add(base, x, ids, A, B, s, ends)
    g = host(y)
    within(g[:, :N], ref, np.abs(ref) * (H + 2 * U) + SUB + spread * ((K / 16 + R + 32) * U + 2.0 ** -20))
    assert np.all(g[:, N:] == 7)


@pytest.mark.parametrize("b", [1, 20, 100, 300])
def test_adapters_of_different_ranks(gpu_lib, b):
    """Entries past an adapter's rank and past K are NaN and stay out of it."""
    rank = [16, 0, 5, 1, 8, 100, -3, 9]
    for K in (64, 203):
        case("adapters ranks", b, K)
        rng = np.random.default_rng(b)
        check_lora(b, 133, K, 16, 2, 8, rng.integers(0, 8, b), 4, rank=rank, junk=True)
        check_lora(b, 77, K, 136, 2, 5, np.sort(rng.integers(-1, 5, b)), 4, rank=[136, 65, 3, 129, 64], junk=True)
        check_lora(b, 133, K, 40, 1, 8, np.sort(rng.integers(0, 8, b)), 4, rank=[40, 33, 31, 1, 8, 25, 17, 39], junk=True)


@pytest.mark.parametrize("b", [1, 7, 200])
def test_adapters_in_place_and_without_a_base(gpu_lib, b):
    rng = np.random.default_rng(b)
    for N, odd in ((64, 0), (99, 1)):
        case("adapters in place", b, N)
        check_lora(b, N, 128, 16, 1, 4, rng.integers(-1, 4, b), 6, place=True, odd=odd)
        check_lora(b, N, 128, 16, 1, 4, rng.integers(-1, 4, b), 6, base=False, odd=odd)


def test_adapters_without_a_pool_or_a_named_adapter(gpu_lib):
    for count in (0, 2):
        check_lora(5, 40, 64, 8, 1, count, [-1, count, 99, -(2 ** 31), 2 ** 31 - 1], 7)


@pytest.mark.parametrize("scale", [2.0 ** -14, 1.0, 200.0, 1e4])
def test_adapters_inner_products_of_any_size(gpu_lib, scale):
    """Activations from subnormals of fp16 to values whose inner products leave
    fp16's range; the outputs stay in it."""
    import torch
    rng = np.random.default_rng(8)
    for b in (3, 90):
        case("adapters range", scale, b)
        N, K, R = 70, 200, 16
        A = (rng.standard_normal((2, R, K))).astype(np.float16)
        B = (rng.standard_normal((2, N, R)) * 1e-3).astype(np.float16)
        s = np.array([1.0, 0.5], np.float32)
        x = (rng.standard_normal((b, K)) * scale).astype(np.float16)
        ids = rng.integers(0, 2, b).astype(np.int32)
        pool = woq.DeviceLora(dev(A), dev(B), dev(s))
        y = full(b, N, 7, "float16")
        ws = torch.empty(woq.woq_lora_workspace(pool.desc, b), dtype=torch.uint8, device="cuda")
        woq.woq_lora_add(pool.desc, dev(x), dev(ids), None, y, ws)
        ref, spread = O.lora_add(np.zeros((b, N)), x, ids, A, B, s, [N])
        within(host(y), ref, np.abs(ref) * (H + 2 * U) + SUB + spread * ((K / 16 + R + 32) * U + 2.0 ** -20))


@pytest.mark.parametrize("b", [3, 90, 300])
@pytest.mark.parametrize("R", [8, 16, 24, 64])
def test_adapters_inner_products_far_apart(gpu_lib, b, R):
    """One rank of every row is larger than another by up to 2^40, and outputs whose B
    has a zero for the large one see the small one alone, to 2^-23 of itself or 2^-38
    of the large one.  The inner products are exact (two terms of 11 bits each, in
    different places); the base takes away the fp16 result, so that the rest shows in
    the output: it is off by that, by an fp32 rounding of the sum, and by its own
    rounding to fp16."""
    import torch
    case("adapters far apart", b, R)
    rng = np.random.default_rng(b + R)
    K, N = 8, 40
    A = np.zeros((1, R, K), np.float16)
    A[0, 0, 0], A[0, R - 1, 1], A[0, R - 1, 2] = 1, 1, 1
    small = (1 + rng.integers(0, 1024, b) / 1024.0) * 2.0 ** rng.integers(-10, 1, b)
    x = np.zeros((b, K), np.float16)
    x[:, 1] = small
    x[:, 2] = small * 2.0 ** -12 * (1 - rng.integers(1, 1024, b) / 2048.0)      # below half a step of x[:, 1]
    x[:, 0] = 2.0 ** rng.integers(-8, 16, b)
    A[0, 0, 0] = 2.0 ** 15
    B = np.zeros((1, N, R), np.float16)
    B[0, :, R - 1] = 1
    B[0, N // 2:, 0] = 2.0 ** -15
    h0, h1 = x[:, 0].astype(np.float64) * 2.0 ** 15, x[:, 1].astype(np.float64) + x[:, 2].astype(np.float64)
    base = np.zeros((b, N), np.float16)
    base[:, :N // 2] = -h1.astype(np.float16)[:, None]
    pool = woq.DeviceLora(dev(A), dev(B), torch.ones(1, device="cuda"))
    y = full(b, N, 7, "float16")
    ws = torch.empty(woq.woq_lora_workspace(pool.desc, b), dtype=torch.uint8, device="cuda")
    woq.woq_lora_add(pool.desc, dev(x), dev(np.zeros(b, np.int32)), dev(base), y, ws)
    g, rest = host(y)[:, :N // 2], (h1 + base[:, 0])[:, None]
    lost = np.maximum(2.0 ** -23 * h1, 2.0 ** -38 * np.maximum(h0, h1))[:, None]
    within(g, np.broadcast_to(rest, g.shape), lost + 2 * U * h1[:, None] + H * (np.abs(rest) + lost) + SUB)


def test_adapters_rows_do_not_touch_each_other(gpu_lib):
    """A NaN or an infinity in one row's input stays in that row; the other rows' bits
    do not depend on it, nor on which rows share the call."""
    import torch
    rng = np.random.default_rng(9)
    for b in (6, 150):
        N, K, R, count = 75, 320, 16, 3
        A, B, s, ends = lora_pool(count, N, K, R, 1, rng)
        pool = woq.DeviceLora(dev(A), dev(B), dev(s))
        x = rng.standard_normal((b, K)).astype(np.float16)
        base = rng.standard_normal((b, N)).astype(np.float16)
        ids = rng.integers(0, count, b).astype(np.int32)
        ws = torch.empty(woq.woq_lora_workspace(pool.desc, b), dtype=torch.uint8, device="cuda")

        def run(x):
            y = full(b, N, 7, "float16")
            woq.woq_lora_add(pool.desc, dev(x), dev(ids), dev(base), y, ws)
            return host(y)

        clean, bad = run(x), x.copy()
        bad[2, 5], bad[4, 0] = np.nan, np.inf
        dirty = run(bad)
        keep = ~np.isin(np.arange(b), (2, 4))
        np.testing.assert_array_equal(clean[keep].view(np.uint16), dirty[keep].view(np.uint16))
        assert np.all(np.isnan(dirty[2])) and not np.isfinite(dirty[4]).any()


# ------------------------------------------------------- a run of them together

class Block:
    """Norm, 8-bit product and adapters in a row, as one layer's q|k|v."""

    def __init__(self, b, K, N, seed):
        import torch
        rng = np.random.default_rng(seed)
        self.x, self.res, self.w = norm_case(b, K, seed)
        ends = [N // 2, N // 2 + N // 4, N]
        self.codes, self.scales, self.w8 = a8_weight(N, K, rng, ends)
        self.scales = [s * np.float32(0.1) for s in self.scales]
        for i, s in enumerate(self.scales):
            self.w8.desc.seg_scale[i] = float(s)
        self.A, self.B, self.s, self.ends = lora_pool(4, N, K, 16, 3, rng)
        self.ids = rng.integers(-1, 4, b).astype(np.int32)
        self.pool = woq.DeviceLora(dev(self.A), dev(self.B), dev(self.s), K=K, segments=ends)
        self.d = {k: dev(v) for k, v in (("x", padded_host(self.x)), ("res", padded_host(self.res)), ("w", self.w),
                                         ("ids", self.ids))}
        half = dict(dtype=torch.float16, device="cuda")
        self.sum, self.n = torch.zeros(b, up(K, 8), **half), torch.zeros(b, up(K, 8), **half)
        self.q = torch.zeros(b, up(K, 16), dtype=torch.int8, device="cuda")
        self.qs, self.y = torch.zeros(b, device="cuda"), torch.zeros(b, N, **half)
        self.ws = torch.zeros(woq.woq_lora_workspace(self.pool.desc, b), dtype=torch.uint8, device="cuda")
        self.b, self.K, self.N = b, K, N

    def run(self, stream=None):
        d = self.d
        woq.woq_add_rmsnorm(d["x"], d["w"], 1e-6, res=d["res"], sum_out=self.sum, y=self.n, q=self.q, q_scale=self.qs,
                            stream=stream)
        woq.woq_qgemm_int8_a8(self.w8.desc, self.q, self.qs, self.y, stream=stream)
        woq.woq_lora_add(self.pool.desc, self.n, d["ids"], self.y, self.y, self.ws, stream=stream)

    def check(self):
        """Each step against the definition on the values the step before gave."""
        q, qs, n = host(self.q)[:, :self.K], host(self.qs), host(self.n)[:, :self.K]
        _, v = O.add_rmsnorm(self.x, self.res, self.w)
        within(n, v, np.abs(v) * (H + 2.0 ** -17) + SUB)
        within(q, v / O.rows_scale(v)[:, None], 0.5 + 127 * 2.0 ** -16)
        base = O.linear_int8_a8(self.codes, self.ends, self.scales, q, qs)
        ref, spread = O.lora_add(base, n, self.ids, self.A, self.B, self.s, self.ends)
        tol = (np.abs(base) + np.abs(ref)) * (H + 4 * U) + 2 * SUB + spread * ((self.K / 16 + 48) * U + 2.0 ** -20)
        within(host(self.y), ref, tol)


def padded_host(a):
    out = np.full((a.shape[0], up(a.shape[1], 8)), np.nan, a.dtype)
    out[:, :a.shape[1]] = a
    return out


@pytest.mark.parametrize("b,K,N", [(1, 512, 256), (8, 1000, 500), (40, 3584, 1024), (70, 512, 130), (500, 640, 300)])
def test_block_in_a_row(gpu_lib, b, K, N):
    case("block", b, K, N)
    blk = Block(b, K, N, b)
    blk.run()
    blk.check()


@pytest.mark.parametrize("b", [4, 100])
def test_block_on_another_stream(gpu_lib, b):
    import torch
    blk = Block(b, 640, 300, 50 + b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        blk.run()
    s.synchronize()
    blk.check()
    first = host(blk.y).copy()
    blk.run(stream=s)
    s.synchronize()
    np.testing.assert_array_equal(host(blk.y).view(np.uint16), first.view(np.uint16))


@pytest.mark.parametrize("b", [3, 64, 130])
def test_block_captured_and_replayed(gpu_lib, b):
    """One graph of the three operators, replayed between eager runs on other
    inputs; every replay gives the eager bits of its inputs."""
    import torch
    blk = Block(b, 512, 200, b)
    blk.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        blk.run()
    x0 = blk.d["x"].clone()
    other = torch.randn_like(x0)
    eager = {}
    for name, x in (("first", x0), ("other", other)):
        blk.d["x"].copy_(x)
        blk.run()
        torch.cuda.synchronize()
        eager[name] = host(blk.y).copy()
    for name, x in (("first", x0), ("other", other), ("other", other), ("first", x0)):
        blk.d["x"].copy_(x)
        blk.y.fill_(5)
        g.replay()
        np.testing.assert_array_equal(host(blk.y).view(np.uint16), eager[name].view(np.uint16))
        Block(b, 64, 48, 1).run()           # the program's own work between replays
        torch.cuda.synchronize()


# ------------------------------------------------- adapters beside a stack's steps

def small_stack(fmt, rng, dims):
    """A chain of linears in one format; each step reads the one before it."""
    steps, keep = [], []
    for i, (N, K) in enumerate(dims):
        W = (rng.standard_normal((N, K)) / np.sqrt(K)).astype(np.float32)
        if fmt == "int8":
            d = woq.DeviceInt8([woq.woq_quantize_int8(W)])
            keep.append(d)
            steps.append(woq.step_int8(d, i, i))
        else:
            g = woq.woq_int4o_geometry(K)
            perm = O.global_perm(K, np.sort(rng.choice(K, g.n_out, replace=False)))
            d, pd = woq.DeviceInt4o([woq.woq_quantize_int4o(W, perm, g.n_out)], g), dev(perm)
            keep += [d, pd]
            steps.append(woq.step_int4o(d, pd, i, i))
    return steps, keep


@pytest.mark.parametrize("fmt,b", [("int8", 1), ("int8", 7), ("int4o", 2), ("int4o", 40)])
def test_stack_with_adapters_equals_its_steps(gpu_lib, fmt, b):
    """A chain of three steps, adapters beside the first and the last: the bits of
    running each step and woq_lora_add by hand, also on replays of a graph."""
    import torch
    case("stack adapters", fmt, b)
    rng = np.random.default_rng(b)
    dims = [(520, 256), (1000, 520), (264, 1000)]
    steps, keep = small_stack(fmt, rng, dims)
    pools = []
    for i, (N, K) in enumerate(dims):
        A, B, s, ends = lora_pool(4, N, K, 16, 2, rng)
        pools.append(None if i == 1 else woq.DeviceLora(dev(A), dev(B), dev(s), K=K, segments=ends))
    ids = dev(rng.integers(-1, 4, b).astype(np.int32))
    x = dev(rng.standard_normal((b, 256)).astype(np.float16))
    outs = [full(b, N, 7, "float16") for N, _ in dims]
    st = woq.Stack(steps, b)
    st.bind([x] + outs[:2], outs)
    ws = torch.empty(st.lora_workspace(pools, b), dtype=torch.uint8, device="cuda")
    st.run_lora(b, pools, ids, ws)
    got = [host(o).copy() for o in outs]

    hand = [full(b, N, 7, "float16") for N, _ in dims]
    src = x
    for step, pool, out in zip(steps, pools, hand):
        step.in_slot = step.out_slot = 0
        one = woq.Stack([step], b)
        one.bind([src], [out])
        one.run(b)
        if pool is not None:
            woq.woq_lora_add(pool.desc, src, ids, out, out, ws)
        src = out
    for g, h in zip(got, hand):
        np.testing.assert_array_equal(g.view(np.uint16), host(h).view(np.uint16))

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.run_lora(b, pools, ids, ws)
    for _ in range(3):
        for o in outs:
            o.fill_(3)
        g.replay()
        for o, h in zip(outs, got):
            np.testing.assert_array_equal(host(o).view(np.uint16), h.view(np.uint16))
    st.run(b)                                      # without adapters the rows without one agree
    assert np.array_equal(host(outs[0])[host(ids) < 0], got[0][host(ids) < 0])
    del keep


def test_stack_with_adapters_refuses_before_the_first_launch(gpu_lib):
    import torch
    rng = np.random.default_rng(0)
    dims = [(64, 128), (48, 64)]
    steps, keep = small_stack("int8", rng, dims)
    st = woq.Stack(steps, 4)
    x, outs = full(4, 128, 1, "float16"), [full(4, N, 7, "float16") for N, _ in dims]
    st.bind([x, outs[0]], outs)
    ids = dev(np.zeros(4, np.int32))

    def pool(N, K, R=16):
        A, B, s, ends = lora_pool(2, N, K, R, 1, rng)
        return woq.DeviceLora(dev(A), dev(B), dev(s), K=K, segments=ends)

    good = pool(64, 128)
    ws = torch.empty(st.lora_workspace([good, None], 4), dtype=torch.uint8, device="cuda")
    for pools in ([None, pool(64, 64)], [None, pool(48, 128)]):           # N or K of another step
        with pytest.raises(woq.WoqError) as e:
            st.run_lora(4, pools, ids, ws)
        assert e.value.status == woq.WOQ_EINVAL
    with pytest.raises(woq.WoqError) as e:
        st.run_lora(4, [None, pool(48, 64)], ids, ws[:16])
    assert e.value.status == woq.WOQ_EINVAL
    with pytest.raises(ValueError):
        st.run_lora(4, [good], ids, ws)                                    # a pool per step
    with pytest.raises(ValueError):
        st.run_lora(4, [good, None], ids[:3], ws)
    assert np.all(host(outs[0]) == 7) and np.all(host(outs[1]) == 7)       # nothing ran
    del keep


def test_empty_calls_are_no_ops(gpu_lib):
    blk = Block(2, 64, 48, 3)
    blk.y.fill_(5)
    blk.n.fill_(5)
    woq.woq_add_rmsnorm(blk.d["x"], blk.d["w"], 1e-6, y=blk.n, b=0)
    woq.woq_qgemm_int8_a8(blk.w8.desc, blk.q, blk.qs, blk.y, b=0)
    woq.woq_lora_add(blk.pool.desc, blk.n, blk.d["ids"], blk.y, blk.y, blk.ws, b=0)
    assert np.all(host(blk.y) == 5) and np.all(host(blk.n) == 5)


@pytest.mark.parametrize("b", [3, 65, 300])
def test_rows_past_the_batch_are_left_as_they_were(gpu_lib, b):
    """Buffers of more rows than the call names: those behind stay untouched."""
    blk = Block(b + 5, 200, 130, b)
    for t in (blk.sum, blk.n, blk.y):
        t.fill_(9)
    blk.q.fill_(9)
    blk.qs.fill_(9)
    d = blk.d
    woq.woq_add_rmsnorm(d["x"], d["w"], 1e-6, res=d["res"], sum_out=blk.sum, y=blk.n, q=blk.q, q_scale=blk.qs, b=b)
    woq.woq_qgemm_int8_a8(blk.w8.desc, blk.q, blk.qs, blk.y, b=b)
    woq.woq_lora_add(blk.pool.desc, blk.n, d["ids"], blk.y, blk.y, blk.ws, b=b)
    for t in (blk.sum, blk.n, blk.y, blk.q):
        assert np.all(host(t)[b:] == 9)
    assert np.all(host(blk.qs)[b:] == 9)
    few = host(blk.y)[:b].copy()
    blk.run()                                     # all rows: the first b are the same
    q, base = host(blk.q), host(blk.n)
    s_ref, v_ref = O.add_rmsnorm(blk.x, blk.res, blk.w)
    within(base[:, :200], v_ref, np.abs(v_ref) * (H + 2.0 ** -17) + SUB)
    ref = O.linear_int8_a8(blk.codes, blk.ends, blk.scales, q[:, :200], host(blk.qs))
    out, spread = O.lora_add(ref, base[:, :200], blk.ids, blk.A, blk.B, blk.s, blk.ends)
    tol = (np.abs(ref) + np.abs(out)) * (H + 4 * U) + 2 * SUB + spread * ((200 / 16 + 48) * U + 2.0 ** -20)
    within(few, out[:b], tol[:b])
    within(host(blk.y), out, tol)


def test_two_streams_at_once(gpu_lib):
    """Runs on two streams with buffers of their own, interleaved, give the bits of
    runs one after the other."""
    import torch
    blocks = [Block(40, 1000, 500, 1), Block(40, 1000, 500, 2), Block(300, 640, 300, 3), Block(1, 2048, 700, 4)]
    want = []
    for blk in blocks:
        blk.run()
        want.append(host(blk.y).copy())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(20):
        for blk, s in zip(blocks, streams):
            blk.run(stream=s)
    torch.cuda.synchronize()
    for blk, w in zip(blocks, want):
        np.testing.assert_array_equal(host(blk.y).view(np.uint16), w.view(np.uint16))


def far_rows(rows, width, ld, dtype):
    import torch
    t = torch.empty((rows - 1) * ld + width, dtype=getattr(torch, dtype), device="cuda")
    return t.as_strided((rows, width), (ld, 1))


def test_offsets_past_32_bits_activations(gpu_lib):
    """Rows of activations, codes and outputs that lie more than 2^31 values apart."""
    import torch
    rows, K, N, ld = 5, 100, 70, 2 ** 29 + 64
    x, res, w = norm_case(rows, K, 1)
    big = {k: far_rows(rows, up(K, 8), ld, "float16") for k in ("x", "sum")}
    big["x"][:, :K] = torch.from_numpy(x).cuda()
    q, qs = far_rows(rows, up(K, 16), ld, "int8"), torch.empty(rows, device="cuda")
    case("norm far rows")
    woq.woq_add_rmsnorm(big["x"], dev(w), 1e-6, sum_out=big["sum"], q=q, q_scale=qs, K=K)
    s_ref, v_ref = O.add_rmsnorm(x, None, w)
    within(host(big["sum"].contiguous())[:, :K], s_ref, np.abs(s_ref) * (H + 2 * U) + SUB)
    qh = host(q.contiguous())
    within(qh[:, :K], v_ref / O.rows_scale(v_ref)[:, None], 0.5 + 127 * 2.0 ** -16)
    case("product far rows")
    rng = np.random.default_rng(2)
    codes, scales, w8 = a8_weight(N, K, rng)
    y = far_rows(rows, N, ld, "float16")
    woq.woq_qgemm_int8_a8(w8.desc, q, qs, y)
    ref = O.linear_int8_a8(codes, [N], scales, qh[:, :K], host(qs))
    within(host(y.contiguous()), ref, np.abs(ref) * (H + 4 * U) + SUB)
    for b in (rows, 300):                        # both forms of the adapters' kernels
        case("adapters far rows", b)
        A, B, s, ends = lora_pool(2, N, K, 16, 1, rng)
        pool = woq.DeviceLora(dev(A), dev(B), dev(s), K=K)
        step = ld if b == rows else 2 ** 23 + 8  # the last row past 2^31 either way
        xs, ys = far_rows(b, up(K, 8), step, "float16"), far_rows(b, N, step, "float16")
        xv = rng.standard_normal((b, K)).astype(np.float16)
        xs[:, :K] = torch.from_numpy(xv).cuda()
        ys.fill_(0.5)
        ids = rng.integers(-1, 2, b).astype(np.int32)
        ws = torch.empty(woq.woq_lora_workspace(pool.desc, b), dtype=torch.uint8, device="cuda")
        woq.woq_lora_add(pool.desc, xs, dev(ids), ys, ys, ws)
        ref, spread = O.lora_add(np.full((b, N), 0.5), xv, ids, A, B, s, ends)
        within(host(ys.contiguous()), ref, np.abs(ref) * (H + 2 * U) + SUB + spread * ((K / 16 + 48) * U + 2.0 ** -20))
        del xs, ys


def test_offsets_past_32_bits_weights(gpu_lib):
    """Weights and pools of more than 2^31 bytes or values: their last rows."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    N, K = 17000, woq.A8_MAX_K
    case("product large weight")
    codes = torch.randint(1, 256, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    w = woq.Int8W()
    w.codes, w.N, w.K, w.nseg = codes.data_ptr(), N, K, 1
    w.seg_end[0], w.seg_scale[0] = N, 2.0 ** -12
    for b in (2, 70):
        q = torch.randint(-127, 128, (b, K), generator=g, device="cuda", dtype=torch.int8)
        qs, y = torch.full((b,), 2.0 ** -6, device="cuda"), full(b, N, 0, "float16")
        woq.woq_qgemm_int8_a8(w, q, qs, y)
        at = torch.cat([torch.arange(20), torch.arange(N - 200, N)]).cuda()
        ref = ((q.double() @ (codes[at].double() - 128).t().contiguous()) * 2.0 ** -18).cpu().numpy()
        within(host(y[:, at]), ref, np.abs(ref) * (H + 4 * U) + SUB)
    del codes, q
    torch.cuda.empty_cache()
    count, N, K, R = 9, 2 ** 20 + 3, 64, 256
    case("adapters large pool")
    A = torch.randn(count, R, K, generator=g, device="cuda").half() * 0.125
    B = torch.zeros(count, N, R, dtype=torch.float16, device="cuda")
    at = torch.cat([torch.arange(40), torch.arange(N - 300, N)]).cuda()
    part = torch.randn(len(at), R, generator=g, device="cuda").half() * 0.25
    B[count - 1, at] = part
    s = torch.ones(count, device="cuda")
    pool = woq.DeviceLora(A, B, s)
    for b in (2, 257):
        x = torch.randn(b, K, generator=g, device="cuda").half()
        ids = torch.full((b,), count - 1, dtype=torch.int32, device="cuda")
        y = torch.empty(b, N, dtype=torch.float16, device="cuda")
        ws = torch.empty(woq.woq_lora_workspace(pool.desc, b), dtype=torch.uint8, device="cuda")
        woq.woq_lora_add(pool.desc, x, ids, None, y, ws)
        xd, Ad, Bd = x.double().cpu().numpy(), A[-1].double().cpu().numpy(), part.double().cpu().numpy()
        ref, spread = xd @ Ad.T @ Bd.T, np.abs(xd) @ np.abs(Ad).T @ np.abs(Bd).T
        within(host(y[:, at]), ref, np.abs(ref) * (H + 2 * U) + SUB + spread * ((K / 16 + R + 32) * U + 2.0 ** -20))
        assert not y[:, 1000:N - 1000].any()
    case("adapters rows of A far apart")
    count, R, K, lda = 3, 16, 40, 2 ** 26
    A = torch.zeros(count, R, lda, dtype=torch.float16, device="cuda")
    A[:, :, :K] = torch.randn(count, R, K, generator=g, device="cuda").half()
    B = torch.randn(count, 50, R, generator=g, device="cuda").half()
    pool = woq.DeviceLora(A, B, torch.ones(count, device="cuda"), K=K)
    for b in (3, 260):
        x = torch.randn(b, K, generator=g, device="cuda").half()
        ids = (torch.arange(b, device="cuda") % count).int()
        y = torch.empty(b, 50, dtype=torch.float16, device="cuda")
        ws = torch.empty(woq.woq_lora_workspace(pool.desc, b), dtype=torch.uint8, device="cuda")
        woq.woq_lora_add(pool.desc, x, ids, None, y, ws)
        ref, spread = O.lora_add(np.zeros((b, 50)), x.cpu().numpy(), host(ids), A[:, :, :K].cpu().numpy(), B.cpu().numpy(),
                                 np.ones(count), [50])
        within(host(y), ref, np.abs(ref) * (H + 2 * U) + SUB + spread * ((K / 16 + 48) * U + 2.0 ** -20))


def test_binding_checks_buffers_before_a_launch(gpu_lib):
    import torch
    blk = Block(4, 64, 48, 3)
    half = dict(dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        woq.woq_add_rmsnorm(blk.d["x"], blk.d["w"], 1e-6, y=torch.empty(3, 64, **half))          # rows
    with pytest.raises(ValueError):
        woq.woq_add_rmsnorm(blk.d["x"], blk.d["w"], 1e-6, y=torch.empty(4, 56, **half))          # width
    with pytest.raises(ValueError):
        woq.woq_add_rmsnorm(blk.d["x"].float(), blk.d["w"], 1e-6, y=blk.n)                       # type
    with pytest.raises(ValueError):
        woq.woq_add_rmsnorm(blk.d["x"].t(), blk.d["w"], 1e-6, y=blk.n, b=4)                      # strides
    with pytest.raises(ValueError):
        woq.woq_add_rmsnorm(blk.d["x"], blk.d["w"], 1e-6, q=blk.q, q_scale=blk.qs[:3])
    with pytest.raises(woq.WoqError) as e:
        woq.woq_add_rmsnorm(blk.d["x"], blk.d["w"], 0.0, y=blk.n)                                # eps
    assert e.value.status == woq.WOQ_EINVAL
    with pytest.raises(ValueError):
        woq.woq_qgemm_int8_a8(blk.w8.desc, blk.q[:, :48], blk.qs, blk.y)
    with pytest.raises(ValueError):
        woq.woq_qgemm_int8_a8(blk.w8.desc, blk.q, blk.qs, blk.y[:, :40])
    with pytest.raises(ValueError):
        woq.woq_lora_add(blk.pool.desc, blk.n, blk.d["ids"][:3], blk.y, blk.y, blk.ws)
    with pytest.raises(ValueError):
        woq.woq_lora_add(blk.pool.desc, blk.n, blk.d["ids"].long(), blk.y, blk.y, blk.ws)
    with pytest.raises(woq.WoqError) as e:
        woq.woq_lora_add(blk.pool.desc, blk.n, blk.d["ids"], blk.y, blk.y, blk.ws[:16])
    assert e.value.status == woq.WOQ_EINVAL
    torch.cuda.synchronize()
