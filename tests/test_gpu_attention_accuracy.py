"""GPU tests of how near the attention over the cache (woq_attn_decode) comes to
the formula in 64 bits: long rows, sharp and bounded scores, values far apart.

Tolerances count roundings as if they were independent, U = 2^-24 half a step of
fp32, H = 2^-11 of fp16, SUB = 2^-25 half the spacing of fp16's subnormals; each test
says how.
"""
import numpy as np
import pytest

import oracle as O
from test_gpu_decode import Cache, H, SUB, U, case, dev, host, tables, within
from weight_only_quantized_quantize_amd import woq

pytestmark = pytest.mark.gpu


def attend(c, q_heads, q, pages, lens, **kw):
    import torch
    b = len(lens)
    y = torch.full((b, q_heads * c.dim), 7.0, dtype=torch.float16, device="cuda")
    ws = torch.empty(woq.woq_attn_decode_workspace(c.desc, q_heads, b), dtype=torch.uint8, device="cuda")
    woq.woq_attn_decode(c.desc, dev(q), dev(np.asarray(pages, np.int32)), dev(np.asarray(lens, np.int32)), y, ws, **kw)
    return host(y).reshape(b, q_heads, c.dim)


def exact(c, q_heads, q, pages, lens, scale, softcap=0.0):
    """The formula over whole pages: y and sum p |v| of every row."""
    y, spread = [], []
    for r, n in enumerate(lens):
        t = np.arange(n)
        slots = np.asarray(pages)[r, t // c.page].astype(np.int64) * c.page + t % c.page
        a, s, _ = O.attend(q[r].reshape(q_heads, c.dim), c.tokens("k", slots), c.tokens("v", slots), scale, softcap)
        y.append(a), spread.append(s)
    return np.stack(y), np.stack(spread)


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("n,heads,q_heads,dim", [(131072, 2, 16, 128), (100001, 3, 12, 64), (60000, 1, 8, 256)])
def test_long_rows_give_the_nearest_fp16(gpu_lib, int8, n, heads, q_heads, dim):
    """Of random values, nearly every result is the fp16 number nearest to the exact
    one.  With independent roundings, relative to a result's usual size: the weights'
    are 2^-20 each (an argument of up to 16, its exponential, two fp16 halves), as is
    their effect on the sum, which is of random signs itself; the n / 8 of the sums (of
    16 tokens, weights in two halves) are U / sqrt(3) of a partial sum, 0.7 of the
    result in the mean: at 131072 tokens 2^-18.3.  Both are 2^-18, and a result is
    rounded to another number where that reaches past the middle between two: 0.8 2^-18
    of a step of 2^-10.5 in the mean of those that are half the usual size at least,
    0.5%.  Four times that is allowed."""
    case("long rows", int8, n, heads, q_heads, dim)
    c = Cache(-(-n // 64) + 1, heads, 64, dim, int8, seed=30)
    rng = np.random.default_rng(31)
    q = rng.standard_normal((1, q_heads * dim)).astype(np.float16)
    pages = tables(rng, c, [n])
    y, ref = attend(c, q_heads, q, pages, [n]), exact(c, q_heads, q, pages, [n], dim ** -0.5)[0]
    large = np.abs(ref) > 0.5 * np.sqrt(np.mean(ref ** 2))
    off = np.mean((y != ref.astype(np.float16))[large])
    print("not the nearest: %.3f%%" % (100 * off), flush=True)
    assert off <= 0.02, off


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("width", [None, 100])
def test_sharp_scores(gpu_lib, int8, width):
    """A few keys along the queries decide.  A score is a sum of dim products, each
    rounding of the sum at most U of the largest partial sum, |q| |k|: sqrt(dim) of
    them, four times that allowed, and eight roundings of the score itself; twice, for
    the row's largest.  Weights, halves and exponentials lose 2^-19, sums of few
    tokens 200 U."""
    case("sharp", int8, width)
    D, q_heads, n = 128, 8, 700
    rng = np.random.default_rng(40)
    c = Cache(50, 2, 16, D, False, seed=41)
    q = rng.standard_normal((2, q_heads, D)).astype(np.float16)
    lens = [n, 33]
    pages = tables(rng, c, lens, width=width)
    k = c.k.astype(np.float32)
    for r, m in enumerate(lens):
        for h in range(q_heads):
            for t in rng.integers(0, m, 3):                     # scores of about 128 * 0.3 * 0.7
                k[pages[r, t // 16], h // 4, t % 16] = 0.3 * q[r, h] + 0.1 * rng.standard_normal(D)
    if int8:
        c.int8, c.vs = True, np.abs(c.v).max(-1).astype(np.float32) / np.float32(127)
        c.ks = np.abs(k).max(-1) / np.float32(127)
        c.v, c.k = ((np.rint(t.astype(np.float32) / s[..., None]) + 128).astype(np.uint8)
                    for t, s in ((c.v, c.vs), (k, c.ks)))
    else:
        c.k = k.astype(np.float16)
    c.upload()
    scale = 0.7
    y, (ref, spread) = attend(c, q_heads, q.reshape(2, -1), pages, lens, scale=scale), \
        exact(c, q_heads, q.reshape(2, -1), pages, lens, scale)
    kn = np.linalg.norm(c.values("k"), axis=-1).max()
    for r in range(2):
        reach = scale * np.linalg.norm(q[r].astype(float), axis=-1).max() * kn
        rel = 2 * (4 * np.sqrt(D) + 8) * U * reach + 2.0 ** -19 + 200 * U
        assert rel < 1e-2
        within(y[r], ref[r], spread[r] * rel + np.abs(ref[r]) * H + SUB, ("row", r))


@pytest.mark.parametrize("int8", [True, False])
def test_scores_of_whole_numbers(gpu_lib, int8):
    """Keys and queries are whole numbers and factors powers of two, so that every
    score is exact in fp32 whatever the order; what is left are three roundings of the
    score in units of log2, |z| <= 64, weights and sums."""
    D, q_heads, n = 64, 4, 400
    rng = np.random.default_rng(50)
    c = Cache(30, 1, 16, D, True, seed=51)
    c.k = (128 + rng.integers(-127, 128, c.k.shape)).astype(np.uint8)
    c.ks[...] = 2.0 ** -6
    q = rng.integers(-4, 5, (1, q_heads * D)).astype(np.float16)
    if not int8:
        c.k = ((c.k.astype(np.float32) - 128) * 2.0 ** -6).astype(np.float16)
        c.v = ((c.v.astype(np.float32) - 128) * c.vs[..., None]).astype(np.float16)
        c.int8 = False
    c.upload()
    pages = tables(rng, c, [n])
    y, (ref, spread) = attend(c, q_heads, q, pages, [n], scale=0.25), exact(c, q_heads, q, pages, [n], 0.25)
    rel = 2 * 3 * 64 * U + 2.0 ** -19 + 200 * U
    within(y, ref, spread * rel + np.abs(ref) * H + SUB)


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("softcap", [1.0, 8.0, 50.0, 1e3, 1e4, 1e6, 1e8, 1e12, 2.0 ** 64])
def test_bounded_scores_of_any_bound(gpu_lib, int8, softcap):
    """Scores of up to some 40 under bounds from far below to far above them.  A score
    is off by a sum's roundings as in the sharp scores' test, which the bound never
    raises (tanh's slope is at most 1), and by 2^-22 of itself for tanh and eight
    roundings, all relative to it however large the bound."""
    case("softcap", int8, softcap)
    D, q_heads, lens = 128, 6, [700, 33, 2, 150]
    c = Cache(80, 2, 16, D, int8, seed=60)
    rng = np.random.default_rng(61)
    q = (rng.standard_normal((4, q_heads * D)) * 4).astype(np.float16)
    pages = tables(rng, c, lens)
    y = attend(c, q_heads, q, pages, lens, softcap=softcap)
    ref, spread = exact(c, q_heads, q, pages, lens, D ** -0.5, softcap)
    kn = np.linalg.norm(c.values("k"), axis=-1).max()
    for r in range(4):
        reach = D ** -0.5 * np.linalg.norm(q[r].reshape(q_heads, D).astype(float), axis=-1).max() * kn
        rel = 2 * ((4 * np.sqrt(D) + 8) * U + 2.0 ** -22) * reach + 2.0 ** -19 + 200 * U
        assert rel < 1e-2
        within(y[r], ref[r], spread[r] * rel + np.abs(ref[r]) * H + SUB, ("row", r))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,width", [([1], None), ([40], None), ([300, 1, 77], None), ([300, 1, 77], 150), ([9000], None)])
def test_values_that_are_infinite(gpu_lib, dim, lens, width):
    """An infinity among the visible values of an fp16 cache gives infinity, as it
    does times any weight and in any sum; two of different signs, or a NaN, give NaN;
    other channels are what they are without it."""
    case("infinite values", dim, lens)
    q_heads, page = 4, 16
    c = Cache(sum(-(-n // page) for n in lens) + 1, 2, page, dim, False, seed=70)
    rng = np.random.default_rng(71)
    q = (rng.standard_normal((len(lens), q_heads * dim)) * 0.5).astype(np.float16)
    pages = tables(rng, c, lens, width=width)
    plain = attend(c, q_heads, q, pages, lens)
    want = plain.copy()

    def put(r, t, h, d, x):
        c.v[pages[r, t // page], h, t % page, d] = x

    for r, n in enumerate(lens):
        at = rng.permutation(n)
        put(r, at[0], 0, 3, np.inf)
        put(r, at[0], 1, 5, -np.inf)
        put(r, at[-1], 0, 17, np.nan)
        for t in at[:5]:
            put(r, t, 1, 40, np.inf)
        want[r, :2, 3], want[r, 2:, 5], want[r, :2, 17], want[r, 2:, 40] = np.inf, -np.inf, np.nan, np.inf
        if n > 1:
            put(r, at[0], 0, dim - 1, np.inf)
            put(r, at[1], 0, dim - 1, -np.inf)
            want[r, :2, dim - 1] = np.nan
    c.upload()
    np.testing.assert_array_equal(attend(c, q_heads, q, pages, lens), want)


@pytest.mark.parametrize("dim,n,width", [(64, 60, None), (128, 700, None), (128, 700, 100), (256, 5000, None)])
@pytest.mark.parametrize("large,small", [(2.0 ** 9, 2.0 ** -20), (2.0 ** 15, 2.0 ** -15), (2.0 ** 30, 2.0 ** -8),
                                         (2.0 ** 30, 2.0 ** 8), (2.0 ** -10, 2.0 ** -20)])
def test_scales_of_values_that_hardly_count(gpu_lib, dim, n, width, large, small):
    """INT8 values of which the largest by far have next to no weight: what counts are
    the others, and they keep their bits.  Weights times their scales below 2^-40 of the
    largest such product may be lost, the rest is as in the sharp scores' test."""
    case("scales apart", dim, n, width, large, small)
    q_heads = 8
    rng = np.random.default_rng(80)
    c = Cache(-(-n // 16) + 1, 2, 16, dim, True, seed=81)
    q = rng.standard_normal((1, q_heads, dim)).astype(np.float16)
    q[0, :, 0] = 8
    pages = tables(rng, c, [n], width=width)
    c.vs = (small * rng.uniform(0.5, 1, c.vs.shape)).astype(np.float32)
    c.k = (128 + np.rint((c.k.astype(float) - 128) / 8)).astype(np.uint8)
    c.k[..., 0] = 128 + 100                 # all keys share a component along the queries,
    c.ks[...] = 0.04
    far = rng.permutation(n)[:max(3, n // 20)]
    for t in far:                           # but for those, whose weights are 2^-80 and less
        c.k[pages[0, t // 16], :, t % 16, 0] = 1
        c.vs[pages[0, t // 16], :, t % 16] = large * rng.uniform(0.5, 1, 2)
    c.upload()
    flat, scale = q.reshape(1, -1), 1.0
    y = attend(c, q_heads, flat, pages, [n], scale=scale)[0]
    ref, spread = (a[0] for a in exact(c, q_heads, flat, pages, [n], scale))
    slots = pages[0, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16
    K, sv = c.tokens("k", slots), c.vs[slots // 16, :, slots % 16].astype(np.float64)
    kn = np.linalg.norm(K, axis=-1).max()
    for h in range(q_heads):
        z = K[:, h // 4] @ q[0, h].astype(np.float64) * scale
        p = np.exp(z - z.max())
        assert p[far].max() / p.sum() * large < 2.0 ** -20 * small
        p /= p.sum()
        lost = n * 2.0 ** -40 * 127 * (p * sv[:, h // 4]).max()
        rel = 2 * (4 * np.sqrt(dim) + 8) * U * scale * np.linalg.norm(q[0, h].astype(float)) * kn + 2.0 ** -19 + (n / 8 + 200) * U
        assert rel < 1e-2
        within(y[h], ref[h], spread[h] * rel + np.abs(ref[h]) * H + SUB + lost, ("head", h))
