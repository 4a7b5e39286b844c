"""GPU tests of the operators between a decode step's products and behind its
head (woq_cache_write, woq_cache_read, woq_attn_decode, woq_sample) against their
float64 definitions.

Tolerances count roundings: U = 2^-24 is half a step of fp32, H = 2^-11 of fp16,
SUB = 2^-25 half the spacing of fp16's subnormals.

* rotation: two products and a sum, at most 3 U of |a c| + |b s|.
* codes of turned keys: |v / scale - code| <= 1/2 plus that error over the scale,
  and 127 * 2 U of the scale's own; values nothing turns are bit for bit the
  encoder's.
* attention: a score is a sum of dim exact products in fp32, then at most 8
  roundings (its factors, the exponential's argument): (dim + 8) U of its terms'
  magnitudes (reach), and as much again for the row's largest score; two fp16
  halves of a weight lose 2^-22 of it, its exponential, its argument and the token's
  scale 2^-19; the sums of n tokens are at most n / 16 + 96 roundings long, twice
  (values and weights): all of them relative to spread = sum p |v|.  Weights below 2^-40 of the largest may be lost: n 2^-40 max |v|.
  The result is rounded to fp16.  INT8 bytes u = code + 128 are multiplied as they
  are and 128 times the factor's sum is taken off in fp32, so the magnitudes that
  fp32's roundings are relative to are those of u, at most |code| + 128: reach grows by
  128 max ks sum |q|, and for the sums (not for the weights' halves, which are the
  same in both) spread by 128 sum p sv.
* a token is the definition's, exactly; its share is rounded to fp32 once.
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


def within(y, ref, tol, what=""):
    y = y.astype(np.float64)
    err = np.abs(y - ref)
    bad = ~(err <= tol)
    assert not bad.any(), (what, np.argwhere(bad)[:4], y[bad][:4], ref[bad][:4], np.broadcast_to(tol, err.shape)[bad][:4])


class Cache:
    """A cache on the device and on the host: random contents, or a poison that no
    call may read as a value (NaN scales, NaN values)."""

    def __init__(self, n_pages, heads, page, dim, int8=True, seed=0, poison=False):
        import torch
        rng = np.random.default_rng(seed)
        shape = (n_pages, heads, page, dim)
        self.shape, self.int8, self.heads, self.page, self.dim = shape, int8, heads, page, dim
        self.k, self.v = (rng.standard_normal(shape).astype(np.float16) for _ in range(2))
        self.k[..., ::7] *= 4
        self.ks = self.vs = None
        if int8:
            self.ks, self.vs = (np.abs(t).max(-1).astype(np.float32) / np.float32(127) for t in (self.k, self.v))
            self.k, self.v = (np.clip(np.rint(t.astype(np.float32) / s[..., None]), -127, 127).astype(np.int64)
                              for t, s in ((self.k, self.ks), (self.v, self.vs)))
            self.k, self.v = (self.k + 128).astype(np.uint8), (self.v + 128).astype(np.uint8)
        if poison:
            for t in (self.k, self.v):
                t[...] = 255 if int8 else np.nan
            if int8:
                self.ks[...] = self.vs[...] = np.nan
        self.upload()

    def upload(self):
        self.d = woq.DeviceCache(dev(self.k), dev(self.v), *((dev(self.ks), dev(self.vs)) if self.int8 else ()))
        self.desc = self.d.desc

    def values(self, which):
        """float64 [n_pages, heads, page, dim] of the host's copy."""
        t, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        return (t.astype(np.float64) - 128) * s[..., None].astype(np.float64) if self.int8 else t.astype(np.float64)

    def tokens(self, which, slots):
        v, slots = self.values(which), np.asarray(slots)
        return v[slots // self.page, :, slots % self.page]

    def now(self):
        """What the device holds: (k, v, k scales, v scales)."""
        return tuple(None if t is None else host(t) for t in (self.d.k, self.d.v, self.d.k_scale, self.d.v_scale))


# ------------------------------------------------------------ write and read

def rope_table(n_pos, rot):
    a = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def check_write(c, b, q_heads, rot, interleaved, slots, pos, seed=0, n_pos=50, pad=0, special=False):
    """One call with q, k and v side by side in rows that are wider by ``pad``;
    everything that no slot names has to stay."""
    import torch
    rng = np.random.default_rng(seed)
    D, Hk = c.dim, c.heads
    n, m = q_heads * D, Hk * D
    x = rng.standard_normal((b, n + 2 * m + pad)).astype(np.float16) * np.float16(3)
    if special:
        x[0, n:n + D] = 0
        x[1, n + m:n + m + D] = np.nan
        x[2, n + D - 1] = np.inf
    before = c.now()
    xd = dev(x)
    rope = rope_table(n_pos, rot) if rot else None
    out = torch.full((b, n + 8), 7.0, dtype=torch.float16, device="cuda")
    kw = dict(rope=dev(rope), pos=dev(np.asarray(pos, np.int32)), interleaved=interleaved) if rot else {}
    if q_heads:
        kw.update(q=xd[:, :n], q_out=out[:, :n])
    slots = np.asarray(slots, np.int32)
    woq.woq_cache_write(c.desc, xd[:, n:n + m], xd[:, n + m:n + 2 * m], dev(slots), **kw)
    after = c.now()
    parts = {"q": x[:, :n].reshape(b, q_heads, D), "k": x[:, n:n + m].reshape(b, Hk, D),
             "v": x[:, n + m:n + 2 * m].reshape(b, Hk, D)}
    ref, mag = {}, {}
    with np.errstate(invalid="ignore"):
        for name, t in parts.items():
            if rot and name != "v":
                at = np.clip(pos, 0, n_pos - 1)
                ref[name] = O.rotate(t, rope, at, interleaved)
                mag[name] = np.abs(ref[name])
                # |a c| + |b s| is at most |a| + |b|
                a = np.abs(t.astype(np.float64))
                pair = np.arange(D)
                i = pair[:rot]
                pair[:rot] = (i ^ 1) if interleaved else (i + rot // 2) % rot
                mag[name][..., :rot] = (a + a[..., pair])[..., :rot]
                lost = [r for r in range(b) if not 0 <= pos[r] < n_pos]
                for r in lost:
                    ref[name][r, :, :rot] = np.nan
            else:
                ref[name], mag[name] = t.astype(np.float64), np.zeros(t.shape)
    if q_heads:
        got = host(out)
        assert np.all(got[:, n:] == 7)
        y, want = got[:, :n].reshape(b, q_heads, D), ref["q"]
        np.testing.assert_array_equal(np.isnan(y), np.isnan(want))
        ok = ~np.isnan(want)
        within(y[ok], want[ok], np.abs(want[ok]) * H + 4 * U * mag["q"][ok] + SUB, "q")
    named = np.zeros(before[0].shape[:3], bool)
    for r, s in enumerate(slots):
        if not 0 <= s < c.shape[0] * c.page:
            continue
        p, o = divmod(int(s), c.page)
        named[p, :, o] = True
        for i, name in enumerate(("k", "v")):
            turned = rot and name == "k"
            for h in range(Hk):
                want, stored = ref[name][r, h], after[i][p, h, o]
                if not c.int8:
                    np.testing.assert_array_equal(np.isnan(stored), np.isnan(want))
                    if not turned:
                        np.testing.assert_array_equal(stored.view(np.uint16), parts[name][r, h].view(np.uint16))
                    elif np.all(np.isfinite(want)):
                        within(stored, want, np.abs(want) * H + 4 * U * mag[name][r, h] + SUB, name)
                    continue
                scale = after[2 + i][p, h, o]
                if not np.all(np.isfinite(want)):
                    assert np.isnan(scale) and np.all(stored == 128), (r, name, h)
                elif not turned:
                    codes, s1 = O.quantize_int8(parts[name][r, h][None].astype(np.float32))
                    assert np.float32(s1) == scale
                    np.testing.assert_array_equal(stored.astype(int) - 128, codes[0])
                elif not want.any():
                    assert scale == 0 and np.all(stored == 128)
                else:
                    true = np.abs(want).max() / 127
                    slack = 4 * U * mag[name][r, h].max()
                    assert abs(scale - true) <= slack / 127 + true * 2 * U
                    within(stored.astype(int) - 128, want / true, 0.5 + 2 * slack / true + 127 * 4 * U, name)
                    assert np.all(np.abs(stored.astype(int) - 128) <= 127)
    for i in range(4):
        if before[i] is not None:
            keep = ~named
            np.testing.assert_array_equal(after[i][keep].view(np.uint8), before[i][keep].view(np.uint8))


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("heads,dim,page,b,q_heads,rot,inter", [
    (1, 16, 16, 1, 1, 16, False), (8, 128, 16, 1, 64, 128, False), (8, 256, 64, 3, 16, 256, True),
    (5, 96, 48, 33, 20, 32, False), (3, 80, 32, 7, 3, 80, True), (12, 64, 128, 5, 12, 64, False),
    (2, 48, 16, 100, 0, 0, False), (1, 240, 16, 9, 2, 224, False), (4, 112, 96, 20, 4, 16, True),
    (7, 32, 16, 64, 0, 32, True)])
def test_write_sizes(gpu_lib, int8, heads, dim, page, b, q_heads, rot, inter):
    case("write", int8, heads, dim, page, b, q_heads, rot, inter)
    rng = np.random.default_rng(b)
    c = Cache(-(-b // page) + 2, heads, page, dim, int8, seed=1)
    slots = rng.permutation(c.shape[0] * page)[:b]
    if b > 4:
        slots[[1, 3]] = -1, c.shape[0] * page
    check_write(c, b, q_heads, rot, inter, slots, rng.integers(0, 50, b), pad=8 * (b % 3))


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("rot", [0, 64])
def test_write_rows_of_zeros_nan_and_infinity(gpu_lib, int8, rot):
    c = Cache(3, 2, 16, 64, int8)
    check_write(c, 6, 4 if rot else 0, rot, False, [5, 40, 17, 0, 47, 31], [0, 1, 49, 3, 50, -1], special=True)


def test_write_keeps_distant_places_and_ties(gpu_lib):
    """A head whose scale is a power of two: halves go to the even code; the first
    and the last slot; -1, -2^31 and 2^31 - 1 are no slots."""
    import torch
    c = Cache(4, 1, 16, 64, True)
    x = np.zeros((2, 64), np.float16)
    x[0] = np.arange(64) / 2 - 16
    x[0, 63] = 127
    x[1] = -x[0]
    rows = dev(np.concatenate([x, x[:1], x[:1], x[:1]]))
    slots = np.array([0, 63, -1, -2 ** 31, 2 ** 31 - 1], np.int32)
    woq.woq_cache_write(c.desc, rows, rows, dev(slots))
    k, v, ks, vs = c.now()
    assert ks[0, 0, 0] == 1 and ks[3, 0, 15] == 1
    np.testing.assert_array_equal(k[0, 0, 0].astype(int) - 128, np.rint(x[0].astype(float)))
    np.testing.assert_array_equal(v[3, 0, 15].astype(int) - 128, np.rint(x[1].astype(float)))
    out = torch.empty(5, 64, dtype=torch.float16, device="cuda")
    woq.woq_cache_read(c.desc, dev(slots), out)
    got = host(out)
    np.testing.assert_array_equal(got[:2], np.rint(x.astype(float)))
    assert not got[2:].any()


def test_write_turns_q_in_place_and_leaves_rows_behind(gpu_lib):
    import torch
    rng = np.random.default_rng(3)
    c = Cache(2, 2, 16, 64, True)
    x = rng.standard_normal((9, 4 * 64 + 256)).astype(np.float16)
    xd, rope, pos = dev(x), rope_table(30, 32), rng.integers(0, 30, 9).astype(np.int32)
    woq.woq_cache_write(c.desc, xd[:, 256:384], xd[:, 384:], dev(np.arange(9, dtype=np.int32)), q=xd[:, :256],
                        q_out=xd[:, :256], rope=dev(rope), pos=dev(pos), b=7)
    got = host(xd)
    np.testing.assert_array_equal(got[7:], x[7:])
    np.testing.assert_array_equal(got[:, 256:], x[:, 256:])
    ref = O.rotate(x[:7, :256].reshape(7, 4, 64), rope, pos).reshape(7, 256)
    within(got[:7, :256], ref, np.abs(ref) * H + 4 * U * 12 + SUB)


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("heads,dim,page,n", [(1, 16, 16, 1), (8, 128, 16, 133), (3, 80, 48, 77), (8, 256, 64, 40),
                                              (5, 64, 32, 1000), (1, 112, 16, 5)])
def test_read_back(gpu_lib, int8, heads, dim, page, n):
    """Slots in any order, some twice, some that are none; one of the two alone."""
    import torch
    case("read", int8, heads, dim, page, n)
    rng = np.random.default_rng(n)
    c = Cache(9, heads, page, dim, int8, seed=2)
    slots = rng.integers(0, 9 * page, n)
    if n > 4:
        slots[[0, 3]] = -5, 9 * page
    width = heads * dim
    k, v = (torch.full((n + 1, width + 16), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    idx = dev(slots.astype(np.int32))
    for ko, vo in ((k[:, :width], v[:, :width]), (k[:, :width], None), (None, v[:, :width])):
        for t in (k, v):
            t.fill_(7.0)
        woq.woq_cache_read(c.desc, idx, ko, vo, n=n)
        for t, asked, which in ((k, ko, "k"), (v, vo, "v")):
            got = host(t)
            assert np.all(got[n] == 7) and np.all(got[:, width:] == 7)
            if asked is None:
                assert np.all(got == 7)
                continue
            on = (slots >= 0) & (slots < 9 * page)
            ref = c.tokens(which, np.where(on, slots, 0)).reshape(n, width)
            if int8:           # the product in fp32, then fp16, both to nearest even
                p, o = np.where(on, slots, 0) // page, np.where(on, slots, 0) % page
                codes, scale = ((c.k, c.ks) if which == "k" else (c.v, c.vs))
                ref = ((codes[p, :, o].astype(np.float32) - 128) * scale[p, :, o][..., None]).reshape(n, width)
            ref = np.where(on[:, None], ref, 0).astype(np.float16)
            np.testing.assert_array_equal(got[:n, :width], ref)


# --------------------------------------------------------------- attention

def tables(rng, c, lens, width=None, spare=0):
    """Pages of a shuffled pool for every row, -1 behind the last."""
    need = [-(-max(int(n), 0) // c.page) for n in lens]
    W = max(max(need), 1) if width is None else width
    order = rng.permutation(c.shape[0])
    t = np.full((len(lens), W + spare), -1, np.int32)
    first = 0
    for r, n in enumerate(need):
        n = min(n, W)
        t[r, :n] = order[first:first + n]
        first += n
    assert first <= c.shape[0]
    return t


def check_attention(c, q_heads, lens, seed=0, window=0, softcap=0.0, scale=None, pages=None, spread=1.0, got=None,
                    q=None, width=None):
    import torch
    rng = np.random.default_rng(seed)
    b, D = len(lens), c.dim
    n = q_heads * D
    if q is None:
        q = (rng.standard_normal((b, n)) * spread).astype(np.float16)
    if pages is None:
        pages = tables(rng, c, lens, width)
    scale = D ** -0.5 if scale is None else scale
    y = torch.full((b + 1, n + 8), 7.0, dtype=torch.float16, device="cuda")
    size = woq.woq_attn_decode_workspace(c.desc, q_heads, b)
    ws = torch.full((size // 4 + 64,), float("nan"), device="cuda")
    if got is None:
        wide = np.full((b, n + 24), np.nan, np.float16)
        wide[:, :n] = q
        woq.woq_attn_decode(c.desc, dev(wide)[:, :n], dev(pages), dev(np.asarray(lens, np.int32)), y[:, :n], ws[:size // 4],
                            scale=scale, softcap=softcap, window=window, b=b)
        got = host(y)
        assert np.all(got[b] == 7) and np.all(got[:, n:] == 7)
        assert np.all(np.isnan(host(ws)[size // 4:]))
        got = got[:b, :n]
    for r in range(b):
        end = min(max(int(lens[r]), 0), pages.shape[1] * c.page)
        t = np.arange(max(0, end - window) if window else 0, end)
        at = pages[r, t // c.page].astype(np.int64)
        on = (at >= 0) & (at < c.shape[0])
        slots = at[on] * c.page + t[on] % c.page
        K, V = c.tokens("k", slots), c.tokens("v", slots)
        ref, mag, reach = O.attend(q[r].reshape(q_heads, D), K, V, scale, softcap)
        m = len(slots)
        sums = mag
        if c.int8 and m:
            ks, sv = (s[slots // c.page, :, slots % c.page].astype(np.float64) for s in (c.ks, c.vs))
            of = np.arange(q_heads) // (q_heads // c.heads)
            reach = reach + 128 * abs(scale) * (ks.max(0)[of] * np.abs(q[r].astype(float)).reshape(q_heads, D).sum(1))[:, None]
            sums = mag + O.attend(q[r].reshape(q_heads, D), K, np.repeat(128 * sv[..., None], D, 2), scale, softcap)[0]
        dz = reach * (D + 8) * U
        rel = 2.0 ** -22 + 3 * dz + 2.0 ** -19 + softcap * 2.0 ** -21
        tol = mag * rel + sums * 2 * (m / 16 + 96) * U + np.abs(ref) * H + SUB + (m * 2.0 ** -40 * np.abs(V).max() if m else 0)
        within(got[r].reshape(q_heads, D), ref, tol, ("row", r, "of", b, "len", int(lens[r])))
    return got


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("heads,q_heads,dim,page", [
    (8, 64, 128, 16), (8, 16, 256, 64), (8, 32, 128, 48), (12, 12, 64, 16), (5, 20, 96, 32), (1, 16, 128, 128),
    (1, 40, 64, 16), (2, 6, 80, 16), (1, 1, 16, 16), (1, 17, 256, 16), (3, 3, 240, 32), (2, 66, 48, 16), (4, 28, 128, 256),
    (1, 32, 64, 16), (1, 32, 128, 16), (1, 48, 128, 32), (2, 128, 64, 16), (1, 71, 64, 16), (1, 33, 80, 16), (2, 40, 96, 48),
    (1, 17, 16, 16)])
def test_attention_head_layouts(gpu_lib, int8, heads, q_heads, dim, page):
    """Over tables of just the pages needed and over wide ones: a short table's
    rows are a workgroup's whole, a long one's are divided."""
    case("attention", int8, heads, q_heads, dim, page)
    lens = [300, 1, 0, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255]
    c = Cache(sum(-(-n // page) for n in lens) + 2, heads, page, dim, int8, seed=heads)
    check_attention(c, q_heads, lens, seed=dim)
    check_attention(c, q_heads, lens, seed=dim, width=2000 // page)


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("b", [1, 2, 3, 7, 64, 257])
def test_attention_batches(gpu_lib, int8, b):
    rng = np.random.default_rng(b)
    lens = rng.integers(0, 200, b)
    lens[0] = 199
    case("attention batch", int8, b)
    c = Cache(int(sum(-(-lens // 16))) + 1, 2, 16, 64, int8, seed=b)
    check_attention(c, 8, lens, seed=b)
    check_attention(c, 8, lens, seed=b, width=100)


@pytest.mark.parametrize("int8,heads,q_heads,dim,page,lens", [
    (True, 8, 64, 128, 64, [5000]), (False, 2, 4, 256, 48, [6001, 3]), (True, 1, 8, 128, 16, [30001]),
    (True, 2, 16, 64, 256, [9000, 0, 1, 12000, 77]), (False, 1, 3, 80, 32, [20011]),
    (True, 2, 2, 64, 16, [0] * 40 + [700] + [0] * 300 + [3, 40] * 60 + [0] * 40),
    (False, 3, 60, 16, 16, [2000, 1, 0, 5000]), (True, 8, 128, 256, 16, [1000, 3000]),
    (True, 1, 40, 64, 64, [30000, 7, 900]), (False, 1, 32, 128, 16, [9000]), (True, 2, 96, 128, 16, [4000, 0, 2100])])
def test_attention_long(gpu_lib, int8, heads, q_heads, dim, page, lens):
    case("attention long", int8, heads, q_heads, dim, page, lens)
    c = Cache(sum(-(-n // page) for n in lens) + 1, heads, page, dim, int8, seed=7)
    check_attention(c, q_heads, lens, seed=3)


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 128, 333, 100000])
def test_attention_window(gpu_lib, int8, window):
    """What lies outside the window is poison, and its pages are not there."""
    case("attention window", int8, window)
    lens = [0, 1, 2, 16, 17, 100, 128, 129, 500, 333, 431]
    page = 16
    rng = np.random.default_rng(window)
    c = Cache(sum(-(-n // page) for n in lens) + 1, 2, page, 64, int8, seed=5, poison=True)
    good = Cache(c.shape[0], 2, page, 64, int8, seed=5)
    pages = tables(rng, c, lens)
    for r, n in enumerate(lens):
        for t in range(max(0, n - window), n):
            p, o = pages[r, t // page], t % page
            for a in ("k", "v", "ks", "vs"):
                if getattr(c, a) is not None:
                    getattr(c, a)[p, :, o] = getattr(good, a)[p, :, o]
        pages[r, :max(0, n - window) // page] = 2 ** 31 - 1
    c.upload()
    check_attention(c, 4, lens, seed=window, window=window, pages=pages)
    wide = np.full((len(lens), 77), -1, np.int32)
    wide[:, :pages.shape[1]] = pages
    check_attention(c, 4, lens, seed=window, window=window, pages=wide)


@pytest.mark.parametrize("int8", [True, False])
def test_attention_does_not_see_past_the_end(gpu_lib, int8):
    """Poison behind the last token of every row, in its page and in others."""
    lens = [1, 5, 16, 20, 31, 33, 64, 100, 250]
    rng = np.random.default_rng(1)
    for page, more in ((16, 3), (64, 3), (16, 40)):
        c = Cache(sum(-(-n // page) for n in lens) + 1, 2, page, 128, int8, seed=6, poison=True)
        good = Cache(c.shape[0], 2, page, 128, int8, seed=6)
        pages = tables(rng, c, lens, width=-(-250 // page) + more)
        for r, n in enumerate(lens):
            for t in range(n):
                for a in ("k", "v", "ks", "vs"):
                    if getattr(c, a) is not None:
                        getattr(c, a)[pages[r, t // page], :, t % page] = getattr(good, a)[pages[r, t // page], :, t % page]
            pages[r, -(-n // page):] = pages[0, 0]       # entries behind the last page name some other
        c.upload()
        check_attention(c, 16, lens, pages=pages)


@pytest.mark.parametrize("int8", [True, False])
def test_attention_pages_that_are_not_there(gpu_lib, int8):
    lens = [200, 200, 40, 16, 90]
    c = Cache(50, 2, 16, 64, int8, seed=8)
    rng = np.random.default_rng(2)
    pages = tables(rng, c, lens)
    pages[0, [0, 3, 4, 12]] = -1, 50, -2 ** 31, 2 ** 31 - 1
    pages[2] = -7                                        # nothing left: zeros
    pages[3, 0] = 50
    pages[4, 1:5] = -1
    for more in (0, 60):
        wide = np.concatenate([pages, np.full((5, more), 3, np.int32)], 1)
        got = check_attention(c, 6, lens, pages=wide)
        assert not got[2].any() and not got[3].any()


def test_attention_lengths_outside_the_table(gpu_lib):
    """Lengths below zero are zero, above the table's pages all of them."""
    c = Cache(12, 1, 16, 64, True, seed=9)
    pages = np.arange(12, dtype=np.int32).reshape(4, 3)
    got = check_attention(c, 2, [-1, -2 ** 31, 49, 2 ** 31 - 1], pages=pages)
    assert not got[:2].any() and got[2].any()


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("softcap,scale,spread", [(50.0, None, 1.0), (5.0, 0.5, 3.0), (0.0, 1.0, 4.0), (0.0, -0.3, 1.0),
                                                  (0.0, 0.0, 1.0), (30.0, 0.0625, 20.0), (0.0, 2.0, 8.0)])
def test_attention_scores(gpu_lib, int8, softcap, scale, spread):
    """Flat, sharp and bounded scores; a negative scale."""
    case("attention scores", int8, softcap, scale, spread)
    lens = [700, 33, 2, 150]
    c = Cache(80, 2, 16, 128, int8, seed=10)
    check_attention(c, 6, lens, softcap=softcap, scale=scale, spread=spread, seed=4)


def test_attention_scales_far_apart(gpu_lib):
    """Values whose scales differ by many powers of two, heads of zeros, and the
    largest values where the weights are smallest."""
    c = Cache(24, 2, 16, 64, True, seed=11)
    rng = np.random.default_rng(5)
    c.vs *= 2.0 ** rng.integers(-25, 12, c.vs.shape).astype(np.float32)
    c.v[3:5], c.vs[3:5] = 128, 0
    c.upload()
    check_attention(c, 8, [300, 64], seed=6)
    check_attention(c, 8, [300, 64], seed=6, spread=6.0)
    # one token decides, with a scale far below that of the tokens that count for nothing
    c = Cache(4, 1, 16, 64, True, seed=12)
    q = np.ones((1, 64), np.float16)
    c.k[...], c.vs[...] = 128 - 100, 2.0 ** 10
    c.k[2, 0, 5], c.vs[2, 0, 5] = 128 + 100, 2.0 ** -14
    c.ks[...] = 1.0
    c.upload()
    pages = np.arange(4, dtype=np.int32)[None]
    check_attention(c, 1, [64], q=q, pages=pages, scale=0.01)
    # heads of zeros only
    c.v[...], c.vs[...] = 128, 0
    c.upload()
    assert not check_attention(c, 1, [64], q=q, pages=pages).any()


def test_attention_of_what_is_not_finite(gpu_lib):
    """A NaN among the visible makes its head NaN, and no other."""
    for int8 in (True, False):
        c = Cache(20, 2, 16, 64, int8, seed=13)
        rng = np.random.default_rng(6)
        pages = tables(rng, c, [100, 100])
        p = pages[0, 3]
        if int8:
            c.ks[p, 0, 2] = np.nan
        else:
            c.k[p, 0, 2, 9] = np.nan
        c.upload()
        q = rng.standard_normal((2, 256)).astype(np.float16)
        import torch
        y = torch.empty(2, 256, dtype=torch.float16, device="cuda")
        ws = torch.empty(woq.woq_attn_decode_workspace(c.desc, 4, 2), dtype=torch.uint8, device="cuda")
        woq.woq_attn_decode(c.desc, dev(q), dev(pages), dev(np.array([100, 100], np.int32)), y, ws)
        got = host(y)
        assert np.all(np.isnan(got[0, :128])) and np.all(np.isfinite(got[0, 128:])) and np.all(np.isfinite(got[1]))


def test_attention_over_its_queries_and_rows_of_a_sequence(gpu_lib):
    """y over q; four new tokens of one sequence as rows with the same pages and
    rising lengths give what each alone gives, bit for bit."""
    import torch
    c = Cache(20, 2, 16, 64, True, seed=14)
    rng = np.random.default_rng(7)
    q = rng.standard_normal((4, 256)).astype(np.float16)
    pages = np.repeat(rng.permutation(20)[None, :9], 4, 0).astype(np.int32)
    lens = np.array([130, 131, 132, 133], np.int32)
    qd = dev(q)
    ws = torch.empty(woq.woq_attn_decode_workspace(c.desc, 4, 4), dtype=torch.uint8, device="cuda")
    woq.woq_attn_decode(c.desc, qd, dev(pages), dev(lens), qd, ws)
    check_attention(c, 4, lens, q=q, pages=pages, got=host(qd))


@pytest.mark.parametrize("b", [63, 64, 65, 130])
def test_attention_many_rows_of_every_length(gpu_lib, b):
    """Ragged rows around the number that a wave holds, some empty, with a window
    and without; one long row among short ones."""
    rng = np.random.default_rng(b)
    lens = rng.integers(0, 60, b)
    lens[rng.random(b) < 0.2] = 0
    lens[b // 2] = 4000
    case("attention ragged", b)
    c = Cache(int(sum(-(-lens // 32))) + 1, 3, 32, 64, True, seed=b)
    check_attention(c, 6, lens, seed=b)
    check_attention(c, 6, lens, seed=b, window=33)
    lens[:] = 0
    assert not check_attention(c, 6, lens, seed=b, width=200).any()


@pytest.mark.parametrize("width", [20, 90])
def test_attention_of_views(gpu_lib, width):
    """Tables, lengths and rows that are pieces of larger tensors, at addresses of
    any 4 (int32) or 16 (rows) bytes; rows behind the batch stay."""
    import torch
    c = Cache(60, 2, 16, 64, True, seed=21)
    rng = np.random.default_rng(width)
    lens = np.array([300, 17, 0, 211], np.int32)
    pages = tables(rng, c, lens, width=width)
    q = rng.standard_normal((4, 4 * 64)).astype(np.float16)
    big = dev(np.full((6, width + 5), 2 ** 30, np.int32))
    big[1:5, 3:3 + width] = dev(pages)
    ld = dev(np.full(9, 777, np.int32))
    ld[3:7] = dev(lens)
    rows = torch.full((6, 3 * 256), 5.0, dtype=torch.float16, device="cuda")
    rows[1:5, 256:512] = dev(q)
    ws = torch.empty(woq.woq_attn_decode_workspace(c.desc, 4, 4) + 16, dtype=torch.uint8, device="cuda")
    woq.woq_attn_decode(c.desc, rows[1:, 256:512], big[1:, 3:3 + width], ld[3:], rows[1:, 512:], ws[16:], b=4)
    got = host(rows)
    check_attention(c, 4, lens, q=q, pages=pages, got=got[1:5, 512:])
    assert np.all(got[[0, 5]] == 5) and np.all(got[:, :256] == 5)
    np.testing.assert_array_equal(got[1:5, 256:512], q)


@pytest.mark.parametrize("int8", [True, False])
def test_attention_captured_where_it_takes_much_shared_memory(gpu_lib, int8):
    """Sixteen heads of 256 to a key head: more than 64 KB a workgroup, short
    tables and long; one graph of both, replayed."""
    import torch
    c = Cache(300, 1, 16, 256, int8, seed=3)
    rng = np.random.default_rng(2)
    lens = np.array([500, 0, 77], np.int32)
    q = rng.standard_normal((3, 16 * 256)).astype(np.float16)
    short = tables(rng, c, lens)
    wide = np.full((3, 280), -1, np.int32)
    wide[:, :short.shape[1]] = short
    qd, ld, pages = dev(q), dev(lens), (dev(short), dev(wide))
    y = [torch.empty(3, 16 * 256, dtype=torch.float16, device="cuda") for _ in pages]
    ws = torch.empty(woq.woq_attn_decode_workspace(c.desc, 16, 3), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for p, out in zip(pages, y):
            woq.woq_attn_decode(c.desc, qd, p, ld, out, ws)
    for _ in range(3):
        for out in y:
            out.fill_(9)
        g.replay()
        for out in y:
            check_attention(c, 16, lens, q=q, pages=short, got=host(out))


# ----------------------------------------------------------------- sampling

def check_sample(x, u, T=None, k=None, p=None, m=None, pad=0):
    import torch
    b, N = x.shape
    ld = -(-N // 8) * 8 + 8 * pad
    wide = np.full((b, ld), 60000, np.float16)           # what stands behind a row is not a logit
    wide[:, :N] = x
    xd = dev(wide)
    token = torch.full((b + 1,), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((b + 1,), -7.0, device="cuda")

    def of(a, t):
        return None if a is None else dev(np.broadcast_to(np.asarray(a, t), (b,)).copy())

    f = np.float32
    woq.woq_sample(xd, of(u, f), token, temperature=of(T, f), top_k=of(k, np.int32), top_p=of(p, f), min_p=of(m, f),
                   prob=prob, N=N)
    got, share = host(token), host(prob)
    assert got[b] == -7 and share[b] == -7

    def at(a, r, none):
        return none if a is None else float(np.broadcast_to(np.asarray(a, f), (b,))[r])

    for r in range(b):
        want, ref = O.sample(x[r], at(u, r, 0), at(T, r, 1.0), int(at(k, r, 0)), at(p, r, 1.0), at(m, r, 0.0))
        assert got[r] == want, (r, got[r], want, x[r, got[r]] if got[r] >= 0 else None, x[r, want])
        assert abs(share[r] - ref) <= ref * 2 * U, (r, share[r], ref)
    return got[:b]


def logits(b, N, seed, spread=3.0):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((b, N)) * spread).astype(np.float16)
    x[::2, 3::17] = -np.inf
    return x, rng


@pytest.mark.parametrize("N", [1, 2, 7, 8, 9, 63, 511, 512, 513, 1000, 8191, 32000, 128256])
def test_sample_sizes(gpu_lib, N):
    case("sample", N)
    b = 24 if N < 10000 else 6
    x, rng = logits(b, N, N)
    u = rng.random(b).astype(np.float32)
    check_sample(x, u)
    check_sample(x, u, T=rng.choice([0.0, 0.3, 1.0, 2.5], b), k=rng.choice([0, 1, 2, 50, 2 ** 30], b), pad=1)
    check_sample(x, u, p=rng.choice([0.1, 0.5, 0.95, 1.0], b), m=rng.choice([0.0, 0.01, 0.2], b))
    check_sample(x, u, T=rng.choice([0.5, 1.0], b), k=rng.choice([5, 40, 400], b), p=rng.choice([0.3, 0.9], b),
                 m=rng.choice([0.0, 0.05], b), pad=2)


@pytest.mark.parametrize("spread", [0.0, 1e-3, 0.1, 30.0, 3000.0])
def test_sample_flat_and_sharp(gpu_lib, spread):
    case("sample spread", spread)
    x, rng = logits(16, 5000, 3, spread)
    u = rng.random(16).astype(np.float32)
    check_sample(x, u)
    check_sample(x, u, T=0.7, p=0.9)
    check_sample(x, u, k=37, m=0.5)


def test_sample_every_draw_of_a_few_tokens(gpu_lib):
    """Numbers at, before and behind the steps of equal weights, and out of range."""
    x = np.zeros((16, 4), np.float16)
    u = np.array([0, 0.2499, 0.25, 0.26, 0.4999, 0.5, 0.7499, 0.75, 0.9999, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, np.nan,
                  np.inf, -np.inf], np.float32)
    got = check_sample(x, u)
    np.testing.assert_array_equal(got, [0, 0, 1, 1, 1, 2, 2, 3, 3, 3, 3, 3, 0, 0, 3, 0])


def test_sample_what_can_not_be_taken(gpu_lib):
    x, rng = logits(10, 3000, 5)
    x[0], x[1] = np.nan, -np.inf
    x[2, 100:], x[2, :100] = np.nan, -np.inf
    x[2, 77] = -65504
    x[3, [5, 9, 2000]] = np.inf
    x[4] = np.where(np.arange(3000) % 2, np.float16(-0.0), np.float16(0.0))
    x[5, 1234] = np.nan
    u = rng.random(10).astype(np.float32)
    got = check_sample(x, u)
    assert got[0] == got[1] == -1 and got[2] == 77 and got[3] in (5, 9, 2000)
    check_sample(x, u, T=0.0)
    check_sample(x, u, T=1e-30, k=7, p=0.9, m=0.3)
    check_sample(x, u, T=np.inf)
    check_sample(x, u, T=np.nan)
    check_sample(x, u, k=-3, p=np.nan, m=np.nan)
    check_sample(x, u, p=-1.0)
    check_sample(x, u, p=0.0, k=100)
    check_sample(x, u, m=1.0)
    check_sample(x, u, m=5.0)


@pytest.mark.parametrize("N", [65535, 65536, 65537, 131080, 200003])
def test_sample_more_equal_logits_than_16_bits_count(gpu_lib, N):
    """One value, two values on either side of zero, and one value among others."""
    case("sample equal", N)
    rng = np.random.default_rng(N)
    x = np.zeros((9, N), np.float16)
    x[1], x[2] = -5, 7
    x[3] = np.where(rng.random(N) < 0.5, np.float16(1.0), np.float16(-1.0))
    x[4:] = rng.standard_normal((5, N)) * 2
    x[5, rng.random(N) < 0.9] = -1.5
    x[6, rng.random(N) < 0.9] = 1.5
    x[7, rng.random(N) < 0.95] = 0.25
    x[8, :] = -np.inf
    x[8, N // 2:] = 3
    u = rng.random(9).astype(np.float32)
    check_sample(x, u)
    check_sample(x, u, T=0.8, p=0.9, m=0.01)
    check_sample(x, u, k=[1, 70000, N, N - 1, 1000, 66000, 60000, 65536, 30000])
    check_sample(x, u, k=66000, p=0.999)


def test_sample_of_views(gpu_lib):
    """Rows inside wider ones, parameters from the middle of vectors."""
    import torch
    x, rng = logits(6, 2000, 4)
    wide = dev(np.full((8, 2400), 60000, np.float16))
    wide[1:7, 200:2200] = dev(x)
    u, top_p = rng.random(6).astype(np.float32), np.array([0.3, 0.9, 1.0, 0.5, 0.99, 0.7], np.float32)
    ud, pd = dev(np.full(9, 0.5, np.float32)), dev(np.full(9, 0.0, np.float32))
    ud[3:], pd[2:8] = dev(u), dev(top_p)
    token = torch.full((8,), -5, dtype=torch.int32, device="cuda")
    woq.woq_sample(wide[1:, 200:2200], ud[3:], token[1:7], top_p=pd[2:], b=6)
    got = host(token)
    assert got[0] == got[7] == -5
    for r in range(6):
        assert got[1 + r] == O.sample(x[r], float(u[r]), top_p=float(top_p[r]))[0]


def test_sample_rows_do_not_touch_each_other(gpu_lib):
    x, rng = logits(300, 1000, 8)
    u = rng.random(300).astype(np.float32)
    together = check_sample(x, u, p=0.9)
    for r in (0, 17, 299):
        assert check_sample(x[r:r + 1], u[r:r + 1], p=0.9)[0] == together[r]


# ------------------------------------------------------- all of them in a row

class Step:
    """A decode step of one small layer and a head: the q|k|v product of an INT8
    weight, the new tokens into the cache, attention, the o product, the head's
    product and the choice of the token."""

    def __init__(self, b, seed=0, heads=2, q_heads=4, dim=64, page=16, length=200, vocab=1000, int8=True):
        import torch
        rng = np.random.default_rng(seed)
        self.b, self.K, self.n, self.m = b, 128, q_heads * dim, heads * dim
        self.heads, self.q_heads, self.dim, self.page, self.vocab = heads, q_heads, dim, page, vocab

        def weight(N, K):
            return woq.DeviceInt8([woq.woq_quantize_int8((rng.standard_normal((N, K)) / np.sqrt(K)).astype(np.float32))])

        self.qkv_w, self.o_w, self.head_w = weight(self.n + 2 * self.m, self.K), weight(self.K, self.n), weight(vocab, self.K)
        W = -(-length // page) + 1
        self.c = Cache(b * W + 1, heads, page, dim, int8, seed=seed)
        self.pages = rng.permutation(b * W).reshape(b, W).astype(np.int32)
        self.lens = rng.integers(1, length, b).astype(np.int32)
        self.rope = rope_table(W * page, dim)
        half = dict(dtype=torch.float16, device="cuda")
        self.d = dict(x=dev(rng.standard_normal((b, self.K)).astype(np.float16)), pages=dev(self.pages), rope=dev(self.rope),
                      u=dev(rng.random(b).astype(np.float32)), top_p=dev(np.full(b, 0.9, np.float32)))
        self.qkv, self.y = torch.empty(b, self.n + 2 * self.m, **half), torch.empty(b, self.n, **half)
        self.h, self.logits = torch.empty(b, self.K, **half), torch.empty(b, vocab, **half)
        self.token = torch.empty(b, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(woq.woq_attn_decode_workspace(self.c.desc, q_heads, b), dtype=torch.uint8, device="cuda")
        self.set_lens()

    def set_lens(self):
        at = self.lens - 1
        slots = self.pages[np.arange(self.b), at // self.page] * self.page + at % self.page
        self.d.update(lens=dev(self.lens), pos=dev(at.astype(np.int32)), slots=dev(slots.astype(np.int32)))

    def run(self, stream=None):
        d, n, m = self.d, self.n, self.m
        woq.woq_qgemv_int8(self.qkv_w.desc, d["x"], self.qkv, stream=stream)
        woq.woq_cache_write(self.c.desc, self.qkv[:, n:n + m], self.qkv[:, n + m:], d["slots"], q=self.qkv[:, :n],
                            q_out=self.qkv[:, :n], rope=d["rope"], pos=d["pos"], stream=stream)
        woq.woq_attn_decode(self.c.desc, self.qkv[:, :n], d["pages"], d["lens"], self.y, self.ws, stream=stream)
        woq.woq_qgemv_int8(self.o_w.desc, self.y, self.h, stream=stream)
        woq.woq_qgemv_int8(self.head_w.desc, self.h, self.logits, stream=stream)
        woq.woq_sample(self.logits, d["u"], self.token, top_p=d["top_p"], stream=stream)

    def results(self):
        return [host(t).copy() for t in (self.qkv, self.y, self.logits, self.token)] + [a.copy() for a in self.c.now()
                                                                                         if a is not None]


def same(a, b):
    for x, y in zip(a, b):
        np.testing.assert_array_equal(x.view(np.uint8), y.view(np.uint8))


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("b", [1, 5, 8])
def test_decode_steps_in_a_row(gpu_lib, int8, b):
    """Four tokens of every request: each operator's result is the definition's of
    what the one before has left."""
    import torch
    case("steps", int8, b)
    s = Step(b, seed=b, int8=int8)
    for _ in range(4):
        s.run()
        qkv, y, x, token = (host(t) for t in (s.qkv, s.y, s.logits, s.token))
        k, v, ks, vs = s.c.now()
        s.c.k, s.c.v, s.c.ks, s.c.vs = k, v, ks, vs
        plain = torch.empty_like(s.qkv)
        woq.woq_qgemv_int8(s.qkv_w.desc, s.d["x"], plain)
        new = host(plain).reshape(b, -1, s.dim)
        turned = O.rotate(new[:, :s.q_heads + s.heads], s.rope, host(s.d["pos"]))
        within(qkv[:, :s.n].reshape(b, s.q_heads, s.dim), turned[:, :s.q_heads],
               np.abs(turned[:, :s.q_heads]) * H + 4 * U * 2 * np.abs(new).max() + SUB)
        slots = host(s.d["slots"])
        for which, ref in (("k", turned[:, s.q_heads:]), ("v", new[:, s.q_heads + s.heads:].astype(np.float64))):
            top = np.abs(ref).max(-1, keepdims=True)
            step = top / 127 * (0.5 + 2.0 ** -10) if int8 else np.abs(ref) * H + SUB
            within(s.c.tokens(which, slots), ref, step + 4 * U * 2 * np.abs(new).max(), which)
        check_attention(s.c, s.q_heads, s.lens, q=qkv[:, :s.n], pages=s.pages, got=y)
        for r in range(b):
            assert token[r] == O.sample(x[r], float(host(s.d["u"])[r]), top_p=float(np.float32(0.9)))[0]
        s.lens += 1
        s.set_lens()
        s.d["u"].copy_(torch.rand(b))
        s.d["x"].copy_(torch.randn(b, s.K))


@pytest.mark.parametrize("length", [200, 1500])
def test_decode_step_captured_and_replayed(gpu_lib, length):
    """One graph replayed between eager runs on other inputs and other work gives
    the eager bits every time; two graphs share a workspace in turn."""
    import torch
    s, t = Step(5, seed=1, length=length), Step(5, seed=2, length=length)
    t.ws = s.ws
    for x in (s, t):
        x.run()
    torch.cuda.synchronize()
    graphs = []
    for x in (s, t):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    for it in range(4):
        for x, g in zip((s, t), graphs):
            x.d["x"].copy_(torch.randn(5, x.K))
            x.lens = 1 + (x.lens + 37) % (length - 1)
            fresh = x.d.copy()
            x.set_lens()
            for name in ("lens", "pos", "slots"):               # into the graph's own buffers
                fresh[name].copy_(x.d[name])
            x.d = fresh
            x.run()
            want = x.results()
            x.y.fill_(3)
            x.token.fill_(-9)
            x.ws.fill_(255)
            g.replay()
            same(x.results(), want)
            torch.randn(1000, 1000, device="cuda").sum().item()  # the program's own work


def test_two_streams_at_once(gpu_lib):
    import torch
    steps = [Step(4, seed=i, length=900) for i in range(4)]
    alone = []
    for s in steps:
        s.run()
        alone.append(s.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(8):
        for s, st in zip(steps, streams):
            s.run(stream=st)
    torch.cuda.synchronize()
    for s, want in zip(steps, alone):
        same(s.results(), want)
    # the stream of the caller, not the default one
    for s, st, want in zip(steps, streams, alone):
        s.y.fill_(0)
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            s.run()
        st.synchronize()
        same(s.results(), want)


@pytest.mark.parametrize("fmt", ["int8", "int4o"])
def test_stack_with_attention_equals_its_steps(gpu_lib, fmt):
    """q|k|v, attention, o of two layers through the runner: the bits of the calls
    one by one, also from a graph; a step without attention between."""
    import torch
    case("stack attention", fmt)
    rng = np.random.default_rng(3)
    b, heads, q_heads, dim, page = 6, 2, 4, 64, 16
    n, m, K = q_heads * dim, heads * dim, 128
    dims = [(n + 2 * m, K), (K, n)] * 2
    steps, keep = [], []
    for i, (N, k) in enumerate(dims):
        W = (rng.standard_normal((N, k)) / np.sqrt(k)).astype(np.float32)
        if fmt == "int8":
            d = woq.DeviceInt8([woq.woq_quantize_int8(W)])
            steps.append(woq.step_int8(d, i, i))
        else:
            geom = woq.woq_int4o_geometry(k)
            perm = O.global_perm(k, np.sort(rng.choice(k, geom.n_out, replace=False)))
            d, pd = woq.DeviceInt4o([woq.woq_quantize_int4o(W, perm, geom.n_out)], geom), dev(perm)
            keep.append(pd)
            steps.append(woq.step_int4o(d, pd, i, i))
        keep.append(d)
    half = dict(dtype=torch.float16, device="cuda")
    lens = np.array([1, 100, 33, 0, 16, 77], np.int32)
    pages = rng.permutation(6 * 8)[:48].reshape(6, 8).astype(np.int32)
    at = np.maximum(lens - 1, 0)
    slots = np.where(lens > 0, pages[np.arange(6), at // page] * page + at % page, -1).astype(np.int32)
    rope = dev(rope_table(128, 32))
    sd, pd, ld, posd = dev(slots), dev(pages), dev(lens), dev(at.astype(np.int32))

    def fresh():
        caches = [Cache(48, heads, page, dim, i == 0, seed=20 + i) for i in range(2)]
        outs = [torch.full((b, N), 7.0, **half) for N, _ in dims]
        ys = [torch.full((b, n), 7.0, **half) for _ in range(2)]
        return caches, outs, ys

    x = dev(rng.standard_normal((b, K)).astype(np.float16))
    caches, outs, ys = fresh()
    st = woq.Stack(steps, 8)
    st.bind([x, ys[0], outs[1], ys[1]], outs)
    attn = [woq.StackAttention(caches[0].d, ys[0], rope=rope, interleaved=True), None,
            woq.StackAttention(caches[1].d, ys[1], softcap=30.0, window=40), None]
    ws = torch.empty(st.attn_workspace(attn, b), dtype=torch.uint8, device="cuda")
    st.run_attn(b, attn, sd, pd, ld, ws, pos=posd)
    got = [host(t).copy() for t in outs + ys] + [a for c in caches for a in c.now() if a is not None]

    hc, ho, hy = fresh()
    src = x
    for layer in range(2):
        for j in range(2):
            i = 2 * layer + j
            step = steps[i]
            step.in_slot = step.out_slot = 0
            one = woq.Stack([step], 8)
            one.bind([src], [ho[i]])
            one.run(b)
            if j == 0:
                q, kv = ho[i][:, :n], ho[i][:, n:]
                kw = dict(q=q, q_out=q, rope=rope, pos=posd, interleaved=True) if layer == 0 else {}
                woq.woq_cache_write(hc[layer].desc, kv[:, :m], kv[:, m:], sd, **kw)
                woq.woq_attn_decode(hc[layer].desc, q, pd, ld, hy[layer], ws, softcap=30.0 * layer, window=40 * layer)
                src = hy[layer]
            else:
                src = ho[i]
    want = [host(t) for t in ho + hy] + [a for c in hc for a in c.now() if a is not None]
    same(got, want)
    assert not host(ys[0])[3].any()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        st.run_attn(b, attn, sd, pd, ld, ws, pos=posd)
    for _ in range(3):
        for t in outs + ys:
            t.fill_(3)
        g.replay()
        same([host(t) for t in outs + ys] + [a for c in caches for a in c.now() if a is not None], want)
    del keep


def test_stack_with_attention_refuses_before_the_first_launch(gpu_lib):
    import torch
    rng = np.random.default_rng(0)
    d = woq.DeviceInt8([woq.woq_quantize_int8(rng.standard_normal((256, 64)).astype(np.float32))])
    st = woq.Stack([woq.step_int8(d, 0, 0)], 4)
    half = dict(dtype=torch.float16, device="cuda")
    x, out, y = torch.ones(4, 64, **half), torch.full((4, 256), 7.0, **half), torch.full((4, 128), 7.0, **half)
    st.bind([x], [out])
    c, idx, pages = Cache(4, 1, 16, 64), dev(np.zeros(4, np.int32)), dev(np.zeros((4, 1), np.int32))
    good = woq.StackAttention(c.d, y, rope=torch.zeros(3, 16, device="cuda"))
    ws = torch.empty(st.attn_workspace([good], 4), dtype=torch.uint8, device="cuda")
    wide = Cache(4, 2, 16, 64)
    for bad in (woq.StackAttention(wide.d, y), woq.StackAttention(c.d, torch.empty(4, 64, **half)),
                woq.StackAttention(c.d, y, rope=torch.zeros(3, 24, device="cuda")),
                woq.StackAttention(c.d, y, window=-1), woq.StackAttention(c.d, y, scale=float("nan"))):
        with pytest.raises(woq.WoqError):
            st.run_attn(4, [bad], idx, pages, idx, ws, pos=idx)
    with pytest.raises(woq.WoqError):
        st.run_attn(4, [good], idx, pages, idx, ws)                       # angles without positions
    with pytest.raises(woq.WoqError):
        st.run_attn(4, [good], idx, pages, idx, ws[:64], pos=idx)
    for args in (([good, None], idx, pages, idx), ([good], idx[:3], pages, idx), ([good], idx, pages[:3], idx)):
        with pytest.raises(ValueError):
            st.run_attn(4, *args, ws, pos=idx)
    with pytest.raises(ValueError):
        st.run_attn(4, [woq.StackAttention(c.d, y[:3])], idx, pages, idx, ws)
    assert np.all(host(out) == 7) and np.all(host(y) == 7)


def test_empty_calls_are_no_ops(gpu_lib):
    s = Step(2, seed=5)
    s.run()
    want = s.results()
    d, n, m = s.d, s.n, s.m
    woq.woq_cache_write(s.c.desc, s.qkv[:, n:n + m], s.qkv[:, n + m:], d["slots"], q=s.qkv[:, :n], q_out=s.qkv[:, :n],
                        rope=d["rope"], pos=d["pos"], b=0)
    woq.woq_cache_read(s.c.desc, d["slots"], s.qkv[:, :m], n=0)
    woq.woq_attn_decode(s.c.desc, s.qkv[:, :n], d["pages"], d["lens"], s.y, s.ws, b=0)
    woq.woq_sample(s.logits, d["u"], s.token, b=0)
    same(s.results(), want)


def test_offsets_past_32_bits(gpu_lib):
    """A cache of more than 2^32 bytes of keys, its tokens at the far end, and
    logits whose rows start past 2^31."""
    import torch
    heads, page, dim = 8, 64, 256
    n_pages = (1 << 32) // (heads * page * dim) + 40
    k, v = (torch.full((n_pages, heads, page, dim), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((n_pages, heads, page), float("nan"), device="cuda") for _ in range(2))
    c = woq.DeviceCache(k, v, ks, vs)
    rng = np.random.default_rng(1)
    b = 130
    x = rng.standard_normal((b, 2 * heads * dim)).astype(np.float16)
    last = np.arange(n_pages - 3, n_pages)
    slots = (last[np.arange(b) // page] * page + np.arange(b) % page).astype(np.int32)
    xd = dev(x)
    woq.woq_cache_write(c.desc, xd[:, :heads * dim], xd[:, heads * dim:], dev(slots))
    ko, vo = (torch.empty(b, heads * dim, dtype=torch.float16, device="cuda") for _ in range(2))
    woq.woq_cache_read(c.desc, dev(slots), ko, vo)
    for got, src in ((host(ko), x[:, :heads * dim]), (host(vo), x[:, heads * dim:])):
        top = np.abs(src.astype(float)).reshape(b, heads, dim).max(-1).repeat(dim, 1)
        within(got, src.astype(np.float64), top / 127 * (0.5 + 2.0 ** -10) + np.abs(src) * H)
    q = rng.standard_normal((1, 16 * dim)).astype(np.float16)
    y = torch.empty(1, 16 * dim, dtype=torch.float16, device="cuda")
    ws = torch.empty(woq.woq_attn_decode_workspace(c.desc, 16, 1), dtype=torch.uint8, device="cuda")
    for width in (3, 40):
        pages = np.full((1, width), -1, np.int32)
        pages[0, :3] = last
        woq.woq_attn_decode(c.desc, dev(q), dev(pages), dev(np.array([b], np.int32)), y, ws)
        small = Cache(3, heads, page, dim)
        small.k, small.v, small.ks, small.vs = (host(t[-3:]) for t in (k, v, ks, vs))
        check_attention(small, 16, [b], q=q, pages=np.arange(3, dtype=np.int32)[None], got=host(y))
    del k, v, ks, vs, c
    N, rows = 256000, 8500
    logit = torch.zeros(rows, N, dtype=torch.float16, device="cuda")
    far = torch.randn(3, N, device="cuda").half()
    logit[-3:] = far
    u = torch.rand(rows, device="cuda")
    token = torch.empty(rows, dtype=torch.int32, device="cuda")
    woq.woq_sample(logit, u, token, top_k=torch.full((rows,), 50, dtype=torch.int32, device="cuda"))
    got, uh, fh = host(token), host(u), host(far)
    for i in range(3):
        assert got[rows - 3 + i] == O.sample(fh[i], float(uh[rows - 3 + i]), top_k=50)[0]
    assert got[0] == O.sample(np.zeros(N), float(uh[0]), top_k=50)[0]
