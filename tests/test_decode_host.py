"""CPU checks of the operators between a decode step's products and behind its
head (woq_cache_write, woq_cache_read, woq_attn_decode, woq_sample): the float64
definitions against explicit loops and closed forms, and every refusal of the C
entry points and of the binding (nothing is launched, so no GPU is needed)."""
import ctypes
import math

import numpy as np
import pytest

import oracle as O
from weight_only_quantized_quantize_amd import woq


# ------------------------------------------------------------- definitions

def test_rotation_definition():
    """A quarter turn takes (a, b) to (-b, a); what lies past rot stays."""
    x = np.arange(2 * 1 * 6, dtype=np.float64).reshape(2, 1, 6)
    rope = np.array([[1.0, 1.0, 0.0, 0.0], [0.0, 0.0, 1.0, 1.0]])
    np.testing.assert_array_equal(O.rotate(x, rope, [0, 0]), x)
    np.testing.assert_array_equal(O.rotate(x, rope, [0, 1])[1, 0], [-8, -9, 6, 7, 10, 11])
    np.testing.assert_array_equal(O.rotate(x, rope, [0, 1], True)[1, 0], [-7, 6, -9, 8, 10, 11])
    # pairs keep their length, and turning back undoes the turn
    a = np.random.default_rng(0).uniform(-3, 3, 2)
    rope = np.stack([np.concatenate([np.cos(a), np.sin(a)]), np.concatenate([np.cos(a), -np.sin(a)])])
    for inter in (False, True):
        y = O.rotate(x, rope, [0, 0], inter)
        np.testing.assert_allclose(O.rotate(y, rope, [1, 1], inter), x, atol=1e-12)


def test_attention_definition_against_loops():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((4, 3)), rng.standard_normal((5, 2, 3)), rng.standard_normal((5, 2, 3))
    for cap in (0.0, 2.0):
        y, spread, _ = O.attend(q, k, v, 0.7, cap)
        for h in range(4):
            z = [0.7 * sum(q[h, d] * k[t, h // 2, d] for d in range(3)) for t in range(5)]
            z = [cap * math.tanh(s / cap) if cap else s for s in z]
            e = [math.exp(s) for s in z]
            for d in range(3):
                assert abs(y[h, d] - sum(e[t] * v[t, h // 2, d] for t in range(5)) / sum(e)) < 1e-12
                assert spread[h, d] >= abs(y[h, d]) - 1e-12
    y, _, _ = O.attend(q, k[:0], v[:0], 1.0)
    assert not y.any()
    y, _, _ = O.attend(q, k[:1], v[:1], 1.0)               # one token: its value
    np.testing.assert_allclose(y, np.repeat(v[0], 2, axis=0))


def test_sampling_definition():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))              # from the largest down: tokens 1, 3, 2, 0
    ends = [0.4, 0.7, 0.9, 1.0]
    for u in np.linspace(0, 0.999, 101):
        want = [1, 3, 2, 0][next(i for i, e in enumerate(ends) if u < e - 1e-12)]
        assert O.sample(x, u)[0] == want, u
    assert O.sample(x, 0.0) == (1, pytest.approx(0.4))
    assert O.sample(x, 0.99, top_k=2) == (3, pytest.approx(3 / 7))
    assert O.sample(x, 0.99, top_p=0.41) == (3, pytest.approx(3 / 7))
    assert O.sample(x, 0.99, top_p=0.39) == (1, 1.0)
    assert O.sample(x, 0.99, top_p=-1.0) == (1, 1.0)
    assert O.sample(x, 0.99, min_p=0.49) == (2, pytest.approx(2 / 9))
    assert O.sample(x, 0.99, min_p=7.0) == (1, 1.0)
    assert O.sample(x, 0.99, temperature=0.0) == (1, 1.0)
    # a temperature of 1/2 squares the shares
    assert O.sample(x, 0.0, temperature=0.5)[1] == pytest.approx(0.16 / 0.3)
    # equal logits by index; top-k and top-p cut among them
    assert [O.sample(np.zeros(4), u)[0] for u in (0.0, 0.3, 0.5, 0.99)] == [0, 1, 2, 3]
    assert O.sample(np.zeros(4), 0.99, top_k=3)[0] == 2 and O.sample(np.zeros(4), 0.99, top_p=0.5)[0] == 1
    assert O.sample(np.array([-0.0, 0.0]), 0.0)[0] == 0
    # what can not be taken
    assert O.sample(np.array([np.nan, -np.inf]), 0.5) == (-1, 0.0)
    assert O.sample(np.array([np.nan, 1.0, -np.inf]), 0.999) == (1, 1.0)
    assert [O.sample(np.array([1.0, np.inf, np.inf]), u)[0] for u in (0.0, 0.9)] == [1, 2]


# ---------------------------------------------------------------- refusals

P = 0x10000          # an aligned address that is never dereferenced
EINVAL, EALIGN, EUNSUPPORTED, OK = woq.WOQ_EINVAL, woq.WOQ_EALIGN, woq.WOQ_EUNSUPPORTED, woq.WOQ_OK


def call(name, *args):
    return getattr(woq.lib(), name)(*args)


def cache(fmt=woq.CACHE_INT8, n_pages=10, heads=2, page=16, dim=64, **ptrs):
    c = woq.Cache()
    c.k, c.v = ptrs.get("k", P), ptrs.get("v", P)
    scale = P if fmt == woq.CACHE_INT8 else None
    c.k_scale, c.v_scale = ptrs.get("k_scale", scale), ptrs.get("v_scale", scale)
    c.n_pages, c.fmt, c.heads, c.page, c.dim = n_pages, fmt, heads, page, dim
    return c


BAD_CACHES = [
    (None, EINVAL), (cache(fmt=0), EINVAL), (cache(fmt=3), EINVAL), (cache(n_pages=0), EINVAL), (cache(heads=0), EINVAL),
    (cache(page=0), EINVAL), (cache(dim=0), EINVAL), (cache(dim=-16), EINVAL), (cache(k=None), EINVAL),
    (cache(v=None), EINVAL), (cache(k_scale=None), EINVAL), (cache(v_scale=None), EINVAL),
    (cache(fmt=woq.CACHE_FP16, k_scale=P), EINVAL), (cache(fmt=woq.CACHE_FP16, v_scale=P), EINVAL),
    (cache(k=P + 8), EALIGN), (cache(v=P + 8), EALIGN), (cache(k_scale=P + 4), EALIGN), (cache(v_scale=P + 4), EALIGN),
    (cache(dim=72), EUNSUPPORTED), (cache(dim=272), EUNSUPPORTED), (cache(page=24), EUNSUPPORTED),
    (cache(page=65552), EUNSUPPORTED), (cache(heads=1025), EUNSUPPORTED),
    (cache(n_pages=1 << 27), EUNSUPPORTED), (cache(n_pages=1 << 60), EUNSUPPORTED),
]


def passed(c):
    return None if c is None else ctypes.byref(c)


def write_args(**kw):
    a = dict(c=cache(), k=P, ldk=128, v=P, ldv=128, slots=P, b=3, q=P, ldq=256, q_heads=4, q_out=P, ldqo=256, rope=P,
             n_pos=10, rot=64, interleaved=0, pos=P, stream=None)
    a.update(kw)
    a["c"] = passed(a["c"])
    return list(a.values())


WIDE = dict(ldk=1 << 20, ldv=1 << 20, ldq=1 << 20, ldqo=1 << 20)


@pytest.mark.parametrize("change,status", [(dict(WIDE, c=c), s) for c, s in BAD_CACHES] + [
    (dict(b=-1), EINVAL), (dict(ldk=120), EINVAL), (dict(ldv=120), EINVAL), (dict(ldq=248), EINVAL),
    (dict(ldqo=248), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(slots=None), EINVAL),
    (dict(q_heads=0), EINVAL), (dict(q_out=None), EINVAL), (dict(rope=None), EINVAL), (dict(pos=None), EINVAL),
    (dict(n_pos=0), EINVAL), (dict(rot=0), EINVAL), (dict(rot=80), EINVAL), (dict(interleaved=2), EINVAL),
    (dict(ldqo=264), EINVAL),                                      # in place with other rows
    (dict(k=P + 8), EALIGN), (dict(v=P + 2), EALIGN), (dict(q=P + 8), EALIGN), (dict(q_out=P + 8), EALIGN),
    (dict(ldk=132), EALIGN), (dict(ldv=132), EALIGN), (dict(ldq=260, ldqo=260), EALIGN), (dict(slots=P + 2), EALIGN),
    (dict(rope=P + 4), EALIGN), (dict(pos=P + 2), EALIGN), (dict(rot=24), EUNSUPPORTED), (dict(b=1 << 28), EUNSUPPORTED),
    (dict(b=1 << 62), EUNSUPPORTED), (dict(b=0, k=None, v=None, slots=None, pos=None), OK), (dict(b=0, k=P + 8), OK),
])
def test_write_refusals(change, status):
    assert call("woq_cache_write", *write_args(**change)) == status


@pytest.mark.parametrize("change,status", [(dict(c=c, ldk=1 << 20, ldv=1 << 20), s) for c, s in BAD_CACHES] + [
    (dict(n=-1), EINVAL), (dict(k=None, v=None), EINVAL), (dict(ldk=120), EINVAL), (dict(ldv=120), EINVAL),
    (dict(slots=None), EINVAL), (dict(k=P + 8), EALIGN), (dict(v=P + 8), EALIGN), (dict(ldk=132), EALIGN),
    (dict(ldv=132), EALIGN), (dict(slots=P + 1), EALIGN), (dict(n=1 << 30), EUNSUPPORTED), (dict(n=0, slots=None), OK),
    (dict(n=0, k=None), OK),
])
def test_read_refusals(change, status):
    a = dict(c=cache(), slots=P, n=3, k=P, ldk=128, v=P, ldv=128, stream=None)
    a.update(change)
    a["c"] = passed(a["c"])
    assert call("woq_cache_read", *a.values()) == status


@pytest.mark.parametrize("change,status", [(dict(c=c, ldq=1 << 20, ldy=1 << 20, q_heads=1025 * 2 if c and c.heads > 1024 else 4), s)
                                           for c, s in BAD_CACHES] + [
    (dict(b=-1), EINVAL), (dict(q_heads=0), EINVAL), (dict(q_heads=3), EINVAL), (dict(ldq=248), EINVAL),
    (dict(ldy=248), EINVAL), (dict(max_pages=0), EINVAL), (dict(ldpages=4), EINVAL), (dict(q=None), EINVAL),
    (dict(pages=None), EINVAL), (dict(lens=None), EINVAL), (dict(y=None), EINVAL), (dict(ws=None), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(softcap=-1.0), EINVAL),
    (dict(softcap=float("nan")), EINVAL), (dict(softcap=float("inf")), EINVAL), (dict(window=-1), EINVAL),
    (dict(ws_bytes=15), EINVAL), (dict(ldy=264), EINVAL), (dict(q=P + 8), EALIGN), (dict(y=P + 4096 + 2), EALIGN),
    (dict(y=P + 4096, ldy=260), EALIGN), (dict(y=P + 4096, ldq=260), EALIGN), (dict(pages=P + 2), EALIGN),
    (dict(lens=P + 1), EALIGN), (dict(ws=P + 8), EALIGN), (dict(b=65537), EUNSUPPORTED),
    (dict(b=1 << 40), EUNSUPPORTED), (dict(q_heads=4098, ldq=1 << 20, ldy=1 << 20), EUNSUPPORTED),
    (dict(max_pages=1 << 27, ldpages=1 << 27), EUNSUPPORTED), (dict(max_pages=(1 << 26) + 1, ldpages=1 << 27), EUNSUPPORTED),
    (dict(max_pages=1 << 24, ldpages=1 << 24, b=65536), EUNSUPPORTED), (dict(scale=1e32), EUNSUPPORTED),
    (dict(scale=1.0, softcap=1e-38), EUNSUPPORTED), (dict(b=0, q=None, lens=None, y=None, ws=None), OK),
])
def test_attention_refusals(change, status):
    a = dict(c=cache(), q=P, ldq=256, q_heads=4, pages=P, ldpages=5, max_pages=5, lens=P, b=3, scale=0.1, softcap=0.0,
             window=0, y=P, ldy=256, ws=P, ws_bytes=1 << 40, stream=None)
    a.update(change)
    a["c"] = passed(a["c"])
    assert call("woq_attn_decode", *a.values()) == status


def test_attention_workspace_sizes():
    for c, s in BAD_CACHES:
        assert call("woq_attn_decode_workspace", passed(c), 1025 * 2 if c and c.heads > 1024 else 4, 1) == s
    for heads, b, s in ((0, 1, EINVAL), (3, 1, EINVAL), (4, -1, EINVAL), (4098, 1, EUNSUPPORTED), (4, 65537, EUNSUPPORTED)):
        assert call("woq_attn_decode_workspace", passed(cache()), heads, b) == s
    last = 0
    for b in (0, 1, 2, 64, 1000, 65536):                   # no less for more rows
        n = woq.woq_attn_decode_workspace(cache(), 4, b)
        assert n >= last
        last = n


@pytest.mark.parametrize("change,status", [
    (dict(b=-1), EINVAL), (dict(N=0), EINVAL), (dict(ld=96), EINVAL), (dict(x=None), EINVAL), (dict(u=None), EINVAL),
    (dict(token=None), EINVAL), (dict(x=P + 8), EALIGN), (dict(ld=100), EALIGN), (dict(T=P + 2), EALIGN),
    (dict(k=P + 1), EALIGN), (dict(p=P + 2), EALIGN), (dict(m=P + 2), EALIGN), (dict(u=P + 2), EALIGN),
    (dict(token=P + 2), EALIGN), (dict(prob=P + 2), EALIGN), (dict(N=(1 << 24) + 1, ld=1 << 25), EUNSUPPORTED),
    (dict(b=1 << 31), EUNSUPPORTED), (dict(b=0, x=None, u=None, token=None), OK),
])
def test_sampling_refusals(change, status):
    a = dict(x=P, ld=104, N=100, b=3, T=P, k=P, p=P, m=P, u=P, token=P, prob=P, stream=None)
    a.update(change)
    assert call("woq_sample", *a.values()) == status


def test_binding_refuses_what_the_library_cannot_see():
    import torch
    half, i32 = torch.float16, torch.int32
    rows, slots, f = torch.zeros(3, 128, dtype=half), torch.zeros(3, dtype=i32), torch.zeros(3)
    q, rope = torch.zeros(3, 256, dtype=half), torch.zeros(10, 64)
    c = cache()
    with pytest.raises(ValueError, match="not on the GPU"):
        woq.woq_cache_write(c, rows, rows, slots)
    for bad in (dict(q=q), dict(q_out=q), dict(rope=rope), dict(pos=slots), dict(q=q[:, :100], q_out=q),
                dict(q=q, q_out=q[:2], rope=rope, pos=slots), dict(rope=rope[0], pos=slots),
                dict(rope=rope.double(), pos=slots), dict(rope=rope, pos=slots[:2])):
        with pytest.raises(ValueError):
            woq.woq_cache_write(c, rows, rows, slots, **bad)
    for args in ((rows[:, :100], rows, slots), (rows, rows[:2], slots), (rows, rows, slots[:2]),
                 (rows, rows.float(), slots), (rows, rows, slots.long())):
        with pytest.raises(ValueError):
            woq.woq_cache_write(c, *args)
    for args in ((slots, rows[:2], rows), (slots, rows, rows[:, :100]), (slots.long(), rows, rows), (slots, rows, rows)):
        with pytest.raises(ValueError):
            woq.woq_cache_read(c, *args)
    pages, ws = torch.zeros(3, 5, dtype=i32), torch.zeros(1 << 20, dtype=torch.uint8)
    for args in ((q, pages, slots, q, ws), (q[:, :100], pages, slots, q, ws), (q, pages[:2], slots, q, ws),
                 (q, pages, slots[:2], q, ws), (q, pages, slots, q[:2], ws), (q, pages.long(), slots, q, ws),
                 (q, pages, slots, q, ws.view(2, -1).t())):
        with pytest.raises(ValueError):
            woq.woq_attn_decode(c, *args)
    for kw in (dict(), dict(N=129), dict(top_k=f), dict(top_p=slots), dict(min_p=f[:2]), dict(temperature=f.double()),
               dict(prob=f[:2])):
        with pytest.raises(ValueError):
            woq.woq_sample(rows, f, slots, **kw)
    for args in ((rows, slots, slots), (rows, f, f), (rows, f[:2], slots), (rows.float(), f, slots)):
        with pytest.raises(ValueError):
            woq.woq_sample(*args)
    k = torch.zeros(10, 2, 16, 64, dtype=torch.uint8)
    s = torch.zeros(10, 2, 16)
    for args in ((k, k), (k, k, s), (k, k, s, s), (k, k[:9], s, s), (k[0], k[0], s, s)):
        with pytest.raises(ValueError):                   # the third is well formed, but not on the GPU
            woq.DeviceCache(*args)


def test_binding_refuses_a_cache_of_another_device():
    import torch
    from test_operators_host import on_gpu
    half, i32 = torch.float16, torch.int32
    rows, slots = on_gpu(torch.zeros(3, 128, dtype=half), 0), on_gpu(torch.zeros(3, dtype=i32), 0)
    c = cache()
    assert c.device is None                       # a descriptor made by hand says nothing
    c.device = 1
    with pytest.raises(ValueError, match="woq_cache_write: the cache"):
        woq.woq_cache_write(c, rows, rows, slots)
    with pytest.raises(ValueError, match="woq_cache_read: the cache"):
        woq.woq_cache_read(c, slots, rows, rows)
    pages, ws = on_gpu(torch.zeros(3, 5, dtype=i32), 0), on_gpu(torch.zeros(1 << 20, dtype=torch.uint8), 0)
    with pytest.raises(ValueError, match="woq_attn_decode: the cache"):
        woq.woq_attn_decode(c, rows, pages, slots, rows, ws)


def test_stack_with_attention_refusals():
    one = (ctypes.c_void_p * 1)(P)
    assert call("woq_stack_run_attn", None, one, one, 1, one, P, P, P, 4, 4, P, P, 1 << 20, None) == EINVAL
    assert call("woq_stack_attn_workspace", None, one, 1) == EINVAL
