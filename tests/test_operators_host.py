"""CPU checks of the operators around a quantised linear (woq_add_rmsnorm,
woq_qgemm_int8_a8, woq_lora_add): the float64 definitions against explicit
loops and closed forms, and every refusal of the C entry points and of the
binding (nothing is launched, so no GPU is needed)."""
import ctypes

import numpy as np
import pytest

import oracle as O
from weight_only_quantized_quantize_amd import woq


# ------------------------------------------------------------- definitions

def test_norm_definition_against_loops():
    rng = np.random.default_rng(0)
    x, res, w = rng.standard_normal((3, 7)), rng.standard_normal((3, 7)), rng.standard_normal(7)
    s, v = O.add_rmsnorm(x, res, w, 1.0, 1e-3)
    for r in range(3):
        t = [x[r, k] + res[r, k] for k in range(7)]
        rms = (sum(a * a for a in t) / 7 + 1e-3) ** 0.5
        for k in range(7):
            assert abs(s[r, k] - t[k]) < 1e-15
            assert abs(v[r, k] - t[k] * (w[k] + 1.0) / rms) < 1e-14
    s, v = O.add_rmsnorm(x)
    np.testing.assert_array_equal(s, x)
    np.testing.assert_array_equal(v, x)
    # a row of one value a has rms |a|: the norm is its sign (eps aside)
    _, v = O.add_rmsnorm(np.full((1, 5), -3.0), None, np.ones(5), 0.0, 1e-12)
    np.testing.assert_allclose(v, -1.0, rtol=1e-9)
    np.testing.assert_allclose(O.rows_scale(np.array([[1.0, -254.0], [0.0, 0.0]])), [2.0, 0.0])


def test_product_definition_against_loops():
    rng = np.random.default_rng(1)
    codes = rng.integers(-127, 128, (5, 6)).astype(np.int8)
    xq = rng.integers(-128, 128, (2, 6)).astype(np.int8)
    y = O.linear_int8_a8(codes, [2, 5], [0.5, 0.25], xq, np.array([2.0, 3.0], np.float32))
    for r in range(2):
        for n in range(5):
            t = sum(int(codes[n, k]) * int(xq[r, k]) for k in range(6))
            assert y[r, n] == t * (0.5 if n < 2 else 0.25) * (2.0 if r == 0 else 3.0)


def test_adapter_definition_against_loops():
    rng = np.random.default_rng(2)
    count, N, K, R, ends = 2, 5, 4, 3, [2, 5]
    A, B = rng.standard_normal((count, 2 * R, K)), rng.standard_normal((count, N, R))
    x, base, scale = rng.standard_normal((4, K)), rng.standard_normal((4, N)), np.array([0.5, 2.0])
    ids, rank = [1, -1, 0, 2], [3, 2]
    y, spread = O.lora_add(base, x, ids, A, B, scale, ends, rank)
    np.testing.assert_array_equal(y[1], base[1])
    np.testing.assert_array_equal(y[3], base[3])
    assert not spread[1].any()
    for r, a in ((0, 1), (2, 0)):
        for n in range(N):
            first = 0 if n < 2 else R
            d = sum(B[a, n, j] * sum(A[a, first + j, k] * x[r, k] for k in range(K)) for j in range(rank[a]))
            assert abs(y[r, n] - base[r, n] - scale[a] * d) < 1e-12


# ---------------------------------------------------------------- refusals

P = 0x10000          # an aligned address that is never dereferenced


def call(name, *args):
    return getattr(woq.lib(), name)(*args)


def norm_args(**kw):
    a = dict(x=P, ldx=64, res=P, ldres=64, weight=P, offset=0.0, eps=1e-6, b=2, K=60, sum_out=P, ldsum=64, y=P,
             ldy=64, q=P, ldq=64, q_scale=P, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("change,status", [
    (dict(b=-1), woq.WOQ_EINVAL), (dict(K=0), woq.WOQ_EINVAL), (dict(x=None), woq.WOQ_EINVAL),
    (dict(ldx=56), woq.WOQ_EINVAL), (dict(ldres=56), woq.WOQ_EINVAL), (dict(ldsum=56), woq.WOQ_EINVAL),
    (dict(ldy=56), woq.WOQ_EINVAL), (dict(ldq=48), woq.WOQ_EINVAL), (dict(q_scale=None), woq.WOQ_EINVAL),
    (dict(sum_out=None, y=None, q=None), woq.WOQ_EINVAL), (dict(eps=0.0), woq.WOQ_EINVAL),
    (dict(eps=-1.0), woq.WOQ_EINVAL), (dict(eps=float("nan")), woq.WOQ_EINVAL),
    (dict(eps=float("inf")), woq.WOQ_EINVAL), (dict(offset=float("nan")), woq.WOQ_EINVAL),
    (dict(x=P + 2), woq.WOQ_EALIGN), (dict(res=P + 8), woq.WOQ_EALIGN), (dict(weight=P + 2), woq.WOQ_EALIGN),
    (dict(ldx=66), woq.WOQ_EALIGN), (dict(ldres=68), woq.WOQ_EALIGN), (dict(sum_out=P + 4), woq.WOQ_EALIGN),
    (dict(ldsum=68), woq.WOQ_EALIGN), (dict(y=P + 2), woq.WOQ_EALIGN), (dict(ldy=68), woq.WOQ_EALIGN),
    (dict(q=P + 8), woq.WOQ_EALIGN), (dict(ldq=72), woq.WOQ_EALIGN), (dict(q_scale=P + 2), woq.WOQ_EALIGN),
    (dict(K=65537, ldx=65544, ldres=65544, ldsum=65544, ldy=65544, ldq=65552), woq.WOQ_EUNSUPPORTED),
    (dict(b=1 << 31), woq.WOQ_EUNSUPPORTED), (dict(b=4000001), woq.WOQ_EUNSUPPORTED),
    (dict(b=0), woq.WOQ_OK), (dict(b=0, x=None), woq.WOQ_OK),
])
def test_norm_refusals(change, status):
    assert call("woq_add_rmsnorm", *norm_args(**change)) == status


def weight8(N=40, K=100, ends=None, codes=P):
    w = woq.Int8W()
    ends = [N] if ends is None else ends
    w.codes, w.N, w.K, w.nseg = codes, N, K, len(ends)
    for i, e in enumerate(ends):
        w.seg_end[i], w.seg_scale[i] = e, 0.01
    return w


@pytest.mark.parametrize("change,status", [
    (dict(w=None), woq.WOQ_EINVAL), (dict(w=weight8(K=0)), woq.WOQ_EINVAL), (dict(w=weight8(N=-1)), woq.WOQ_EINVAL),
    (dict(w=weight8(ends=[39])), woq.WOQ_EINVAL), (dict(w=weight8(ends=[30, 20, 40])), woq.WOQ_EINVAL),
    (dict(w=weight8(codes=None)), woq.WOQ_EINVAL), (dict(w=weight8(codes=P + 8)), woq.WOQ_EALIGN),
    (dict(b=-1), woq.WOQ_EINVAL), (dict(ldq=96), woq.WOQ_EINVAL), (dict(ldy=39), woq.WOQ_EINVAL),
    (dict(xq=None), woq.WOQ_EINVAL), (dict(xs=None), woq.WOQ_EINVAL), (dict(y=None), woq.WOQ_EINVAL),
    (dict(xq=P + 8), woq.WOQ_EALIGN), (dict(ldq=120), woq.WOQ_EALIGN), (dict(xs=P + 2), woq.WOQ_EALIGN),
    (dict(y=P + 1), woq.WOQ_EALIGN), (dict(w=weight8(K=131073), ldq=131088), woq.WOQ_EUNSUPPORTED),
    (dict(w=weight8(N=1 << 31), ldy=1 << 31), woq.WOQ_EUNSUPPORTED), (dict(b=1 << 31), woq.WOQ_EUNSUPPORTED),
    (dict(w=weight8(N=1 << 22), ldy=1 << 22, b=1 << 18), woq.WOQ_EUNSUPPORTED),
    (dict(b=0, xq=None), woq.WOQ_OK), (dict(w=weight8(N=0, codes=None)), woq.WOQ_OK),
])
def test_product_refusals(change, status):
    a = dict(w=weight8(), xq=P, ldq=112, xs=P, b=3, y=P, ldy=40, stream=None)
    a.update(change)
    if a["w"] is not None:
        a["w"] = ctypes.byref(a["w"])
    assert call("woq_qgemm_int8_a8", *a.values()) == status


def test_product_tiles():
    """The GPU's cases reach every tile that any size takes (on 256 compute units)."""
    from test_gpu_operators import PRODUCT_TILES
    tiles = {woq.woq_qgemm_int8_a8_tile(N, b) for N in list(range(1, 70000, 97)) + [128256, 262144, 1 << 24]
             for b in (1, 2, 16, 17, 32, 33, 50, 64, 65, 128, 129, 200, 256, 257, 400, 512, 1000, 1021, 3001, 4096, 70000)}
    assert tiles == {woq.woq_qgemm_int8_a8_tile(N, b) for N, _, b, _ in PRODUCT_TILES}
    for N, _, b, tile in PRODUCT_TILES:
        assert woq.woq_qgemm_int8_a8_tile(N, b) == tile, (N, b)
    for N, b, status in ((0, 1, woq.WOQ_EINVAL), (1, 0, woq.WOQ_EINVAL), (1 << 31, 1, woq.WOQ_EUNSUPPORTED),
                         (1, 1 << 31, woq.WOQ_EUNSUPPORTED)):
        with pytest.raises(woq.WoqError) as e:
            woq.woq_qgemm_int8_a8_tile(N, b)
        assert e.value.status == status
    assert call("woq_qgemm_int8_a8_tile", 1, 1, None, None) == woq.WOQ_EINVAL


@pytest.mark.parametrize("N", [1, 1000, 16400, 28672, 32768, 32784, 57344, 65536, 65552, 131072, 152064, 1 << 24])
def test_product_tiles_are_not_far_taller_than_the_batch(N):
    """However wide the weight: a workgroup of 128 or 256 rows for a batch of few
    would multiply mostly rows that are not there."""
    for b in (1, 2, 8, 15, 16, 17, 31, 32, 33, 50, 61, 64, 65, 100, 128):
        rows, _ = woq.woq_qgemm_int8_a8_tile(N, b)
        assert rows <= (64 if b <= 64 else 128), (N, b, rows)
        if N > 1 << 16:                     # several rounds of workgroups, whatever the tile
            assert rows == min(r for r in (16, 32, 64, 128) if r >= b), (N, b, rows)
    for n, b in ((N, 1), (1 << 30, 1), (1 << 30, 33), (1 << 24, 16384)):    # a launch has fewer than 2^32 threads
        rows, cols = woq.woq_qgemm_int8_a8_tile(n, b)
        assert -(-n // cols) * -(-b // rows) * 512 < 1 << 32


def pool(N=40, K=100, lda=104, R=16, count=3, ends=None, **ptrs):
    w = woq.LoraW()
    ends = [N] if ends is None else ends
    for name in ("A", "B", "scale"):
        setattr(w, name, ptrs.get(name, P))
    w.rank = ptrs.get("rank")
    w.N, w.K, w.lda, w.R, w.count, w.nseg = N, K, lda, R, count, len(ends)
    for i, e in enumerate(ends):
        w.seg_end[i] = e
    return w


@pytest.mark.parametrize("change,status", [
    (dict(w=None), woq.WOQ_EINVAL), (dict(w=pool(K=0)), woq.WOQ_EINVAL), (dict(w=pool(N=-1)), woq.WOQ_EINVAL),
    (dict(w=pool(lda=96)), woq.WOQ_EINVAL), (dict(w=pool(R=0)), woq.WOQ_EINVAL), (dict(w=pool(count=-1)), woq.WOQ_EINVAL),
    (dict(w=pool(ends=[39])), woq.WOQ_EINVAL), (dict(w=pool(ends=[30, 20, 40])), woq.WOQ_EINVAL),
    (dict(w=pool(A=None)), woq.WOQ_EINVAL), (dict(w=pool(B=None)), woq.WOQ_EINVAL),
    (dict(w=pool(scale=None)), woq.WOQ_EINVAL), (dict(b=-1), woq.WOQ_EINVAL), (dict(ldx=96), woq.WOQ_EINVAL),
    (dict(ldy=39), woq.WOQ_EINVAL), (dict(ldbase=39), woq.WOQ_EINVAL), (dict(x=None), woq.WOQ_EINVAL),
    (dict(ids=None), woq.WOQ_EINVAL), (dict(y=None), woq.WOQ_EINVAL), (dict(ws=None), woq.WOQ_EINVAL),
    (dict(ws_bytes=16), woq.WOQ_EINVAL),
    (dict(w=pool(A=P + 8)), woq.WOQ_EALIGN), (dict(w=pool(B=P + 8)), woq.WOQ_EALIGN),
    (dict(w=pool(scale=P + 2)), woq.WOQ_EALIGN), (dict(w=pool(rank=P + 2)), woq.WOQ_EALIGN),
    (dict(w=pool(lda=100)), woq.WOQ_EALIGN), (dict(x=P + 8), woq.WOQ_EALIGN), (dict(ldx=108), woq.WOQ_EALIGN),
    (dict(ids=P + 2), woq.WOQ_EALIGN), (dict(y=P + 1), woq.WOQ_EALIGN), (dict(base=P + 1), woq.WOQ_EALIGN),
    (dict(ws=P + 8), woq.WOQ_EALIGN), (dict(w=pool(R=12)), woq.WOQ_EUNSUPPORTED),
    (dict(w=pool(R=264)), woq.WOQ_EUNSUPPORTED), (dict(w=pool(N=1 << 31), ldy=1 << 31, ldbase=1 << 31), woq.WOQ_EUNSUPPORTED),
    (dict(w=pool(N=(1 << 28) + 1), ldy=1 << 29, ldbase=1 << 29), woq.WOQ_EUNSUPPORTED),
    (dict(b=1 << 31), woq.WOQ_EUNSUPPORTED), (dict(b=1000001), woq.WOQ_EUNSUPPORTED),
    (dict(b=0, x=None), woq.WOQ_OK), (dict(w=pool(N=0, A=None)), woq.WOQ_OK),
])
def test_adapter_refusals(change, status):
    a = dict(w=pool(), x=P, ldx=104, ids=P, b=3, base=P, ldbase=40, y=P, ldy=40, ws=P, ws_bytes=1 << 40, stream=None)
    a.update(change)
    if a["w"] is not None:
        a["w"] = ctypes.byref(a["w"])
    assert call("woq_lora_add", *a.values()) == status


def test_adapter_workspace_sizes():
    for w, b in ((pool(), -1), (pool(R=0), 4), (pool(ends=[39]), 4)):
        assert call("woq_lora_workspace", ctypes.byref(w), b) == woq.WOQ_EINVAL
    for w, b in ((pool(R=12), 4), (pool(R=264), 4), (pool(), 1 << 31)):
        assert call("woq_lora_workspace", ctypes.byref(w), b) == woq.WOQ_EUNSUPPORTED
    assert call("woq_lora_workspace", ctypes.byref(pool()), 0) >= 0
    # at least the inner products of every row, and no less for more rows
    last = 0
    for b in (1, 2, 15, 16, 17, 64, 65, 100, 1000, 4096, 100000):
        n = woq.woq_lora_workspace(pool(ends=[10, 20, 40]), b)
        assert n >= b * 3 * 16 * 4 and n >= last, b
        last = n


def test_binding_refuses_what_the_library_cannot_see():
    import torch
    half, cpu = torch.float16, torch.zeros(2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):                       # not on the GPU
        woq.woq_add_rmsnorm(cpu, torch.ones(64, dtype=half), 1e-6, y=cpu)
    with pytest.raises(ValueError):                       # codes without scales
        woq.woq_add_rmsnorm(cpu, None, 1e-6, q=torch.zeros(2, 64, dtype=torch.int8))
    with pytest.raises(ValueError):
        woq.woq_qgemm_int8_a8(weight8(), torch.zeros(2, 112, dtype=torch.int8), torch.zeros(2), cpu)
    with pytest.raises(ValueError):
        woq.woq_lora_add(pool(), cpu, torch.zeros(2, dtype=torch.int32), None, cpu, torch.zeros(8))
    A, B, s = torch.zeros(2, 32, 64, dtype=half), torch.zeros(2, 40, 16, dtype=half), torch.zeros(2)
    for bad in (dict(segments=[40]), dict(segments=[10, 39]), dict(segments=[])):
        with pytest.raises(ValueError):
            woq.DeviceLora(A, B, s, **bad)
    with pytest.raises(ValueError):
        woq.DeviceLora(A, B, s, segments=[10, 40], K=65)
    with pytest.raises(ValueError):                       # well formed, but not on the GPU
        woq.DeviceLora(A, B, s, segments=[10, 40])


def on_gpu(t, index):
    """The CPU tensor t, said to lie on a GPU: enough for checks that come before any launch."""
    import torch

    class Placed(torch.Tensor):
        def get_device(self):
            return index

    return t.as_subclass(Placed)


def test_binding_refuses_weights_and_pools_of_another_device():
    import torch
    half = torch.float16
    x, ids = on_gpu(torch.zeros(2, 64, dtype=half), 0), on_gpu(torch.zeros(2, dtype=torch.int32), 0)
    y, ws = on_gpu(torch.zeros(2, 40, dtype=half), 0), on_gpu(torch.zeros(1 << 16, dtype=torch.uint8), 0)
    q, qs = on_gpu(torch.zeros(2, 64, dtype=torch.int8), 0), on_gpu(torch.zeros(2), 0)

    host_weight = woq.DeviceInt8([(np.zeros((40, 64), np.int8), 1.0)], device="cpu")
    assert host_weight.desc.device == -1
    with pytest.raises(ValueError, match="woq_qgemm_int8_a8: the weight"):
        woq.woq_qgemm_int8_a8(host_weight.desc, q, qs, y)
    w = pool(K=64, lda=64)
    assert w.device is None                       # a descriptor made by hand says nothing
    w.device = 1
    with pytest.raises(ValueError, match="woq_lora_add: the pool"):
        woq.woq_lora_add(w, x, ids, None, y, ws)

    class Pool:
        desc = w

    st = woq.Stack.__new__(woq.Stack)
    st.n, st.handle, st._in, st._out, st._pin, st._pout = 2, None, [x], [y], None, None
    with pytest.raises(ValueError, match="woq_stack_run_lora: the pool"):
        st.run_lora(2, [None, Pool()], ids, ws)
    del st.handle


def test_stack_with_adapters_refusals():
    one = (ctypes.c_void_p * 1)(P)
    for args in ((None, one, one, 1, one, P, P, 1 << 20, None),):
        assert call("woq_stack_run_lora", *args) == woq.WOQ_EINVAL
    assert call("woq_stack_lora_workspace", None, one, 1) == woq.WOQ_EINVAL
