"""CPU checks of limits of the operators between a decode step's products that
were found too wide: what they refuse, before anything is launched."""
import pytest

from test_decode_host import EUNSUPPORTED, P, cache, call, passed, write_args
from weight_only_quantized_quantize_amd import woq


@pytest.mark.parametrize("fmt", [woq.CACHE_INT8, woq.CACHE_FP16])
@pytest.mark.parametrize("softcap", [2.0 ** 64 * (1 + 2.0 ** -23), 1e30, 2.4e38, 3.4e38])
def test_attention_refuses_bounds_that_fp32_scores_vanish_under(fmt, softcap):
    """A bound times log2(e) has to be finite, and a score divided by it normal."""
    a = dict(c=passed(cache(fmt=fmt)), q=P, ldq=256, q_heads=4, pages=P, ldpages=5, max_pages=5, lens=P, b=3, scale=0.1,
             softcap=softcap, window=0, y=P, ldy=256, ws=P, ws_bytes=1 << 40, stream=None)
    assert call("woq_attn_decode", *a.values()) == EUNSUPPORTED


@pytest.mark.parametrize("dim,lanes", [(16, 4), (64, 4), (80, 8), (128, 8), (144, 16), (256, 16)])
def test_cache_refuses_what_one_launch_can_not_take(dim, lanes):
    """A head takes 4, 8 or 16 threads and a launch fewer than 2^32, in whole
    workgroups of 256: the smallest batches that do not fit, and some that are larger."""
    c = cache(heads=2, dim=dim)
    heads = (2 ** 32 - 256) // lanes                # of a call, at most
    for rows in (1, 7, heads // 8):
        b = -(-(heads + 1) // 8) + rows - 1         # 4 heads of queries, 2 of keys and values each
        w = write_args(c=c, b=b, rot=16, ldk=1024, ldv=1024, ldq=1024, ldqo=1024, q_out=P + 4096)
        assert call("woq_cache_write", *w) == EUNSUPPORTED, b
        n = -(-(heads + 1) // 4) + rows - 1
        assert call("woq_cache_read", passed(c), P, n, P, 1024, P, 1024, None) == EUNSUPPORTED, n
