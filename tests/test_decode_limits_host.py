"""CPU checks of limits of the operators between a decode step's products that
were found too wide: what they refuse, before anything is launched."""
import pytest

from test_decode_host import EUNSUPPORTED, P, cache, call, passed
from weight_only_quantized_quantize_amd import woq


@pytest.mark.parametrize("fmt", [woq.CACHE_INT8, woq.CACHE_FP16])
@pytest.mark.parametrize("softcap", [2.0 ** 64 * (1 + 2.0 ** -23), 1e30, 2.4e38, 3.4e38])
def test_attention_refuses_bounds_that_fp32_scores_vanish_under(fmt, softcap):
    """A bound times log2(e) has to be finite, and a score divided by it normal."""
    a = dict(c=passed(cache(fmt=fmt)), q=P, ldq=256, q_heads=4, pages=P, ldpages=5, max_pages=5, lens=P, b=3, scale=0.1,
             softcap=softcap, window=0, y=P, ldy=256, ws=P, ws_bytes=1 << 40, stream=None)
    assert call("woq_attn_decode", *a.values()) == EUNSUPPORTED
