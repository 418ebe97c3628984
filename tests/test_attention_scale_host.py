"""The scores' scale of attention over the cache: where log2(e) times it is infinite, the call is refused."""
import pytest

from tests.test_abi_host import OK, VALUE
from tests.test_attention_logprobs_host import attend, nrt  # noqa: F401
from tests.test_kv_cache_host import cache


@pytest.mark.parametrize("scale,want", [(2.0 ** 127, OK), (-2.0 ** 127, OK), (0.0, OK), (2.4e38, VALUE),
                                        (-3.4e38, VALUE), (float("-inf"), VALUE)])
def test_scales(nrt, scale, want):  # noqa: F811
    assert attend(nrt, cache(), tokens=0, scale=scale) == want
