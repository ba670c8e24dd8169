"""Pointers that the raw calls take: where C has no use for NULL, None is an error in Python; where it has, None is NULL."""
import pytest

import tiered_kv_cache_gqa_gb300 as tkv


@pytest.mark.parametrize("call", [
    lambda: tkv.tkv_append(None, 0, None, 0x1000, 1), lambda: tkv.tkv_append(None, 0, 0x1000, None, 1),
    lambda: tkv.tkv_decode_step(None, 0, None, 0x1000), lambda: tkv.tkv_decode_step(None, 0, 0x1000, None)])
def test_none_is_no_pointer(call):
    with pytest.raises(TypeError):
        call()


def test_none_is_null_where_c_says_so():
    c = tkv.PagedDesc()
    assert tkv.tkv_paged_attention(c, 0x1000, 0x2000, None, tkv.TKV_BF16, 1, 2, (128, 64), (128, 64), 0x3000, 1, 1, 0, 0.1, None, 0,
                                   status=None, stream=1) == tkv.TKV_EINVAL
