"""Reordering of more caches of one shape than a launch takes."""
import numpy as np
import pytest

import tiered_kv_cache_gqa_gb300 as tkv
from test_gpu_beam import Beams

pytestmark = pytest.mark.gpu


def kinds_of(first, second, third, n):
    """n caches, seven in ten of the first kind, the others between them."""
    return tuple(second if i % 10 in (3, 8) else third if i % 10 == 6 else first for i in range(n))


@pytest.mark.parametrize("kinds,heads,d", [(kinds_of("e4m3", "bf16", "int4", 190), 2, 64), (kinds_of("e4m3", "fp16", "int4", 370), 1, 64),
                                           (kinds_of("bf16", "e4m3", "fp16", 190), 1, 64), (kinds_of("int4", "e4m3", "bf16", 187), 1, 128)])
@pytest.mark.parametrize("groups,beams,length,page", [(2, 3, 41, 16), (1, 9, 33, 32)])
def test_two_and_three_launches_of_one_shape(kinds, heads, d, groups, beams, length, page):
    b = Beams(groups, beams, length, page, kinds, heads, d)
    rng = np.random.default_rng(length)
    b.check(rng.permuted(np.tile(np.arange(beams), (groups, 1)), axis=1))
    b.check(rng.integers(-1, beams, (groups, beams)))
    b.check(np.zeros((groups, beams), int))


@pytest.mark.parametrize("at", [3, 127, 128, 200])
def test_one_cache_with_fewer_pages_among_many(at):
    """In whichever launch it is: its beams without a page stay, all others of all caches follow."""
    b = Beams(2, 5, 41, 16, ("e4m3",) * 201)
    left = b.num_pages - 7
    b.pages[at], b.np_pages[at] = b.pages[at][:left], b.np_pages[at][:left]
    b.caches[at] = tkv.PagedCache(b.pages[at], b.table, b.lens)
    b.layers = tkv.PagedLayers(b.caches)
    parents = np.array([[1, 2, 3, 4, 0], [4, 0, 0, 1, 1]])
    moved = np.concatenate([np.stack([b.pt[5 * g:5 * g + 5, 2], b.pt[5 * g + parents[g], 2]], 1) for g in range(2)])
    assert (moved >= left).any()
    b.check(parents, tkv.TKV_ECAPACITY)
