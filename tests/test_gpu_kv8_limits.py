"""The 8-bit cache at the ends of what its header allows: rows that fill no warp, sizes of values that meet the ends of
fp32 and of the weights' types, non-finite inputs, calls in place and on several streams.

Bounds as in test_gpu_kv8; what a test adds to them stands beside it."""

import numpy as np
import pytest

from oracle import kv8

from .gpu_common import DEV, to_dev, torch, tq, wl
from .test_gpu_kv8 import DT, Cache, _attend, _bound, _causal_case, _check, _decode_case, _table, ctx_for, values

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g,n_new,starts,lens", [(1, 17, [0, 100], None), (5, 4, [0, 700, 3000], None),
                                                 (3, 11, [2300], None), (1, 129, [0, 40], [129, 33]),
                                                 (1, 161, [900, 0], [161, 160]), (7, 31, [5, 2000], [31, 29])])
def test_causal_rows_that_fill_no_warp(d, g, n_new, starts, lens):
    """Row counts that leave a warp of the tcgen05 form with some rows and some lanes without: items of one tile, of
    several that the halves share, of more than 128 rows, whole and in parts."""
    rng = np.random.default_rng(60)
    _causal_case(rng, "bf16", d, 2, 2 * g, starts, n_new, lens, rows=24)
    _causal_case(rng, "bf16", d, 2, 2 * g, starts, n_new, lens, window=150, sinks=5, rows=24)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq", [17, 40, 131])
def test_decode_rows_that_fill_no_warp(d, hq):
    rng = np.random.default_rng(61)
    _decode_case(rng, "bf16", d, 1, hq, [1, 0, 100, 1500])
    _decode_case(rng, "bf16", d, 2, 2 * hq, [5000])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g", [1, 3, 5, 11])
def test_decode_short_contexts_with_odd_rows(dtype, d, g):
    """A cluster's CTAs share out an item's rows: shares that end inside a warp, and CTAs with none."""
    rng = np.random.default_rng(62)
    for lens in ([700], [400, 0, 33], [2500]):
        _decode_case(rng, dtype, d, 1, g, lens)
    _decode_case(rng, dtype, d, 1, g, [2500], window=300, sinks=3)
