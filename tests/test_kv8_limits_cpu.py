"""The 8-bit cache's entry points at the ends of their sizes, without a GPU (see test_kv8_cpu for how)."""

import ctypes
import itertools

import pytest

from .test_kv8_cpu import Fake, _append, _attend, _cache, _rope, f, tq  # noqa: F401


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("h", [1, 4, 8])
def test_a_workspace_for_the_largest_call_serves_the_smaller_ones(d, h):
    """Never less for more sequences, tokens, heads or length: across the blocks of 8 and 16 rows, the two forms, and
    what one list of blocks holds."""
    fake = Fake(d)                                  # its memory has to last
    ctx = fake.ctx
    batches, news, groups, lens = [0, 1, 2, 31, 32, 33, 64, 2049], [1, 2, 5, 8, 9, 16, 17, 255, 1000, 4096], [1, 4, 8], [0, 100, 8192, 1 << 20]
    size = {(b, t, g, n): tq.tq_kv8_workspace_size(ctx, b, t, g * h, h, n)
            for b, t, g, n in itertools.product(batches, news, groups, lens) if b * t * g * h < 1 << 27}
    axes = (batches, news, groups, lens)
    for at, n in size.items():
        for i, axis in enumerate(axes):
            j = axis.index(at[i])
            less = at[:i] + (axis[j - 1],) + at[i + 1:]
            if j and less in size:
                assert size[less] <= n, (less, size[less], at, n)


def test_a_call_asks_for_no_workspace_of_a_form_that_it_does_not_take(f):
    """Few rows, fp32 and larger scales never run on tcgen05, whose parts are the larger ones."""
    size = lambda b, t, n: tq.tq_kv8_workspace_size(f.ctx, b, t, 8, 4, n)  # noqa: E731
    cache = _cache(f, max_pages_per_seq=512, num_pages=1000)
    few, sixteen, many = size(1, 1, 8192), size(1, 8, 8192), size(8, 1000, 8192)
    assert few < sixteen < many
    ask = lambda ws, t, **kw: _attend(f, True, cache=cache, batch=8, n_new=t, max_len=8192, ws_bytes=ws, **kw)  # noqa: E731
    assert _attend(f, False, cache=cache, batch=8, max_len=8192, ws_bytes=few) == tq.TQ_ERR_CUDA
    assert ask(sixteen, 1000, dtype=1) == ask(sixteen, 1000, scale=1.0) == tq.TQ_ERR_CUDA
    assert ask(sixteen, 1000, scale=0.05) == ask(many - 1, 1000, scale=0.05) == tq.TQ_ERR_WORKSPACE
    assert ask(many, 1000, scale=0.05) == tq.TQ_ERR_CUDA
    assert ask(many, 1000, scale=0.05) == ask(many, 8, scale=0.05) == tq.TQ_ERR_CUDA


@pytest.mark.parametrize("batch,n_new,hq", [(2 ** 31 - 1, 2 ** 31 - 1, 4), (2 ** 31 - 1, 2 ** 31 - 1, 8), (2 ** 30, 2 ** 30, 16),
                                            (2 ** 30, 2 ** 31 - 1, 32), (1 << 26, 1, 4), (1, 1 << 26, 4)])
def test_sizes_whose_product_passes_64_bits_are_refused(f, batch, n_new, hq):
    n = ctypes.c_size_t()
    assert tq.raw_status("tq_kv8_workspace_size", f.ctx, batch, n_new, hq, 4, 100, ctypes.byref(n)) == tq.TQ_ERR_UNSUPPORTED
    for dtype in (0, 1):
        assert _attend(f, True, batch=batch, n_new=n_new, hq=hq, dtype=dtype, ws_bytes=2 ** 63) == tq.TQ_ERR_UNSUPPORTED


def test_in_place_is_refused_where_a_row_has_two_items(f):
    g = Fake(256)
    one = dict(q=1 << 20, out=1 << 20)
    assert _attend(g, True, n_new=9, **one) == _attend(g, False, hq=4 * 17, **one) == tq.TQ_ERR_INVALID_ARG
    assert _attend(g, True, n_new=8, **one) == _attend(g, False, hq=4 * 16, **one) == tq.TQ_ERR_CUDA
    assert _attend(g, True, n_new=9, q=1 << 20, out=1 << 21) == tq.TQ_ERR_CUDA
    assert _attend(f, True, n_new=9, **one) == _attend(f, False, hq=4 * 17, **one) == tq.TQ_ERR_CUDA
