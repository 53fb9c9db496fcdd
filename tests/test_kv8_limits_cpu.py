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


def test_arrays_off_their_elements_boundary_are_refused(f):
    """int32 and fp32 arrays: a kernel's load from there would end the process's use of the GPU."""
    odd = (1 << 20) + 2
    for name in ("k_scale", "v_scale", "block_table"):
        c = _cache(f, **{name: odd})
        assert _append(f, cache=c) == _attend(f, False, cache=c) == _attend(f, True, cache=c) == tq.TQ_ERR_INVALID_ARG, name
    assert _append(f, start=odd) == _attend(f, False, lens=odd) == _attend(f, True, lens=odd) == tq.TQ_ERR_INVALID_ARG
    assert _append(f, rope=_rope(f, pos=odd)) == tq.TQ_ERR_INVALID_ARG
    new = lambda at: tq.raw_status("tq_kv8_append", f.ctx, f.cache, f.buf, f.buf, f.buf, 0, 2, 3, 8, f.buf, at, None, f.buf,  # noqa: E731
                                   0, 0, 0, None)
    assert new(odd) == tq.TQ_ERR_INVALID_ARG and new(f.buf) == tq.TQ_ERR_CUDA
    causal = lambda at: tq.raw_status("tq_kv8_causal_attention", f.ctx, f.cache, f.buf, 0, 2, 3, 8, f.buf, at, 100, 0, 0,  # noqa: E731
                                      ctypes.c_float(0.1), f.buf, f.buf, 1 << 40, None)
    assert causal(odd) == tq.TQ_ERR_INVALID_ARG
    assert causal(f.buf) == tq.TQ_ERR_CUDA
    # of a cache that is only half used, the other half is not looked at
    assert _append(f, cache=_cache(f, k_scale=odd), k=None) == tq.TQ_ERR_CUDA


def test_the_section_of_a_single_axis_is_not_read(f):
    for section in ((-1, 0, 0, 0), (2 ** 31 - 1, -5, 0, 0), (0, 0, 0, 0)):
        assert _append(f, rope=_rope(f, section=section)) == tq.TQ_ERR_CUDA
    assert _append(f, rope=_rope(f, num_axes=2, section=(-1, 65, 0, 0), pos=f.buf)) == tq.TQ_ERR_INVALID_ARG
