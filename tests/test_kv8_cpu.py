"""The 8-bit cache without a GPU: its oracle against torch's own e4m3, and the entry points' refusals.

A context cannot be made here, so the refusals are asked of a zeroed block of memory that starts with a
configuration, as a context does; a call that passes every check ends at the missing device."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import kv8

tq = pytest.importorskip("online_kv_cache_02_gb300.tq")


def test_e4m3_values_and_rounding():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(kv8.VALUES))
    assert np.array_equal(t[~np.isnan(t)], kv8.VALUES[~np.isnan(t)])
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * np.exp(rng.uniform(-12, 6, 20000)), t[~np.isnan(t)],
                        (kv8.VALUES[:126] + kv8.VALUES[1:127]) / 2])          # every tie
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = kv8.e4m3_encode(x.astype(np.float64))
    assert np.array_equal(got, want)
    assert np.array_equal(kv8.e4m3_encode([np.nan, np.inf, -np.inf, 1e9]), [0, 0x7E, 0xFE, 0x7E])


@pytest.mark.parametrize("amax,e", [(448.0, 0), (np.nextafter(448.0, 500.0), 1), (447.0, 0), (224.0, -1), (0.0, -100),
                                    (1e-40, -100), (3e38, 119), (448.0 * 2.0 ** -30, -30)])
def test_block_exponent(amax, e):
    assert kv8.block_exponent(amax) == e


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_relative_positions(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 64))
    f = 100.0 ** (-np.arange(24) / 24)
    turn = lambda x, p: kv8.rotate(x, np.cos(p * f), np.sin(p * f), interleaved)  # noqa: E731
    assert np.allclose(np.linalg.norm(turn(q, 7)), np.linalg.norm(q))
    assert np.allclose(turn(q, 9) @ turn(k, 4), turn(q, 25) @ turn(k, 20))
    assert np.array_equal(turn(q, 5)[48:], q[48:])


def test_growing_block_equals_one_call_but_for_the_smallest_codes():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((16, 2, 64)) * np.exp2(np.arange(16))[:, None, None]
    row = [0]
    a, sa = np.zeros((1, 2, 16, 64), np.uint8), np.ones((1, 2))
    b, sb = a.copy(), sa.copy()
    kv8.append(a, sa, row, 0, x)
    for i in range(16):
        kv8.append(b, sb, row, i, x[i:i + 1])
    assert np.array_equal(sa, sb)
    d = np.abs(kv8.VALUES[a] - kv8.VALUES[b])
    assert d.max() <= 2.0 ** -9                     # one step of the subnormals: rounded twice


class Fake:
    """Memory that looks like a context's first bytes, and buffers that look like device memory."""

    def __init__(self, d=128):
        self.mem = ctypes.create_string_buffer(1 << 16)
        ctypes.memmove(self.mem, ctypes.byref(tq.make_config(d=d)), ctypes.sizeof(tq.TQConfig))
        self.ctx = ctypes.addressof(self.mem)
        self.buf = 1 << 20                          # an aligned address; nothing may read it
        self.cache = tq.make_kv8_cache(self.buf, self.buf, self.buf, self.buf, self.buf, 8, 100, 4)
        self.rope = tq.make_rope(self.buf, 64, d)


def _append(f, cache="-", k="-", v="-", q="-", dtype=0, batch=2, n_new=3, hq=8, start="-", rope="-", q_out="-",
            strides=(0, 0, 0)):
    v_ = lambda x: f.buf if isinstance(x, str) else x  # noqa: E731
    return tq.raw_status("tq_kv8_append", f.ctx, f.cache if cache == "-" else cache, v_(k), v_(v), v_(q), dtype, batch,
                         n_new, hq, v_(start), None, f.rope if rope == "-" else rope, v_(q_out), *strides, None)


def _attend(f, causal, cache="-", q="-", dtype=0, batch=2, n_new=3, hq=8, lens="-", max_len=100, window=0, sinks=0,
            scale=0.1, out="-", ws="-", ws_bytes=1 << 40):
    v_ = lambda x: f.buf if isinstance(x, str) else x  # noqa: E731
    c = f.cache if cache == "-" else cache
    if causal:
        return tq.raw_status("tq_kv8_causal_attention", f.ctx, c, v_(q), dtype, batch, n_new, hq, v_(lens), None,
                             max_len, window, sinks, ctypes.c_float(scale), v_(out), v_(ws), ws_bytes, None)
    return tq.raw_status("tq_kv8_decode_attention", f.ctx, c, v_(q), dtype, batch, hq, v_(lens), max_len, window, sinks,
                         ctypes.c_float(scale), v_(out), v_(ws), ws_bytes, None)


def _cache(f, **kw):
    c = tq.make_kv8_cache(f.buf, f.buf, f.buf, f.buf, f.buf, 8, 100, 4)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.fixture
def f():
    if torch.cuda.is_available():
        pytest.skip("the addresses here are not device memory: a call that is not refused must not be made")
    return Fake()


def _rope(f, **kw):
    sec = kw.pop("section", None)
    r = tq.make_rope(f.buf, 64, 128)
    for k, v in kw.items():
        setattr(r, k, v)
    if sec is not None:
        r.section = (ctypes.c_int * 4)(*sec)
    return r


def test_calls_that_pass_every_check_end_at_the_missing_device(f):
    assert _append(f) == tq.TQ_ERR_CUDA
    assert _append(f, k=None, q=None) == tq.TQ_ERR_CUDA
    assert _append(f, strides=(4 * 128, 2000, 1024)) == tq.TQ_ERR_CUDA
    assert _append(f, rope=None) == tq.TQ_ERR_CUDA
    assert _append(f, rope=_rope(f, num_axes=3, section=(16, 24, 24), pos=f.buf)) == tq.TQ_ERR_CUDA
    assert _attend(f, False) == tq.TQ_ERR_CUDA
    assert _attend(f, True, window=5, sinks=2) == tq.TQ_ERR_CUDA
    assert _attend(f, True, hq=4 * 33) == tq.TQ_ERR_CUDA


def test_nothing_to_do_is_no_error(f):
    assert _append(f, batch=0) == tq.TQ_OK
    assert _append(f, n_new=0) == tq.TQ_OK
    assert _attend(f, False, batch=0) == tq.TQ_OK


@pytest.mark.parametrize("kw", [dict(cache=None), dict(k=None, v=None, q=None), dict(dtype=2), dict(batch=-1),
                                dict(n_new=-1), dict(hq=0), dict(start=None), dict(q_out=None), dict(q_out=(1 << 20) + 8),
                                dict(k=(1 << 20) + 1), dict(strides=(511, 0, 0)), dict(strides=(0, -4, 0)),
                                dict(strides=(0, 0, 1023)), dict(q_out=1 << 20, strides=(0, 0, 2048))])
def test_append_refuses(f, kw):
    assert _append(f, **kw) == tq.TQ_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(k_codes=None), dict(v_scale=None), dict(k_codes=(1 << 20) + 8), dict(block_table=None),
                                dict(max_pages_per_seq=0), dict(num_pages=0), dict(num_kv_heads=0)])
def test_bad_caches_are_refused(f, kw):
    c = _cache(f, **kw)
    assert _append(f, cache=c) == tq.TQ_ERR_INVALID_ARG
    assert _attend(f, False, cache=c) == tq.TQ_ERR_INVALID_ARG
    assert _attend(f, True, cache=c) == tq.TQ_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(cos_sin=None), dict(cos_sin=(1 << 20) + 4), dict(max_pos=0), dict(rot_dim=0),
                                dict(rot_dim=8), dict(rot_dim=144), dict(rot_dim=40), dict(interleaved=2),
                                dict(num_axes=0), dict(num_axes=5), dict(num_axes=2, section=(32, 32, 0, 0)),
                                dict(num_axes=2, section=(32, 31, 0, 0), pos=1 << 20),
                                dict(num_axes=2, section=(65, -1, 0, 0), pos=1 << 20)])
def test_bad_rotations_are_refused(f, kw):
    assert _append(f, rope=_rope(f, **kw)) == tq.TQ_ERR_INVALID_ARG


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("kw", [dict(cache=None), dict(q=None), dict(q=(1 << 20) + 8), dict(dtype=7), dict(batch=-1),
                                dict(hq=0), dict(hq=6), dict(lens=None), dict(max_len=-1), dict(window=-1), dict(sinks=-1),
                                dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None), dict(out=(1 << 20) + 4),
                                dict(ws=None), dict(ws=(1 << 20) + 8)])
def test_attention_refuses(f, causal, kw):
    assert _attend(f, causal, **kw) == tq.TQ_ERR_INVALID_ARG


def test_attention_refuses_small_workspaces_and_other_head_dims(f):
    n = tq.tq_kv8_workspace_size(f.ctx, 2, 3, 8, 4, 100)
    assert n > 0
    assert _attend(f, True, ws_bytes=n - 1) == tq.TQ_ERR_WORKSPACE
    assert _attend(f, True, ws_bytes=n) == tq.TQ_ERR_CUDA
    assert _attend(f, True, n_new=0) == tq.TQ_ERR_INVALID_ARG
    for d in (32, 96, 192):
        g = Fake(d)
        assert _attend(g, False) == tq.TQ_ERR_UNSUPPORTED
        assert _append(g) == tq.TQ_ERR_UNSUPPORTED
        assert tq.raw_status("tq_kv8_cache_layout", g.ctx, 4, ctypes.byref(ctypes.c_size_t()), None) == tq.TQ_ERR_UNSUPPORTED
    assert tq.tq_kv8_cache_layout(f.ctx, 4) == (4 * 16 * 128, 16)


def test_sizes_beyond_the_kernels_arithmetic_are_refused(f):
    assert _append(f, batch=2, n_new=(1 << 29) + 1) == tq.TQ_ERR_UNSUPPORTED
    assert _append(f, cache=_cache(f, num_kv_heads=65536, num_pages=1), k=None, v=None) == tq.TQ_ERR_UNSUPPORTED
    assert _append(f, cache=_cache(f, num_pages=1 << 29, num_kv_heads=4)) == tq.TQ_ERR_UNSUPPORTED
    for causal in (False, True):
        assert _attend(f, causal, cache=_cache(f, num_pages=1 << 29)) == tq.TQ_ERR_UNSUPPORTED
        assert _attend(f, causal, batch=1 << 20, hq=128, n_new=1) == tq.TQ_ERR_UNSUPPORTED
        assert _attend(f, causal, cache=_cache(f, max_pages_per_seq=1 << 26), max_len=1 << 30) == tq.TQ_ERR_UNSUPPORTED


def test_null_context_is_refused():
    n = ctypes.c_size_t()
    c = tq.make_kv8_cache(16, 16, 16, 16, 16, 1, 1, 1)
    assert tq.raw_status("tq_kv8_cache_layout", None, 8, ctypes.byref(n), None) == tq.TQ_ERR_INVALID_ARG
    assert tq.raw_status("tq_kv8_workspace_size", None, 1, 1, 8, 8, 16, ctypes.byref(n)) == tq.TQ_ERR_INVALID_ARG
    assert tq.raw_status("tq_kv8_append", None, c, 16, 16, 16, 0, 1, 1, 8, 16, None, None, 16, 0, 0, 0,
                         None) == tq.TQ_ERR_INVALID_ARG
    assert tq.raw_status("tq_kv8_decode_attention", None, c, 16, 0, 1, 8, 16, 8, 0, 0, ctypes.c_float(1), 16, 16, 1 << 30,
                         None) == tq.TQ_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        tq.make_rope(None, 1, 128, sections=[])
    with pytest.raises(ValueError):
        tq.make_rope(None, 1, 128, sections=[1] * 5)
