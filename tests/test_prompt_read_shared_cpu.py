"""Refusals of the calls around the caches (packed prompts, reading back, shared prefixes), without a GPU.

A context cannot be made here, so the refusals are asked of a zeroed block of memory that starts with a configuration, as
a context does; a call that passes every check ends at the missing device."""

import ctypes

import pytest
import torch

tq = pytest.importorskip("online_kv_cache_02_gb300.tq")

BIG = 1 << 40


class Fake:
    def __init__(self, d=128):
        self.mem = ctypes.create_string_buffer(1 << 16)
        ctypes.memmove(self.mem, ctypes.byref(tq.make_config(d=d)), ctypes.sizeof(tq.TQConfig))
        self.ctx = ctypes.addressof(self.mem)
        self.buf = 1 << 20                          # aligned addresses; nothing may read them
        self.far = 1 << 44
        self.cache = tq.make_kv8_cache(self.buf, self.buf, self.buf, self.buf, self.buf, 8, 100, 4)


@pytest.fixture
def f():
    if torch.cuda.is_available():
        pytest.skip("the addresses here are not device memory: a call that is not refused must not be made")
    return Fake()


def prompt(f, **kw):
    a = dict(ctx=f.ctx, q=f.buf, k=f.buf, v=f.buf, dtype=0, seqs=2, cu_q=f.buf, cu_k=f.buf, tq=10, tk=20, mq=9, mk=20, hq=8, h=4, window=0,
             sinks=0, scale=0.1, out=f.far, ws=f.buf, size=BIG, qs=0, ks=0, vs=0)
    a.update(kw)
    return tq.raw_status("tq_prompt_attention", a["ctx"], a["q"], a["k"], a["v"], a["dtype"], a["seqs"], a["cu_q"], a["cu_k"], a["tq"],
                         a["tk"], a["mq"], a["mk"], a["hq"], a["h"], a["window"], a["sinks"], ctypes.c_float(a["scale"]), a["out"],
                         a["ws"], a["size"], a["qs"], a["ks"], a["vs"], None)


def test_prompt_attention(f):
    ok, bad, uns = tq.TQ_ERR_CUDA, tq.TQ_ERR_INVALID_ARG, tq.TQ_ERR_UNSUPPORTED
    assert prompt(f) == ok
    assert prompt(f, dtype=1, qs=8 * 128 + 4, ks=4 * 128 + 4) == ok
    for kw in (dict(ctx=None), dict(q=None), dict(k=None), dict(v=None), dict(cu_q=None), dict(cu_k=None), dict(out=None), dict(ws=None),
               dict(dtype=2), dict(seqs=-1), dict(tq=-1), dict(tk=-1), dict(mq=-1), dict(mk=-1), dict(hq=0), dict(h=0), dict(hq=6),
               dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(qs=8 * 128 - 8),
               dict(ks=4 * 128 - 8), dict(vs=-8), dict(qs=8 * 128 + 4), dict(dtype=1, vs=4 * 128 + 2)):
        assert prompt(f, **kw) == bad, kw
    for name in ("q", "k", "v", "ws"):
        assert prompt(f, **{name: f.buf + 8}) == bad
    for name in ("cu_q", "cu_k"):
        assert prompt(f, **{name: f.buf + 2}) == bad
    assert prompt(f, out=f.far + 8) == bad
    assert prompt(f, size=15) == tq.TQ_ERR_WORKSPACE
    # nothing to do
    assert prompt(f, seqs=0, q=None) == tq.TQ_OK and prompt(f, tq=0, q=None) == tq.TQ_OK and prompt(f, mq=0) == tq.TQ_OK
    assert prompt(f, tk=0, k=None, v=None) == ok
    # what 32 bits do not hold
    assert prompt(f, tq=1 << 28) == uns and prompt(f, tk=(1 << 30) + 1) == uns and prompt(f, mk=(1 << 29) + 1) == uns
    assert prompt(f, tq=1 << 27, hq=8) == ok
    # results where inputs are read
    row = 8 * 128 * 2
    assert prompt(f, out=f.buf) == bad and prompt(f, q=f.far + 9 * row) == bad and prompt(f, q=f.far + 10 * row) == ok
    assert prompt(f, k=f.far - 20 * 1024 + 16) == bad and prompt(f, k=f.far - 20 * 1024) == ok
    assert prompt(f, v=f.far - 19 * 2048 - 1024, vs=1024) == ok and prompt(f, v=f.far - 19 * 2048 - 1008, vs=1024) == bad


def test_prompt_workspace(f):
    n = ctypes.c_size_t()
    ask = lambda *a: tq.raw_status("tq_prompt_workspace_size", f.ctx, *a, ctypes.byref(n))  # noqa: E731
    assert ask(3, 100, 8, 4, 1000) == tq.TQ_OK and n.value > 0
    least = n.value
    assert ask(300, 10000, 64, 4, 100000) == tq.TQ_OK and n.value >= least
    for a in ((-1, 1, 8, 4, 1), (1, -1, 8, 4, 1), (1, 1, 0, 4, 1), (1, 1, 6, 4, 1), (1, 1, 8, 0, 1), (1, 1, 8, 4, -1)):
        assert ask(*a) == tq.TQ_ERR_INVALID_ARG
    assert tq.raw_status("tq_prompt_workspace_size", f.ctx, 1, 1, 8, 4, 1, None) == tq.TQ_ERR_INVALID_ARG
    assert tq.raw_status("tq_prompt_workspace_size", None, 1, 1, 8, 4, 1, ctypes.byref(n)) == tq.TQ_ERR_INVALID_ARG


def read(f, eight, **kw):
    a = dict(ctx=f.ctx, cache=f.cache, kc=f.buf, vc=f.buf, dtype=0, batch=2, h=4, start=f.buf, lens=f.buf, max_len=20, bt=f.buf, maxp=8,
             pages=100, k=f.buf, v=f.buf, first=f.buf, rows=50, ks=0, vs=0)
    a.update(kw)
    if eight:
        return tq.raw_status("tq_kv8_dequantize", a["ctx"], a["cache"], a["dtype"], a["batch"], a["start"], a["lens"], a["max_len"], a["k"],
                             a["v"], a["first"], a["rows"], a["ks"], a["vs"], None)
    return tq.raw_status("tq_dequantize", a["ctx"], a["kc"], a["vc"], a["dtype"], a["batch"], a["h"], a["start"], a["lens"], a["max_len"],
                         a["bt"], a["maxp"], a["pages"], a["k"], a["v"], a["first"], a["rows"], a["ks"], a["vs"], None)


@pytest.mark.parametrize("eight", [False, True])
def test_reading_back(f, eight):
    ok, bad, uns = tq.TQ_ERR_CUDA, tq.TQ_ERR_INVALID_ARG, tq.TQ_ERR_UNSUPPORTED
    assert read(f, eight) == ok and read(f, eight, k=None) == ok and read(f, eight, v=None, ks=520) == ok
    for kw in (dict(ctx=None), dict(k=None, v=None), dict(dtype=-1), dict(batch=-1), dict(max_len=-1), dict(rows=-1), dict(start=None),
               dict(lens=None), dict(first=None), dict(ks=504), dict(vs=516), dict(dtype=1, vs=514), dict(k=f.buf + 8), dict(v=f.buf + 4),
               dict(start=f.buf + 1), dict(lens=f.buf + 2), dict(first=f.buf + 2)):
        assert read(f, eight, **kw) == bad, kw
    assert read(f, eight, batch=0, start=None) == tq.TQ_OK and read(f, eight, max_len=0, lens=None) == tq.TQ_OK and read(f, eight, rows=0) == tq.TQ_OK
    if eight:
        c = tq.make_kv8_cache(f.buf, None, f.buf, None, f.buf, 8, 100, 4)
        assert read(f, True, cache=c) == bad and read(f, True, cache=c, v=None) == ok
        assert read(f, True, cache=None) == bad and read(f, True, ctx=Fake(96).ctx) == uns
    else:
        assert read(f, False, kc=None) == bad and read(f, False, kc=None, k=None) == ok and read(f, False, vc=f.buf + 8) == bad
        for kw in (dict(h=0), dict(bt=None), dict(bt=f.buf + 2), dict(maxp=0), dict(pages=0)):
            assert read(f, False, **kw) == bad, kw
        assert read(f, False, h=1 << 16) == uns and read(f, False, maxp=(1 << 26) + 1) == uns and read(f, False, pages=1 << 30) == uns


def shared(f, **kw):
    a = dict(ctx=f.ctx, cache=f.cache, q=f.buf, dtype=0, batch=6, hq=8, lens=f.buf, max_len=100, groups=2, start=f.buf, prefix=f.buf, most=4,
             scale=0.1, out=f.buf, ws=f.buf, size=BIG)
    a.update(kw)
    return tq.raw_status("tq_kv8_shared_decode_attention", a["ctx"], a["cache"], a["q"], a["dtype"], a["batch"], a["hq"], a["lens"],
                         a["max_len"], a["groups"], a["start"], a["prefix"], a["most"], ctypes.c_float(a["scale"]), a["out"], a["ws"],
                         a["size"], None)


def test_shared_prefixes(f):
    ok, bad, uns = tq.TQ_ERR_CUDA, tq.TQ_ERR_INVALID_ARG, tq.TQ_ERR_UNSUPPORTED
    assert shared(f) == ok and shared(f, dtype=1) == ok
    for kw in (dict(ctx=None), dict(cache=None), dict(q=None), dict(lens=None), dict(out=None), dict(ws=None), dict(start=None),
               dict(prefix=None), dict(dtype=2), dict(batch=-1), dict(hq=0), dict(hq=6), dict(max_len=-1), dict(groups=0), dict(most=0),
               dict(scale=float("nan")), dict(q=f.buf + 8), dict(out=f.buf + 8), dict(ws=f.buf + 8), dict(lens=f.buf + 2),
               dict(start=f.buf + 2), dict(prefix=f.buf + 1)):
        assert shared(f, **kw) == bad, kw
    assert shared(f, batch=0, q=None) == tq.TQ_OK
    assert shared(f, ctx=Fake(96).ctx) == uns
    assert shared(f, batch=1 << 27) == uns and shared(f, groups=1 << 20, most=1 << 10) == uns and shared(f, max_len=(1 << 29) + 1) == uns
    n = ctypes.c_size_t()
    ask = lambda *a: tq.raw_status("tq_kv8_shared_workspace_size", f.ctx, *a, ctypes.byref(n))  # noqa: E731
    assert ask(6, 8, 4, 2, 4, 100) == tq.TQ_OK
    need = n.value
    assert shared(f, size=need) == ok and shared(f, size=need - 1) == tq.TQ_ERR_WORKSPACE
    for a in ((-1, 8, 4, 2, 4, 100), (6, 0, 4, 2, 4, 100), (6, 6, 4, 2, 4, 100), (6, 8, 4, 0, 4, 100), (6, 8, 4, 2, 0, 100), (6, 8, 4, 2, 4, -1)):
        assert ask(*a) == bad
    assert ask(6, 8, 4, 1 << 20, 1 << 10, 100) == uns


@pytest.mark.parametrize("d", [64, 128, 256])
def test_shared_workspace_never_falls(d):
    f = Fake(d)
    n = ctypes.c_size_t()

    def ask(batch, hq, h, groups, most, max_len):
        assert tq.raw_status("tq_kv8_shared_workspace_size", f.ctx, batch, hq, h, groups, most, max_len, ctypes.byref(n)) == tq.TQ_OK
        return n.value
    base = [12, 8, 2, 2, 6, 1000]
    for i, steps in ((0, (1, 5, 13, 100)), (1, (2, 4, 6, 8, 10, 18, 32, 34, 66)), (3, (1, 2, 3, 9, 40)), (4, (1, 2, 3, 4, 5, 8, 9, 17, 33, 65, 200)),
                     (5, (0, 1, 16, 100, 5000, 100000))):
        sizes = []
        for x in steps:
            a = list(base)
            a[i] = x
            sizes.append(ask(*a))
        assert sizes == sorted(sizes), (i, sizes)
