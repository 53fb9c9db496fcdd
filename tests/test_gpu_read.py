"""Reading the 2-4-bit and the 8-bit caches back into rows, against the formulas in 64 bits.

Bounds per element of the 2-4-bit cache, x = sum_k P_k y_k with y_k = norm/sqrt(d) c (and the signs' terms, P the rotation or
the projections), against the root of the sum of the terms' squares, which is the size of a sum of random signs:
  - fp32 rows: 2^-22 of it, counted eight times: each factor's rounding (2^-24 three times a term, independent) and those
    of the sums, at most 32 terms at a time (2^-24 of running sizes below half of it, 256 of them, then 8 of the whole);
  - bf16 rows may be formed from the tables in fp16: 2^-11 of each factor, independent, counted eight times;
  - half a step of the rows' type.
The 8-bit cache is exact.
"""

import math

import numpy as np
import pytest

import oracle
from oracle import kv8

from .gpu_common import DEV, to_dev, torch, tq

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, tq.TQ_BF16), "f32": (torch.float32, tq.TQ_F32)}


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


class Pool:
    """Caches of random records: any bits are codes and signs, norms in the usual range; on both sides."""

    def __init__(self, rng, ctx, p, h, pages, batch, maxp):
        self.p, self.h, self.pages, self.maxp = p, h, pages, maxp
        self.bytes, self.dev = {}, {}
        for kind, page_bytes in zip("kv", tq.tq_cache_layout(ctx, h)):
            blk = rng.integers(0, 256, (pages * h, page_bytes // h), dtype=np.uint8)
            cb = oracle.turboquant.code_bytes(p, kind)
            at = 16 * (cb + (p.m // 8 if kind == "k" and p.k_qjl else 0))
            norm = rng.uniform(5, 30, (pages * h, 16)).astype(np.float16)
            norm[rng.random(norm.shape) < 0.02] = 0
            blk[:, at:at + 32] = norm.view(np.uint8)
            if kind == "k" and p.k_qjl:
                blk[:, at + 32:at + 64] = rng.uniform(0, 9, (pages * h, 16)).astype(np.float16).view(np.uint8)
            self.bytes[kind] = blk.reshape(-1)
            self.dev[kind] = to_dev(self.bytes[kind])
        self.table = rng.permutation(pages)[:batch * maxp].reshape(batch, maxp).astype(np.int32)

    def values(self, kind, b, positions):
        """[n][h][d] in fp64 and the sum of squares behind each element's bounds."""
        p, pos = self.p, np.repeat(np.asarray(positions), self.h)
        rec = oracle.turboquant.read_paged(p, kind, self.bytes[kind], self.table[b, pos // 16], pos % 16, np.tile(np.arange(self.h), len(positions)), self.h)
        unpack = oracle.turboquant.unpack_k_records if kind == "k" else oracle.turboquant.unpack_v_records
        r = unpack(p, rec)
        table = oracle.turboquant._centroid_table(p, kind)
        c = np.stack([table[j].centroids[r["codes"][:, j]] for j in range(p.d)], axis=1)
        y = c * r["n16"][:, None] / math.sqrt(p.d)
        x, size = y @ p.Pi, (y ** 2) @ (p.Pi ** 2)
        if kind == "k" and p.k_qjl:
            w = (2.0 * r["signs"] - 1.0) * (math.sqrt(math.pi / 2) / p.m) * r["rho16"][:, None]
            sp = p.S @ p.Pi
            x, size = x + w @ sp, size + (w ** 2) @ (sp ** 2)
        return x.reshape(len(positions), self.h, p.d), np.sqrt(size).reshape(len(positions), self.h, p.d)


def config(d, k_bits, v_bits, m=128, split=None, qjl=True, seed=3):
    split = d // 64 * 32 if split is None else split
    cfg = tq.make_config(k_bits=k_bits, v_bits=v_bits, m=m, seed=seed, k_split=split, v_split=split, k_qjl=qjl, d=d)
    p = oracle.turboquant.make_params(d=d, m=m, k_bits=k_bits, k_split=split, v_bits=v_bits, v_split=split, k_qjl=qjl, seed=seed)
    return tq.tq_create_ex(cfg), p


def read(ctx, pool, dtype, starts, lens, gap=0, strides=(0, 0), kinds="kv", flags=0, max_len=None, first=None, total=None):
    dt, code = DT[dtype]
    h, d = pool.h, pool.p.d
    first = np.cumsum([0] + [n + gap for n in lens])[:-1].tolist() if first is None else first
    total = int(max([f + n for f, n in zip(first, lens)] + [0])) + 5 if total is None else total
    out = {k: torch.full((total + 3, (s or h * d)), -7.0, dtype=dt, device=DEV) for k, s in zip("kv", strides)}
    tq.tq_dequantize(ctx, pool.dev["k"], pool.dev["v"], code, len(lens), h, ints(starts), ints(lens), max(lens) if max_len is None else max_len,
                     to_dev(pool.table), pool.maxp, pool.pages, out["k"] if "k" in kinds else None, out["v"] if "v" in kinds else None,
                     ints(first), total, k_stride=strides[0], v_stride=strides[1], stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == flags
    return out, first


def check(pool, dtype, out, starts, lens, first, kinds="kv"):
    dt = DT[dtype][0]
    h, d = pool.h, pool.p.d
    for kind in "kv":
        got = out[kind].double().cpu().numpy()
        seen = np.zeros(got.shape, bool)
        for b, (s, n, f) in enumerate(zip(starts, lens, first)):
            if n == 0 or kind not in kinds:
                continue
            want, size = pool.values(kind, b, range(s, s + n))
            tol = size * (8 * 2.0 ** -22 if dtype == "f32" else 8 * 2.0 ** -11 * math.sqrt(2)) + torch.finfo(dt).eps / 2 * np.abs(want) * 1.01
            x = got[f:f + n, :h * d].reshape(n, h, d)
            worst = float((np.abs(x - want) / (tol + 1e-30)).max())
            assert worst <= 1.0, (kind, b, worst)
            seen[f:f + n, :h * d] = True
        assert np.all(got[~seen] == -7.0), kind


BITS = [((4, 3), (4, 3)), ((3, 3), (3, 3)), ((3, 2), (3, 2)), ((4, 4), (4, 4)), ((2, 2), (2, 2)), ((4, 4), (2, 2)), ((1, 1), (1, 4)), ((2, 3), (1, 2))]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k_bits,v_bits", BITS)
def test_bit_widths(dtype, k_bits, v_bits):
    ctx, p = config(128, k_bits, v_bits)
    pool = Pool(np.random.default_rng(0), ctx, p, 3, 40, 3, 9)
    starts, lens = [0, 37, 5], [70, 1, 100]
    out, first = read(ctx, pool, dtype, starts, lens, gap=2)
    check(pool, dtype, out, starts, lens, first)
    tq.tq_destroy(ctx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,m,split,qjl", [(32, 32, 0, True), (64, 128, 32, True), (96, 64, 32, True), (128, 64, 64, True), (128, 128, 96, True),
                                           (128, 128, 64, False), (160, 96, 64, True), (256, 128, 128, True), (128, 32, 0, True)])
def test_head_dimensions_projections_and_splits(dtype, d, m, split, qjl):
    ctx, p = config(d, (4, 3), (3, 2), m=m, split=split, qjl=qjl)
    pool = Pool(np.random.default_rng(1), ctx, p, 2, 20, 2, 8)
    starts, lens = [3, 16], [33, 48]
    out, first = read(ctx, pool, dtype, starts, lens)
    check(pool, dtype, out, starts, lens, first)
    tq.tq_destroy(ctx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h", [1, 5, 8, 16])
def test_heads_lengths_and_rows(dtype, h):
    """From nothing to many pages, runs that start and end inside one, rows in another order than the sequences."""
    ctx, p = config(128, (4, 3), (4, 3))
    pool = Pool(np.random.default_rng(2), ctx, p, h, 200, 9, 20)
    starts, lens = [0, 15, 16, 17, 31, 300, 2, 7, 0], [0, 1, 16, 15, 2, 20, 14, 250, 320]
    first = [0, 900, 10, 30, 50, 60, 100, 400, 1000]
    out, first = read(ctx, pool, dtype, starts, lens, first=first)
    check(pool, dtype, out, starts, lens, first)
    tq.tq_destroy(ctx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_one_of_both(dtype):
    ctx, p = config(128, (3, 3), (3, 3))
    pool = Pool(np.random.default_rng(3), ctx, p, 2, 20, 2, 5)
    starts, lens = [9, 0], [40, 80]
    for strides, kinds in (((2 * 128 + 8, 3 * 128), "kv"), ((0, 512), "v"), ((256, 0), "k")):
        out, first = read(ctx, pool, dtype, starts, lens, strides=strides, kinds=kinds)
        check(pool, dtype, out, starts, lens, first, kinds)
    tq.tq_destroy(ctx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_is_out_of_range_is_skipped_and_flagged(dtype):
    ctx, p = config(128, (4, 3), (4, 3))
    rng = np.random.default_rng(4)
    pool = Pool(rng, ctx, p, 2, 20, 3, 5)
    keep = pool.table.copy()
    pool.table[0, 1], pool.table[1, 0] = 20, -1
    out, first = read(ctx, pool, dtype, [0, 0, 0], [40, 20, 16], flags=1)
    pool.table = keep
    for kind in "kv":                             # the other pages' tokens are there
        left = (out[kind] == -7).all(1).tolist()
        assert left == [16 <= r < 32 or 40 <= r < 56 or r >= 76 for r in range(len(left))]
    out, first = read(ctx, pool, dtype, [70, 80, 1 << 30], [20, 5, 5], flags=2)          # the table holds 80 positions
    check(pool, dtype, out, [70, 0, 0], [10, 0, 0], [0, 20, 25])
    out, first = read(ctx, pool, dtype, [0, 0, 0], [20, 30, 7], flags=4, max_len=25)     # cut to max_len
    check(pool, dtype, out, [0, 0, 0], [20, 25, 7], first)
    out, first = read(ctx, pool, dtype, [-1, 0, 0], [20, -30, 7], flags=4, max_len=30, first=[0, 20, 30], total=40)
    check(pool, dtype, out, [0, 0, 0], [0, 0, 7], first)
    out, first = read(ctx, pool, dtype, [0, 0, 0], [20, 30, 7], flags=4, first=[0, 20, 60], total=45)     # rows that are not there
    check(pool, dtype, out, [0, 0, 0], [20, 25, 0], first)
    out, first = read(ctx, pool, dtype, [0, 0, 0], [20, 30, 7], flags=4, first=[0, -3, 2 ** 31 - 5], total=45)
    check(pool, dtype, out, [0, 0, 0], [20, 0, 0], first)
    tq.tq_destroy(ctx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch", [511, 512, 513, 1500])
def test_many_sequences(dtype, batch):
    """As many as the list of pages holds, and more."""
    ctx, p = config(128, (4, 3), (3, 3))
    rng = np.random.default_rng(8)
    pool = Pool(rng, ctx, p, 2, 2 * batch + 3, batch, 2)
    lens = rng.integers(0, 18, batch)
    lens[rng.random(batch) < 0.2] = 0
    lens[-1] = 9
    starts = rng.integers(0, 32 - lens + 1).tolist()
    out, first = read(ctx, pool, dtype, starts, lens.tolist())
    check(pool, dtype, out, starts, lens.tolist(), first)
    tq.tq_destroy(ctx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed(dtype):
    """Two reads in graphs, replayed at once on two streams as starts and lengths change."""
    ctx, p = config(128, (4, 3), (4, 3))
    pool = Pool(np.random.default_rng(9), ctx, p, 2, 40, 3, 10)
    dt, code = DT[dtype]
    starts, lens, first = ints([0, 0, 0]), ints([1, 1, 1]), ints([0, 160, 320])
    table = to_dev(pool.table)
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for _ in range(2):
        out = {k: torch.empty(480, 2 * 128, dtype=dt, device=DEV) for k in "kv"}
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tq.tq_dequantize(ctx, pool.dev["k"], pool.dev["v"], code, 3, 2, starts, lens, 160, table, pool.maxp, pool.pages, out["k"], out["v"],
                             first, 480, stream=torch.cuda.current_stream())
        outs.append(out)
        graphs.append(g)
    for s, n in (([0, 5, 30], [160, 20, 1]), ([100, 0, 3], [0, 33, 150]), ([15, 16, 17], [17, 16, 15])):
        starts.copy_(ints(s))
        lens.copy_(ints(n))
        for out in outs:
            for x in out.values():
                x.fill_(-7)
        torch.cuda.synchronize()
        for _ in range(3):
            for g, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    g.replay()
        torch.cuda.synchronize()
        assert tq.tq_check_device_status(ctx) == 0
        for out in outs:
            check(pool, dtype, out, s, n, [0, 160, 320])
    tq.tq_destroy(ctx)


@pytest.mark.parametrize("d,bits", [(128, (4, 3)), (64, (3, 3))])
def test_scores_of_rows_that_were_read_are_the_decodes(d, bits):
    """Quantize, read back, and attend over the rows: the decode's results."""
    ctx, p = config(d, bits, bits)
    rng = np.random.default_rng(5)
    b, h, hq, L = 2, 2, 8, 203
    maxp = (L + 15) // 16
    table = to_dev(rng.permutation(b * maxp).reshape(b, maxp).astype(np.int32))
    kpb, vpb = tq.tq_cache_layout(ctx, h)
    kc, vc = (torch.zeros(b * maxp * x, dtype=torch.uint8, device=DEV) for x in (kpb, vpb))
    k, v, q = (torch.randn(*s, device=DEV) for s in ((b, L, h, d), (b, L, h, d), (b, hq, d)))
    tq.tq_quantize(ctx, k, v, tq.TQ_F32, b, L, h, ints([0] * b), table, maxp, b * maxp, kc, vc)
    n = tq.tq_workspace_size(ctx, b, hq, L, 0)
    ws, out = torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty(b, hq, d, device=DEV)
    lens = ints([L] * b)
    tq.tq_decode_attention(ctx, q, tq.TQ_F32, b, hq, h, lens, L, table, maxp, b * maxp, kc, vc, 0, d ** -0.5, out, ws, n)
    kr, vr = (torch.empty(b * L, h, d, device=DEV) for _ in range(2))
    tq.tq_dequantize(ctx, kc, vc, tq.TQ_F32, b, h, ints([0] * b), lens, L, table, maxp, b * maxp, kr, vr, ints(range(0, b * L, L)), b * L)
    n2 = tq.tq_prompt_workspace_size(ctx, b, 1, hq, h, L)
    ws2, got = torch.empty(n2, dtype=torch.uint8, device=DEV), torch.empty_like(q)
    tq.tq_prompt_attention(ctx, q, kr, vr, tq.TQ_F32, b, ints([0, 1, 2]), ints([0, L, 2 * L]), b, b * L, 1, L, hq, h, 0, 0, d ** -0.5, got, ws2, n2)
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == 0
    err = ((got - out).abs().amax(-1) / got.abs().amax(-1)).max()
    assert float(err) <= 2e-3                     # the decode's own bar
    # and the stored records are near what was stored: 3 bits and more keep the values within their codebook's distortion
    assert float((vr.view(b, L, h, d) - v).pow(2).mean() / v.pow(2).mean()) < (0.03 if bits == (4, 3) else 0.05)
    tq.tq_destroy(ctx)


@pytest.mark.parametrize("d,m,k_bits,v_bits,qjl", [(128, 128, (4, 3), (4, 3), True), (128, 128, (3, 3), (2, 2), True), (128, 128, (4, 4), (1, 1), False),
                                                   (64, 64, (4, 3), (3, 2), True), (128, 64, (4, 3), (4, 3), True), (256, 128, (3, 3), (4, 3), True)])
def test_bf16_rows_within_the_stated_bounds(d, m, k_bits, v_bits, qjl):
    """2^-8 of the root of the terms' squares and 2^-8 of the element where fp16 tables form them (d = m = 128), elsewhere the
    fp32 rows' bound and half a step of bf16."""
    ctx, p = config(d, k_bits, v_bits, m=m, qjl=qjl)
    pool = Pool(np.random.default_rng(14), ctx, p, 3, 60, 2, 30)
    lens, h = [470, 333], 3
    out, first = read(ctx, pool, "bf16", [0, 5], lens)
    for kind in "kv":
        got = out[kind].double().cpu().numpy()
        for b, (s, n, f) in enumerate(zip([0, 5], lens, first)):
            want, root = pool.values(kind, b, range(s, s + n))
            over = (np.abs(got[f:f + n].reshape(n, h, d) - want)) / (root * (2.0 ** -8 if d == m == 128 else 2.0 ** -19) + 2.0 ** -8 * np.abs(want) + 1e-30)
            assert float(over.max()) <= 1.0, (kind, float(over.max()))
    tq.tq_destroy(ctx)


@pytest.mark.parametrize("k_bits,v_bits,split", [((3, 3), (2, 2), 0), ((4, 3), (3, 2), 64), ((4, 4), (1, 1), 64)])
def test_fp32_rows_within_the_stated_bounds(k_bits, v_bits, split):
    """Half a million elements, some of them several times the root of their terms' squares: 2^-19 of that root, and 2^-20 of the
    element for the tensor cores' cut sums."""
    ctx, p = config(128, k_bits, v_bits, split=split)
    pool = Pool(np.random.default_rng(5), ctx, p, 8, 42, 2, 20)
    out, first = read(ctx, pool, "f32", [0, 0], [320, 320])
    most = 0.0
    for kind in "kv":
        got = out[kind].double().cpu().numpy()
        for b in range(2):
            want, root = pool.values(kind, b, range(320))
            most = max(most, float((np.abs(want) / (root + 1e-30)).max()))
            tol = root * 2.0 ** -19 + np.abs(want) * (2.0 ** -20 + 2.0 ** -24)
            assert np.all(np.abs(got[first[b]:first[b] + 320].reshape(want.shape) - want) <= tol), kind
    assert most > 3.5
    tq.tq_destroy(ctx)


# ---------------------------------------------------------------------------
# the 8-bit cache
# ---------------------------------------------------------------------------
def _kv8(rng, d, h, pages, batch, maxp):
    codes = {k: rng.integers(0, 256, (pages, h, 16, d)).astype(np.uint8) for k in "kv"}
    for c in codes.values():
        c[(c & 127) == 127] = 0
    scales = {k: np.exp2(rng.integers(-100, 120, (pages, h))).astype(np.float32) for k in "kv"}
    table = rng.permutation(pages)[:batch * maxp].reshape(batch, maxp).astype(np.int32)
    dev = [to_dev(x) for x in (codes["k"], codes["v"], scales["k"], scales["v"], table)]
    return codes, scales, table, tq.make_kv8_cache(*dev, maxp, pages, h)


def _kv8_read(ctx, cache, dtype, h, d, starts, lens, first, total, max_len, strides=(0, 0), kinds="kv", flags=0):
    dt, code = DT[dtype]
    out = {k: torch.full((total + 3, (s or h * d)), -7.0, dtype=dt, device=DEV) for k, s in zip("kv", strides)}
    tq.tq_kv8_dequantize(ctx, cache, code, len(lens), ints(starts), ints(lens), max_len, out["k"] if "k" in kinds else None,
                         out["v"] if "v" in kinds else None, ints(first), total, k_stride=strides[0], v_stride=strides[1],
                         stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == flags
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,h,strides,kinds", [(64, 3, (0, 0), "kv"), (128, 8, (0, 0), "kv"), (256, 2, (0, 0), "kv"), (128, 1, (136, 384), "kv"),
                                               (64, 5, (0, 320), "v"), (128, 2, (256, 0), "k")])
def test_kv8_values_are_exact(dtype, d, h, strides, kinds):
    rng = np.random.default_rng(6)
    ctx = tq.tq_create(d, 3, 128, 0)
    codes, scales, table, cache = _kv8(rng, d, h, 70, 6, 11)
    starts, lens, first = [0, 15, 16, 33, 5, 9], [0, 1, 16, 30, 160, 25], [0, 300, 400, 30, 100, 0]
    out = _kv8_read(ctx, cache, dtype, h, d, starts, lens, first, 420, 170, strides, kinds)
    for kind in "kv":
        got = out[kind].double().cpu().numpy()
        seen = np.zeros(got.shape, bool)
        for b, (s, n, f) in enumerate(zip(starts, lens, first)):
            if kind not in kinds:
                continue
            pos = np.arange(s, s + n)
            x = kv8.VALUES[codes[kind][table[b, pos // 16], :, pos % 16]] * scales[kind][table[b, pos // 16]].astype(np.float64)[..., None]
            assert np.array_equal(got[f:f + n, :h * d].reshape(n, h, d), x)
            seen[f:f + n, :h * d] = True
        assert np.all(got[~seen] == -7.0)
    tq.tq_destroy(ctx)


def test_kv8_what_is_out_of_range_is_skipped_and_flagged():
    rng = np.random.default_rng(7)
    d, h = 128, 2
    ctx = tq.tq_create(d, 3, 128, 0)
    codes, scales, table, cache = _kv8(rng, d, h, 20, 2, 4)
    run = lambda *a, **kw: _kv8_read(ctx, cache, "f32", h, d, *a, **kw)  # noqa: E731
    full = run([0, 0], [64, 64], [0, 64], 128, 64)
    out = run([60, 64], [9, 1], [0, 9], 10, 9, flags=2)
    assert torch.equal(out["k"][:4], full["k"][60:64]) and bool((out["k"][4:] == -7).all())
    out = run([0, -1], [64, 3], [0, 70], 50, 30, flags=4)
    assert torch.equal(out["v"][:30], full["v"][:30]) and bool((out["v"][30:] == -7).all())
    cache.buffers[4][1, 2] = 20
    out = run([0, 30], [5, 20], [0, 5], 25, 20, flags=1)
    assert torch.equal(out["v"][:7], torch.cat([full["v"][:5], full["v"][94:96]]))
    assert bool((out["v"][7:23] == -7).all()) and torch.equal(out["v"][23:25], full["v"][112:114])
    tq.tq_destroy(ctx)


@pytest.mark.parametrize("eight", [False, True])
def test_a_length_of_zero_reads_nothing_wherever_it_starts(eight):
    """(A negative start is flagged all the same.)"""
    rng = np.random.default_rng(10)
    for starts, flags in (([1 << 20, 3], 0), ([81, 3], 0), ([2 ** 31 - 1, 3], 0), ([-1, 3], 4)):
        if eight:
            ctx = tq.tq_create(128, 3, 128, 0)
            cache = _kv8(rng, 128, 2, 20, 2, 5)[3]
            out = _kv8_read(ctx, cache, "f32", 2, 128, starts, [0, 5], [0, 0], 5, 5, flags=flags)
            assert not bool((out["k"][:5] == -7).any()) and bool((out["k"][5:] == -7).all())
        else:
            ctx, p = config(128, (4, 3), (4, 3))
            pool = Pool(rng, ctx, p, 2, 20, 2, 5)
            out, first = read(ctx, pool, "f32", starts, [0, 5], flags=flags)
            check(pool, "f32", out, starts, [0, 5], first)
        tq.tq_destroy(ctx)


def test_reads_beyond_32_bit_offsets():
    """Pages and rows whose elements lie beyond 2^31."""
    d, h, pages = 128, 8, (1 << 17) + 999
    ctx = tq.tq_create(d, 3, 128, 0)
    codes = torch.zeros(pages, h, 16, d, dtype=torch.uint8, device=DEV)
    scale = torch.ones(pages, h, device=DEV)
    codes[-1] = torch.randint(0, 120, (h, 16, d), device=DEV, dtype=torch.uint8)
    rows = (1 << 21) + 999
    out = torch.zeros(rows, h * d, dtype=torch.bfloat16, device=DEV)
    cache = tq.make_kv8_cache(codes, codes, scale, scale, ints([pages - 1]), 1, pages, h)
    tq.tq_kv8_dequantize(ctx, cache, tq.TQ_BF16, 1, ints([0]), ints([16]), 16, out, None, ints([rows - 16]), rows)
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == 0
    want = codes[-1].view(torch.float8_e4m3fn).float().transpose(0, 1).reshape(16, h * d).bfloat16()
    assert torch.equal(out[-16:], want) and not bool(out[:-16].any())
    tq.tq_destroy(ctx)
