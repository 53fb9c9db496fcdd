"""The 8-bit cache at the ends of what its header allows: rows that fill no warp, sizes of values that meet the ends of
fp32 and of the weights' types, non-finite inputs, calls in place and on several streams.

Bounds as in test_gpu_kv8; what a test adds to them stands beside it."""

import numpy as np
import pytest

from oracle import kv8

from .gpu_common import DEV, to_dev, torch, tq
from .test_gpu_kv8 import DT, Cache, _append_case, _attend, _bound, _causal_case, _check, _decode_case, ctx_for, values

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


# ---------------------------------------------------------------------------
# sizes of values
# ---------------------------------------------------------------------------
# (dtype, d, query heads of the one KV head): mma.sync in both types, tcgen05 with the halves in turn and with both halves' rows
FORMS = [("bf16", 128, 4), ("f32", 128, 4), ("f32", 64, 11), ("bf16", 64, 20), ("bf16", 128, 20), ("bf16", 256, 20),
         ("bf16", 64, 150), ("bf16", 128, 150), ("bf16", 256, 150)]


def _one_head(rng, d, n, pages=None, maxp=None):
    pages = pages or (n + 15) // 16 + 1
    c = Cache(rng, pages, 1, d, 1, maxp or pages)
    c.clean(rng, 0, range(n))
    return c


def _tails(c, x, p, scale):
    """Per row, what weights below the normal numbers of fp16 add to a bound: half a step of the subnormals is 2^-25, and
    the largest weight 2^3 at least (tcgen05; 2^8 on mma.sync), so each key's weight is off by 2^-28 of the largest
    weight times its code."""
    j = np.arange(p + 1)
    pg, sl = c.table[0][j // 16], j % 16
    k = kv8.VALUES[c.codes["k"][pg, 0, sl]] * c.scales["k"][pg, 0].astype(np.float64)[:, None]
    vc, vs = kv8.VALUES[c.codes["v"][pg, 0, sl]], c.scales["v"][pg, 0].astype(np.float64)
    out = []
    for row in x.astype(np.float64):
        s = (k @ row) * scale
        w = np.exp(s - s.max())
        out.append(2.0 ** -28 * (w / w.sum() * vs).max() * np.abs(vc).sum(axis=0))
    return np.stack(out)


def _check_one(c, got, x, dtype, p, two_parts=None):
    scale = 1.0 / np.sqrt(c.d)
    want, mag, dots, ksum, n = kv8.attention(x, c.codes["k"], c.scales["k"], c.codes["v"], c.scales["v"], c.table[0], p, 0, 0, scale)
    two_parts = dtype == "bf16" and len(x) > 16 if two_parts is None else two_parts
    parts = 2.0 ** -17 * np.abs(x).max(axis=-1) * ksum if two_parts else 0.0
    tol = _bound(dtype, want, mag, dots, n, c.d, scale, parts) + _tails(c, x, p, scale)
    err = np.abs(got - want)
    assert np.all(err <= tol), (float(np.nanmax(err / tol)), int(np.isnan(got).sum()), np.argwhere(~(err <= tol))[:4].tolist())


@pytest.mark.parametrize("dtype,d,g", FORMS)
@pytest.mark.parametrize("n", [100, 310, 5000])
def test_value_scales_far_apart(dtype, d, g, n):
    """Value scales 2^-50 to 2^49, queries from 2^-100 to 2^20 and zero: each half of an item and each part of a split one
    has a maximum of its own."""
    rng = np.random.default_rng(70)
    c = _one_head(rng, d, n)
    c.scales["v"][:] = np.exp2(rng.integers(-50, 50, c.scales["v"].shape))
    c.scales["k"][:] = np.exp2(rng.integers(-40, -6, c.scales["k"].shape))
    c.to_device()
    q = values(rng, dtype, 1, g, d)
    q[0, 1] *= 2.0 ** -100
    q[0, 2] *= 2.0 ** 20
    q[0, 3] = 0
    q[0, 4::7] *= 2.0 ** 9
    got = _attend(c, q, dtype, False, [n])
    assert tq.tq_check_device_status(ctx_for(d)) == 0
    _check_one(c, got[0], q[0], dtype, n - 1)


@pytest.mark.parametrize("dtype,d,g", FORMS)
def test_blocks_of_zeros_keep_their_weight(dtype, d, g):
    """Zero values have the smallest scale, 2^-100: their weights count in the sum all the same."""
    rng = np.random.default_rng(71)
    c = _one_head(rng, d, 310)
    zero = c.table[0][[1, 3, 8, 9, 12]]
    c.codes["v"][zero] = 0
    c.scales["v"][zero] = 2.0 ** -100
    c.scales["v"][c.table[0][5]] = 2.0 ** -9
    c.to_device()
    q = values(rng, dtype, 1, g, d)
    _check_one(c, _attend(c, q, dtype, False, [310])[0], q[0], dtype, 309)


@pytest.mark.parametrize("dtype,d,g", FORMS)
def test_tiny_queries_against_huge_keys(dtype, d, g):
    """Scores of usual size from queries of 2^-106 and keys of 2^111: no product on the way may pass fp32."""
    rng = np.random.default_rng(72)
    c = _one_head(rng, d, 310)
    c.scales["k"][:] = 2.0 ** 106
    c.scales["k"][c.table[0][::3]] = 2.0 ** 104
    c.to_device()
    q = values(rng, dtype, 1, g, d) * np.float32(2.0 ** -106)
    _check_one(c, _attend(c, q, dtype, False, [310])[0], q[0], dtype, 309)


@pytest.mark.parametrize("dtype,d,g", FORMS)
@pytest.mark.parametrize("n", [60, 310, 5000])
def test_a_query_that_is_not_finite_spoils_only_its_row(dtype, d, g, n):
    rng = np.random.default_rng(75)
    c = _one_head(rng, d, n)
    c.to_device()
    q = values(rng, dtype, 1, g, d)
    bad = {0: np.nan, 2: np.inf, 3: -np.inf, g - 1: np.nan}
    for r, x in bad.items():
        q[0, r, (5 + r) % d] = x
    got = _attend(c, q, dtype, False, [n])
    assert np.isnan(got[0, list(bad)]).all()
    keep = [r for r in range(g) if r not in bad]
    _check_one(c, got[0, keep], q[0, keep], dtype, n - 1, two_parts=dtype == "bf16" and g > 16)


@pytest.mark.parametrize("dtype,d,g", FORMS)
def test_keys_of_zeros_beside_huge_ones(dtype, d, g):
    """Scores beyond fp32 on one side (minus infinity there, weight zero) and exact zeros in the same block."""
    rng = np.random.default_rng(73)
    n = 310
    c = _one_head(rng, d, n)
    q = np.zeros((1, g, d), np.float32)
    q[..., 0] = 2.0 ** 20
    c.codes["k"][:, :, :, 0] = 0x7E                 # the largest code
    q[..., 0] *= -1
    c.codes["k"][c.table[0][2], 0, 3] = 0           # three keys of zeros
    c.codes["k"][c.table[0][11], 0, [0, 15]] = 0
    c.scales["k"][:] = 2.0 ** 119
    c.to_device()
    got = _attend(c, q, dtype, False, [n])
    v = lambda pg, s: kv8.VALUES[c.codes["v"][c.table[0][pg], 0, s]] * c.scales["v"][c.table[0][pg], 0]  # noqa: E731
    three = np.stack([v(2, 3), v(11, 0), v(11, 15)]).astype(np.float64)
    # weights of a third, each off by 2^-11 (bf16; 2^-21), and the output's rounding; subnormal weights: none
    tol = np.abs(three.mean(0)) * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) + np.abs(three).mean(0) * (
        (2.0 ** -11 if dtype == "bf16" else 2.0 ** -21) + 2.0 ** -19)
    assert np.all(np.abs(got[0] - three.mean(0)) <= tol)


@pytest.mark.parametrize("dtype,d,g", FORMS)
@pytest.mark.parametrize("best", [0, 17, 140, 309])
def test_scores_far_below_zero(dtype, d, g, best):
    """Every score near -2^116 but one at -2^110: that one's value is the result."""
    rng = np.random.default_rng(74)
    n = 310
    c = _one_head(rng, d, n)
    c.codes["k"][:] = 0x7E
    c.scales["k"][:] = 2.0 ** 104
    c.codes["k"][c.table[0][best // 16], 0, best % 16] = 0x4E           # 7 = 448 / 64
    c.to_device()
    q = np.full((1, g, d), -(2.0 ** -1), np.float32)
    got = _attend(c, q, dtype, False, [n])
    want = kv8.VALUES[c.codes["v"][c.table[0][best // 16], 0, best % 16]] * c.scales["v"][c.table[0][best // 16], 0]
    assert np.all(np.abs(got[0] - want) <= np.abs(want) * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -22))


@pytest.mark.parametrize("dtype,d,g", FORMS)
@pytest.mark.parametrize("n", [60, 310, 5000])
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_scores_win_at_every_size(dtype, d, g, n, sign):
    """Scores of 2^12 to 2^110: a few keys share the largest one exactly, every other lies far below.  The result is the
    mean of those keys' values, whatever the scales of their blocks."""
    rng = np.random.default_rng(76)
    for size in (12, 15, 17, 20, 23, 24, 25, 26, 27, 28, 29, 30, 31, 32, 33, 35, 40, 64, 110):
        c = _one_head(rng, d, n)
        c.scales["v"][:] = np.exp2(rng.integers(-50, 50, c.scales["v"].shape))
        step = rng.integers(0, 2, c.scales["k"].shape)
        c.scales["k"][:] = np.exp2(step + size // 2)
        best = sorted({int(x) for x in rng.integers(0, n, 4)} | {n - 1})
        # channel 0 decides: 64 times the smaller scale for the best, half (or, against a negative query, twice) for others
        for kv in range(n):
            pg, s = c.table[0][kv // 16], kv % 16
            v = 64.0 if kv in best else 32.0 if sign > 0 else 128.0
            c.codes["k"][pg, 0, s, 0] = kv8.e4m3_encode([v / 2.0 ** step[pg, 0]])[0]
        c.to_device()
        q = np.zeros((1, g, d), np.float32)
        q[..., 0] = sign * 2.0 ** (size - size // 2 - 3)
        got = _attend(c, q, dtype, False, [n])[0]
        pg, s = c.table[0][np.asarray(best) // 16], np.asarray(best) % 16
        codes, scales = kv8.VALUES[c.codes["v"][pg, 0, s]], c.scales["v"][pg, 0].astype(np.float64)
        v = codes * scales[:, None]
        # each rounding of a weight, of the exponents' sum (2^-21 of the score while one number holds it) and of the
        # result; weights below the normal ones as in _tails
        w = (2.0 ** -11 if dtype == "bf16" else 2.0 ** -21) + 2 * 2.0 ** (min(size, 17) + 1 - 21)
        tol = np.abs(v.mean(0)) * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) + np.abs(v).mean(0) * w + (
            2.0 ** -28 * scales.max() * np.abs(codes).mean(0))
        err = np.abs(got - v.mean(0))
        assert np.all(err <= tol), (size, best, float(np.nanmax(err / tol)), int(np.isnan(got).sum()))


# ---------------------------------------------------------------------------
# buffers and streams
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,d,h,hq,n_new,starts", [("bf16", 128, 2, 8, 1, [700, 20]), ("bf16", 128, 2, 8, 4, [9000, 40]),
                                                       ("f32", 64, 2, 4, 30, [500, 3]), ("bf16", 64, 2, 8, 150, [0, 900]),
                                                       ("bf16", 128, 2, 8, 70, [5000, 1]), ("bf16", 128, 1, 20, 1, [3000]),
                                                       ("bf16", 256, 2, 8, 4, [2000, 1])])
def test_results_in_the_queries_place(dtype, d, h, hq, n_new, starts):
    rng = np.random.default_rng(77)
    b = len(starts)
    maxp = (max(starts) + n_new) // 16 + 2
    c = Cache(rng, b * maxp, h, d, b, maxp)
    for i, s in enumerate(starts):
        c.clean(rng, i, range(s + n_new))
    c.to_device()
    dt, code = DT[dtype]
    q = values(rng, dtype, b, n_new, hq, d)
    n = tq.tq_kv8_workspace_size(ctx_for(d), b, n_new, hq, h, 16 * maxp)
    ws, at = torch.empty(n, dtype=torch.uint8, device=DEV), to_dev(np.asarray(starts, np.int32))
    want = _attend(c, q, dtype, True, starts)
    for _ in range(5):
        x = to_dev(q).to(dt)
        tq.tq_kv8_causal_attention(ctx_for(d), c.desc, x, code, b, n_new, hq, at, None, 16 * maxp, 0, 0, d ** -0.5, x, ws, n)
        torch.cuda.synchronize()
        assert np.array_equal(x.float().cpu().numpy(), want)
    _check(c, want, q, dtype, True, starts, rows={(i, t) for i in range(b) for t in (0, n_new - 1)})


@pytest.mark.parametrize("d", [64, 128, 256])
def test_two_streams_at_once_on_tcgen05(d):
    """Two calls that overlap on the GPU, items cut over many CTAs, each call with its own workspace."""
    rng = np.random.default_rng(78)
    c = Cache(rng, 400, 2, d, 1, 330)
    c.clean(rng, 0, range(5200))
    c.to_device()
    n_new, start = 90, 5000
    q = values(rng, "bf16", 1, n_new, 8, d)
    want = _attend(c, q, "bf16", True, [start])
    ctx, dt = ctx_for(d), torch.bfloat16
    n = tq.tq_kv8_workspace_size(ctx, 1, n_new, 8, 2, 5280)
    qd, at = to_dev(q).to(dt), to_dev(np.asarray([start], np.int32))
    runs = [(torch.cuda.Stream(), torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty(1, n_new, 8, d, dtype=dt, device=DEV))
            for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, ws, out in runs:
            tq.tq_kv8_causal_attention(ctx, c.desc, qd, tq.TQ_BF16, 1, n_new, 8, at, None, 5280, 0, 0, d ** -0.5, out, ws, n, st)
    torch.cuda.synchronize()
    for _, _, out in runs:
        assert np.array_equal(out.float().cpu().numpy(), want)
    _check(c, want, q, "bf16", True, [start], rows={(0, 0), (0, 45), (0, 89)})


# ---------------------------------------------------------------------------
# append: what is stored, where only the flags were looked at
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,d,rot,interleaved", [("f32", 128, 128, False), ("bf16", 128, 128, False), ("f32", 64, 32, True),
                                                     ("bf16", 256, 240, False), ("f32", 256, 256, True)])
def test_append_of_pairs_that_are_not_finite(dtype, d, rot, interleaved):
    """Of a turned pair with an infinity or NaN the infinite halves become the largest code, NaN zero; neither counts for
    the scale, and every other code is exact."""
    rng = np.random.default_rng(80)
    h, n, start = 2, 37, 6
    x = {"k": values(rng, dtype, 1, n, h, d) * 5, "v": values(rng, dtype, 1, n, h, d), "q": values(rng, dtype, 1, n, 2, d)}
    for t, head, ch, bad in ((0, 0, 3, np.inf), (3, 1, 5, -np.inf), (9, 0, rot // 2 + 2, np.nan), (10, 1, rot - 1, np.inf),
                             (25, 0, 0, np.nan), (26, 0, 1, np.inf), (36, 1, rot // 2, -np.inf)):
        x["k"][0, t, head, ch] = bad
        x["v"][0, t, head, (ch + 7) % d] = bad
    x["k"][0, 12, 0, 4] = x["k"][0, 12, 0, 4 + (1 if interleaved else rot // 2)] = np.inf     # both of a pair
    if rot < d:
        x["k"][0, 20, 1, d - 1] = np.inf            # a channel that does not turn
    c = _append_case(rng, dtype, d, h, 2, [start], n, rot=rot, interleaved=interleaved, x=x, kinds="kv", flags=32)
    for kind in "kv":
        codes = c.dev[kind + "c"].cpu().numpy()
        assert not ((codes & 127) == 127).any()     # no NaN code anywhere


def test_append_behind_a_scale_that_is_none():
    """An earlier token's block without a power of two as its scale: taken as 2^-100, so that its codes round to zero, and
    the new token has the scale that it needs."""
    rng = np.random.default_rng(81)
    h, d = 2, 128
    ctx = ctx_for(d)
    c = Cache(rng, 3, h, d, 1, 2, nan=False)
    desc = c.to_device()
    x = values(rng, "bf16", 1, 1, h, d)
    dev = to_dev(x).to(torch.bfloat16)
    page = int(c.table[0, 0])
    before = c.dev["kc"].cpu().numpy()[page]
    for bad in (3.0, 0.0, float("nan"), float("inf"), 2.0 ** 120, 2.0 ** -101, -1.0):
        c.dev["ks"][page] = bad
        c.dev["kc"][page] = to_dev(before)
        tq.tq_kv8_append(ctx, desc, dev, None, None, tq.TQ_BF16, 1, 1, 0, to_dev(np.asarray([2], np.int32)))
        torch.cuda.synchronize()
        assert tq.tq_check_device_status(ctx) == 64, bad
        codes, scales = c.dev["kc"].cpu().numpy()[page], c.dev["ks"].cpu().numpy()[page]
        for head in range(h):
            e = kv8.block_exponent(np.abs(x[0, 0, head]).max())
            assert scales[head] == 2.0 ** e
            assert np.all(kv8.VALUES[codes[head, :2]] == 0)
            assert np.array_equal(codes[head, 2], kv8.e4m3_encode(x[0, 0, head].astype(np.float64) * 2.0 ** -e))
            assert np.array_equal(codes[head, 3:], before[head, 3:])


@pytest.mark.parametrize("dtype,d,n_new", [("bf16", 128, 100), ("bf16", 64, 100), ("bf16", 256, 100), ("f32", 128, 30), ("bf16", 128, 3)])
def test_causal_calls_that_are_cut_answer_what_is_left(dtype, d, n_new):
    """Queries beyond max_seq_len, a padded count that is none and a negative start: the rows that remain are right, and the
    others stay."""
    rng = np.random.default_rng(82)
    c = Cache(rng, 40, 2, d, 3, 13)
    for b in range(3):
        c.clean(rng, b, range(200))
    c.to_device()
    q = values(rng, dtype, 3, n_new, 8, d)
    most = 130 + n_new * 7 // 10
    got = _attend(c, q, dtype, True, [130, -3, 50], lens=[1000, 5, n_new - 1], max_len=most)
    assert tq.tq_check_device_status(ctx_for(d)) == 4
    assert np.all(got[1] == -7)
    keep = [0, 2]
    sub = Cache.__new__(Cache)
    sub.__dict__.update(c.__dict__, table=c.table[keep])
    _check(sub, got[keep], q[keep], dtype, True, [130, 50], [most - 130, n_new - 1])


@pytest.mark.parametrize("dtype,d,g,n_new", [("bf16", 128, 4, 3), ("f32", 64, 3, 30), ("f32", 256, 2, 9), ("bf16", 64, 4, 30),
                                             ("bf16", 128, 4, 30), ("bf16", 256, 4, 30), ("bf16", 64, 4, 100), ("bf16", 128, 4, 100)])
@pytest.mark.parametrize("window,sinks,start", [(0, 0, 0), (0, 0, 3000), (100, 3, 350), (37, 20, 5)])
def test_large_scores_behind_masks(dtype, d, g, n_new, window, sinks, start):
    """Large scores in causal calls with windows, first tokens and rows at different positions: the mean over the visible
    keys of the largest score."""
    rng = np.random.default_rng(83)
    n = start + n_new
    for size in (17, 27, 60):
        c = _one_head(rng, d, n)
        c.scales["v"][:] = np.exp2(rng.integers(-20, 20, c.scales["v"].shape))
        c.scales["k"][:] = np.exp2(size // 2)
        c.codes["k"][:, :, :, 0] = kv8.e4m3_encode(rng.choice([32.0, 64.0, 128.0], c.codes["k"].shape[:3]))
        c.to_device()
        q = np.zeros((1, n_new, g, d), np.float32)
        q[..., 0] = rng.choice([-1.0, 1.0], (n_new, g)) * 2.0 ** (size - size // 2 - 2)
        q[0, 0, 0] = values(rng, dtype, d) * 2.0 ** -(size // 2)           # a row of usual scores among them
        got = _attend(c, q, dtype, True, [start], window=window, sinks=sinks)
        assert tq.tq_check_device_status(ctx_for(d)) == 0
        two_parts = dtype == "bf16" and n_new * g > 16
        for t in {0, 1, n_new // 2, n_new - 1}:
            want, mag, dots, ksum, keys = kv8.attention(q[0, t], c.codes["k"], c.scales["k"], c.codes["v"], c.scales["v"], c.table[0],
                                                        start + t, window, sinks, d ** -0.5)
            # exact scores but for the first row: no bound on a logit counts beyond 2^17 (where one number holds it)
            dots = np.where(q[0, t, :, 1] == 0, np.minimum(dots, 2.0 ** 17 * d ** 0.5), dots)
            parts = np.where(q[0, t, :, 1] == 0, 0.0, 2.0 ** -17 * np.abs(q[0, t]).max(axis=-1) * ksum if two_parts else 0.0)
            j = np.arange(start + t + 1)
            j = j[kv8.visible(start + t, j, window, sinks)]
            pg, sl = c.table[0][j // 16], j % 16
            tail = 2.0 ** -28 * c.scales["v"][pg, 0].max() * np.abs(kv8.VALUES[c.codes["v"][pg, 0, sl]]).sum(axis=0)
            tol = _bound(dtype, want, mag, dots, keys, d, d ** -0.5, parts) + tail
            err = np.abs(got[0, t] - want)
            assert np.all(err <= tol), (size, t, float(np.nanmax(err / tol)), int(np.isnan(got[0, t]).sum()))
