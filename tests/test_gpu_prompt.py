"""Attention over packed prompts on the GPU against plain attention in 64 bits, within bounds that count each rounding.

Per output element, with A = sum_j w_j |v_j| (w the weights, which add up to 1) and m keys:
  - the output's own rounding: half a step of its type, finfo.eps / 2 of the value;
  - a logit <q, k> in fp32: a sum of d products whose running size stays near the root of the sum of their squares, or the
    result; roundings of 2^-24 (2^-23 where a tensor core cuts a sum) add up like sqrt(d) of them, counted eight times;
  - its scaling and the exponential: 2^-22 of the logit's size in powers of two and 2^-22; a logit that is off by x moves
    a result by at most 2 x A;
  - bf16 on the tensor cores: the weights are rounded to bf16 for the value product, by half a step, 2^-8 of each at most;
  - the sums over keys: 2^-23 of A for each of sqrt(m) steps, counted eight times.
"""

import math

import numpy as np
import pytest

from .gpu_common import DEV, torch, tq

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, tq.TQ_BF16), "f32": (torch.float32, tq.TQ_F32)}
_CTX = {}


def ctx_for(d):
    if d not in _CTX:
        _CTX[d] = tq.tq_create(d, 3, 128, 0)
    return _CTX[d]


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def ends(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(int).tolist()


def reference(q, k, v, window, sinks, scale, weight_step):
    """q [n][hq][d], k, v [m][h][d], all in fp64: results [n][hq][d] and their bounds without the output's rounding."""
    n, hq, d = q.shape
    m, h = k.shape[:2]
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    p = torch.arange(m - n, m, device=DEV)[:, None]
    j = torch.arange(m, device=DEV)[None]
    seen = j <= p
    if window:
        seen = seen & ((j > p - window) | (j < sinks))
    any_seen = seen.any(1)
    if not bool(any_seen.any()):
        return out, bound
    for a in range(hq):
        kk, vv = k[:, a // (hq // h)], v[:, a // (hq // h)]
        # what nobody may look at does not enter the plain form either
        ks = torch.where(seen.any(0)[:, None], kk, 0.0)
        s = q[:, a] @ ks.T
        x = (s * scale).masked_fill(~seen, -math.inf)
        w = torch.softmax(x[any_seen], dim=-1)
        vs = torch.where(seen.any(0)[:, None], vv, 0.0)
        if bool(torch.isfinite(vs).all()):
            o = w @ vs
            size = w @ vs.abs()
        else:                               # a value that some rows see and others do not
            sr = seen[any_seen]
            each = [torch.where(sr[i][:, None], vs, 0.0) * w[i][:, None] for i in range(len(w))]
            o = torch.stack([x.sum(0) for x in each])
            size = torch.stack([x.abs().sum(0) for x in each])              # A, not the sum's size: its terms cancel
        rough = 8 * math.sqrt(d) * 2.0 ** -24 * (torch.sqrt((q[:, a] ** 2) @ (ks ** 2).T) + s.abs()) * abs(scale)
        rough = rough + 2.0 ** -22 * (s * scale).abs()
        e = torch.where(seen, rough, 0.0).amax(1)[any_seen][:, None]
        out[any_seen, a] = o
        bound[any_seen, a] = size * (2 * e + weight_step + 2.0 ** -21 + 8 * math.sqrt(m) * 2.0 ** -23)
    return out, bound


def attend(dtype, d, hq, h, new, keys, window=0, sinks=0, scale=None, strides="dense", pad=0, seed=0, change=None, flags=0,
           out=None, repeat=1):
    """One call, checked; `change(q, k, v)` edits the inputs, `pad` rows stand behind the last sequence."""
    dt, code = DT[dtype]
    gen = torch.Generator(device=DEV).manual_seed(seed)
    tq_, tk = sum(new) + pad, sum(keys) + pad
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(dt)  # noqa: E731
    row = {"q": 0, "k": 0, "v": 0}
    if strides == "fused":
        assert tq_ == tk
        big = rnd(tq_, (hq + 2 * h) * d)
        q, k, v = (x.unflatten(-1, (-1, d)) for x in big.split([hq * d, h * d, h * d], dim=-1))
        row = dict.fromkeys("qkv", (hq + 2 * h) * d)
    elif strides == "odd":                    # rows apart, each its own way
        step = 16 // dt.itemsize
        row = {"q": hq * d + 3 * step, "k": h * d + step, "v": h * d + 5 * step}
        q, k, v = (rnd(n, row[x])[:, step:step + hh * d].unflatten(-1, (hh, d)) if n else rnd(0, hh, d)
                   for x, n, hh in (("q", tq_, hq), ("k", tk, h), ("v", tk, h)))
    else:
        q, k, v = rnd(tq_, hq, d), rnd(tk, h, d), rnd(tk, h, d)
    if change:
        change(q, k, v)
    ctx = ctx_for(d)
    size = tq.tq_prompt_workspace_size(ctx, len(new), max(new), hq, h, max(keys))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)          # a workspace needs no contents
    got = torch.full((tq_, hq, d), -7.0, dtype=dt, device=DEV) if out is None else out
    for _ in range(repeat):
        tq.tq_prompt_attention(ctx, q, k, v, code, len(new), ints(ends(new)), ints(ends(keys)), tq_, tk, max(new), max(keys), hq,
                               h, window, sinks, scale, got, ws, size, q_stride=row["q"], k_stride=row["k"],
                               v_stride=row["v"], stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == flags
    step = 2.0 ** -8 if dtype == "bf16" else 0.0
    aq = ak = 0
    worst = 0.0
    for n, m in zip(new, keys):
        want, bound = reference(q[aq:aq + n].double(), k[ak:ak + m].double(), v[ak:ak + m].double(), window, sinks, scale, step)
        bound = bound + torch.finfo(dt).eps / 2 * (want.abs() + bound) + torch.finfo(dt).tiny
        x = got[aq:aq + n].double()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(x), nan)
        same = (x == want) | nan                                            # infinities among them
        over = torch.where(same, 0.0, (x - want).abs() / bound)
        if n:
            worst = max(worst, float(over.max()))
        aq, ak = aq + n, ak + m
    assert worst <= 1.0, worst
    assert bool((got[aq:] == -7.0).all())
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,hq,h", [(32, 4, 2), (64, 8, 1), (96, 3, 3), (128, 8, 2), (128, 7, 1), (160, 4, 4), (192, 2, 1),
                                    (224, 2, 2), (256, 6, 2)])
def test_packed_prompts(dtype, d, hq, h):
    attend(dtype, d, hq, h, [1, 70, 0, 129, 17], [1, 70, 0, 129, 17], pad=3)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 128)])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
def test_lengths_around_the_tiles(dtype, d, n):
    attend(dtype, d, 4, 1, [n], [n], seed=n)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("bf16", 96)])
@pytest.mark.parametrize("new,keys", [([1], [5000]), ([3, 1, 40], [3000, 1, 41]), ([100, 7], [1000, 2007]), ([1] * 9, list(range(1, 10))),
                                      ([200], [20000])])
def test_chunks_behind_cached_keys(dtype, d, new, keys):
    attend(dtype, d, 8, 2, new, keys)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 0), (100, 200), (128, 4), (300, 129), (5000, 9), (333, 0)])
def test_windows_and_first_tokens(dtype, d, window, sinks):
    attend(dtype, d, 6, 2, [700, 33, 1], [700, 900, 650], window=window, sinks=sinks)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 32)])
def test_more_queries_than_keys(dtype, d):
    """Rows that see nothing give zeros, beside rows that see something."""
    got = attend(dtype, d, 4, 2, [5, 300, 70, 3], [0, 11, 69, 700])
    assert bool((got[:5] == 0).all()) and bool((got[5:5 + 289] == 0).all()) and bool((got[305] == 0).all())
    assert not bool((got[306] == 0).all())


@pytest.mark.parametrize("strides", ["fused", "odd"])
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 128), ("f32", 96)])
def test_strides(dtype, d, strides):
    attend(dtype, d, 4, 2, [90, 1, 200], [90, 1, 200], strides=strides)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 128)])
@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0, 5.0, 1e-6])
def test_softmax_scales(dtype, d, scale):
    attend(dtype, d, 4, 1, [150, 20], [150, 400], scale=scale)


@pytest.mark.parametrize("g", [1, 3, 5, 16, 40, 300])
def test_heads_per_kv_head(g):
    attend("bf16", 128, 2 * g, 2, [1, 50], [200, 51])
    attend("f32", 64, g, 1, [1, 50], [200, 51])


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 128)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_hidden_keys_may_hold_anything(dtype, d, bad):
    """Keys and values that are not finite: behind the last row, in another sequence, at later positions and before a
    window; rows that do not see them stay what they are."""
    def poison(q, k, v):
        k[-3:], v[-3:] = bad, bad                       # behind the last sequence
        v[200:210] = bad                                # at the end of the first sequence, seen by its last rows alone
        k[205] = bad
        v[210 + 100] = bad                              # second sequence: seen by what stands behind
    got = attend_poisoned(dtype, d, poison, 0, 0)
    assert bool(torch.isfinite(got[:200]).all()) and bool(torch.isfinite(got[210:310]).all()) and bool(torch.isfinite(got[410:430]).all())
    assert not bool(torch.isfinite(got[205:210]).any()) and not bool(torch.isfinite(got[310:410]).all())

    def old(q, k, v):
        k[:40], v[:40] = bad, bad
        v[215:230] = -math.inf
    got = attend_poisoned(dtype, d, old, 33, 0)
    assert bool(torch.isfinite(got[39 + 33:210]).all()) and bool(torch.isfinite(got[229 + 33:430]).all())


def attend_poisoned(dtype, d, change, window, sinks):
    """Compared row by row: rows whose seen keys and values are all finite are held to the bounds, the others are not finite."""
    dt, code = DT[dtype]
    hq, h, new = 4, 2, [210, 200, 20]
    n = sum(new) + 3
    gen = torch.Generator(device=DEV).manual_seed(5)
    q, k, v = (torch.randn(n, x, d, generator=gen, device=DEV).to(dt) for x in (hq, h, h))
    clean = [x.clone() for x in (q, k, v)]
    change(q, k, v)
    ctx = ctx_for(d)
    size = tq.tq_prompt_workspace_size(ctx, 3, 210, hq, h, 210)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    got = torch.full((n, hq, d), -7.0, dtype=dt, device=DEV)
    tq.tq_prompt_attention(ctx, q, k, v, code, 3, ints(ends(new)), ints(ends(new)), n, n, 210, 210, hq, h, window, sinks,
                           1 / math.sqrt(d), got, ws, size)
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == 0
    at = 0
    for m in new:
        ok = (torch.isfinite(k[at:at + m]) & torch.isfinite(v[at:at + m])).flatten(1).all(1)
        p = torch.arange(m, device=DEV)
        seen = (p[None] <= p[:, None]) & ((p[None] > p[:, None] - window) if window else True)
        good = ~(seen & ~ok[None]).any(1)
        want, bound = reference(*(x[at:at + m].double() for x in clean), window, sinks, 1 / math.sqrt(d), 2.0 ** -8 if dtype == "bf16" else 0.0)
        bound = bound + torch.finfo(dt).eps / 2 * (want.abs() + bound)
        assert bool(((got[at:at + m].double() - want).abs() <= bound)[good].all())
        at += m
    return got


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 128)])
@pytest.mark.parametrize("new,keys", [([200, 9], [200, 400]), ([1], [3000])])
def test_queries_that_are_not_finite_spoil_only_their_rows(dtype, d, new, keys):
    dt, code = DT[dtype]
    gen = torch.Generator(device=DEV).manual_seed(6)
    nq, nk = sum(new), sum(keys)
    q, k, v = torch.randn(nq, 4, d, generator=gen, device=DEV).to(dt), *(torch.randn(nk, 2, d, generator=gen, device=DEV).to(dt) for _ in range(2))
    ctx = ctx_for(d)
    size = tq.tq_prompt_workspace_size(ctx, len(new), max(new), 4, 2, max(keys))
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    outs = []
    for bad in (None, math.nan, math.inf):
        x = q.clone()
        if bad is not None:
            x[0, 1, 3] = bad
        o = torch.empty_like(q)
        tq.tq_prompt_attention(ctx, x, k, v, code, len(new), ints(ends(new)), ints(ends(keys)), nq, nk, max(new), max(keys), 4, 2, 0, 0,
                               0.1, o, ws, size)
        outs.append(o)
    torch.cuda.synchronize()
    aq = ak = 0
    for n, m in zip(new, keys):
        want, bound = reference(q[aq:aq + n].double(), k[ak:ak + m].double(), v[ak:ak + m].double(), 0, 0, 0.1, 2.0 ** -8 if dtype == "bf16" else 0.0)
        bound = bound + torch.finfo(dt).eps / 2 * (want.abs() + bound)
        for i, o in enumerate(outs):
            good = (o[aq:aq + n].double() - want).abs() <= bound
            if i and aq == 0:
                assert bool(torch.isnan(o[0, 1]).all())               # (of an infinite channel: infinity less itself)
                good[0, 1] = True
            assert bool(good.all())
        aq, ak = aq + n, ak + m


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 128)])
@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 12, 2.0 ** 30])
def test_large_scores(dtype, d, size):
    """Scores far beyond what an exponent holds: powers of two, so that every score is exact and the largest keys share
    the weight; results are means of their values."""
    dt, code = DT[dtype]
    n = 300
    q = torch.full((n, 2, d), 1.0, device=DEV, dtype=dt) * size
    k = torch.zeros((n, 1, d), device=DEV, dtype=dt)
    k[:, 0, 0] = (torch.arange(n, device=DEV) % 7).to(dt) * size * 2.0 ** -4       # scores 0 .. 6 times size^2 / 16
    gen = torch.Generator(device=DEV).manual_seed(1)
    v = torch.randn(n, 1, d, generator=gen, device=DEV).to(dt)
    ctx = ctx_for(d)
    ws_n = tq.tq_prompt_workspace_size(ctx, 1, n, 2, 1, n)
    ws, out = torch.zeros(ws_n, dtype=torch.uint8, device=DEV), torch.empty_like(q)
    tq.tq_prompt_attention(ctx, q, k, v, code, 1, ints([0, n]), ints([0, n]), n, n, n, n, 2, 1, 0, 0, 1.0, out, ws, ws_n)
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == 0
    for t in range(n):
        best = torch.arange(t + 1, device=DEV) % 7 == min(t, 6)
        vals = v[:t + 1, 0][best].double()
        want, a = vals.mean(0), vals.abs().mean(0)
        tol = torch.finfo(dt).eps / 2 * want.abs() * 1.01 + a * (2.0 ** -20 + (2.0 ** -8 if dtype == "bf16" else 0.0))
        assert bool(((out[t].double() - want).abs() <= tol).all()), t


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 128)])
@pytest.mark.parametrize("kind", ["rising", "falling", "tiles", "rows", "far below", "steps"])
@pytest.mark.parametrize("new,keys,window", [([700], [700], 0), ([300, 1, 20, 200], [1300, 900, 20, 333], 0), ([260, 70], [1500, 70], 400)])
def test_maxima_that_move(dtype, d, kind, new, keys, window):
    """Scores whose size changes along the keys and the rows: hundreds and thousands (in powers of two) up or down from one
    tile to the next, in one half's tiles and not in the other's, all of them far below zero."""
    def change(q, k, v):
        j = torch.arange(k.shape[0], device=DEV)
        t = torch.arange(q.shape[0], device=DEV)
        size = {"rising": 1.0 + j / 16, "falling": 80.0 - (j % 1500) / 20, "tiles": torch.where(j // 128 % 2 == 0, 1.0, 60.0),
                "rows": torch.ones_like(j, dtype=torch.float), "far below": 40.0 + j % 128 / 8,
                "steps": 2.0 ** (j // 100 % 9).float()}[kind]
        if kind == "far below":                       # a direction that every key has and every query is against
            k[:, :, 0], q[:, :, 0] = 0.0, -30.0
            k += 0.0
            k[:, :, 0] = size[:, None].to(k.dtype)
        else:
            k *= size.to(k.dtype)[:, None, None]
        if kind == "rows":
            q *= (2.0 ** (t % 11 - 2).float()).to(q.dtype)[:, None, None]
    attend(dtype, d, 8, 2, new, keys, window=window, change=change)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 128)])
def test_many_sequences_and_blocks(dtype, d):
    """More sequences than the list of spans holds, and more blocks."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 9, 2500).tolist()
    attend(dtype, d, 2, 1, lens, [n + (i % 5) for i, n in enumerate(lens)])
    if dtype == "f32":
        attend(dtype, 32, 64, 1, [2100, 50], [2100, 50], window=40)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,h", [(4, 1), (24, 3)])
def test_short_and_long_prompts_in_any_order(d, hq, h):
    """Items of one tile, of several in one half and of two halves follow each other in a block, in every order."""
    rng = np.random.default_rng(5)
    new = rng.choice([1, 1, 1, 2, 5, 20, 33, 40, 64, 65, 130], 400).tolist()
    keys = [n + int(k) for n, k in zip(new, rng.choice([0, 0, 0, 1, 100, 127, 128, 300, 700], 400))]
    attend("bf16", d, hq, h, new, keys)
    attend("bf16", d, hq, h, new, keys, window=90, sinks=3)
    attend("bf16", d, hq, h, [1] * 700 + [90] + [1] * 700, [3] * 700 + [500] + [2] * 700)


@pytest.mark.parametrize("d", [64, 256])
def test_more_sequences_than_the_list(d):
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 6, 2200).tolist()
    lens[700], lens[1500] = 300, 129
    attend("bf16", d, 2, 1, lens, [n + (i % 4) for i, n in enumerate(lens)], window=100, sinks=2)


@pytest.mark.parametrize("d", [64, 128])
def test_fp32_of_many_sequences(d):
    """More than the list holds, prompts of one tile and of several in turn."""
    rng = np.random.default_rng(6)
    new = rng.integers(0, 5, 2200).tolist()
    new[300], new[900] = 150, 64
    attend("f32", d, 2, 1, new, [n + (i % 70) for i, n in enumerate(new)])
    new = rng.choice([1, 2, 30, 64, 65, 129], 150).tolist()
    attend("f32", d, 4, 2, new, [n + int(k) for n, k in zip(new, rng.choice([0, 63, 64, 200, 900], 150))], window=130, sinks=2)


@pytest.mark.parametrize("dtype,d,scale", [("f32", 128, None), ("f32", 64, 0.01), ("bf16", 128, -0.01)])
def test_sums_of_one_sign(dtype, d, scale):
    """Long sums of values, and scores, that do not cancel."""
    def change(q, k, v):
        v.abs_().add_(1.0)
        q.abs_()
        k.abs_().mul_(0.25)
    attend(dtype, d, 4, 2, [70, 3], [6000, 2500], scale=scale, change=change)


def two_keys(d, q, k, v, scale):
    """Single queries (of many heads) that see two keys each, fp32 on both sides."""
    s, hq = q.shape[:2]
    ctx = ctx_for(d)
    q, k, v = (torch.from_numpy(x).to(DEV) for x in (q, k, v))
    size = tq.tq_prompt_workspace_size(ctx, s, 1, hq, 1, 2)
    ws, out = torch.zeros(size, dtype=torch.uint8, device=DEV), torch.empty_like(q)
    tq.tq_prompt_attention(ctx, q, k, v, tq.TQ_F32, s, ints(range(s + 1)), ints(range(0, 2 * s + 1, 2)), s, 2 * s, 1, 2, hq, 1, 0, 0, scale,
                           out, ws, size)
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == 0
    return out.double().cpu().numpy()


@pytest.mark.parametrize("d", [64, 128])
def test_fp32_products_keep_24_bits(d):
    """Scores of one product each, of numbers whose parts are as large as parts can be, against a score that is exact: what the
    two weights show of the difference.  Counted: 2^-24 of the product for what six products of parts leave out, a cut of the
    sum twice (2^-23), and both scores' scaling (2^-24 each); the exponentials and the rest 2^-20 of the result."""
    rng = np.random.default_rng(11)
    s, hq, big = 64, 20, 2.0 ** 13
    low = [(1 << 16) - 1, 1 << 16, 0x7FFF, 0x8000, 0xFFFF, 0x17FFF, 0x18000, 0x1FFFF, 0xFF7F, 0x7F80]
    pick = lambda *shape: ((1 << 23) + (rng.integers(0, 64, shape) << 17) * (rng.random(shape) < 0.5) + rng.choice(low, shape)) / 2.0 ** 23  # noqa: E731
    a, b = pick(s, hq), pick(s, 1)
    a[:8], b[:8] = 1 + 2.0 ** -7 - 2.0 ** -23, 1 + 2.0 ** -7 - 2.0 ** -23
    q, k, v = (np.zeros((n, h, d), np.float32) for n, h in ((s, hq), (2 * s, 1), (2 * s, 1)))
    c = (a * b * big).astype(np.float32)
    q[:, :, 0], q[:, :, 1] = a * big, c
    k[::2, 0, 0], k[1::2, 0, 1] = b[:, 0], 1.0
    v[::2] = 1.0
    scale = math.log(2.0)
    f = float(np.float32(scale) * np.float32(1.4426950408889634))
    got = two_keys(d, q, k, v, scale)
    apart = f * (a * b * big - c.astype(np.float64))
    tol = f * a * b * big * (0.5 + 2 + 1) * 2.0 ** -23
    lo, hi = (1 / (1 + np.exp2(-(apart + x))) for x in (-tol, tol))
    assert np.all(got >= lo[..., None] * (1 - 2.0 ** -20)) and np.all(got <= hi[..., None] * (1 + 2.0 ** -20))


@pytest.mark.parametrize("d", [64, 128])
def test_fp32_keys_beyond_the_largest_bf16_number(d):
    """Finite ones: two scores that are exact and equal, so that the values' mean comes out, and a value that size alone."""
    most = np.array([0x7F7FFFFF, 0x7F7F8000, 0x7F7F7FFF, 0x7F7FC001], np.uint32).view(np.float32)
    s, hq = len(most), 20
    q, k, v = (np.zeros((n, h, d), np.float32) for n, h in ((s, hq), (2 * s, 1), (2 * s, 1)))
    q[:, :, 0], q[:, :, 1] = 2.0 ** -114, most[:, None] * np.float32(2.0 ** -114)
    k[::2, 0, 0], k[1::2, 0, 1] = most, 1.0
    v[::2], v[1::2] = 3.0, 1.0
    got = two_keys(d, q, k, v, 1.0)
    assert np.abs(got - 2.0).max() <= 2.0 ** -20
    v[1::2, 0, :] = np.where(np.arange(d) % 2, most[:, None], -most[:, None])
    k[::2], k[1::2, 0, 1] = 0.0, 1.0                                # (the other key's weight is nothing)
    got = two_keys(d, q, k, v, 1.0)
    assert np.array_equal(got, np.broadcast_to(v[1::2].astype(np.float64), got.shape))


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 60, 2.0 ** 99])
def test_fp32_sizes(size):
    """Values of any size, queries and keys whose sizes cancel in the scores."""
    def change(q, k, v):
        q.mul_(size)
        k.div_(size)
        v.mul_(size)
    attend("f32", 128, 4, 2, [130, 17], [300, 900], change=change)


@pytest.mark.parametrize("dtype,d,scale", [("f32", 64, None), ("bf16", 64, -0.05), ("bf16", 128, -0.05)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_that_are_not_finite_spoil_only_who_sees_them(dtype, d, scale, bad):
    def change(q, k, v):
        v[5, 0, 3] = v[120, 1, 7] = v[199, 0, 0] = bad
    attend(dtype, d, 4, 2, [200], [200], scale=scale, change=change)
    attend(dtype, d, 4, 2, [200], [200], scale=scale, change=change, window=40)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g", [64, 65, 100, 128, 129])
def test_many_heads_per_kv_head(d, g):
    attend("bf16", d, 2 * g, 2, [5, 1, 40], [5, 300, 200])


def test_offsets_that_are_none_are_skipped_and_flagged():
    d, h = 128, 2
    ctx = ctx_for(d)
    x = torch.randn(100, h, d, device=DEV).bfloat16()
    ws_n = tq.tq_prompt_workspace_size(ctx, 3, 100, h, h, 100)
    ws = torch.zeros(ws_n, dtype=torch.uint8, device=DEV)

    def run(cu_q, cu_k, max_q=100, max_k=100):
        out = torch.full_like(x, -7.0)
        tq.tq_prompt_attention(ctx, x, x, x, tq.TQ_BF16, 3, ints(cu_q), ints(cu_k), 100, 100, max_q, max_k, h, h, 0, 0, 0.1, out, ws, ws_n)
        torch.cuda.synchronize()
        return out, tq.tq_check_device_status(ctx)
    good, flags = run([0, 30, 60, 100], [0, 30, 60, 100])
    assert flags == 0 and not bool((good == -7).any())
    # (in the first, rows 20 .. 29 are the third sequence's, too)
    for cu_q, cu_k, kept in (([0, 30, 20, 100], [0, 30, 60, 100], slice(0, 20)), ([0, 30, 60, 101], [0, 30, 60, 100], slice(0, 60)),
                             ([0, 30, 60, 100], [0, 30, 60, 1 << 30], slice(0, 60)), ([-5, 30, 60, 100], [0, 30, 60, 100], slice(30, 100))):
        out, flags = run(cu_q, cu_k)
        assert flags == 4
        assert torch.equal(out[kept], good[kept])
    out, flags = run([0, 30, 60, 100], [0, 30, 60, 100], max_q=35)
    assert flags == 4 and torch.equal(out[:60], good[:60]) and bool((out[60:] == -7).all())
    out, flags = run([0, 30, 60, 100], [0, 30, 60, 100], max_k=35)
    assert flags == 4 and torch.equal(out[:60], good[:60]) and bool((out[60:] == -7).all())


# a form each: tcgen05, three parts on tcgen05 (fp32, and bf16 at a scale below 0), CUDA cores; with the query rows of a block
FORMS = [("bf16", 64, None, 256), ("bf16", 128, None, 256), ("bf16", 256, None, 128), ("f32", 64, None, 128), ("f32", 128, None, 128),
         ("bf16", 128, -0.05, 128), ("f32", 96, None, 64), ("bf16", 96, None, 64), ("f32", 256, None, 64)]


def by_offsets(dtype, d, scale, cu_q, cu_k, total, hq=4, h=1, max_q=None, max_k=None, seed=0, flags=4):
    """A call with any offsets: its inputs and what it leaves of an output of -7."""
    dt, code = DT[dtype]
    gen = torch.Generator(device=DEV).manual_seed(seed)
    q, k, v = (torch.randn(total, x, d, generator=gen, device=DEV).to(dt) for x in (hq, h, h))
    ctx, max_q, max_k = ctx_for(d), total if max_q is None else max_q, total if max_k is None else max_k
    size = tq.tq_prompt_workspace_size(ctx, len(cu_q) - 1, max_q, hq, h, max_k)
    ws, out = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV), torch.full_like(q, -7.0)
    tq.tq_prompt_attention(ctx, q, k, v, code, len(cu_q) - 1, ints(cu_q), ints(cu_k), total, total, max_q, max_k, hq, h, 0, 0,
                           1 / math.sqrt(d) if scale is None else scale, out, ws, size)
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == flags
    return q, k, v, out


def near(dtype, d, scale, q, k, v, got):
    want, bound = reference(q.double(), k.double(), v.double(), 0, 0, 1 / math.sqrt(d) if scale is None else scale, 2.0 ** -8 if dtype == "bf16" else 0.0)
    return bool(((got.double() - want).abs() <= bound + torch.finfo(got.dtype).eps / 2 * (want.abs() + bound)).all())


@pytest.mark.parametrize("dtype,d,scale,rows", FORMS)
def test_offsets_that_fall_again_and_again(dtype, d, scale, rows):
    """The same rows in every second pair of offsets: more blocks than rows of that number make."""
    n = 700
    q, k, v, out = by_offsets(dtype, d, scale, [0, n] * 40, [0, n] * 40, n + 9)
    assert near(dtype, d, scale, q[:n], k[:n], v[:n], out[:n]) and bool((out[n:] == -7).all())


@pytest.mark.parametrize("dtype,d,scale,rows", FORMS[:-1])
def test_offsets_that_fall_behind_many_blocks(dtype, d, scale, rows):
    """Twice the rows that the list of 2,048 blocks takes once: the second time they are left out."""
    n = 1560 * rows // 4
    q, k, v, out = by_offsets(dtype, d, scale, [0, n, 0, n], [0, n, 0, n], n + 9)
    for at in (0, n // 2, n - 40):
        assert near(dtype, d, scale, q[at:at + 40], k[:at + 40], v[:at + 40], out[at:at + 40])
    assert not bool((out[:n] == -7).all(-1).any()) and bool((out[n:] == -7).all())


@pytest.mark.parametrize("dtype,d,scale,rows", FORMS)
@pytest.mark.parametrize("cu_q,cu_k,max_q,max_k,left", [
    ([0, 600, 400, 2000], [0, 600, 1500, 2000], 2000, 2000, [1]),             # falls: rows 400 .. 599 are the third sequence's, too
    ([0, 600, 1500, 2001], [0, 600, 1500, 2000], 2000, 2000, [2]),
    ([0, 600, 1500, 2000], [0, 600, 1500, 1 << 30], 2000, 2000, [2]),
    ([-5, 600, 1500, 2000], [0, 600, 1500, 2000], 2000, 2000, [0]),
    ([0, 600, 1500, 2000], [-(1 << 31), 600, 1500, 2000], 2000, 2000, [0]),
    ([0, 600, 1500, 2000], [0, 600, 300, 2000], 2000, 2000, [1]),
    ([0, 600, 1500, 2000], [0, 600, 1500, 2000], 700, 2000, [1]),
    ([0, 600, 1500, 2000], [0, 600, 1500, 2000], 2000, 599, [0, 1]),
    ([3000, 2000, 1000, -7], [0, 600, 1500, 2000], 2000, 2000, [0, 1, 2])])
def test_offsets_that_are_none_among_cut_items(dtype, d, scale, rows, cu_q, cu_k, max_q, max_k, left):
    """Lists that are cut into spans: what is no sequence is left as it was, the others are right."""
    q, k, v, out = by_offsets(dtype, d, scale, cu_q, cu_k, 2000, 4, 2, max_q, max_k, seed=3)
    taken = [(cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]) for s in range(3) if s not in left]
    owners = torch.zeros(2000, dtype=torch.int32, device=DEV)
    for a, b, *_ in taken:
        owners[a:b] += 1
    for a, b, c, e in taken:
        want, bound = reference(q[a:b].double(), k[c:e].double(), v[c:e].double(), 0, 0, 1 / math.sqrt(d) if scale is None else scale,
                                2.0 ** -8 if dtype == "bf16" else 0.0)
        bound = bound + torch.finfo(out.dtype).eps / 2 * (want.abs() + bound)
        assert bool(((out[a:b].double() - want).abs() <= bound)[owners[a:b] == 1].all())
    assert bool((out[owners == 0] == -7).all())


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 128)])
def test_results_repeat_bit_for_bit(dtype, d):
    outs = [attend(dtype, d, 8, 2, [300, 1, 45], [1300, 2000, 45], repeat=3) for _ in range(4)]
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed_with_new_inputs(dtype):
    """Two graphs that share a workspace, replayed with other inputs, offsets among them."""
    dt, code = DT[dtype]
    step = 2.0 ** -8 if dtype == "bf16" else 0.0
    d, hq, h, n = 128, 8, 2, 400
    ctx = ctx_for(d)
    bufs = [torch.zeros(n, x, d, dtype=dt, device=DEV) for x in (hq, h, h)]
    cu = ints([0, 0, 0])
    ws_n = tq.tq_prompt_workspace_size(ctx, 2, n, hq, h, n)
    ws = torch.zeros(ws_n, dtype=torch.uint8, device=DEV)
    outs = [torch.zeros(n, hq, d, dtype=dt, device=DEV) for _ in range(2)]
    graphs = []
    for window, out in zip((0, 50), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tq.tq_prompt_attention(ctx, *bufs, code, 2, cu, cu, n, n, n, n, hq, h, window, 0, 0.1, out, ws, ws_n,
                                   stream=torch.cuda.current_stream())
        graphs.append(g)
    for seed, offsets in ((1, [0, 100, 400]), (2, [0, 399, 400]), (3, [0, 0, 350])):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        for b in bufs:
            b.copy_(torch.randn(b.shape, generator=gen, device=DEV))
        cu.copy_(ints(offsets))
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        for window, out in zip((0, 50), outs):
            for a, b in zip(offsets[:-1], offsets[1:]):
                want, bound = reference(*(x[a:b].double() for x in bufs), window, 0, 0.1, step)
                assert bool(((out[a:b].double() - want).abs() <= bound + torch.finfo(dt).eps / 2 * (want.abs() + bound)).all())
    assert tq.tq_check_device_status(ctx) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_streams_at_once(dtype):
    dt, code = DT[dtype]
    step = 2.0 ** -8 if dtype == "bf16" else 0.0
    d, hq, h, n = 128, 8, 2, 500
    ctx = ctx_for(d)
    ws_n = tq.tq_prompt_workspace_size(ctx, 1, n, hq, h, n)
    sets = []
    for seed in (1, 2):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        sets.append([torch.randn(n, x, d, generator=gen, device=DEV).to(dt) for x in (hq, h, h)] +
                    [torch.zeros(n, hq, d, dtype=dt, device=DEV), torch.zeros(ws_n, dtype=torch.uint8, device=DEV), torch.cuda.Stream()])
    cu = ints([0, n])
    want = []
    for rounds in (1, 8):
        torch.cuda.synchronize()
        for _ in range(rounds):
            for q, k, v, out, ws, s in sets:
                tq.tq_prompt_attention(ctx, q, k, v, code, 1, cu, cu, n, n, n, n, hq, h, 0, 0, 0.1, out, ws, ws_n, stream=s)
            if rounds == 1:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        want.append([x[3].clone() for x in sets])
    assert all(torch.equal(a, b) for a, b in zip(*want))
    for q, k, v, out, ws, s in sets:
        r, bound = reference(q.double(), k.double(), v.double(), 0, 0, 0.1, step)
        assert bool(((out.double() - r).abs() <= bound + torch.finfo(dt).eps / 2 * (r.abs() + bound)).all())


def test_rows_beyond_32_bit_offsets():
    """Keys whose elements lie beyond 2^31 (and bytes beyond 2^32): the last sequence of a long buffer."""
    d, h, rows = 128, 8, (1 << 21) + 4096 + 77
    k = torch.zeros(rows, h, d, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    n = 90
    gen = torch.Generator(device=DEV).manual_seed(4)
    q = torch.randn(n, 2 * h, d, generator=gen, device=DEV).bfloat16()
    k[-n:] = torch.randn(n, h, d, generator=gen, device=DEV).bfloat16()
    v[-n:] = torch.randn(n, h, d, generator=gen, device=DEV).bfloat16()
    ctx = ctx_for(d)
    ws_n = tq.tq_prompt_workspace_size(ctx, 2, n, 2 * h, h, rows)
    ws, out = torch.zeros(ws_n, dtype=torch.uint8, device=DEV), torch.zeros_like(q)
    tq.tq_prompt_attention(ctx, q, k, v, tq.TQ_BF16, 2, ints([0, 0, n]), ints([0, rows - n, rows]), n, rows, n, rows, 2 * h, h, 0, 0, 0.1,
                           out, ws, ws_n)
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == 0
    want, bound = reference(q.double(), k[-n:].double(), v[-n:].double(), 0, 0, 0.1, 2.0 ** -8)
    assert bool(((out.double() - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound)).all())
