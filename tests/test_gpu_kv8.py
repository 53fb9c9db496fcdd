"""The 8-bit paged cache on the GPU against the fp64 oracle: appended codes and scales bit for bit, attention within
bounds that count each rounding.

Attention's bounds, per output element, with A = sum_j p_j |v_j| and the seen keys n:
  - the output's own rounding: half a step of its type, finfo.eps / 2 of the value;
  - the weights as fp16 (2^-11 of each; fp32 input: hi + lo, 2^-22);
  - a logit's error: fp32 sums of exact products over d channels in the tensor core, at most d/16 + 1 steps
    each off by 2^-23 of the running size, times scale * sum |q k|; its scaling and the exponential: 2^-21 of
    its own size and 2^-21 more; a logit off by x moves the weights' share by at most 2 x A;
  - bf16, more than 16 rows per KV head: the query as two e4m3 parts, off by at most 2^-17 of the row's
    largest value per channel: scale * 2^-17 * max |q| * sum |k| on a logit;
  - the sums over keys: n/16 steps in the value product and the joins, each off by 2^-23 of A.
"""

import numpy as np
import pytest

from oracle import kv8

from .gpu_common import DEV, th, to_dev, torch, tq, wl

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, tq.TQ_BF16), "f32": (torch.float32, tq.TQ_F32)}
_CTX = {}


def ctx_for(d):
    if d not in _CTX:
        _CTX[d] = tq.tq_create_ex(tq.make_config(d=d, k_split=d // 64 * 32, v_split=d // 64 * 32))
    return _CTX[d]


def values(rng, dtype, *shape):
    x = rng.standard_normal(shape).astype(np.float32)
    return wl.bf16_round(x) if dtype == "bf16" else x


class Cache:
    """A pool on both sides, filled alike: random codes (NaN codes among them where nobody may look) and scales."""

    def __init__(self, rng, pages, h, d, batch, maxp, spread=3, nan=True):
        self.h, self.d, self.pages, self.maxp = h, d, pages, maxp
        self.codes, self.scales = {}, {}
        for kind in "kv":
            c = rng.integers(0, 256, (pages, h, 16, d)).astype(np.uint8)
            if not nan:
                c[(c & 127) == 127] = 0
            self.codes[kind] = c
            self.scales[kind] = np.exp2(rng.integers(-6 - spread, -5 + spread, (pages, h))).astype(np.float32)
        self.table = rng.permutation(pages)[:batch * maxp].reshape(batch, maxp).astype(np.int32)
        self.dev = None

    def clean(self, rng, b, positions):
        """Plain random values (no NaN codes) at the given positions of sequence b."""
        pos = np.asarray(positions)
        for kind in "kv":
            x = rng.standard_normal((pos.size, self.h, self.d)) * 60
            self.codes[kind][self.table[b, pos // 16], :, pos % 16] = kv8.e4m3_encode(x)

    def to_device(self):
        t = {k: to_dev(v) for k, v in (("kc", self.codes["k"]), ("vc", self.codes["v"]), ("ks", self.scales["k"]),
                                       ("vs", self.scales["v"]), ("bt", self.table))}
        self.dev = t
        self.desc = tq.make_kv8_cache(t["kc"], t["vc"], t["ks"], t["vs"], t["bt"], self.maxp, self.pages, self.h)
        return self.desc

    def same_as_device(self):
        for kind in "kv":
            got, want = self.dev[kind + "c"].cpu().numpy(), self.codes[kind]
            bad = np.argwhere(got != want)
            assert bad.size == 0, (kind, len(bad), bad[:4].tolist(), [(int(got[tuple(i)]), int(want[tuple(i)])) for i in bad[:4]])
            assert np.array_equal(self.dev[kind + "s"].cpu().numpy(), self.scales[kind]), kind


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def _table(rng, max_pos, rot):
    ang = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


def _append_case(rng, dtype, d, h, hq, starts, n_new, lens=None, rot=None, interleaved=False, sections=None, fused=False,
                 kinds="kvq", x=None, inplace=False, flags=0):
    b = len(starts)
    rot = d if rot is None else rot
    maxp = (max(starts) + n_new + 15) // 16 + 1
    c = Cache(rng, b * maxp + 2, h, d, b, maxp, nan=False)
    dt, code = DT[dtype]
    hosts = x or {"k": values(rng, dtype, b, n_new, h, d) * 5, "v": values(rng, dtype, b, n_new, h, d),
                  "q": values(rng, dtype, b, n_new, hq, d)}
    if dtype == "bf16":
        hosts = {k: wl.bf16_round(v) for k, v in hosts.items()}
    max_pos = max(starts) + n_new + 3
    cs = _table(rng, max_pos, rot) if rot else None
    pos = None
    if rot and sections:
        pos = rng.integers(0, max_pos, (len(sections), b, n_new)).astype(np.int32)
    desc = c.to_device()
    dev, strides = {}, {"k": 0, "v": 0, "q": 0}
    if fused:
        row = torch.cat([to_dev(hosts[k]).to(dt).flatten(2) for k in "qkv"], dim=-1).contiguous()
        at = 0
        for k, heads in (("q", hq), ("k", h), ("v", h)):
            dev[k] = row[..., at * d:(at + heads) * d]
            strides[k] = row.stride(1)
            at += heads
    else:
        dev = {k: to_dev(hosts[k]).to(dt) for k in "kvq"}
    q_out = dev["q"] if inplace else torch.full((b, n_new, hq, d), -7.0, dtype=dt, device=DEV)
    rope = tq.make_rope(to_dev(cs), max_pos, rot, interleaved, sections, None if pos is None else to_dev(pos)) if rot else None
    ctx = ctx_for(d)
    get = lambda k: dev[k] if k in kinds else None  # noqa: E731
    tq.tq_kv8_append(ctx, desc, get("k"), get("v"), get("q"), code, b, n_new, hq, to_dev(np.asarray(starts, np.int32)),
                     None if lens is None else to_dev(np.asarray(lens, np.int32)), rope, q_out if "q" in kinds else None,
                     strides["k"], strides["v"], strides["q"])
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == flags

    def turned(y, s, t):      # one token's heads, as fp64
        if not rot:
            return y.astype(np.float64)
        p = [starts[s] + t] if pos is None else pos[:, s, t]
        axis = np.repeat(np.arange(len(sections)), sections) if pos is not None else np.zeros(rot // 2, int)
        at = np.asarray(p)[axis]
        i = np.arange(rot // 2)
        return kv8.rotate(y.astype(np.float64), cs[at, i].astype(np.float64), cs[at, rot // 2 + i].astype(np.float64),
                          interleaved)

    got_q = q_out.float().cpu().numpy()
    for s in range(b):
        n = n_new if lens is None else lens[s]
        if n and "k" in kinds:
            kv8.append(c.codes["k"], c.scales["k"], c.table[s], starts[s],
                       np.stack([turned(hosts["k"][s, t], s, t) for t in range(n)]))
        if n and "v" in kinds:
            kv8.append(c.codes["v"], c.scales["v"], c.table[s], starts[s], hosts["v"][s, :n].astype(np.float64))
        if "q" in kinds:
            for t in range(n):
                want = turned(hosts["q"][s, t], s, t)
                # one rounding to the type, and fp32's two products and one sum before it
                size = np.abs(hosts["q"][s, t]).max(axis=-1, keepdims=True)
                tol = np.abs(want) * torch.finfo(dt).eps / 2 + 2.0 ** -22 * size
                assert np.all(np.abs(got_q[s, t] - want) <= tol), (s, t)
            if not inplace:
                assert np.all(got_q[s, n:] == -7.0)
    c.same_as_device()
    return c


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h,hq,starts,n_new,fused", [(2, 8, [0, 5, 16, 31], 1, False), (3, 3, [7], 1, True),
                                                     (1, 16, [0, 3, 15], 37, True), (8, 8, [33, 0], 16, False)])
def test_append(dtype, d, h, hq, starts, n_new, fused):
    rng = np.random.default_rng(3)
    _append_case(rng, dtype, d, h, hq, starts, n_new, fused=fused)


@pytest.mark.parametrize("d,rot,interleaved,sections", [(128, 128, True, None), (128, 64, False, None), (128, 32, True, None),
                                                        (128, 0, False, None), (128, 128, False, [16, 24, 24]),
                                                        (128, 128, False, [13, 50, 1]), (64, 32, True, [5, 11]),
                                                        (256, 240, False, [100, 0, 19, 1]), (64, 64, False, [32])])
def test_append_rotations(d, rot, interleaved, sections):
    rng = np.random.default_rng(4)
    _append_case(rng, "bf16", d, 2, 6, [4, 18], 21, rot=rot, interleaved=interleaved, sections=sections)
    _append_case(rng, "f32", d, 2, 6, [4, 18], 5, rot=rot, interleaved=interleaved, sections=sections, fused=True)


@pytest.mark.parametrize("kinds", ["k", "v", "q", "kv", "kq"])
def test_append_parts(kinds):
    _append_case(np.random.default_rng(5), "bf16", 128, 4, 8, [9, 0], 20, kinds=kinds)


def test_append_padded_batch_and_queries_in_place():
    rng = np.random.default_rng(6)
    _append_case(rng, "bf16", 128, 2, 4, [3, 16, 40, 0], 35, lens=[35, 0, 1, 17])
    _append_case(rng, "f32", 64, 2, 4, [3, 16], 35, inplace=True)


def test_append_unaligned_rows():
    """Token strides that are no multiple of 16 bytes, and a base that is not 16-byte aligned."""
    rng = np.random.default_rng(7)
    for dtype in ("bf16", "f32"):
        dt, code = DT[dtype]
        h, d, n = 2, 128, 19
        c = Cache(rng, 6, h, d, 1, 3, nan=False)
        desc = c.to_device()
        x = values(rng, dtype, 1, n, 1, h * d + 3)[:, :, 0]
        dev = to_dev(x).to(dt)
        k = dev[..., 1:1 + h * d]
        tq.tq_kv8_append(ctx_for(d), desc, k, k, None, code, 1, n, 0, to_dev(np.asarray([5], np.int32)), None, None, None,
                         k.stride(1), k.stride(1), 0)
        torch.cuda.synchronize()
        y = x[0, :, 1:1 + h * d].reshape(n, h, d).astype(np.float64)
        for kind in "kv":
            kv8.append(c.codes[kind], c.scales[kind], c.table[0], 5, y)
        c.same_as_device()


def test_append_ties_and_scale_borders():
    """Values half way between codes, maxima on a border (448 * 2^e exactly, and one step of the type above), and
    rotations whose exact results stand on ties (cosine 1/2, sine 1/2 in binary)."""
    rng = np.random.default_rng(8)
    h, d, n = 4, 128, 16
    ties = (kv8.VALUES[:126] + kv8.VALUES[1:127]) / 2
    x = rng.choice(np.concatenate([ties, -ties]), (1, n, h, d)).astype(np.float32)
    x[..., 5] = 448.0
    x[:, :, 1, 5] = 450.0                          # bf16 just above the border: the next scale
    x[:, :, 2] /= 2.0 ** 40
    x[:, :, 3] *= 2.0 ** 30
    c = Cache(rng, 4, h, d, 1, 2, nan=False)
    cs = np.full((64, d), 0.5, np.float32)
    desc = c.to_device()
    ctx = ctx_for(d)
    for dtype in ("f32", "bf16"):
        dt, code = DT[dtype]
        y = wl.bf16_round(x) if dtype == "bf16" else x
        dev = to_dev(y).to(dt)
        tq.tq_kv8_append(ctx, desc, dev, dev, None, code, 1, n, 0, to_dev(np.asarray([16], np.int32)), None,
                         tq.make_rope(to_dev(cs), 64, d), None)
        torch.cuda.synchronize()
        assert tq.tq_check_device_status(ctx) == 0
        half = np.full(d // 2, 0.5)
        kv8.append(c.codes["k"], c.scales["k"], c.table[0], 16, kv8.rotate(y[0].astype(np.float64), half, half, False))
        kv8.append(c.codes["v"], c.scales["v"], c.table[0], 16, y[0].astype(np.float64))
        c.same_as_device()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64), ("bf16", 256)])
def test_append_token_by_token_with_growth_rollback_and_reuse(dtype, d):
    """One token at a time, sizes up and down by 2^20 (blocks grow, old codes go down into the subnormals), then a
    rollback into the middle of a page, then the pages again for another sequence."""
    rng = np.random.default_rng(9)
    h = 2
    c = Cache(rng, 5, h, d, 1, 3, nan=False)
    desc = c.to_device()
    ctx = ctx_for(d)
    dt, code = DT[dtype]
    steps = list(range(0, 21)) + list(range(9, 24)) + list(range(0, 5))
    for p in steps:
        x = values(rng, dtype, 1, 1, h, d) * np.float32(2.0 ** rng.integers(-10, 11))
        dev = to_dev(x).to(dt)
        tq.tq_kv8_append(ctx, desc, dev, dev, None, code, 1, 1, 0, to_dev(np.asarray([p], np.int32)))
        torch.cuda.synchronize()
        for kind in "kv":
            kv8.append(c.codes[kind], c.scales[kind], c.table[0], p, x[0].astype(np.float64))
        c.same_as_device()
    assert tq.tq_check_device_status(ctx) == 0


def test_append_values_that_are_not_finite():
    rng = np.random.default_rng(10)
    h, d = 2, 128
    x = {"k": values(rng, "f32", 1, 20, h, d), "v": values(rng, "f32", 1, 20, h, d), "q": values(rng, "f32", 1, 20, 2, d)}
    x["v"][0, 3, 0, 7] = np.nan
    x["v"][0, 4, 0, 9] = np.inf
    x["v"][0, 17, 1, 100] = -np.inf
    x["v"][0, 18, 1, 1] = 3.3e38
    x["k"][0, 2, 1, 70] = np.nan                    # without a rotation: one channel
    _append_case(rng, "f32", d, h, 2, [6], 20, x=x, rot=0, flags=32)
    x["k"][0, 2, 1, 70] = 1e30
    x["v"] = values(rng, "f32", 1, 20, h, d) * 0    # blocks of zeros take the smallest scale
    _append_case(rng, "f32", d, h, 2, [6], 20, x=x, rot=0)
    x["k"][0, 5, 0, 3] = np.inf                     # with one: both of the pair
    c = _append_nonfinite_rotated(rng, x["k"])
    assert not np.isnan(kv8.VALUES[c]).any()


def _append_nonfinite_rotated(rng, k):
    h, d = k.shape[2:]
    c = Cache(rng, 4, h, d, 1, 2, nan=False)
    for kind in "kv":
        c.codes[kind][:] = 0
    desc = c.to_device()
    tq.tq_kv8_append(ctx_for(d), desc, to_dev(k), None, None, tq.TQ_F32, 1, 20, 0, to_dev(np.asarray([6], np.int32)), None,
                     tq.make_rope(to_dev(_table(rng, 64, d)), 64, d))
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx_for(d)) == 32
    return c.dev["kc"].cpu().numpy()


def test_append_skips_and_flags_what_is_out_of_range():
    rng = np.random.default_rng(11)
    h, d, dt = 2, 128, torch.bfloat16
    ctx = ctx_for(d)
    x = values(rng, "bf16", 3, 20, h, d)
    dev = to_dev(x).to(dt)
    c = Cache(rng, 8, h, d, 3, 2, nan=False)
    c.table[0, 1] = 8                               # no such page
    c.table[2, 0] = -1
    desc = c.to_device()
    tq.tq_kv8_append(ctx, desc, dev, dev, None, tq.TQ_BF16, 3, 20, 0, to_dev(np.asarray([0, 25, 12], np.int32)))
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == 1 | 2  # bad pages; positions 32 .. 44 behind the table
    for kind in "kv":
        kv8.append(c.codes[kind], c.scales[kind], c.table[0], 0, x[0, :16].astype(np.float64))
        kv8.append(c.codes[kind], c.scales[kind], c.table[1], 25, x[1, :7].astype(np.float64))
        kv8.append(c.codes[kind], c.scales[kind], c.table[2], 16, x[2, 4:20].astype(np.float64))
    c.same_as_device()
    # positions outside the cosines' table: those tokens are skipped, queries among them
    q_out = torch.full((1, 4, 2, d), -7.0, dtype=dt, device=DEV)
    pos = to_dev(np.asarray([[[0, 9, -1, 3]]], np.int32))
    before = c.dev["kc"].clone()
    tq.tq_kv8_append(ctx, desc, dev[:1, :4].contiguous(), None, dev[:1, :4].contiguous(), tq.TQ_BF16, 1, 4, 2,
                     to_dev(np.asarray([0], np.int32)), None, tq.make_rope(to_dev(_table(rng, 9, d)), 9, d, pos=pos), q_out)
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == 2
    after = c.dev["kc"]
    page = int(c.table[0, 0])
    assert torch.equal(before[page, :, 1:3], after[page, :, 1:3]) and not torch.equal(before[page, :, 0], after[page, :, 0])
    assert bool((q_out[0, 1:3] == -7).all()) and not bool((q_out[0, 0] == -7).all())
    # a start before the sequence and too many tokens
    tq.tq_kv8_append(ctx, desc, dev, dev, None, tq.TQ_BF16, 3, 20, 0, to_dev(np.asarray([-1, -30, -2], np.int32)))
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == 4
    assert torch.equal(after, c.dev["kc"])
    # an earlier block whose scale is none: taken as the smallest
    c.dev["ks"][c.table[0, 0].item()] = 3.0
    tq.tq_kv8_append(ctx, desc, dev[:1, :1].contiguous(), None, None, tq.TQ_BF16, 1, 1, 0,
                     to_dev(np.asarray([2], np.int32)))
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == 64


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _attend(c, q, dtype, causal, starts, lens=None, window=0, sinks=0, scale=None, max_len=None, stream=None, out=None):
    """starts: cached tokens with the query's own (decode) or before the queries (causal)."""
    dt, code = DT[dtype]
    d = c.d
    b, hq = q.shape[0], q.shape[-2]
    n_new = q.shape[1] if causal else 1
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    max_len = c.maxp * 16 if max_len is None else max_len
    ctx = ctx_for(d)
    n = tq.tq_kv8_workspace_size(ctx, b, n_new, hq, c.h, max_len)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full(q.shape, -7.0, dtype=dt, device=DEV) if out is None else out
    qd, ld = to_dev(q).to(dt), to_dev(np.asarray(starts, np.int32))
    if causal:
        tq.tq_kv8_causal_attention(ctx, c.desc, qd, code, b, n_new, hq, ld,
                                   None if lens is None else to_dev(np.asarray(lens, np.int32)), max_len, window, sinks,
                                   scale, out, ws, n, stream)
    else:
        tq.tq_kv8_decode_attention(ctx, c.desc, qd, code, b, hq, ld, max_len, window, sinks, scale, out, ws, n, stream)
    torch.cuda.synchronize()
    return out.float().cpu().numpy()


def _bound(dtype, want, mag, dots, n, d, scale, parts=0.0):
    eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    w = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
    logit = abs(scale) * (dots * ((d / 16 + 1) * 2.0 ** -23 + 2.0 ** -21) + parts) + 2.0 ** -21
    return np.abs(want) * eps + mag * (w + 2 * logit[:, None] + (n / 16 + 40) * 2.0 ** -23) * (1 + eps) + 1e-38


def _check(c, got, q, dtype, causal, starts, lens=None, window=0, sinks=0, scale=None, rows=None, hidden=None):
    d = c.d
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    for b, s in enumerate(starts):
        n = (q.shape[1] if lens is None else lens[b]) if causal else 1
        for t in range(n):
            if rows is not None and (b, t) not in rows:
                continue
            p = s + t if causal else s - 1
            x = q[b, t] if causal else q[b]
            want, mag, dots, ksum, keys = kv8.attention(x, c.codes["k"], c.scales["k"], c.codes["v"], c.scales["v"],
                                                        c.table[b], p, window, sinks, scale,
                                                        () if hidden is None else hidden.get(b, ()))
            y = got[b, t] if causal else got[b]
            two_parts = dtype == "bf16" and q[0].size // d // c.h > 16
            tol = _bound(dtype, want, mag, dots, keys, d, scale,
                         2.0 ** -17 * np.abs(x).max(axis=-1) * ksum if two_parts else 0.0)
            err = np.abs(y - want)
            assert np.all(err <= tol), (b, t, keys, float(np.nanmax(err / tol)), int(np.isnan(y).sum()))
        if causal:
            assert np.all(got[b, n:] == -7.0), b


def _seen(p, window, sinks):
    j = np.arange(p + 1)
    return j[kv8.visible(p, j, window, sinks)]


def _decode_case(rng, dtype, d, h, hq, lens, window=0, sinks=0, scale=None, spread=3, extra=1):
    b = len(lens)
    maxp = max(1, (max(lens) + 15) // 16 + extra)
    c = Cache(rng, b * maxp + 1, h, d, b, maxp, spread)
    for i, n in enumerate(lens):
        if n:
            c.clean(rng, i, _seen(n - 1, window, sinks))
    c.to_device()
    q = values(rng, dtype, b, hq, d)
    got = _attend(c, q, dtype, False, lens, window=window, sinks=sinks, scale=scale)
    assert tq.tq_check_device_status(ctx_for(d)) == 0
    _check(c, got, q, dtype, False, lens, window=window, sinks=sinks, scale=scale)
    return c, q, got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,h,hq", [(128, 2, 8), (128, 1, 40), (64, 3, 3), (256, 1, 5), (128, 1, 16), (128, 4, 28), (64, 1, 40), (256, 2, 24)])
def test_decode(dtype, d, h, hq):
    _decode_case(np.random.default_rng(20), dtype, d, h, hq, [1, 0, 15, 16, 17, 130, 301, 64])


@pytest.mark.parametrize("dtype,window,sinks", [("bf16", 1, 0), ("bf16", 16, 1), ("bf16", 17, 16), ("f32", 40, 20),
                                                ("bf16", 1000, 4), ("f32", 100, 0), ("bf16", 33, 300), ("bf16", 0, 5)])
def test_decode_window_and_sinks(dtype, window, sinks):
    """Everything outside the window and the first tokens holds NaN codes."""
    _decode_case(np.random.default_rng(21), dtype, 128, 2, 8, [1, 2, 16, 17, 18, 100, 333, 48], window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5, 3.0])
def test_decode_softmax_scales(dtype, scale):
    _decode_case(np.random.default_rng(22), dtype, 128, 2, 6, [70, 333], scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_block_scales_far_apart(dtype):
    """Scales from 2^-60 to 2^60 across pages: the value scale rides in the weights' exponents."""
    rng = np.random.default_rng(23)
    c = Cache(rng, 24, 2, 128, 1, 20)
    c.clean(rng, 0, range(310))
    c.scales["v"][:] = np.exp2(rng.integers(-60, 61, c.scales["v"].shape))
    c.scales["k"][:] = np.exp2(rng.integers(-40, -4, c.scales["k"].shape))
    c.to_device()
    q = values(rng, dtype, 1, 4, 128)
    q[0, 1] *= 2.0 ** -100
    q[0, 2] *= 2.0 ** 20
    q[0, 3] = 0
    _check(c, _attend(c, q, dtype, False, [310]), q, dtype, False, [310])


@pytest.mark.parametrize("dtype,d,h,hq,lens", [("bf16", 128, 8, 32, [9000]), ("f32", 128, 1, 4, [40000]),
                                               ("bf16", 64, 2, 4, [5000, 1, 12000]), ("bf16", 256, 2, 4, [20001])])
def test_decode_split_over_the_context(dtype, d, h, hq, lens):
    _decode_case(np.random.default_rng(24), dtype, d, h, hq, lens)


def test_decode_many_short_sequences():
    rng = np.random.default_rng(25)
    _decode_case(rng, "bf16", 128, 8, 16, [int(x) for x in rng.integers(0, 40, 420)])
    _decode_case(rng, "bf16", 64, 1, 2, [int(x) for x in rng.integers(0, 20, 2100)])
    # more sequences than a list holds, with one long context among them
    lens = [int(x) for x in rng.integers(0, 6, 2060)]
    lens[1234] = 2100
    b = len(lens)
    c = Cache(rng, b + 140, 1, 64, 1, 140, nan=False)
    c.table = np.zeros((b, 140), np.int32)
    c.table[:, 0] = np.arange(b)
    c.table[1234] = b + np.arange(140)
    c.maxp = 140
    for i, n in enumerate(lens):
        if n:
            c.clean(rng, i, range(n))
    c.to_device()
    q = values(rng, "bf16", b, 2, 64)
    _check(c, _attend(c, q, "bf16", False, lens), q, "bf16", False, lens)


def test_decode_query_that_is_not_finite_spoils_only_its_row():
    rng = np.random.default_rng(26)
    c = Cache(rng, 9, 1, 128, 1, 8)
    c.clean(rng, 0, range(100))
    c.to_device()
    q = values(rng, "f32", 1, 4, 128)
    q[0, 1, 5] = np.nan
    q[0, 2, 5] = np.inf
    got = _attend(c, q, "f32", False, [100])
    assert np.isnan(got[0, 1]).all() and np.isnan(got[0, 2]).all()
    keep = [0, 3]
    _check(c, got[:, keep], q[:, keep], "f32", False, [100])


def test_decode_bad_pages_and_lengths():
    rng = np.random.default_rng(27)
    lens = [100, 40, 16]
    c = Cache(rng, 30, 2, 128, 3, 8)
    for i, n in enumerate(lens):
        c.clean(rng, i, range(n))
    c.table[0, 2], c.table[0, 5], c.table[2, 0] = 30, -1, 1 << 30
    c.to_device()
    q = values(rng, "bf16", 3, 4, 128)
    got = _attend(c, q, "bf16", False, lens)
    ctx = ctx_for(128)
    assert tq.tq_check_device_status(ctx) == 1
    _check(c, got, q, "bf16", False, lens, hidden={0: [*range(32, 48), *range(80, 96)], 2: range(16)})
    assert np.all(got[2] == 0)
    # lengths: negative counts as empty, beyond max_seq_len or the table as cut
    got = _attend(c, q, "bf16", False, [-5, 41, 16], max_len=40)
    assert tq.tq_check_device_status(ctx) == 4 | 1
    assert np.all(got[0] == 0)
    want, mag, dots, _, n = kv8.attention(q[1], c.codes["k"], c.scales["k"], c.codes["v"], c.scales["v"], c.table[1], 39, 0, 0,
                                       1 / np.sqrt(128))
    assert np.all(np.abs(got[1] - want) <= _bound("bf16", want, mag, dots, n, 128, 1 / np.sqrt(128)))


def _causal_case(rng, dtype, d, h, hq, starts, n_new, lens=None, window=0, sinks=0, scale=None, rows=None):
    b = len(starts)
    real = [n_new] * b if lens is None else lens
    maxp = max(1, (max(s + n for s, n in zip(starts, real)) + 15) // 16 + 1)
    c = Cache(rng, b * maxp + 1, h, d, b, maxp)
    for i, (s, n) in enumerate(zip(starts, real)):
        if n:
            see = sorted(set().union(*[set(_seen(p, window, sinks).tolist()) for p in range(s, s + n)])) if window else range(s + n)
            c.clean(rng, i, list(see))
    c.to_device()
    q = values(rng, dtype, b, n_new, hq, d)
    got = _attend(c, q, dtype, True, starts, lens, window, sinks, scale)
    assert tq.tq_check_device_status(ctx_for(d)) == 0
    if rows is not None:
        rows = {(b_, int(t)) for b_ in range(b) for t in rng.integers(0, max(1, real[b_]), rows) if real[b_]}
        rows |= {(b_, t) for b_ in range(b) for t in (0, real[b_] - 1) if real[b_]}
    _check(c, got, q, dtype, True, starts, lens, window, sinks, scale, rows)
    return c, q, got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,h,hq,starts,n_new,lens", [(128, 2, 8, [0, 17, 100], 5, None), (128, 1, 4, [0, 31], 1, None),
                                                      (64, 2, 2, [3, 0, 50, 9], 33, [33, 0, 1, 20]),
                                                      (256, 1, 6, [10], 9, None), (128, 4, 28, [64, 0], 7, [7, 2]),
                                                      (128, 1, 12, [200], 3, None)])
def test_causal_few_rows(dtype, d, h, hq, starts, n_new, lens):
    _causal_case(np.random.default_rng(30), dtype, d, h, hq, starts, n_new, lens)


@pytest.mark.parametrize("dtype,window,sinks", [("bf16", 1, 0), ("f32", 7, 3), ("bf16", 24, 16), ("bf16", 200, 4), ("bf16", 16, 40)])
def test_causal_few_rows_window(dtype, window, sinks):
    _causal_case(np.random.default_rng(31), dtype, 128, 2, 6, [0, 40, 150], 5, None, window, sinks)


@pytest.mark.parametrize("dtype,d,h,hq,starts,n_new,lens,window,sinks", [
    ("bf16", 128, 2, 8, [0], 300, None, 0, 0), ("bf16", 128, 1, 4, [1000, 0], 200, [200, 77], 0, 0),
    ("bf16", 128, 2, 14, [130, 5, 0], 257, [257, 1, 128], 64, 4), ("bf16", 128, 1, 1, [31], 700, None, 100, 0),
    ("bf16", 128, 1, 4, [20000], 130, None, 0, 0), ("bf16", 128, 1, 5, [9], 513, None, 1, 1),
    ("f32", 128, 2, 4, [50], 200, None, 90, 3), ("bf16", 64, 1, 8, [77], 150, None, 0, 0), ("bf16", 64, 2, 6, [0, 1000, 5], 301, [301, 0, 99], 0, 0),
    ("bf16", 64, 3, 3, [40, 0], 333, [333, 200], 70, 20), ("bf16", 64, 1, 4, [9000], 40, None, 0, 0),
    ("f32", 256, 1, 2, [3], 100, None, 0, 0), ("bf16", 256, 2, 8, [0, 40], 150, [150, 31], 0, 0),
    ("bf16", 256, 1, 5, [700], 333, None, 200, 9), ("bf16", 256, 1, 1, [9000], 30, None, 0, 0), ("bf16", 256, 3, 12, [5], 37, None, 0, 0),
    ("bf16", 128, 8, 32, [0, 300], 160, None, 128, 17)])
def test_causal_many_rows(dtype, d, h, hq, starts, n_new, lens, window, sinks):
    _causal_case(np.random.default_rng(32), dtype, d, h, hq, starts, n_new, lens, window, sinks, rows=40)


@pytest.mark.parametrize("scale", [0.0, -0.08, 0.7])
def test_causal_softmax_scales(scale):
    _causal_case(np.random.default_rng(33), "bf16", 128, 2, 8, [60], 140, scale=scale, rows=40)


def test_causal_bad_pages_and_lengths():
    rng = np.random.default_rng(34)
    c = Cache(rng, 40, 2, 128, 2, 16)
    c.clean(rng, 0, range(230))
    c.clean(rng, 1, range(200))
    c.table[0, 3] = -7
    c.to_device()
    q = values(rng, "bf16", 2, 100, 8, 128)
    ctx = ctx_for(128)
    got = _attend(c, q, "bf16", True, [130, 100])
    assert tq.tq_check_device_status(ctx) == 1
    _check(c, got, q, "bf16", True, [130, 100], hidden={0: range(48, 64)}, rows={(0, 0), (0, 57), (0, 99), (1, 0), (1, 99)})
    # queries beyond max_seq_len and a padded count that is none are cut; rows that are not answered stay
    got = _attend(c, q, "bf16", True, [130, -3], lens=[1000, 5], max_len=200)
    assert tq.tq_check_device_status(ctx) == 4 | 1
    assert np.all(got[0, 70:] == -7) and np.all(got[1] == -7) and not np.any(np.all(got[0, :70] == -7, axis=-1))


def test_many_heads_per_kv_head():
    """More query heads per KV head than a block of query rows, in both forms, with windows and empty sequences."""
    for dtype, d, hq in (("bf16", 64, 300), ("f32", 64, 37), ("bf16", 128, 260), ("bf16", 256, 150)):
        _decode_case(np.random.default_rng(35), dtype, d, 1, hq, [20, 0, 333])
        _decode_case(np.random.default_rng(35), dtype, d, 1, hq, [20, 0, 333], 30, 5)
    _causal_case(np.random.default_rng(36), "bf16", 64, 1, 300, [100], 3)


def test_bounds_on_the_length_far_above_the_lengths():
    """max_seq_len up to the largest int: the work is not listed (its count passes 32 bits) but taken item by item."""
    rng = np.random.default_rng(37)
    lens = [int(x) for x in rng.integers(1, 300, 20)]
    c = Cache(rng, 20 * 20, 2, 128, 20, 20)
    for i, n in enumerate(lens):
        c.clean(rng, i, range(n))
    c.to_device()
    q = values(rng, "bf16", 20, 8, 128)
    for most in (320, 1 << 20, 2 ** 31 - 1):
        _check(c, _attend(c, q, "bf16", False, lens, max_len=most), q, "bf16", False, lens)
    q = values(rng, "bf16", 20, 9, 8, 128)
    starts = [max(n - 9, 0) for n in lens]
    new = [n - s for n, s in zip(lens, starts)]
    for most in (320, 2 ** 31 - 1):
        _check(c, _attend(c, q, "bf16", True, starts, new, max_len=most), q, "bf16", True, starts, new)


@pytest.mark.parametrize("causal", [False, True])
def test_output_on_a_16_byte_boundary(causal):
    rng = np.random.default_rng(38)
    c = Cache(rng, 20, 2, 128, 1, 20)
    c.clean(rng, 0, range(310))
    c.to_device()
    q = values(rng, "bf16", 1, 300, 8, 128) if causal else values(rng, "bf16", 1, 8, 128)
    room = torch.full((q.size + 16,), -7.0, dtype=torch.bfloat16, device=DEV)
    out = room[8:8 + q.size].view(q.shape)
    assert out.data_ptr() % 32 == 16
    got = _attend(c, q, "bf16", causal, [10] if causal else [310], out=out)
    _check(c, got, q, "bf16", causal, [10] if causal else [310], rows={(0, t) for t in (0, 1, 31, 127, 128, 299)})
    assert bool((room[:8] == -7).all()) and bool((room[8 + q.size:] == -7).all())


def test_pools_beyond_32_bit_offsets():
    """Codes of 4.4 GB each: a sequence's pages lie at both ends and in the middle."""
    rng = np.random.default_rng(39)
    h, d, pages, n = 8, 128, 270000, 330
    maxp = 21
    small = Cache(rng, maxp, h, d, 1, maxp)
    small.clean(rng, 0, range(n))
    far = np.concatenate([np.arange(7), 131068 + np.arange(7), pages - 7 + np.arange(7)])     # where its pages really are
    at = torch.from_numpy(far).to(DEV)
    t = {k: torch.empty(pages, h, 16, d, dtype=torch.uint8, device=DEV) for k in ("kc", "vc")}
    t.update({k: torch.empty(pages, h, dtype=torch.float32, device=DEV) for k in ("ks", "vs")})
    for kind in "kv":
        t[kind + "c"][at] = to_dev(small.codes[kind])
        t[kind + "s"][at] = to_dev(small.scales[kind])
    t["bt"] = to_dev(far[small.table].astype(np.int32))
    small.dev = t
    small.desc = tq.make_kv8_cache(t["kc"], t["vc"], t["ks"], t["vs"], t["bt"], maxp, pages, h)
    q = values(rng, "bf16", 1, 32, d)
    _check(small, _attend(small, q, "bf16", False, [n]), q, "bf16", False, [n])
    q = values(rng, "bf16", 1, 40, 32, d)
    _check(small, _attend(small, q, "bf16", True, [n - 40]), q, "bf16", True, [n - 40], rows={(0, 0), (0, 39)})
    x = values(rng, "bf16", 1, n - 40, h, d)
    dev = to_dev(x).to(torch.bfloat16)
    tq.tq_kv8_append(ctx_for(d), small.desc, dev, dev, None, tq.TQ_BF16, 1, n - 40, 0, to_dev(np.asarray([0], np.int32)))
    torch.cuda.synchronize()
    for kind in "kv":
        kv8.append(small.codes[kind], small.scales[kind], small.table[0], 0, x[0].astype(np.float64))
        assert np.array_equal(t[kind + "c"][at].cpu().numpy(), small.codes[kind])
        assert np.array_equal(t[kind + "s"][at].cpu().numpy(), small.scales[kind])


def test_pages_shared_by_sequences_and_seen_twice():
    rng = np.random.default_rng(43)
    c = Cache(rng, 30, 2, 128, 3, 10, nan=False)
    c.table = np.asarray([[0, 1, 2, 3, 4, 5, 6, 7, 8, 9], [0, 1, 2, 3, 10, 11, 4, 5, 0, 0], [7, 7, 7, 7, 7, 7, 7, 7, 7, 7]], np.int32)
    for b in range(3):
        c.clean(rng, b, range(160))
    c.to_device()
    for dtype in ("bf16", "f32"):
        q = values(rng, dtype, 3, 8, 128)
        _check(c, _attend(c, q, dtype, False, [160, 155, 130]), q, dtype, False, [160, 155, 130])
        q = values(rng, dtype, 3, 20, 8, 128)
        _check(c, _attend(c, q, dtype, True, [140, 100, 3]), q, dtype, True, [140, 100, 3])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def _steps(dtype, d, h, hq, window, sinks, graph=False):
    """A prompt of each sequence, then single tokens, then five drafted ones: append + attention on one stream."""
    rng = np.random.default_rng(40)
    b, dt, code = 3, DT[dtype][0], DT[dtype][1]
    ctx = ctx_for(d)
    maxp = 14
    c = Cache(rng, b * maxp, h, d, b, maxp)
    desc = c.to_device()
    cs = _table(rng, 300, d)
    rope = tq.make_rope(to_dev(cs), 300, d)
    lens = np.asarray([0, 0, 0], np.int32)
    stream = torch.cuda.Stream()
    for n_new, new in ((150, [150, 97, 16]), (1, [1, 1, 1]), (1, [1, 1, 1]), (5, [5, 5, 5]), (1, [1, 1, 1])):
        x = {k: values(rng, dtype, b, n_new, hh, d) for k, hh in (("k", h), ("v", h), ("q", hq))}
        dev = {k: to_dev(v).to(dt) for k, v in x.items()}
        n = tq.tq_kv8_workspace_size(ctx, b, n_new, hq, h, 16 * maxp)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        q_rot = torch.zeros(b, n_new, hq, d, dtype=dt, device=DEV)
        out = torch.full((b, n_new, hq, d), -7.0, dtype=dt, device=DEV)
        start, cnt, after = to_dev(lens), to_dev(np.asarray(new, np.int32)), to_dev(lens + np.asarray(new, np.int32))
        torch.cuda.synchronize()

        def call(st):
            tq.tq_kv8_append(ctx, desc, dev["k"], dev["v"], dev["q"], code, b, n_new, hq, start, cnt, rope, q_rot, stream=st)
            if n_new == 1:
                tq.tq_kv8_decode_attention(ctx, desc, q_rot, code, b, hq, after, 16 * maxp, window, sinks, d ** -0.5, out, ws,
                                           n, st)
            else:
                tq.tq_kv8_causal_attention(ctx, desc, q_rot, code, b, n_new, hq, start, cnt, 16 * maxp, window, sinks,
                                           d ** -0.5, out, ws, n, st)

        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                call(torch.cuda.current_stream())
            out.fill_(-7.0)
            torch.cuda.synchronize()
            g.replay()
            g.replay()                      # a step again: the same positions, the same bytes
        else:
            call(stream)
        torch.cuda.synchronize()
        assert tq.tq_check_device_status(ctx) == 0
        got, q_got = out.float().cpu().numpy(), q_rot.float().cpu().numpy()
        for s in range(b):
            p0 = int(lens[s])
            ks = np.stack([kv8.rotate(x["k"][s, t].astype(np.float64), cs[p0 + t, :d // 2].astype(np.float64),
                                      cs[p0 + t, d // 2:].astype(np.float64), False) for t in range(new[s])])
            kv8.append(c.codes["k"], c.scales["k"], c.table[s], p0, ks)
            kv8.append(c.codes["v"], c.scales["v"], c.table[s], p0, x["v"][s, :new[s]].astype(np.float64))
        c.same_as_device()
        _check(c, got, q_got, dtype, True, [int(v) for v in lens], new, window, sinks)
        lens = lens + np.asarray(new, np.int32)


@pytest.mark.parametrize("dtype,d,h,hq,window,sinks", [("bf16", 128, 2, 8, 0, 0), ("bf16", 128, 1, 4, 40, 4),
                                                       ("f32", 64, 2, 4, 0, 0), ("bf16", 256, 1, 3, 33, 16)])
def test_prompt_then_steps_then_drafts(dtype, d, h, hq, window, sinks):
    _steps(dtype, d, h, hq, window, sinks)


def test_prompt_then_steps_then_drafts_captured():
    _steps("bf16", 128, 2, 8, 0, 0, graph=True)


def test_captured_graphs_share_a_workspace():
    """A decode step and a drafted step, captured once with one workspace between them and replayed in turn while the
    lengths on the device grow, with eager calls among them: what each would give alone."""
    rng = np.random.default_rng(44)
    h, hq, d, maxp = 2, 16, 128, 400
    c = Cache(rng, 2 * maxp, h, d, 2, maxp)
    for b in range(2):
        c.clean(rng, b, range(16 * maxp))
    c.to_device()
    ctx, dt = ctx_for(d), torch.bfloat16
    q = {1: values(rng, "bf16", 2, 1, hq, d), 4: values(rng, "bf16", 2, 4, hq, d)}
    dev = {t: to_dev(x).to(dt) for t, x in q.items()}
    out = {t: torch.empty(2, t, hq, d, dtype=dt, device=DEV) for t in q}
    n = max(tq.tq_kv8_workspace_size(ctx, 2, t, hq, h, 16 * maxp) for t in q)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    lens, starts = (torch.zeros(2, dtype=torch.int32, device=DEV) for _ in range(2))

    def call(t, st):
        if t == 1:
            tq.tq_kv8_decode_attention(ctx, c.desc, dev[1], tq.TQ_BF16, 2, hq, lens, 16 * maxp, 0, 0, d ** -0.5, out[1], ws, n, st)
        else:
            tq.tq_kv8_causal_attention(ctx, c.desc, dev[4], tq.TQ_BF16, 2, 4, hq, starts, None, 16 * maxp, 0, 0, d ** -0.5,
                                       out[4], ws, n, st)

    graphs, stream = {}, torch.cuda.Stream()
    torch.cuda.synchronize()
    for t in q:
        graphs[t] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[t], stream=stream):
            call(t, torch.cuda.current_stream())
    for now in ([6000, 3], [1, 5999], [40, 77], [6070, 6060]):
        lens.copy_(to_dev(np.asarray(now, np.int32)))
        starts.copy_(to_dev(np.asarray(now, np.int32)))
        for _ in range(3):
            graphs[1].replay()
            graphs[4].replay()
        call(1, torch.cuda.current_stream())
        graphs[4].replay()
        graphs[1].replay()
        call(4, torch.cuda.current_stream())
        torch.cuda.synchronize()
        _check(c, out[1].float().cpu().numpy(), q[1], "bf16", True, [x - 1 for x in now])
        _check(c, out[4].float().cpu().numpy(), q[4], "bf16", True, now)
    assert tq.tq_check_device_status(ctx) == 0


@pytest.mark.parametrize("dtype,d,h,hq", [("bf16", 128, 2, 8), ("bf16", 64, 1, 32), ("f32", 128, 2, 8)])
def test_steps_without_a_wait_between_them(dtype, d, h, hq):
    """Forty steps of append and attention enqueued one behind the other: each sees the tokens of those before it."""
    rng = np.random.default_rng(45)
    n, dt, code = 40, DT[dtype][0], DT[dtype][1]
    c = Cache(rng, 4, h, d, 1, 4, nan=False)
    desc = c.to_device()
    x = {k: values(rng, dtype, n, 1, 1, hh, d) for k, hh in (("k", h), ("v", h), ("q", hq))}
    dev = {k: to_dev(v).to(dt) for k, v in x.items()}
    q_rot = torch.empty(n, 1, 1, hq, d, dtype=dt, device=DEV)
    out = torch.empty(n, 1, hq, d, dtype=dt, device=DEV)
    at = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    size = tq.tq_kv8_workspace_size(ctx_for(d), 1, 1, hq, h, 64)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for i in range(n):
        tq.tq_kv8_append(ctx_for(d), desc, dev["k"][i], dev["v"][i], dev["q"][i], code, 1, 1, hq, at[i:i + 1], None, None, q_rot[i])
        tq.tq_kv8_decode_attention(ctx_for(d), desc, q_rot[i], code, 1, hq, at[i + 1:i + 2], 64, 0, 0, d ** -0.5, out[i], ws, size)
    torch.cuda.synchronize()
    got = out.float().cpu().numpy()
    for i in range(n):
        for kind in "kv":
            kv8.append(c.codes[kind], c.scales[kind], c.table[0], i, x[kind][i, 0].astype(np.float64))
        _check(c, got[i], x["q"][i, 0], dtype, False, [i + 1])
    c.same_as_device()


def test_results_repeat_bit_for_bit():
    rng = np.random.default_rng(41)
    c = Cache(rng, 700, 2, 128, 2, 300)
    c.clean(rng, 0, range(4700))
    c.clean(rng, 1, range(900))
    c.to_device()
    q = values(rng, "bf16", 2, 70, 8, 128)
    a = _attend(c, q, "bf16", True, [4600, 800])
    b = _attend(c, q, "bf16", True, [4600, 800])
    assert np.array_equal(a, b)
    a = _attend(c, q[:, 0], "bf16", False, [4700, 900])
    assert np.array_equal(a, _attend(c, q[:, 0], "bf16", False, [4700, 900]))


@pytest.mark.parametrize("dtype,d,h,hq,n_new,starts", [("f32", 128, 8, 32, 100, [100, 2000]), ("f32", 64, 8, 32, 50, [1500, 300]),
                                                       ("f32", 256, 4, 16, 20, [900, 2000]), ("bf16", 128, 8, 32, 4, [9000, 500, 4000]),
                                                       ("bf16", 256, 4, 8, 3, [5000, 70]), ("bf16", 64, 4, 16, 60, [2000, 100])])
def test_many_runs_give_the_same_bits(dtype, d, h, hq, n_new, starts):
    """Copies race with nothing: forty runs, and a sample of rows of each distinct result against the oracle."""
    rng = np.random.default_rng(46)
    b = len(starts)
    maxp = (max(starts) + n_new) // 16 + 2
    c = Cache(rng, b * maxp, h, d, b, maxp)
    for i, s in enumerate(starts):
        c.clean(rng, i, range(s + n_new))
    c.to_device()
    q = values(rng, dtype, b, n_new, hq, d)
    first = _attend(c, q, dtype, True, starts)
    _check(c, first, q, dtype, True, starts, rows={(i, t) for i in range(b) for t in (0, n_new // 2, n_new - 1)})
    for _ in range(40):
        assert np.array_equal(first, _attend(c, q, dtype, True, starts))
    assert tq.tq_check_device_status(ctx_for(d)) == 0


def test_two_streams_at_once():
    """Two calls that overlap on the GPU, each with its own workspace."""
    rng = np.random.default_rng(42)
    c = Cache(rng, 600, 4, 128, 1, 550)
    c.clean(rng, 0, range(8700))
    c.to_device()
    q = values(rng, "bf16", 1, 16, 128)
    want = _attend(c, q, "bf16", False, [8700])
    ctx, dt = ctx_for(128), torch.bfloat16
    n = tq.tq_kv8_workspace_size(ctx, 1, 1, 16, 4, 8800)
    qd, ld = to_dev(q).to(dt), to_dev(np.asarray([8700], np.int32))
    runs = [(torch.cuda.Stream(), torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty(1, 16, 128, dtype=dt, device=DEV))
            for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, ws, out in runs:
            tq.tq_kv8_decode_attention(ctx, c.desc, qd, tq.TQ_BF16, 1, 16, ld, 8800, 0, 0, 128 ** -0.5, out, ws, n, st)
    torch.cuda.synchronize()
    for _, _, out in runs:
        assert np.array_equal(out.float().cpu().numpy(), want)
