"""Decode attention of sequences that share a prefix, over the 8-bit cache, against plain attention in 64 bits.

Bounds per output element, with A = sum_j w_j |v_j| and n keys:
  - half a step of the output's type;
  - a logit's fp32 sum over d channels (2^-23 a step where a tensor core cuts it, adding up like the root of the steps,
    counted eight times), its scaling and exponential (2^-21 of its size and 2^-21), a logit off by x counting 2 x A;
  - bf16 queries on tcgen05 as two e4m3 parts: 2^-17 of the row's largest value per channel, scale * 2^-17 max|q| sum|k|;
  - the weights as fp16, 2^-11 of each (fp32 inputs: in two parts, 2^-21);
  - the sums over keys, 2^-23 of A for each of sqrt(n) steps, counted eight times, and the join's 2^-20.
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
        _CTX[d] = tq.tq_create_ex(tq.make_config(d=d, k_split=d // 64 * 32, v_split=d // 64 * 32))
    return _CTX[d]


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


class Batch:
    """Groups of sequences with a prefix each, and pages of their own behind it; what no one may look at is NaN."""

    def __init__(self, seed, d, hq, h, sizes, prefixes, tails, dtype, spread=3):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.d, self.hq, self.h, self.dtype = d, hq, h, dtype
        self.sizes, self.prefixes = sizes, prefixes
        pages0 = [p // 16 for p in prefixes]
        self.lens = [16 * pages0[g] + t for g, t in zip(np.repeat(range(len(sizes)), sizes), tails)]
        b = len(self.lens)
        self.maxp = max(max((n + 15) // 16 for n in self.lens), max(pages0)) + 1
        pool = sum(pages0) + sum((t + 15) // 16 + 1 for t in tails) + 2
        ids = torch.randperm(pool, generator=gen, device=DEV).int().tolist()
        table = torch.full((b, self.maxp), pool, dtype=torch.int32)                 # (no such page)
        at = i = 0
        for g, n in enumerate(sizes):
            shared, at = ids[at:at + pages0[g]], at + pages0[g]
            for _ in range(n):
                own = (tails[i] + 15) // 16
                table[i, :pages0[g] + own] = torch.tensor(shared + ids[at:at + own], dtype=torch.int32)
                at += own
                i += 1
        self.table = table.to(DEV)
        rnd = torch.randn(2, pool, h, 16, d, generator=gen, device=DEV) * 60
        self.codes = rnd.clamp(-448, 448).to(torch.float8_e4m3fn)
        self.scale = torch.exp2(torch.randint(-7 - spread, -5 + spread, (2, pool, h), generator=gen, device=DEV).float())
        for i, n in enumerate(self.lens):                                           # slots behind the ends
            if n % 16 and n > 0:
                self.codes[:, self.table[i, n // 16].item(), :, n % 16:].view(torch.uint8)[...] = 0x7F
        self.pool = pool
        self.q = torch.randn(b, hq, d, generator=gen, device=DEV).to(DT[dtype][0])
        self.cache = tq.make_kv8_cache(self.codes[0], self.codes[1], self.scale[0], self.scale[1], self.table, self.maxp, pool, h)
        self.starts = np.concatenate([[0], np.cumsum(sizes)]).tolist()

    def run(self, scale=None, flags=0, out=None, prefix_lens=None, starts=None, lens=None, q=None, max_group=None, ws=None, stream=None):
        ctx = ctx_for(self.d)
        b, groups = len(self.lens), len(self.sizes)
        scale = self.d ** -0.5 if scale is None else scale
        max_len = max(max(self.lens), max(self.prefixes))
        g = max(self.sizes) if max_group is None else max_group
        size = tq.tq_kv8_shared_workspace_size(ctx, b, self.hq, self.h, groups, g, max_len)
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV) if ws is None else ws
        out = torch.full_like(self.q, -7.0) if out is None else out
        tq.tq_kv8_shared_decode_attention(ctx, self.cache, self.q if q is None else q, DT[self.dtype][1], b, self.hq,
                                          ints(self.lens if lens is None else lens), max_len, groups,
                                          ints(self.starts if starts is None else starts),
                                          ints(self.prefixes if prefix_lens is None else prefix_lens), g, scale, out, ws, size,
                                          torch.cuda.current_stream() if stream is None else stream)
        torch.cuda.synchronize()
        assert tq.tq_check_device_status(ctx) == flags
        return out

    def plain(self, scale=None, lens=None):
        """The same by the decode call, sequence by sequence."""
        ctx = ctx_for(self.d)
        lens = self.lens if lens is None else lens
        size = tq.tq_kv8_workspace_size(ctx, len(lens), 1, self.hq, self.h, max(lens))
        ws, out = torch.empty(max(16, size), dtype=torch.uint8, device=DEV), torch.empty_like(self.q)
        tq.tq_kv8_decode_attention(ctx, self.cache, self.q, DT[self.dtype][1], len(lens), self.hq, ints(lens), max(lens), 0, 0,
                                   self.d ** -0.5 if scale is None else scale, out, ws, size)
        torch.cuda.synchronize()
        assert tq.tq_check_device_status(ctx) == 0
        return out

    def check(self, got, scale=None, rows=None, lens=None):
        h, d, g = self.h, self.d, self.hq // self.h
        scale = d ** -0.5 if scale is None else scale
        dt = DT[self.dtype][0]
        for b, n in enumerate(self.lens if lens is None else lens):
            if rows is not None and b not in rows:
                continue
            if n == 0:
                assert bool((got[b] == 0).all())
                continue
            ids = self.table[b, :(n + 15) // 16].long()
            k, v = ((self.codes[x].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * self.scale[x][ids].double()[:, :, None, None])
                    .transpose(0, 1).reshape(h, -1, d)[:, :n] for x in (0, 1))
            q = self.q[b].double().view(h, g, d)
            s = q @ k.mT
            w = torch.softmax(s * scale, dim=-1)
            want, size = w @ v, w @ v.abs()
            e = abs(scale) * (8 * math.sqrt(d) * 2.0 ** -23 * (torch.sqrt((q ** 2) @ (k ** 2).mT) + s.abs()) + 2.0 ** -20 * s.abs())
            if self.dtype == "bf16":
                e = e + abs(scale) * 2.0 ** -17 * q.abs().amax(-1, keepdim=True) * k.abs().sum(-1)[:, None]
            e = e.amax(-1, keepdim=True)
            tol = size * (2 * e + (2.0 ** -11 if self.dtype == "bf16" else 2.0 ** -21) + 2.0 ** -20 + 8 * math.sqrt(n) * 2.0 ** -23)
            tol = tol + torch.finfo(dt).eps / 2 * (want.abs() + tol)
            over = ((got[b].double().view(h, g, d) - want).abs() / tol).max()
            assert float(over) <= 1.0, (b, n, float(over))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,hq,h", [(64, 8, 2), (128, 8, 2), (128, 7, 1), (256, 4, 2), (128, 3, 3), (64, 40, 2)])
def test_groups(dtype, d, hq, h):
    b = Batch(0, d, hq, h, [5, 1, 9, 3], [160, 0, 1000, 48], [1, 17, 16, 200, 33, 5] + list(range(1, 13)), dtype)
    b.check(b.run())


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 128)])
@pytest.mark.parametrize("size", [1, 2, 4, 5, 16, 31, 32, 33, 65, 130])
def test_group_sizes(dtype, d, size):
    """From one sequence to more rows than a block has (4 rows per sequence and KV head)."""
    b = Batch(size, d, 4, 1, [size], [333], [1 + 7 * i % 40 for i in range(size)], dtype)
    b.check(b.run(), rows=set(range(0, size, max(1, size // 8))) | {size - 1})


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64), ("bf16", 256)])
@pytest.mark.parametrize("prefix", [15, 16, 17, 127, 128, 144, 2048, 20000])
def test_prefix_lengths(dtype, d, prefix):
    """Whole pages are shared; from none to a prefix that many CTAs split."""
    b = Batch(prefix, d, 8, 2, [6], [prefix], [40, 1, 300, 16, 15, 2], dtype)
    b.check(b.run())


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 128), ("bf16", 64)])
def test_long_tails_and_empty_sequences(dtype, d):
    b = Batch(3, d, 8, 2, [7, 2], [64, 640], [9000, 1, 500, 5000, 3, 100, 70, 3000, 20], dtype)
    b.check(b.run())
    lens = list(b.lens)
    lens[2] = lens[7] = 0                             # empty places of a batch
    b.check(b.run(lens=lens), lens=lens)
    lens[4] = 64                                      # nothing behind the prefix
    b.check(b.run(lens=lens), lens=lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0, 3.0])
def test_softmax_scales(dtype, scale):
    b = Batch(4, 128, 8, 2, [12], [500], [30 * i + 1 for i in range(12)], dtype)
    b.check(b.run(scale=scale), scale=scale)


@pytest.mark.parametrize("dtype,d,hq", [("bf16", 128, 8), ("bf16", 256, 8), ("bf16", 64, 8), ("f32", 128, 8)])
def test_results_are_the_decodes(dtype, d, hq):
    """Within twice the bounds of each; and at scores beyond 2^16, where both keep the largest."""
    b = Batch(5, d, hq, 2, [10, 6], [1024, 96], [50 * i + 1 for i in range(16)], dtype)
    got, want = b.run(), b.plain()
    tol = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -18
    assert float((got.float() - want.float()).abs().max()) <= tol * float(want.float().abs().max())
    b.q *= 2.0 ** 12
    b.scale[0] *= 2.0 ** 10
    got, want = b.run(), b.plain()
    assert bool(torch.isfinite(got).all())
    assert float((got.float() - want.float()).abs().max()) <= tol * float(want.float().abs().max())


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64), ("bf16", 256)])
def test_results_in_the_queries_place(dtype, d):
    b = Batch(6, d, 8, 2, [9], [480], [3 + 20 * i for i in range(9)], dtype)
    want = b.run()
    q = b.q.clone()
    assert torch.equal(b.run(q=q, out=q), want)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_a_query_that_is_not_finite_spoils_only_its_row(dtype, d):
    b = Batch(7, d, 8, 2, [9, 3], [480, 64], [3 + 20 * i for i in range(12)], dtype)
    keep = b.q.clone()
    want = b.run()
    b.q[2, 3, 5], b.q[10, 0, 0] = math.nan, math.inf
    got = b.run()
    assert bool(torch.isnan(got[2, 3]).all()) and bool(torch.isnan(got[10, 0]).all())
    got[2, 3], got[10, 0] = want[2, 3], want[10, 0]
    b.q = keep
    b.check(got)                                      # (rows of a warp decide together when a maximum is taken)


def test_what_is_out_of_range_is_flagged():
    for dtype, hq in (("bf16", 8), ("f32", 8), ("bf16", 2)):
        b = Batch(8, 128, hq, 2, [6, 6], [320, 160], [20 + i for i in range(12)], dtype)
        good = b.run()
        # a bad page of the prefix is left out for its group, one of a tail for its sequence
        keep = b.table.clone()
        b.table[0, 3] = -5
        got = b.run(flags=1)
        assert torch.equal(got[6:], good[6:]) and bool(torch.isfinite(got).all()) and not torch.equal(got[:6], good[:6])
        b.table.copy_(keep)
        b.table[7, 10] = b.pool
        got = b.run(flags=1)
        ok = [i for i in range(12) if i != 7]
        assert torch.equal(got[ok], good[ok]) and bool(torch.isfinite(got).all())
        b.table.copy_(keep)
        # a sequence shorter than its group's prefix counts as that long
        lens = list(b.lens)
        lens[2] = 100
        got = b.run(lens=lens, flags=4)
        ok = [i for i in range(12) if i != 2]
        lens[2] = 320
        assert torch.equal(got[ok], good[ok])
        b.check(got, lens=lens)
        # a negative length: zeros
        lens = list(b.lens)
        lens[2] = -1
        got = b.run(lens=lens, flags=4)
        assert bool((got[2] == 0).all()) and torch.equal(got[[0, 1] + list(range(3, 12))], good[[0, 1] + list(range(3, 12))])
        # starts that are no list: those groups share nothing, and results stay right
        for starts in ([0, 20, 12], [0, 6, 13], [-1, 6, 12], [3, 6, 12]):
            got = b.run(starts=starts, flags=4)
            b.check(got)
        got = b.run(flags=4, max_group=5)                        # groups larger than stated
        b.check(got)
        got = b.run(prefix_lens=[-16, 160], flags=4)
        b.check(got)


@pytest.mark.parametrize("dtype,d,hq", [("bf16", 128, 8), ("f32", 64, 8), ("bf16", 256, 4)])
def test_groups_that_overlap_share_nothing_twice(dtype, d, hq):
    """Starts that fall put sequences into two groups: one of them at most shares its pages, and every result is right."""
    b = Batch(15, d, hq, 2, [6, 0, 6], [320, 0, 160], [20 + i for i in range(12)], dtype)
    for starts, prefixes in (([0, 6, 0, 6], [320, 0, 160]), ([0, 6, 0, 6], [160, 0, 320]), ([0, 6, 2, 12], [320, 0, 0])):
        for _ in range(5):
            b.check(b.run(starts=starts, prefix_lens=prefixes, flags=4))
    b = Batch(16, d, hq, 2, [8, 0, 8], [320, 0, 160], [20 + i for i in range(16)], dtype)
    for _ in range(5):
        b.check(b.run(starts=[0, 8, 4, 8], prefix_lens=[320, 0, 160], flags=4))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64), ("bf16", 256)])
def test_a_workspace_may_hold_anything(dtype, d):
    """Also what looks like the records of other items."""
    b = Batch(17, d, 8, 2, [9, 1, 20], [3000, 0, 500], [1 + 40 * i for i in range(30)], dtype)
    want = b.run()
    b.check(want)
    for fill in (0, 1, 0x7F, None):
        size = 1 << 26
        ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device=DEV) if fill is None else torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(b.run(ws=ws), want)


def test_prefix_beyond_the_table_is_cut():
    b = Batch(9, 128, 8, 2, [6], [320], [20 + i for i in range(6)], "bf16")
    got = b.run(prefix_lens=[1 << 30], flags=4)          # to the 21 whole pages of the longest sequence, all of the first's
    b.check(got, rows={0})
    assert bool(torch.isfinite(got).all())


@pytest.mark.parametrize("dtype,d,hq", [("bf16", 128, 8), ("f32", 128, 8), ("bf16", 64, 8), ("bf16", 256, 4)])
def test_results_repeat_bit_for_bit(dtype, d, hq):
    b = Batch(10, d, hq, 2, [20, 3], [3000, 500], [1 + 30 * i for i in range(23)], dtype)
    want = b.run()
    for _ in range(8):
        assert torch.equal(b.run(), want)


@pytest.mark.parametrize("dtype,d,hq,h", [("bf16", 64, 4, 1), ("bf16", 128, 32, 1), ("f32", 64, 4, 1)])
def test_many_groups(dtype, d, hq, h):
    """More groups than the list of spans holds."""
    rng = np.random.default_rng(13)
    sizes = rng.integers(1, 3, 2100).tolist()
    b = Batch(13, d, hq, h, sizes, rng.choice([0, 16, 32, 160], 2100).tolist(), rng.integers(1, 40, sum(sizes)).tolist(), dtype)
    b.check(b.run(), rows=set(range(0, sum(sizes), 37)) | {sum(sizes) - 1})


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_two_streams_at_once(dtype, d):
    """A workspace each."""
    b = Batch(14, d, 8, 2, [9, 4], [2000, 300], [1 + 40 * i for i in range(13)], dtype)
    want = b.run()
    ctx = ctx_for(d)
    max_len = max(b.lens)
    size = tq.tq_kv8_shared_workspace_size(ctx, 13, 8, 2, 2, 9, max_len)
    lens, starts, prefix = ints(b.lens), ints(b.starts), ints(b.prefixes)
    work = [(torch.cuda.Stream(), torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV), torch.zeros_like(b.q)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for stream, ws, out in work:
            tq.tq_kv8_shared_decode_attention(ctx, b.cache, b.q, DT[dtype][1], 13, 8, lens, max_len, 2, starts, prefix, 9, d ** -0.5, out, ws, size,
                                              stream)
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == 0
    assert all(torch.equal(out, want) for _, _, out in work)


def test_captured_and_replayed():
    """A step in a graph, replayed as lengths, prefixes and groups change, two graphs on one workspace."""
    b = Batch(11, 128, 8, 2, [8, 4], [640, 320], [100 + i for i in range(12)], "bf16")
    ctx = ctx_for(128)
    max_len = max(b.lens)
    size = tq.tq_kv8_shared_workspace_size(ctx, 12, 8, 2, 2, 12, max_len)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    lens, starts, prefix = ints(b.lens), ints(b.starts), ints(b.prefixes)
    outs = [torch.zeros_like(b.q) for _ in range(2)]
    graphs = []
    for scale, out in zip((0.05, 0.02), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tq.tq_kv8_shared_decode_attention(ctx, b.cache, b.q, tq.TQ_BF16, 12, 8, lens, max_len, 2, starts, prefix, 12, scale, out, ws,
                                              size, torch.cuda.current_stream())
        graphs.append(g)
    for s, p, cut in (([0, 8, 12], [640, 320], 0), ([0, 8, 12], [160, 0], 7), ([0, 8, 12], [639, 321], 20), ([0, 5, 8], [640, 640], 3)):
        now = [n - cut for n in b.lens]
        lens.copy_(ints(now))
        starts.copy_(ints(s))
        prefix.copy_(ints(p))
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        assert tq.tq_check_device_status(ctx) == (4 if s[-1] != 12 else 0)
        for scale, out in zip((0.05, 0.02), outs):
            b.check(out, scale=scale, lens=now)


def test_prompt_append_samples_and_read_back():
    """A prompt's exact attention, its append to the 8-bit cache, samples behind it, and the cache read back: the decode of
    each sample is the prompt attention over the rows that were read."""
    d, hq, h, n, samples = 128, 8, 2, 213, 6
    ctx = ctx_for(d)
    gen = torch.Generator(device=DEV).manual_seed(12)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV).bfloat16()  # noqa: E731
    shared, own_pages = n // 16, 2
    pool = (n + 15) // 16 + samples * own_pages
    kc, vc = (torch.zeros(pool, h, 16, d, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(pool, h, device=DEV) for _ in range(2))
    table = torch.zeros(samples, shared + own_pages, dtype=torch.int32, device=DEV)
    table[:, :shared] = torch.arange(shared, device=DEV, dtype=torch.int32)
    table[:, shared:] = shared + torch.arange(samples * own_pages, device=DEV, dtype=torch.int32).view(samples, own_pages)
    cache = tq.make_kv8_cache(kc, vc, ks, vs, table, shared + own_pages, pool, h)
    k, v, q = rnd(n, h, d), rnd(n, h, d), rnd(n, hq, d)
    # the prompt: attention, then its tokens into the first sample's pages, the last partial page into every sample's
    ws_n = tq.tq_prompt_workspace_size(ctx, 1, n, hq, h, n)
    ws, o = torch.zeros(ws_n, dtype=torch.uint8, device=DEV), torch.zeros_like(q)
    tq.tq_prompt_attention(ctx, q, k, v, tq.TQ_BF16, 1, ints([0, n]), ints([0, n]), n, n, n, n, hq, h, 0, 0, d ** -0.5, o, ws, ws_n)
    tq.tq_kv8_append(ctx, cache, k, v, None, tq.TQ_BF16, 1, n, 0, ints([0]))
    rest = n % 16
    many = lambda x: x[n - rest:].expand(samples, -1, -1, -1).contiguous()  # noqa: E731
    tq.tq_kv8_append(ctx, cache, many(k), many(v), None, tq.TQ_BF16, samples, rest, 0, ints([n - rest] * samples))
    for step in range(12):
        kn, vn, qn = rnd(samples, 1, h, d), rnd(samples, 1, h, d), rnd(samples, hq, d)
        tq.tq_kv8_append(ctx, cache, kn, vn, None, tq.TQ_BF16, samples, 1, 0, ints([n + step] * samples))
    L = n + 12
    size = tq.tq_kv8_shared_workspace_size(ctx, samples, hq, h, 1, samples, L)
    ws2, got = torch.zeros(size, dtype=torch.uint8, device=DEV), torch.zeros_like(qn)
    tq.tq_kv8_shared_decode_attention(ctx, cache, qn, tq.TQ_BF16, samples, hq, ints([L] * samples), L, 1, ints([0, samples]), ints([n]), samples,
                                      d ** -0.5, got, ws2, size)
    kr, vr = (torch.zeros(samples * L, h, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    tq.tq_kv8_dequantize(ctx, cache, tq.TQ_BF16, samples, ints([0] * samples), ints([L] * samples), L, kr, vr, ints(range(0, samples * L, L)), samples * L)
    ws_n = tq.tq_prompt_workspace_size(ctx, samples, 1, hq, h, L)
    ws3, want = torch.zeros(ws_n, dtype=torch.uint8, device=DEV), torch.zeros_like(qn)
    tq.tq_prompt_attention(ctx, qn, kr, vr, tq.TQ_BF16, samples, ints(range(samples + 1)), ints(range(0, samples * L + 1, L)), samples, samples * L,
                           1, L, hq, h, 0, 0, d ** -0.5, want, ws3, ws_n)
    torch.cuda.synchronize()
    assert tq.tq_check_device_status(ctx) == 0
    # both within 2^-8 of the weights and half a step of the result: 2^-8 each, of the largest
    assert float((got.float() - want.float()).abs().max()) <= 4 * 2.0 ** -8 * float(want.float().abs().max())
    # the stored keys and values differ from the fresh ones by half a step of e4m3, 2^-4, at most (or half a subnormal's)
    assert float((kr[:n].float() - k.float()).abs().max()) <= 2.0 ** -4 * float(k.float().abs().max())
    assert bool(torch.isfinite(o).all())
