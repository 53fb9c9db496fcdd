"""Cases of what stands around a paged cache: attention over whole prompts (packed sequences of fresh keys and values),
reading the 2-4-bit and the 8-bit cache back into rows, and single-token attention of sequences that share a prefix.

``own`` false: the operators in plain torch operations; true: the library's calls (online_kv_cache_02_gb300.tq).
A page holds 16 tokens.  A block of the 2-4-bit cache is one KV head of one page, its fields one after the other
(codes, signs, norms); a block of the 8-bit cache is e4m3 codes with a power-of-two scale.
"""

import functools
import math

import numpy as np
import torch

own = False

PAGE = 16
M = 128                                    # projections of the keys' residual sketch
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _prompt(dtype, heads, kv_heads, d, seqs, q_lo, q_hi, past_lo=0, past_hi=0, window=0, sinks=0, fused=False):
    return dict(op="prompt", dtype=dtype, heads=heads, kv_heads=kv_heads, d=d, seqs=seqs, q_lo=q_lo, q_hi=q_hi,
                past_lo=past_lo, past_hi=past_hi, window=window, sinks=sinks, fused=fused)


def _read(dtype, kv_heads, d, batch, len_lo, len_hi, bits, start=0, gap=0):
    return dict(op="read", dtype=dtype, kv_heads=kv_heads, d=d, batch=batch, len_lo=len_lo, len_hi=len_hi,
                k_hi=bits[0], k_lo=bits[1], v_hi=bits[2], v_lo=bits[3], start=start, gap=gap)


def _read8(dtype, kv_heads, d, batch, len_lo, len_hi, start=0, gap=0):
    return dict(op="read8", dtype=dtype, kv_heads=kv_heads, d=d, batch=batch, len_lo=len_lo, len_hi=len_hi, start=start,
                gap=gap)


def _shared(dtype, heads, kv_heads, d, groups, size_lo, size_hi, prefix_lo, prefix_hi, tail_lo, tail_hi):
    return dict(op="shared", dtype=dtype, heads=heads, kv_heads=kv_heads, d=d, groups=groups, size_lo=size_lo,
                size_hi=size_hi, prefix_lo=prefix_lo, prefix_hi=prefix_hi, tail_lo=tail_lo, tail_hi=tail_hi)


def listed():
    return [
        # a question of a few words: the latency of the call
        dict(_prompt("bf16", 32, 8, 128, 1, 57, 57, fused=True), name="prompt_short"),
        # one long document
        dict(_prompt("bf16", 32, 8, 128, 1, 8192, 8192), name="prompt_long"),
        # a scheduler's batch: 24 prompts of very different lengths, slices of one fused projection
        dict(_prompt("bf16", 28, 4, 128, 24, 1, 2500, fused=True), name="prompt_packed"),
        # a sliding-window layer with a small head dimension, the first tokens visible
        dict(_prompt("bf16", 32, 8, 64, 3, 3001, 5000, window=1024, sinks=4), name="prompt_window"),
        # chunks of long prompts behind what was read back from a cache, a large head dimension
        dict(_prompt("bf16", 16, 4, 256, 2, 700, 1024, 9000, 15000), name="prompt_chunk"),
        # fp32 activations
        dict(_prompt("f32", 16, 8, 128, 3, 300, 1111), name="prompt_f32"),
        # the cache of eight conversations read back, 3.5-bit keys (with their sketch) and values
        dict(_read("bf16", 8, 128, 8, 16384, 16384, (4, 3, 4, 3)), name="read_context"),
        # parts of caches, 3-bit, into fp32 rows with room for new tokens behind each sequence
        dict(_read("f32", 4, 128, 5, 100, 999, (3, 3, 3, 3), start=333, gap=64), name="read_parts"),
        # the 8-bit cache of eight conversations read back
        dict(_read8("bf16", 8, 128, 8, 16384, 16384), name="read8_context"),
        # and a short part of it
        dict(_read8("f32", 8, 64, 3, 20, 150, start=77, gap=16), name="read8_parts"),
        # 64 answers sampled behind one long prompt
        dict(_shared("bf16", 32, 8, 128, 1, 64, 64, 32768, 32768, 20, 600), name="shared_samples"),
        # assistants with system prompts of their own: groups of requests, each with its conversation behind
        dict(_shared("bf16", 28, 4, 128, 3, 3, 17, 1000, 6000, 1, 1500), name="shared_groups"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "read", "read8", "shared", "shared"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    heads, kv_heads = rng.choice([(32, 8), (28, 4), (8, 1), (16, 8), (12, 12), (40, 8)])
    d = rng.choice([128, 128, 128, 64, 256])
    if op == "prompt":
        if rng.random() < 0.1:
            d = rng.choice([32, 96, 160])
        # (query, key) pairs times heads times channels; fp32 and other head dimensions run without tensor cores
        most = (1 << 36) if dtype == "bf16" and d in (64, 128, 256) else (1 << 32)
        n = _log_int(rng, 1, 8000)
        past = _log_int(rng, 1, 20000) if rng.random() < 0.4 else 0
        n = max(1, min(n, int(math.sqrt(most / (heads * d))), most // (heads * d * (past + 1))))
        seqs = min(_log_int(rng, 1, 32), max(1, most // (n * (n + past) * heads * d)))
        windowed = rng.random() < 0.3
        return _prompt(dtype, heads, kv_heads, d, seqs, max(1, n // rng.choice([1, 3, 50])), n, past // 2, past,
                       _log_int(rng, 64, 4096) if windowed else 0, rng.choice([0, 4, 17]) if windowed else 0,
                       past == 0 and rng.random() < 0.5)
    if op in ("read", "read8"):
        if op == "read":
            # other head dimensions than 128 run without tensor cores
            d = rng.choice([128, 128, 128, 128, 64])
        hi = _log_int(rng, 1, 16384)
        most = (1 << 27) if d == 128 or op == "read8" else (1 << 23)      # values
        batch = max(1, min(_log_int(rng, 1, 64), most // (hi * kv_heads * d)))
        hi = min(hi, max(1, most // (batch * kv_heads * d)))
        start, gap = rng.choice([0, 0, rng.randrange(1, 500)]), rng.choice([0, 0, rng.randrange(1, 100)])
        lo = max(1, hi // rng.choice([1, 2, 10]))
        if op == "read8":
            return _read8(dtype, kv_heads, d, batch, lo, hi, start, gap)
        bits = rng.choice([(4, 3, 4, 3), (3, 3, 3, 3), (3, 2, 3, 2), (4, 4, 4, 4), (2, 2, 2, 2), (4, 4, 2, 2)])
        return _read(dtype, kv_heads, d, batch, lo, hi, bits, start, gap)
    groups = _log_int(rng, 1, 6)
    prefix, tail = _log_int(rng, 64, 32768), _log_int(rng, 1, 3000)
    most = (1 << 30) if dtype == "bf16" else (1 << 28)     # rows times keys times channels
    size = max(1, min(_log_int(rng, 1, 64), most * 8 // (groups * (prefix + tail) * heads * d)))
    return _shared(dtype, heads, kv_heads, d, groups, max(1, size // rng.choice([1, 2, 5])), size,
                   max(16, prefix // rng.choice([1, 3])), prefix, max(1, tail // rng.choice([1, 10])), tail)


def _spread(lo, hi, n):
    """n numbers from lo to hi, not in order."""
    order = [(5 * i + 3) % n if n % 5 else i for i in range(n)]
    return [lo + (hi - lo) * i // (n - 1) if n > 1 else hi for i in order]


def _prompt_lens(case):
    """Queries and keys of each sequence."""
    new = _spread(case["q_lo"], case["q_hi"], case["seqs"])
    past = _spread(case["past_lo"], case["past_hi"], case["seqs"])[::-1]
    return new, [n + p for n, p in zip(new, past)]


def _shared_lens(case):
    """Sizes and prefixes of the groups, lengths of the sequences."""
    sizes = _spread(case["size_lo"], case["size_hi"], case["groups"])
    prefixes = [p // PAGE * PAGE for p in _spread(case["prefix_lo"], case["prefix_hi"], case["groups"])]
    tails = _spread(case["tail_lo"], case["tail_hi"], sum(sizes))
    lens, at = [], 0
    for s, p in zip(sizes, prefixes):
        lens += [p + t for t in tails[at:at + s]]
        at += s
    return sizes, prefixes, lens


def _visible(p, case):
    """Keys that the query at position p sees."""
    w, s = case["window"], case["sinks"]
    return p + 1 if not w or p < w else w + min(s, p + 1 - w)


def _code_bytes(hi, lo, d):
    split = d // 2
    return (hi * split + lo * (d - split)) // 8


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    d, h = case["d"], case["kv_heads"]
    if case["op"] == "prompt":
        new, keys = _prompt_lens(case)
        pairs = sum(_visible(p, case) for n, k in zip(new, keys) for p in range(k - n, k))
        seen = 0
        for n, k in zip(new, keys):
            first = max(0, k - n + 1 - case["window"]) if case["window"] else 0
            seen += k - first + min(first, case["sinks"])
        return {"bytes": (2 * sum(new) * case["heads"] + 2 * seen * h) * d * e, "flops": 4 * pairs * case["heads"] * d}
    if case["op"] == "shared":
        sizes, prefixes, lens = _shared_lens(case)
        at, keys = 0, sum(prefixes)
        for s, p in zip(sizes, prefixes):
            keys += sum(n - p for n in lens[at:at + s])
            at += s
        return {"bytes": 2 * keys * h * d + 8 * h * keys // PAGE + 2 * len(lens) * case["heads"] * d * e,
                "flops": 4 * sum(lens) * case["heads"] * d}
    n = sum(_spread(case["len_lo"], case["len_hi"], case["batch"])) * h
    if case["op"] == "read8":
        return {"bytes": 2 * n * d * (1 + e) + 8 * n // PAGE, "flops": 2 * n * d}
    k = _code_bytes(case["k_hi"], case["k_lo"], d) + M // 8 + 4
    v = _code_bytes(case["v_hi"], case["v_lo"], d) + 2
    return {"bytes": n * (k + v + 2 * d * e), "flops": 2 * n * d * (2 * d + M)}


# ---------------------------------------------------------------------------
# the 2-4-bit method's tables, which every program of a context shares
# ---------------------------------------------------------------------------
def _normals(stream, n):
    """Standard normals of seed 0: SplitMix64 in counter form, Box-Muller pairs."""
    i = np.arange(1, n + 1, dtype=np.uint64)
    z = np.uint64(stream << 40) + i * np.uint64(0x9E3779B97F4A7C15)
    z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
    z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    z ^= z >> np.uint64(31)
    u = ((z >> np.uint64(11)).astype(np.float64) + 0.5) * 2.0 ** -53
    r, t = np.sqrt(-2.0 * np.log(u[0::2])), 2.0 * np.pi * u[1::2]
    return np.stack([r * np.cos(t), r * np.sin(t)], axis=1).ravel()


@functools.lru_cache(maxsize=None)
def _matrices(d):
    """The rotation (d x d) and the residual's projections (M x d), fp64 on the GPU."""
    q, r = np.linalg.qr(_normals(1, d * d).reshape(d, d))
    pi = q * np.sign(np.diag(r))[None, :]
    return torch.from_numpy(pi).cuda(), torch.from_numpy(_normals(2, M * d).reshape(M, d)).cuda()


@functools.lru_cache(maxsize=None)
def _centroids(bits):
    """Lloyd-Max centroids of N(0,1): each the mean of the density between the midpoints beside it."""
    a = (np.arange(1 << (bits - 1)) + 0.5) * 3.0 / (1 << (bits - 1))
    phi = lambda t: np.exp(-0.5 * t * t) / math.sqrt(2.0 * math.pi)  # noqa: E731
    erfc = np.vectorize(math.erfc)
    for _ in range(20000):
        lo = np.concatenate([[0.0], 0.5 * (a[:-1] + a[1:])])
        hi = np.concatenate([lo[1:], [40.0]])
        new = (phi(lo) - phi(hi)) / (0.5 * (erfc(lo / math.sqrt(2.0)) - erfc(hi / math.sqrt(2.0))))
        done = np.max(np.abs(new - a)) <= 1e-15
        a = new
        if done:
            break
    return np.concatenate([-a[::-1], a])


def _fields(hi, lo, d):
    """Of each channel: the stream bits of its stored value (low bit first), its width, and the value of each stored value."""
    split, out, base = d // 2, [], 0
    for bits, n in ((hi, split), (lo, d - split)):
        c = _centroids(bits)
        if bits == 4:          # sign and magnitude: the upper half's rank, or the lower half's from the middle down
            c = np.concatenate([c[15 - np.arange(8)][::-1], c[7 - np.arange(8)]])
        for i in range(n):
            if bits != 3:
                at = [base + bits * i + j for j in range(bits)]
            else:              # eight channels in 24 bits: six in the low bits of nibbles, two in the spare ones
                o, k = base + 24 * (i // 8), i % 8
                at = [o + 4 * k + j for j in range(3)] if k < 6 else [o + (3 if k == 6 else 7) + 8 * j for j in range(3)]
            out.append((at, c))
        base += bits * n
    return out


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _ends(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _table(gen, need):
    """A block table of sequences with so many pages each, and the pool's size."""
    pool = sum(need) + 3
    ids = torch.randperm(pool, generator=gen, device="cuda").int()
    table = torch.zeros(len(need), max(1, max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = ids[at:at + k]
        at += k
    return table, pool


def _cached_pages(gen, pages, h, d, outliers):
    """A pool of filled 8-bit blocks: codes [pages][h][16][d] and scales [pages][h]."""
    codes = torch.empty(pages, h, PAGE, d, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(pages, h, device="cuda")
    for p in range(0, pages, 16384):
        n = min(16384, pages - p)
        x = torch.randn(n, h, PAGE, d, generator=gen, device="cuda")
        x *= torch.exp2(torch.randint(-2, 2, (n, h, 1, 1), generator=gen, device="cuda").float())
        x[..., :outliers] *= 4
        m, e = torch.frexp(x.abs().amax(dim=(2, 3)))
        s = torch.exp2((e - 9 + (m > 0.875).int()).float())       # the smallest 2^e with |x| <= 448 * 2^e
        codes[p:p + n] = (x / s[..., None, None]).to(torch.float8_e4m3fn)
        scale[p:p + n] = s
    return codes, scale


def _records(gen, pages, h, code_bytes, key):
    """A pool of 2-4-bit blocks: any bits are codes and signs, norms about those of 128 normal channels with outliers."""
    n = pages * h
    codes = torch.randint(0, 256, (n, PAGE * code_bytes), generator=gen, device="cuda", dtype=torch.uint8)
    norm = (12.0 + 20.0 * torch.rand(n, PAGE, generator=gen, device="cuda")).half()
    if not key:
        return torch.cat([codes, norm.view(torch.uint8)], dim=1).flatten()
    signs = torch.randint(0, 256, (n, PAGE * M // 8), generator=gen, device="cuda", dtype=torch.uint8)
    rest = (norm.float() * (0.08 + 0.3 * torch.rand(n, PAGE, generator=gen, device="cuda"))).half()
    return torch.cat([codes, signs, norm.view(torch.uint8), rest.view(torch.uint8)], dim=1).flatten()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, d, h = DTYPES[case["dtype"]], case["d"], case["kv_heads"]
    st = dict(case=case, dtype=dt)
    if case["op"] == "prompt":
        hq = case["heads"]
        new, keys = _prompt_lens(case)
        tq, tk = sum(new), sum(keys)
        if case["fused"]:
            qkv = torch.randn(tq, (hq + 2 * h) * d, generator=gen, device="cuda").to(dt)
            q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([hq * d, h * d, h * d], dim=-1))
        else:
            q = torch.randn(tq, hq, d, generator=gen, device="cuda").to(dt)
            k, v = (torch.randn(tk, h, d, generator=gen, device="cuda").to(dt) for _ in range(2))
        k[..., :4] *= 4
        st.update(q=q, k=k, v=v, new=new, keys=keys, cu_q=_ints(_ends(new)), cu_k=_ints(_ends(keys)), tq=tq, tk=tk,
                  out=torch.zeros(tq, hq, d, dtype=dt, device="cuda"))
        return st
    if case["op"] == "shared":
        hq = case["heads"]
        sizes, prefixes, lens = _shared_lens(case)
        firsts = _ends(sizes)
        need = [(n + PAGE - 1) // PAGE for n in lens]
        for g, p in enumerate(prefixes):               # the first sequence brings the prefix's pages, the others share them
            for b in range(firsts[g] + 1, firsts[g + 1]):
                need[b] -= p // PAGE
        own_pages, pool = _table(gen, need)
        maxp = max((n + PAGE - 1) // PAGE for n in lens)
        table = torch.zeros(len(lens), maxp, dtype=torch.int32, device="cuda")
        for g, p in enumerate(prefixes):
            f = firsts[g]
            table[f, :need[f]] = own_pages[f, :need[f]]
            for b in range(f + 1, firsts[g + 1]):
                table[b, :p // PAGE] = own_pages[f, :p // PAGE]
                table[b, p // PAGE:p // PAGE + need[b]] = own_pages[b, :need[b]]
        kc, ks = _cached_pages(gen, pool, h, d, 4)
        vc, vs = _cached_pages(gen, pool, h, d, 0)
        st.update(kc=kc, ks=ks, vc=vc, vs=vs, table=table, maxp=maxp, pool=pool, sizes=sizes, prefixes=prefixes, lens=lens,
                  seq_lens=_ints(lens), group_start=_ints(firsts), prefix_lens=_ints(prefixes),
                  q=torch.randn(len(lens), hq, d, generator=gen, device="cuda").to(dt),
                  out=torch.zeros(len(lens), hq, d, dtype=dt, device="cuda"))
        return st
    lens = _spread(case["len_lo"], case["len_hi"], case["batch"])
    table, pool = _table(gen, [(case["start"] + n + PAGE - 1) // PAGE for n in lens])
    first = _ends([n + case["gap"] for n in lens])
    rows = first[-1]
    st.update(lens=lens, first=first[:-1], rows=rows, table=table, maxp=table.shape[1], pool=pool,
              start_pos=_ints([case["start"]] * len(lens)), dev_lens=_ints(lens), first_row=_ints(first[:-1]),
              k_out=torch.zeros(rows, h, d, dtype=dt, device="cuda"), v_out=torch.zeros(rows, h, d, dtype=dt, device="cuda"))
    if case["op"] == "read8":
        st["kc"], st["ks"] = _cached_pages(gen, pool, h, d, 4)
        st["vc"], st["vs"] = _cached_pages(gen, pool, h, d, 0)
        return st
    st["kc"] = _records(gen, pool, h, _code_bytes(case["k_hi"], case["k_lo"], d), True)
    st["vc"] = _records(gen, pool, h, _code_bytes(case["v_hi"], case["v_lo"], d), False)
    pi, s = _matrices(d)
    st.update(pi=pi, s=s, pi32=pi.float(), s32=s.float())
    for kind in "kv":
        fields = _fields(case[kind + "_hi"], case[kind + "_lo"], d)
        at = torch.tensor([(f[0] + [0] * 4)[:4] for f in fields], device="cuda")
        width = torch.tensor([len(f[0]) for f in fields], device="cuda")
        value = torch.tensor(np.stack([np.resize(f[1], 16) for f in fields]), device="cuda")
        st[kind + "_fields"] = (at, width, value)
    return st


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _handle(d, k_bits, v_bits):
    from online_kv_cache_02_gb300 import tq
    return tq, tq.tq_create_ex(tq.make_config(k_bits=k_bits, v_bits=v_bits, m=M, seed=0, k_split=d // 2, v_split=d // 2, d=d))


def _plan(st):
    """What a program keeps: the context, the cache's descriptor and a workspace."""
    if "plan" not in st:
        c = st["case"]
        if c["op"] == "read":
            tq, ctx = _handle(c["d"], (c["k_hi"], c["k_lo"]), (c["v_hi"], c["v_lo"]))
        else:
            tq, ctx = _handle(c["d"], (3, 3), (3, 3)) if c["d"] % 64 == 0 else _odd_handle(c["d"])
        cache, size = None, 0
        if c["op"] in ("read8", "shared"):
            cache = tq.make_kv8_cache(st["kc"], st["vc"], st["ks"], st["vs"], st["table"], st["maxp"], st["pool"], c["kv_heads"])
        if c["op"] == "prompt":
            size = tq.tq_prompt_workspace_size(ctx, c["seqs"], max(st["new"]), c["heads"], c["kv_heads"], max(st["keys"]))
        elif c["op"] == "shared":
            size = tq.tq_kv8_shared_workspace_size(ctx, len(st["lens"]), c["heads"], c["kv_heads"], c["groups"],
                                                   max(st["sizes"]), max(st["lens"]))
        ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
        st["plan"] = (tq, ctx, tq.TQ_BF16 if c["dtype"] == "bf16" else tq.TQ_F32, cache, ws, size)
    return st["plan"]


@functools.lru_cache(maxsize=None)
def _odd_handle(d):
    """A head dimension whose half is no multiple of 32: the context's default split."""
    from online_kv_cache_02_gb300 import tq
    return tq, tq.tq_create(d, 3, M, 0)


def _run_own(st):
    c = st["case"]
    tq, ctx, code, cache, ws, size = _plan(st)
    stream = torch.cuda.current_stream()
    h, d = c["kv_heads"], c["d"]
    if c["op"] == "prompt":
        row = (c["heads"] + 2 * h) * d if c["fused"] else 0      # elements from token to token
        tq.tq_prompt_attention(ctx, st["q"], st["k"], st["v"], code, c["seqs"], st["cu_q"], st["cu_k"], st["tq"], st["tk"],
                               max(st["new"]), max(st["keys"]), c["heads"], h, c["window"], c["sinks"], 1.0 / math.sqrt(d),
                               st["out"], ws, size, q_stride=row, k_stride=row, v_stride=row, stream=stream)
        return st["out"]
    if c["op"] == "shared":
        tq.tq_kv8_shared_decode_attention(ctx, cache, st["q"], code, len(st["lens"]), c["heads"], st["seq_lens"],
                                          max(st["lens"]), c["groups"], st["group_start"], st["prefix_lens"],
                                          max(st["sizes"]), 1.0 / math.sqrt(d), st["out"], ws, size, stream)
        return st["out"]
    if c["op"] == "read8":
        tq.tq_kv8_dequantize(ctx, cache, code, c["batch"], st["start_pos"], st["dev_lens"], max(st["lens"]), st["k_out"],
                             st["v_out"], st["first_row"], st["rows"], stream=stream)
    else:
        tq.tq_dequantize(ctx, st["kc"], st["vc"], code, c["batch"], h, st["start_pos"], st["dev_lens"], max(st["lens"]),
                         st["table"], st["maxp"], st["pool"], st["k_out"], st["v_out"], st["first_row"], st["rows"],
                         stream=stream)
    return {"k": st["k_out"], "v": st["v_out"]}


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _run_prompt(st):
    c = st["case"]
    h, g, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["d"]
    outs, aq, ak = [], 0, 0
    for n, m in zip(st["new"], st["keys"]):
        q, k, v = st["q"][aq:aq + n].float(), st["k"][ak:ak + m].float(), st["v"][ak:ak + m].float()
        aq, ak = aq + n, ak + m
        p = torch.arange(m - n, m, device=q.device)[:, None]
        j = torch.arange(m, device=q.device)
        seen = j <= p
        if c["window"]:
            seen &= (j > p - c["window"]) | (j < c["sinks"])
        rows = q.view(n, h, g, d).permute(1, 2, 0, 3)                                   # [h][g][n][d]
        s = (rows @ k.permute(1, 2, 0)[:, None]) * (1.0 / math.sqrt(d))
        s = s.masked_fill_(~seen, float("-inf"))
        s -= s.amax(-1, keepdim=True)
        s = s.exp_()
        o = (s @ v.transpose(0, 1)[:, None]) / s.sum(-1, keepdim=True)
        outs.append(o.permute(2, 0, 1, 3).reshape(n, h * g, d).to(st["dtype"]))
    return torch.cat(outs)


def _positions(st):
    """Sequence, position and output row of every token that is read."""
    n = st["dev_lens"].long()
    b = torch.repeat_interleave(torch.arange(len(st["lens"]), device=n.device), n, output_size=sum(st["lens"]))
    t = torch.arange(sum(st["lens"]), device=n.device) - (n.cumsum(0) - n)[b]
    return b, st["start_pos"].long()[b] + t, st["first_row"].long()[b] + t


def _run_read8(st):
    b, pos, row = _positions(st)
    ids, slot = st["table"].long()[b, pos // PAGE], pos % PAGE
    for kind in "kv":
        x = st[kind + "c"].view(torch.uint8)[ids, :, slot].view(torch.float8_e4m3fn).float() * st[kind + "s"][ids][..., None]
        st[kind + "_out"][row] = x.to(st["dtype"])
    return {"k": st["k_out"], "v": st["v_out"]}


def _stored(raw, fields):
    """Centroids [n][d] of code bytes raw [n][bytes]."""
    at, width, value = fields
    got = torch.zeros(raw.shape[0], at.shape[0], dtype=torch.int64, device=raw.device)
    for j in range(4):
        bit = (raw[:, at[:, j] // 8] >> (at[:, j] % 8).to(torch.uint8)) & 1
        got |= torch.where(j < width, bit.long(), 0) << j
    return value[torch.arange(at.shape[0], device=raw.device), got]


def _run_read(st):
    c = st["case"]
    d, h = c["d"], c["kv_heads"]
    b, pos, row = _positions(st)
    for kind in "kv":
        cb = _code_bytes(c[kind + "_hi"], c[kind + "_lo"], d)
        blocks = st[kind + "c"].view(st["pool"], h, -1)
        x_of = st[kind + "_out"]
        for i in range(0, len(pos), 1 << 15):                                           # what temporaries fit in
            bi, pi = b[i:i + (1 << 15)], pos[i:i + (1 << 15)]
            blk = blocks[st["table"].long()[bi, pi // PAGE]]                            # [n][h][block]
            slot = (pi % PAGE)[:, None, None].expand(-1, h, 1)

            def field(offset, width):
                at = offset + slot * width + torch.arange(width, device=blk.device)
                return torch.gather(blk, 2, at).flatten(0, 1)

            y = _stored(field(0, cb), st[kind + "_fields"]).float()
            after = PAGE * (cb + (M // 8 if kind == "k" else 0))
            norm = field(after, 2).contiguous().view(torch.half).float()
            x = (y @ st["pi32"]) * (norm / math.sqrt(d))
            if kind == "k":
                bits = field(PAGE * cb, M // 8)
                signs = ((bits[..., None] >> torch.arange(8, device=bits.device, dtype=torch.uint8)) & 1).flatten(1).float() * 2 - 1
                rest = field(after + 2 * PAGE, 2).contiguous().view(torch.half).float()
                x = x + ((signs @ st["s32"]) @ st["pi32"]) * (rest * (math.sqrt(math.pi / 2) / M))
            x_of[row[i:i + (1 << 15)]] = x.view(-1, h, d).to(st["dtype"])
    return {"k": st["k_out"], "v": st["v_out"]}


def _run_shared(st):
    c = st["case"]
    h, g, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["d"]
    gathered = lambda codes, scale, t: (  # noqa: E731
        codes.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * scale[t][..., None, None]).transpose(0, 1).flatten(1, 2)
    outs, at = [], 0
    for size, prefix in zip(st["sizes"], st["prefixes"]):
        shared = st["table"][at, :prefix // PAGE].long()
        kp, vp = gathered(st["kc"], st["ks"], shared), gathered(st["vc"], st["vs"], shared)      # [h][prefix][d]
        q = st["q"][at:at + size].float().view(size, h, g, d).transpose(0, 1) * (1.0 / math.sqrt(d))      # [h][size][g][d]
        s0 = (q.reshape(h, size * g, d) @ kp.mT).view(h, size, g, prefix)
        for i in range(size):
            n = st["lens"][at + i] - prefix
            tail = st["table"][at + i, prefix // PAGE:(st["lens"][at + i] + PAGE - 1) // PAGE].long()
            k, v = gathered(st["kc"], st["ks"], tail)[:, :n], gathered(st["vc"], st["vs"], tail)[:, :n]
            s = torch.cat([s0[:, i], q[:, i] @ k.mT], dim=-1)
            s = (s - s.amax(-1, keepdim=True)).exp()
            o = (s[..., :prefix] @ vp + s[..., prefix:] @ v) / s.sum(-1, keepdim=True)
            outs.append(o.reshape(h * g, d).to(st["dtype"]))
        at += size
    return torch.stack(outs)


def run(state):
    if own:
        return _run_own(state)
    return {"prompt": _run_prompt, "read": _run_read, "read8": _run_read8, "shared": _run_shared}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# 64 bits, from the definition
# ---------------------------------------------------------------------------
def _exact_prompt(case, seed):
    st = prepare(case, seed)
    new, keys = _prompt_lens(case)
    g, d = case["heads"] // case["kv_heads"], case["d"]
    out = st["out"].double()
    for i, (n, m) in enumerate(zip(new, keys)):
        fq, fk = sum(new[:i]), sum(keys[:i])
        for a in range(case["heads"]):
            k, v = st["k"][fk:fk + m, a // g].double(), st["v"][fk:fk + m, a // g].double()
            for r in range(0, n, 4096):
                q = st["q"][fq + r:fq + min(n, r + 4096), a].double()
                here = torch.arange(m - n + r, m - n + r + len(q), device="cuda")[:, None]
                there = torch.arange(m, device="cuda")[None]
                hidden = there > here
                if case["window"]:
                    hidden = hidden | ((here - there >= case["window"]) & (there >= case["sinks"]))
                w = torch.softmax(((q @ k.T) / math.sqrt(d)).masked_fill(hidden, float("-inf")), dim=-1)
                out[fq + r:fq + r + len(q), a] = w @ v
    return out


def _exact_read8(case, seed):
    st = prepare(case, seed)
    out = {"k": st["k_out"].double(), "v": st["v_out"].double()}
    for b, n in enumerate(st["lens"]):
        s, f = case["start"], st["first"][b]
        ids = st["table"][b, :(s + n + PAGE - 1) // PAGE].long()
        for kind in "kv":
            x = st[kind + "c"][ids].double() * st[kind + "s"][ids].double()[:, :, None, None]
            out[kind][f:f + n] = x.transpose(1, 2).reshape(-1, case["kv_heads"], case["d"])[s:s + n]
    return out


def _exact_read(case, seed):
    st = prepare(case, seed)
    d, h = case["d"], case["kv_heads"]
    out = {"k": st["k_out"].double(), "v": st["v_out"].double()}
    turn = {"k": torch.cat([st["pi"], (math.sqrt(math.pi / 2) / M) * (st["s"] @ st["pi"])]), "v": st["pi"]}
    for b, n in enumerate(st["lens"]):
        s, f = case["start"], st["first"][b]
        ids = st["table"][b, :(s + n + PAGE - 1) // PAGE].long()
        for kind in "kv":
            cb = _code_bytes(case[kind + "_hi"], case[kind + "_lo"], d)
            blk = st[kind + "c"].view(st["pool"], h, -1)[ids]                           # [pages][h][block]
            parts = [PAGE * cb] + ([PAGE * M // 8, 2 * PAGE, 2 * PAGE] if kind == "k" else [2 * PAGE])
            parts = blk.split(parts, dim=2)
            stream = parts[0].reshape(-1, cb)
            bits = torch.stack([(stream >> j) & 1 for j in range(8)], dim=-1).flatten(1)
            y = torch.empty(len(stream), d, dtype=torch.float64, device="cuda")
            for ch, (at, values) in enumerate(_fields(case[kind + "_hi"], case[kind + "_lo"], d)):
                number = sum(bits[:, p].long() << j for j, p in enumerate(at))
                y[:, ch] = torch.from_numpy(values).cuda()[number]
            norm = parts[-1 if kind == "v" else 2].contiguous().view(torch.half).double().reshape(-1, 1)
            y = y * norm / math.sqrt(d)
            if kind == "k":
                raw = parts[1].reshape(-1, M // 8)
                sign = torch.stack([(raw >> j) & 1 for j in range(8)], dim=-1).flatten(1).double() * 2 - 1
                y = torch.cat([y, sign * parts[3].contiguous().view(torch.half).double().reshape(-1, 1)], dim=1)
            x = (y @ turn[kind]).view(len(ids), h, PAGE, d).transpose(1, 2).reshape(-1, h, d)
            out[kind][f:f + n] = x[s:s + n]
    return out


def _exact_shared(case, seed):
    st = prepare(case, seed)
    h, g, d = case["kv_heads"], case["heads"] // case["kv_heads"], case["d"]
    out = st["out"].double()
    for b, n in enumerate(st["lens"]):
        ids = st["table"][b, :(n + PAGE - 1) // PAGE].long()
        k, v = ((st[x + "c"][ids].double() * st[x + "s"][ids].double()[:, :, None, None]).transpose(0, 1).reshape(h, -1, d)[:, :n]
                for x in "kv")
        q = st["q"][b].double().view(h, g, d)
        out[b] = (torch.softmax((q @ k.mT) / math.sqrt(d), dim=-1) @ v).reshape(h * g, d)
    return out


def exact(case, seed):
    return {"prompt": _exact_prompt, "read": _exact_read, "read8": _exact_read8, "shared": _exact_shared}[case["op"]](case, seed)
