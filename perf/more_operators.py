"""A long prompt that arrives in chunks, in a cache of bounded size: plain forms, calls, and cases to measure them by.

    rope     norms of queries and keys for each head, the position rotation and the append, in one pass (``qk_norm_rope``)
    chunk    attention of a chunk of new tokens of each sequence over the paged cache (``chunk_attn``)
    weight   the attention weight that each cached key collects from a chunk (``key_weights``)
    evict    the rows of most weight move to other pages, for each KV head (``kv_evict``)

``run`` computes the plain form in elementary torch operations; with ``own`` it
makes the library's calls.  Inputs come from the seed alone.  Pools are made by
quantizing normal rows under the block rules of ``include/memra.h``.
"""
import functools
import math

import numpy as np
import torch

own = False

PAGE = 16


def listed():
    return [
        # one decode token of one short request, with its log-sum-exp: latency
        dict(name="chunk_1_256", op="chunk", new="1", past="255", heads=8, kv_heads=2, dim=128, k="q8_0", v="q5_1",
             window=0, lse=True, pad=0),
        # continuous batching: one request's prompt goes in while fifteen others decode
        dict(name="chunk_mixed_512", op="chunk", new="1,1,1,1,1,512,1,1,1,1,1,1,1,1,1,1",
             past="4859,700,8191,6303,1,5120,2047,4095,333,7777,6303,16,3000,8000,4859,1500", heads=32, kv_heads=4,
             dim=128, k="q8_0", v="q5_1", window=0, lse=False, pad=3),
        # a chunk of a long document, deep in it
        dict(name="chunk_2048_32048", op="chunk", new="2048", past="30000", heads=32, kv_heads=4, dim=128, k="q8_0",
             v="q5_1", window=0, lse=False, pad=0),
        # wide heads with a sliding window over ring page tables, chunks of several requests
        dict(name="chunk_d256_window", op="chunk", new="700,1,257,512", past="6301,16001,512,0", heads=16, kv_heads=2,
             dim=256, k="fp8", v="fp8", window=1024, lse=True, pad=0),
        # eight sequences decode: their rows are normalized, rotated and stored
        dict(name="rope_8", op="rope", tokens=8, heads=32, kv_heads=4, dim=128, rotary=128, interleaved=False,
             norm=True, append=True),
        # a prompt whose rows prompt attention reads next: rotated keys come out as rows
        dict(name="rope_2048", op="rope", tokens=2048, heads=32, kv_heads=4, dim=128, rotary=128, interleaved=False,
             norm=True, append=False),
        # a large chunk of wide heads that rotate a quarter of their dims, stored as it passes
        dict(name="rope_16384_d256", op="rope", tokens=16384, heads=16, kv_heads=2, dim=256, rotary=64,
             interleaved=True, norm=True, append=True),
        # one decode step of eight sequences adds to what their keys have collected
        dict(name="weight_8x1_6316", op="weight", new="1,1,1,1,1,1,1,1",
             past="6315,6315,6315,6315,6315,6315,6315,6315", heads=32, kv_heads=4, dim=128, k="q8_0", v="q5_1",
             keep=1.0),
        # the last tokens of a long prompt weigh all of its keys
        dict(name="weight_64_262144", op="weight", new="64", past="262080", heads=32, kv_heads=4, dim=128, k="q8_0",
             v="q5_1", keep=0.0),
        # a short request is cut to half
        dict(name="evict_512", op="evict", lens="512", budgets="256", sink=4, recent=32, kv_heads=2, dim=128, k="q8_0",
             v="q5_1"),
        # a batch is cut to a common budget, some sequences below it
        dict(name="evict_16x8192", op="evict",
             lens="8192,4860,7001,2049,8191,1500,6304,8192,5120,31,8000,2048,7777,4096,6000,8100",
             budgets="2048,2048,2048,2048,2048,2048,2048,2048,1000,2048,2048,2048,2048,2048,2048,2048", sink=4,
             recent=128, kv_heads=4, dim=128, k="q8_0", v="q5_1"),
        # the longest context is cut to a sixteenth
        dict(name="evict_262144", op="evict", lens="262144", budgets="16384", sink=64, recent=1024, kv_heads=4,
             dim=128, k="q8_0", v="q5_1"),
    ]


PAIRS = (("q8_0", "q5_1"), ("q8_0", "q4_0"), ("fp8", "fp8"), ("nvfp4", "nvfp4"), ("fp8", "q5_1"), ("nvfp4", "q4_0"))
HEADS = ((8, 2), (32, 4), (16, 2), (4, 4), (12, 4), (8, 1), (40, 8), (24, 8))


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _commas(values):
    return ",".join(map(str, values))


def draw(rng):
    op = rng.choice(("chunk", "chunk", "rope", "weight", "evict"))
    dim = rng.choice((128, 256))
    heads, kv_heads = rng.choice(HEADS)
    k, v = rng.choice(PAIRS)
    if op == "rope":
        tokens = min(_log(rng, 1, 32768), 16384 * 20 * 256 // ((heads + 2 * kv_heads) * dim))
        return dict(op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim,
                    rotary=rng.choice((dim, dim // 2, dim // 4, 0)), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.7, append=rng.random() < 0.5)
    if op == "evict":
        n = _log(rng, 1, 32)
        lens = [_log(rng, 1, min(262144, 262144 * 4 * 128 // (n * kv_heads * dim))) for _ in range(n)]
        budget = _log(rng, 1, min(16384, max(lens)))
        return dict(op=op, lens=_commas(lens), budgets=_commas([rng.randint((budget + 1) // 2, budget) for _ in lens]),
                    sink=rng.choice((0, 1, 4, 33)), recent=rng.choice((0, 1, 16, 100)), kv_heads=kv_heads, dim=dim,
                    k=k, v=v)
    # the plain form holds the scores of the longest chunk over the longest context for every sequence
    n = _log(rng, 1, 16)
    past = [_log(rng, 1, 32768 if op == "chunk" else 262144) - 1 for _ in range(n)]
    room = 2 ** 38 // (n * heads * dim) if op == "chunk" else 2 ** 36 // (n * heads * dim)
    longest = max(1, min(2048, room // max(4096, max(past))))
    past = [min(p, max(0, room - longest)) for p in past]
    new = [1 if rng.random() < 0.4 else _log(rng, 1, longest) for _ in range(n)]
    case = dict(op=op, new=_commas(new), past=_commas(past), heads=heads, kv_heads=kv_heads, dim=dim, k=k, v=v)
    if op == "weight":
        return dict(case, keep=rng.choice((0.0, 0.5, 1.0)))
    return dict(case, window=rng.choice((0, 0, _log(rng, 1, 4096))), lse=rng.random() < 0.5, pad=rng.choice((0, 3)))


# --------------------------------------------------------- the pools' byte layout --

def _segment(fmt, dim):
    return {"q8_0": 17, "fp8": 16, "nvfp4": 9, "q5_1": 12, "q4_0": 9}[fmt] * dim


def _grid(dim):
    return np.meshgrid(np.arange(PAGE), np.arange(dim), indexing="ij")


def _places(fmt, side, dim):
    """Where the code of token t, element j of a page lies: (byte, shift), each [16, dim]."""
    t, j = _grid(dim)
    nb, b, r = dim // 32, j // 32, j % 32
    b16, r16 = j // 16, j % 16
    if side == "k" and fmt in ("q8_0", "fp8"):
        return ((t // 8 * (nb // 2) + b // 2) * 32 + 4 * (t % 8) + r // 8) * 16 + b % 2 * 8 + r % 8, np.zeros_like(t)
    if side == "k":
        e = r % 8
        w = 2 * b + e // 4
        return (w // 4 * 32 + 4 * (t % 8) + r // 8) * 16 + w % 4 * 4 + t // 8 + 2 * (e % 4 // 2), 4 * (e % 2)
    lane, h, k = 4 * (r // 4) + t % 8 // 2, r % 4 // 2, 2 * (t % 2) + t // 8
    if fmt == "fp8":
        return (b * 32 + lane) * 16 + 8 * h + 2 * (2 * (t // 8) + r % 2) + t % 2, np.zeros_like(t)
    if fmt == "nvfp4":
        lane = 4 * (r16 % 8) + t % 8 // 2
        return (b16 // 4 * 32 + lane) * 16 + b16 % 4 * 4 + t % 2 + 2 * (t // 8), 4 * (r16 // 8)
    return (b // 2 * 32 + lane) * 16 + b % 2 * 8 + 4 * h + k, 4 * (r % 2)


def _fifth(dim):
    """Where bit 4 of a q5_1 code lies: (byte, bit)."""
    t, j = _grid(dim)
    b, r = j // 32, j % 32
    lane = 4 * (r // 4) + t % 8 // 2
    return 8 * dim + (lane * (dim // 64) + b // 2) * 4 + 2 * (t % 2) + t // 8, 4 * (r % 2) + 2 * (b % 2) + r % 4 // 2


def _scales(fmt, side, dim):
    """First byte of the block scale of token t, block b: [16, blocks] (q5_1: the minimum lies dim bytes further)."""
    if fmt == "fp8":
        return None
    n = dim // (16 if fmt == "nvfp4" else 32)
    t, b = np.meshgrid(np.arange(PAGE), np.arange(n), indexing="ij")
    at = (t % 8 // 2 * n + b) * 4 + 2 * (t // 8) + t % 2
    if fmt == "nvfp4":
        return 8 * dim + (t * n + b if side == "k" else (t % 8 // 2 * n + b) * 4 + t % 2 + 2 * (t // 8))
    if fmt == "q8_0":
        return 16 * dim + (t * n + b) * 2
    return (10 if fmt == "q5_1" else 8) * dim + at * 2


def _token_bytes(fmt, side, dim):
    """The bytes that hold token t of a page, in the same order for every t: [16, segment / 16]."""
    parts = [np.sort(_places(fmt, side, dim)[0], 1)]
    if fmt == "q5_1":
        parts.append(np.sort(_fifth(dim)[0], 1))
    at = _scales(fmt, side, dim)
    for first in [] if at is None else [at] if fmt != "q5_1" else [at, at + dim]:
        parts += [first] if fmt == "nvfp4" else [first, first + 1]
    per = {"q8_0": 1, "fp8": 1, "nvfp4": 2, "q5_1": 2, "q4_0": 2}[fmt]
    parts[0] = parts[0][:, ::per]
    if fmt == "q5_1":
        parts[1] = parts[1][:, ::8]
    return np.concatenate(parts, 1)


@functools.lru_cache(None)
def _table_of(what, *args):
    """What one of the functions above says, as index tensors on the GPU (built once)."""
    got = what(*args)
    return tuple(torch.from_numpy(a).cuda() for a in got) if isinstance(got, tuple) else torch.from_numpy(got).cuda()


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


@functools.lru_cache(None)
def _e2m1_values(dtype):
    return torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda", dtype=dtype)


def _nearest_e2m1(x):
    """E2M1 codes of x, round to nearest, saturating."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    return torch.bucketize(x.abs(), mids).to(torch.uint8) | ((x < 0).to(torch.uint8) << 3)


def _pack(codes, byte, slot, first, n, bits):
    """Bytes first .. first + n - 1 of the segments: the codes [..., 16, dim] whose (byte, slot) lie there, ORed."""
    inverse = np.zeros((n, 8 // bits), np.int64)
    inverse[byte - first, slot // bits] = np.arange(byte.size).reshape(byte.shape)
    got = codes.flatten(-2)[..., torch.from_numpy(inverse).to(codes.device)]
    weight = torch.tensor([1 << (bits * i) for i in range(8 // bits)], device=codes.device, dtype=torch.int32)
    return (got.to(torch.int32) * weight).sum(-1).to(torch.uint8)


def _quantize(x, fmt, side):
    """Rows x [pages, heads, 16, dim] as pool bytes [pages, heads, segment], and the tensor scale."""
    dim = x.shape[-1]
    seg = torch.zeros(*x.shape[:2], _segment(fmt, dim), dtype=torch.uint8, device=x.device)
    byte, shift = _places(fmt, side, dim)
    scale = 1.0
    blocks = x.unflatten(-1, (-1, 16 if fmt == "nvfp4" else 32))
    top = blocks.abs().amax(-1, keepdim=True)
    if fmt == "fp8":
        scale = float(np.float32(x.abs().max().item() / 448))
        codes = (x / scale).to(torch.float8_e4m3fn).view(torch.uint8)
        seg[..., :16 * dim] = _pack(codes, byte, shift, 0, 16 * dim, 8)
        return seg, scale
    if fmt == "nvfp4":
        scale = float(np.float32(x.abs().max().item() / 2688))
        block = (top / (6 * scale)).to(torch.float8_e4m3fn)
        codes = _nearest_e2m1(blocks / (block.float() * scale).clamp_min(1e-30)).flatten(-2)
        seg[..., :8 * dim] = _pack(codes, byte, shift, 0, 8 * dim, 4)
        seg[..., _table_of(_scales, fmt, side, dim)] = block.squeeze(-1).view(torch.uint8)
        return seg, scale
    low = blocks.amin(-1, keepdim=True)
    d = {"q8_0": top / 127, "q4_0": top / 7, "q5_1": (blocks.amax(-1, keepdim=True) - low) / 31}[fmt].half()
    shifted = blocks - low if fmt == "q5_1" else blocks
    q = (shifted / d.float().clamp_min(1e-30)).round()
    bias, lo, hi = {"q8_0": (128, -127, 127), "q4_0": (8, -8, 7), "q5_1": (0, 0, 31)}[fmt]
    codes = (q.clamp(lo, hi) + bias).to(torch.uint8).flatten(-2)
    if fmt == "q8_0":
        seg[..., :16 * dim] = _pack(codes, byte, shift, 0, 16 * dim, 8)
    else:
        seg[..., :8 * dim] = _pack(codes & 15, byte, shift, 0, 8 * dim, 4)
    if fmt == "q5_1":
        fifth, bit = _fifth(dim)
        seg[..., 8 * dim:10 * dim] = _pack(codes >> 4, fifth, bit, 8 * dim, 2 * dim, 1)
        minimum = _table_of(_scales, fmt, side, dim) + dim
        halves = low.half().view(torch.uint8)
        seg[..., minimum], seg[..., minimum + 1] = halves[..., 0], halves[..., 1]
    first, halves = _table_of(_scales, fmt, side, dim), d.view(torch.uint8)
    seg[..., first], seg[..., first + 1] = halves[..., 0], halves[..., 1]
    return seg, scale


def _half_at(seg, first):
    return torch.stack((seg[..., first], seg[..., first + 1]), -1).view(torch.float16).squeeze(-1)


def _values(seg, fmt, side, dim, scale, dtype):
    """The values that segments [..., segment] stand for: [..., 16, dim] in `dtype`."""
    byte, shift = _table_of(_places, fmt, side, dim)
    code = seg[..., byte]
    if fmt == "fp8":
        return code.view(torch.float8_e4m3fn).to(dtype) * scale
    if fmt == "q8_0":
        q = code.to(dtype) - 128
    else:
        code = (code >> shift.to(torch.uint8)) & 15
        if fmt == "nvfp4":
            table = _e2m1_values(dtype)
            block = seg[..., _table_of(_scales, fmt, side, dim)].view(torch.float8_e4m3fn)
            return table[code.int()] * (block.to(dtype) * scale).repeat_interleave(16, -1)
        if fmt == "q5_1":
            fifth, bit = _table_of(_fifth, dim)
            code = code | (((seg[..., fifth] >> bit.to(torch.uint8)) & 1) << 4)
        q = code.to(dtype) - (8 if fmt == "q4_0" else 0)
    at = _table_of(_scales, fmt, side, dim)
    x = q * _half_at(seg, at).to(dtype).repeat_interleave(32, -1)
    return x + _half_at(seg, at + dim).to(dtype).repeat_interleave(32, -1) if fmt == "q5_1" else x


# ------------------------------------------------------------------------ states --

def _ints(text):
    return [int(n) for n in text.split(",")]


def _pools(case, pages, g):
    """A cache of `pages` pages of quantized normal rows: the K and V segments and their scales."""
    shape = (pages, case["kv_heads"], PAGE, case["dim"])
    k, ks = _quantize(torch.randn(shape, generator=g, device="cuda"), case["k"], "k")
    v, vs = _quantize(torch.randn(shape, generator=g, device="cuda"), case["v"], "v")
    return dict(k=k, v=v, k_scale=ks, v_scale=vs)


def _table(rng, columns, spare=2):
    """Page tables of `columns[b]` pages a sequence, drawn from a shuffled pool; and the pool's size."""
    pages = sum(columns) + spare
    table = np.zeros((len(columns), max(columns)), np.int32)
    table[np.arange(max(columns)) < np.array(columns)[:, None]] = rng.permutation(pages)[:sum(columns)]
    return table, pages


def _attended(case, g, rng):
    """What chunk attention and the key weights share: the cache, the packed queries and the lengths."""
    new, past = _ints(case["new"]), _ints(case["past"])
    lens, window = [n + p for n, p in zip(new, past)], case.get("window", 0)
    if window:
        table, pages = _table(rng, [(window + max(new) - 2) // PAGE + 2] * len(new))
    else:
        table, pages = _table(rng, [-(-n // PAGE) for n in lens])
    st = _pools(case, pages, g)
    total = sum(new) + case.get("pad", 0)
    starts = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    first = torch.tensor([max(0, p - window + 1) if window else 0 for p in past]).cuda()
    span = max(n - max(0, p - window + 1 if window else 0) for n, p in zip(lens, past))
    st.update(case=case, table=torch.from_numpy(table).cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda(),
              starts=starts, longest_new=max(new), longest=max(lens), first=first, span=span,
              q=torch.randn(total, case["heads"], case["dim"], generator=g, device="cuda").half())
    return st


def _chunk_state(case, g, rng):
    st = _attended(case, g, rng)
    st["out"] = torch.zeros_like(st["q"])
    st["lse"] = torch.zeros(st["q"].shape[:2], device="cuda") if case["lse"] else None
    # float32 partial rows of the splits of the keys: the call never needs more
    st["workspace"] = torch.empty(128 << 20, dtype=torch.uint8, device="cuda")
    return st


def _weight_state(case, g, rng):
    st = _attended(case, g, rng)
    s, _ = _scores(st)
    lse = torch.logsumexp(s, -1)                                   # [B, hk, group, n]
    rows, live = _chunk_rows(st)
    st["lse"] = torch.zeros(st["q"].shape[:2], device="cuda")
    st["lse"][rows[live]] = lse.permute(0, 3, 1, 2).flatten(2, 3)[live]
    shape = (len(st["lens"]), case["kv_heads"], st["longest"])
    st["weights"] = torch.rand(shape, generator=g, device="cuda") ** 4
    return st


def _rope_state(case, g, rng):
    n, dim, hq, hk = case["tokens"], case["dim"], case["heads"], case["kv_heads"]
    fused = torch.randn(n, hq + 2 * hk, dim, generator=g, device="cuda").half()
    st = dict(case=case, q=fused[:, :hq], k=fused[:, hq:hq + hk], v=fused[:, hq + hk:])
    first = rng.integers(0, 262144 - n)
    st["positions"] = torch.arange(first, first + n, dtype=torch.int32, device="cuda")
    half = case["rotary"] // 2
    freq = 1e6 ** (-np.arange(half) / max(1, half))
    st["inv_freq"] = torch.from_numpy(freq.astype(np.float32)).cuda() if half else None
    for side in ("q_weight", "k_weight"):
        st[side] = 1 + 0.1 * torch.randn(dim, generator=g, device="cuda") if case["norm"] else None
    st["q_out"] = torch.zeros(n, hq, dim, device="cuda").half()
    if case["append"]:
        pages = -(-n // PAGE) + 3
        st["k_scale"], st["v_scale"] = (float(np.float32(x / 448)) for x in (16.0, 6.0))
        st["k_pool"], st["v_pool"] = (torch.zeros(pages, hk, PAGE * dim, dtype=torch.uint8, device="cuda")
                                      for _ in range(2))
        slots = rng.permutation(pages)[:, None] * PAGE + np.arange(PAGE)
        st["slots"] = torch.from_numpy(slots.reshape(-1)[5:5 + n].astype(np.int32)).cuda()
    else:
        st["k_out"] = torch.zeros(n, hk, dim, device="cuda").half()
    return st


def _evict_state(case, g, rng):
    lens, budgets = _ints(case["lens"]), _ints(case["budgets"])
    used = [-(-n // PAGE) for n in lens]
    per = -(-max(budgets) // PAGE)
    table, pages = _table(rng, used, spare=per * len(lens))
    st = _pools(case, pages, g)
    free = np.setdiff1d(np.arange(pages), table[np.arange(max(used)) < np.array(used)[:, None]])
    shape = (len(lens), case["kv_heads"], max(lens))
    # a few keys collect most of the weight, some none at all
    weights = torch.rand(shape, generator=g, device="cuda") ** 8
    weights *= torch.rand(shape, generator=g, device="cuda") > 0.1
    st.update(case=case, table=torch.from_numpy(table).cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda(),
              longest=max(lens), weights=weights, budgets=torch.tensor(budgets, dtype=torch.int32).cuda(),
              most=max(budgets), to=torch.from_numpy(free.reshape(len(lens), per).astype(np.int32)).cuda(),
              kept=torch.zeros(len(lens), case["kv_heads"], max(budgets), dtype=torch.int32, device="cuda"),
              new_weights=torch.zeros(len(lens), case["kv_heads"], max(budgets), device="cuda"),
              new_lens=torch.zeros(len(lens), dtype=torch.int32, device="cuda"))
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    make = {"chunk": _chunk_state, "weight": _weight_state, "rope": _rope_state, "evict": _evict_state}
    return make[case["op"]](case, g, rng)


# ------------------------------------------------------------------------- plain --

def _chunk_rows(st):
    """[B, n]: the packed rows of each sequence's chunk, and which of them exist."""
    at = torch.arange(st["longest_new"], device="cuda")
    rows = (st["starts"][:-1, None].long() + at).clamp_max(st["q"].shape[0] - 1)
    return rows, at < st["starts"].diff()[:, None]


def _keys(st, side):
    """[B, hk, span, dim] float32: the cached rows from each sequence's first visible key on."""
    case = st["case"]
    at = st["first"][:, None] + torch.arange(st["span"], device="cuda")
    column = at // PAGE % st["table"].shape[1]
    x = _values(st[side][st["table"]], case[side], side, case["dim"], st[side + "_scale"], torch.float32)
    x = x.transpose(2, 3).flatten(1, 2)                            # [B, tokens, hk, dim]
    return x[torch.arange(x.shape[0], device="cuda")[:, None], column * PAGE + at % PAGE].transpose(1, 2)


def _scores(st):
    """[B, hk, group, n, span] float32: scaled scores, -inf where the row does not see the key; and the keys' positions."""
    case, n = st["case"], st["longest_new"]
    hk, group, dim = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    rows, _ = _chunk_rows(st)
    q = st["q"][rows].float().unflatten(2, (hk, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)    # [B, hk, group n, dim]
    s = (q @ _keys(st, "k").transpose(2, 3)).mul_(dim ** -0.5).unflatten(2, (group, n))
    key = st["first"][:, None] + torch.arange(st["span"], device="cuda")
    row = (st["lens"] - st["starts"].diff())[:, None] + torch.arange(n, device="cuda")
    back = row[:, :, None] - key[:, None]                          # [B, n, span]
    window = case.get("window", 0)
    hidden = (back < 0) | (back >= window) if window else back < 0
    return s.masked_fill_(hidden[:, None, None], -math.inf), key


def _chunk_plain(st):
    case = st["case"]
    s, _ = _scores(st)
    top = s.amax(-1, keepdim=True)                                 # (a row sees its own key at least)
    total = s.sub_(top).exp_().sum(-1, keepdim=True)
    o = (s.flatten(2, 3) @ _keys(st, "v")).unflatten(2, s.shape[2:4]) / total
    rows, live = _chunk_rows(st)
    st["out"][rows[live]] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[live].half()
    if not case["lse"]:
        return st["out"]
    lse = (top + total.log()).squeeze(-1)
    st["lse"][rows[live]] = lse.permute(0, 3, 1, 2).flatten(2, 3)[live]
    return st["out"], st["lse"]


def _weight_plain(st):
    case = st["case"]
    s, key = _scores(st)
    rows, live = _chunk_rows(st)
    lse = st["lse"][rows].masked_fill(~live[..., None], math.inf)  # rows that do not exist weigh nothing
    lse = lse.unflatten(2, s.shape[1:3]).permute(0, 2, 3, 1)
    got = s.sub_(lse[..., None]).exp_().sum((2, 3))                # [B, hk, span]
    exists = (key < st["lens"][:, None])[:, None]
    w = st["weights"]
    w.copy_(torch.where(exists, case["keep"] * w + got if case["keep"] else got, w))
    return w


def _normed(x, weight):
    x = x.float()
    return x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * weight if weight is not None else x


def _rotated(x, st):
    """The first dims of rows x [tokens, heads, dim] turned by their positions (angles in 64 bits)."""
    case, r = st["case"], st["case"]["rotary"]
    if not r:
        return x
    angle = st["positions"].double()[:, None] * st["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _rope_plain(st):
    case = st["case"]
    st["q_out"].copy_(_rotated(_normed(st["q"], st["q_weight"]), st).half())
    k = _rotated(_normed(st["k"], st["k_weight"]), st).half()
    if not case["append"]:
        st["k_out"].copy_(k)
        return st["q_out"], st["k_out"]
    page, t = st["slots"].long() // PAGE, st["slots"].long() % PAGE
    heads = torch.arange(case["kv_heads"], device="cuda")[:, None]
    for side, x in (("k", k), ("v", st["v"])):
        codes = (x.float() / st[side + "_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        at = _table_of(_places, "fp8", side, case["dim"])[0][t]
        st[side + "_pool"][page[:, None, None], heads, at[:, None]] = codes
    return _rope_stored(st)


def _rope_stored(st):
    # fp8 codes, as the values they stand for (but for the tensor's scale)
    return (st["q_out"],) + tuple(st[side].view(torch.float8_e4m3fn) for side in ("k_pool", "v_pool"))


def _evict_kept(st):
    """[B, hk, most] the kept tokens in order, -1 behind the last; and how many each sequence keeps."""
    case, most = st["case"], st["most"]
    lens = st["lens"].long()[:, None]
    n = torch.minimum(lens, st["budgets"].long()[:, None])
    recent = n.clamp_max(case["recent"])
    sink = (n - recent).clamp_max(case["sink"])
    at = torch.arange(st["weights"].shape[2], device="cuda")
    forced, exists = ((at < sink) | (at >= lens - recent)) & (at < lens), at < lens
    rank = st["weights"].masked_fill(forced[:, None], math.inf).masked_fill(~exists[:, None], -math.inf)
    first = rank.sort(dim=-1, descending=True, stable=True).indices[..., :most]
    spare = torch.arange(first.shape[2], device="cuda") >= n[..., None]
    kept = first.masked_fill(spare, at.numel()).sort(-1).values
    return kept.masked_fill(spare, -1), n[:, 0]


def _evict_plain(st):
    case = st["case"]
    kept, n = _evict_kept(st)
    st["kept"].fill_(-1)
    st["kept"][..., :kept.shape[2]] = kept.int()
    st["new_lens"].copy_(n)
    b, h, j = (kept >= 0).nonzero(as_tuple=True)
    frm = kept[b, h, j]
    st["new_weights"][b, h, j] = st["weights"][b, h, frm]
    src, dst = st["table"].long()[b, frm // PAGE], st["to"].long()[b, j // PAGE]
    for side in ("k", "v"):
        own_bytes, pool = _table_of(_token_bytes, case[side], side, case["dim"]), st[side]
        pool[dst[:, None], h[:, None], own_bytes[j % PAGE]] = pool[src[:, None], h[:, None], own_bytes[frm % PAGE]]
    return st["kept"], st["new_weights"], st["new_lens"], st["k"], st["v"]


# --------------------------------------------------------------------------- own --

def _cache(st):
    import decode_attention_block_memra_gb300 as memra
    case = st["case"]
    if "cache" not in st:
        k, v = (st[s] if s in st and case["op"] != "rope" else st[s + "_pool"] for s in ("k", "v"))
        formats = ("fp8", "fp8") if case["op"] == "rope" else (case["k"], case["v"])
        st["cache"] = memra.KVCache(*formats, k.shape[0], case["kv_heads"], case["dim"], st["k_scale"], st["v_scale"],
                                    k_pool=k.view(-1), v_pool=v.view(-1))
    return memra, st["cache"]


def _own(st):
    import decode_attention_block_memra_gb300 as memra
    case = st["case"]
    if case["op"] == "rope":
        turn = dict(q_weight=st["q_weight"], k_weight=st["k_weight"], eps=1e-6, interleaved=case["interleaved"])
        if not case["append"]:
            memra.qk_norm_rope(st["q"], st["k"], st["positions"], st["inv_freq"], st["q_out"], st["k_out"], **turn)
            return st["q_out"], st["k_out"]
        memra, cache = _cache(st)
        memra.qk_norm_rope(st["q"], st["k"], st["positions"], st["inv_freq"], st["q_out"], cache=cache, v=st["v"],
                           slot_mapping=st["slots"], **turn)
        return _rope_stored(st)
    memra, cache = _cache(st)
    if case["op"] == "chunk":
        memra.chunk_attn(cache, st["q"], st["starts"], st["table"], st["lens"], st["longest"], st["out"],
                         st["workspace"], window=case["window"], lse=st["lse"])
        return (st["out"], st["lse"]) if case["lse"] else st["out"]
    if case["op"] == "weight":
        memra.key_weights(cache, st["q"], st["lse"], st["starts"], st["table"], st["lens"], st["longest"],
                          st["weights"], keep=case["keep"])
        return st["weights"]
    memra.kv_evict(cache, st["table"], st["lens"], st["longest"], st["weights"], st["budgets"], st["to"], st["kept"],
                   sink=case["sink"], recent=case["recent"], new_weights=st["new_weights"], new_lens=st["new_lens"])
    return st["kept"], st["new_weights"], st["new_lens"], st["k"], st["v"]


def run(state):
    if own:
        return _own(state)
    plain = {"chunk": _chunk_plain, "weight": _weight_plain, "rope": _rope_plain, "evict": _evict_plain}
    return plain[state["case"]["op"]](state)


# -------------------------------------------------------------------------- work --

def _visible(case):
    """Keys that the rows of a chunk see, all together; and the keys that any of them sees."""
    pairs = keys = 0
    for n, p in zip(_ints(case["new"]), _ints(case["past"])):
        w = case.get("window", 0) or n + p
        full = max(0, min(n, w - p))                               # rows whose window reaches back to key 0
        pairs += full * p + full * (full + 1) // 2 + (n - full) * w
        keys += n + p - max(0, p - w + 1)
    return float(pairs), float(keys)


def work(case):
    dim, hk = case["dim"], case["kv_heads"]
    if case["op"] == "rope":
        rows = case["tokens"] * (2 * case["heads"] + 2 * hk) * dim * 2.0
        if case["append"]:                                         # V in, one byte a code out for K and V; K not written as rows
            rows += case["tokens"] * hk * dim * 2.0
        return {"bytes": rows, "flops": 0.0}
    ks, vs = _segment(case["k"], dim) / PAGE, _segment(case["v"], dim) / PAGE
    if case["op"] == "evict":
        lens, kept = _ints(case["lens"]), [min(a, b) for a, b in zip(_ints(case["lens"]), _ints(case["budgets"]))]
        return {"bytes": float(hk * (4 * sum(lens) + sum(kept) * (2 * (ks + vs) + 8))), "flops": 0.0}
    pairs, keys = _visible(case)
    tokens, hq = sum(_ints(case["new"])), case["heads"]
    if case["op"] == "weight":
        rw = 8 if case["keep"] else 4
        return {"bytes": float(keys * hk * (ks + rw) + tokens * hq * (2 * dim + 4)), "flops": 2.0 * dim * hq * pairs}
    return {"bytes": float(keys * hk * (ks + vs) + tokens * hq * (4 * dim + 4 * case["lse"])),
            "flops": 4.0 * dim * hq * pairs}


# ------------------------------------------------------------------------- exact --

def _exact_values(seg, fmt, side, dim, scale):
    """Segments [n, segment] of pages read as the strided arrays that the header's formulas describe: [n, 16, dim]."""
    n, nb = seg.shape[0], dim // 32
    x = seg.cpu().numpy()

    def part(first, size, shape):
        return x[:, first:first + size].reshape((n,) + shape)

    def halves(first, shape):
        return np.ascontiguousarray(x[:, first:first + dim]).view(np.float16).reshape((n,) + shape).astype(np.float64)

    def e4m3(a):
        sign, e, m = 1.0 - 2.0 * (a >> 7), (a >> 3 & 15).astype(np.int64), (a & 7).astype(np.float64)
        return sign * np.where(e == 0, np.ldexp(m / 8, -6), np.ldexp(1 + m / 8, e - 7))

    def e2m1(a):
        e, m = (a >> 1 & 3).astype(np.int64), (a & 1).astype(np.float64)
        return (1.0 - 2.0 * (a >> 3)) * np.where(e == 0, m / 2, np.ldexp(1 + m / 2, e - 1))

    def nibbles(a):
        return np.stack((a & 15, a >> 4), -1)

    if side == "k" and fmt != "nvfp4":                       # tp b2 tg kc b1 e
        code = part(0, 16 * dim, (2, nb // 2, 8, 4, 2, 8)).transpose(0, 1, 3, 2, 5, 4, 6).reshape(n, PAGE, dim)
        if fmt == "fp8":
            return torch.from_numpy(e4m3(code) * scale)
        d = halves(16 * dim, (PAGE, nb))
        return torch.from_numpy((code.astype(np.float64) - 128) * np.repeat(d, 32, -1))
    if side == "k":                                          # w4 tg c b1 e2 eh tp el
        code = nibbles(part(0, 8 * dim, (nb // 2, 8, 4, 2, 2, 2, 2))).transpose(0, 7, 2, 1, 4, 3, 5, 6, 8)
        block = e4m3(part(8 * dim, dim, (PAGE, dim // 16))) * scale
        return torch.from_numpy(e2m1(code.reshape(n, PAGE, dim)) * np.repeat(block, 16, -1))
    if fmt == "fp8":                                         # b vg c h p s f
        code = part(0, 16 * dim, (nb, 8, 4, 2, 2, 2, 2)).transpose(0, 5, 3, 7, 1, 2, 4, 6)
        return torch.from_numpy(e4m3(code.reshape(n, PAGE, dim)) * scale)
    if fmt == "nvfp4":                                       # b4 r8 c b1 p f rh
        code = nibbles(part(0, 8 * dim, (dim // 64, 8, 4, 4, 2, 2))).transpose(0, 5, 3, 6, 1, 4, 7, 2)
        block = e4m3(part(8 * dim, dim, (4, dim // 16, 2, 2))).transpose(0, 3, 1, 4, 2).reshape(n, PAGE, dim // 16)
        return torch.from_numpy(e2m1(code.reshape(n, PAGE, dim)) * np.repeat(block * scale, 16, -1))
    low = nibbles(part(0, 8 * dim, (nb // 2, 8, 4, 2, 2, 2, 2)))                  # b2 vg c b1 h f p s
    code = low.transpose(0, 7, 3, 6, 1, 4, 2, 5, 8).reshape(n, PAGE, dim).astype(np.float64)

    def blocks(first):                                       # c b p f
        return np.repeat(halves(first, (4, nb, 2, 2)).transpose(0, 3, 1, 4, 2).reshape(n, PAGE, nb), 32, -1)

    if fmt == "q4_0":
        return torch.from_numpy((code - 8) * blocks(8 * dim))
    bits = np.unpackbits(part(8 * dim, 2 * dim, (8, 4, nb // 2, 2, 2, 1)), axis=-1, bitorder="little")
    high = bits.reshape(n, 8, 4, nb // 2, 2, 2, 2, 2, 2)                          # vg c b2 f p s b1 h
    code += 16.0 * high.transpose(0, 5, 2, 4, 3, 7, 1, 8, 6).reshape(n, PAGE, dim)
    return torch.from_numpy(code * blocks(10 * dim) + blocks(11 * dim))


def _exact_sequence(case, st, b):
    """Of sequence b: its packed rows, the positions and pages of the keys that its chunk may see, and what sees what."""
    begin, end = (int(x) for x in st["starts"][b:b + 2])
    length, window, n = int(st["lens"][b]), case.get("window", 0), end - begin
    key = np.arange(max(0, length - n - window + 1) if window else 0, length)
    row = np.arange(length - n, length)
    sees = key <= row[:, None]
    if window:
        sees &= key > row[:, None] - window
    at = key // PAGE % st["table"].shape[1]
    used, where = np.unique(at, return_inverse=True)
    pages = st["table"][b].cpu().numpy()[used]
    return slice(begin, end), torch.from_numpy(pages).long().cuda(), where * PAGE + key % PAGE, torch.from_numpy(sees).cuda()


def _exact_logits(case, st, rows, h, k, sees):
    z = torch.einsum("rd,kd->rk", st["q"][rows, h].double(), k) / math.sqrt(case["dim"])
    return torch.where(sees, z, torch.full_like(z, -math.inf))


def _exact_attended(case, st, each):
    """Calls each(b, head, rows, logits, values of V of the KV head, keys' positions) for every head, in 64 bits."""
    group = case["heads"] // case["kv_heads"]
    for b in range(len(st["lens"])):
        rows, pages, at, sees = _exact_sequence(case, st, b)
        at = torch.from_numpy(at).cuda()
        for g in range(case["kv_heads"]):
            k, v = (_exact_values(st[s][pages, g], case[s], s, case["dim"], st[s + "_scale"]).flatten(0, 1).cuda()[at]
                    for s in ("k", "v"))
            for h in range(g * group, (g + 1) * group):
                each(b, h, rows, _exact_logits(case, st, rows, h, k, sees), v)


def _exact_chunk(case, st):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device="cuda")

    def each(b, h, rows, z, v):
        out[rows, h] = torch.softmax(z, 1) @ v
        lse[rows, h] = torch.logsumexp(z, 1)

    _exact_attended(case, st, each)
    return (out, lse) if case["lse"] else out


def _exact_weight(case, st):
    group, start = case["heads"] // case["kv_heads"], st["weights"].double()
    got = torch.zeros_like(start)

    def each(b, h, rows, z, v):
        got[b, h // group, :z.shape[1]] += torch.exp(z - st["lse"][rows, h].double()[:, None]).sum(0)

    _exact_attended(case, st, each)
    for b, n in enumerate(st["lens"].tolist()):
        got[b, :, :n] += case["keep"] * start[b, :, :n] if case["keep"] else 0.0
        got[b, :, n:] = start[b, :, n:]
    return got


def _exact_turned(case, st, x, weight):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + 1e-6) * weight.double()
    half = case["rotary"] // 2
    if half:
        dims = torch.arange(half, device="cuda")
        first, second = (2 * dims, 2 * dims + 1) if case["interleaved"] else (dims, dims + half)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           torch.outer(st["positions"].double(), st["inv_freq"].double()))[:, None]
        z = torch.complex(x[..., first], x[..., second]) * turn
        x = x.index_copy(-1, first, z.real).index_copy(-1, second, z.imag)
    return x


def _exact_e4m3(x):
    """The nearest e4m3 values, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -12))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_rope(case, st):
    q = _exact_turned(case, st, st["q"], st["q_weight"])
    k = _exact_turned(case, st, st["k"], st["k_weight"])
    if not case["append"]:
        return q, k
    pools = []
    for side, x in (("k", k.half()), ("v", st["v"])):
        pool = torch.zeros(st[side + "_pool"].shape, dtype=torch.float64, device="cuda")
        codes = _exact_e4m3((x.float() / np.float32(st[side + "_scale"])).double())
        at = torch.from_numpy(_places("fp8", side, case["dim"])[0]).cuda()
        for t in range(PAGE):
            here = st["slots"] % PAGE == t
            pages = (st["slots"][here] // PAGE).long()
            for h in range(case["kv_heads"]):
                pool[pages[:, None], h, at[t]] = codes[here, h]
        pools.append(pool)
    return (q, *pools)


def _exact_evict(case, st):
    """The kept tokens' weights: budgets met by comparing each middle token with every other."""
    out = torch.zeros(st["new_weights"].shape, dtype=torch.float64)
    weights = st["weights"].cpu().numpy()
    for b, (length, budget) in enumerate(zip(_ints(case["lens"]), _ints(case["budgets"]))):
        n = min(length, budget)
        recent = min(case["recent"], n)
        sink = min(case["sink"], n - recent)
        for h in range(case["kv_heads"]):
            w = weights[b, h, :length]
            middle = np.arange(sink, length - recent)
            best = middle[np.lexsort((middle, -w[middle]))][:n - sink - recent]
            kept = np.concatenate((np.arange(sink), np.sort(best), np.arange(length - recent, length)))
            out[b, h, :n] = torch.from_numpy(w[kept].astype(np.float64))
    return None, out, None, None, None


def exact(case, seed):
    """The numbers in 64 bits (an eviction moves bytes and picks by comparison: of its outputs the weights are numbers)."""
    st = prepare(case, seed)
    numbers = {"chunk": _exact_chunk, "weight": _exact_weight, "rope": _exact_rope, "evict": _exact_evict}
    return numbers[case["op"]](case, st)
