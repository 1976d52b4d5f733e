"""The library's operators around the decode step: their plain forms, their calls, and cases to measure them by.

    prompt   causal attention of whole prompts, packed one behind the other (``prompt_attn``)
    tree     attention of a tree of drafted tokens over the paged cache (``tree_attn``)
    copy     copies of cache pages inside the pools (``kv_copy_pages``)
    compact  the accepted rows of a verified tree move to its front (``kv_compact``)

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
        # the smallest prompt a server sees: one short request, where latency counts
        dict(name="prompt_256", op="prompt", lens="256", heads=8, kv_heads=2, dim=128, window=0, fused=False, pad=0),
        # admission of several requests at once: a shared-prefix prompt's length, ragged ones, a one-token one
        dict(name="prompt_ragged_4860", op="prompt", lens="4860,4096,1,2047,700,4859,3333,17", heads=32, kv_heads=4,
             dim=128, window=0, fused=True, pad=5),
        # one long document
        dict(name="prompt_16384", op="prompt", lens="16384", heads=32, kv_heads=4, dim=128, window=0, fused=False,
             pad=0),
        # wide heads with a sliding window
        dict(name="prompt_d256_window", op="prompt", lens="6301,512,2900", heads=16, kv_heads=2, dim=256, window=1024,
             fused=False, pad=0),
        # a small tree of drafts over a short context, batch 1
        dict(name="tree_8_256", op="tree", lens="256", nodes=8, heads=8, kv_heads=2, dim=128, k="q8_0", v="q5_1"),
        # eight sequences verifying 16 drafts each
        dict(name="tree_16_6316", op="tree", lens="6316,6316,6316,6316,6316,6316,6316,6316", nodes=16, heads=32,
             kv_heads=4, dim=128, k="q8_0", v="q5_1"),
        # the widest tree over the longest context
        dict(name="tree_64_262144", op="tree", lens="262144", nodes=64, heads=32, kv_heads=4, dim=128, k="q8_0",
             v="q5_1"),
        # ragged contexts at head_dim 256 in fp8
        dict(name="tree_d256_fp8", op="tree", lens="512,32768,777,9000,16001,4860,31,2049,12288,20000,6304,1025",
             nodes=31, heads=16, kv_heads=2, dim=256, k="fp8", v="fp8"),
        # sixteen sequences fork: their last, partial pages are copied
        dict(name="copy_16", op="copy", pages=16, pool=4096, kv_heads=4, dim=128, k="q8_0", v="q5_1"),
        # a 262,144-token cache moves
        dict(name="copy_16384", op="copy", pages=16384, pool=40000, kv_heads=4, dim=128, k="q8_0", v="q5_1"),
        # eight sequences keep up to 5 of 16 drafts
        dict(name="compact_8x16", op="compact", batch=8, nodes=16, most=5, length=6316, kv_heads=4, dim=128, k="q8_0",
             v="q5_1"),
        # many sequences, wide trees, four-bit rows
        dict(name="compact_256x64", op="compact", batch=256, nodes=64, most=64, length=700, kv_heads=2, dim=256,
             k="nvfp4", v="q4_0"),
    ]


PAIRS = (("q8_0", "q5_1"), ("q8_0", "q4_0"), ("fp8", "fp8"), ("nvfp4", "nvfp4"), ("fp8", "q5_1"), ("nvfp4", "q4_0"))
HEADS = ((8, 2), (32, 4), (16, 2), (4, 4), (12, 4), (8, 1), (40, 8), (24, 8))


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "tree", "tree", "copy", "compact"))
    dim = rng.choice((128, 256))
    heads, kv_heads = rng.choice(HEADS)
    k, v = rng.choice(PAIRS)
    if op == "prompt":
        n = _log(rng, 1, 12)
        longest = int(min(16384, math.sqrt(16384 ** 2 * 32 * 128 / (n * heads * dim))))
        lens = [_log(rng, 1, longest) for _ in range(n)]
        return dict(op=op, lens=",".join(map(str, lens)), heads=heads, kv_heads=kv_heads, dim=dim,
                    window=rng.choice((0, 0, _log(rng, 1, 4096))), fused=rng.random() < 0.5, pad=rng.choice((0, 3)))
    if op == "tree":
        n, nodes = _log(rng, 1, 24), _log(rng, 1, 64)
        longest = min(262144, 262144 * 32 * 128 // (n * heads * dim))
        lens = [nodes + _log(rng, 1, longest) - 1 for _ in range(n)]
        return dict(op=op, lens=",".join(map(str, lens)), nodes=nodes, heads=heads, kv_heads=kv_heads, dim=dim, k=k, v=v)
    if op == "copy":
        pages = min(_log(rng, 1, 16384), 16384 * 4 * 128 // (kv_heads * dim))
        return dict(op=op, pages=pages, pool=2 * pages + rng.randrange(1, 5000), kv_heads=kv_heads, dim=dim, k=k, v=v)
    nodes = _log(rng, 2, 64)
    return dict(op=op, batch=_log(rng, 1, 256), nodes=nodes, most=rng.randint(1, nodes), length=nodes + _log(rng, 1, 900),
                kv_heads=kv_heads, dim=dim, k=k, v=v)


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
def _table(what, *args):
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
        seg[..., _table(_scales, fmt, side, dim)] = block.squeeze(-1).view(torch.uint8)
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
        minimum = _table(_scales, fmt, side, dim) + dim
        halves = low.half().view(torch.uint8)
        seg[..., minimum], seg[..., minimum + 1] = halves[..., 0], halves[..., 1]
    first, halves = _table(_scales, fmt, side, dim), d.view(torch.uint8)
    seg[..., first], seg[..., first + 1] = halves[..., 0], halves[..., 1]
    return seg, scale


def _half_at(seg, first):
    return torch.stack((seg[..., first], seg[..., first + 1]), -1).view(torch.float16).squeeze(-1)


def _values(seg, fmt, side, dim, scale, dtype):
    """The values that segments [..., segment] stand for: [..., 16, dim] in `dtype`."""
    byte, shift = _table(_places, fmt, side, dim)
    code = seg[..., byte]
    if fmt == "fp8":
        return code.view(torch.float8_e4m3fn).to(dtype) * scale
    if fmt == "q8_0":
        q = code.to(dtype) - 128
    else:
        code = (code >> shift.to(torch.uint8)) & 15
        if fmt == "nvfp4":
            table = _e2m1_values(dtype)
            block = seg[..., _table(_scales, fmt, side, dim)].view(torch.float8_e4m3fn)
            return table[code.int()] * (block.to(dtype) * scale).repeat_interleave(16, -1)
        if fmt == "q5_1":
            fifth, bit = _table(_fifth, dim)
            code = code | (((seg[..., fifth] >> bit.to(torch.uint8)) & 1) << 4)
        q = code.to(dtype) - (8 if fmt == "q4_0" else 0)
    at = _table(_scales, fmt, side, dim)
    x = q * _half_at(seg, at).to(dtype).repeat_interleave(32, -1)
    return x + _half_at(seg, at + dim).to(dtype).repeat_interleave(32, -1) if fmt == "q5_1" else x


# ------------------------------------------------------------------------ states --

def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def _pools(case, pages, g):
    """A cache of `pages` pages of quantized normal rows: the K and V segments and their scales."""
    shape = (pages, case["kv_heads"], PAGE, case["dim"])
    k, ks = _quantize(torch.randn(shape, generator=g, device="cuda"), case["k"], "k")
    v, vs = _quantize(torch.randn(shape, generator=g, device="cuda"), case["v"], "v")
    return dict(k=k, v=v, k_scale=ks, v_scale=vs)


def _ancestors(nodes, rng):
    """A random tree of drafts: bit j of word i says that node i's path from the root passes node j."""
    words = np.zeros(nodes, np.uint64)
    for i in range(nodes):
        words[i] = np.uint64(1 << i) | (words[rng.integers(0, i)] if i else np.uint64(0))
    return words.view(np.int64)


def _prompt_state(case, g):
    lens, dim, hq, hk = _lens(case), case["dim"], case["heads"], case["kv_heads"]
    total = sum(lens) + case["pad"]
    rows = torch.randn(total, hq + 2 * hk, dim, generator=g, device="cuda").half()
    q, k, v = rows[:, :hq], rows[:, hq:hq + hk], rows[:, hq + hk:]
    if not case["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    starts = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    return dict(q=q, k=k, v=v, starts=starts, longest=max(lens), out=torch.zeros(total, hq, dim, device="cuda").half())


def _tree_state(case, g, rng):
    lens, dim = _lens(case), case["dim"]
    need = [-(-n // PAGE) for n in lens]
    pages = sum(need) + 2
    state = _pools(case, pages, g)
    order = rng.permutation(pages)
    table = np.zeros((len(lens), max(need)), np.int32)
    mask = np.arange(max(need)) < np.array(need)[:, None]
    table[mask] = order[:sum(need)]
    words = np.stack([_ancestors(case["nodes"], rng) for _ in lens])
    state.update(table=torch.from_numpy(table).cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                 longest=max(lens), mask=torch.from_numpy(words).cuda(),
                 q=torch.randn(len(lens), case["nodes"], case["heads"], dim, generator=g, device="cuda").half())
    state["out"] = torch.empty_like(state["q"])
    # float32 partial rows and their log-sum-exp, one for each 256 keys and 512 at most: the call never needs more
    rows = len(lens) * case["nodes"] * case["heads"]
    parts = min(512, -(-max(lens) // 256))
    state["workspace"] = torch.empty(rows * parts * (dim + 1) * 4 + 1024, dtype=torch.uint8, device="cuda")
    return state


def _compact_state(case, g, rng):
    batch, nodes, length = case["batch"], case["nodes"], case["length"]
    lens = np.maximum(nodes, length - rng.integers(0, PAGE, batch)).astype(np.int32)
    per = -(-length // PAGE)
    first = (length - nodes) // PAGE - 1                  # pages before the trees' are not part of the pools
    used = per - max(first, 0)
    state = _pools(case, batch * used + 1, g)
    table = np.zeros((batch, per), np.int32)
    table[:, per - used:] = rng.permutation(batch * used + 1)[:batch * used].reshape(batch, used)
    count = rng.integers(0, case["most"] + 1, batch).astype(np.int32)
    kept = np.sort(np.argsort(rng.random((batch, nodes)), 1)[:, :case["most"]], 1)
    state.update(table=torch.from_numpy(table).cuda(), lens=torch.from_numpy(lens).cuda(), longest=int(lens.max()),
                 kept=torch.from_numpy(kept.astype(np.int32)).cuda(), count=torch.from_numpy(count).cuda())
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    if case["op"] == "prompt":
        state = _prompt_state(case, g)
    elif case["op"] == "tree":
        state = _tree_state(case, g, rng)
    elif case["op"] == "copy":
        state = _pools(case, case["pool"], g)
        order = rng.permutation(case["pool"])[:2 * case["pages"]].astype(np.int32)
        state["src"], state["dst"] = (torch.from_numpy(a.copy()).cuda() for a in np.split(order, 2))
    else:
        state = _compact_state(case, g, rng)
    state["case"] = case
    return state


# ------------------------------------------------------------------------- plain --

def _softmax_product(s, v):
    """softmax(s) v over the last axis of s; rows that see nothing (all -inf) are zeros.  Overwrites s."""
    top = s.amax(-1, keepdim=True)
    s.sub_(top.masked_fill_(top == -math.inf, 0)).exp_()
    return (s @ v) / s.sum(-1, keepdim=True).clamp_min(1e-30)


def _prompt_plain(st):
    case, n = st["case"], st["longest"]
    hk, group, dim = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    first, size = st["starts"][:-1].long(), st["starts"].diff()
    at = torch.arange(n, device="cuda")
    rows = (first[:, None] + at).clamp_max(st["q"].shape[0] - 1)
    q = st["q"][rows].float().unflatten(2, (hk, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)    # [B, hk, group n, dim]
    k = st["k"][rows].float().permute(0, 2, 3, 1)
    v = st["v"][rows].float().transpose(1, 2)
    s = (q @ k).mul_(dim ** -0.5).unflatten(2, (group, n))
    back = at[:, None] - at
    hidden = (back < 0) | ((back >= case["window"]) if case["window"] else False)
    s.masked_fill_(hidden, -math.inf)
    o = _softmax_product(s.flatten(2, 3), v).unflatten(2, (group, n)).permute(0, 3, 1, 2, 4).flatten(2, 3)
    live = at < size[:, None]
    st["out"][rows[live]] = o[live].half()
    return st["out"]


def _tree_visible(st, nodes):
    """[B, nodes, keys]: which keys a node sees: every one before the tree's, and the tree's by its word."""
    key = torch.arange(st["table"].shape[1] * PAGE, device="cuda") - (st["lens"].long()[:, None] - nodes)
    bit = (st["mask"][:, :, None] >> key.clamp(0, nodes - 1)[:, None]) & 1
    return (key < 0)[:, None] | ((key < nodes)[:, None] & (bit != 0))


def _tree_plain(st):
    case = st["case"]
    hk, group, dim, nodes = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"], case["nodes"]
    k = _values(st["k"][st["table"]], case["k"], "k", dim, st["k_scale"], torch.float32)    # [B, pages, hk, 16, dim]
    v = _values(st["v"][st["table"]], case["v"], "v", dim, st["v_scale"], torch.float32)
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))
    q = st["q"].float().unflatten(2, (hk, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)      # [B, hk, nodes group, dim]
    s = (q @ k.transpose(2, 3)).mul_(dim ** -0.5).unflatten(2, (nodes, group))
    s.masked_fill_(~_tree_visible(st, nodes)[:, None, :, None], -math.inf)
    o = _softmax_product(s.flatten(2, 3), v).unflatten(2, (nodes, group)).transpose(1, 2).flatten(2, 3)
    return o.half()


def _compact_plain(st):
    case = st["case"]
    base = st["lens"].long()[:, None] - case["nodes"]
    live = torch.arange(st["kept"].shape[1], device="cuda") < st["count"][:, None]
    frm, to = (base + st["kept"])[live], (base + torch.arange(st["kept"].shape[1], device="cuda"))[live]
    row = torch.arange(case["batch"], device="cuda")[:, None].expand_as(live)[live]
    src, dst = (st["table"].long()[row, p // PAGE] for p in (frm, to))
    for side in ("k", "v"):
        own_bytes = _table(_token_bytes, case[side], side, case["dim"])
        pool, heads = st[side], torch.arange(case["kv_heads"], device="cuda")[:, None]
        moved = pool[src[:, None, None], heads, own_bytes[frm % PAGE][:, None]]
        pool[dst[:, None, None], heads, own_bytes[to % PAGE][:, None]] = moved
    return st["k"], st["v"]


def _copy_plain(st):
    st["k"][st["dst"]] = st["k"][st["src"]]
    st["v"][st["dst"]] = st["v"][st["src"]]
    return st["k"], st["v"]


# --------------------------------------------------------------------------- own --

def _cache(st):
    import decode_attention_block_memra_gb300 as memra
    case = st["case"]
    if "cache" not in st:
        st["cache"] = memra.KVCache(case["k"], case["v"], st["k"].shape[0], case["kv_heads"], case["dim"],
                                    st["k_scale"], st["v_scale"], k_pool=st["k"].view(-1), v_pool=st["v"].view(-1))
    return memra, st["cache"]


def _own(st):
    import decode_attention_block_memra_gb300 as memra
    case = st["case"]
    if case["op"] == "prompt":
        memra.prompt_attn(st["q"], st["k"], st["v"], st["starts"], st["out"], window=case["window"])
        return st["out"]
    memra, cache = _cache(st)
    if case["op"] == "tree":
        memra.tree_attn(cache, st["q"], st["table"], st["lens"], st["longest"], st["mask"], st["out"], st["workspace"])
        return st["out"]
    if case["op"] == "copy":
        memra.kv_copy_pages(cache, st["src"], st["dst"])
    else:
        memra.kv_compact(cache, st["table"], st["lens"], st["longest"], st["kept"], st["count"], case["nodes"])
    return st["k"], st["v"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "prompt":
        return _prompt_plain(state)
    if op == "tree":
        return _tree_plain(state)
    return _copy_plain(state) if op == "copy" else _compact_plain(state)


# -------------------------------------------------------------------------- work --

def work(case):
    dim, hk = case["dim"], case["kv_heads"]
    if case["op"] == "prompt":
        lens, w = np.array(_lens(case), np.float64), case["window"]
        full = np.minimum(lens, w) if w else lens
        keys = full * (full + 1) / 2 + (lens - full) * w
        return {"bytes": float(2 * dim * (2 * case["heads"] + 2 * hk) * lens.sum()),
                "flops": float(4 * dim * case["heads"] * keys.sum())}
    segments = _segment(case["k"], dim) + _segment(case["v"], dim)
    if case["op"] == "tree":
        lens, rows = _lens(case), case["nodes"] * case["heads"]
        return {"bytes": float(sum(n * hk * segments / PAGE + 4 * rows * dim for n in lens)),
                "flops": float(sum(4 * dim * rows * n for n in lens))}
    if case["op"] == "copy":
        return {"bytes": float(2 * case["pages"] * hk * segments), "flops": 0.0}
    return {"bytes": float(2 * case["batch"] * case["most"] / 2 * hk * segments / PAGE), "flops": 0.0}


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


def _exact_rows(q, k, v, sees, scale):
    """One sequence and KV head in 64 bits: q [rows, dim], k, v [keys, dim], sees [rows, keys]."""
    z = torch.einsum("rd,kd->rk", q.double(), k.double()) * scale
    z = torch.where(sees, z, torch.full_like(z, -math.inf))
    weight = torch.softmax(z, 1).nan_to_num(0.0)
    return torch.einsum("rk,kd->rd", weight, v.double())


def _exact_prompt(case, st):
    group, scale = case["heads"] // case["kv_heads"], 1 / math.sqrt(case["dim"])
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    begin = 0
    for n in _lens(case):
        at = torch.arange(n, device="cuda")
        for lo in range(0, n, 4096):                        # rows lo .. hi - 1 of the sequence see keys below hi
            hi = min(n, lo + 4096)
            sees = at[:hi] <= at[lo:hi, None]
            if case["window"]:
                sees &= at[:hi] > at[lo:hi, None] - case["window"]
            for h in range(case["heads"]):
                out[begin + lo:begin + hi, h] = _exact_rows(
                    st["q"][begin + lo:begin + hi, h], st["k"][begin:begin + hi, h // group],
                    st["v"][begin:begin + hi, h // group], sees, scale)
        begin += n
    return out


def _exact_tree(case, st):
    group, scale, nodes = case["heads"] // case["kv_heads"], 1 / math.sqrt(case["dim"]), case["nodes"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    words = st["mask"].cpu().numpy().view(np.uint64)
    for b, n in enumerate(_lens(case)):
        sees = np.ones((nodes, n), bool)
        for j in range(nodes):
            sees[:, n - nodes + j] = (words[b] >> np.uint64(j)) & np.uint64(1)
        sees = torch.from_numpy(sees).cuda().repeat_interleave(group, 0)
        pages = st["table"][b, :-(-n // PAGE)].long()
        for h in range(case["kv_heads"]):
            k = _exact_values(st["k"][pages, h], case["k"], "k", case["dim"], st["k_scale"]).cuda().flatten(0, 1)[:n]
            v = _exact_values(st["v"][pages, h], case["v"], "v", case["dim"], st["v_scale"]).cuda().flatten(0, 1)[:n]
            heads = slice(h * group, (h + 1) * group)
            rows = _exact_rows(st["q"][b, :, heads].flatten(0, 1), k, v, sees, scale)
            out[b, :, heads] = rows.unflatten(0, (nodes, group))
    return out


def exact(case, seed):
    """The attention in 64 bits; the cache's upkeep moves bytes and has no computed number."""
    if case["op"] not in ("prompt", "tree"):
        return None
    st = prepare(case, seed)
    return _exact_prompt(case, st) if case["op"] == "prompt" else _exact_tree(case, st)
