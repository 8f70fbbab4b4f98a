"""The cache-compression operators as measured cases: 4-bit K/V caches and eviction by attention weight.

Five operators over paged K/V pools ``[num_blocks, num_kv_heads, block_size, row]``:

* append  -- new tokens' K/V rounded to 4 bits into their slots of a 4-bit pool;
* expand  -- whole blocks of a 4-bit pool widened into blocks of an f32/f16/bf16 pool;
* decode  -- single-token attention over a 4-bit pool through block tables;
* weights -- the attention probabilities of a decode step added to per-token accumulators;
* evict   -- the heaviest and the most recent rows of every (sequence, KV head) kept, in
  order, in fresh blocks.

A row of a 4-bit pool holds D values in 5 D / 8 bytes: D/2 bytes of codes (byte i: value 2i
in the low half, 2i + 1 in the high half), then one (step, lo) pair of float16 for each 32
values.  A code c stands for ``lo + c * step``, rounded once to float16.

``run`` computes the operators in elementary torch operations where ``own`` is false and
calls the library where it is true.  ``exact`` states them again in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
GROUP = 32          # values that share one (step, lo) pair
LARGEST = 65408.0   # values beyond it are stored as it: lo + 15 * step then stays a finite float16
DEVICE = "cuda"


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step's new tokens of 64 sequences: a call whose launch is its cost
        dict(name="append step", op="append", tokens=64, kv_heads=8, head_dim=128, block_size=16, dtype="bf16",
             scattered=True),
        # a prompt chunk of an odd number of tokens, and its blocks widened for prefill attention
        dict(name="append chunk", op="append", tokens=8191, kv_heads=8, head_dim=128, block_size=16, dtype="f16",
             scattered=False),
        # a few short blocks, head_dim 64
        dict(name="expand few", op="expand", blocks=9, kv_heads=4, head_dim=64, block_size=8, dtype="f32"),
        # the 4-bit blocks of a batch of long prompts widened for prefill attention
        dict(name="expand prompts", op="expand", blocks=16384, kv_heads=8, head_dim=128, block_size=16, dtype="bf16"),
        # the first tokens of a single chat: latency
        dict(name="decode one short", op="decode", seqs=1, lo=33, hi=33, q_heads=32, kv_heads=8, head_dim=64,
             block_size=16, dtype="f16", out="f16"),
        # the batch of 64 sequences with one query head per KV head
        dict(name="decode batch g1", op="decode", seqs=64, lo=128, hi=2048, q_heads=32, kv_heads=32, head_dim=128,
             block_size=16, dtype="bf16", out="bf16"),
        # the batch of 128 sequences with eight query heads per KV head
        dict(name="decode batch g8", op="decode", seqs=128, lo=512, hi=4096, q_heads=64, kv_heads=8, head_dim=128,
             block_size=16, dtype="bf16", out="bf16"),
        # two long documents: the split over a long axis, f32 in and out
        dict(name="decode two long", op="decode", seqs=2, lo=120001, hi=131072, q_heads=32, kv_heads=8, head_dim=128,
             block_size=64, dtype="f32", out="f32"),
        # accumulators of a 16-bit batch after a decode step
        dict(name="weights batch", op="weights", seqs=64, lo=128, hi=2048, q_heads=32, kv_heads=8, head_dim=128,
             block_size=16, dtype="bf16", pool="bf16"),
        # accumulators of long contexts held in 4 bits
        dict(name="weights long kv4", op="weights", seqs=8, lo=20000, hi=32768, q_heads=64, kv_heads=8, head_dim=128,
             block_size=32, dtype="f16", pool="kv4"),
        # a batch that is cut to half its room
        dict(name="evict batch", op="evict", seqs=32, lo=512, hi=4096, keep=2048, recent=256, kv_heads=8,
             head_dim=128, block_size=16, pool="bf16"),
        # one long sequence cut to a short budget
        dict(name="evict one long", op="evict", seqs=1, lo=32767, hi=32767, keep=4096, recent=511, kv_heads=4,
             head_dim=64, block_size=32, pool="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "expand", "decode", "decode", "weights", "evict"])
    case = dict(op=op, kv_heads=rng.choice([1, 2, 3, 4, 5, 8, 8, 16, 32]), head_dim=rng.choice([64, 128, 128]),
                block_size=rng.choice([8, 16, 16, 32, 64]))
    heads, bs = case["kv_heads"], case["block_size"]
    if op == "append":
        return dict(case, tokens=_log(rng, 1, 65536 // heads), dtype=rng.choice(["f32", "f16", "bf16"]),
                    scattered=rng.random() < 0.5)
    if op == "expand":
        return dict(case, blocks=_log(rng, 1, 2000000 // (heads * bs)), dtype=rng.choice(["f32", "f16", "bf16"]))
    # sequences and lengths: the padded number of (token, KV head) rows stays within the listed cases'
    hi = _log(rng, 1, 100000)
    seqs = _log(rng, 1, max(1, min(256, 1500000 // (hi * heads))))
    lo = rng.choice([0, 1, hi // 4, hi // 2, hi])
    case.update(seqs=seqs, lo=min(lo, hi), hi=hi)
    if op == "evict":
        keep = max(1, int(hi * rng.uniform(0.05, 1.0)))
        return dict(case, keep=keep, recent=int(keep * rng.choice([0.0, 0.1, 0.5, 1.0])),
                    pool=rng.choice(["f32", "f16", "bf16"]))
    group = rng.choice([1, 2, 3, 4, 6, 7, 8, 8, 12, 16])
    case["q_heads"] = heads * group
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "decode":
        return dict(case, dtype=dtype, out=rng.choice([dtype, "f32"]))
    pool = rng.choice(["f32", "f16", "bf16", "kv4", "kv4"])
    return dict(case, dtype=dtype if pool == "kv4" else pool, pool=pool)


# ----------------------------------------------------------------------------- the format

def _round16(x):
    """float64 -> the nearest float16 value, ties to even, still as float64 (one rounding)."""
    power = (x.view(torch.int64) & 0x7FF0000000000000).view(torch.float64)
    step = power.clamp(min=2.0 ** -14) * 2.0 ** -10
    return torch.where(x.isfinite(), (x / step).round() * step, x)


def quantise(x):
    """[..., D] values -> [..., 5 D / 8] bytes of a 4-bit row."""
    x = x.float()
    d = x.shape[-1]
    g = x.reshape(*x.shape[:-1], d // GROUP, GROUP)
    bad = ~g.isfinite().all(-1, keepdim=True)
    g = torch.where(bad, torch.zeros_like(g), g.clamp(-LARGEST, LARGEST))
    lo = g.amin(-1, keepdim=True).half()
    spread = (g.amax(-1, keepdim=True) - lo.float()).clamp(min=0)
    step = (spread.double() / 15).float().half()
    quotient = (g - lo.float()).double() / torch.where(step == 0, torch.ones_like(step), step).double()
    code = torch.where(step == 0, torch.zeros_like(quotient), quotient.round().clamp(0, 15))
    code = code.to(torch.uint8).reshape(*x.shape[:-1], d // 2, 2)
    pair = torch.cat([step, lo], -1)
    pair = torch.where(bad, torch.full_like(pair, math.nan), pair)
    packed = code[..., 0] | (code[..., 1] << 4)
    return torch.cat([packed, pair.flatten(-2).contiguous().view(torch.uint8)], -1)


def widen(rows):
    """[..., 5 D / 8] bytes -> the [..., D] float32 values they stand for."""
    d = rows.shape[-1] * 8 // 5
    packed = rows[..., :d // 2]
    code = torch.stack([packed & 15, packed >> 4], -1).reshape(*rows.shape[:-1], d // GROUP, GROUP)
    pair = rows[..., d // 2:].contiguous().view(torch.float16).reshape(*rows.shape[:-1], d // GROUP, 2, 1).double()
    return _round16(pair[..., 1, :] + code.double() * pair[..., 0, :]).float().reshape(*rows.shape[:-1], d)


# ------------------------------------------------------------------------------- the inputs

def _normal(gen, shape, heads, head_dim):
    """K or V rows: normal values around a mean and with a spread of each channel's own."""
    mean = torch.randn(heads, 1, head_dim, generator=gen, device=DEVICE)
    spread = 0.5 + torch.rand(heads, 1, head_dim, generator=gen, device=DEVICE)
    return torch.randn(*shape, generator=gen, device=DEVICE) * spread + 0.5 * mean


def _pool(gen, blocks, case, kind):
    shape = (blocks, case["kv_heads"], case["block_size"], case["head_dim"])
    x = _normal(gen, shape, case["kv_heads"], case["head_dim"])
    return quantise(x) if kind == "kv4" else x.to(DTYPES[kind])


def _lengths(gen, case):
    return torch.randint(case["lo"], case["hi"] + 1, (case["seqs"],), generator=gen, device=DEVICE, dtype=torch.int32)


def _tables(lens, block_size, width, perm, first):
    """Tables of ceil(len / block_size) blocks a sequence, taken from perm[first:]; -1 beyond; and the next free place."""
    need = (lens.long() + block_size - 1) // block_size
    start = first + need.cumsum(0) - need
    col = torch.arange(width, device=DEVICE)
    at = (start[:, None] + col).clamp(max=perm.numel() - 1)
    table = torch.where(col < need[:, None], perm[at], torch.full_like(at, -1))
    return table.to(torch.int32).contiguous(), first + int(need.sum())


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    bs, heads, d = case["block_size"], case["kv_heads"], case["head_dim"]
    s = dict(case=case)
    if case["op"] == "append":
        tokens = case["tokens"]
        # a decode step's tokens land anywhere in blocks of their own; a chunk's fill its sequence's blocks
        used = tokens if case["scattered"] else -(-tokens // bs)
        blocks = max(2, int(used * 1.25))
        perm = torch.randperm(blocks, generator=gen, device=DEVICE)[:used]
        at = torch.arange(tokens, device=DEVICE)
        if case["scattered"]:
            s["slots"] = perm * bs + torch.randint(0, bs, (tokens,), generator=gen, device=DEVICE)
        else:
            s["slots"] = perm[at // bs] * bs + at % bs
        for n in ("k", "v"):
            s[n] = _normal(gen, (tokens, heads, 1, d), heads, d).reshape(tokens, heads, d).to(DTYPES[case["dtype"]])
            s[n + "_cache"] = _pool(gen, blocks, case, "kv4")
            s[n + "_wide"] = torch.zeros(used, heads, bs, d, dtype=DTYPES[case["dtype"]], device=DEVICE)
        s["pairs"] = torch.stack([perm, torch.arange(used, device=DEVICE)], -1).contiguous()
    elif case["op"] == "expand":
        n = case["blocks"]
        blocks = max(2, int(n * 1.25))
        src = torch.randperm(blocks, generator=gen, device=DEVICE)[:n]
        dst = torch.randperm(n, generator=gen, device=DEVICE)
        s["pairs"] = torch.stack([src, dst], -1).contiguous()
        for name in ("k", "v"):
            s[name + "_cache"] = _pool(gen, blocks, case, "kv4")
            s[name + "_wide"] = torch.zeros(n, heads, bs, d, dtype=DTYPES[case["dtype"]], device=DEVICE)
    else:
        lens = s["lens"] = _lengths(gen, case)
        hi = case["hi"]
        width = max(1, -(-hi // bs))
        blocks = max(2, int(int(((lens.long() + bs - 1) // bs).sum()) * 1.1))
        if case["op"] == "evict":  # the pools are among its outputs: their size does not go by the lengths drawn
            s["keep"] = torch.full_like(lens, case["keep"])
            left = torch.minimum(lens, s["keep"])
            blocks = case["seqs"] * (width + -(-case["keep"] // bs)) + 1
        perm = torch.randperm(blocks, generator=gen, device=DEVICE)
        s["tables"], used = _tables(lens, bs, width, perm, 0)
        if case["op"] == "evict":
            s["new_tables"], _ = _tables(left, bs, max(1, -(-case["keep"] // bs)), perm, used)
            s["k_cache"], s["v_cache"] = (_pool(gen, blocks, case, case["pool"]) for _ in range(2))
            # accumulated probabilities: few heavy rows, many light ones, and equal ones among them
            w = torch.rand(case["seqs"], heads, max(1, hi), generator=gen, device=DEVICE) ** 8
            s["weights"] = torch.where(w < 1e-3, torch.zeros_like(w), w)
            s["weights_out"] = torch.zeros_like(s["weights"])
            s["kept"] = torch.full((case["seqs"], heads, case["keep"]), -1, dtype=torch.int32, device=DEVICE)
        else:
            s["scale"] = d ** -0.5
            q = torch.randn(case["seqs"], case["q_heads"], d, generator=gen, device=DEVICE)
            s["q"] = q.to(DTYPES[case["dtype"]])
            s["k_cache"] = _pool(gen, blocks, case, case.get("pool", "kv4"))
            if case["op"] == "decode":
                s["v_cache"] = _pool(gen, blocks, case, "kv4")
                s["out"] = torch.zeros(q.shape, dtype=DTYPES[case["out"]], device=DEVICE)
            else:
                s["weights"] = torch.rand(case["seqs"], heads, max(1, hi), generator=gen, device=DEVICE)
                s["tracked"] = (lens - 1).clamp(min=0)  # the newest token has no accumulator yet
                s["weights_out"] = torch.zeros_like(s["weights"])
    return s


# ------------------------------------------------------------------------------ the operators

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_append(s):
    import paged_kv_cache_310_gb300 as pkv
    pkv.paged_kv4_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
    pkv.paged_kv4_expand(s["pairs"], s["k_cache"], s["v_cache"], s["k_wide"], s["v_wide"])
    return s["k_wide"], s["v_wide"]


def _own_expand(s):
    import paged_kv_cache_310_gb300 as pkv
    pkv.paged_kv4_expand(s["pairs"], s["k_cache"], s["v_cache"], s["k_wide"], s["v_wide"])
    return s["k_wide"], s["v_wide"]


def _own_decode(s):
    import paged_kv_cache_310_gb300 as pkv
    return pkv.paged_attention_decode_kv4(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"],
                                          s["out"], max_context_len=s["case"]["hi"])


def _own_weights(s):
    import paged_kv_cache_310_gb300 as pkv
    return pkv.paged_attention_weights(s["q"], s["k_cache"], s["tables"], s["lens"], s["scale"], s["weights"],
                                       weights_out=s["weights_out"], tracked_lens=s["tracked"],
                                       max_context_len=s["case"]["hi"])


def _own_evict(s):
    import paged_kv_cache_310_gb300 as pkv
    pkv.paged_kv_evict(s["weights"], s["tables"], s["lens"], s["keep"], s["new_tables"], s["k_cache"], s["v_cache"],
                       s["weights_out"], s["kept"], recent=s["case"]["recent"], max_context_len=s["case"]["hi"])
    return s["kept"], s["weights_out"], s["k_cache"], s["v_cache"]


def _plain_expand(s):
    src, dst = s["pairs"].unbind(-1)
    for n in ("k", "v"):
        s[n + "_wide"][dst] = widen(s[n + "_cache"][src]).to(s[n + "_wide"].dtype)
    return s["k_wide"], s["v_wide"]


def _plain_append(s):
    bs = s["case"]["block_size"]
    for n in ("k", "v"):
        s[n + "_cache"][s["slots"] // bs, :, s["slots"] % bs] = quantise(s[n])
    return _plain_expand(s)


def _rows(pool, tables):
    """Each sequence's rows through its block table, as float32 [S, heads, padded length, D]."""
    got = pool[tables.clamp(min=0).long()]
    got = widen(got) if pool.dtype == torch.uint8 else got.float()
    n, width, heads, bs, d = got.shape
    return got.transpose(1, 2).reshape(n, heads, width * bs, d)


def _probabilities(s):
    """[S, KV heads, query heads of each, padded length] softmax over the first lens tokens, and the mask of those."""
    k = _rows(s["k_cache"], s["tables"])
    n, heads, length, d = k.shape
    q = s["q"].float().reshape(n, heads, -1, d)
    seen = torch.arange(length, device=DEVICE) < s["lens"][:, None]
    x = (q @ k.transpose(-1, -2)) * s["scale"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    x = x - x.amax(-1, keepdim=True).masked_fill(s["lens"][:, None, None, None] == 0, 0)
    e = x.exp()
    return e / e.sum(-1, keepdim=True).masked_fill(s["lens"][:, None, None, None] == 0, 1), seen


def _plain_decode(s):
    p, seen = _probabilities(s)
    v = _rows(s["v_cache"], s["tables"]).masked_fill(~seen[:, None, :, None], 0)
    return (p @ v).reshape(s["q"].shape).to(s["out"].dtype)


def _plain_weights(s):
    p, seen = _probabilities(s)
    width = s["weights"].shape[-1]
    at = torch.arange(width, device=DEVICE)
    before = torch.where((at < s["tracked"][:, None])[:, None], s["weights"], torch.zeros_like(s["weights"]))
    s["weights_out"].copy_(torch.where(seen[:, None, :width], before + p.sum(2)[..., :width], s["weights_out"]))
    return s["weights_out"]


def _plain_evict(s):
    case, w = s["case"], s["weights"]
    n_seqs, heads, width = w.shape
    at = torch.arange(width, device=DEVICE)
    left = torch.minimum(s["lens"], s["keep"])
    last = s["lens"] - left.clamp(max=case["recent"])
    order = torch.sort(torch.where(w.isnan(), torch.full_like(w, -math.inf), w), descending=True, stable=True).indices
    rank = (at >= last[:, None]).int() - (at >= s["lens"][:, None]).int() * 2  # 1: kept, 0: by weight, -1: no row
    rank = rank[:, None].expand_as(w).gather(-1, order)
    order = order.gather(-1, torch.sort(rank, descending=True, stable=True).indices)
    chosen = torch.zeros_like(order).scatter_(-1, order, (at < left[:, None])[:, None].expand_as(order).long()) > 0
    seq, head, row = chosen.nonzero().unbind(-1)  # ascending rows of each (sequence, head)
    place = (chosen.cumsum(-1) - 1)[seq, head, row]
    s["kept"][seq, head, place] = row.int()
    s["weights_out"][seq, head, place] = w[seq, head, row]
    bs = case["block_size"]
    src, dst = s["tables"].long()[seq, row // bs], s["new_tables"].long()[seq, place // bs]
    for n in ("k_cache", "v_cache"):
        s[n][dst, head, place % bs] = s[n][src, head, row % bs]
    return s["kept"], s["weights_out"], s["k_cache"], s["v_cache"]


_own = dict(append=_own_append, expand=_own_expand, decode=_own_decode, weights=_own_weights, evict=_own_evict)
_plain = dict(append=_plain_append, expand=_plain_expand, decode=_plain_decode, weights=_plain_weights,
              evict=_plain_evict)


# ----------------------------------------------------------------------- what a pass cannot do without

def work(case):
    heads, d, op = case["kv_heads"], case["head_dim"], case["op"]
    row4 = d * 5 // 8
    if op == "append":
        rows = 2 * case["tokens"] * heads
        blocks = case["tokens"] if case["scattered"] else -(-case["tokens"] // case["block_size"])
        wide = 2 * blocks * heads * case["block_size"]
        # the new rows read and written, then their blocks read and written wide (16 bytes a pair)
        return dict(bytes=rows * (d * BYTES[case["dtype"]] + row4) + 8 * case["tokens"]
                    + wide * (row4 + d * BYTES[case["dtype"]]) + 16 * blocks, flops=6 * rows * d + 2 * wide * d)
    if op == "expand":
        rows = 2 * case["blocks"] * heads * case["block_size"]
        return dict(bytes=rows * (row4 + d * BYTES[case["dtype"]]) + 16 * case["blocks"], flops=2 * rows * d)
    tokens = case["seqs"] * (case["lo"] + case["hi"]) / 2
    table = 4 * tokens / case["block_size"] + 4 * case["seqs"]
    if op == "evict":
        row = d * BYTES[case["pool"]]
        mean = max(1.0, (case["lo"] + case["hi"]) / 2)
        kept = case["seqs"] * min(mean, case["keep"])
        return dict(bytes=tokens * heads * 4 + kept * heads * (4 * row + 4 + 4) + 2 * table, flops=4 * tokens * heads)
    group = case["q_heads"] // heads
    ask = case["seqs"] * case["q_heads"] * d
    if op == "decode":
        return dict(bytes=tokens * heads * 2 * row4 + ask * (BYTES[case["dtype"]] + BYTES[case["out"]]) + table,
                    flops=tokens * heads * (4 * group + 4) * d)
    row = row4 if case["pool"] == "kv4" else d * BYTES[case["pool"]]
    return dict(bytes=tokens * heads * (row + 8) + ask * BYTES[case["dtype"]] + table,
                flops=tokens * heads * (2 * group + 2) * d)


# ------------------------------------------------------------------------------- in 64 bits

def _exact_half(x):
    """float64 -> float16 as float64, through a float32 rounded to odd (which a second rounding cannot spoil)."""
    f = x.float()
    over = f.double().abs() > x.abs()
    bits = f.view(torch.int32)
    bits = torch.where(over, bits - 1, bits)
    cut = bits.view(torch.float32)
    odd = torch.where(cut.double() != x, bits | 1, bits).view(torch.float32)
    return torch.where(x == 0, x, odd.half().double())


def _exact_values(rows):
    """float64 values of 4-bit rows: the 16 values of each group listed, then picked by code."""
    d = rows.shape[-1] * 8 // 5
    pair = rows[..., d // 2:].contiguous().view(torch.float16).double().reshape(*rows.shape[:-1], d // GROUP, 2)
    ladder = _exact_half(pair[..., 1:] + torch.arange(16, dtype=torch.float64, device=rows.device) * pair[..., :1])
    low, high = rows[..., :d // 2] % 16, rows[..., :d // 2] // 16
    codes = torch.stack((low, high), -1).flatten(-2).reshape(*rows.shape[:-1], d // GROUP, GROUP).long()
    return ladder.gather(-1, codes).flatten(-2)


def _exact_row(x):
    """The numpy float64 values that a [rows, D] numpy float64 array is held as."""
    out = np.empty_like(x)
    for at in range(0, x.shape[1], GROUP):
        g = np.clip(x[:, at:at + GROUP], -LARGEST, LARGEST)
        lo = g.min(1, keepdims=True).astype(np.float16).astype(np.float64)
        spread = np.maximum(0, g.max(1, keepdims=True).astype(np.float32) - lo.astype(np.float32)).astype(np.float64)
        step = (spread / 15).astype(np.float32).astype(np.float16).astype(np.float64)
        up = (g.astype(np.float32) - lo.astype(np.float32)).astype(np.float64)
        code = np.where(step > 0, np.clip(np.rint(up / np.where(step > 0, step, 1)), 0, 15), 0)
        out[:, at:at + GROUP] = (lo + code * step).astype(np.float16)
    return out


def _exact_sequence(pool, table, n, bs):
    blocks = pool[table[:-(-n // bs)].long()]
    got = _exact_values(blocks) if pool.dtype == torch.uint8 else blocks.double()
    return got.transpose(0, 1).reshape(pool.shape[1], -1, got.shape[-1])[:, :n]


def exact(case, seed):
    s = prepare(case, seed)
    bs = case["block_size"]
    if case["op"] in ("append", "expand"):
        src, dst = s["pairs"][:, 0], s["pairs"][:, 1]
        outs = []
        for n in ("k", "v"):
            wide = _exact_values(s[n + "_cache"][src])
            if case["op"] == "append":
                place = torch.full((s[n + "_cache"].shape[0],), -1, dtype=torch.int64, device=DEVICE)
                place[src] = torch.arange(src.numel(), device=DEVICE)
                rows = s[n].double().cpu().numpy()
                held = torch.from_numpy(_exact_row(rows.reshape(-1, rows.shape[-1])).reshape(rows.shape)).to(DEVICE)
                wide[place[s["slots"] // bs], :, s["slots"] % bs] = held
            out = torch.empty_like(wide)
            out[dst] = wide
            outs.append(out)
        return tuple(outs)
    lens = s["lens"].tolist()
    if case["op"] == "evict":
        kept = np.full(s["kept"].shape, -1, dtype=np.int32)
        weights = s["weights"].double().cpu().numpy()
        moved = np.zeros_like(weights)
        for i, n in enumerate(lens):
            k = min(n, case["keep"])
            r = min(k, case["recent"])
            for h in range(case["kv_heads"]):
                by_weight = np.lexsort((np.arange(n - r), -weights[i, h, :n - r]))[:k - r]
                rows = np.sort(np.concatenate([by_weight, np.arange(n - r, n)]))
                kept[i, h, :k] = rows
                moved[i, h, :k] = weights[i, h, rows]
        return kept, moved, None, None  # the pools: copies of their own rows
    out = torch.zeros(s["q"].shape if case["op"] == "decode" else s["weights"].shape, dtype=torch.float64, device=DEVICE)
    for i, n in enumerate(lens):
        if n == 0:
            continue
        k = _exact_sequence(s["k_cache"], s["tables"][i], n, bs)
        q = s["q"][i].double().reshape(case["kv_heads"], -1, k.shape[-1])
        p = torch.softmax(torch.bmm(q, k.mT) * s["scale"], -1)
        if case["op"] == "decode":
            v = _exact_sequence(s["v_cache"], s["tables"][i], n, bs)
            out[i] = torch.bmm(p, v).reshape(out[i].shape)
        else:
            out[i, :, :n] = p.sum(1)
            t = int(s["tracked"][i])
            out[i, :, :t] += s["weights"][i, :, :t].double()
    return out
