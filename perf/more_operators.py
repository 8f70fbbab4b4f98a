"""The step of a model with rotary positions and sliding-window layers, as measured cases.

Four operators around paged K/V pools ``[num_blocks, num_kv_heads, block_size, head_dim]``:

* rotary  -- queries and keys normed per head and rotated by their positions, in one pass;
* append  -- the same on the way into the cache: keys (normed, rotated) and values into their
  slots, queries into a buffer;
* decode  -- single-token attention over the last ``window`` tokens and the first ``sinks``;
* prefill -- the same for several new tokens per sequence.

Blocks that a window has left behind have no block any more: their table entries are -1.

``run`` computes the operators in elementary torch operations where ``own`` is false and
calls the library where it is true.  ``exact`` states them again in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
DEVICE = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of 64 sequences whose keys go to a 4-bit pool afterwards: latency
        dict(name="rotary step", op="rotary", tokens=64, q_heads=64, kv_heads=8, head_dim=128, rotary_dim=128,
             interleaved=False, norm=True, factor=1.0, dtype="bf16", far=131072),
        # an odd number of prompt tokens, a quarter of each head rotated, in pairs of neighbours
        dict(name="rotary prompt part", op="rotary", tokens=4097, q_heads=32, kv_heads=8, head_dim=64, rotary_dim=16,
             interleaved=True, norm=False, factor=1.0, dtype="f32", far=4097),
        # the new token of a single chat
        dict(name="append one", op="append", tokens=1, q_heads=32, kv_heads=8, head_dim=128, rotary_dim=128,
             interleaved=False, norm=False, factor=1.0, dtype="f16", far=32768, block_size=16, fused=True),
        # the step of a batch of long contexts, with a scaled rotation and norms
        dict(name="append batch", op="append", tokens=256, q_heads=64, kv_heads=8, head_dim=128, rotary_dim=64,
             interleaved=False, norm=True, factor=1.25, dtype="bf16", far=1000000, block_size=32, fused=True),
        # a long prompt, q, k and v as the projection left them: parts of one row
        dict(name="append prompt", op="append", tokens=16384, q_heads=64, kv_heads=8, head_dim=128, rotary_dim=128,
             interleaved=False, norm=True, factor=1.0, dtype="bf16", far=16384, block_size=16, fused=True),
        # one long chat in a windowed layer: latency
        dict(name="decode one", op="decode", seqs=1, lo=100001, hi=100001, window=1024, sinks=4, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, dtype="f16"),
        # narrow windows at head_dim 64
        dict(name="decode narrow", op="decode", seqs=64, lo=100, hi=20000, window=128, sinks=0, q_heads=64, kv_heads=8,
             head_dim=64, block_size=16, dtype="bf16"),
        # odd window and sinks in f32, lengths from nothing
        dict(name="decode f32", op="decode", seqs=32, lo=0, hi=6000, window=1021, sinks=5, q_heads=32, kv_heads=8,
             head_dim=128, block_size=8, dtype="f32"),
        # the batch of 128 sequences with eight query heads per KV head, a wide window
        dict(name="decode batch", op="decode", seqs=128, lo=512, hi=32768, window=4096, sinks=64, q_heads=64, kv_heads=8,
             head_dim=128, block_size=16, dtype="bf16"),
        # drafted tokens to verify: a few new tokens for each of many sequences
        dict(name="prefill drafts", op="prefill", seqs=32, lo=2000, hi=20000, new_lo=3, new_hi=8, window=4096, sinks=4,
             q_heads=64, kv_heads=8, head_dim=128, block_size=16, dtype="bf16"),
        # short prompts of odd lengths from their first token on, a narrow window
        dict(name="prefill ragged", op="prefill", seqs=9, lo=0, hi=300, new_lo=1, new_hi=517, window=130, sinks=3,
             q_heads=16, kv_heads=4, head_dim=64, block_size=32, dtype="f16"),
        # chunks of four long prompts
        dict(name="prefill chunks", op="prefill", seqs=4, lo=0, hi=6000, new_lo=1000, new_hi=2000, window=1024, sinks=0,
             q_heads=64, kv_heads=8, head_dim=128, block_size=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "decode", "decode", "prefill", "prefill"])
    heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 16, 32])
    case = dict(op=op, kv_heads=heads, head_dim=rng.choice([64, 128, 128]))
    if op in ("rotary", "append"):
        case["q_heads"] = heads * rng.choice([1, 2, 3, 4, 6, 7, 8, 8, 12, 16])
        case.update(tokens=_log(rng, 1, max(1, 1300000 // (case["q_heads"] + 2 * heads))),
                    rotary_dim=rng.choice([case["head_dim"], 16 * rng.randint(1, case["head_dim"] // 16)]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.5, factor=rng.choice([1.0, 1.0, 1.139]),
                    dtype=rng.choice(["f32", "f16", "bf16", "bf16"]), far=_log(rng, 16, 1000000))
        if case["dtype"] == "f32":
            case["tokens"] = (case["tokens"] + 1) // 2
        if op == "append":
            case.update(block_size=rng.choice([8, 16, 16, 32, 64]), fused=rng.random() < 0.6)
        return case
    case.update(block_size=rng.choice([8, 16, 16, 32, 64]), window=_log(rng, 1, 8192),
                sinks=rng.choice([0, 0, 1, 4, 4, 5, 64, rng.randint(0, 300)]))
    hi = _log(rng, 1, 100000)
    case.update(hi=hi, lo=min(hi, rng.choice([0, 1, hi // 4, hi // 2, hi])))
    seen = min(hi, case["window"] + case["sinks"])
    if op == "decode":
        dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
        group = rng.choice([1, 2, 3, 4, 6, 7, 8, 8] + ([12, 16] if dtype != "f32" else []))
        return dict(case, seqs=_log(rng, 1, max(1, min(256, (1500000 if dtype == "f32" else 3000000) // (seen * heads)))),
                    q_heads=heads * group, dtype=dtype)
    case.update(q_heads=heads * rng.choice([1, 2, 3, 4, 6, 7, 8, 8, 12, 16]), dtype=rng.choice(["f16", "bf16"]))
    new = _log(rng, 1, 4096)
    case.update(new_hi=new, new_lo=max(1, min(new, rng.choice([1, new // 2, new]))))
    # padded scores (sequences x query heads x new tokens x tokens) within the listed cases'
    pairs = case["q_heads"] * new * (hi + new)
    while pairs > 4000000000 and case["new_hi"] > 1:
        case.update(new_hi=case["new_hi"] // 2, new_lo=max(1, case["new_lo"] // 2))
        pairs = case["q_heads"] * case["new_hi"] * (hi + case["new_hi"])
    return dict(case, seqs=_log(rng, 1, max(1, min(64, 4000000000 // pairs, 1500000 // (heads * (hi + case["new_hi"]))))))


# ------------------------------------------------------------------------------- the inputs

def _frequencies(case):
    """base^(-2 i / rotary_dim), the low frequencies divided by 8 where the rotation is scaled."""
    i = torch.arange(0, case["rotary_dim"], 2, dtype=torch.float64)
    freq = 10000.0 ** (-i / case["rotary_dim"])
    if case["factor"] != 1.0:
        kept = ((freq * 8192 / (2 * math.pi) - 1) / 31).clamp(0, 1)  # turns within the first 8192 tokens: from 1 to 32
        freq = freq / 8 * (1 - kept) + freq * kept
    return freq.to(DEVICE)


def _tables(kept, perm):
    """Block tables with blocks of perm where `kept` [S, width] says that a block is held, -1 elsewhere."""
    place = kept.flatten().cumsum(0).reshape(kept.shape) - 1
    return torch.where(kept, perm[place.clamp(min=0)], torch.full_like(place, -1)).to(torch.int32).contiguous()


def _spread(gen, lo, hi, n):
    """n whole numbers from lo to hi, evenly spread, in an order of the seed's."""
    x = torch.linspace(lo, hi, n, dtype=torch.float64, device=DEVICE) if n > 1 else torch.full((1,), (lo + hi) / 2, device=DEVICE)
    return x.round().to(torch.int32)[torch.randperm(n, generator=gen, device=DEVICE)].contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    heads, hq, d, dtype = case["kv_heads"], case["q_heads"], case["head_dim"], DTYPES[case["dtype"]]
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=DEVICE)
    s = dict(case=case)
    if case["op"] in ("rotary", "append"):
        t = case["tokens"]
        s["inv_freq"] = _frequencies(case)
        if case.get("fused"):  # one row a token: the heads of q, of k, of v
            rows = rand(t, hq + 2 * heads, d).to(dtype)
            s["q"], s["k"], s["v"] = rows.split([hq, heads, heads], 1)
        else:
            s["q"], s["k"], s["v"] = (rand(t, h, d).to(dtype) for h in (hq, heads, heads))
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"], s["k_weight"] = ((1 + 0.2 * rand(d)).to(dtype) for _ in range(2))
        if t > 256:  # a prompt's tokens follow one another
            first = int(torch.randint(0, max(1, case["far"] - t) + 1, (1,), generator=gen, device=DEVICE))
            s["positions"] = torch.arange(first, first + t, device=DEVICE, dtype=torch.int32)
        else:
            s["positions"] = torch.randint(0, case["far"], (t,), generator=gen, device=DEVICE, dtype=torch.int32)
        s["q_out"] = torch.zeros(t, hq, d, dtype=dtype, device=DEVICE)
        if case["op"] == "rotary":
            s["k_out"] = torch.zeros(t, heads, d, dtype=dtype, device=DEVICE)
            return s
        bs = case["block_size"]
        used = -(-t // bs) if t > 256 else t
        blocks = max(2, int(used * 1.25))
        perm = torch.randperm(blocks, generator=gen, device=DEVICE)[:used]
        at = torch.arange(t, device=DEVICE)
        if t > 256:
            s["slots"] = perm[at // bs] * bs + at % bs
        else:
            s["slots"] = perm * bs + torch.randint(0, bs, (t,), generator=gen, device=DEVICE)
        s["k_cache"], s["v_cache"] = (rand(blocks, heads, bs, d).to(dtype) for _ in range(2))
        return s

    n, bs, window, sinks = case["seqs"], case["block_size"], case["window"], case["sinks"]
    new = torch.ones(n, dtype=torch.int32, device=DEVICE)
    lens = torch.randint(case["lo"], case["hi"] + 1, (n,), generator=gen, device=DEVICE, dtype=torch.int32)
    longest = case["hi"]
    if case["op"] == "prefill":  # lo to hi tokens before the chunk
        new = _spread(gen, case["new_lo"], case["new_hi"], n)
        lens = lens + new
        longest += case["new_hi"]
    s.update(lens=lens, longest=longest, scale=d ** -0.5)
    # blocks that hold a token which some new token sees
    width = max(1, -(-longest // bs))
    first = torch.arange(width, device=DEVICE) * bs
    n_blocks = (lens.long() + bs - 1) // bs
    oldest = (lens - new - window + 1)[:, None]
    kept = (first < n_blocks[:, None] * bs) & ((first + bs > oldest) | (first < sinks))
    blocks = max(2, int(int(kept.sum()) * 1.1))
    s["tables"] = _tables(kept, torch.randperm(blocks, generator=gen, device=DEVICE))
    s["k_cache"], s["v_cache"] = (rand(blocks, heads, bs, d).to(dtype) for _ in range(2))
    if case["op"] == "prefill":
        s["start"] = torch.cat([new.new_zeros(1), new.cumsum(0).to(torch.int32)])
        s["q"] = rand(int(new.sum()), hq, d).to(dtype)
    else:
        s["q"] = rand(n, hq, d).to(dtype)
    s["out"] = torch.zeros_like(s["q"])
    return s


# ------------------------------------------------------------------------------ the operators

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_rotary(s):
    import paged_kv_cache_310_gb300 as pkv
    case = s["case"]
    pkv.paged_qk_rotary(s["q"], s["k"], s["positions"], s["q_out"], s["k_out"], s["inv_freq"],
                        interleaved=case["interleaved"], factor=case["factor"], q_weight=s["q_weight"],
                        k_weight=s["k_weight"], eps=EPS)
    return s["q_out"], s["k_out"]


def _own_append(s):
    import paged_kv_cache_310_gb300 as pkv
    case = s["case"]
    pkv.paged_kv_append_rotary(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                               s["q_out"], s["inv_freq"], interleaved=case["interleaved"], factor=case["factor"],
                               q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_decode(s):
    import paged_kv_cache_310_gb300 as pkv
    case = s["case"]
    return pkv.paged_attention_decode_window(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"],
                                             s["out"], window=case["window"], sinks=case["sinks"],
                                             max_context_len=s["longest"])


def _own_prefill(s):
    import paged_kv_cache_310_gb300 as pkv
    case = s["case"]
    return pkv.paged_attention_prefill_window(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["start"],
                                              s["scale"], s["out"], window=case["window"], sinks=case["sinks"],
                                              max_context_len=s["longest"])


def _normed_rotated(s, x, weight):
    case = s["case"]
    r, y = case["rotary_dim"], x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.float()
    angle = s["positions"].double()[:, None, None] * s["inv_freq"]
    c, sn = (case["factor"] * angle.cos()).float(), (case["factor"] * angle.sin()).float()
    if case["interleaved"]:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([turned, y[..., r:]], -1).to(x.dtype)


def _plain_rotary(s):
    s["q_out"].copy_(_normed_rotated(s, s["q"], s["q_weight"]))
    s["k_out"].copy_(_normed_rotated(s, s["k"], s["k_weight"]))
    return s["q_out"], s["k_out"]


def _plain_append(s):
    bs = s["case"]["block_size"]
    s["q_out"].copy_(_normed_rotated(s, s["q"], s["q_weight"]))
    s["k_cache"][s["slots"] // bs, :, s["slots"] % bs] = _normed_rotated(s, s["k"], s["k_weight"])
    s["v_cache"][s["slots"] // bs, :, s["slots"] % bs] = s["v"]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _softmax_product(x, seen, v):
    """softmax of x over the places that are seen, times v; zeros where none is."""
    top = x.masked_fill_(~seen, -math.inf).amax(-1, keepdim=True)
    e = x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = e.sum(-1, keepdim=True)
    return e.div_(torch.where(total == 0, torch.ones_like(total), total)) @ v


def _plain_decode(s):
    case, bs = s["case"], s["case"]["block_size"]
    n = s["lens"].long()[:, None]
    # the tokens that a sequence sees, in order: its sinks, then its window
    most = min(case["hi"], case["window"] + case["sinks"])
    at = torch.arange(max(1, most), device=DEVICE)
    cut = n > case["window"] + case["sinks"]
    place = torch.where(cut & (at >= case["sinks"]), n - case["window"] - case["sinks"] + at, at)
    seen = at < n.clamp(max=most)
    place = torch.where(seen, place, torch.zeros_like(place))
    block = s["tables"].long().gather(1, place // bs).clamp(min=0)
    k, v = (c[block, :, place % bs].float().transpose(1, 2) for c in (s["k_cache"], s["v_cache"]))  # [S, heads, most, D]
    v = v.masked_fill(~seen[:, None, :, None], 0)
    q = s["q"].float().reshape(n.shape[0], case["kv_heads"], -1, case["head_dim"])
    x = (q @ k.transpose(-1, -2)) * s["scale"]
    s["out"].copy_(_softmax_product(x, seen[:, None, None], v).reshape(s["q"].shape))
    return s["out"]


def _plain_prefill(s):
    case, bs = s["case"], s["case"]["block_size"]
    heads, d = case["kv_heads"], case["head_dim"]
    lens, start = s["lens"].long(), s["start"].long()
    seqs, new = lens.numel(), start[1:] - start[:-1]
    rows = torch.arange(case["new_hi"], device=DEVICE)
    live = rows < new[:, None]                                              # [S, rows]
    row = torch.where(live, start[:-1, None] + rows, torch.zeros_like(rows))
    q = s["q"][row].float().reshape(seqs, -1, heads, case["q_heads"] // heads, d).permute(0, 2, 3, 1, 4)
    k, v = (c[s["tables"].long().clamp(min=0)].float().transpose(1, 2).reshape(seqs, heads, 1, -1, d)
            for c in (s["k_cache"], s["v_cache"]))
    at = torch.arange(k.shape[3], device=DEVICE)
    p = ((lens - new)[:, None] + rows)[..., None]
    seen = (at <= p) & ((at > p - case["window"]) | (at < case["sinks"])) & live[..., None]   # [S, rows, tokens]
    v = v.masked_fill(~seen.any(1)[:, None, None, :, None], 0)
    o = _softmax_product((q @ k.transpose(-1, -2)).mul_(s["scale"]), seen[:, None, None], v)
    s["out"][row[live]] = o.permute(0, 3, 1, 2, 4).reshape(seqs, -1, case["q_heads"], d)[live].to(s["out"].dtype)
    return s["out"]


_own = dict(rotary=_own_rotary, append=_own_append, decode=_own_decode, prefill=_own_prefill)
_plain = dict(rotary=_plain_rotary, append=_plain_append, decode=_plain_decode, prefill=_plain_prefill)


# ----------------------------------------------------------------------- what a pass cannot do without

def _sum_seen(lo, hi, most):
    """The sum over n = lo..hi of min(n, most)."""
    ramp = lambda m: m * (m + 1) // 2
    small = min(hi, most)
    total = ramp(small) - ramp(lo - 1) if lo <= small else 0
    return total + max(0, hi - max(lo - 1, most)) * most


def work(case):
    heads, hq, d, size = case["kv_heads"], case["q_heads"], case["head_dim"], BYTES[case["dtype"]]
    if case["op"] in ("rotary", "append"):
        t, rows = case["tokens"], hq + heads
        moved = rows + (heads if case["op"] == "append" else 0)
        once = 4 * case["rotary_dim"] + (2 * d * size if case["norm"] else 0)
        return dict(bytes=2 * t * moved * d * size + t * (12 if case["op"] == "append" else 4) + once,
                    flops=t * rows * (3 * case["rotary_dim"] + (4 * d if case["norm"] else 0)))
    most, n, bs = case["window"] + case["sinks"], case["seqs"], case["block_size"]
    if case["op"] == "decode":
        tokens = n * _sum_seen(case["lo"], case["hi"], most) / (case["hi"] - case["lo"] + 1)
        return dict(bytes=tokens * heads * 2 * d * size + 2 * n * hq * d * size + 4 * tokens / bs + 4 * n,
                    flops=tokens * hq * 4 * d)
    before, new = (case["lo"] + case["hi"]) // 2, (case["new_lo"] + case["new_hi"]) / 2
    pairs = n * _sum_seen(before + 1, before + int(new), most)
    tokens = n * (min(before, most) + new)  # rows that any new token sees
    return dict(bytes=tokens * heads * 2 * d * size + 2 * n * new * hq * d * size + 4 * tokens / bs + 8 * n,
                flops=pairs * hq * 4 * d)


# ------------------------------------------------------------------------------- in 64 bits

def _exact_rows(s, x, weight):
    """x [T, H, D], each pair of dimensions a complex number that is multiplied by factor e^(i position f)."""
    case = s["case"]
    r, y = case["rotary_dim"], x.double()
    if weight is not None:
        y = y / (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + EPS).sqrt() * weight.double()
    i = torch.arange(r // 2, device=DEVICE)
    one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
    z = torch.complex(y[..., one], y[..., two])
    angle = torch.outer(s["positions"].double(), s["inv_freq"])[:, None]
    z = z * torch.polar(torch.full_like(angle, case["factor"]), angle)
    out = y.clone()
    out[..., one], out[..., two] = z.real, z.imag
    return out


def _exact_attention(s, i, q, positions):
    """Softmax products in 64 bits of q [rows, Hq, D], new tokens of sequence i at `positions`, a KV head at a time."""
    case, bs = s["case"], s["case"]["block_size"]
    heads, last = case["kv_heads"], int(positions[-1])
    oldest = max(0, int(positions[0]) - case["window"] + 1)
    place = torch.cat([torch.arange(min(case["sinks"], oldest), device=DEVICE), torch.arange(oldest, last + 1, device=DEVICE)])
    block = s["tables"][i].long()[torch.div(place, bs, rounding_mode="floor")]
    gap = positions[:, None] - place
    hidden = (gap < 0) | ((gap >= case["window"]) & (place >= case["sinks"]))
    outs = []
    for g in range(heads):
        k, v = (c[block, g, place % bs].double() for c in (s["k_cache"], s["v_cache"]))
        mine = q[:, g * (q.shape[1] // heads):(g + 1) * (q.shape[1] // heads)].double()
        x = torch.einsum("rhd,nd->hrn", mine, k) * s["scale"]
        p = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
        outs.append(torch.einsum("hrn,nd->rhd", p, v))
    return torch.cat(outs, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rotary", "append"):
        q, k = _exact_rows(s, s["q"], s["q_weight"]), _exact_rows(s, s["k"], s["k_weight"])
        if case["op"] == "rotary":
            return q, k
        bs, pools = case["block_size"], [s["k_cache"].double(), s["v_cache"].double()]
        for pool, rows in zip(pools, (k, s["v"].double())):
            pool[torch.div(s["slots"], bs, rounding_mode="floor"), :, s["slots"] % bs] = rows
        return q, pools[0], pools[1]
    lens = s["lens"].tolist()
    starts = s["start"].tolist() if case["op"] == "prefill" else list(range(len(lens) + 1))
    pairs = sum((b - a) * min(n, case["window"] + case["sinks"] + b - a) for n, a, b in zip(lens, starts, starts[1:]))
    if pairs * case["q_heads"] * 4 * case["head_dim"] > 1e13:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    for i, n in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        step = max(1, 100000000 // max(1, n * case["q_heads"] // case["kv_heads"]))
        for at in range(a, b, step):
            to = min(b, at + step)
            if n:
                positions = torch.arange(n - (b - at), n - (b - to), device=DEVICE)
                out[at:to] = _exact_attention(s, i, s["q"][at:to], positions)
    return out
