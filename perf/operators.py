"""Workloads of the paged-cache operators, with their plain forms.

Three operators work on a paged K/V cache held in 16 bits, in FP8 or in 4 bits:

  append   rotates q and k by their tokens' positions and writes k and v into
           the cache slots of the tokens (kv.store_kv_rope_paged);
  load     reads rows back out of the cache as 16-bit values (kv.load_kv_paged);
  attend   attention of new tokens over the cached sequences, causal, with an
           optional sliding window and first tokens that stay visible
           (kv.attention_paged), for single tokens and for runs of them.

The 4-bit cache holds e2m1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives), two to a byte with the even element low, and one power-of-two
scale byte (exponent + 127) for each block of 32 dims of a head.

A case is a dict of plain values; `listed()` holds the fixed ones, `draw()`
makes more of the same ranges, `prepare()` makes the inputs on the GPU,
`run()` is one pass and `exact()` the same in 64 bits.
"""
import math
import random

import torch

own = False

LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
FP8 = {"e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3fn": 448.0, "e5m2": 57344.0}
FP4_MIN_SCALE = 27      # smallest scale byte: 2^-100
SRC = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _append(name, tokens, q_heads, kv_heads, dim, rot, cache, page, src="bf16",
            interleaved=False):
    return dict(name=name, kind="append", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads,
                dim=dim, rot=rot, cache=cache, page=page, src=src, interleaved=interleaved)


def _load(name, tokens, kv_heads, dim, cache, scales, page, src="bf16"):
    return dict(name=name, kind="load", tokens=tokens, kv_heads=kv_heads, dim=dim, cache=cache,
                scales=scales, page=page, src=src)


def _attend(name, seqs, queries, context, q_heads, kv_heads, dim, cache, scales, page, window=0,
            sinks=0, src="bf16", ragged=True, mix=1):
    return dict(name=name, kind="attend", seqs=seqs, queries=queries, context=context,
                q_heads=q_heads, kv_heads=kv_heads, dim=dim, cache=cache, scales=scales,
                page=page, window=window, sinks=sinks, src=src, ragged=ragged, mix=mix)


def listed():
    return [
        # one decode step of a small batch: bound by launch latency
        _append("append step", 16, 32, 8, 128, 128, "16", 16),
        # a long prompt into an FP8 cache: bound by HBM
        _append("append prompt e4m3fn", 16384, 32, 8, 128, 128, "e4m3fn", 64),
        # few narrow heads, half of each rotated, odd token count, pages that are no power of two
        _append("append odd e5m2", 1777, 14, 2, 64, 32, "e5m2", 24, "fp16", True),
        # a prompt into a 4-bit cache, and its rows read back (moving a prefix to another cache)
        _append("append and load 4 bit", 8192, 32, 8, 128, 128, "fp4", 64),
        # a prefix out of an FP8 cache with a scale for each token and head
        _load("load prefix e4m3fn", 16384, 8, 128, "e4m3fn", "head", 64),
        # a short prefix, odd row count, one scale for the tensor
        _load("load short e5m2", 333, 2, 64, "e5m2", "tensor", 16, "fp16"),
        # one sequence's next token over a short context: latency
        _attend("decode one", 1, 1, 777, 32, 8, 128, "16", "none", 16, ragged=False),
        # a serving batch's next tokens, long contexts behind a window with first tokens kept
        _attend("decode window e4m3fn", 64, 1, 32768, 32, 8, 128, "e4m3fn", "tensor", 64,
                window=4096, sinks=4, mix=2),
        # a serving batch's next tokens over whole contexts held in 4 bits: bound by HBM
        _attend("decode 4 bit", 32, 1, 32768, 32, 8, 128, "fp4", "block", 64, mix=3),
        # one long prompt over itself: bound by the matrix cores
        _attend("prompt", 1, 8192, 8192, 32, 8, 128, "16", "none", 16, ragged=False),
        # chunks of several prompts over their earlier parts, ragged, window and first tokens
        _attend("chunks window e4m3fn", 6, 1024, 16384, 16, 2, 64, "e4m3fn", "head", 16,
                window=2048, sinks=16, src="fp16", mix=4),
        # the next chunk of two prompts over 4-bit contexts
        _attend("chunks 4 bit", 2, 2048, 8192, 32, 8, 128, "fp4", "block", 64, mix=5),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(("append", "append", "load", "attend", "attend", "attend"))
    src = rng.choice(("bf16", "bf16", "fp16"))
    page = rng.choice((16, 16, 24, 64, 64, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    dim = rng.choice((64, 96, 128, 128))
    cache = rng.choice(("16", "e4m3fn", "e4m3fn", "e5m2", "fp4"))
    scales = {"16": "none", "fp4": "block", "e5m2": "tensor"}.get(cache) or rng.choice(
        ("tensor", "token", "head"))
    group = rng.choice((1, 2, 4, 7, 8))
    tokens = _between(rng, 1, 16384)
    if kind == "append":
        rot = rng.choice((dim, dim, dim // 2))
        case = _append("", tokens, kv_heads * group, kv_heads, dim, rot, cache, page, src,
                       rng.random() < 0.3)
        while case["tokens"] > 1 and work(case)["bytes"] > work(listed()[1])["bytes"]:
            case["tokens"] = case["tokens"] * 2 // 3
    elif kind == "load":
        case = _load("", tokens, kv_heads, dim, cache, scales, page, src)
    else:
        window = rng.choice((0, 0, _between(rng, 16, 4096)))
        queries = rng.choice((1, 1, _between(rng, 2, 16), _between(rng, 17, 2048)))
        case = _attend("", _between(rng, 1, 64), queries, _between(rng, 1, 32768),
                       kv_heads * group, kv_heads, dim, cache, scales, page, window,
                       rng.choice((0, 4, _between(rng, 1, 64))) if window else 0, src,
                       rng.random() < 0.8, rng.randrange(1 << 30))
        case["context"] = max(case["context"], queries)
        big = {c["name"]: c for c in listed()}
        most_bytes, most_flops = work(big["decode 4 bit"])["bytes"], work(big["prompt"])["flops"]
        while case["seqs"] > 1 and (work(case)["bytes"] > most_bytes or
                                    work(case)["flops"] > most_flops or
                                    _plain_size(case) > 2 << 30):
            case["seqs"] = case["seqs"] * 2 // 3
        while case["context"] > 1 and (work(case)["bytes"] > most_bytes or
                                       work(case)["flops"] > most_flops or
                                       _plain_size(case) > 2 << 30):
            case["context"] = case["context"] * 2 // 3
            case["queries"] = min(case["queries"], case["context"])
    del case["name"]
    return case


def _lengths(case):
    """(context length, new tokens) of each sequence; the context counts the new tokens."""
    r = random.Random(case["mix"])
    got = []
    for b in range(case["seqs"]):
        if b == 0 or not case["ragged"]:
            got.append((case["context"], case["queries"]))
        else:
            length = max(1, int(case["context"] * r.random() ** 1.5))
            got.append((length, min(length, max(1, int(case["queries"] * (0.1 + 0.9 * r.random()))))))
    return got


def _far(case):
    """How many tokens back the first new token of any sequence sees, plus the new ones: the
    plain form's keys beside the first tokens."""
    return max((n if not case["window"] else min(n, case["window"] + q - 1))
               for n, q in _lengths(case))


def _plain_size(case):
    """Values of the largest tensor of the plain form."""
    keys = case["sinks"] + _far(case)
    return max(case["seqs"] * case["q_heads"] * case["queries"] * keys,
               case["seqs"] * case["kv_heads"] * case["dim"] * keys)


def _row_bytes(case):
    """Bytes of one token's K row in the cache, with its scales."""
    n = case["kv_heads"] * case["dim"]
    if case["cache"] == "16":
        return 2 * n
    if case["cache"] == "fp4":
        return n // 2 + n // 32
    scales = case.get("scales")
    return n + (4 if scales == "token" else 4 * case["kv_heads"] if scales == "head" else 0)


def _ramp(n, most):
    """The sum of min(x, most) over x = 1 ... n."""
    n = max(0, n)
    m = min(n, most)
    return m * (m + 1) // 2 + (n - m) * most


def work(case):
    if case["kind"] == "append":
        T, H, Hq, D = case["tokens"], case["kv_heads"], case["q_heads"], case["dim"]
        moved = T * (2 * Hq + 2 * H) * D * 2             # q, k and v in, q out
        moved += T * (2 * _row_bytes(case) + 4 + 8 + 4 * case["rot"])
        if case["cache"] == "fp4":                       # the rows are read back
            moved += T * (2 * _row_bytes(case) + 2 * H * D * 2 + 4)
        return {"bytes": moved, "flops": 3 * T * (Hq + H) * case["rot"] + 2 * T * H * D}
    if case["kind"] == "load":
        T, n = case["tokens"], case["kv_heads"] * case["dim"]
        return {"bytes": T * (2 * _row_bytes(case) + 4 * n + 4), "flops": 2 * T * n}
    rows = keys = pairs = 0
    w, s = case["window"] or 1 << 40, case["sinks"]
    for length, n in _lengths(case):
        first = length - n                               # position of the first new token
        low = max(0, first - w + 1)
        rows += n
        keys += length - low + min(s, low)
        # a token at position p sees min(p + 1, w) keys of its window, and
        # min(p + 1 - w, s) first tokens behind it
        pairs += _ramp(length, w) - _ramp(first, w) + _ramp(length - w, s) - _ramp(first - w, s)
    return {"bytes": rows * case["q_heads"] * case["dim"] * 4 + keys * 2 * _row_bytes(case) +
            4 * (keys // case["page"] + 2 * case["seqs"]),
            "flops": 4 * pairs * case["q_heads"] * case["dim"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

class State:
    pass


def _rows(g, n, heads, dim, src, outliers):
    """[n, heads, dim] normal values, one in a thousand of them fifty times as large."""
    x = torch.randn((n, heads, dim), generator=g, device="cuda")
    if outliers:
        x *= torch.where(torch.rand((n, heads, dim), generator=g, device="cuda") < 1e-3, 50.0, 1.0)
    return x.to(SRC[src])


def _empty_cache(case, pages):
    """Zeroed K or V cache and scale cache (None where the format has none)."""
    shape = (pages, case["page"], case["kv_heads"], case["dim"])
    if case["cache"] == "16":
        return torch.zeros(shape, dtype=SRC[case["src"]], device="cuda"), None
    if case["cache"] == "fp4":
        codes = torch.zeros(shape[:3] + (case["dim"] // 2,), dtype=torch.uint8, device="cuda")
        scales = torch.full(shape[:3] + (case["dim"] // 32,), 127, dtype=torch.uint8, device="cuda")
        return codes.view(torch.float4_e2m1fn_x2), scales.view(torch.float8_e8m0fnu)
    codes = torch.zeros(shape, dtype=torch.uint8, device="cuda").view(FP8[case["cache"]])
    if case.get("scales") in ("token", "head"):
        return codes, torch.ones(shape[:2 if case["scales"] == "token" else 3], device="cuda")
    return codes, None


def _fill(case, g, cache, scales):
    """Fills a cache with what a serving engine stored there: normal rows in the cache's format."""
    flat = cache.view(-1, *cache.shape[2:])
    slots, step = flat.shape[0], max(1, (1 << 28) // (case["kv_heads"] * case["dim"]))
    fs = None if scales is None else scales.view(slots, *scales.shape[2:])
    for a in range(0, slots, step):
        b = min(slots, a + step)
        x = _rows(g, b - a, case["kv_heads"], case["dim"], case["src"], False)
        if case["cache"] == "16":
            flat[a:b] = x
        elif case["cache"] == "fp4":
            codes, e = _to_fp4(x.float())
            flat.view(torch.uint8)[a:b] = codes
            fs.view(torch.uint8)[a:b] = e
        else:
            x = x.float()
            if scales is not None:
                amax = x.abs().amax(dim=(1, 2) if case["scales"] == "token" else 2)
                fs[a:b] = amax / 448.0
                x = x / fs[a:b].view(b - a, -1, 1)
            flat.view(torch.uint8)[a:b] = x.clamp(-448.0, 448.0).to(FP8[case["cache"]]).view(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = State()
    s.case, s.page = case, case["page"]
    src = SRC[case["src"]]
    H, D = case["kv_heads"], case["dim"]
    s.inv_k = s.inv_v = s.k_scale = s.v_scale = None
    if case["cache"] in FP8 and case.get("scales", "tensor") == "tensor":
        s.k_scale = torch.tensor([2.5], device="cuda")
        s.v_scale = torch.tensor([1.7], device="cuda")
        s.inv_k, s.inv_v = 1.0 / s.k_scale, 1.0 / s.v_scale
    if case["kind"] in ("append", "load"):
        T = case["tokens"]
        pages = max(2, 2 * -(-T // s.page))              # half of the cache belongs to others
        s.k_cache, s.ks_cache = _empty_cache(case, pages)
        s.v_cache, s.vs_cache = _empty_cache(case, pages)
        order = torch.randperm(pages, generator=g, device="cuda")[:-(-T // s.page)]
        slots = order[:, None] * s.page + torch.arange(s.page, device="cuda")
        s.loc = slots.view(-1)[:T].to(torch.int32)
        s.k_out = torch.zeros((T, H, D), dtype=src, device="cuda")
        s.v_out = torch.zeros((T, H, D), dtype=src, device="cuda")
    if case["kind"] == "append":
        s.k = _rows(g, T, H, D, case["src"], True)
        s.v = _rows(g, T, H, D, case["src"], True)
        s.q = _rows(g, T, case["q_heads"], D, case["src"], False)
        s.q_out = torch.zeros_like(s.q)
        start = int(torch.randint(0, 32768 - T, (1,), generator=g, device="cuda"))
        s.positions = torch.arange(start, start + T, device="cuda")
        half = case["rot"] // 2
        freq = 1e4 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        angle = torch.arange(32768, dtype=torch.float64, device="cuda")[:, None] * freq
        s.cos_sin = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    elif case["kind"] == "load":
        _fill(case, g, s.k_cache, s.ks_cache)
        _fill(case, g, s.v_cache, s.vs_cache)
    else:
        lengths = _lengths(case)
        need = [-(-n // s.page) for n, _ in lengths]
        pages = sum(need) + 1
        s.k_cache, s.ks_cache = _empty_cache(case, pages)
        s.v_cache, s.vs_cache = _empty_cache(case, pages)
        _fill(case, g, s.k_cache, s.ks_cache)
        _fill(case, g, s.v_cache, s.vs_cache)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        s.table = torch.zeros((len(need), max(need)), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            s.table[b, :n] = order[at:at + n]
            at += n
        s.lens = torch.tensor([n for n, _ in lengths], dtype=torch.int32, device="cuda")
        starts = [0]
        for _, n in lengths:
            starts.append(starts[-1] + n)
        s.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s.q = (2.0 * torch.randn((starts[-1], case["q_heads"], D), generator=g, device="cuda")).to(src)
        s.out = torch.zeros_like(s.q)
        s.max_queries = max(n for _, n in lengths)
        s.max_length = max(n for n, _ in lengths)
        s.far = _far(case)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _to_fp4(x):
    """fp32 [..., D] -> (packed codes [..., D/2], scale bytes [..., D/32]).

    A block's scale is the smallest power of two, at least 2^-100, for which
    its largest magnitude is at most 7 scales; elements go to the nearest
    e2m1 value, ties to the even code, and values above 6 scales to 6."""
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    m, e = torch.frexp(blocks.abs().amax(dim=-1))        # amax = m * 2^e, m in [0.5, 1)
    e = e - 3 + (m > 0.875).int()
    byte = (e + 127).clamp(FP4_MIN_SCALE, 254)
    y = torch.ldexp(blocks, (127 - byte)[..., None])
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() +
            (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    code = (code + 8 * torch.signbit(y).int()).reshape(*x.shape[:-1], -1, 2)
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), byte.to(torch.uint8)


def _fp4_values(codes, scales):
    """Packed codes [..., D/2] and scale bytes [..., D/32] -> fp32 [..., D]."""
    pairs = torch.tensor([[(LUT + tuple(-v for v in LUT))[b & 15], (LUT + tuple(-v for v in LUT))[b >> 4]]
                          for b in range(256)], device=codes.device)
    x = pairs[codes.int()].reshape(*scales.shape, 32)
    x = torch.ldexp(x, scales.int()[..., None] - 127)
    return x.reshape(*codes.shape[:-1], -1)


def _cached(case, cache, scale_cache, scale, slots):
    """fp32 values of the cache rows at `slots`: [*slots.shape, H, D]."""
    flat = cache.view(-1, *cache.shape[2:])
    if case["cache"] == "16":
        return flat[slots].float()
    if case["cache"] == "fp4":
        fs = scale_cache.view(torch.uint8).view(flat.shape[0], *scale_cache.shape[2:])
        return _fp4_values(flat.view(torch.uint8)[slots], fs[slots])
    x = flat.view(torch.uint8)[slots].view(FP8[case["cache"]]).float()
    if scale_cache is not None:
        fs = scale_cache.view(flat.shape[0], -1)
        return x * fs[slots][..., None]
    return x * scale


def _rotated(x, positions, table, interleaved):
    """fp32 rotation of the first table.shape[1] dims of x [T, H, D], in pairs
    (i, i + half), or (2i, 2i + 1) where interleaved."""
    x = x.float()
    rot = table.shape[1]
    half = rot // 2
    row = table[positions][:, None]
    c, n = row[..., :half], row[..., half:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * c - b * n, b * c + a * n], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_append(s):
    case = s.case
    k = _rotated(s.k, s.positions, s.cos_sin, case["interleaved"])
    v = s.v.float()
    s.q_out.copy_(_rotated(s.q, s.positions, s.cos_sin, case["interleaved"]))
    loc = s.loc.long()
    for x, cache, scales, inv in ((k, s.k_cache, s.ks_cache, s.inv_k),
                                  (v, s.v_cache, s.vs_cache, s.inv_v)):
        flat = cache.view(-1, *cache.shape[2:])
        if case["cache"] == "16":
            flat[loc] = x.to(flat.dtype)
        elif case["cache"] == "fp4":
            codes, e = _to_fp4(x)
            flat.view(torch.uint8)[loc] = codes
            scales.view(torch.uint8).view(flat.shape[0], *scales.shape[2:])[loc] = e
        else:
            most = FP8_MAX[case["cache"]]
            y = (x * inv).clamp(-most, most).to(FP8[case["cache"]])
            flat.view(torch.uint8)[loc] = y.view(torch.uint8)


def _plain_load(s):
    loc = s.loc.long()
    s.k_out.copy_(_cached(s.case, s.k_cache, s.ks_cache, s.k_scale, loc))
    s.v_out.copy_(_cached(s.case, s.v_cache, s.vs_cache, s.v_scale, loc))


def _plain_attend(s):
    case = s.case
    dev, sinks, window = s.q.device, case["sinks"], case["window"]
    B, H, D, n = case["seqs"], case["kv_heads"], case["dim"], s.max_queries
    group = case["q_heads"] // H
    lens, starts = s.lens.long(), s.starts.long()
    new = starts[1:] - starts[:-1]
    # queries padded to [B, n], their positions and rows of q
    at = torch.arange(n, device=dev)
    q_pos = (lens - new)[:, None] + at
    real = at < new[:, None]
    q_row = torch.where(real, starts[:-1, None] + at, 0)
    # keys: the first tokens, then everything from the first new token's window on
    low = (lens - new - window + 1 if window else torch.zeros_like(lens)).clamp(min=sinks)
    i = torch.arange(sinks + s.far, device=dev)
    k_pos = torch.where(i < sinks, i, low[:, None] + i - sinks)
    there = k_pos < lens[:, None]
    k_pos = torch.where(there, k_pos, 0)
    slots = s.table.long().gather(1, k_pos // s.page) * s.page + k_pos % s.page
    k = _cached(case, s.k_cache, s.ks_cache, s.k_scale, slots).permute(0, 2, 3, 1).contiguous()
    v = _cached(case, s.v_cache, s.vs_cache, s.v_scale, slots).permute(0, 2, 1, 3).contiguous()
    q = s.q[q_row].float().view(B, n, H, group, D).permute(0, 2, 3, 1, 4).reshape(B, H, group * n, D)
    score = torch.matmul(q, k).view(B, H, group, n, -1) / math.sqrt(D)
    seen = there[:, None] & (k_pos[:, None] <= q_pos[..., None]) & real[..., None]
    if window:
        seen &= (q_pos[..., None] - k_pos[:, None] < window) | (k_pos[:, None] < sinks)
    seen = seen[:, None, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(dim=-1, keepdim=True)
    p = p.view(B, H, group * n, -1)
    o = torch.matmul(p, v).view(B, H, group, n, D) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, H * group, D)
    s.out[q_row[real]] = o[real].to(s.out.dtype)


def run(s):
    case = s.case
    if case["kind"] == "append":
        if own:
            import fp8_kv_quantization_amd as kv
            kv.store_kv_rope_paged(s.k, s.v, s.k_cache, s.v_cache, s.loc, s.positions, s.cos_sin,
                                   q=s.q, q_out=s.q_out, interleaved=case["interleaved"],
                                   page_size=s.page, inv_k_scale=s.inv_k, inv_v_scale=s.inv_v,
                                   k_scale_cache=s.ks_cache, v_scale_cache=s.vs_cache)
        else:
            _plain_append(s)
        if case["cache"] != "fp4":
            return {"q": s.q_out, "k_cache": s.k_cache, "v_cache": s.v_cache}
    if case["kind"] in ("append", "load"):
        if own:
            import fp8_kv_quantization_amd as kv
            kv.load_kv_paged(s.k_cache, s.v_cache, s.loc, s.k_out, s.v_out, page_size=s.page,
                             k_scale=s.k_scale, v_scale=s.v_scale, k_scale_cache=s.ks_cache,
                             v_scale_cache=s.vs_cache)
        else:
            _plain_load(s)
        rows = {"k": s.k_out, "v": s.v_out}
        return rows if case["kind"] == "load" else {"q": s.q_out, **rows}
    if own:
        import fp8_kv_quantization_amd as kv
        kv.attention_paged(s.q, s.k_cache, s.v_cache, s.table, s.lens, cu_q=s.starts,
                           max_q=s.max_queries, max_len=s.max_length, window=case["window"],
                           sinks=case["sinks"], page_size=s.page, k_scale=s.k_scale,
                           v_scale=s.v_scale, k_scale_cache=s.ks_cache,
                           v_scale_cache=s.vs_cache, out=s.out)
    else:
        _plain_attend(s)
    return s.out


# ---------------------------------------------------------------------------
# The same in 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _exact_turn(x, positions, table, interleaved):
    x, row = x.double().clone(), table.double()[positions]
    half = row.shape[1] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        z = torch.complex(x[..., a], x[..., b]) * torch.complex(row[:, i], row[:, i + half])[:, None]
        x[..., a], x[..., b] = z.real, z.imag
    return x


def _exact_fp4(x):
    """Every value replaced by the one that a 4-bit cache holds for it."""
    flat = x.reshape(-1, 32)
    amax = flat.abs().amax(dim=1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, 1.0) / 7.0)).clamp(min=-100.0)
    scale = torch.exp2(e)
    values = torch.tensor(LUT, dtype=torch.float64, device=x.device)
    y = flat / scale
    best = torch.zeros_like(y)
    for code in (0, 2, 4, 6, 1, 3, 5, 7):                # the even codes first: they win ties
        better = (y.abs() - values[code]).abs() < (y.abs() - best).abs()
        best = torch.where(better, values[code], best)
    return (torch.copysign(best, y) * scale).reshape(x.shape)


def _exact_cached(s, cache, scale_cache, scale):
    """The whole cache in 64 bits, [slots, H, D]."""
    case = s.case
    if case["cache"] == "16":
        return cache.double().flatten(0, 1)
    if case["cache"] == "fp4":
        raw = cache.view(torch.uint8).flatten(0, 1)
        nibbles = torch.stack([raw & 15, raw >> 4], dim=-1).flatten(-2).long()
        values = torch.tensor(LUT + tuple(-v for v in LUT), dtype=torch.float64, device=raw.device)
        e = scale_cache.view(torch.uint8).flatten(0, 1).double() - 127.0
        return values[nibbles] * torch.exp2(e).repeat_interleave(32, dim=-1)
    x = cache.float().double().flatten(0, 1)
    if scale_cache is not None:
        return x * scale_cache.double().flatten(0, 1).view(x.shape[0], -1, 1)
    return x * scale.double()


def _picked(cache, pages):
    """The pages of a cache, whatever its type (indexing wants one that torch computes with)."""
    if cache is None or cache.element_size() > 1:
        return None if cache is None else cache[pages]
    return cache.view(torch.uint8)[pages].view(cache.dtype)


def exact(case, seed):
    s = prepare(case, seed)
    H, D = case["kv_heads"], case["dim"]
    if case["kind"] == "append":
        q = _exact_turn(s.q, s.positions, s.cos_sin, case["interleaved"])
        k = _exact_turn(s.k, s.positions, s.cos_sin, case["interleaved"])
        v = s.v.double()
        if case["cache"] == "fp4":
            return {"q": q, "k": _exact_fp4(k), "v": _exact_fp4(v)}
        out = {"q": q}
        for name, x, cache, inv in (("k_cache", k, s.k_cache, s.inv_k), ("v_cache", v, s.v_cache, s.inv_v)):
            whole = cache.double().flatten(0, 1)
            if case["cache"] in FP8:
                most = FP8_MAX[case["cache"]]
                x = (x * inv.double()).clamp(-most, most).float().to(FP8[case["cache"]]).double()
            whole[s.loc.long()] = x
            out[name] = whole.view(cache.shape)
        return out
    if case["kind"] == "load":
        loc = s.loc.long()
        return {"k": _exact_cached(s, s.k_cache, s.ks_cache, s.k_scale)[loc],
                "v": _exact_cached(s, s.v_cache, s.vs_cache, s.v_scale)[loc]}
    out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    starts, lens = s.starts.tolist(), s.lens.tolist()
    group = case["q_heads"] // H
    for b in range(case["seqs"]):
        pages = s.table[b, :-(-lens[b] // s.page)].long()
        k = _exact_cached(s, _picked(s.k_cache, pages), _picked(s.ks_cache, pages), s.k_scale)[:lens[b]]
        v = _exact_cached(s, _picked(s.v_cache, pages), _picked(s.vs_cache, pages), s.v_scale)[:lens[b]]
        n = starts[b + 1] - starts[b]
        where = torch.arange(lens[b], device="cuda")
        mine = torch.arange(lens[b] - n, lens[b], device="cuda")[:, None]
        hidden = where > mine
        if case["window"]:
            hidden |= (where <= mine - case["window"]) & (where >= case["sinks"])
        for h in range(case["q_heads"]):
            q = s.q[starts[b]:starts[b + 1], h].double()
            score = q @ k[:, h // group].T / math.sqrt(D)
            out[starts[b]:starts[b + 1], h] = score.masked_fill_(hidden, -math.inf).softmax(dim=1) @ v[:, h // group]
    return out
