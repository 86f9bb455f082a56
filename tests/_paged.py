"""Test-side references of the paged-cache operators, in numpy and in 64 bits,
written from the formats' and the operators' definitions."""
from __future__ import annotations

import numpy as np
import torch

from tests import _ref

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}
FP4_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([_ref.e4m3fn_decode(c) for c in range(256)])
E5M2 = np.array([_ref.e5m2_decode(c) for c in range(256)])


def bits_of(x: torch.Tensor) -> np.ndarray:
    """The 16-bit patterns of a bf16 / fp16 tensor."""
    return x.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def round16(x: np.ndarray, src: str) -> np.ndarray:
    """float32 -> the nearest bf16 / fp16 value's pattern (ties to even)."""
    return bits_of(torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TORCH[src]))


def rotate32(x: np.ndarray, positions, table: np.ndarray, interleaved: bool) -> np.ndarray:
    """float32 x [T, H, D] with its first table.shape[1] dims turned, every
    product and sum rounded to float32 on its own."""
    x = x.astype(np.float32).copy()
    rot = table.shape[1]
    half = rot // 2
    c, s = table[positions][:, None, :half], table[positions][:, None, half:]
    a = x[..., 0:rot:2].copy() if interleaved else x[..., :half].copy()
    b = x[..., 1:rot:2].copy() if interleaved else x[..., half:rot].copy()
    with np.errstate(all="ignore"):
        p = (a * c).astype(np.float32) - (b * s).astype(np.float32)
        q = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    if interleaved:
        x[..., 0:rot:2], x[..., 1:rot:2] = p, q
    else:
        x[..., :half], x[..., half:rot] = p, q
    return x


def fp4_encode(x: np.ndarray):
    """float32 [..., D] -> (packed codes [..., D/2], scale bytes [..., D/32]),
    from the definition: smallest power of two s >= 2^-100 with amax <= 7 s,
    nearest e2m1 value of x / s, ties to the even code."""
    blocks = x.astype(np.float64).reshape(-1, 32)
    codes = np.zeros(blocks.shape, np.uint8)
    scales = np.zeros(blocks.shape[0], np.uint8)
    for i, b in enumerate(blocks):
        if not np.isfinite(b).all():
            scales[i] = 255
            continue
        e = -100
        while np.abs(b).max() > 7.0 * 2.0 ** e:
            e += 1
        scales[i] = e + 127
        y = np.abs(b) / 2.0 ** e
        d = np.abs(np.minimum(y, 6.0)[:, None] - FP4_VALUES[None])
        near = d == d.min(axis=1, keepdims=True)
        code = np.array([min(np.flatnonzero(n), key=lambda c: (c % 2, c)) for n in near])
        codes[i] = code + 8 * np.signbit(b)
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    return (packed.reshape(*x.shape[:-1], -1),
            scales.reshape(*x.shape[:-1], -1))


def fp4_decode(packed: np.ndarray, scales: np.ndarray) -> np.ndarray:
    both = np.concatenate([FP4_VALUES, -FP4_VALUES])
    n = np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], -1)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return both[n] * np.repeat(s, 32, axis=-1)


class Cache:
    """K and V caches of one format on the GPU, [pages, P, H, D] inside larger
    allocations (padded strides), and their values in 64 bits.  fmt: "bf16",
    "fp16", "e4m3fn", "e5m2", "fp4"; kind: "tensor", "token", "head" or
    "block"."""

    def __init__(self, rng, fmt, pages, P, H, D, kind="tensor", pad=0, device="cuda", spread=1.0):
        self.fmt, self.kind, self.P, self.H, self.D, self.pages = fmt, kind, P, H, D, pages
        self.k_scale = self.v_scale = self.ks = self.vs = None
        self.tensors, self.values, self.scales = [], [], []
        for side in range(2):
            x = rng.standard_normal((pages, P, H, D)).astype(np.float32) * spread
            if fmt in ("bf16", "fp16"):
                t = torch.from_numpy(x).to(TORCH[fmt])
                value = t.double().numpy()
                scale = None
            elif fmt == "fp4":
                packed, byte = fp4_encode(x)
                value = fp4_decode(packed, byte)
                t, scale = torch.from_numpy(packed), torch.from_numpy(byte)
            else:
                codes = rng.integers(0, 256, (pages, P, H, D), dtype=np.uint8)
                table = E4M3 if fmt == "e4m3fn" else E5M2
                big = 16.0       # keep the codes' values moderate, and finite
                codes[~(np.abs(table[codes]) <= big)] = 0x31
                t = torch.from_numpy(codes)
                if kind == "tensor":
                    s = np.float32(rng.uniform(0.05, 0.2))
                    value = table[codes] * float(s)
                    scale = torch.tensor([s])
                else:
                    s = rng.uniform(0.02, 0.3, (pages, P) if kind == "token" else (pages, P, H))
                    s = s.astype(np.float32)
                    value = table[codes] * s.astype(np.float64).reshape(pages, P, -1, 1)
                    scale = torch.from_numpy(s)
            if pad:
                room = torch.zeros((pages, P + 1, H + 1, t.shape[-1] + pad), dtype=t.dtype, device=device)
                room[:, :P, :H, :t.shape[-1]] = t.to(device)
                t = room[:, :P, :H, :t.shape[-1]]
            else:
                t = t.to(device)
            self.tensors.append(t)
            self.values.append(value)
            self.scales.append(None if scale is None else scale.to(device))
        if fmt == "fp4" or kind in ("token", "head"):
            self.ks, self.vs = self.scales
        elif fmt in ("e4m3fn", "e5m2"):
            self.k_scale, self.v_scale = self.scales

    def typed(self, t):
        if self.fmt in ("bf16", "fp16"):
            return t
        return t.view({"e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2,
                       "fp4": torch.float4_e2m1fn_x2}[self.fmt])

    @property
    def k(self):
        return self.typed(self.tensors[0])

    @property
    def v(self):
        return self.typed(self.tensors[1])

    def kwargs(self):
        return dict(page_size=self.P, k_scale=self.k_scale, v_scale=self.v_scale,
                    k_scale_cache=self.ks, v_scale_cache=self.vs)


def attention(q, cache, table, lens, starts, window=0, sinks=0, scale=None):
    """(out, bound) in 64 bits: q [T, Hq, D] float64.  Only the keys that a row
    sees are ever read.  bound: how far a result may be off, elementwise, for a
    16-bit source type of unit roundoff u: (u + slack) * sum_j p_j |v_j| for
    the rounded weights, and what the scores' fp32 sums add, returned as the
    factor's parts (weights, scores)."""
    T, Hq, D = q.shape
    G = Hq // cache.H
    scale = D ** -0.5 if scale is None else scale
    out = np.zeros((T, Hq, D))
    weights, scores = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    counts = np.zeros((T, Hq, D))
    seen_rows = np.zeros(T, bool)
    kv, vv = cache.values
    for b in range(len(lens)):
        n = starts[b + 1] - starts[b]
        for r in range(n):
            p = lens[b] - n + r
            row = starts[b] + r
            seen_rows[row] = True
            keys = np.arange(0, max(p + 1, 0))
            if window:
                keys = keys[(p - keys < window) | (keys < sinks)]
            pages = table[b][keys // cache.P]
            good = (pages >= 0) & (pages < cache.pages)
            keys, pages = keys[good], pages[good]
            if len(keys) == 0:
                continue
            K, V = kv[pages, keys % cache.P], vv[pages, keys % cache.P]   # [n, H, D]
            for h in range(Hq):
                with np.errstate(all="ignore"):
                    s = K[:, h // G] @ q[row, h] * scale
                    e = np.exp(s - s.max())
                    w = e / e.sum()
                    out[row, h] = w @ V[:, h // G]
                    weights[row, h] = w @ np.abs(V[:, h // G])
                    d = np.abs(K[:, h // G]) @ np.abs(q[row, h]) * scale
                    scores[row, h] = d.max() * weights[row, h]
                    counts[row, h] = len(keys) * np.abs(V[:, h // G]).max()
    return out, dict(weights=weights, scores=scores, counts=counts, rows=seen_rows)


def attention_bound(ref, parts, src, D):
    """Elementwise bound on |kernel - reference|:

    * each weight is rounded once to the source type: u * sum p |v|;
    * a score is an fp32 sum of D exact products plus a few more roundings, off
      by at most (D + 8) 2^-24 sum |q k| scale, which moves its weight and the
      weights' sum by that factor each; exponentials and the running sums add
      some 2^-18 for the few thousand keys of these tests;
    * fp16 weights below 2^-14 have an absolute step: 2^-25 each;
    * the result is rounded once: u |out|."""
    u = torch.finfo(TORCH[src]).eps / 2
    bound = u * parts["weights"] + 2 * (D + 8) * 2.0 ** -24 * parts["scores"] * 1.5
    bound += 2.0 ** -18 * parts["weights"] + u * np.abs(ref) * (1 + 2.0 ** -6)
    if src == "fp16":
        bound += 2.0 ** -25 * parts["counts"] + 2.0 ** -25
    return bound + 1e-30


def assert_attention(got: torch.Tensor, ref, parts, src, what=""):
    g = got.detach().double().cpu().numpy()
    rows = parts["rows"]
    g, ref = g[rows], ref[rows]
    cut = {k: (v[rows] if k != "rows" else v) for k, v in parts.items()}
    nan = np.isnan(ref)
    assert np.array_equal(nan, np.isnan(g)), f"{what}: NaN in other places than the reference"
    with np.errstate(all="ignore"):
        off = np.abs(g - ref) - attention_bound(ref, cut, src, ref.shape[-1])
    off[nan] = -1
    if (off > 0).any():
        i = np.unravel_index(np.argmax(off), off.shape)
        raise AssertionError(f"{what}: {int((off > 0).sum())} values outside the bound; worst at {i}: "
                             f"got {g[i]} want {ref[i]} (over by {off[i]:.3g})")
