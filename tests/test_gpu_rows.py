"""GPU: rotated append into paged caches and load out of them, against numpy
references, bit for bit (every step is one fp32 rounding)."""
import numpy as np
import pytest
import torch

import fp8_kv_quantization_amd as kv
from tests import _paged, _ref
from tests._gpu import check_flag
from tests._paged import TORCH, Cache, attention, assert_attention, bits_of, fp4_decode, fp4_encode, rotate32, round16

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_flag(request):
    print(f"[gpu-case] {request.node.name}", flush=True)
    check_flag()
    yield
    torch.cuda.synchronize()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def table_of(n, rot, base=1e4):
    half = rot // 2
    a = np.arange(n, dtype=np.float64)[:, None] * base ** (-np.arange(half) / half)
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


def rows(rng, T, H, D, src):
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    x[rng.random(x.shape) < 0.01] *= 50.0
    return torch.from_numpy(x).to(TORCH[src])


class Target:
    """Sentinel-filled caches of one format, and the bytes that they should hold."""

    def __init__(self, fmt, src, pages, P, H, D, pad=0):
        self.fmt, self.src, self.P, self.H, self.D, self.slots = fmt, src, P, H, D, pages * P
        width = {"16": 2 * D, "fp4": D // 2}.get(fmt, D)
        self.room = torch.full((2, pages, P + (1 if pad else 0), H + (1 if pad else 0), width + pad), 0xEE,
                               dtype=torch.uint8, device="cuda")
        self.raw = self.room[:, :, :P, :H, :width]
        self.want = self.room.cpu().numpy().copy()
        self.view = self.want[:, :, :P, :H, :width]
        self.scales = torch.full((2, pages, P, H, max(D // 32, 1)), 0xEE, dtype=torch.uint8, device="cuda")
        self.want_scales = self.scales.cpu().numpy().copy()

    def cache(self, side):
        t = self.raw[side]
        if self.fmt == "16":
            return t.view(TORCH[self.src])
        return t.view({"e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2,
                       "fp4": torch.float4_e2m1fn_x2}[self.fmt])

    def kwargs(self):
        return dict(k_scale_cache=self.scales[0], v_scale_cache=self.scales[1]) if self.fmt == "fp4" else {}

    def put(self, side, slot, row32, inv=None):
        """row32: [H, D] float32, the value that is quantised."""
        at = self.view[side, slot // self.P, slot % self.P]
        if self.fmt == "16":
            at[:] = round16(row32, self.src).view(np.uint8).reshape(self.H, -1)
        elif self.fmt == "fp4":
            at[:], self.want_scales[side, slot // self.P, slot % self.P] = fp4_encode(row32)
        else:
            y = row32 if inv is None else (row32 * np.float32(inv)).astype(np.float32)
            f = _ref.nearest_e5m2 if self.fmt == "e5m2" else _ref.nearest_e4m3fn
            at[:] = f(y, nan_sign_from=y).reshape(self.H, -1)

    def check(self):
        np.testing.assert_array_equal(self.room.cpu().numpy(), self.want)
        if self.fmt == "fp4":
            np.testing.assert_array_equal(self.scales.cpu().numpy(), self.want_scales)


def append_case(rng, fmt, src, T, Hq, H, D, rot, interleaved, P, pad=0, in_place=False, idx=np.int32,
                pos_t=np.int64, scales=True, wide=0):
    pages = max(2, -(-T // P) + 3)
    t = Target(fmt, src, pages, P, H, D, pad)
    k, v = rows(rng, T, H, D, src), rows(rng, T, H, D, src)
    q = rows(rng, T, Hq, D, src) if Hq else None
    slots = rng.permutation(t.slots)[:T].astype(idx)
    positions = rng.integers(0, 500, T).astype(pos_t)
    table = table_of(500, rot) if rot else None
    fp8 = fmt in ("e4m3fn", "e5m2")
    inv = (0.4, 1.7) if fp8 and scales else (None, None)

    def on_gpu(x):       # inside wider rows where asked
        if not wide:
            return x.cuda()
        room = torch.zeros((x.shape[0], x.shape[1] + 1, x.shape[2] + wide), dtype=x.dtype, device="cuda")
        room[:, 1:, :x.shape[2]] = x.cuda()
        return room[:, 1:, :x.shape[2]]

    gq = None if q is None else on_gpu(q)
    out = None if q is None or in_place else torch.full((T, Hq, D), 9.0, dtype=TORCH[src], device="cuda")
    kv.store_kv_rope_paged(on_gpu(k), on_gpu(v), t.cache(0), t.cache(1), dev(slots),
                           dev(positions) if rot else None, dev(table) if rot else None, q=gq, q_out=out,
                           interleaved=interleaved, page_size=P,
                           inv_k_scale=dev(np.float32([inv[0]])) if inv[0] else None,
                           inv_v_scale=dev(np.float32([inv[1]])) if inv[1] else None, **t.kwargs())
    turn = (lambda x: rotate32(x.float().numpy(), positions, table, interleaved)) if rot else (
        lambda x: x.float().numpy())
    kr = turn(k)
    for i in range(T):
        t.put(0, int(slots[i]), kr[i], inv[0])
        t.put(1, int(slots[i]), v[i].float().numpy(), inv[1])
    t.check()
    if q is not None:
        got = gq if in_place else out
        np.testing.assert_array_equal(bits_of(got), round16(turn(q), src))
    assert check_flag() == (kv.OK, -1, 0)


@pytest.mark.parametrize("src", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["16", "e4m3fn", "e5m2", "fp4"])
@pytest.mark.parametrize("D,rot", [(32, 32), (64, 32), (96, 96), (96, 48), (128, 128), (128, 80), (256, 64), (512, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(src, fmt, D, rot, interleaved):
    rng = np.random.default_rng(D + rot)
    append_case(rng, fmt, src, 13, 5, 2, D, rot, interleaved, 16)


@pytest.mark.parametrize("fmt", ["16", "e4m3fn"])
@pytest.mark.parametrize("D", [16, 48, 80, 208])
def test_append_odd_dims(fmt, D):
    append_case(np.random.default_rng(D), fmt, "bf16", 9, 3, 3, D, 16, False, 24)


@pytest.mark.parametrize("fmt", ["16", "e5m2", "fp4"])
def test_append_without_rotation_or_q(fmt):
    append_case(np.random.default_rng(1), fmt, "bf16", 21, 0, 3, 64, 0, False, 7)
    append_case(np.random.default_rng(2), fmt, "fp16", 21, 0, 3, 64, 64, False, 7, scales=False)


@pytest.mark.parametrize("T,H,Hq", [(1, 1, 1), (1, 8, 32), (700, 2, 14), (2100, 8, 32)])
@pytest.mark.parametrize("D", [64, 96])
def test_append_sizes(T, H, Hq, D):
    """One head a lane and four, heads that do not fill the last group."""
    append_case(np.random.default_rng(T), "e4m3fn", "bf16", T, Hq, H, D, D, False, 64)


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("T", [5, 3000])
def test_append_in_place(D, T):
    append_case(np.random.default_rng(D), "16", "bf16", T, 6, 2, D, D, False, 16, in_place=True)


def test_append_strides_and_index_types():
    for idx, pos in ((np.int64, np.int32), (np.int32, np.int64)):
        append_case(np.random.default_rng(5), "16", "fp16", 40, 4, 2, 64, 32, False, 16, pad=16, idx=idx, pos_t=pos,
                    wide=8)
        append_case(np.random.default_rng(6), "fp4", "bf16", 40, 4, 2, 64, 64, True, 10, pad=16, idx=idx, pos_t=pos,
                    wide=8)


@pytest.mark.parametrize("fmt", ["16", "e4m3fn", "fp4"])
def test_append_bad_slots_and_positions(fmt):
    rng = np.random.default_rng(7)
    T, H, Hq, D, P = 20, 2, 4, 64, 16
    t = Target(fmt, "bf16", 4, P, H, D)
    k, v, q = (rows(rng, T, n, D, "bf16") for n in (H, H, Hq))
    slots = rng.permutation(t.slots)[:T].astype(np.int64)
    positions = rng.integers(0, 100, T)
    table = table_of(100, D)
    slots[3], slots[11], slots[12] = -1, t.slots, 2 ** 40
    positions[5], positions[12], positions[19] = -1, 3, 100
    out = torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    kv.store_kv_rope_paged(k.cuda(), v.cuda(), t.cache(0), t.cache(1), dev(slots), dev(positions), dev(table),
                           q=q.cuda(), q_out=out, page_size=P, **t.kwargs())
    kr = rotate32(k.float().numpy(), np.clip(positions, 0, 99), table, False)
    qr = round16(rotate32(q.float().numpy(), np.clip(positions, 0, 99), table, False), "bf16")
    nine = bits_of(torch.full((1,), 9.0, dtype=torch.bfloat16))[0]
    for i in range(T):
        if i in (5, 19):
            qr[i] = nine
        elif i not in (3, 11, 12):
            t.put(0, int(slots[i]), kr[i])
            t.put(1, int(slots[i]), v[i].float().numpy())
    t.check()
    np.testing.assert_array_equal(bits_of(out), qr)
    assert check_flag() == (kv.ERR_OOB, 3, 5)
    # the cache's own limit
    kv.store_kv_rope_paged(k.cuda(), v.cuda(), t.cache(0), t.cache(1), dev(np.arange(T)), None, None, page_size=P,
                           size_limit=18, **t.kwargs())
    assert check_flag() == (kv.ERR_OOB, 18, 2)


def test_fp4_codes_of_every_pattern():
    """Every finite bf16 pattern next to a block maximum that sets the scale,
    NaN and infinity blocks, zeros and the smallest magnitudes."""
    D, H = 32, 1
    pats = np.arange(65536, dtype=np.uint32)
    x = (pats << 16).astype(np.uint32).view(np.float32)
    blocks = []
    for top in (1.0, 1.75, 1.7578125, 448.0, 1e-30, 3e38, 0.0):
        keep = x[np.abs(np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0)) <= top]
        keep = keep[np.isfinite(keep)]
        keep = np.concatenate([keep, np.zeros(-len(keep) % 31, np.float32)]).reshape(-1, 31)
        blocks.append(np.concatenate([np.full((len(keep), 1), top, np.float32), keep], axis=1))
    special = np.zeros((4, 32), np.float32)
    special[0, 3], special[1, 31], special[2, 0], special[3, :] = np.nan, np.inf, -np.inf, -0.0
    b = np.concatenate(blocks + [special])
    b = b[np.linspace(0, len(b) - 1, 6000).astype(int).tolist() + list(range(len(b) - 4, len(b)))]
    T = len(b)
    k = torch.from_numpy(b.reshape(T, H, D)).to(torch.bfloat16)
    t = Target("fp4", "bf16", -(-T // 16), 16, H, D)
    kv.store_kv_fp4_paged(k.cuda(), k.flip(0).contiguous().cuda(), t.cache(0), t.cache(1), dev(np.arange(T)),
                          t.scales[0], t.scales[1], page_size=16)
    codes, scales = fp4_encode(k.float().numpy())
    got = t.raw.cpu().numpy().reshape(2, -1, H, D // 2)[:, :T]
    got_s = t.scales.cpu().numpy().reshape(2, -1, H, 1)[:, :T]
    np.testing.assert_array_equal(got_s[0], scales)
    np.testing.assert_array_equal(got[0], codes)
    np.testing.assert_array_equal(got_s[1], scales[::-1])
    np.testing.assert_array_equal(got[1], codes[::-1])


def load_case(rng, fmt, src, T, H, D, P, kind, pad=0, flat=False):
    cache = Cache(rng, fmt if fmt != "16" else src, max(2, -(-T // P) + 2), P, H, D, kind, pad)
    if fmt in ("e4m3fn", "e5m2"):       # every code, NaN and infinity among them
        codes = np.resize(np.arange(256, dtype=np.uint8), (cache.pages, P, H, D))
        tab = _paged.E4M3 if fmt == "e4m3fn" else _paged.E5M2
        for side in range(2):
            cache.tensors[side].copy_(dev(codes))
            s = cache.scales[side].cpu().numpy()
            with np.errstate(all="ignore"):
                s = s.reshape(cache.pages, P, -1, 1) if kind != "tensor" else s
                cache.values[side] = (tab[codes].astype(np.float32) * s).astype(np.float32)
    slots = rng.integers(0, cache.pages * P, T)
    slots[T // 2] = -1
    ko = torch.full((T, H + 1, D + 8), 9.0, dtype=TORCH[src], device="cuda")
    vo = torch.full((T, H, D), 9.0, dtype=TORCH[src], device="cuda")
    args = (cache.k, cache.v)
    kw = cache.kwargs()
    if flat:
        args = tuple(a.flatten(0, 1) for a in args)
        kw = {n: (x.flatten(0, 1) if n.endswith("cache") and x is not None else x) for n, x in kw.items()}
    kv.load_kv_paged(*args, dev(slots), ko[:, :H, :D], vo, **kw)
    for side, got in ((0, ko[:, :H, :D]), (1, vo)):
        want = cache.values[side].reshape(-1, H, D)[slots].astype(np.float32)
        want = torch.from_numpy(want).to(TORCH[src])
        want[T // 2] = 9.0
        np.testing.assert_array_equal(np.nan_to_num(got.cpu().float().numpy(), nan=12345.0),
                                      np.nan_to_num(want.float().numpy(), nan=12345.0))
    assert (ko[:, H:] == 9.0).all() and (ko[:, :, D:] == 9.0).all()
    assert check_flag() == (kv.ERR_OOB, T // 2, 1)


@pytest.mark.parametrize("src", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,kind", [("16", "tensor"), ("e4m3fn", "tensor"), ("e4m3fn", "token"), ("e4m3fn", "head"),
                                      ("e5m2", "tensor"), ("e5m2", "head"), ("fp4", "block")])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 512])
def test_load(src, fmt, kind, D):
    load_case(np.random.default_rng(D), fmt, src, 40, 3, D, 16, kind)


@pytest.mark.parametrize("T", [1, 600, 5000])
def test_load_sizes(T):
    load_case(np.random.default_rng(T), "e4m3fn", "bf16", T, 2, 128, 24, "head")
    load_case(np.random.default_rng(T), "fp4", "bf16", T, 8, 64, 64, "block", flat=True)
    load_case(np.random.default_rng(T), "16", "fp16", T, 8, 48, 64, "tensor", pad=16)


def test_a_serving_loop():
    """Prompt, then single tokens: append and attend, in every format, against
    attention over the values that the cache then holds."""
    rng = np.random.default_rng(61)
    H, Hq, D, P, src = 2, 8, 64, 16, "bf16"
    prompts, steps = [70, 5, 110], 4
    table_rows = table_of(300, D)
    for fmt in ("16", "e4m3fn", "e5m2", "fp4"):
        t = Target(fmt, src, 24, P, H, D)
        order = rng.permutation(24).reshape(3, 8).astype(np.int32)
        inv, scale = np.float32(2.0), np.float32(0.5)
        fp8 = fmt in ("e4m3fn", "e5m2")
        lens = [0, 0, 0]
        for step in range(steps + 1):
            new = prompts if step == 0 else [1, 1, 1]
            T = sum(new)
            starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
            positions = np.concatenate([np.arange(n, n + m) for n, m in zip(lens, new)])
            slots = np.concatenate([order[b][p // P] * P + p % P for b, p in
                                    ((b, np.arange(lens[b], lens[b] + new[b])) for b in range(3))])
            lens = [n + m for n, m in zip(lens, new)]
            k, v, q = (rows(rng, T, n, D, src).cuda() for n in (H, H, Hq))
            one = dev(np.float32([inv])) if fp8 else None
            kv.store_kv_rope_paged(k, v, t.cache(0), t.cache(1), dev(slots.astype(np.int64)), dev(positions),
                                   dev(table_rows), q=q, page_size=P, inv_k_scale=one, inv_v_scale=one, **t.kwargs())
            back = dev(np.float32([scale])) if fp8 else None
            out = kv.attention_paged(q, t.cache(0), t.cache(1), dev(order), dev(np.array(lens, np.int32)),
                                     cu_q=dev(starts), page_size=P, window=60, sinks=2, k_scale=back, v_scale=back,
                                     **t.kwargs())
            raw = t.raw.cpu().numpy()
            c = Cache.__new__(Cache)
            c.P, c.H, c.D, c.pages = P, H, D, 24
            if fmt == "16":
                c.values = [t.cache(s).double().cpu().numpy() for s in (0, 1)]
            elif fmt == "fp4":
                c.values = [fp4_decode(raw[s], t.scales[s].cpu().numpy()) for s in (0, 1)]
            else:
                tab = _paged.E4M3 if fmt == "e4m3fn" else _paged.E5M2
                c.values = [tab[raw[s]] * float(scale) for s in (0, 1)]
            ref, parts = attention(q.double().cpu().numpy(), c, order, lens, starts, 60, 2)
            assert_attention(out, ref, parts, src, f"{fmt} step {step}")
        assert check_flag() == (kv.OK, -1, 0)
