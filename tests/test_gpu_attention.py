"""GPU: attention over paged caches against a reference in 64 bits that reads
only the keys a row sees."""
import numpy as np
import pytest
import torch

import fp8_kv_quantization_amd as kv
from tests import _paged
from tests._gpu import check_flag
from tests._paged import TORCH, Cache, assert_attention, attention

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_flag(request):
    print(f"[gpu-case] {request.node.name}", flush=True)
    check_flag()
    yield
    torch.cuda.synchronize()


def make_table(rng, cache, lens, spare=0):
    need = [-(-n // cache.P) for n in lens]
    order = rng.permutation(cache.pages)
    table = np.full((len(lens), max(max(need), 1) + spare), -7, np.int32)   # unused entries name no page
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def pages_for(lens, P):
    return sum(-(-n // P) for n in lens) + 2


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def queries(rng, T, Hq, D, src, spread=2.0):
    return torch.from_numpy(rng.standard_normal((T, Hq, D)).astype(np.float32) * spread).to(TORCH[src]).cuda()


def check(rng, src, fmt, kind, lens, new, Hq, H, D, P, window=0, sinks=0, pad=0, cu=False, **kw):
    cache = Cache(rng, fmt if fmt != "16" else src, pages_for(lens, P), P, H, D, kind, pad)
    table = make_table(rng, cache, lens)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = queries(rng, int(starts[-1]), Hq, D, src)
    out = torch.full_like(q, 77.0)
    single = all(n == 1 for n in new)
    got = kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array(lens, np.int32)),
                             cu_q=None if single and not cu else dev(starts),
                             window=window, sinks=sinks, out=out, **cache.kwargs(), **kw)
    assert got is out
    ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, starts, window, sinks)
    assert_attention(out, ref, parts, src)
    assert check_flag() == (kv.OK, -1, 0)


FORMATS = [("16", "tensor"), ("e4m3fn", "tensor"), ("e4m3fn", "token"), ("e4m3fn", "head"),
           ("e5m2", "tensor"), ("e5m2", "head"), ("fp4", "block")]


@pytest.mark.parametrize("src", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,kind", FORMATS)
@pytest.mark.parametrize("D", [32, 64, 96, 128, 256])
def test_single_tokens(src, fmt, kind, D):
    rng = np.random.default_rng(D + len(fmt))
    check(rng, src, fmt, kind, [1, 2, 31, 32, 33, 77, 130], [1] * 7, 8, 2, D, 16)


@pytest.mark.parametrize("src", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,kind", FORMATS)
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_runs_of_tokens(src, fmt, kind, D):
    """Ragged runs: the tile kernel (more than 64 rows a sequence)."""
    rng = np.random.default_rng(D + 10 + len(fmt))
    check(rng, src, fmt, kind, [97, 1, 64, 200], [97, 1, 30, 41], 4, 2, D, 16)


@pytest.mark.parametrize("D", [16, 48, 80, 112, 144, 240])
@pytest.mark.parametrize("fmt", ["16", "e4m3fn"])
@pytest.mark.parametrize("new", [1, 70])
def test_head_dims(D, fmt, new):
    rng = np.random.default_rng(D)
    check(rng, "bf16", fmt, "tensor", [100, 71], [new, 1], 3, 3, D, 32)


@pytest.mark.parametrize("Hq,H", [(1, 1), (7, 7), (14, 2), (16, 1), (20, 1), (40, 1), (71, 1), (24, 8)])
@pytest.mark.parametrize("new", [1, 3, 9])
def test_head_groups(Hq, H, new):
    """Groups below, at and above a tile's rows."""
    rng = np.random.default_rng(Hq * 10 + new)
    check(rng, "bf16", "16", "tensor", [50, 9, 140], [new, new, new], Hq, H, 64, 16, cu=True)


@pytest.mark.parametrize("P", [1, 3, 16, 24, 33, 64, 100])
@pytest.mark.parametrize("new", [1, 5, 66])
def test_page_sizes(P, new):
    rng = np.random.default_rng(P * 7 + new)
    check(rng, "bf16", "e4m3fn", "head", [150, 66, 201], [new, new, new], 4, 2, 64, P)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (32, 4), (33, 40), (64, 64), (100, 1),
                                          (5000, 2), (17, 5000)])
@pytest.mark.parametrize("new", [1, 6, 80])
def test_windows_and_first_tokens(window, sinks, new):
    rng = np.random.default_rng(window + sinks + new)
    for fmt, kind in (("16", "tensor"), ("fp4", "block")):
        check(rng, "bf16", fmt, kind, [300, 80, 133], [new, new, new], 4, 2, 64, 16, window, sinks)


def test_first_tokens_without_a_window_change_nothing():
    rng = np.random.default_rng(3)
    check(rng, "bf16", "16", "tensor", [90, 40], [1, 1], 4, 2, 64, 16, window=0, sinks=9)


@pytest.mark.parametrize("fmt,kind", [("16", "tensor"), ("e4m3fn", "token"), ("fp4", "block")])
@pytest.mark.parametrize("new", [1, 4, 90])
def test_padded_strides(fmt, kind, new):
    """Caches inside larger allocations, q and out as slices of wider rows."""
    rng = np.random.default_rng(5)
    lens, P, H, Hq, D = [100, 93], 16, 2, 6, 64
    cache = Cache(rng, fmt if fmt != "16" else "bf16", pages_for(lens, P), P, H, D, kind, pad=16)
    table = make_table(rng, cache, lens, spare=3)
    starts = np.array([0, new, 2 * new], np.int32)
    q = queries(rng, 2 * new, Hq + 2, D + 8, "bf16")[:, 1:Hq + 1, :D]
    room = torch.full((2 * new, Hq + 1, D + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    out = room[:, :Hq, 8:D + 8]
    wide = dev(np.concatenate([table, table], axis=1))
    kv.attention_paged(q, cache.k, cache.v, wide[:, :table.shape[1]], dev(np.array(lens, np.int32)),
                       cu_q=dev(starts), out=out, **cache.kwargs())
    ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, starts)
    assert_attention(out, ref, parts, "bf16")
    assert (room[:, Hq:] == 5.0).all() and (room[:, :, :8] == 5.0).all() and (room[:, :, D + 8:] == 5.0).all()


@pytest.mark.parametrize("fmt,kind,D", [("16", "tensor", 128), ("e4m3fn", "head", 128), ("fp4", "block", 64)])
@pytest.mark.parametrize("new", [1, 2])
def test_long_contexts_are_split(fmt, kind, D, new):
    rng = np.random.default_rng(11)
    lens = [5000, 1, 2777]
    check(rng, "bf16", fmt, kind, lens, [min(new, n) for n in lens], 4, 1, D, 16, cu=True)


def test_long_context_split_for_many_rows():
    rng = np.random.default_rng(12)
    check(rng, "fp16", "16", "tensor", [2500], [70], 2, 1, 64, 64)


@pytest.mark.parametrize("hint", [1, 40, 5000])
def test_lengths_beyond_the_hints(hint):
    """max_len and max_q only steer the launch."""
    rng = np.random.default_rng(13)
    check(rng, "bf16", "16", "tensor", [4000, 100, 5000], [1, 3, 40], 4, 2, 64, 16, max_len=hint,
          max_q=min(hint, 2))


@pytest.mark.parametrize("P", [16, 10])
@pytest.mark.parametrize("new", [1, 3, 70])
@pytest.mark.parametrize("fmt,kind", [("16", "tensor"), ("e4m3fn", "head"), ("e5m2", "tensor"), ("fp4", "block")])
def test_nan_and_infinity_in_unseen_places(P, new, fmt, kind):
    """Slots behind a sequence's end, keys that a window hides, pages of others
    and dims beyond the head hold NaN and infinity; rows that do not see them
    do not notice, rows that see one get what the formula gives."""
    rng = np.random.default_rng(P + new)
    lens, H, Hq, D, window, sinks = [150, 80], 1, 2, 64, 40, 3
    src = "fp16" if fmt == "e5m2" else "bf16"
    cache = Cache(rng, fmt if fmt != "16" else src, pages_for(lens, P), P, H, D, kind)
    table = make_table(rng, cache, lens)
    used = np.zeros((cache.pages, P), bool)
    for b, n in enumerate(lens):
        hidden = max(0, n - new - window + 1)      # first key of the first new token's window
        for k in list(range(min(sinks, n))) + list(range(hidden, n)):
            used[table[b, k // P], k % P] = True
    bad = dict(e4m3fn=[0x7F, 0xFF], e5m2=[0x7C, 0xFD], fp4=[255]).get(fmt)
    for side, t in enumerate(cache.tensors):
        where = ~used
        if fmt == "fp4":
            s = cache.scales[side].cpu()
            s[torch.from_numpy(where)] = 255
            cache.scales[side].copy_(s)
        else:
            h = t.cpu()
            fill = h[torch.from_numpy(where)]
            if bad:
                fill[:] = torch.tensor(bad, dtype=torch.uint8).repeat(D // 2)
            else:
                fill[:] = torch.tensor([float("nan"), float("inf")]).repeat(D // 2).to(fill.dtype)
            h[torch.from_numpy(where)] = fill
            t.copy_(h)
    if kind == "head":
        for s in cache.scales:
            h = s.cpu()
            h[torch.from_numpy(~used)] = float("nan")
            s.copy_(h)
    # one visible key that only the later rows see: the last key of sequence 0
    starts = np.array([0, new, 2 * new], np.int32)
    q = queries(rng, 2 * new, Hq, D, src)
    out = torch.empty_like(q)

    def run():
        kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array(lens, np.int32)), cu_q=dev(starts),
                           window=window, sinks=sinks, out=out, **cache.kwargs())
        ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, starts, window, sinks)
        assert_attention(out, ref, parts, src)
        return ref

    assert np.isfinite(run()).all()
    if fmt != "fp4":
        # an infinity in V at the last key, in one dim, reaches the last row alone
        at = (table[0, (lens[0] - 1) // P], (lens[0] - 1) % P)
        value = {"e4m3fn": 0x7F, "e5m2": 0x7C}.get(fmt, float("inf"))
        cache.tensors[1][at[0], at[1], 0, 5] = value
        cache.values[1][at[0], at[1], 0, 5] = np.nan if fmt == "e4m3fn" else np.inf
        got = run()
        assert not np.isfinite(got[new - 1, :, 5]).any() and np.isfinite(got[:new - 1]).all()
        assert np.isfinite(got[new:]).all()


def test_empty_rows_are_zero_and_other_rows_are_left():
    """No keys (length 0), positions before the sequence (more new tokens than
    keys), rows before and behind the sequences."""
    rng = np.random.default_rng(17)
    P, H, Hq, D = 16, 2, 4, 64
    lens = [0, 3, 40, -5]
    cache = Cache(rng, "bf16", 8, P, H, D)
    table = make_table(rng, cache, [16, 16, 40, 16])
    for new, kwargs in (([1, 5, 2, 1], {}), ([2, 90, 3, 4], {})):
        starts = (np.concatenate([[0], np.cumsum(new)]) + 2).astype(np.int32)
        T = int(starts[-1]) + 3
        q = queries(rng, T, Hq, D, "bf16")
        out = torch.full_like(q, 77.0)
        kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array(lens, np.int32)), cu_q=dev(starts),
                           out=out, **cache.kwargs(), **kwargs)
        o = out.double().cpu().numpy()
        assert (o[:2] == 77.0).all() and (o[starts[-1]:] == 77.0).all()
        ref, parts = attention(q.double().cpu().numpy(), cache, table, [max(n, 0) for n in lens], starts)
        assert_attention(out, ref, parts, "bf16")
        assert (o[starts[0]:starts[1]] == 0).all() and (o[starts[3]:starts[4]] == 0).all()
        assert (o[starts[1]:starts[2] - 3] == 0).all()
    assert check_flag() == (kv.OK, -1, 0)


def test_lengths_are_cut_to_the_table():
    rng = np.random.default_rng(18)
    cache = Cache(rng, "bf16", 6, 16, 1, 64)
    table = rng.permutation(6)[:4].astype(np.int32).reshape(2, 2)
    q = queries(rng, 2, 2, 64, "bf16")
    out = kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array([1000, 2 ** 31 - 1], np.int32)),
                             **cache.kwargs())
    ref, parts = attention(q.double().cpu().numpy(), cache, table, [32, 32], [0, 1, 2])
    assert_attention(out, ref, parts, "bf16")


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("P", [16, 7])
def test_bad_pages_hold_no_keys_and_are_recorded(new, P):
    rng = np.random.default_rng(19)
    lens, H, Hq, D = [100, 90, 75], 2, 4, 64
    cache = Cache(rng, "bf16", pages_for(lens, P), P, H, D)
    table = make_table(rng, cache, lens)
    table[1, 2] = cache.pages
    table[2, 0] = -1
    starts = np.array([0, new, 2 * new, 3 * new], np.int32)
    q = queries(rng, 3 * new, Hq, D, "bf16")
    out = kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array(lens, np.int32)), cu_q=dev(starts),
                             **cache.kwargs())
    ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, starts)
    assert_attention(out, ref, parts, "bf16")
    st, first, count = check_flag()
    assert st == kv.ERR_OOB and first == new and count >= 2
    # a sequence of bad pages only
    table[:] = 2 ** 31 - 1
    out = kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array(lens, np.int32)), cu_q=dev(starts),
                             **cache.kwargs())
    assert (out == 0).all()
    assert check_flag()[:2] == (kv.ERR_OOB, 0)


@pytest.mark.parametrize("B", [63, 64, 65, 300, 4200])
def test_many_sequences(B):
    """Runs of 0 to 3 tokens: sequences are found among many."""
    rng = np.random.default_rng(B)
    P, H, Hq, D = 16, 1, 2, 16
    lens = rng.integers(1, 30, B).tolist()
    new = [int(min(n, k)) for n, k in zip(lens, rng.integers(0, 4, B))]
    cache = Cache(rng, "bf16", pages_for(lens, P), P, H, D)
    table = make_table(rng, cache, lens)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = queries(rng, int(starts[-1]), Hq, D, "bf16")
    ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, starts)
    for max_q in (3, None):       # tiles of 16 rows, and of 128
        out = torch.full_like(q, 77.0)
        kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array(lens, np.int32)), cu_q=dev(starts),
                           max_q=max_q, out=out, **cache.kwargs())
        assert_attention(out, ref, parts, "bf16")


def test_starts_outside_the_rows_are_cut():
    rng = np.random.default_rng(23)
    cache = Cache(rng, "bf16", 12, 16, 1, 64)
    lens = [50, 60]
    table = make_table(rng, cache, lens)
    q = queries(rng, 6, 2, 64, "bf16")
    out = torch.full_like(q, 77.0)
    kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array(lens, np.int32)),
                       cu_q=dev(np.array([-9, 2, 900], np.int32)), out=out, **cache.kwargs())
    ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, [0, 2, 6])
    assert_attention(out, ref, parts, "bf16")


@pytest.mark.parametrize("new", [1, 70])
def test_cache_offsets_past_32_bits(new):
    """Pages at the end of caches of 5 GiB each."""
    rng = np.random.default_rng(29)
    P, H, D, lens = 16, 2, 64, [100, 40]
    small = Cache(rng, "e4m3fn", pages_for(lens, P), P, H, D)
    total = (5 << 30) // (P * H * D)
    far = total - small.pages
    big = []
    for t in small.tensors:
        c = torch.empty((total, P, H, D), dtype=torch.uint8, device="cuda")
        c[far:] = t
        big.append(c.view(torch.float8_e4m3fn))
    table = make_table(rng, small, lens)
    starts = np.array([0, new, new + 1], np.int32)
    q = queries(rng, new + 1, 4, D, "bf16")
    out = kv.attention_paged(q, big[0], big[1], dev(np.where(table < 0, table, table + far).astype(np.int32)),
                             dev(np.array(lens, np.int32)), cu_q=dev(starts), **small.kwargs())
    ref, parts = attention(q.double().cpu().numpy(), small, table, lens, starts)
    assert_attention(out, ref, parts, "bf16")


@pytest.mark.parametrize("scale", [0.0, 0.3, 4.0])
@pytest.mark.parametrize("new", [1, 70])
def test_score_scales(scale, new):
    rng = np.random.default_rng(31)
    lens = [100, 70]
    cache = Cache(rng, "bf16", pages_for(lens, 16), 16, 1, 64)
    table = make_table(rng, cache, lens)
    starts = np.array([0, new, 2 * new], np.int32)
    q = queries(rng, 2 * new, 2, 64, "bf16")
    out = kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array(lens, np.int32)), cu_q=dev(starts),
                             sm_scale=scale, **cache.kwargs())
    ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, starts, scale=scale)
    assert_attention(out, ref, parts, "bf16")


@pytest.mark.parametrize("new", [1, 70])
def test_large_scores_rise_along_the_sequence(new):
    """Scores that grow by hundreds from key to key, and fall: the running
    maximum is raised many times, and weights underflow."""
    rng = np.random.default_rng(37)
    lens = [400, 200]
    cache = Cache(rng, "bf16", pages_for(lens, 16), 16, 1, 64)
    table = make_table(rng, cache, lens)
    for b, n in enumerate(lens):
        for k in range(n):
            at = table[b, k // 16], k % 16
            row = cache.values[0][at][0] * (k if b == 0 else n - k) / 8.0
            t = torch.from_numpy(row).to(torch.bfloat16)
            cache.tensors[0][at[0], at[1], 0] = t.cuda()
            cache.values[0][at][0] = t.double().numpy()
    starts = np.array([0, new, 2 * new], np.int32)
    q = queries(rng, 2 * new, 2, 64, "bf16")
    out = kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array(lens, np.int32)), cu_q=dev(starts),
                             **cache.kwargs())
    ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, starts)
    assert_attention(out, ref, parts, "bf16")


@pytest.mark.parametrize("new", [1, 70])
def test_negative_tensor_scales(new):
    rng = np.random.default_rng(41)
    lens = [100, 70]
    cache = Cache(rng, "e4m3fn", pages_for(lens, 16), 16, 1, 64)
    cache.k_scale.neg_()
    cache.v_scale.neg_()
    cache.values = [-x for x in cache.values]
    table = make_table(rng, cache, lens)
    starts = np.array([0, new, 2 * new], np.int32)
    q = queries(rng, 2 * new, 2, 64, "bf16")
    out = kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array(lens, np.int32)), cu_q=dev(starts),
                             **cache.kwargs())
    ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, starts)
    assert_attention(out, ref, parts, "bf16")


@pytest.mark.parametrize("new", [1, 70])
def test_same_page_twice_and_shared_pages(new):
    """Sequences that share a prefix's pages, and one that repeats a page."""
    rng = np.random.default_rng(43)
    lens = [120, 120, 64]
    cache = Cache(rng, "bf16", 20, 16, 2, 64)
    table = make_table(rng, cache, lens)
    table[1, :5] = table[0, :5]
    table[2, 1] = table[2, 0]
    starts = np.array([0, new, 2 * new, 2 * new + 1], np.int32)
    q = queries(rng, 2 * new + 1, 4, 64, "bf16")
    out = kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array(lens, np.int32)), cu_q=dev(starts),
                             **cache.kwargs())
    ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, starts)
    assert_attention(out, ref, parts, "bf16")


@pytest.mark.parametrize("new", [1, 70])
def test_two_runs_agree_bit_for_bit(new):
    rng = np.random.default_rng(47)
    lens = [3000, 1200]
    cache = Cache(rng, "bf16", pages_for(lens, 16), 16, 1, 64)
    table, n = dev(make_table(rng, cache, lens)), dev(np.array(lens, np.int32))
    starts = dev(np.array([0, new, 2 * new], np.int32))
    q = queries(rng, 2 * new, 2, 64, "bf16")
    a = [kv.attention_paged(q, cache.k, cache.v, table, n, cu_q=starts, **cache.kwargs()) for _ in range(3)]
    assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[2])


def test_given_workspace_and_flat_cache():
    rng = np.random.default_rng(53)
    lens = [4000, 90]
    cache = Cache(rng, "bf16", pages_for(lens, 16), 16, 1, 64)
    table = make_table(rng, cache, lens)
    q = queries(rng, 2, 2, 64, "bf16")
    args = (q, cache.k.flatten(0, 1), cache.v.flatten(0, 1), dev(table), dev(np.array(lens, np.int32)))
    need = kv.attention_paged_workspace(*args)
    assert need > 0
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    out = kv.attention_paged(*args, workspace=ws[:need])
    assert (ws[need:] == 0xFF).all()
    ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, [0, 1, 2])
    assert_attention(out, ref, parts, "bf16")
    with pytest.raises(kv.KVStoreError):
        kv.attention_paged(*args, workspace=ws[:need - 16])


@pytest.mark.parametrize("new", [1, 70])
def test_captured_and_replayed(new):
    """Two graphs captured from the same call, replayed in turn with eager calls
    between, inputs overwritten between replays; then on another stream."""
    rng = np.random.default_rng(59)
    lens = [3000, 500]
    cache = Cache(rng, "e4m3fn", pages_for(lens, 16), 16, 1, 64, "head")
    table = make_table(rng, cache, lens)
    starts = np.array([0, new, 2 * new], np.int32)
    d_table, d_lens, d_starts = dev(table), dev(np.array(lens, np.int32)), dev(starts)
    q = queries(rng, 2 * new, 2, 64, "bf16")
    outs = [torch.empty_like(q) for _ in range(3)]

    def call(i):
        kv.attention_paged(q, cache.k, cache.v, d_table, d_lens, cu_q=d_starts, out=outs[i], **cache.kwargs())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(0)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for k in range(4):
        q.copy_(queries(rng, 2 * new, 2, 64, "bf16"))
        lens = [3000 - 700 * k, 500 - k]
        if min(lens) < new:
            lens = [new, new]
        d_lens.copy_(dev(np.array(lens, np.int32)))
        torch.cuda.synchronize()
        graphs[k % 2].replay()
        call(2)
        graphs[1 - k % 2].replay()
        torch.cuda.synchronize()
        ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, starts)
        for o in outs:
            assert_attention(o, ref, parts, "bf16", f"replay {k}")
            assert torch.equal(o, outs[0])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = kv.attention_paged(q, cache.k, cache.v, d_table, d_lens, cu_q=d_starts, stream=other, **cache.kwargs())
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(got, outs[0])
