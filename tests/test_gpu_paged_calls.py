"""GPU: how calls of the paged-cache operators meet each other: threads,
streams, captured graphs, hints, empty calls, shared tables."""
import threading

import numpy as np
import pytest
import torch

import fp8_kv_quantization_amd as kv
from tests._gpu import check_flag
from tests._paged import Cache, assert_attention, attention
from tests.test_gpu_attention import dev, make_table, pages_for, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_flag(request):
    print(f"[gpu-case] {request.node.name}", flush=True)
    check_flag()
    yield
    torch.cuda.synchronize()


class Case:
    """Attention of `new` tokens a sequence, and its call."""

    def __init__(self, seed, lens, new, fmt="bf16", kind="tensor", H=2, Hq=4, D=64, P=16):
        rng = np.random.default_rng(seed)
        self.lens, self.cache = lens, Cache(rng, fmt, pages_for(lens, P), P, H, D, kind)
        self.table = make_table(rng, self.cache, lens)
        self.starts = np.arange(len(lens) + 1, dtype=np.int32) * new
        self.q = queries(rng, new * len(lens), Hq, D, "bf16")
        self.args = (self.q, self.cache.k, self.cache.v, dev(self.table), dev(np.array(lens, np.int32)))
        self.d_starts = dev(self.starts)

    def __call__(self, **kw):
        return kv.attention_paged(*self.args, cu_q=self.d_starts, **self.cache.kwargs(), **kw)

    def workspace(self):
        need = kv.attention_paged_workspace(*self.args, cu_q=self.d_starts, **self.cache.kwargs())
        return torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")

    def check(self, out):
        ref, parts = attention(self.q.double().cpu().numpy(), self.cache, self.table, self.lens, self.starts)
        assert_attention(out, ref, parts, "bf16")


# splits of long contexts (with a workspace), tiles of many rows, 4 bits
CASES = [dict(lens=[3000, 900], new=1), dict(lens=[400, 333], new=90),
         dict(lens=[2500, 64], new=3, fmt="fp4", kind="block"), dict(lens=[1500, 200], new=80, fmt="e4m3fn", kind="head")]


def test_calls_of_several_threads_and_streams():
    cases = [Case(i, **c) for i, c in enumerate(CASES)]
    alone = [c() for c in cases]
    torch.cuda.synchronize()
    for case, out in zip(cases, alone):
        case.check(out)
    wrong = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(10):
                out = cases[i](stream=stream)
                stream.synchronize()
                if not torch.equal(out, alone[i]):
                    wrong.append(i)
        except Exception as e:   # shown by the assertion below
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []
    assert check_flag() == (kv.OK, -1, 0)


def test_two_graphs_replayed_at_once():
    """Each graph has a workspace of its own; they run side by side on two
    streams, with eager calls between the replays."""
    cases = [Case(10 + i, **c) for i, c in enumerate((CASES[0], CASES[2]))]
    alone = [c() for c in cases]
    outs = [torch.zeros_like(c.q) for c in cases]
    spaces = [c.workspace() for c in cases]
    torch.cuda.synchronize()
    graphs = []
    for c, out, ws in zip(cases, outs, spaces):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c(out=out, workspace=ws)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = cases[0]()
        torch.cuda.synchronize()
        assert torch.equal(eager, alone[0])
        for out, want in zip(outs, alone):
            assert torch.equal(out, want)


def test_append_attend_and_load_in_one_graph():
    """A decode step as a serving loop captures it; positions, slots, lengths and
    rows are overwritten between replays."""
    rng = np.random.default_rng(20)
    B, H, Hq, D, P, pages = 3, 2, 4, 64, 16, 12
    cache = [torch.zeros(pages, P, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = dev(rng.permutation(pages).reshape(B, 4).astype(np.int32))
    angles = np.arange(64)[:, None] / 10000.0 ** (np.arange(D // 2) / (D // 2))
    cos_sin = dev(np.concatenate([np.cos(angles), np.sin(angles)], 1).astype(np.float32))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    slots, positions = (torch.zeros(B, dtype=torch.int64, device="cuda") for _ in range(2))
    k, v = (queries(rng, B, H, D, "bf16") for _ in range(2))
    q, out = queries(rng, B, Hq, D, "bf16"), torch.zeros(B, Hq, D, dtype=torch.bfloat16, device="cuda")
    q_out, back = torch.empty_like(q), [torch.empty_like(k) for _ in range(2)]

    def step(cache, q_out, out, back):
        kv.store_kv_rope_paged(k, v, *cache, slots, positions, cos_sin, q=q, q_out=q_out, page_size=P)
        kv.attention_paged(q_out, *cache, table, lens, out=out, page_size=P)
        kv.load_kv_paged(*cache, slots, *back, page_size=P)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, q_out, out, back)
    eager_cache = [c.clone() for c in cache]
    eager = torch.empty_like(q), torch.empty_like(q), [torch.empty_like(k) for _ in range(2)]
    for n in range(1, 40):
        for x, heads in ((k, H), (v, H), (q, Hq)):
            x.copy_(queries(rng, B, heads, D, "bf16"))
        lens.fill_(n)
        positions.fill_(n - 1)
        slots.copy_(table[:, (n - 1) // P].long() * P + (n - 1) % P)
        torch.cuda.synchronize()
        graph.replay()
        step(eager_cache, *eager)
        torch.cuda.synchronize()
        assert torch.equal(q_out, eager[0]) and torch.equal(out, eager[1])
        for a, b in zip(cache + back, eager_cache + eager[2]):
            assert torch.equal(a, b)
    for side, raw in enumerate((k, v)):
        if side:   # v is stored as it is
            assert torch.equal(back[1], raw)


@pytest.mark.parametrize("hint", [1, 5, 20, 10000])
@pytest.mark.parametrize("case", [0, 1, 3])
def test_wrong_hints_of_new_tokens(case, hint):
    c = Case(30 + case, **CASES[case])
    c.check(c(max_q=hint))


def test_a_table_that_sequences_share():
    c = Case(40, lens=[700, 700, 700], new=2)
    c.table = np.repeat(c.table[:1], 3, 0)
    args = list(c.args)
    args[3] = dev(c.table[:1]).expand(3, -1)
    c.args = tuple(args)
    c.check(c())


def test_empty_calls():
    c = Case(50, lens=[30, 40], new=2)
    none = c.q[:0]
    loc = torch.zeros(0, dtype=torch.int64, device="cuda")
    empty = dev(np.zeros(3, np.int32))
    assert kv.attention_paged(none, *c.args[1:], cu_q=empty, **c.cache.kwargs()).shape == none.shape
    out = torch.full_like(c.q, 5.0)     # no sequences: no rows of out are written
    kv.attention_paged(c.q, *c.args[1:3], c.args[3][:0], c.args[4][:0], cu_q=empty[:1], out=out,
                       **c.cache.kwargs())
    assert (out == 5.0).all()
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    kv.store_kv_rope_paged(k, k, c.cache.k, c.cache.v, loc, None, None, page_size=16)
    kv.load_kv_paged(c.cache.k, c.cache.v, loc, k, k, page_size=16)
    assert check_flag() == (kv.OK, -1, 0)


def test_the_same_slot_loaded_twice():
    c = Case(60, lens=[64], new=1)
    loc = torch.tensor([3, 9, 3, 3], dtype=torch.int32, device="cuda")
    out = [torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kv.load_kv_paged(c.cache.k, c.cache.v, loc, *out, page_size=16)
    for o, side in zip(out, (c.cache.k, c.cache.v)):
        assert torch.equal(o, side.flatten(0, 1)[loc.long()])


def test_in_place_attention_is_refused():
    c = Case(70, lens=[64], new=1)
    with pytest.raises(kv.KVStoreError):
        c(out=c.q)


@pytest.mark.parametrize("D", [80, 128, 256])
@pytest.mark.parametrize("P", [16, 7])
@pytest.mark.parametrize("lens", [[1, 0, 63], [64, 65, 900], [2500, 128, 3]])
def test_single_tokens_where_much_may_be_read(D, P, lens):
    """Tables wide enough for long contexts, whatever the sequences hold."""
    rng = np.random.default_rng(D + P)
    cache = Cache(rng, "bf16", pages_for(lens, P), P, 2, D, "tensor")
    table = make_table(rng, cache, lens, spare=60000 // P)
    q = queries(rng, 3, 8, D, "bf16")
    out = kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array(lens, np.int32)), **cache.kwargs())
    ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, [0, 1, 2, 3])
    assert_attention(out, ref, parts, "bf16")
    assert check_flag() == (kv.OK, -1, 0)


@pytest.mark.parametrize("new", [4, 5, 33])
@pytest.mark.parametrize("fmt,kind", [("bf16", "tensor"), ("e5m2", "token"), ("fp4", "block")])
def test_short_runs_over_long_contexts(new, fmt, kind):
    c = Case(80 + new, lens=[6000, 40, 1111], new=new, fmt=fmt, kind=kind)
    c.check(c(max_q=new, max_len=6000))


@pytest.mark.parametrize("P", [16, 10])
@pytest.mark.parametrize("window,sinks", [(0, 0), (24600, 5)])
def test_unseen_nan_where_much_is_read(P, window, sinks):
    """Single tokens over long 16-bit contexts: slots that no token sees hold NaN
    and infinity."""
    rng = np.random.default_rng(P + window)
    lens, D = [25000, 24700], 128
    cache = Cache(rng, "bf16", pages_for(lens, P), P, 2, D, "tensor")
    table = make_table(rng, cache, lens)
    unseen = np.ones((cache.pages, P), bool)
    for b, n in enumerate(lens):
        for k in list(range(min(sinks, n))) + list(range(max(0, n - window) if window else 0, n)):
            unseen[table[b, k // P], k % P] = False
    where = torch.from_numpy(unseen)
    for t in cache.tensors:
        h = t.cpu()
        h[where] = torch.tensor([float("nan"), float("inf")]).repeat(D // 2).to(h.dtype)
        t.copy_(h)
    q = queries(rng, 2, 4, D, "bf16")
    out = kv.attention_paged(q, cache.k, cache.v, dev(table), dev(np.array(lens, np.int32)), window=window,
                             sinks=sinks, **cache.kwargs())
    ref, parts = attention(q.double().cpu().numpy(), cache, table, lens, [0, 1, 2], window, sinks)
    assert np.isfinite(ref).all()
    assert_attention(out, ref, parts, "bf16")
    assert check_flag() == (kv.OK, -1, 0)
