"""The C boundary of the paged-cache operators (include/kvstore_paged.h): its
functions are exported, and bad arguments are refused before anything is
launched (CPU only: fake device addresses, so a slip would be a failed launch).

Each rejected case changes one thing of an otherwise valid call.
"""
import ctypes as C
import os
import re

import pytest

from tests.test_abi import A, cpu_only

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kvstore_paged.h")
NULL, SHAPE, ALIGN, DTYPE, HIP = -1, -2, -3, -4, -5

i32, i64, u32, ptr = C.c_int32, C.c_int64, C.c_uint32, C.c_void_p


class Cache(C.Structure):
    _fields_ = [("k", ptr), ("v", ptr), ("format", i32), ("scale_kind", i32), ("num_heads", i32),
                ("head_dim", i32), ("page_size", i64), ("num_slots", i64),
                ("k_page", i64), ("k_offset", i64), ("k_head", i64),
                ("v_page", i64), ("v_offset", i64), ("v_head", i64),
                ("k_scales", ptr), ("v_scales", ptr),
                ("ks_page", i64), ("ks_offset", i64), ("ks_head", i64),
                ("vs_page", i64), ("vs_offset", i64), ("vs_head", i64)]


class Rows(C.Structure):
    _fields_ = [("q", ptr), ("q_out", ptr), ("k", ptr), ("v", ptr), ("src_dtype", i32),
                ("q_heads", i32), ("q_token", i64), ("q_head", i64), ("qo_token", i64),
                ("qo_head", i64), ("k_token", i64), ("k_head", i64), ("v_token", i64),
                ("v_head", i64)]


class Attention(C.Structure):
    _fields_ = [("q", ptr), ("out", ptr), ("q_token", i64), ("q_head", i64), ("o_token", i64),
                ("o_head", i64), ("src_dtype", i32), ("q_heads", i32), ("cu_q", ptr),
                ("tokens", u32), ("seqs", u32), ("max_q", u32), ("page_table", ptr),
                ("table_stride", i64), ("max_pages", u32), ("seq_lens", ptr), ("max_len", i64),
                ("window", i64), ("sinks", i64), ("sm_scale", C.c_float), ("workspace", ptr),
                ("workspace_bytes", i64)]


def declared_functions():
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^(?:int|int64_t) (kvstore_\w+)\s*\(", text, re.M)))


@pytest.fixture(scope="module")
def lib():
    import fp8_kv_quantization_amd as kv
    lib = C.CDLL(kv.LIB_PATH)
    lib.kvstore_attention_workspace.restype = i64
    lib.kvstore_attention_workspace.argtypes = [ptr, ptr]
    lib.kvstore_attention_paged.argtypes = [ptr, ptr, ptr]
    lib.kvstore_rope_paged.argtypes = [ptr, ptr, C.c_int, ptr, i64, i64, i32, C.c_int, ptr, C.c_int,
                                       i64, ptr, ptr, ptr, u32, ptr]
    lib.kvstore_load_paged.argtypes = [ptr, ptr, C.c_int, i64, ptr, i64, i64, ptr, i64, i64, C.c_int,
                                       u32, ptr]
    return lib


def test_header_and_exports(lib):
    names = declared_functions()
    assert names == ["kvstore_attention_paged", "kvstore_attention_workspace", "kvstore_load_paged",
                     "kvstore_rope_paged"]
    import fp8_kv_quantization_amd as kv
    for name in names:
        assert hasattr(lib, name), name
        assert type(getattr(kv, name)).__name__ == "builtin_function_or_method", name


# 8 heads of 128 dims, 64 pages of 16 slots, by format: (format, kind, bytes of a head)
FORMATS = {"bf16": (0, 0, 256), "fp16": (1, 0, 256), "e4m3fn": (2, 0, 128), "e4m3fn token": (2, 1, 128),
           "e5m2 head": (3, 2, 128), "fp4": (4, 3, 64)}


def cache(fmt="bf16", **over):
    code, kind, head = FORMATS[fmt]
    unit = 1 if fmt == "fp4" else 4
    per = 4 if fmt == "fp4" else 1 if kind == 2 else 0   # scales of a head
    c = dict(k=A, v=A + 0x1000000, format=code, scale_kind=kind, num_heads=8, head_dim=128,
             page_size=16, num_slots=1024, k_page=128 * head, k_offset=8 * head, k_head=head,
             v_page=128 * head, v_offset=8 * head, v_head=head,
             k_scales=A + 0x2000000 if kind else None, v_scales=A + 0x3000000 if kind else None,
             ks_page=512 * unit, ks_offset=32 * unit, ks_head=per * unit,
             vs_page=512 * unit, vs_offset=32 * unit, vs_head=per * unit)
    c.update(over)
    return Cache(**c)


def rope(lib, fmt="bf16", cache_over={}, rows_over={}, **over):
    r = dict(q=A + 0x4000000, q_out=A + 0x5000000, k=A + 0x6000000, v=A + 0x7000000,
             src_dtype=1 if fmt == "fp16" else 0, q_heads=32, q_token=8192, q_head=256, qo_token=8192,
             qo_head=256, k_token=2048, k_head=256, v_token=2048, v_head=256)
    r.update(rows_over)
    a = dict(positions=A + 0x8000000, pos_dtype=1, cos_sin=A + 0x9000000, cs_stride=512, num=4096,
             rot=128, inter=0, indices=A + 0xA000000, idx_dtype=0, idx_stride=1, inv_k=None, inv_v=None,
             batch=16)
    a.update(over)
    return lib.kvstore_rope_paged(
        C.byref(Rows(**r)), a["positions"], a["pos_dtype"], a["cos_sin"], a["cs_stride"], a["num"],
        a["rot"], a["inter"], a["indices"], a["idx_dtype"], a["idx_stride"],
        C.byref(cache(fmt, **cache_over)), a["inv_k"], a["inv_v"], a["batch"], None)


def load(lib, fmt="bf16", cache_over={}, **over):
    a = dict(indices=A + 0xA000000, idx_dtype=0, idx_stride=1, k_out=A + 0x4000000, ko_token=2048,
             ko_head=256, v_out=A + 0x5000000, vo_token=2048, vo_head=256,
             dst=1 if fmt == "fp16" else 0, batch=16)
    a.update(over)
    return lib.kvstore_load_paged(C.byref(cache(fmt, **cache_over)), *a.values(), None)


def attention_args(fmt="bf16", **over):
    a = dict(q=A + 0x4000000, out=A + 0x5000000, q_token=8192, q_head=256, o_token=8192, o_head=256,
             src_dtype=1 if fmt == "fp16" else 0, q_heads=32, cu_q=A + 0x6000000, tokens=64, seqs=4,
             max_q=0, page_table=A + 0x7000000, table_stride=64, max_pages=64,
             seq_lens=A + 0x8000000, max_len=0, window=0, sinks=0, sm_scale=0.1,
             workspace=A + 0x9000000, workspace_bytes=1 << 40)
    a.update(over)
    return Attention(**a)


def attend(lib, fmt="bf16", cache_over={}, **over):
    return lib.kvstore_attention_paged(C.byref(attention_args(fmt, **over)),
                                       C.byref(cache(fmt, **cache_over)), None)


@cpu_only
@pytest.mark.parametrize("fmt", FORMATS)
def test_valid_arguments_reach_the_runtime(lib, fmt):
    assert load(lib, fmt) == HIP
    assert attend(lib, fmt) == HIP
    assert attend(lib, fmt, cu_q=None, seqs=64) == HIP
    assert rope(lib, fmt) == (DTYPE if fmt in ("e4m3fn token", "e5m2 head") else HIP)
    if fmt == "e4m3fn":
        assert rope(lib, fmt, inv_k=A, inv_v=A + 4) == HIP
    if fmt == "fp4":
        assert rope(lib, fmt, cos_sin=None, positions=None, rows_over=dict(q=None, q_out=None)) == HIP


# A cache's own rules: the same for all three calls.
CACHE_BAD = [
    ("bf16", dict(k=None), NULL), ("bf16", dict(v=None), NULL),
    ("bf16", dict(format=5), DTYPE), ("bf16", dict(format=-1), DTYPE),
    ("bf16", dict(scale_kind=1), DTYPE), ("fp4", dict(scale_kind=0), DTYPE),
    ("e4m3fn", dict(scale_kind=3), DTYPE), ("e4m3fn", dict(scale_kind=-1), DTYPE),
    ("fp4", dict(k_scales=None), NULL), ("fp4", dict(v_scales=None), NULL),
    ("bf16", dict(num_heads=0), SHAPE), ("bf16", dict(num_heads=-8), SHAPE),
    ("bf16", dict(head_dim=0), SHAPE), ("bf16", dict(head_dim=120), SHAPE),
    ("fp4", dict(head_dim=48), SHAPE), ("bf16", dict(head_dim=528), SHAPE),
    ("bf16", dict(page_size=0), SHAPE), ("bf16", dict(num_slots=0), SHAPE),
    ("bf16", dict(num_slots=-16), SHAPE),
    ("bf16", dict(k_page=-32768), SHAPE), ("bf16", dict(v_head=-256), SHAPE),
    ("bf16", dict(k_offset=2056), ALIGN), ("fp4", dict(v_head=72), ALIGN),
    ("bf16", dict(k=A + 8), ALIGN), ("bf16", dict(v=A + 0x1000002), ALIGN),
    ("bf16", dict(k_page=1 << 62), SHAPE), ("bf16", dict(v_offset=1 << 60, num_slots=64), SHAPE),
    ("bf16", dict(k_head=1 << 31), SHAPE),
    ("fp4", dict(ks_page=-1), SHAPE), ("fp4", dict(vs_page=1 << 62), SHAPE),
    ("fp4", dict(vs_head=1 << 31), SHAPE),
]


@cpu_only
@pytest.mark.parametrize("fmt,over,status", CACHE_BAD)
def test_caches_refused(lib, fmt, over, status):
    assert rope(lib, fmt, cache_over=over) == status
    assert load(lib, fmt, cache_over=over) == status
    assert attend(lib, fmt, cache_over=over) == status


@cpu_only
@pytest.mark.parametrize("fmt,over,status", [
    ("e4m3fn token", dict(k_scales=None), NULL), ("e5m2 head", dict(v_scales=None), NULL),
    ("e4m3fn token", dict(k_scales=A + 2), ALIGN), ("e5m2 head", dict(vs_head=2), ALIGN),
    ("e4m3fn token", dict(ks_offset=-4), SHAPE), ("e4m3fn", dict(k_scales=A + 2), ALIGN),
])
def test_fp8_scales_refused_by_readers(lib, fmt, over, status):
    assert load(lib, fmt, cache_over=over) == status
    assert attend(lib, fmt, cache_over=over) == status


@cpu_only
@pytest.mark.parametrize("over,status", [
    (dict(idx_dtype=2), DTYPE), (dict(pos_dtype=2), DTYPE), (dict(rows_over=dict(src_dtype=2)), DTYPE),
    (dict(rows_over=dict(src_dtype=1)), DTYPE),                 # fp16 rows, bf16 cache
    (dict(rows_over=dict(k=None)), NULL), (dict(rows_over=dict(v=None)), NULL),
    (dict(rows_over=dict(q_out=None)), NULL), (dict(indices=None), NULL),
    (dict(positions=None), NULL), (dict(cos_sin=None), NULL),
    (dict(rows_over=dict(q_heads=0)), SHAPE), (dict(rows_over=dict(q_heads=1 << 25, q_head=0, qo_head=0)), SHAPE),
    (dict(rows_over=dict(q_token=-16)), SHAPE), (dict(rows_over=dict(qo_head=-16)), SHAPE),
    (dict(rows_over=dict(k_token=2056)), ALIGN), (dict(rows_over=dict(v=A + 0x7000008)), ALIGN),
    (dict(rows_over=dict(q=A + 0x4000004)), ALIGN), (dict(rows_over=dict(q_out=A + 0x5000004)), ALIGN),
    (dict(rows_over=dict(q_out=A + 0x4000000, qo_token=16384)), SHAPE),   # in place, other strides
    (dict(rows_over=dict(k_token=1 << 60)), SHAPE), (dict(rows_over=dict(q_head=1 << 31)), SHAPE),
    (dict(rot=0), SHAPE), (dict(rot=24), SHAPE), (dict(rot=144), SHAPE), (dict(rot=-16), SHAPE),
    (dict(num=0), SHAPE), (dict(cs_stride=256), SHAPE), (dict(cs_stride=1 << 62), SHAPE),
    (dict(cs_stride=520), ALIGN), (dict(cos_sin=A + 0x9000008), ALIGN),
    (dict(positions=A + 0x8000004), ALIGN), (dict(positions=A + 0x8000002, pos_dtype=0), ALIGN),
    (dict(indices=A + 2), ALIGN), (dict(idx_stride=0), SHAPE), (dict(idx_stride=1 << 62), SHAPE),
    (dict(inv_k=A + 2), ALIGN),
])
def test_rope_refused(lib, over, status):
    assert rope(lib, **over) == status


@cpu_only
@pytest.mark.parametrize("over,status", [
    (dict(idx_dtype=2), DTYPE), (dict(dst=2), DTYPE), (dict(dst=1), DTYPE), (dict(indices=None), NULL),
    (dict(k_out=None), NULL), (dict(v_out=None), NULL), (dict(ko_token=-16), SHAPE),
    (dict(vo_head=264), ALIGN), (dict(k_out=A + 0x4000008), ALIGN), (dict(vo_token=1 << 61), SHAPE),
    (dict(indices=A + 4, idx_dtype=1), ALIGN), (dict(idx_stride=0), SHAPE),
])
def test_load_refused(lib, over, status):
    assert load(lib, **over) == status


@cpu_only
@pytest.mark.parametrize("over,status", [
    (dict(src_dtype=2), DTYPE), (dict(src_dtype=1), DTYPE),
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(page_table=None), NULL), (dict(seq_lens=None), NULL),
    (dict(out=A + 0x4000000), SHAPE),                            # in place
    (dict(q_heads=0), SHAPE), (dict(q_heads=12), SHAPE), (dict(q_heads=-32), SHAPE),
    (dict(cu_q=None), SHAPE),                                    # 64 rows, 4 sequences
    (dict(tokens=1 << 31, q_heads=8), SHAPE), (dict(tokens=1 << 27), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 27), SHAPE), (dict(max_len=-1), SHAPE),
    (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE),
    (dict(sm_scale=-0.1), SHAPE), (dict(sm_scale=float("nan")), SHAPE), (dict(sm_scale=float("inf")), SHAPE),
    (dict(sm_scale=3e38), SHAPE),                                # times log2(e) past fp32's range
    (dict(table_stride=-1), SHAPE), (dict(table_stride=1 << 61), SHAPE),
    (dict(q_token=-16), SHAPE), (dict(q_head=264), ALIGN), (dict(o_token=8200), ALIGN),
    (dict(o_head=-256), SHAPE), (dict(q_token=1 << 60), SHAPE),
    (dict(q=A + 0x4000008), ALIGN), (dict(out=A + 0x5000008), ALIGN), (dict(page_table=A + 2), ALIGN),
    (dict(seq_lens=A + 2), ALIGN), (dict(cu_q=A + 2), ALIGN),
    (dict(cache_over=dict(head_dim=272, k_head=544, v_head=544, k_offset=4352, v_offset=4352)), SHAPE),
    (dict(cache_over=dict(page_size=1 << 31, num_slots=1 << 32)), SHAPE),
    (dict(cache_over=dict(num_slots=15)), SHAPE),                # not one page
])
def test_attention_refused(lib, over, status):
    assert attend(lib, **over) == status


SPLIT = dict(tokens=1, seqs=1, cu_q=None, max_pages=4096)   # one row over a long context


@cpu_only
def test_workspace_is_asked_for_and_checked(lib):
    need = lib.kvstore_attention_workspace(C.byref(attention_args(**SPLIT)), C.byref(cache()))
    assert need > 0 and need % 16 == 0
    # it depends on shapes alone
    bare = attention_args(**SPLIT, q=None, out=None, page_table=None, seq_lens=None, workspace=None)
    assert lib.kvstore_attention_workspace(C.byref(bare), C.byref(cache(k=None, v=None))) == need
    assert attend(lib, **SPLIT, workspace_bytes=need) == HIP
    assert attend(lib, **SPLIT, workspace_bytes=need - 1) == SHAPE
    assert attend(lib, **SPLIT, workspace=None) == NULL
    assert attend(lib, **SPLIT, workspace=A + 8) == ALIGN
    # calls that need none read none of it
    none = dict(tokens=1, seqs=1, cu_q=None, max_pages=1)
    assert lib.kvstore_attention_workspace(C.byref(attention_args(**none)), C.byref(cache())) == 0
    assert attend(lib, **none, workspace=None, workspace_bytes=0) == HIP
    # refused arguments have no workspace
    assert lib.kvstore_attention_workspace(C.byref(attention_args(q_heads=12)), C.byref(cache())) == SHAPE
    assert lib.kvstore_attention_workspace(None, C.byref(cache())) == NULL
    assert lib.kvstore_attention_workspace(C.byref(attention_args()), None) == NULL


@cpu_only
@pytest.mark.parametrize("tokens,seqs,pages,heads", [
    (1, 1, 1 << 20, 1), (65535, 65535, 8192, 8), (1 << 20, 1, 1 << 17, 8), (1 << 22, 1 << 22, 64, 8),
    (4096, 7, 100000, 64)])
def test_workspace_stays_in_bounds(lib, tokens, seqs, pages, heads):
    for cu in (None, A):
        if cu is None and tokens != seqs:
            continue
        args = attention_args(tokens=tokens, seqs=seqs, max_pages=pages, q_heads=2 * heads, cu_q=cu)
        need = lib.kvstore_attention_workspace(C.byref(args), C.byref(cache(num_heads=heads)))
        assert need == SHAPE or 0 <= need <= (1 << 30) + 16


@cpu_only
def test_empty_calls_launch_nothing(lib):
    assert rope(lib, batch=0, cache_over=dict(k=None), rows_over=dict(k=None)) == 0
    assert load(lib, batch=0, k_out=None) == 0
    assert attend(lib, tokens=0, q=None) == 0 and attend(lib, seqs=0, q=None) == 0
    assert rope(lib, batch=0, idx_dtype=2) == DTYPE and load(lib, batch=0, dst=7) == DTYPE
    assert lib.kvstore_rope_paged(None, None, 0, None, 0, 0, 0, 0, None, 0, 1, C.byref(cache()), None,
                                  None, 1, None) == NULL
    assert lib.kvstore_load_paged(None, None, 0, 1, None, 0, 0, None, 0, 0, 0, 1, None) == NULL
    assert lib.kvstore_attention_paged(None, None, None) == NULL
