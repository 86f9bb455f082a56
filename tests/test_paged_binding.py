"""Refusals of the tensor-level paged operators, with CPU tensors: shapes, types
and combinations are looked at before the tensors' device, so every call here
ends before the library, a correct one with "must be a GPU tensor"."""
import pytest
import torch

import fp8_kv_quantization_amd as kv

T, H, HQ, D, P, PAGES = 5, 2, 4, 64, 16, 3
BF16 = torch.bfloat16


def rows(heads=H, dtype=BF16, n=T):
    return torch.zeros(n, heads, D, dtype=dtype)


def caches(fmt="16", flat=False):
    shape = (PAGES * P, H, D) if flat else (PAGES, P, H, D)
    if fmt == "fp4":
        make = lambda: torch.zeros(*shape[:-1], D // 2, dtype=torch.uint8).view(torch.float4_e2m1fn_x2)
    else:
        dtype = {"16": BF16, "e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "u8": torch.uint8}[fmt]
        make = lambda: torch.zeros(shape, dtype=torch.uint8 if dtype.itemsize == 1 else dtype).view(dtype)
    return make(), make()


def scales(kind, flat=False):
    lead = (PAGES * P,) if flat else (PAGES, P)
    shape = {"token": lead, "head": lead + (H,), "block": lead + (H, D // 32)}[kind]
    return tuple(torch.zeros(shape, dtype=torch.uint8 if kind == "block" else torch.float32) for _ in range(2))


def rope_args(fmt="16", **over):
    kc, vc = caches(fmt)
    a = dict(k=rows(), v=rows(), k_cache=kc, v_cache=vc, cache_loc=torch.arange(T),
             positions=torch.arange(T), cos_sin=torch.zeros(8, D), page_size=P)
    if fmt == "fp4":
        a["k_scale_cache"], a["v_scale_cache"] = scales("block")
    a.update(over)
    return a


def load_args(fmt="16", **over):
    kc, vc = caches(fmt)
    a = dict(k_cache=kc, v_cache=vc, cache_loc=torch.arange(T), k_out=rows(), v_out=rows(), page_size=P)
    if fmt == "fp4":
        a["k_scale_cache"], a["v_scale_cache"] = scales("block")
    a.update(over)
    return a


def attention_args(fmt="16", **over):
    kc, vc = caches(fmt)
    a = dict(q=rows(HQ), k_cache=kc, v_cache=vc, page_table=torch.zeros(2, PAGES, dtype=torch.int32),
             seq_lens=torch.zeros(2, dtype=torch.int32), cu_q=torch.zeros(3, dtype=torch.int32), page_size=P)
    if fmt == "fp4":
        a["k_scale_cache"], a["v_scale_cache"] = scales("block")
    a.update(over)
    return a


CALLS = {"rope": (kv.store_kv_rope_paged, rope_args), "load": (kv.load_kv_paged, load_args),
         "attention": (kv.attention_paged, attention_args)}


def refused(call, error, text, fmt="16", **over):
    fn, make = CALLS[call]
    with pytest.raises(error, match=text):
        fn(**make(fmt, **over))


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("fmt", ["16", "e4m3fn", "e5m2", "u8", "fp4"])
def test_correct_calls_are_stopped_by_the_device_alone(call, fmt):
    refused(call, ValueError, "must be a GPU tensor", fmt)


def test_other_forms_that_are_correct():
    gpu = dict(error=ValueError, text="must be a GPU tensor")
    two_d = lambda heads: torch.zeros(T, heads * D, dtype=BF16)
    refused("rope", **gpu, k=two_d(H), v=two_d(H), q=two_d(HQ))
    refused("rope", **gpu, q=rows(HQ), q_out=rows(HQ), interleaved=True)
    refused("rope", **gpu, positions=None, cos_sin=None)
    refused("rope", **gpu, fmt="e4m3fn", inv_k_scale=torch.ones(1), inv_v_scale=torch.ones(()))
    kc, vc = caches("fp4", flat=True)
    ks, vs = scales("block", flat=True)
    refused("load", **gpu, k_cache=kc, v_cache=vc, k_scale_cache=ks, v_scale_cache=vs)
    for kind in ("token", "head"):
        ks, vs = scales(kind)
        refused("load", **gpu, fmt="e5m2", k_scale_cache=ks, v_scale_cache=vs)
        refused("attention", **gpu, fmt="e4m3fn", k_scale_cache=ks, v_scale_cache=vs)
    refused("attention", **gpu, cu_q=None, q=rows(HQ, n=2), out=rows(HQ, n=2))
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        kv.attention_paged_workspace(**attention_args())
    kc, vc = caches("fp4")
    ks, vs = scales("block")
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        kv.store_kv_fp4_paged(rows(), rows(), kc, vc, torch.arange(T), ks, vs, page_size=P)


@pytest.mark.parametrize("call", CALLS)
def test_caches_refused(call):
    kc, vc = caches()
    refused(call, TypeError, "k_cache must be a tensor", k_cache=None)
    refused(call, TypeError, "share one dtype", v_cache=caches("e4m3fn")[0])
    refused(call, ValueError, "page_size must be positive", page_size=0)
    refused(call, ValueError, "must not be negative", page_size=-16)
    refused(call, ValueError, "slots per page", page_size=8)
    refused(call, ValueError, "does not split", k_cache=kc.reshape(-1, H, D)[:40],
            v_cache=vc.reshape(-1, H, D)[:40])
    refused(call, ValueError, "3-D .* or 4-D", k_cache=kc[0, 0], v_cache=vc[0, 0])
    refused(call, ValueError, "shapes differ", v_cache=vc[:2])
    refused(call, ValueError, "dim stride must be 1", k_cache=torch.zeros(PAGES, P, H, 2 * D, dtype=BF16)[..., ::2])
    refused(call, TypeError, "go with rows of that type", k_cache=kc.half(), v_cache=vc.half())
    refused(call, TypeError, "none of the formats", k_cache=kc.float(), v_cache=vc.float())
    one = torch.ones(1)
    ks, vs = scales("token")
    bs, _ = scales("block")
    refused(call, ValueError, "both scale caches or neither", "e4m3fn", k_scale_cache=ks)
    refused(call, ValueError, "16-bit caches have no scales", k_scale_cache=ks, v_scale_cache=vs)
    refused(call, ValueError, "need k_scale_cache", "fp4", k_scale_cache=None, v_scale_cache=None)
    refused(call, TypeError, "uint8 or float8_e8m0fnu", "fp4", k_scale_cache=bs.float())
    refused(call, ValueError, "4-bit scale caches must be", "fp4", k_scale_cache=bs[..., :1])
    refused(call, ValueError, "cover the same slots", "fp4", k_scale_cache=bs[:2])
    if call == "rope":
        refused(call, ValueError, "takes inverse scales", "e4m3fn", k_scale_cache=ks, v_scale_cache=vs)
        refused(call, ValueError, "only FP8 caches", inv_k_scale=one)
        refused(call, TypeError, "one-element fp32", "e5m2", inv_k_scale=one.double())
        return
    refused(call, ValueError, "not both", "e4m3fn", k_scale=one, k_scale_cache=ks, v_scale_cache=vs)
    refused(call, ValueError, "16-bit caches have no scales", k_scale=one)
    refused(call, ValueError, "block scales, not tensor", "fp4", k_scale=one)
    refused(call, TypeError, "one-element fp32", "e5m2", k_scale=torch.ones(2))
    refused(call, TypeError, "must be float32", "e4m3fn", k_scale_cache=ks.double(), v_scale_cache=vs)
    refused(call, ValueError, "unsupported scale cache shape", "e4m3fn", k_scale_cache=ks[0], v_scale_cache=vs)
    refused(call, ValueError, "cover the same slots", "e4m3fn", k_scale_cache=ks[:2], v_scale_cache=vs)
    refused(call, ValueError, r"\[pages, page_size", "e4m3fn", k_scale_cache=ks[:, :8], v_scale_cache=vs)


def test_rope_rows_refused():
    refused("rope", TypeError, "bfloat16 or float16", k=rows(dtype=torch.float32))
    refused("rope", TypeError, "share one dtype", v=rows(dtype=torch.float16))
    refused("rope", TypeError, "share one dtype", q=rows(HQ, torch.float16))
    refused("rope", ValueError, "do not match heads/dim", k=rows(H + 1))
    refused("rope", ValueError, "row width", v=torch.zeros(T, D, dtype=BF16))
    refused("rope", ValueError, "rows are 2-D", k=torch.zeros(D, dtype=BF16))
    refused("rope", ValueError, "row dim stride", k=torch.zeros(T, H, 2 * D, dtype=BF16)[..., ::2])
    refused("rope", ValueError, "same tokens", v=rows(n=T - 1))
    refused("rope", ValueError, "one slot for each row", cache_loc=torch.arange(T - 1))
    refused("rope", TypeError, "int32 or int64", cache_loc=torch.zeros(T))
    refused("rope", TypeError, "int32 or int64", positions=torch.zeros(T))
    refused("rope", ValueError, "contiguous", positions=torch.arange(2 * T)[::2])
    refused("rope", ValueError, "contiguous", positions=torch.arange(T + 1))
    refused("rope", ValueError, "or neither", positions=None)
    refused("rope", ValueError, "or neither", cos_sin=None)
    refused("rope", TypeError, "cos_sin must be fp32", cos_sin=torch.zeros(8, D, dtype=BF16))
    refused("rope", TypeError, "cos_sin must be fp32", cos_sin=torch.zeros(D, 8).T)
    refused("rope", ValueError, "q_out without q", q_out=rows(HQ))
    refused("rope", ValueError, "of one dtype", q=rows(HQ), q_out=rows(HQ + 1))
    refused("rope", ValueError, "of one dtype", q=rows(HQ, n=T + 1))
    refused("rope", ValueError, "exceeds the cache", size_limit=PAGES * P + 1)
    refused("rope", ValueError, "must not be negative", size_limit=-1)
    with pytest.raises(TypeError, match="4-bit codes go into"):
        kv.store_kv_fp4_paged(rows(), rows(), *caches(), torch.arange(T), *scales("block"), page_size=P)


def test_load_rows_refused():
    refused("load", TypeError, "bfloat16 or float16", "e4m3fn", k_out=rows(dtype=torch.float32))
    refused("load", TypeError, "share one dtype", "e4m3fn", v_out=rows(dtype=torch.float16))
    refused("load", ValueError, "do not match heads/dim", k_out=rows(H + 1))
    refused("load", ValueError, "same rows", v_out=rows(n=T - 1))
    refused("load", ValueError, "one slot for each row", cache_loc=torch.arange(T + 1))
    refused("load", TypeError, "int32 or int64", cache_loc=torch.zeros(T, dtype=torch.int16))


def test_attention_rows_refused():
    refused("attention", TypeError, "bfloat16 or float16", q=rows(HQ, torch.float32))
    refused("attention", ValueError, "multiple of 2", q=rows(3))
    refused("attention", ValueError, "q must be", q=rows(HQ)[..., :48])
    refused("attention", ValueError, "q must be", q=torch.zeros(T, HQ * D, dtype=BF16))
    refused("attention", ValueError, "dim stride of 1", q=torch.zeros(T, HQ, 2 * D, dtype=BF16)[..., ::2])
    refused("attention", ValueError, r"page_table \[B, pages\]", seq_lens=torch.zeros(3, dtype=torch.int32))
    refused("attention", TypeError, "must be int32", seq_lens=torch.zeros(2, dtype=torch.int64))
    refused("attention", TypeError, "must be int32", page_table=torch.zeros(2, PAGES, dtype=torch.int64))
    refused("attention", TypeError, "must be int32", cu_q=torch.zeros(3, dtype=torch.int64))
    refused("attention", ValueError, "must be contiguous", seq_lens=torch.zeros(4, dtype=torch.int32)[::2])
    refused("attention", ValueError, "must be contiguous", page_table=torch.zeros(PAGES, 2, dtype=torch.int32).T)
    refused("attention", ValueError, "one token", cu_q=None)
    refused("attention", ValueError, r"\[B \+ 1\]", cu_q=torch.zeros(2, dtype=torch.int32))
    refused("attention", ValueError, "q's shape and dtype", out=rows(HQ, n=T + 1))
    refused("attention", ValueError, "q's shape and dtype", out=rows(HQ, torch.float16))
    for name in ("window", "sinks", "max_q", "max_len"):
        refused("attention", ValueError, "must not be negative", **{name: -1})
    refused("attention", TypeError, None, window="8")
    refused("attention", TypeError, None, sm_scale="1")
    refused("attention", TypeError, "page_table must be a tensor", page_table=[[0]])


def test_tensors_that_wait_for_a_gradient_are_refused():
    refused("attention", ValueError, "no backward pass", q=rows(HQ).requires_grad_())
    refused("rope", ValueError, "no backward pass", k=rows().requires_grad_())
    refused("rope", ValueError, "no backward pass", q=rows(HQ).requires_grad_())
    refused("load", ValueError, "no backward pass", v_out=rows().requires_grad_())
    with torch.no_grad():
        refused("attention", ValueError, "must be a GPU tensor", q=rows(HQ).requires_grad_())


def test_argument_counts():
    from fp8_kv_quantization_amd import _kvstore_torch as calls
    for name in ("store_kv_rope_paged", "load_kv_paged", "attention_paged"):
        with pytest.raises(TypeError, match="expected .* arguments"):
            getattr(calls, name)(None)
