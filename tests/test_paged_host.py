"""Refusals of the rotary and paged entry points that need no GPU: the C ABI checks its arguments before
it touches the device, and the Python binding refuses host tensors."""
import ctypes

import pytest
import torch

import attention_attn_fwd_10_b200 as attn
from attention_attn_fwd_10_b200 import _abi, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def _cache(**kw):
    a = dict(k=0x1000, v=0x2000, e4m3=0, n_pages=4, page_size=16, H_kv=2, D=64, page_stride=2048, token_stride=128,
             head_stride=64, k_scale=1.0, v_scale=1.0, page_table=0x3000, table_stride=4, max_pages=4, seq_len=0x4000,
             q_start=0x5000, n_seq=1)
    a.update(kw)
    return _abi.PagedKVStruct(**a)


BAD_CACHE = [
    (dict(k=0), 1), (dict(v=None), 1), (dict(page_table=0), 1), (dict(seq_len=0), 1), (dict(q_start=0), 1),
    (dict(n_pages=0), 1), (dict(H_kv=0), 1), (dict(max_pages=0), 1), (dict(n_seq=0), 1), (dict(page_size=8), 1),
    (dict(page_size=24), 1), (dict(D=96), 2), (dict(e4m3=2), 1), (dict(k_scale=0.0), 1), (dict(v_scale=float("nan")), 1),
    (dict(k_scale=2.0), 1), (dict(table_stride=3), 1), (dict(max_pages=2 ** 28, table_stride=2 ** 28), 2),
    (dict(k=0x1008), 3), (dict(v=0x2002), 3), (dict(seq_len=0x4001), 3), (dict(token_stride=132), 3),
    (dict(head_stride=0), 1), (dict(page_stride=1024), 1), (dict(token_stride=64), 1), (dict(page_stride=-2048), 1),
    (dict(e4m3=1, token_stride=136), 3), (dict(token_stride=64, head_stride=512), 1),
]


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_cache_refusals(lib, kw, code):
    c = _cache(**kw)
    assert lib.attn_fwd_paged(ctypes.byref(c), 16, 32, 48, 64, 1, 4, 256, 0, 1, 0.125, None) == code
    assert lib.attn_paged_append(ctypes.byref(c), None, 16, 32, None, 1, 0, 0, 128, 128, None, None) == code


def test_other_layouts_pass_the_checks(lib):
    # zero tokens: nothing to do, and no device is needed
    for kw in (dict(), dict(token_stride=64, head_stride=1024), dict(page_stride=4096), dict(e4m3=1, k_scale=0.5),
               dict(n_pages=1, page_stride=0), dict(H_kv=1, head_stride=0, token_stride=64)):
        c = _cache(**kw)
        assert lib.attn_fwd_paged(ctypes.byref(c), 16, 32, 48, 64, 0, 4, 256, 0, 1, 0.125, None) == 0
        assert lib.attn_paged_append(ctypes.byref(c), None, 16, 32, None, 0, 0, 0, 128, 128, None, None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(o=0), 1), (dict(lse=0), 1), (dict(ws=0), 1), (dict(T=-1), 1), (dict(H_q=3), 1), (dict(H_q=0), 1),
    (dict(stride=248), 1), (dict(stride=260), 1), (dict(max_new=-1), 1), (dict(causal=2), 1), (dict(scale=0.0), 1),
    (dict(scale=float("inf")), 1), (dict(H_q=258, stride=258 * 64), 2), (dict(q=24), 3), (dict(ws=40), 3), (dict(ws=48), 3), (dict(lse=36), 3)])
def test_attend_refusals(lib, kw, code):
    a = dict(q=16, o=32, lse=48, ws=64, T=1, H_q=4, stride=256, max_new=0, causal=1, scale=0.125)
    a.update(kw)
    c = _cache()
    assert lib.attn_fwd_paged(ctypes.byref(c), a["q"], a["o"], a["lse"], a["ws"], a["T"], a["H_q"], a["stride"], a["max_new"],
                              a["causal"], a["scale"], None) == code
    assert lib.attn_fwd_paged(None, a["q"], a["o"], a["lse"], a["ws"], a["T"], a["H_q"], a["stride"], 0, 1, 0.125, None) == 1


@pytest.mark.parametrize("scale,k_scale,code", [(1e30, 1e10, 1), (3e38, 1.5, 1), (2.5e38, 1.0, 1), (2.3e38, 1.0, 0), (1e-30, 1e30, 0)])
def test_scales_whose_product_overflows_are_refused(lib, scale, k_scale, code):
    # scale * k_scale * log2(e) is held in 32 bits: infinite, it would make NaN of a score of 0
    c = _cache(e4m3=1, k_scale=k_scale)
    assert lib.attn_fwd_paged(ctypes.byref(c), 16, 32, 48, 64, 0, 4, 256, 0, 1, scale, None) == code


def _rotary(**kw):
    a = dict(inv_freq=0x6000, positions=0x7000, n_freq=32, n_axes=1, section=(ctypes.c_int * 4)(32, 0, 0, 0), interleaved=0)
    a.update(kw)
    return _abi.RotaryStruct(**a)


BAD_ROTARY = [
    (dict(inv_freq=0), 1), (dict(n_freq=0), 1), (dict(n_freq=6), 1), (dict(n_freq=36), 1), (dict(n_axes=0), 1),
    (dict(n_axes=5), 1), (dict(interleaved=2), 1), (dict(section=(ctypes.c_int * 4)(28, 0, 0, 0)), 1),
    (dict(n_axes=2, section=(ctypes.c_int * 4)(40, -8, 0, 0)), 1), (dict(inv_freq=0x6001), 3), (dict(positions=0x7002), 3),
    (dict(n_axes=2, positions=None), 1)]


@pytest.mark.parametrize("kw,code", BAD_ROTARY)
def test_rotary_refusals(lib, kw, code):
    r = _rotary(**kw)
    assert lib.attn_rope(16, 32, 48, 64, 4, 4, 2, 64, 256, 128, 256, 128, 4, ctypes.byref(r), 0, None) == code
    c = _cache()
    assert lib.attn_paged_append(ctypes.byref(c), 16, 32, 48, 64, 1, 4, 256, 128, 128, ctypes.byref(r), None) == code


@pytest.mark.parametrize("args,code", [
    ((0, 32, 48, 64, 4, 4, 2, 64, 256, 128, 256, 128, 4), 1), ((16, 32, 0, 64, 4, 4, 2, 64, 256, 128, 256, 128, 4), 1),
    ((16, 32, 48, 0, 4, 4, 2, 64, 256, 128, 256, 128, 4), 1), ((16, 32, 48, 64, -1, 4, 2, 64, 256, 128, 256, 128, 4), 1),
    ((16, 32, 48, 64, 4, 0, 2, 64, 256, 128, 256, 128, 4), 1), ((16, 32, 48, 64, 4, 4, 0, 64, 256, 128, 256, 128, 4), 1),
    ((16, 32, 48, 64, 4, 4, 2, 80, 320, 160, 320, 160, 4), 2), ((16, 32, 48, 64, 4, 4, 2, 64, 248, 128, 256, 128, 4), 1),
    ((16, 32, 48, 64, 4, 4, 2, 64, 256, 0, 256, 128, 4), 1), ((16, 32, 16, 64, 4, 4, 2, 64, 512, 128, 256, 128, 4), 1),
    ((24, 32, 48, 64, 4, 4, 2, 64, 256, 128, 256, 128, 4), 3), ((16, 32, 48, 72, 4, 4, 2, 64, 256, 128, 256, 128, 4), 3)])
def test_rope_refusals(lib, args, code):
    assert lib.attn_rope(*args, ctypes.byref(_rotary()), 0, None) == code


def test_rope_needs_a_period_without_positions(lib):
    r = _rotary(positions=None)
    assert lib.attn_rope(16, None, 48, None, 4, 4, 0, 64, 256, 0, 256, 0, 0, ctypes.byref(r), 0, None) == 1
    assert lib.attn_rope(16, None, 48, None, 0, 4, 0, 64, 256, 0, 256, 0, 1, ctypes.byref(r), 0, None) == 0
    assert lib.attn_rope(16, None, 48, None, 0, 4, 0, 64, 256, 0, 256, 0, 1, ctypes.byref(r), 2, None) == 1


def test_append_refusals(lib):
    c, r = _cache(), _rotary()

    def call(q=16, k=32, v=48, q_out=64, T=1, H_q=4, qs=256, ks=128, vs=128, rot=True):
        return lib.attn_paged_append(ctypes.byref(c), q, k, v, q_out, T, H_q, qs, ks, vs, ctypes.byref(r) if rot else None, None)

    for kw, code in ((dict(k=0), 1), (dict(v=0), 1), (dict(q_out=0), 1), (dict(rot=False), 1), (dict(ks=64), 1), (dict(vs=132), 1),
                     (dict(qs=128), 1), (dict(H_q=0), 1), (dict(q=16, q_out=16, qs=512), 1), (dict(k=40), 3), (dict(q=24), 3),
                     (dict(T=-1), 1)):
        assert call(**kw) == code, kw
    assert call(T=0) == 0


def test_workspace_size(lib):
    assert lib.attn_fwd_paged_workspace_size(32, 8, 128) > 0
    for bad in ((0, 8, 128), (32, 0, 128), (33, 8, 128), (32, 8, 96), (129, 1, 64)):
        assert lib.attn_fwd_paged_workspace_size(*bad) == 0


def test_host_tensors_are_refused():
    bf = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    i32 = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        attn.PagedKV(bf, bf.clone(), i32, i32[0, :1], i32[0])
    with pytest.raises(ValueError, match="CUDA"):
        attn.Rotary(torch.ones(32))
    with pytest.raises(ValueError, match="float32"):
        attn.Rotary(torch.ones(32, dtype=torch.float64))
