"""Refusals of the paged-cache entry points on the host (CPU only: every check
comes before the first CUDA call), and the binding's own checks."""
import ctypes

import pytest

from sparse_attention_13_b200 import dsa

A = 1 << 20  # aligned, never dereferenced: the checks fail first


def _kv(**kw):
    d = dict(n_pages=4, page=64, n_kv=2, D=128, fmt=dsa.DSA_KV_E4M3, k=A, v=A, k_scale=A, v_scale=A, sum=A, sum_scale=A)
    d.update(kw)
    return dsa.PagedKVDesc(**d)


def _pb(**kw):
    d = dict(B=2, cu_q=A, start_pos=A, block_table=A, max_pages=4, total_q=8, max_Lq=4, max_Lk=200)
    d.update(kw)
    return dsa.PagedBatchDesc(**d)


def _append(kv=None, pb=None, **kw):
    d = dict(k=A, ks=256, v=A, vs=256, cos=A, sin=A, n_pos=256, rot=128, inter=0, q=A, qs=1024, n_h=8, q_out=A)
    d.update(kw)
    return dsa.lib().dsa_paged_append(ctypes.byref(kv or _kv()), ctypes.byref(pb or _pb()), d["k"], d["ks"], d["v"], d["vs"], d["cos"],
                                      d["sin"], d["n_pos"], d["rot"], d["inter"], d["q"], d["qs"], d["n_h"], d["q_out"], None)


def _topk(kv=None, pb=None, **kw):
    d = dict(q=A, n_h=8, inc=0, n_sel=4, first=1, last=1, sel=A)
    d.update(kw)
    return dsa.lib().dsa_page_topk(d["q"], d["n_h"], ctypes.byref(kv or _kv()), ctypes.byref(pb or _pb()), d["inc"], d["n_sel"], d["first"],
                                   d["last"], d["sel"], None)


def _attn(kv=None, pb=None, **kw):
    d = dict(q=A, n_h=8, inc=0, sel=None, n_sel=0, scale=1.0, out=A, lse=None, ws=A, wsb=1 << 40)
    d.update(kw)
    return dsa.lib().dsa_paged_attn(d["q"], d["n_h"], ctypes.byref(kv or _kv()), ctypes.byref(pb or _pb()), d["inc"], d["sel"], d["n_sel"],
                                    d["scale"], d["out"], d["lse"], d["ws"], d["wsb"], None)


INV, UNS, WS = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_ERR_WORKSPACE


@pytest.mark.parametrize("call", [_append, _topk, _attn])
@pytest.mark.parametrize("kv,pb,want", [
    (dict(k=None), {}, INV), (dict(v=A + 8), {}, INV), (dict(n_pages=0), {}, INV), (dict(n_kv=0), {}, INV),
    (dict(page=48), {}, UNS), (dict(page=256), {}, UNS), (dict(D=96), {}, UNS), (dict(fmt=7), {}, UNS),
    (dict(k_scale=None), {}, INV), (dict(fmt=dsa.DSA_KV_BF16), {}, INV), (dict(sum=None), {}, INV),
    (dict(n_kv=129), {}, UNS), (dict(n_pages=1 << 30, n_kv=4), {}, UNS),
    ({}, dict(B=0), INV), ({}, dict(cu_q=None), INV), ({}, dict(start_pos=A + 2), INV), ({}, dict(block_table=None), INV),
    ({}, dict(total_q=0), INV), ({}, dict(max_Lq=9), INV), ({}, dict(max_Lk=257), INV), ({}, dict(max_pages=0), INV),
    ({}, dict(max_Lk=(1 << 30) + 1, max_pages=1 << 25), UNS),
])
def test_descriptor_refusals(call, kv, pb, want):
    assert call(_kv(**kv), _pb(**pb)) == want
    assert dsa.lib().dsa_last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INV), (dict(v=A + 2), INV), (dict(ks=248), INV), (dict(vs=260), INV), (dict(q=None), INV), (dict(q_out=None), INV),
    (dict(qs=1000), INV), (dict(n_h=0), INV), (dict(rot=120), UNS), (dict(rot=144), UNS), (dict(rot=-16), UNS), (dict(inter=2), INV),
    (dict(cos=None), INV), (dict(n_pos=199), INV), (dict(qs=1032, q_out=A), INV),
])
def test_append_refusals(kw, want):
    assert _append(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INV), (dict(sel=None), INV), (dict(sel=A + 4), INV), (dict(n_h=7), INV), (dict(n_h=0), INV), (dict(inc=2), INV),
    (dict(n_sel=0), INV), (dict(last=0), INV), (dict(first=-1), INV), (dict(first=4), INV), (dict(n_sel=1025), UNS), (dict(n_h=258), UNS),
])
def test_topk_refusals(kw, want):
    assert _topk(**kw) == want
    assert _topk(kv=_kv(sum=None, sum_scale=None)) == INV


def test_topk_refuses_more_pages_than_it_can_hold():
    assert _topk(kv=_kv(page=16), pb=_pb(max_Lk=49152 * 16 + 1, max_pages=49153)) == UNS


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INV), (dict(out=None), INV), (dict(out=A + 2), INV), (dict(lse=A + 4), INV), (dict(n_h=7), INV), (dict(n_h=130), UNS),
    (dict(inc=-1), INV), (dict(n_sel=3), INV), (dict(sel=A), INV), (dict(sel=A, n_sel=1025), UNS), (dict(scale=0.0), INV),
    (dict(scale=-1.0), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(ws=None), WS), (dict(ws=A + 8), WS),
    (dict(wsb=0), WS),
])
def test_attention_refusals(kw, want):
    assert _attn(**kw) == want


def test_null_descriptors_and_workspace_query():
    lib = dsa.lib()
    kv, pb = _kv(), _pb()
    assert lib.dsa_paged_attn(A, 8, None, ctypes.byref(pb), 0, None, 0, 1.0, A, None, A, 1 << 40, None) == INV
    assert lib.dsa_check_paged(ctypes.byref(kv), ctypes.byref(pb), None, None) == INV
    assert lib.dsa_paged_attn_workspace(None, ctypes.byref(pb), 8, 0) == 0
    assert lib.dsa_paged_attn_workspace(ctypes.byref(kv), ctypes.byref(pb), 8, 0) >= 16
    assert lib.dsa_paged_attn_workspace(ctypes.byref(kv), ctypes.byref(pb), 0, 0) == 0


def test_the_binding_takes_cuda_tensors_only():
    import torch
    x = torch.zeros((2, 2, 64, 128), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        dsa.PagedKV(x, x)
    with pytest.raises(TypeError):
        dsa.PagedBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros((2, 4), dtype=torch.int32),
                       total_q=2, max_Lq=1, max_Lk=5)
    with pytest.raises(ValueError):
        dsa.PagedKV.empty(2, 64, 2, 128, fmt="int8", device="cpu")
