"""Refusals of the prompt-path entry points, on the CPU: shapes, types and devices in the binding,
pointers, strides, sizes and workspaces in the library (nothing reaches a device)."""
import ctypes
import re

import pytest
import torch

import memory_bounded_kv_b200 as kvb
from memory_bounded_kv_b200 import _lib

T, Hq, Hkv, d, N = 12, 8, 2, 64, 2
bf = torch.bfloat16


def args():
    return dict(q=torch.zeros(T, Hq, d, dtype=bf), k=torch.zeros(T, Hkv, d, dtype=bf), v=torch.zeros(T, Hkv, d, dtype=bf),
                log_beta=torch.zeros(T, Hkv), cu=torch.zeros(N + 1, dtype=torch.int32), o=torch.zeros(T, Hq, d, dtype=bf),
                lse=torch.zeros(T, Hq))


def grads():
    return dict(d_o=torch.zeros(T, Hq, d, dtype=bf), d_lse=None, dq=torch.zeros(T, Hq, d, dtype=bf),
                dk=torch.zeros(T, Hkv, d, dtype=bf), dv=torch.zeros(T, Hkv, d, dtype=bf), d_log_beta=torch.zeros(T, Hkv),
                workspace=torch.zeros(T * Hq * 600, dtype=torch.uint8))


@pytest.mark.parametrize("name,value,error", [
    ("q", torch.zeros(T, Hq, d), TypeError), ("q", torch.zeros(T, Hq * d, dtype=bf), ValueError),
    ("k", torch.zeros(T, Hkv, d + 8, dtype=bf), ValueError), ("v", torch.zeros(T - 1, Hkv, d, dtype=bf), ValueError),
    ("log_beta", torch.zeros(T, Hq), ValueError), ("log_beta", torch.zeros(T, Hkv, dtype=bf), TypeError),
    ("o", torch.zeros(T, Hq, d), TypeError), ("o", torch.zeros(T, Hkv, d, dtype=bf), ValueError),
    ("lse", torch.zeros(Hq, T), ValueError), ("cu", torch.zeros(N + 1, dtype=torch.int64), TypeError),
    ("cu", torch.zeros(0, dtype=torch.int32), ValueError), ("q", None, TypeError),
    ("o", None, TypeError), ("q", torch.zeros(T, Hq, d, dtype=bf), TypeError),          # CPU tensors come last
])
def test_forward_binding_refuses(name, value, error):
    a = dict(args(), **{name: value})
    with pytest.raises(error):
        kvb.kvb_prefill_attn(**a)
    with pytest.raises(error):
        kvb.kvb_prefill_attn_bwd(**a, **grads())


def test_binding_refuses_prefix_and_strides():
    with pytest.raises(ValueError, match="prefix_len"):
        kvb.kvb_prefill_attn(**args(), prefix_len=torch.zeros(N + 1, dtype=torch.int32))
    wide = torch.zeros(T, Hkv, 2 * d, dtype=bf)
    with pytest.raises(ValueError):   # innermost dim not contiguous
        kvb.kvb_prefill_attn(**dict(args(), k=wide[:, :, ::2]))
    with pytest.raises(ValueError, match="equal strides"):
        kvb.kvb_prefill_attn(**dict(args(), k=wide[:, :, :d]))


@pytest.mark.parametrize("name,value,error", [
    ("d_o", torch.zeros(T, Hq, d), TypeError), ("dq", torch.zeros(T, Hkv, d, dtype=bf), ValueError),
    ("dk", None, TypeError), ("dv", torch.zeros(T, Hkv, dtype=bf), ValueError),
    ("d_lse", torch.zeros(T, Hkv), ValueError), ("d_log_beta", None, ValueError),
    ("dq", torch.zeros(Hq, T, d, dtype=bf).transpose(0, 1), ValueError),
    ("workspace", torch.zeros(4), TypeError),
])
def test_backward_binding_refuses(name, value, error):
    with pytest.raises(error):
        kvb.kvb_prefill_attn_bwd(**args(), **dict(grads(), **{name: value}))


def test_backward_needs_lse():
    with pytest.raises(ValueError, match="lse"):
        kvb.kvb_prefill_attn_bwd(**dict(args(), lse=None), **grads())


def test_paged_bindings_refuse():
    pool = kvb.PagedPool(N, Hkv, d, 2, 4, True, device="cpu")
    cu, sm = torch.zeros(N + 1, dtype=torch.int32), torch.zeros(Hkv, T, dtype=torch.int32)
    ws = torch.zeros(1024, dtype=torch.uint8)
    for bad in (dict(cu=cu[:-1]), dict(slot_map=sm.t().contiguous()), dict(slot_map=sm[:, 0])):
        with pytest.raises(ValueError):
            kvb.kvb_paged_plan(**dict(dict(pool=pool, cu=cu, slot_map=sm, workspace=ws), **bad))
    for bad in (dict(pool=None), dict(cu=cu.long()), dict(workspace=torch.zeros(4)), dict()):
        with pytest.raises(TypeError):
            kvb.kvb_paged_plan(**dict(dict(pool=pool, cu=cu, slot_map=sm, workspace=ws), **bad))
    a = args()
    w = dict(pool=pool, k=a["k"], v=a["v"], log_beta=a["log_beta"], pos=torch.zeros(T, dtype=torch.int32), slot_map=sm)
    for bad in (dict(k=a["q"]), dict(log_beta=None), dict(pos=torch.zeros(T - 1, dtype=torch.int32)), dict(slot_map=sm[:, 1:])):
        with pytest.raises(ValueError):
            kvb.kvb_paged_write(**dict(w, **bad))
    for bad in (dict(v=a["v"].float()), dict(pos=torch.zeros(T)), dict()):
        with pytest.raises(TypeError):
            kvb.kvb_paged_write(**dict(w, **bad))


F = 1 << 20   # a 16-byte aligned non-null value; the host checks never dereference it


def c_args(**kw):
    a = dict(q=F, q_stride_t=Hq * d, q_stride_h=d, k=F, v=F, kv_stride_t=Hkv * d, kv_stride_h=d, log_beta=F, lb_stride_t=Hkv,
             lb_stride_h=1, cu=F, prefix_len=None, T=T, N=N, Hq=Hq, Hkv=Hkv, d=d, scale=0.0, softcap=0.0, o=F, lse=F)
    a.update(kw)
    return _lib.PrefillArgs(**a)


BAD = [dict(d=96), dict(Hq=6), dict(Hq=32), dict(Hkv=0), dict(T=-1), dict(T=(1 << 24) + 1), dict(N=-1), dict(N=8193),
       dict(q=None), dict(k=F + 2), dict(v=None), dict(cu=None), dict(o=F + 4), dict(log_beta=F + 2),
       dict(q_stride_t=Hq * d + 4), dict(q_stride_h=0), dict(kv_stride_t=-Hkv * d), dict(kv_stride_h=d - 8),
       dict(lb_stride_t=-1), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=2.0 ** -21), dict(scale=float("inf")),
       dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(softcap=1e-9)]


@pytest.mark.parametrize("bad", BAD)
def test_library_refuses(bad):
    L = _lib.lib()
    assert L.kvb_prefill_attn(ctypes.byref(c_args(**bad)), None) == _lib.KVB_EINVAL
    g = _lib.PrefillGrads(d_o=F, d_lse=None, dq=F, dk=F, dv=F, d_log_beta=F, workspace=F, workspace_bytes=1 << 40)
    assert L.kvb_prefill_attn_bwd(ctypes.byref(c_args(**bad)), ctypes.byref(g), None) == _lib.KVB_EINVAL


@pytest.mark.parametrize("bad", [dict(d_o=None), dict(dq=F + 8), dict(dk=None), dict(dv=None), dict(d_log_beta=None),
                                 dict(workspace=None), dict(workspace=F + 4), dict(workspace_bytes=_lib.lib().kvb_prefill_attn_bwd_workspace_bytes(T, Hq) - 1)])
def test_library_refuses_gradient_arguments(bad):
    g = dict(d_o=F, d_lse=None, dq=F, dk=F, dv=F, d_log_beta=F, workspace=F, workspace_bytes=1 << 30)
    L = _lib.lib()
    assert L.kvb_prefill_attn_bwd(ctypes.byref(c_args()), ctypes.byref(_lib.PrefillGrads(**dict(g, **bad))),
                                  None) == _lib.KVB_EINVAL
    assert L.kvb_prefill_attn_bwd(ctypes.byref(c_args(lse=None)), ctypes.byref(_lib.PrefillGrads(**g)),
                                  None) == _lib.KVB_EINVAL
    # without log_beta there is no d_log_beta
    assert L.kvb_prefill_attn_bwd(ctypes.byref(c_args(log_beta=None)), ctypes.byref(_lib.PrefillGrads(**g)),
                                  None) == _lib.KVB_EINVAL


def test_empty_calls_are_ok():
    L = _lib.lib()
    assert L.kvb_prefill_attn(ctypes.byref(c_args(N=0)), None) == _lib.KVB_OK
    assert L.kvb_prefill_attn(ctypes.byref(c_args(T=0)), None) == _lib.KVB_OK
    assert L.kvb_prefill_attn(None, None) == _lib.KVB_EINVAL
    assert L.kvb_prefill_attn_bwd_workspace_bytes(0, 4) == 0 and L.kvb_paged_plan_workspace_bytes(0, 1) == 0


def test_library_refuses_paged_arguments():
    L = _lib.lib()
    pc = dict(k_pages=F, v_pages=F, log_beta_pages=None, pos_pages=F, table=F, len=F, free_pages=F, free_count=F, B=2, Hkv=2,
              d=128, max_pages=4, num_pages=16)
    c = ctypes.byref(_lib.PagedCacheArgs(**pc))
    ws = L.kvb_paged_plan_workspace_bytes(2, 2)
    assert L.kvb_paged_plan(c, F, -1, F, 0, F, ws, None) == _lib.KVB_EINVAL
    assert L.kvb_paged_plan(c, None, 8, F, 0, F, ws, None) == _lib.KVB_EINVAL
    assert L.kvb_paged_plan(c, F, 8, None, 0, F, ws, None) == _lib.KVB_EINVAL
    assert L.kvb_paged_plan(c, F, 8, F, 0, F, ws - 1, None) == _lib.KVB_EINVAL
    assert L.kvb_paged_plan(c, F, 8, F, 0, F + 4, ws, None) == _lib.KVB_EINVAL
    assert L.kvb_paged_plan(ctypes.byref(_lib.PagedCacheArgs(**dict(pc, num_pages=0))), F, 8, F, 0, F, ws, None) == _lib.KVB_EINVAL
    for bad in ((F + 2, F, 256, 128, None), (F, F, 252, 128, None), (F, F, -256, 128, None), (F, F, 256, 128, F)):
        assert L.kvb_paged_write(c, bad[0], bad[1], bad[2], bad[3], bad[4], 2, 1, F, F, 8, None) == _lib.KVB_EINVAL
    assert L.kvb_paged_write(c, F, F, 256, 128, None, 0, 0, None, F, 8, None) == _lib.KVB_EINVAL
    assert L.kvb_paged_write(c, F, F, 256, 128, None, 0, 0, F, F, 0, None) == _lib.KVB_OK


@pytest.mark.parametrize("struct,mirror", [("kvb_prefill_args", _lib.PrefillArgs), ("kvb_prefill_grads", _lib.PrefillGrads)])
def test_structs_match_the_header(struct, mirror):
    import os
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kvb.h")).read()
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), src, re.S).group(1)
    names = []
    for decl in body.split(";"):
        decl = re.sub(r"^(const\s+)?\w+\s*\**\s*", "", decl.strip())
        names += [n.strip().lstrip("*") for n in decl.split(",") if n.strip()]
    assert names == [f[0] for f in mirror._fields_]


def test_packed_structs_have_the_mirrors_layout():
    """The binding packs the structs as bytes: field by field the same as the ctypes mirrors."""
    a = dict(q=1, q_stride_t=2, q_stride_h=3, k=4, v=5, kv_stride_t=6, kv_stride_h=7, log_beta=8, lb_stride_t=9, lb_stride_h=10,
             cu=11, prefix_len=12, T=13, N=14, Hq=15, Hkv=16, d=17, scale=0.5, softcap=2.0, o=18, lse=19)
    assert bytes(_lib.PrefillArgs(**a)) == _lib.PREFILL_ARGS.pack(*a.values())
    g = dict(d_o=1, d_lse=2, dq=3, dk=4, dv=5, d_log_beta=6, workspace=7, workspace_bytes=8)
    assert bytes(_lib.PrefillGrads(**g)) == _lib.PREFILL_GRADS.pack(*g.values())
    c = [n for n, _ in _lib.PagedCacheArgs._fields_]
    values = dict(zip(c, range(1, len(c) + 1)))
    assert bytes(_lib.PagedCacheArgs(**values)) == _lib.PAGED_CACHE.pack(*values.values())


def test_cache_prefill_refuses_before_it_changes_anything(monkeypatch):
    from memory_bounded_kv_b200 import cache as cache_mod
    monkeypatch.setattr(kvb, "kvb_paged_reset", lambda pool, stream=None: None)
    c = cache_mod.PagedKVCache(N, Hq, Hkv, d, max_pages=2, num_pages=8, M=64, device="cpu")
    called = []
    for f in ("kvb_prefill_attn", "kvb_paged_plan", "kvb_paged_write"):
        monkeypatch.setattr(kvb, f, lambda *a, _f=f, **k: called.append(_f))
    a = args()
    good = dict(q=a["q"], k=a["k"], v=a["v"], log_beta=a["log_beta"], cu=a["cu"], pos=torch.zeros(T, dtype=torch.int32), o=a["o"])
    for bad in (dict(log_beta=None), dict(pos=torch.zeros(T)), dict(pos=torch.zeros(T - 1, dtype=torch.int32)),
                dict(k=a["k"][:, :1]), dict(cu=a["cu"][:-1]), dict(q=a["k"])):
        with pytest.raises(ValueError):
            c.prefill(**dict(good, **bad))
    assert called == []
