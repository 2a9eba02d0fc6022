"""Refusals of the tree, mass and eviction calls: a bad argument gives a status and a message
and nothing is launched or written."""
import ctypes as C

import numpy as np
import pytest
import torch

from packed_cache_decode_b200 import binding as B


def test_calls_before_upload_report_device(lib):
    lay = B.Layout(np.full(64, 2), 2, 0)
    h = lay.handle
    assert lib.bgtq_tree_attention(h, None, 0, 1, 1, 1, 1, None, None, None, None, 64, 64, 0.1, None, 0, None, 0,
                                   None) == B.ERR_DEVICE
    assert lib.bgtq_tree_attention_paged(h, None, 0, 1, 1, 1, 1, None, None, None, 1, None, 1, None, 64, 0.1, None, 0,
                                         None, 0, None) == B.ERR_DEVICE
    assert lib.bgtq_tree_commit(h, None, 1, None, None, 1, 1, 1, None, None, None, 64, None) == B.ERR_DEVICE
    assert lib.bgtq_tree_commit_paged(h, None, 1, None, None, 1, 1, 1, None, 1, None, 1, None, None, None) == B.ERR_DEVICE
    assert lib.bgtq_decode_attention_mass(h, None, 0, 1, 1, 1, None, None, 64, 64, 0.1, 1.0, None, 64, None, 0, None, 0,
                                          None) == B.ERR_DEVICE
    assert lib.bgtq_cache_evict(h, 1, 1, None, 64, None, 64, None, 64, 1, 0, 0, None, 64, None, 64, None, None,
                                None) == B.ERR_DEVICE
    assert lib.bgtq_tree_attention(None, None, 0, 1, 1, 1, 1, None, None, None, None, 64, 64, 0.1, None, 0, None, 0,
                                   None) == B.ERR_INVALID
    for bad in ((0, 8, 2, 4, 64), (1, 7, 2, 4, 64), (1, 66, 2, 4, 64), (1, 8, 2, 0, 64), (1, 8, 2, 65, 64), (1, 8, 2, 4, -1)):
        assert lib.bgtq_tree_workspace_bytes(h, *bad) == 0
    assert lib.bgtq_mass_workspace_bytes(h, 1, 7, 2, 64) == 0


def _ptr(t):
    return C.c_void_p(t.data_ptr())


@pytest.mark.gpu
def test_tree_refusals(lib):
    lay = B.Layout(np.full(64, 2), 2, 0).upload(0)
    z = dict(dtype=torch.int32, device="cuda")
    q, out = torch.zeros(1, 4, 8, 128, device="cuda"), torch.full((1, 4, 8, 128), 5.0, device="cuda")
    mask, lens = torch.ones(1, 4, dtype=torch.int64, device="cuda"), torch.full((1,), 64, **z)
    cache = torch.zeros(lay.cache_bytes(1, 2, 128) + 16, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(B.tree_workspace_bytes(lay, 1, 8, 2, 4, 128) + 16, dtype=torch.uint8, device="cuda")

    def call(q=_ptr(q), qt=0, b=1, n=4, hq=8, hkv=2, mask=_ptr(mask), cache=_ptr(cache), lens=_ptr(lens), cap=128, most=128,
             scale=0.1, out=_ptr(out), ot=0, ws=_ptr(ws), nb=ws.numel()):
        return lib.bgtq_tree_attention(lay.handle, q, qt, b, n, hq, hkv, mask, None, cache, lens, cap, most, scale, out, ot,
                                       ws, nb, None)

    for kw, want in (({"q": None}, B.ERR_INVALID), ({"qt": 3}, B.ERR_INVALID), ({"ot": -1}, B.ERR_INVALID),
                     ({"b": 0}, B.ERR_INVALID), ({"n": 0}, B.ERR_INVALID), ({"n": 65}, B.ERR_INVALID),
                     ({"hq": 7}, B.ERR_INVALID), ({"hq": 66}, B.ERR_INVALID), ({"mask": None}, B.ERR_INVALID),
                     ({"cache": None}, B.ERR_INVALID), ({"lens": None}, B.ERR_INVALID), ({"out": None}, B.ERR_INVALID),
                     ({"cap": 100}, B.ERR_CAPACITY), ({"most": 129}, B.ERR_CAPACITY), ({"most": -1}, B.ERR_CAPACITY),
                     ({"scale": float("nan")}, B.ERR_INVALID), ({"ws": None}, B.ERR_WORKSPACE),
                     ({"nb": 100}, B.ERR_WORKSPACE),
                     ({"cache": C.c_void_p(cache.data_ptr() + 8)}, B.ERR_INVALID),
                     ({"ws": C.c_void_p(ws.data_ptr() + 16)}, B.ERR_WORKSPACE)):
        assert call(**kw) == want or (kw == {"most": -1} and call(**kw) == B.ERR_INVALID), kw
        assert lib.bgtq_last_error_string()
    path, cnt, new = torch.zeros(1, 4, **z), torch.zeros(1, **z), torch.zeros(1, **z)

    def commit(path=_ptr(path), ld=4, cnt=_ptr(cnt), n=4, b=1, hkv=2, cache=_ptr(cache), lens=_ptr(lens), new=_ptr(new),
               cap=128):
        return lib.bgtq_tree_commit(lay.handle, path, ld, cnt, None, n, b, hkv, cache, lens, new, cap, None)

    for kw, want in (({"path": None}, B.ERR_INVALID), ({"ld": 3}, B.ERR_INVALID), ({"cnt": None}, B.ERR_INVALID),
                     ({"n": 0}, B.ERR_INVALID), ({"n": 65}, B.ERR_INVALID), ({"b": 0}, B.ERR_INVALID),
                     ({"hkv": 0}, B.ERR_INVALID), ({"cache": None}, B.ERR_INVALID), ({"lens": None}, B.ERR_INVALID),
                     ({"new": None}, B.ERR_INVALID), ({"new": _ptr(lens)}, B.ERR_INVALID), ({"cap": 0}, B.ERR_CAPACITY),
                     ({"cache": C.c_void_p(cache.data_ptr() + 4)}, B.ERR_INVALID)):
        assert commit(**kw) == want, kw
    torch.cuda.synchronize()
    assert (out == 5).all() and (cache == 0).all() and lay.status() == 0


@pytest.mark.gpu
def test_mass_and_evict_refusals(lib):
    lay = B.Layout(np.full(64, 2), 2, 0).upload(0)
    z = dict(dtype=torch.int32, device="cuda")
    q, out = torch.zeros(1, 8, 128, device="cuda"), torch.full((1, 8, 128), 5.0, device="cuda")
    lens, mass = torch.full((1,), 64, **z), torch.zeros(1, 2, 128, device="cuda")
    cache = torch.zeros(lay.cache_bytes(1, 2, 128), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(B.mass_workspace_bytes(lay, 1, 8, 2, 128), dtype=torch.uint8, device="cuda")

    def call(mass=_ptr(mass), ld=128, decay=1.0, ot=0, nb=ws.numel(), out=_ptr(out), most=128, hq=8, ws=_ptr(ws)):
        return lib.bgtq_decode_attention_mass(lay.handle, _ptr(q), 0, 1, hq, 2, _ptr(cache), _ptr(lens), 128, most, 0.1,
                                              decay, mass, ld, out, ot, ws, nb, None)

    for kw, want in (({"mass": None}, B.ERR_INVALID), ({"ld": 127}, B.ERR_INVALID), ({"decay": float("inf")}, B.ERR_INVALID),
                     ({"ot": 7}, B.ERR_INVALID), ({"nb": ws.numel() - 1}, B.ERR_WORKSPACE), ({"out": None}, B.ERR_INVALID),
                     ({"most": 200}, B.ERR_CAPACITY), ({"hq": 9}, B.ERR_INVALID), ({"ws": None}, B.ERR_WORKSPACE)):
        assert call(**kw) == want, kw
    dst = torch.full((lay.cache_bytes(1, 2, 64),), 9, dtype=torch.uint8, device="cuda")
    mo, kept, new = torch.zeros(1, 2, 32, device="cuda"), torch.zeros(1, 2, 32, **z), torch.zeros(1, **z)

    def evict(src=_ptr(cache), cap=128, lens=_ptr(lens), most=128, mass=_ptr(mass), ld=128, keep=32, sink=2, recent=4,
              dst=_ptr(dst), dcap=64, mo=_ptr(mo), mold=32, kept=_ptr(kept), new=_ptr(new), b=1, hkv=2):
        return lib.bgtq_cache_evict(lay.handle, b, hkv, src, cap, lens, most, mass, ld, keep, sink, recent, dst, dcap, mo,
                                    mold, kept, new, None)

    for kw, want in (({"src": None}, B.ERR_INVALID), ({"cap": 65}, B.ERR_CAPACITY), ({"most": 129}, B.ERR_CAPACITY),
                     ({"lens": None}, B.ERR_INVALID), ({"mass": None}, B.ERR_INVALID), ({"ld": 100}, B.ERR_INVALID),
                     ({"keep": 0}, B.ERR_INVALID), ({"sink": -1}, B.ERR_INVALID), ({"recent": -1}, B.ERR_INVALID),
                     ({"sink": 30}, B.ERR_INVALID), ({"dst": None}, B.ERR_INVALID), ({"dcap": 63}, B.ERR_CAPACITY),
                     ({"keep": 65}, B.ERR_CAPACITY), ({"mo": None}, B.ERR_INVALID), ({"mold": 31}, B.ERR_INVALID),
                     ({"kept": None}, B.ERR_INVALID), ({"new": None}, B.ERR_INVALID), ({"new": _ptr(lens)}, B.ERR_INVALID),
                     ({"mo": _ptr(mass)}, B.ERR_INVALID), ({"dst": _ptr(cache)}, B.ERR_INVALID), ({"b": 0}, B.ERR_INVALID),
                     ({"b": 40000}, B.ERR_INVALID)):
        assert evict(**kw) == want, kw
    torch.cuda.synchronize()
    assert (out == 5).all() and (dst == 9).all() and (mass == 0).all() and lay.status() == 0
