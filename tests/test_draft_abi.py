"""The calls around drafted tokens refuse bad arguments on the host, before any launch (no GPU)."""
import ctypes

import pytest
import torch

import bit_asymmetric_kv_quantize_b200 as kivi
from bit_asymmetric_kv_quantize_b200 import KiviCacheC, KiviDims, KiviRope

ERR_ARG, ERR_UNSUPPORTED, ERR_STATE = 1, 2, 3
P = ctypes.c_void_p(0x5000)
ODD = ctypes.c_void_p(0x5008)


def cache(ragged=False, paged=False, **kw):
    d = dict(B=2, Hkv=4, D=128, bits=2, G=32, Gv=32, R=128, capacity=512, dtype=0, meta=0, k_out=0, v_out=0)
    d.update(kw)
    dims, c = KiviDims(*d.values()), KiviCacheC()
    ptrs = (ctypes.c_void_p * 8)(*[0x10000 * (i + 1) for i in range(8)])
    if paged:
        rc = kivi.lib().kivi_paged_cache_init(ctypes.byref(c), ctypes.byref(dims), ctypes.byref(ptrs), P, 3, 6)
    else:
        rc = kivi.lib().kivi_cache_init(ctypes.byref(c), ctypes.byref(dims), ctypes.byref(ptrs))
    assert rc == 0
    if dims.k_out:
        o = (ctypes.c_void_p * 4)(*[0x100000 * (i + 1) for i in range(4)])
        assert kivi.lib().kivi_cache_set_outliers(ctypes.byref(c), ctypes.byref(o)) == 0
    if ragged:
        c.n_q = -1
    else:
        c.n_q, c.r = 128, 5
    return c


def tree(c, state="none", **kw):
    a = dict(q=P, k=P, v=P, mask=P, N=4, Hq=8, scale=1.0, out=P, ws=P, nbytes=1 << 30, stream=None)
    a.update(kw)
    if state == "none":
        return kivi.lib().kivi_tree_decode(ctypes.byref(c), *a.values())
    return kivi.lib().kivi_ragged_tree_decode(ctypes.byref(c), state, *a.values())


@pytest.mark.parametrize("ragged", [False, True])
def test_tree_arguments(ragged):
    c, st = cache(ragged), (P if ragged else "none")
    for name in ("q", "k", "v", "mask", "out"):
        assert tree(c, st, **{name: None}) == ERR_ARG, name
    assert tree(c, st, mask=ctypes.c_void_p(0x5002)) == ERR_ARG
    assert tree(c, st, N=0) == ERR_ARG
    assert tree(c, st, N=-5) == ERR_ARG
    assert tree(c, st, N=257) == ERR_UNSUPPORTED
    assert tree(c, st, Hq=0) == ERR_ARG
    assert tree(c, st, Hq=6) == ERR_ARG
    assert tree(c, st, Hq=4 * 65) == ERR_UNSUPPORTED
    sparse = cache(ragged, k_out=1)
    assert tree(sparse, st) == ERR_UNSUPPORTED


def test_tree_wants_its_kind_of_cache():
    assert tree(cache(True)) == ERR_STATE
    assert tree(cache(paged=True)) == ERR_STATE
    assert tree(cache(False), P) == ERR_STATE
    assert tree(cache(True), None) == ERR_ARG
    assert tree(cache(True), ODD) == ERR_ARG


def test_tree_workspace_refusals():
    L, c = kivi.lib(), cache()
    for N, Hq in ((0, 8), (257, 8), (4, 0), (4, 6), (4, 4 * 65)):
        assert L.kivi_tree_workspace_bytes(ctypes.byref(c), N, Hq) == 0


def test_commit_arguments():
    def commit(c, st=P, k=P, v=P, N=4, path=P, count=P, most=3):
        return kivi.lib().kivi_ragged_tree_commit(ctypes.byref(c), st, k, v, N, path, count, most, None)
    c = cache(True)
    for kw in (dict(st=None), dict(st=ODD), dict(k=None), dict(v=None), dict(path=None), dict(count=None),
               dict(path=ctypes.c_void_p(0x5002)), dict(count=ctypes.c_void_p(0x5001)), dict(N=0), dict(most=0),
               dict(most=129)):
        assert commit(c, **kw) == ERR_ARG, kw
    assert commit(c, N=257) == ERR_UNSUPPORTED
    assert commit(cache(False)) == ERR_STATE
    assert commit(cache(paged=True)) == ERR_STATE  # not filled


def test_read_arguments():
    L = kivi.lib()

    def read(c, t0, T, K=P, V=P):
        return L.kivi_read_tokens(ctypes.byref(c), t0, T, K, V, None)

    def ragged(c, t0, T, st=P, K=P, V=P):
        return L.kivi_ragged_read_tokens(ctypes.byref(c), st, t0, T, K, V, None)
    c = cache()  # 133 tokens
    big = (1 << 63) - 1
    for t0, T in ((-1, 1), (0, -1), (0, 134), (133, 1), (134, 0), (big, big), (1, big)):
        assert read(c, t0, T) == ERR_ARG, (t0, T)
    assert read(c, 0, 1, K=None) == ERR_ARG and read(c, 0, 1, V=None) == ERR_ARG
    assert read(c, 133, 0, K=None, V=None) == 0
    assert read(cache(True), 0, 1) == ERR_STATE and read(cache(paged=True), 0, 1) == ERR_STATE
    r = cache(True)
    for t0, T in ((-1, 1), (0, -1), (0, 513), (512, 1), (big, big)):
        assert ragged(r, t0, T) == ERR_ARG, (t0, T)
    assert ragged(r, 0, 1, st=None) == ERR_ARG and ragged(r, 0, 1, st=ODD) == ERR_ARG
    assert ragged(r, 512, 0) == 0
    assert ragged(cache(), 0, 1) == ERR_STATE


def test_rope_arguments():
    def rope(shape=None, stride=12 * 128, **kw):
        s = dict(B=2, N=3, Hq=8, Hkv=2, D=128, dtype=0, rot=64, axes=2, sections=(20, 12), interleaved=0, eps=1e-6)
        s.update(shape or {})
        s["sections"] = (ctypes.c_int * 4)(*s["sections"])
        a = dict(qkv=P, stride=stride, pos=P, f=P, qw=P, kw=P, q=P, k=P, v=P, stream=None)
        a.update(kw)
        return kivi.lib().kivi_qk_norm_rope(ctypes.byref(KiviRope(*s.values())), *a.values())
    for name in ("qkv", "pos", "f", "q", "k", "v"):
        assert rope(**{name: None}) == ERR_ARG, name
    assert kivi.lib().kivi_qk_norm_rope(None, P, 1536, P, P, P, P, P, P, P, None) == ERR_ARG
    for name in ("qkv", "q", "k", "v"):
        assert rope(**{name: ODD}) == ERR_ARG, name
    for name in ("pos", "f"):
        assert rope(**{name: ctypes.c_void_p(0x5004)}) == ERR_ARG, name
    assert rope(qw=ctypes.c_void_p(0x5001)) == ERR_ARG
    for kw in (dict(B=0), dict(N=0), dict(Hq=0), dict(Hkv=0), dict(axes=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(sections=(20, 11)), dict(sections=(33, -1)), dict(sections=(32, 1))):
        assert rope(kw) == ERR_ARG, kw
    for kw in (dict(D=96), dict(dtype=2), dict(rot=72), dict(rot=8), dict(rot=144), dict(axes=5)):
        assert rope(kw) == ERR_UNSUPPORTED, kw
    assert rope(dict(Hq=1 << 20)) == ERR_UNSUPPORTED
    assert rope(dict(B=1 << 16, N=1 << 16)) == ERR_UNSUPPORTED
    assert rope(stride=12 * 128 - 8) == ERR_ARG
    assert rope(stride=12 * 128 + 4) == ERR_ARG


def test_rope_struct_matches_the_header():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "kivi.h")).read()
    end = text.index("} kivi_rope;")
    body = text[text.rindex("typedef struct {", 0, end):end]
    assert re.findall(r"\b(?:int|float)\s+(\w+)(?:\[4\])?;", body) == [f[0] for f in KiviRope._fields_]


def test_tree_mask():
    m = kivi.tree_mask(torch.tensor([[-1, 0, 0, 2], [-1, -1, 1, 2]]))
    assert m.tolist() == [[[1], [3], [5], [13]], [[1], [2], [6], [14]]]
    chain = kivi.tree_mask(torch.arange(-1, 69)[None])
    assert chain.shape == (1, 70, 3) and chain.dtype == torch.int32
    assert chain[0, 31].tolist() == [-1, 0, 0] and chain[0, 69].tolist() == [-1, -1, 63]
    for bad in ([[0]], [[-1, 1]], [[-2]], [[-1, 5]]):
        with pytest.raises(ValueError):
            kivi.tree_mask(torch.tensor(bad))
    with pytest.raises(ValueError):
        kivi.tree_mask(torch.tensor([-1, 0]))
