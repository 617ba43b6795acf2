"""Pointers that are not aligned to their elements are refused on the host, by every call around drafted
tokens (no GPU): a kernel's loads would fault on them."""
import ctypes

import pytest

import bit_asymmetric_kv_quantize_b200 as kivi
from test_draft_abi import ERR_ARG, P, cache, tree


def off(n):
    return ctypes.c_void_p(P.value + n)


@pytest.mark.parametrize("dtype,by", [(0, 1), (1, 1), (1, 2), (1, 3)])
@pytest.mark.parametrize("ragged", [False, True])
def test_tree(ragged, dtype, by):
    c, st = cache(ragged, dtype=dtype), (P if ragged else "none")
    for name in ("q", "k", "v", "out"):
        assert tree(c, st, **{name: off(by)}) == ERR_ARG, name


@pytest.mark.parametrize("dtype,by", [(0, 1), (1, 1), (1, 2)])
def test_commit(dtype, by):
    c = cache(True, dtype=dtype)
    for k, v in ((off(by), P), (P, off(by))):
        assert kivi.lib().kivi_ragged_tree_commit(ctypes.byref(c), P, k, v, 4, P, P, 3, None) == ERR_ARG


@pytest.mark.parametrize("dtype,by", [(0, 1), (1, 1), (1, 2)])
def test_read(dtype, by):
    for K, V in ((off(by), P), (P, off(by))):
        c = cache(dtype=dtype)
        assert kivi.lib().kivi_read_tokens(ctypes.byref(c), 0, 1, K, V, None) == ERR_ARG
        c = cache(True, dtype=dtype)
        assert kivi.lib().kivi_ragged_read_tokens(ctypes.byref(c), P, 0, 1, K, V, None) == ERR_ARG


@pytest.mark.parametrize("dtype,by", [(0, 1), (1, 2)])
def test_weights_of_projections(dtype, by):
    s = kivi.KiviRope(2, 3, 8, 2, 128, dtype, 64, 1, (ctypes.c_int * 4)(32), 0, 1e-6)
    for qw, kw in ((off(by), P), (P, off(by))):
        assert kivi.lib().kivi_qk_norm_rope(ctypes.byref(s), P, 1536, P, P, qw, kw, P, P, P, None) == ERR_ARG
