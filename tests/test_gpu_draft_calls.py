"""What the Python calls around drafted tokens hold and refuse, beside their numbers."""
import gc
import weakref

import pytest
import torch

import bit_asymmetric_kv_quantize_b200 as kivi

pytestmark = pytest.mark.gpu


def filled(T=4000):
    c = kivi.KiviCache(1, 1, 64, 2, 4096, R=64)
    g = torch.Generator(device="cuda").manual_seed(T)
    c.prefill(*(torch.randn(1, 1, T, 64, generator=g, device="cuda").half() for _ in "kv"))
    return c, g


def tree_of(c, g, N):
    q, k, v = (torch.randn(1, 1, N, 64, generator=g, device="cuda").half() for _ in "qkv")
    return q, k, v, kivi.tree_mask((torch.arange(N) - 1)[None]).cuda(), 0.125


def test_outgrown_workspaces_are_given_back():
    """A larger tree takes a larger workspace; the one before it goes unless a captured graph has it."""
    c, g = filled()
    seen = []
    for N in (9, 30, 45):
        c.tree_decode(*tree_of(c, g, N))
        seen.append(weakref.ref(c._ws_tree))
    gc.collect()
    assert [s() is None for s in seen] == [True, True, False]
    small = tree_of(c, g, 100)
    out = torch.zeros_like(small[0])
    want = c.tree_decode(*small)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.tree_decode(*small, out=out)
    captured = weakref.ref(c._ws_tree)
    c.tree_decode(*tree_of(c, g, 128))
    gc.collect()
    assert captured() is not None and c._ws_tree is not captured()
    graph.replay()
    assert torch.equal(out, want)


def test_workspace_given_back_while_another_stream_uses_it():
    """An outgrown workspace is not handed out before the other stream's call is done with it."""
    c, g = filled()
    small, large = tree_of(c, g, 9), tree_of(c, g, 60)
    want = c.tree_decode(*small)
    c._ws_tree = None
    c.tree_decode(*small)  # the workspace of this stream
    size = c._ws_tree.numel()
    s = torch.cuda.Stream()
    spin = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x = spin
        for _ in range(40):  # keeps the stream busy while the host goes on
            x = x @ spin
        got = c.tree_decode(*small)
    c.tree_decode(*large)
    others = [torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(bool((o == 0xA5).all()) for o in others)


@pytest.mark.parametrize("t0,T", [(0, 1 << 40), (-1, 1), (0, -1), (4096, 1), (1 << 50, 1)])
def test_read_refuses_a_range_before_it_makes_room_for_it(t0, T):
    c, _ = filled()
    before = torch.cuda.memory_allocated()
    with pytest.raises(kivi.KiviError):
        c.read_tokens(t0, T)
    r = kivi.KiviCache(1, 1, 64, 2, 4096, R=64)
    x = torch.zeros(1, 1, 100, 64, dtype=torch.float16, device="cuda")
    st = r.ragged_prefill(x, x, torch.tensor([100], device="cuda"))
    with pytest.raises(kivi.KiviError):
        r.ragged_read_tokens(st, t0, T)
    del r, x, st
    assert torch.cuda.memory_allocated() == before


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_cache_that_is_all_window(dtype):
    """capacity == R: no store, and no flush that could have room."""
    R, D = 32, 64
    c = kivi.KiviCache(2, 2, D, 2, R, R=R, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    K, V = (torch.randn(2, 2, 30, D, generator=g, device="cuda").to(dtype) for _ in "kv")
    st = c.ragged_prefill(K, V, torch.tensor([30, 7], device="cuda"))
    k, v = (torch.randn(2, 2, 4, D, generator=g, device="cuda").to(dtype) for _ in "kv")
    q = torch.randn(2, 4, 4, D, generator=g, device="cuda").to(dtype)
    mask = kivi.tree_mask((torch.arange(4) - 1).expand(2, 4)).cuda()
    see = torch.tril(torch.ones(4, 4, dtype=torch.bool))
    out = c.ragged_tree_decode(st, q, k, v, mask, 0.125).cpu().double()
    for b, n in ((0, 30), (1, 7)):
        for h in range(4):
            ks = torch.cat([K[b, h // 2, :n], k[b, h // 2]]).cpu().double()
            vs = torch.cat([V[b, h // 2, :n], v[b, h // 2]]).cpu().double()
            s = q[b, h].cpu().double() @ ks.T * 0.125
            s = s.masked_fill(torch.cat([torch.zeros(4, n).bool(), ~see], 1), -float("inf"))
            ref = torch.softmax(s, -1) @ vs
            # raw keys and values lose nothing, weights and the output are rounded to the type:
            # 2 half steps of sum p |V| (numerator and denominator), one of the output, and the
            # binary32 sums of D and n products
            half = torch.finfo(dtype).eps / 2
            A = torch.softmax(s, -1) @ vs.abs()
            top = (q[b, h].cpu().double().abs() @ ks.abs().T).amax(1, keepdim=True) * 0.125
            tol = 2 * (half + (2 * top * (D + 8) + 140 + n) * 2.0 ** -24) * A + half * ref.abs() + 2.0 ** -25
            assert ((out[b, h] - ref).abs() <= tol).all()
    path = torch.arange(4, dtype=torch.int32, device="cuda").expand(2, 4).contiguous()
    c.ragged_tree_commit(st, k, v, path, torch.tensor([3, 4], dtype=torch.int32, device="cuda"))
    assert kivi.ragged_lengths(st) == ([0, 0], [30, 11], [1, 0])
    Kr, Vr = c.ragged_read_tokens(st, 0, R)
    assert (Kr[0] == 0).all() and torch.equal(Kr[1, :, 7:11], k[1]) and torch.equal(Vr[1, :, :7], V[1, :, :7])
