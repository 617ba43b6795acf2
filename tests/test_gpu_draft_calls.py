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
