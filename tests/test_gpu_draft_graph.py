"""A whole drafted step captured once and replayed, against the same calls made one by one."""
import pytest
import torch

import bit_asymmetric_kv_quantize_b200 as kivi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("store,dtype", [("ragged", torch.float16), ("paged", torch.float16),
                                         ("ragged", torch.float32)])
@pytest.mark.parametrize("N", [6, 40])
def test_captured_step_is_the_eager_one(store, dtype, N):
    """Projections -> tree -> commit -> decode -> read-back in one graph over two caches that take turns
    on its workspaces; positions, counts and paths change in place between replays, flushes included."""
    B, Hq, Hkv, D, R, P = 5, 8, 2, 64, 32, 6
    g = torch.Generator(device="cuda").manual_seed(N)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    lens = [40, 1, 300, 64, 31]
    K, V = rnd(B, Hkv, 300, D), rnd(B, Hkv, 300, D)
    f = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    w = torch.ones(D, dtype=dtype, device="cuda")
    mask = kivi.tree_mask((torch.arange(N) - 2).clamp(min=-1).expand(B, N)).cuda()

    def fill():
        if store == "paged":
            pages = 20
            bt = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(pages, B).T.contiguous()
            c = kivi.PagedKiviCache(B, Hkv, D, 2, pages, B * pages, bt, R=R, dtype=dtype)
        else:
            c = kivi.KiviCache(B, Hkv, D, 2, 640, R=R, dtype=dtype)
        return c, c.ragged_prefill(K, V, torch.tensor(lens, device="cuda"))

    qkv, pos = rnd(B, N, (Hq + 2 * Hkv) * D), torch.zeros(B, N, dtype=torch.int64, device="cuda")
    path = torch.zeros(B, P, dtype=torch.int32, device="cuda")
    count = torch.zeros(B, dtype=torch.int32, device="cuda")

    def step(c, st):
        q, k, v = kivi.qk_norm_rope(qkv, pos, f, Hq, Hkv, q_weight=w, k_weight=w)
        out = c.ragged_tree_decode(st, q, k, v, mask, 0.125)
        c.ragged_tree_commit(st, k, v, path, count)
        after = c.ragged_decode(st, q[:, :, 0].contiguous(), 0.125)
        return out, after, *c.ragged_read_tokens(st, 250, 150)

    eager, graphed = [fill(), fill()], [fill(), fill()]
    for c, st in graphed:  # what a first call makes is made
        step(c, st.clone())
    fresh = [fill() for _ in graphed]
    for (c, st), (d, s) in zip(graphed, fresh):
        st.copy_(s)
        for n in c.buffers:
            c.buffers[n].copy_(d.buffers[n])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [step(c, st) for c, st in graphed]
    for i in range(12):
        qkv.copy_(rnd(*qkv.shape))
        pos.copy_(torch.randint(0, 100000, pos.shape, generator=g, device="cuda"))
        path.copy_(torch.randint(0, N, path.shape, generator=g, device="cuda"))
        count.copy_(torch.randint(0, P + 1, count.shape, generator=g, device="cuda"))
        graph.replay()
        for (c, st), mine, (d, s) in zip(eager, got, graphed):
            for x, y in zip(step(c, st), mine):
                assert torch.equal(x, y), i
            assert torch.equal(st, s)
    assert kivi.ragged_lengths(eager[0][1])[2] == [0] * B
