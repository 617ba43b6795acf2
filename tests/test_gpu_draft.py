"""The operators around drafted tokens on the GPU, against 64-bit plain implementations
(draft_testlib): attention of a tree over the cache, commit of accepted paths, read-back, and the
normed and turned projections."""
import ctypes
import math

import pytest
import torch

import bit_asymmetric_kv_quantize_b200 as kivi
from draft_testlib import assert_tree, fills, rope_reference, tokens, tree_reference

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, dtype, *shape, by=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * by).to(dtype)


def make_cache(seed, B, Hkv, D, bits, lens, R=32, dtype=torch.float16, meta=torch.float32,
               store="uniform", room=2, outliers=(0, 0)):
    """A filled cache and its state (None for host counters); lens: an int, or one per sequence."""
    g = gen(seed)
    ragged = store != "uniform"
    lens = [lens] * B if isinstance(lens, int) else list(lens)
    T = max(lens + [1])
    big = torch.ones(Hkv, 1, D, device="cuda")
    big[:, :, torch.randperm(D, generator=g, device="cuda")[:3]] = 20.0
    K = (torch.randn(B, Hkv, T, D, generator=g, device="cuda") * big).to(dtype)
    V = rnd(g, dtype, B, Hkv, T, D)
    pages = (T - 1) // R + room
    if store == "paged":
        bt = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages)
        c = kivi.PagedKiviCache(B, Hkv, D, bits, pages, B * pages, bt.contiguous(), R=R, dtype=dtype,
                                meta=meta)
    else:
        c = kivi.KiviCache(B, Hkv, D, bits, (pages + 1) * R, R=R, dtype=dtype, meta=meta,
                           outliers=outliers)
    for b in c.buffers.values():
        b.fill_(0xFF)  # what no call has written is NaN
    if ragged:
        return c, c.ragged_prefill(K, V, torch.tensor(lens, device="cuda"))
    if T and lens[0]:
        c.prefill(K, V)
    return c, None


def draft(seed, c, gq, N):
    g = gen(seed + 1)
    return (rnd(g, c.dtype, c.B, c.Hkv * gq, N, c.D, by=1.5), rnd(g, c.dtype, c.B, c.Hkv, N, c.D, by=2.0),
            rnd(g, c.dtype, c.B, c.Hkv, N, c.D))


def random_tree(seed, B, N):
    g = torch.Generator()
    g.manual_seed(seed)
    p = torch.arange(N) - torch.randint(1, 5, (B, N), generator=g)
    return kivi.tree_mask(p.clamp(min=-1)).cuda()


def tree(c, st, q, k, v, mask, scale, out=None):
    if st is None:
        return c.tree_decode(q, k, v, mask, scale, out=out)
    return c.ragged_tree_decode(st, q, k, v, mask, scale, out=out)


def check_tree(c, st, gq, N, seed=7, scale=None, mask=None):
    q, k, v = draft(seed, c, gq, N)
    mask = random_tree(seed, c.B, N) if mask is None else mask
    scale = 1 / math.sqrt(c.D) if scale is None else scale
    got = tree(c, st, q, k, v, mask, scale)
    assert_tree(got, tree_reference(c, st, q, k, v, mask, scale))


# ---- attention of a tree ------------------------------------------------------------------------


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("bits", [1, 2, 3, 4])
@pytest.mark.parametrize("kind", ["f16", "f16-meta16", "f32"])
def test_tree_every_format(D, bits, kind):
    dtype = torch.float32 if kind == "f32" else torch.float16
    meta = torch.float16 if kind == "f16-meta16" else torch.float32
    c, st = make_cache(D + bits, 2, 2, D, bits, 231, dtype=dtype, meta=meta)
    check_tree(c, st, 2, 7)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("T", [0, 1, 31, 32, 33, 64, 65, 96, 97, 128, 129, 160, 161, 700])
def test_tree_every_end(T, dtype):
    c, st = make_cache(T, 2, 1, 64, 2, T, R=64, dtype=dtype)
    check_tree(c, st, 4, 5)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("gq,N", [(1, 1), (8, 1), (1, 15), (1, 16), (1, 17), (2, 32), (1, 33), (4, 31),
                                  (8, 16), (1, 64), (1, 65), (2, 64), (1, 127), (1, 128), (1, 129),
                                  (8, 40), (1, 256), (2, 200), (3, 7),
                                  (5, 13), (64, 3)])
def test_tree_every_row_count(gq, N, dtype):
    c, st = make_cache(N, 1, 2, 64, 4, 150, dtype=dtype)
    check_tree(c, st, gq, N)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("store", ["ragged", "paged"])
@pytest.mark.parametrize("R", [32, 96, 128])
def test_tree_ragged(store, R, dtype):
    lens = [1, 700, 2, R, R + 1, 64, 333]
    c, st = make_cache(R, len(lens), 2, 128, 2, lens, R=R, dtype=dtype, store=store)
    check_tree(c, st, 2, 21)


def test_tree_many_sequences():
    lens = [(37 * i) % 200 + 1 for i in range(75)]
    c, st = make_cache(5, 75, 1, 32, 2, lens, store="ragged")
    check_tree(c, st, 1, 3)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_tree_long_cache_few_heads(dtype):
    """One group, split over all CTAs and joined."""
    c, st = make_cache(11, 1, 1, 128, 2, 20011, R=128, dtype=dtype)
    check_tree(c, st, 1, 9)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_tree_masks(dtype):
    """Causal chains, rows that see nothing of the draft, everything, and any pattern."""
    for T in (0, 40):
        c, st = make_cache(3, 2, 2, 64, 2, T, dtype=dtype)
        N = 40
        low = torch.tril(torch.ones(N, N, dtype=torch.bool)).expand(2, N, N).clone()
        low[0, 5] = False
        low[1, :] = False
        rand = torch.rand(2, N, N) < 0.2
        for see in (low, torch.ones(2, N, N, dtype=torch.bool), rand):
            w = torch.zeros(2, N, 64, dtype=torch.int64)
            w[:, :, :N] = see
            w[:, :, N:] = 1  # bits behind the last node are ignored
            words = (w.view(2, N, 2, 32) << torch.arange(32)).sum(-1)
            words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).cuda()
            check_tree(c, st, 2, N, mask=words)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_tree_masked_places_hold_anything(dtype, value):
    """A node's result is the same whatever stands in drafted tokens that it does not see; the
    nodes that see them get what the definition gives."""
    c, st = make_cache(4, 2, 2, 64, 2, 70, dtype=dtype)
    N = 12
    q, k, v = draft(9, c, 2, N)
    parents = torch.full((2, N), -1)
    parents[:, 1:] = torch.arange(N - 1)
    parents[:, 4] = -1  # 4 .. 11 do not see 0 .. 3
    mask = kivi.tree_mask(parents).cuda()
    clean = tree(c, st, q, k, v, mask, 0.1)
    for what in ("k", "v", "both"):
        k2, v2 = k.clone(), v.clone()
        if what != "v":
            k2[:, :, 2] = value
        if what != "k":
            v2[:, :, 2, ::3] = value
        got = tree(c, st, q, k2, v2, mask, 0.1)
        assert torch.equal(got[:, :, 4:], clean[:, :, 4:]), what
        assert torch.equal(got[:, :, :2], clean[:, :, :2]), what
        if what == "v":
            bad = got[:, :, 2:4, ::3]
            assert (torch.isnan(bad) if math.isnan(value) else bad == value).all()
            rest = torch.ones(c.D, dtype=torch.bool)
            rest[::3] = False
            assert torch.equal(got[:, :, 2:4][..., rest], clean[:, :, 2:4][..., rest])


def test_tree_large_scores():
    """Scores far apart: weights underflow, the running maximum jumps from tile to tile."""
    for dtype in (torch.float16, torch.float32):
        c, st = make_cache(6, 1, 2, 64, 4, 500, dtype=dtype)
        check_tree(c, st, 2, 6, scale=30.0)
        check_tree(c, st, 2, 6, scale=-1.0)
        check_tree(c, st, 2, 6, scale=0.0)


def test_tree_many_small_weights_beside_a_large_one():
    """One token far above thousands that follow it, each 2^-25 of its weight: together they count.
    The score between them, 25 ln 2 = 17.33, is off by 17.33 * 2^-11 = 0.0085 (its key is rounded to
    binary16), so a weight that stands in binary16 at 2^-21 or above lies within 0.85 % of a whole
    number of its steps of 2^-24 and is rounded to that; the output is rounded to binary16
    (2^-11), the scores are as in tree_reference (3 * 2^-17 * 17.33): within 1 % in all."""
    for dtype in (torch.float16, torch.float32):
        B, Hkv, D, T = 8, 8, 32, 4096
        c = kivi.KiviCache(B, Hkv, D, 2, T + 32, R=32, dtype=dtype)
        K = torch.zeros(B, Hkv, T, D, device="cuda", dtype=dtype)
        K[:, :, 0] = 25 * math.log(2) / D
        V = torch.full_like(K, 64.0)
        V[:, :, 0] = 0
        c.prefill(K, V)
        q = torch.ones(B, Hkv, 3, D, device="cuda", dtype=dtype)
        none = torch.zeros(B, 3, 1, dtype=torch.int32, device="cuda")
        out = c.tree_decode(q, q, q, none, 1.0)
        ref, _ = tree_reference(c, None, q, q, q, none, 1.0)
        assert ((out.cpu().double() - ref).abs() <= 0.01 * ref).all()


@pytest.mark.parametrize("N", [3, 80])
def test_tree_long_sums_do_not_drift(N):
    """Equal weights (powers of two, so exact) over a long cache whose values are spread around zero:
    the mean is small beside the codes' products, and cuts toward zero at each step of a sum would
    pull it down.  Off by at most, with c' s + z' a stored value and c' its code about the
    center: half a step of the output; 2^-17 of |c' s| for the two parts of s; and for the sums of
    c' s (two parts), of z' and of the weights 2^-23 of the largest partial sum at each of their
    n / 16 steps."""
    B, D, T = 32 if N == 80 else 64, 32, 16384
    c, st = make_cache(17, B, 2, D, 2, T, R=32)
    c.view("k_codes").zero_()
    for n in ("k_scale", "k_zero", "k_res"):
        c.view(n).zero_()
    q, k, v = draft(1, c, 1, N)
    none = torch.zeros(B, N, (N + 31) // 32, dtype=torch.int32, device="cuda")
    out = c.tree_decode(q, k, v, none, 1.0).cpu().double()
    for b in (0, B // 2 - 1, B - 1):
        _, V = tokens(c, b, c.n_q, c.r)
        z = torch.zeros_like(V)
        z[:, : c.n_q] = (c.view("v_zero")[b].double() + 1.5 * c.view("v_scale")[b].double())[:, : c.n_q].cpu()
        ref = V.mean(1)
        steps = T / 16 * 2.0 ** -23
        tol = (2.0 ** -11 * ref.abs() + 2.0 ** -17 * (V - z).abs().mean(1)
               + steps * ref.abs() + 2 * steps * (V - z).cumsum(1).abs().amax(1) / T
               + steps * z.cumsum(1).abs().amax(1) / T)
        assert ((out[b] - ref[:, None]).abs() <= tol[:, None]).all()


def test_tree_refused_sequences_give_nan():
    lens = [40, 300, 200]
    c, st = make_cache(8, 3, 2, 64, 2, lens, store="paged")
    c.block_table[1, 3] = 999  # a page of sequence 1 outside the pool
    st2 = st.clone()
    st2.view(torch.int64).view(3, 2)[2, 0] = 33  # no fill of a cache
    q, k, v = draft(3, c, 1, 4)
    mask = random_tree(3, 3, 4)
    got = tree(c, st2, q, k, v, mask, 0.2)
    assert torch.isnan(got[1:]).all()
    c.block_table[1, 3] = 0
    ref = tree(c, st, q, k, v, mask, 0.2)
    assert torch.equal(got[0], ref[0]) and torch.isfinite(ref).all()


def test_tree_unaligned_tensors():
    for dtype in (torch.float16, torch.float32):
        c, st = make_cache(2, 2, 2, 32, 2, 100, dtype=dtype)
        q, k, v = draft(2, c, 2, 6)

        def off(t):
            big = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            big[1:] = t.reshape(-1)
            return big[1:].view(t.shape)
        mask = random_tree(2, 2, 6)
        want = tree(c, st, q, k, v, mask, 0.3)
        out = off(torch.zeros_like(q))
        got = tree(c, st, off(q), off(k), off(v), mask, 0.3, out=out)
        assert got is out and torch.equal(got, want)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_tree_is_the_same_each_time_and_in_graphs(dtype):
    """No atomics order results; one workspace serves two captured graphs and eager calls."""
    c, st = make_cache(12, 3, 2, 128, 2, [900, 33, 400], dtype=dtype, store="ragged")
    q, k, v = draft(5, c, 4, 9)
    q2, k2, v2 = draft(50, c, 1, 20)
    m1, m2 = random_tree(1, 3, 9), random_tree(2, 3, 20)
    w1, w2 = tree(c, st, q, k, v, m1, 0.1), tree(c, st, q2, k2, v2, m2, 0.1)
    o1, o2 = torch.zeros_like(q), torch.zeros_like(q2)
    torch.cuda.synchronize()
    graphs = []
    for args, o in (((q, k, v, m1), o1), ((q2, k2, v2, m2), o2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tree(c, st, *args, 0.1, out=o)
        graphs.append(g)
    for _ in range(3):
        o1.zero_()
        o2.zero_()
        graphs[0].replay()
        graphs[1].replay()
        e = tree(c, st, q, k, v, m1, 0.1)
        assert torch.equal(o1, w1) and torch.equal(o2, w2) and torch.equal(e, w1)
    # the state is read at each replay
    st2 = st.clone()
    st.view(torch.int32).view(3, 4)[:, 3] = 1
    graphs[0].replay()
    assert torch.isnan(o1).all()
    st.copy_(st2)
    graphs[0].replay()
    assert torch.equal(o1, w1)


def test_tree_workspace_of_a_captured_graph_stays():
    """A later call with a larger tree takes a larger workspace; a graph captured before it still
    writes its partials into its own."""
    c, st = make_cache(12, 1, 1, 64, 2, 4000)
    q, k, v = draft(5, c, 1, 9)
    m = random_tree(1, 1, 9)
    want = tree(c, st, q, k, v, m, 0.1)
    out = torch.zeros_like(q)
    size = c._ws_tree.numel()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tree(c, st, q, k, v, m, 0.1, out=out)
    check_tree(c, st, 1, 60)
    others = [torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(4)]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(bool((o == 0xA5).all()) for o in others)


def test_tree_on_another_stream():
    c, st = make_cache(13, 2, 2, 64, 2, 300)
    q, k, v = draft(5, c, 2, 9)
    m = random_tree(1, 2, 9)
    want = tree(c, st, q, k, v, m, 0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = tree(c, st, q, k, v, m, 0.1)
    s.synchronize()
    assert torch.equal(got, want)


def test_tree_calls_at_once_on_two_streams():
    """Two caches, trees of both block forms under way together: neither result changes."""
    work = []
    for seed, N in ((31, 20), (32, 90), (33, 5)):
        c, st = make_cache(seed, 4, 8, 32, 2, 3000)
        q, k, v = draft(seed, c, 1, N)
        m = random_tree(seed, 4, N)
        work.append((c, st, q, k, v, m, tree(c, st, q, k, v, m, 0.2), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[] for _ in work]
    for _ in range(10):
        for (c, st, q, k, v, m, _, s), g in zip(work, got):
            with torch.cuda.stream(s):
                g.append(tree(c, st, q, k, v, m, 0.2))
    torch.cuda.synchronize()
    for w, g in zip(work, got):
        assert all(torch.equal(x, w[6]) for x in g)


def test_tree_of_one_node_is_append_and_decode():
    """A chain of one node is the next token: the result of kivi_append_decode, within both bars."""
    c, st = make_cache(14, 2, 4, 128, 2, 600, R=128)
    q, k, v = draft(6, c, 2, 1)
    one = torch.ones(2, 1, 1, dtype=torch.int32, device="cuda")
    got = tree(c, st, q, k, v, one, 0.05)
    want = c.append_decode(k[:, :, 0].contiguous(), v[:, :, 0].contiguous(), q[:, :, 0].contiguous(), 0.05)
    assert (got[:, :, 0].float() - want.float()).abs().max() <= 2e-3 + 2e-3


# ---- commit -----------------------------------------------------------------------------------


def copies(seed, store, B, Hkv, D, bits, lens, **kw):
    """The batch, and each of its sequences as a batch of its own, filled alike."""
    c, st = make_cache(seed, B, Hkv, D, bits, lens, store=store, **kw)
    ones = []
    g = gen(seed)
    T = max(lens)
    big = torch.ones(Hkv, 1, D, device="cuda")
    big[:, :, torch.randperm(D, generator=g, device="cuda")[:3]] = 20.0
    K = (torch.randn(B, Hkv, T, D, generator=g, device="cuda") * big).to(c.dtype)
    V = rnd(g, c.dtype, B, Hkv, T, D)
    for b in range(B):
        o = kivi.KiviCache(1, Hkv, D, bits, c.capacity, R=c.R, dtype=c.dtype, meta=c.meta,
                           outliers=c.__dict__.get("outliers", (0, 0)))
        for x in o.buffers.values():
            x.fill_(0xFF)
        s = o.ragged_prefill(K[b:b + 1].contiguous(), V[b:b + 1].contiguous(),
                             torch.tensor([lens[b]], device="cuda"))
        ones.append((o, s))
    return c, st, ones


def assert_same_cache(c, st, ones):
    got = kivi.ragged_lengths(st)
    for b, (o, s) in enumerate(ones):
        n_q, r, status = (x[0] for x in kivi.ragged_lengths(s))
        assert (got[0][b], got[1][b], got[2][b]) == (n_q, r, status), b
        for n in kivi.BUFFER_NAMES + (("k_out_idx", "k_out_val", "v_out_idx", "v_out_val")
                                      if o.outliers != (0, 0) else ()):
            a, w = c.view(n), o.view(n)[0]
            if hasattr(c, "block_table") and not n.endswith("_res"):
                pages = c.block_table[b, : n_q // c.R].long()
                a = torch.cat(list(a[pages]), 1) if len(pages) else a[0][:, :0]
                w = w[:, : a.shape[1]]
            else:
                a = a[b]
            assert torch.equal(a.contiguous().view(torch.uint8), w.contiguous().view(torch.uint8)), (b, n)


@pytest.mark.parametrize("store", ["ragged", "paged"])
@pytest.mark.parametrize("D,bits,kind", [(32, 1, "f32"), (64, 2, "f16"), (128, 2, "f16"), (128, 3, "f32"),
                                         (64, 4, "m16"), (128, 3, "m16"), (32, 4, "f16"), (128, 1, "f16")])
def test_commit_equals_appends(D, bits, kind, store):
    dtype = torch.float32 if kind == "f32" else torch.float16
    meta = torch.float16 if kind == "m16" else torch.float32
    R, N, P = 64, 40, 33
    lens = [1, 64, 63, 130, 100, 32, 95, 128]
    counts = [0, 1, 1, 33, 28, 33, 33, 2]
    c, st, ones = copies(D + bits, store, len(lens), 2, D, bits, lens, R=R, dtype=dtype, meta=meta, room=4)
    assert_same_cache(c, st, ones)
    for step in range(3):
        _, k, v = draft(step, c, 1, N)
        g = torch.Generator()
        g.manual_seed(step)
        path = torch.randint(0, N, (len(lens), P), generator=g)  # the same node twice among them
        for b, m in enumerate(counts):
            path[b, m:] = -7  # not read
        c.ragged_tree_commit(st, k, v, path.to(torch.int32).cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda"))
        for b, (o, s) in enumerate(ones):
            for i in range(counts[b]):
                o.ragged_append(s, k[b:b + 1, :, path[b, i]].contiguous(), v[b:b + 1, :, path[b, i]].contiguous())
        assert_same_cache(c, st, ones)


def test_commit_with_outlier_lists():
    lens, counts = [64, 50], [3, 20]
    c, st, ones = copies(3, "ragged", 2, 2, 64, 2, lens, R=64, room=3, outliers=(1, 2))
    _, k, v = draft(0, c, 1, 24)
    path = torch.arange(24).flip(0).expand(2, 24).to(torch.int32).contiguous().cuda()
    c.ragged_tree_commit(st, k, v, path, torch.tensor(counts, dtype=torch.int32, device="cuda"))
    for b, (o, s) in enumerate(ones):
        for i in range(counts[b]):
            n = int(path[b, i])
            o.ragged_append(s, k[b:b + 1, :, n].contiguous(), v[b:b + 1, :, n].contiguous())
    assert_same_cache(c, st, ones)


def test_commit_refusals_touch_only_their_sequence():
    """A count or a node out of range, no room, a page outside the pool: status 1 and nothing else."""
    R, N, P = 32, 8, 8
    lens = [30, 30, 30, 30, 96, 30, 30]
    c, st = make_cache(1, 7, 2, 64, 2, lens, R=R, store="paged", room=0)  # capacity 3 pages of tokens
    assert c.capacity == 96
    c.block_table[5, 0] = -1
    before = {n: b.clone() for n, b in c.buffers.items()}
    _, k, v = draft(0, c, 1, N)
    path = torch.arange(8).expand(7, 8).clone()
    path[1, 2] = 8
    path[2, 0] = -1
    counts = [9, 3, 1, -1, 1, 5, 4]
    c.ragged_tree_commit(st, k, v, path.to(torch.int32).cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda"))
    n_q, r, status = kivi.ragged_lengths(st)
    assert status == [1, 1, 1, 1, 1, 1, 0] and (n_q[6], r[6]) == (32, 2)
    assert (n_q[:6], r[:6]) == ([0, 0, 0, 0, 64, 0], [30, 30, 30, 30, 32, 30])
    for n in ("k_res", "v_res"):
        old = before[n].view(c.dtype).view(c.view(n).shape) if before[n].numel() else None
        assert torch.equal(c.view(n)[:6].view(torch.uint8), old[:6].view(torch.uint8))
    page = int(c.block_table[6, 0])
    for n in kivi.BUFFER_NAMES[:6]:
        was = before[n].view(c.view(n).dtype).view(c.view(n).shape)
        for p in range(c.num_pages):
            if p != page:
                assert torch.equal(c.view(n)[p].view(torch.uint8), was[p].view(torch.uint8)), (n, p)
    # a refused sequence takes nothing afterwards either
    ok = torch.ones(7, dtype=torch.int32, device="cuda")
    c.ragged_tree_commit(st, k, v, torch.zeros(7, 8, dtype=torch.int32, device="cuda"), ok)
    assert kivi.ragged_lengths(st)[1] == [30, 30, 30, 30, 32, 30, 3]


def test_commit_captured_and_unaligned():
    c, st, ones = copies(9, "ragged", 2, 2, 32, 2, [40, 60], R=32, room=6)
    _, k, v = draft(0, c, 1, 5)
    big = torch.empty(k.numel() + 1, dtype=k.dtype, device="cuda")
    big[1:] = k.reshape(-1)
    ku = big[1:].view(k.shape)
    path = torch.tensor([[4, 0, 2], [1, 1, 3]], dtype=torch.int32, device="cuda")
    count = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.ragged_tree_commit(st, ku, v, path, count)
    for _ in range(25):
        g.replay()
        for b, (o, s) in enumerate(ones):
            for i in range(int(count[b])):
                n = int(path[b, i])
                o.ragged_append(s, k[b:b + 1, :, n].contiguous(), v[b:b + 1, :, n].contiguous())
    assert_same_cache(c, st, ones)


# ---- read-back ----------------------------------------------------------------------------------


def check_read(c, st, t0, T, K=None, V=None):
    fill = [x.clone() if x is not None else torch.zeros(c.B, c.Hkv, T, c.D, dtype=c.dtype) for x in (K, V)]
    got = c.read_tokens(t0, T, K=K, V=V) if st is None else c.ragged_read_tokens(st, t0, T, K=K, V=V)
    # c s + z rounded to binary32 (half a step of 2^-24 relative), then to the cache's type
    half = torch.finfo(c.dtype).eps / 2 + 2.0 ** -24
    for b, (n_q, r, status) in enumerate(fills(c, st)):
        ref = tokens(c, b, n_q, r) if not status else (torch.zeros(c.Hkv, 0, c.D),) * 2
        for x, y, was in zip(got, ref, fill):
            y = y[:, t0:t0 + T]
            x = x[b].cpu()
            assert ((x[:, : y.shape[1]].double() - y).abs() <= half * y.abs() + 2.0 ** -25).all()
            assert torch.equal(x[:, y.shape[1]:], was[b].cpu()[:, y.shape[1]:])


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("bits", [1, 2, 3, 4])
@pytest.mark.parametrize("kind", ["f16", "f16-meta16", "f32"])
def test_read_every_format(D, bits, kind):
    dtype = torch.float32 if kind == "f32" else torch.float16
    meta = torch.float16 if kind == "f16-meta16" else torch.float32
    c, st = make_cache(D + bits, 2, 3, D, bits, 231, R=64, dtype=dtype, meta=meta)
    for t0, T in ((0, 231), (0, 1), (230, 1), (191, 2), (33, 60), (5, 0), (231, 0)):
        check_read(c, st, t0, T)


@pytest.mark.parametrize("store", ["ragged", "paged"])
def test_read_ragged_leaves_what_is_not_there(store):
    lens = [1, 300, 64, 65, 130]
    c, st = make_cache(2, 5, 2, 64, 2, lens, R=64, store=store, room=3)
    st.view(torch.int32).view(5, 4)[4, 3] = 1  # refused
    for t0, T in ((0, c.capacity), (60, 10), (299, 20), (c.capacity - 1, 1), (c.capacity, 0)):
        K = torch.full((5, 2, T, 64), 7.0, dtype=c.dtype, device="cuda")
        check_read(c, st, t0, T, K=K, V=K.clone() * 2)


def test_read_page_outside_the_pool():
    c, st = make_cache(2, 2, 2, 64, 4, [200, 100], R=32, store="paged")
    c.block_table[0, 2] = c.num_pages
    K, V = c.ragged_read_tokens(st, 0, 200)
    assert (K[0, :, 64:96] == 0).all() and (V[0, :, 64:96] == 0).all()
    assert (K[0, :, 96:] != 0).any() and (K[0, :, :64] != 0).any()


def test_read_outlier_lists_and_unaligned():
    c, st = make_cache(2, 2, 2, 64, 2, 200, R=32, outliers=(2, 3))
    check_read(c, st, 3, 190)
    for dtype in (torch.float16, torch.float32):
        c, st = make_cache(2, 2, 2, 32, 3, 100, dtype=dtype)
        want = c.read_tokens(1, 99)
        K, V = (torch.empty(want[0].numel() + 1, dtype=dtype, device="cuda")[1:].view(want[0].shape) for _ in "kv")
        got = c.read_tokens(1, 99, K=K, V=V)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_read_after_prefill_requantizes_to_the_same_cache():
    """What is read back quantizes to the same codes: a group's numbers hit its own grid (up to the
    group's own scale, so codes are compared, not scales)."""
    c, _ = make_cache(2, 2, 2, 64, 2, 129, R=32, dtype=torch.float32)
    K, V = c.read_tokens(0, 129)
    d = kivi.KiviCache(2, 2, 64, 2, c.capacity, R=32, dtype=torch.float32)
    d.prefill(K, V)
    for n in ("k_codes", "v_codes"):
        rows = c.n_q if n == "k_codes" else c.n_q // 16
        assert torch.equal(c.view(n)[:, :, :rows], d.view(n)[:, :, :rows])


# ---- projections ----------------------------------------------------------------------------------


def check_rope(dtype, B, N, Hq, Hkv, D, rot, axes=1, interleaved=False, norm="both", start=0, pad=0, seed=1):
    g = gen(seed)
    width = (Hq + 2 * Hkv) * D
    qkv = rnd(g, dtype, B, N, width + pad, by=3.0)[:, :, :width]
    pos = torch.randint(start, start + 5000, (axes, B, N), generator=g, device="cuda")
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    share = rot // 2 // axes
    sections = [rot // 2 - share * (axes - 1)] + [share] * (axes - 1)
    w = [(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in "qk"]
    qw, kw = w[0] if norm in ("both", "q") else None, w[1] if norm in ("both", "k") else None
    got = kivi.qk_norm_rope(qkv, pos, f, Hq, Hkv, q_weight=qw, k_weight=kw, eps=1e-5, sections=sections,
                            interleaved=interleaved)
    ref, tol = rope_reference(qkv, pos, f, Hq, Hkv, qw, kw, 1e-5, sections, interleaved)
    for x, y, t in zip(got, ref, tol):
        err = (x.cpu().double() - y).abs()
        assert (err <= t).all(), float((err / t).max())
    assert torch.equal(got[2].cpu().double(), ref[2])


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(32, 32), (32, 16), (64, 64), (64, 48), (64, 16), (128, 128), (128, 64),
                                   (128, 96), (128, 16)])
def test_rope_every_shape(D, rot, interleaved, dtype):
    check_rope(dtype, 2, 5, 6, 2, D, rot, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("axes", [2, 3, 4])
def test_rope_axes(axes, dtype):
    check_rope(dtype, 2, 33, 4, 2, 128, 128, axes=axes)


@pytest.mark.parametrize("norm", ["none", "q", "k", "both"])
def test_rope_norms(norm):
    check_rope(torch.float16, 3, 1, 8, 1, 64, 64, norm=norm)
    check_rope(torch.float32, 1, 3, 1, 1, 64, 32, norm=norm)


@pytest.mark.parametrize("start", [0, 10 ** 6, 2 ** 31, 2 ** 40, -5000])
def test_rope_far_positions(start):
    check_rope(torch.float32, 1, 9, 2, 1, 64, 64, start=start)


def test_rope_strided_rows_odd_counts():
    check_rope(torch.float16, 3, 7, 3, 1, 128, 128, pad=64)
    check_rope(torch.float16, 5, 1, 5, 3, 32, 32, pad=8)
    check_rope(torch.float32, 1, 301, 7, 5, 32, 32, pad=4)


def test_rope_zero_rows_and_infinite_channels():
    """A head of zeros stays zero; an infinity in a channel that does not turn spoils no other."""
    f = torch.ones(8, dtype=torch.float64, device="cuda")
    pos = torch.ones(1, 2, dtype=torch.int64, device="cuda")
    for inter in (False, True):
        x = torch.zeros(1, 2, 3 * 32, device="cuda", dtype=torch.float16)
        w = torch.ones(32, device="cuda", dtype=torch.float16)
        for t in kivi.qk_norm_rope(x, pos, f, 1, 1, q_weight=w, k_weight=w, interleaved=inter):
            assert (t == 0).all()
        x[:, :, 20] = math.inf
        q, _, _ = kivi.qk_norm_rope(x, pos, f, 1, 1, interleaved=inter)
        assert (q[..., 20] == math.inf).all() and torch.isfinite(q).sum() == q.numel() - 2


# ---- the step as it is used -------------------------------------------------------------------------


@pytest.mark.parametrize("store,dtype", [("ragged", torch.float16), ("paged", torch.float16),
                                         ("ragged", torch.float32)])
def test_steps_of_speculative_decoding(store, dtype):
    """Projections -> tree -> accepted path -> cache, several times across flushes; the tree's last
    accepted node and the same token decoded by kivi_ragged_decode from the cache agree."""
    B, Hq, Hkv, D, R, N = 3, 4, 2, 64, 32, 10
    lens = [40, 31, 90]
    c, st = make_cache(21, B, Hkv, D, 4, lens, R=R, dtype=dtype, store=store, room=4)
    g = gen(5)
    f = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    w = torch.ones(D, dtype=dtype, device="cuda")
    parents = torch.tensor([[-1, 0, 1, 1, 3, 4, 0, 6, 7, 8]]).expand(B, N)
    depth = torch.tensor([0, 1, 2, 2, 3, 4, 1, 2, 3, 4], device="cuda")
    mask = kivi.tree_mask(parents).cuda()
    path = torch.tensor([[0, 1, 3, 4, 5], [0, 6, 7, 8, 9], [0, 1, 2, 0, 0]], dtype=torch.int32, device="cuda")
    for step in range(8):
        count = torch.tensor([(step + 2) % 6, 5, min(3, step)], dtype=torch.int32, device="cuda")
        n_q, r, status = kivi.ragged_lengths(st)
        assert status == [0] * B
        base = torch.tensor([a + b for a, b in zip(n_q, r)], device="cuda")
        qkv = rnd(g, dtype, B, N, (Hq + 2 * Hkv) * D)
        q, k, v = kivi.qk_norm_rope(qkv, base[:, None] + depth, f, Hq, Hkv, q_weight=w, k_weight=w)
        out = c.ragged_tree_decode(st, q, k, v, mask, 0.125)
        assert_tree(out, tree_reference(c, st, q, k, v, mask, 0.125))
        flushed = [a + int(m) > R for a, m in zip(r, count)]
        c.ragged_tree_commit(st, k, v, path, count)
        last = torch.stack([q[b, :, path[b, max(int(count[b]) - 1, 0)]] for b in range(B)])
        again = c.ragged_decode(st, last.contiguous(), 0.125)
        for b in range(B):
            m = int(count[b])
            if m and not flushed[b]:  # a flush quantizes what the tree saw in full precision
                d = (again[b].float() - out[b, :, path[b, m - 1]].float()).abs().max()
                assert d <= 4e-3, (step, b, float(d))
        K, V = c.ragged_read_tokens(st, 0, c.capacity)
        for b, (a, e, _) in enumerate(fills(c, st)):
            if e and int(count[b]):
                assert torch.equal(K[b, :, a + e - 1], k[b, :, path[b, int(count[b]) - 1]])


def test_draft_calls_stay_inside_their_buffers():
    """Guard bands around every output and the workspace."""
    def guarded(nbytes):
        raw = torch.full((4096 + nbytes + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        return raw, raw[4096:4096 + nbytes]
    for D, dtype, gq, N in ((64, torch.float16, 2, 9), (128, torch.float16, 1, 70), (32, torch.float32, 8, 33)):
        c, st = make_cache(3, 3, 2, D, 2, [100, 1, 333], dtype=dtype, store="ragged")
        q, k, v = draft(1, c, gq, N)
        need = int(kivi.lib().kivi_tree_workspace_bytes(ctypes.byref(c._c), N, 2 * gq))
        raws = [guarded(need), guarded(q.numel() * q.element_size()), guarded(3 * 2 * 77 * D * q.element_size()),
                guarded(3 * 2 * 77 * D * q.element_size())]
        c._ws_tree = raws[0][1]
        out = raws[1][1].view(dtype).view(q.shape)
        c.ragged_tree_decode(st, q, k, v, random_tree(1, 3, N), 0.1, out=out)
        assert c._ws_tree is raws[0][1]
        c.ragged_read_tokens(st, 30, 77, K=raws[2][1].view(dtype).view(3, 2, 77, D),
                             V=raws[3][1].view(dtype).view(3, 2, 77, D))
        torch.cuda.synchronize()
        for raw, inner in raws:
            n = inner.numel()
            assert (raw[:4096] == 0xA5).all() and (raw[4096 + n:] == 0xA5).all()
