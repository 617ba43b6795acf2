"""Numbers of the attention of drafted tokens: references that rise in the middle of a range, scores
far apart, weights far below the largest, narrow groups far from zero, infinite and NaN values.
Against 64-bit sums over the bytes that the cache holds (draft_testlib.tokens)."""
import math
from types import SimpleNamespace

import pytest
import torch

import bit_asymmetric_kv_quantize_b200 as kivi
from draft_testlib import U, sees, tokens

pytestmark = pytest.mark.gpu

HALF = {torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def weigh(c, b, h, gq, q, k, v, mask, scale):
    """Row h of sequence b in 64 bits: (out, sum p |V|, scores, l, max |V|), p = exp(s - max) / l."""
    K, V = tokens(c, b, c.n_q, c.r)
    K = torch.cat([K, k[b].cpu().double()], 1)[h // gq]
    V = torch.cat([V, v[b].cpu().double()], 1)[h // gq]
    N = q.shape[2]
    m = torch.cat([torch.ones(N, c.n_q + c.r, dtype=torch.bool), sees(mask[b:b + 1], N)[0]], 1)
    s = torch.where(m, q[b, h].cpu().double() @ K.T * scale, -math.inf)
    p = torch.exp(s - s.amax(1, keepdim=True))
    l = p.sum(1, keepdim=True)
    p = p / l
    return p @ V, p @ V.abs(), s, l, V.abs().max()


def head_of(c, h):
    """KV head h of a cache, for weigh."""
    return SimpleNamespace(bits=c.bits, D=c.D, R=c.R, n_q=c.n_q, r=c.r, view=lambda n: c.view(n)[:, h:h + 1])


def split_of(c, rows, N):
    """Tiles of a CTA's range in the tensor-core kernel, for one row block and equal lengths."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = -(-c.n_q // 128) + -(-(c.r + N) // 128)
    return -(-c.B * c.Hkv * tiles // (2 * sms if rows <= 64 else sms))


@pytest.mark.parametrize("heights", [(11.25,), (11.25, 22.5)])
@pytest.mark.parametrize("N", [9, 40, 80])
def test_tree_reference_rises_within_a_range(N, heights):
    """Tokens 11.25 (and 22.5) log2 units above the many others stand in known tiles, for the even rows only:
    just enough for the references to rise there (11 units above the tiles before), so that the sums so
    far are rescaled and still count.  One height: one token in six tiles, whose other 767 are a
    quarter of the sum.  Two: the 128 tokens of a tile at 11.25, one at 22.5 two tiles on, of which they are 5 %.
    Bound: as in tree_reference of draft_testlib, where a key is carried to 2^-17 of its group's range
    and 2^-22 of its middle (3 * 2^-17 max|K| is above both)."""
    B, Hkv, D, T = 32, 2, 32, 2990
    g = torch.Generator().manual_seed(N)
    c = kivi.KiviCache(B, Hkv, D, 2, 3200, R=32)
    K = torch.zeros(B, Hkv, T, D)
    K[..., 0] = 0.1 * torch.rand(B, Hkv, T, generator=g) - 0.05
    V = 0.25 * torch.randn(B, Hkv, T, D, generator=g) + 1.0
    if len(heights) == 1:
        high = {128 * t + 37: heights[0] for t in range(3, 23, 6)}
    else:
        high = {128 * t + i: heights[0] for t in range(0, 23, 4) for i in range(128)}
        high |= {128 * t + 37: heights[1] for t in range(2, 23, 4)}
    at = torch.tensor(list(high))
    K[:, :, at, 1] = torch.tensor(list(high.values()), dtype=torch.float)
    V[:, :, at] = -1.0 if len(heights) == 1 else torch.where(K[:, :, at, 1:2] == heights[1], -1.0, 3.0)
    c.prefill(K.half().cuda(), V.half().cuda())
    assert split_of(c, N, N) >= 4
    q = torch.zeros(B, Hkv, N, D)
    q[..., 0] = 1.0
    q[:, :, ::2, 1] = math.log(2)
    q = q.half().cuda()
    k, v = (0.3 * torch.randn(B, Hkv, N, D, generator=g).half().cuda() for _ in "kv")
    mask = kivi.tree_mask((torch.arange(N) - 2).clamp(min=-1).expand(B, N)).cuda()
    got = c.tree_decode(q, k, v, mask, 1.0).cpu().double()
    for b, h in ((0, 0), (7, 1), (13, 0), (14, 1), (22, 0), (31, 1)):
        ref, A, s, l, vmax = weigh(c, b, h, 1, q, k, v, mask, 1.0)
        n = s.shape[1]
        kmax = tokens(c, b, c.n_q, c.r)[0][h].abs().amax(0).maximum(k[b, h].cpu().double().abs().amax(0))
        e_s = (q[b, h].cpu().double().abs() @ kmax[:, None]) * (3 * 2.0 ** -17 + (D + 8) * U)
        eps = 2 * e_s + 140 * U + n * U + 2.0 ** -11 + 2.0 ** -17
        tol = 2 * eps * A + 2.0 ** -11 * ref.abs() + n * 2.0 ** -29 / l * vmax + 2.0 ** -17 * vmax
        # the sums over a range grow by steps of 16 tokens, each cut off by 2^-23 of them
        tol = tol + 2 * n / 16 * 2.0 ** -23 * A
        assert (tol <= 0.005 * A).all()  # nor would a few per cent of the sum pass
        assert ((got[b, h] - ref).abs() <= tol).all(), (b, h)


@pytest.mark.parametrize("scale", [30.0, -30.0, 3.0])
@pytest.mark.parametrize("N", [7, 70])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_tree_scores_far_apart(dtype, N, scale):
    """Scores up to 700 log2 units apart that are exact up to binary32: the keys of a group are equal (its
    scale is 0 and its zero the key, a binary16 number), queries are powers of two in one channel.
    So a score is off by the roundings of its product with the scale, of that product with log2 e and of
    the difference, 6 half steps of the largest; the rest is a weight's and the output's rounding."""
    B, Hkv, D, T = 2, 3, 64, 500
    g = torch.Generator().manual_seed(N)
    c = kivi.KiviCache(B, Hkv, D, 4, 1024, R=32, dtype=dtype)
    level = torch.randint(-256, 257, (B, Hkv, T // 32 + 1), generator=g) / 64.0
    K = torch.zeros(B, Hkv, T, D)
    K[..., 5] = level.repeat_interleave(32, 2)[:, :, :T]
    V = torch.randn(B, Hkv, T, D, generator=g)
    c.prefill(K.to(dtype).cuda(), V.to(dtype).cuda())
    q = torch.zeros(B, Hkv, N, D)
    q[..., 5] = (2.0 ** (torch.arange(N) % 5 - 3)) * (1 - 2 * (torch.arange(N) % 2))
    k = torch.zeros(B, Hkv, N, D)
    k[..., 5] = torch.randint(-256, 257, (B, Hkv, N), generator=g) / 64.0
    v = torch.randn(B, Hkv, N, D, generator=g)
    q, k, v = (x.to(dtype).cuda() for x in (q, k, v))
    mask = kivi.tree_mask((torch.arange(N) - 3).clamp(min=-1).expand(B, N)).cuda()
    got = c.tree_decode(q, k, v, mask, scale).cpu().double()
    f16 = dtype == torch.float16
    for b in range(B):
        for h in range(Hkv):
            ref, A, s, l, vmax = weigh(c, b, h, 1, q, k, v, mask, scale)
            n = s.shape[1]
            e_s = torch.where(s > -math.inf, s.abs(), 0.0).amax(1, keepdim=True) * 6 * U
            eps = 2 * e_s + 140 * U + n * U + ((2.0 ** -11 + 2.0 ** -17) if f16 else 0.0)
            tol = 2 * eps * A + HALF[dtype] * ref.abs() + 2.0 ** -25 * HALF[dtype]
            if f16:
                tol = tol + n * 2.0 ** -29 / l * vmax + 2.0 ** -25 + 2.0 ** -17 * vmax
            assert (tol <= (0.005 if f16 else 0.0005) * A + 2.0 ** -14).all()
            assert ((got[b, h] - ref).abs() <= tol).all(), (b, h)


@pytest.mark.parametrize("gap", [14.0, 17.3, 20.5, 23.4, 25.6, 27.5, 28.8])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_tree_small_weights_at_any_gap(dtype, gap):
    """Thousands of tokens `gap` log2 units below one: with binary16 operands each keeps its weight to
    2^-11 of itself and 2^-29 of the largest, as include/kivi.h states, whatever the gap is."""
    B, Hkv, D, T = 8, 8, 32, 4096
    c = kivi.KiviCache(B, Hkv, D, 2, T + 32, R=32, dtype=dtype)
    K = torch.zeros(B, Hkv, T, D, device="cuda", dtype=dtype)
    K[:, :, 0] = gap * math.log(2) / D
    V = torch.full_like(K, 64.0)
    V[:, :, 0] = 0
    c.prefill(K, V)
    q = torch.ones(B, Hkv, 3, D, device="cuda", dtype=dtype)
    none = torch.zeros(B, 3, 1, dtype=torch.int32, device="cuda")
    got = c.tree_decode(q, q, q, none, 1.0).cpu().double()
    f16 = dtype == torch.float16
    for b, h in ((0, 0), (3, 7), (7, 4)):
        ref, A, s, l, vmax = weigh(c, b, h, 1, q, q, q, none, 1.0)
        e_s = gap * ((3 * 2.0 ** -17 if f16 else 0.0) + (D + 8) * U)
        eps = 2 * e_s + (140 + T) * U + (2.0 ** -11 if f16 else 0.0)
        tol = 2 * eps * A + HALF[dtype] * ref.abs()
        if f16:
            tol = tol + T * 2.0 ** -29 / l * vmax + 2 * T / 16 * 2.0 ** -23 * A
        assert ((got[b, h] - ref).abs() <= tol).all(), (b, h)


@pytest.mark.parametrize("bits", [1, 2, 4])
@pytest.mark.parametrize("meta", [torch.float32, torch.float16])
def test_tree_narrow_groups_far_from_zero(bits, meta):
    """Groups of keys a unit wide around 1400, where a group's middle is most of what is carried: a stored
    key is off by 2^-17 of its group's range, 2^-22 of its middle and 2^-21, as include/kivi.h states.
    One channel of q is not 0, so a score has 6 roundings to binary32 more."""
    B, Hkv, D, T, N = 2, 2, 64, 600, 5
    g = torch.Generator().manual_seed(bits)
    c = kivi.KiviCache(B, Hkv, D, bits, 1024, R=32, meta=meta)
    mid = 1400 + torch.randint(0, 8, (B, Hkv, T // 32 + 1, 1), generator=g).float()
    K = (mid.repeat_interleave(32, 2)[:, :, :T] + torch.rand(B, Hkv, T, D, generator=g))
    V = torch.randn(B, Hkv, T, D, generator=g)
    c.prefill(K.half().cuda(), V.half().cuda())
    q = torch.zeros(B, Hkv, N, D)
    q[..., 9] = 1.0
    k, v = torch.full((B, Hkv, N, D), 1404.0), torch.randn(B, Hkv, N, D, generator=g)
    q, k, v = (x.half().cuda() for x in (q, k, v))
    mask = kivi.tree_mask(torch.full((B, N), -1)).cuda()
    for scale in (1.0, 4.0):
        got = c.tree_decode(q, k, v, mask, scale).cpu().double()
        for b in range(B):
            for h in range(Hkv):
                ref, A, s, l, vmax = weigh(c, b, h, 1, q, k, v, mask, scale)
                n = s.shape[1]
                e_s = scale * (2.0 ** -17 + 1409 * 2.0 ** -22 + 2.0 ** -21) + scale * 1409 * 6 * U
                eps = 2 * e_s + 140 * U + n * U + 2.0 ** -11 + 2.0 ** -17
                tol = (2 * eps * A + 2.0 ** -11 * ref.abs() + n * 2.0 ** -29 / l * vmax + 2.0 ** -25
                       + 2.0 ** -17 * vmax)
                assert ((got[b, h] - ref).abs() <= tol).all(), (scale, b, h)


# ---- infinite and NaN values and keys of tokens that a node attends to ---------------------------


def words(see):
    """int32 mask words of bool [B][N][N]."""
    B, N, _ = see.shape
    w = torch.zeros(B, N, -(-N // 32) * 32, dtype=torch.int64)
    w[..., :N] = see
    w = (w.view(B, N, -1, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).cuda()


def same(x, value):
    return torch.isnan(x) if math.isnan(value) else x == value


@pytest.mark.parametrize("where", ["draft", "window"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("B,Hkv,T", [(16, 32, 40), (1, 1, 700), (1, 2, 130), (40, 8, 200)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_tree_attended_values_that_are_not_finite(dtype, B, Hkv, T, value, where):
    """A value that is infinite or NaN makes its channel so for every node that attends to it, whether
    its weight is 2^-200 of the largest or not, and however the work is split; it has no part in
    the other channels and nodes."""
    D, N, R = 32, 40, 64
    g = torch.Generator().manual_seed(T)
    c = kivi.KiviCache(B, Hkv, D, 2, T // R * R + 2 * R, R=R, dtype=dtype)
    K = torch.zeros(B, Hkv, T, D)
    V = torch.randn(B, Hkv, T, D, generator=g)
    r = (T - 1) % R + 1
    q, k = torch.zeros(B, Hkv, N, D), torch.zeros(B, Hkv, N, D)
    q[..., 0] = math.log(2)
    K[:, :, : T - r, 0] = 200.0  # the store's tokens, where there are any: all other weights are 0
    k[:, :, 33, 0] = 250.0  # and one late node, above them
    v = torch.randn(B, Hkv, N, D, generator=g)
    see = torch.zeros(B, N, N, dtype=torch.bool)
    see[:, ::2, 2] = True
    see[:, 1::4, 33] = True
    see[:, 4, 33] = True
    mask = words(see)
    q, k, v = (x.to(dtype).cuda() for x in (q, k, v))
    K, V = K.to(dtype).cuda(), V.to(dtype).cuda()
    c.prefill(K, V)
    clean = c.tree_decode(q, k, v, mask, 1.0)
    assert torch.isfinite(clean).all()
    if where == "draft":
        v[:, :, 2, 1::3] = value
        rows = see[0, :, 2].cuda()
    else:
        c.view("v_res")[:, :, min(3, r - 1), 1::3] = value
        rows = torch.ones(N, dtype=torch.bool, device="cuda")
    got = c.tree_decode(q, k, v, mask, 1.0)
    assert same(got[:, :, rows][..., 1::3], value).all()
    rest = torch.ones(D, dtype=torch.bool)
    rest[1::3] = False
    assert torch.equal(got[..., rest], clean[..., rest])
    assert torch.equal(got[:, :, ~rows], clean[:, :, ~rows])


@pytest.mark.parametrize("T", [0, 40, 700])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_tree_attended_keys_that_are_infinite(dtype, T):
    """A score of -inf is a weight of 0, and a node with no other gets 0; +inf and NaN give NaN.  The
    other nodes keep their results."""
    B, Hkv, D, N = 2, 2, 32, 40
    c = kivi.KiviCache(B, Hkv, D, 2, 1024, R=64, dtype=dtype)
    g = torch.Generator().manual_seed(T)
    if T:
        c.prefill(*(torch.randn(B, Hkv, T, D, generator=g).to(dtype).cuda() for _ in "kv"))
    q, k, v = (torch.randn(B, Hkv, N, D, generator=g).to(dtype).cuda() for _ in "qkv")
    q[..., 0] = 1.0
    mask = words(torch.eye(N, dtype=torch.bool).expand(B, N, N))
    none = torch.zeros_like(mask)
    clean, alone = c.tree_decode(q, k, v, mask, 0.5), c.tree_decode(q, k, v, none, 0.5)
    low, high, odd = (3, 35), (5, 36), (7, 39)
    for n in low:
        k[:, :, n, 0] = -math.inf
    for n in high:
        k[:, :, n, 0] = math.inf
    for n in odd:
        k[:, :, n, 0] = math.nan
    got = c.tree_decode(q, k, v, mask, 0.5)
    touched = torch.zeros(N, dtype=torch.bool)
    touched[list(low + high + odd)] = True
    assert torch.equal(got[:, :, ~touched], clean[:, :, ~touched])
    assert torch.isnan(got[:, :, list(high + odd)]).all()
    assert torch.equal(got[:, :, list(low)], alone[:, :, list(low)])
    if not T:
        assert (got[:, :, list(low)] == 0).all()
        v[:, :, list(low)] = math.inf  # no weight is left: still 0
        assert (c.tree_decode(q, k, v, mask, 0.5)[:, :, list(low)] == 0).all()


def long_groups(N, dtype=torch.float16):
    """Groups of which a CTA has about one (rows = N)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if dtype == torch.float32:
        return 4 * sms + 4 if N <= 16 else 3 * sms + 4
    return 2 * sms + 4 if N <= 64 else sms + 2


@pytest.mark.parametrize("N", [3, 80])
def test_tree_sums_of_one_sign_over_a_million_tokens(N):
    """Equal weights and, in each channel, equal values: partial sums only grow, and the tensor cores cut each
    addition off toward zero.  A segment has 128 tiles at most, 1024 steps of 16 tokens: its sums of c' s
    (two planes) lose up to 2 * 1024 * 2^-23 / 2 of themselves (a step 2^-23 of the sum so far, which
    grows evenly), those of z' and of the weights 1024 * 2^-23 / 2; the segments are joined in binary32 (64
    of them, 3 roundings each); a stored value is carried to 2^-17; the output is rounded."""
    D, T, H = 32, 1 << 20, long_groups(N)
    c = kivi.KiviCache(1, H, D, 2, T + 32, R=32)
    for n in ("k_codes", "k_scale", "k_zero", "v_zero", "k_res", "v_res"):
        c.buffers[n].zero_()
    code = torch.arange(D) % 4  # of channel d, for every token
    w = torch.tensor([0, 0x55555555, 0xAAAAAAAA - (1 << 32), -1])[code].to(torch.int32).cuda()
    c.view("v_codes").copy_(w.expand(c.view("v_codes").shape))
    c._c.n_q, c._c.r = T, 32
    q = torch.zeros(1, H, N, D, dtype=torch.float16, device="cuda")
    none = torch.zeros(1, N, -(-N // 32), dtype=torch.int32, device="cuda")
    for s, z in ((2 / 3, -1.0), (0.0, 1.0), (2 / 3, 1.0)):
        c.view("v_scale").fill_(s)
        c.view("v_zero").fill_(z)
        want = code.double() * float(torch.tensor(s)) + z
        c.view("v_res").copy_(want.half().cuda().expand(c.view("v_res").shape))
        got = c.tree_decode(q, q, q, none, 1.0)[0].cpu().double()
        part = (code - 1.5).abs() * s + abs(z + 1.5 * s)
        tol = (2.0 ** -13 + 2 * 2.0 ** -14 + 3 * 64 * U + 2.0 ** -17) * part + 2.0 ** -11 * want.abs()
        assert ((got - want).abs() <= tol).all(), (s, z, float(((got - want).abs() / tol).max()))


@pytest.mark.parametrize("N", [3, 20])
def test_tree_binary32_sums_of_one_sign(N):
    """The same in binary32, where an addition is off by half a unit of the sum's last place, to one side for
    equal steps: 512 of them in a segment, whose sum grows evenly (512 / 2 half steps); 3 roundings for each
    of T / 512 joins; the value itself, the quotient, and the window's tile 8 more."""
    D, T, H = 32, 1 << 17, long_groups(N, torch.float32)
    c = kivi.KiviCache(1, H, D, 2, T + 32, R=32, dtype=torch.float32)
    for n in ("k_codes", "k_scale", "k_zero", "v_zero", "k_res", "v_res"):
        c.buffers[n].zero_()
    code = torch.arange(D) % 4
    w = torch.tensor([0, 0x55555555, 0xAAAAAAAA - (1 << 32), -1])[code].to(torch.int32).cuda()
    c.view("v_codes").copy_(w.expand(c.view("v_codes").shape))
    c._c.n_q, c._c.r = T, 32
    q = torch.zeros(1, H, N, D, device="cuda")
    none = torch.zeros(1, N, 1, dtype=torch.int32, device="cuda")
    for s, z in ((2 / 3, -1.0), (0.1, 0.7), (1 / 3, 1.0)):
        c.view("v_scale").fill_(s)
        c.view("v_zero").fill_(z)
        want = code.double() * float(torch.tensor(s)) + float(torch.tensor(z))
        c.view("v_res").copy_(want.float().cuda().expand(c.view("v_res").shape))
        got = c.tree_decode(q, q, q, none, 1.0)[0].cpu().double()
        tol = (512 / 2 + 3 * T / 512 + 8) * U * want.abs()
        assert ((got - want).abs() <= tol).all(), (s, z, float(((got - want).abs() / tol).max()))


@pytest.mark.parametrize("N,dtype", [(9, torch.float16), (80, torch.float16), (9, torch.float32),
                                     (50, torch.float32)])
def test_tree_ranges_of_several_segments(N, dtype):
    """Ranges of more than 128 tiles (16 in binary32), whose segments are joined in the kernel: references
    that rise or fall from one to the next, whole groups and parts of groups, an infinite value, each
    against its own sums.  Bound as in test_tree_reference_rises_within_a_range; binary32: a
    segment's sums are off by 512 half steps at most, the joins (40) by 3 each."""
    D, T, H = 32, 20011, long_groups(N, dtype)
    f16 = dtype == torch.float16
    g = torch.Generator(device="cuda").manual_seed(N)
    c = kivi.KiviCache(1, H, D, 2, 20096, R=32, dtype=dtype)
    K = torch.zeros(1, H, T, D, device="cuda")
    K[..., 0] = 0.1 * torch.rand(1, H, T, generator=g, device="cuda") - 0.05
    ramp = torch.linspace(0, 16, T, device="cuda")
    K[:, ::2, :, 1] = ramp
    K[:, 1::2, :, 1] = ramp.flip(0)
    V = 0.25 * torch.randn(1, H, T, D, generator=g, device="cuda") + torch.linspace(-1, 1, T, device="cuda")[:, None]
    c.prefill(K.to(dtype), V.to(dtype))
    assert not f16 or split_of(c, N, N) > 128
    q = torch.zeros(1, H, N, D, device="cuda")
    q[..., 0] = 1.0
    q[:, :, ::2, 1] = 0.25 * math.log(2)
    q[:, :, 1::4, 1] = 2 * math.log(2)
    q = q.to(dtype)
    k, v = ((0.3 * torch.randn(1, H, N, D, generator=g, device="cuda")).to(dtype) for _ in "kv")
    mask = kivi.tree_mask((torch.arange(N) - 2).clamp(min=-1)[None]).cuda()
    got = c.tree_decode(q, k, v, mask, 1.0)
    for h in (0, 1, 2, 51, 100, H // 2, H // 2 + 1, H - 2, H - 1):
        ref, A, s, l, vmax = weigh(head_of(c, h), 0, 0, 1, *(x[:, h:h + 1] for x in (q, k, v)), mask, 1.0)
        n = s.shape[1]
        kmax = torch.cat([K[0, h].to(dtype), k[0, h]]).abs().amax(0).cpu().double()
        e_s = (q[0, h].cpu().double().abs() @ kmax[:, None]) * ((3 * 2.0 ** -17 if f16 else 0.0) + (D + 8) * U)
        eps = 2 * e_s + (140 + 512 + 3 * 40) * U
        if f16:
            eps = 2 * e_s + 140 * U + 2.0 ** -11 + 2.0 ** -17 + 2.0 ** -13 + 2 * 2.0 ** -14
        tol = 2 * eps * A + HALF[dtype] * ref.abs()
        if f16:
            tol = tol + n * 2.0 ** -29 / l * vmax + 2.0 ** -17 * vmax
        assert (tol <= (0.006 if f16 else 0.0005) * A).all()  # (2 * 2 e_s = 4 * 22 * 40 u = 2.1e-4 for q = 2 ln 2)
        assert ((got[0, h].cpu().double() - ref).abs() <= tol).all(), h
    v[:, :, 2, 1::3] = math.inf
    sees2 = sees(mask, N)[0, :, 2].cuda()
    odd = c.tree_decode(q, k, v, mask, 1.0)
    assert (odd[:, :, sees2][..., 1::3] == math.inf).all()
    assert torch.equal(odd[:, :, ~sees2], got[:, :, ~sees2])
    rest = torch.ones(D, dtype=torch.bool)
    rest[1::3] = False
    assert torch.equal(odd[..., rest], got[..., rest])
    assert torch.equal(c.tree_decode(q, k, v, mask, 1.0), odd)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_tree_bad_pages_in_ranges_of_several_segments(dtype):
    """A page outside the pool in any segment of a sequence makes all of it NaN, and no other."""
    D, R, N = 32, 128, 5
    B = long_groups(N, dtype)
    pages = 160
    g = torch.Generator(device="cuda").manual_seed(1)
    bt = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    c = kivi.PagedKiviCache(B, 1, D, 2, pages, B * pages, bt, R=R, dtype=dtype)
    K = torch.randn(B, 1, 20400, D, generator=g, device="cuda").to(dtype)
    st = c.ragged_prefill(K, K, torch.full((B,), 20400, device="cuda"))
    q, k, v = (torch.randn(B, 1, N, D, generator=g, device="cuda").to(dtype) for _ in "qkv")
    mask = kivi.tree_mask((torch.arange(N) - 1).expand(B, N)).cuda()
    clean = c.ragged_tree_decode(st, q, k, v, mask, 0.2)
    bad = {0: 0, 5: 3, 6: 150, 100: 70, B - 1: 158}
    for b, p in bad.items():
        c.block_table[b, p] = -1
    got = c.ragged_tree_decode(st, q, k, v, mask, 0.2)
    rows = torch.tensor(list(bad), device="cuda")
    good = torch.ones(B, dtype=torch.bool, device="cuda")
    good[rows] = False
    assert torch.isnan(got[rows]).all() and torch.isfinite(clean).all()
    assert torch.equal(got[good], clean[good])


# ---- largest tree, first call in a capture ---------------------------------------------------------


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_tree_of_the_largest_size(dtype):
    """256 nodes of 64 query heads to a KV head: 16384 rows, each against its own reference."""
    B, Hkv, D, T, gq, N = 1, 1, 32, 300, 64, 256
    g = torch.Generator().manual_seed(1)
    c = kivi.KiviCache(B, Hkv, D, 2, 512, R=32, dtype=dtype)
    c.prefill(*(torch.randn(B, Hkv, T, D, generator=g).to(dtype).cuda() for _ in "kv"))
    q = torch.randn(B, gq, N, D, generator=g).to(dtype).cuda()
    k, v = (torch.randn(B, Hkv, N, D, generator=g).to(dtype).cuda() for _ in "kv")
    mask = words(torch.rand(B, N, N, generator=g) < 0.3)
    got = c.tree_decode(q, k, v, mask, 0.2).cpu().double()
    f16 = dtype == torch.float16
    kmax = torch.cat([tokens(c, 0, c.n_q, c.r)[0][0], k[0, 0].cpu().double()]).abs().amax(0)
    for h in (0, 1, 31, 63):
        ref, A, s, l, vmax = weigh(c, 0, h, gq, q, k, v, mask, 0.2)
        n = s.shape[1]
        e_s = 0.2 * (q[0, h].cpu().double().abs() @ kmax[:, None]) * ((D + 8) * U + (3 * 2.0 ** -17 if f16 else 0.0))
        eps = 2 * e_s + 140 * U + n * U + ((2.0 ** -11 + 2.0 ** -17) if f16 else 0.0)
        tol = 2 * eps * A + HALF[dtype] * ref.abs() + 2.0 ** -25 * HALF[dtype]
        if f16:
            tol = tol + n * 2.0 ** -29 / l * vmax + 2.0 ** -25 + 2.0 ** -17 * vmax
        assert ((got[0, h] - ref).abs() <= tol).all(), h


def test_tree_first_call_of_a_cache_in_a_capture():
    """The workspace made under capture serves the graph and eager calls after it."""
    c = kivi.KiviCache(1, 2, 64, 2, 2048, R=64)
    g = torch.Generator(device="cuda").manual_seed(3)
    c.prefill(*(torch.randn(1, 2, 1500, 64, generator=g, device="cuda").half() for _ in "kv"))
    q, k, v = (torch.randn(1, 2, 6, 64, generator=g, device="cuda").half() for _ in "qkv")
    mask = kivi.tree_mask((torch.arange(6) - 1)[None]).cuda()
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.tree_decode(q, k, v, mask, 0.125, out=out)
    graph.replay()
    eager = c.tree_decode(q, k, v, mask, 0.125)
    graph.replay()
    del graph
    again = c.tree_decode(q, k, v, mask, 0.125)
    assert torch.equal(out, eager) and torch.equal(out, again)
