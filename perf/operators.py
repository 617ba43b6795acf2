"""Cases and plain forms of the operators of speculative decoding over a quantized cache.

Four operators work together in one step of such a decoder:

  rope    the projections of N drafted tokens, norms of queries and keys for each head and
          rotary positions (one or several axes), laid out by heads as the cache takes them
  tree    attention of a tree of N drafted tokens over the cache and over their own ancestors
  commit  the accepted path of the tree written into the cache, window flush included
  read    a range of the cache's tokens read back as numbers

Cache layout (codes, scales, zeros, residual window; pages of R tokens) is that of include/kivi.h.
Lengths of a ragged batch follow from the case alone, so that its work does too.
"""
import math

import torch

own = False

G = 32  # tokens per key group, and channels per value group
STORE = ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale", "v_zero")
BUFFERS = STORE + ("k_res", "v_res")


# ---- the cases ---------------------------------------------------------------------------------


def _cache(name, kind, B, Hq, Hkv, D, T, bits, **more):
    c = {"kind": kind, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "T": T, "bits": bits, "R": 128, "f32": False,
         "meta16": False, "store": "uniform", "N": 1}
    c.update(more)
    return c if name is None else dict(c, name=name)


def _rope(name, B, N, Hq, Hkv, D, **more):
    c = {"kind": "rope", "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": D, "axes": 1, "interleaved": False,
         "norm": True, "f32": False, "start": 4096}
    c.update(more)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # one user, a short context, a chain of five drafted tokens: the step's latency
        _cache("tree-b1-t300-n5", "tree", 1, 32, 32, 128, 300, 2, N=5),
        # the Llama-2-7B-shaped layer of the benchmark, a tree of 16 nodes for each of 8 users
        _cache("tree-mha-b8-t4096-n16", "tree", 8, 32, 32, 128, 4096, 2, N=16),
        # the Mistral-7B-shaped GQA layer at its long context, 4 query heads to a cache head, binary16 scales
        _cache("tree-gqa-b16-t16384-n24", "tree", 16, 32, 8, 128, 16384, 2, N=24, meta16=True),
        # a serving batch of unequal lengths in a paged pool at 4 bits, a wide tree
        _cache("tree-paged-b24-t6000-n61", "tree", 24, 32, 8, 128, 6000, 4, N=61, store="paged"),
        # a binary32 cache of small heads, unequal lengths, 3 bits
        _cache("tree-f32-b6-t2999-n13", "tree", 6, 12, 4, 64, 2999, 3, N=13, R=64, f32=True, store="ragged"),
        # what a verified tree leaves: up to 8 accepted tokens for each of 8 users, half of the windows due for a flush
        _cache("commit-b8-t4096-p8", "commit", 8, 32, 32, 128, 4096, 2, N=16, P=8, store="ragged"),
        # a large paged batch, 4 bits, a long accepted path
        _cache("commit-paged-b64-t2000-p24", "commit", 64, 32, 8, 128, 2000, 4, N=64, P=24, store="paged"),
        # the new tokens of one decode step of 16 users
        _rope("rope-step-b16-n1", 16, 1, 32, 8, 128, start=16384),
        # a prompt with images: positions in time, height and width
        _rope("rope-prompt-b4-n8191-3axes", 4, 8191, 32, 8, 128, axes=3),
        # binary32, a rotated part of small heads, neighbouring channels paired, far positions
        _rope("rope-f32-b6-n517", 6, 517, 12, 4, 64, rot=32, interleaved=True, f32=True, start=1000003),
        # the last pages of a conversation read back to be moved or attended to by other means
        _cache("read-tail-b2-t5001", "read", 2, 32, 8, 128, 5001, 4, t0=4600, n=401),
        # a whole layer of the 7B-shaped batch read back
        _cache("read-all-b8-t4096", "read", 8, 32, 32, 128, 4096, 2, t0=0, n=4096, store="ragged"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("tree", "tree", "tree", "commit", "rope", "rope", "read"))
    D = rng.choice((32, 64, 128, 128, 128))
    Hkv = rng.choice((1, 2, 4, 8, 8, 32))
    gq = rng.choice((1, 2, 4, 8)) if Hkv <= 8 else 1
    f32 = rng.random() < 0.2
    if kind == "rope":
        B, N = _log(rng, 1, 32), _log(rng, 1, 8192)
        while B * N * (gq + 2) * Hkv * D > 4 * 8191 * 48 * 128:
            N = max(1, N // 2)
            B = max(1, B - 1)
        return _rope(None, B, N, gq * Hkv, Hkv, D, rot=rng.choice((D, D, D // 2)), axes=rng.choice((1, 1, 2, 3)),
                     interleaved=rng.random() < 0.5, norm=rng.random() < 0.8, f32=f32, start=_log(rng, 1, 1000003))
    B, T = _log(rng, 1, 32), _log(rng, 1, 16384)
    most = 16 * 8 * 128 * 16384 // (2 if kind == "tree" else 4)  # the largest listed of its kind
    while B * Hkv * D * T > most:
        T = max(1, T // 2)
        B = max(1, B - 1)
    more = {"R": rng.choice((32, 64, 128, 128)), "f32": f32, "meta16": not f32 and rng.random() < 0.3,
            "store": rng.choice(("uniform", "ragged", "paged")), "N": _log(rng, 1, 64)}
    if kind == "tree":  # no more products than the largest listed
        while 4 * gq * more["N"] * B * Hkv * D * T > 4 * 96 * 16 * 8 * 128 * 16384:
            more["N"] = more["N"] // 2
    if kind == "commit":
        more["store"] = rng.choice(("ragged", "paged"))
        more["P"] = rng.randint(1, min(24, more["N"], more["R"]))
    if kind == "read":
        more["t0"] = rng.randrange(T)
        more["n"] = rng.randint(1, T - more["t0"])
    return _cache(None, kind, B, gq * Hkv, Hkv, D, T, rng.choice((1, 2, 2, 3, 4, 4)), **more)


def _lens(c):
    """Tokens of each sequence. A commit's windows stand a few tokens before they are full."""
    B, T, R = c["B"], c["T"], c["R"]
    if c["store"] == "uniform":
        return [T] * B
    lens = [max(1, T - (b * T * 3) // (4 * B) - (b * 5) % 3 * (b > 0)) for b in range(B)]
    if c["kind"] == "commit":
        lens = [max(1, n // R * R - b % c["P"]) for b, n in enumerate(lens)]
    return lens


def _counts(c):
    """Tokens that each sequence accepts, none of them in some."""
    return [(3 * b + c["P"]) % (c["P"] + 1) for b in range(c["B"])]


def _fill(n, R):
    """(quantized tokens, window tokens) of a sequence of n tokens."""
    r = (n - 1) % R + 1
    return n - r, r


def _token_bytes(c):
    """Bytes of a quantized token of one cache head, keys and values."""
    D, m = c["D"], 2 if c["meta16"] else 4
    return 2 * (D * c["bits"] / 8 + 2 * m * D / G)


def work(case):
    c, e = case, 4 if case["f32"] else 2
    B, Hq, Hkv, D, N = c["B"], c["Hq"], c["Hkv"], c["D"], c["N"]
    if c["kind"] == "rope":
        n = B * N * (Hq + 2 * Hkv) * D
        return {"bytes": 2 * n * e + 8 * c["axes"] * B * N, "flops": B * N * (Hq + Hkv) * (4 * D + 3 * c["rot"])}
    fills = [_fill(n, c["R"]) for n in _lens(c)]
    if c["kind"] == "tree":
        stored = sum(nq * _token_bytes(c) + 2 * r * D * e for nq, r in fills) * Hkv
        drafted = B * N * D * e * (2 * Hkv + 2 * Hq) + B * N * 4 * ((N + 31) // 32)
        return {"bytes": stored + drafted, "flops": sum(4 * N * D * (nq + r + (N + 1) / 2) for nq, r in fills) * Hq}
    if c["kind"] == "commit":
        moved = 0
        for (nq, r), m in zip(fills, _counts(c)):
            moved += 4 * m * D * e  # read once, written once, keys and values
            if r + m > c["R"]:  # the window that is quantized: the old part read, its codes written
                moved += 2 * r * D * e + c["R"] * _token_bytes(c)
        return {"bytes": moved * Hkv + B * (16 * 2 + 4 * c["P"]), "flops": 0}
    got, told = 0, 0
    for nq, r in fills:
        a, b = min(c["t0"], nq + r), min(c["t0"] + c["n"], nq + r)
        told += (b - a) * 2 * D * e
        got += max(0, min(b, nq) - a) * _token_bytes(c) + max(0, b - max(a, nq)) * 2 * D * e
    return {"bytes": (got + told) * Hkv, "flops": 0}


# ---- inputs ------------------------------------------------------------------------------------


def _gen(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    return g


def _randn(g, dtype, *shape, by=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * by).to(dtype)


def _tree(case, seed):
    """The ancestors of each node, itself among them, as bits of 32-bit words [B][N][ceil(N / 32)]."""
    B, N = case["B"], case["N"]
    g = torch.Generator()
    g.manual_seed(seed * 7919 + 3)
    sees = torch.zeros(B, N, N, dtype=torch.bool)
    rows = torch.arange(B)
    for i in range(N):
        back = torch.randint(1, 5, (B,), generator=g)  # a parent among the last four nodes
        parent = i - back
        sees[:, i] = sees[rows, parent.clamp(min=0)] & (parent >= 0)[:, None]
        sees[:, i, i] = True
    W = (N + 31) // 32
    bits = torch.zeros(B, N, W * 32, dtype=torch.int64)
    bits[:, :, :N] = sees
    words = (bits.view(B, N, W, 32) << torch.arange(32)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).cuda()


def _prompt(case, g):
    """Keys with four channels of large values in each head, values without."""
    dtype = torch.float32 if case["f32"] else torch.float16
    B, Hkv, D, T = case["B"], case["Hkv"], case["D"], case["T"]
    big = torch.ones(Hkv, D, device="cuda")
    at = torch.rand(Hkv, D, generator=g, device="cuda").argsort(dim=1)[:, :4]
    big.scatter_(1, at, 20.0)
    K = torch.randn(B, Hkv, T, D, generator=g, device="cuda").mul_(big[:, None, :]).to(dtype)
    return K, torch.randn(B, Hkv, T, D, generator=g, device="cuda").to(dtype), big


def _pages(case):
    return (case["T"] + case["R"] - 1) // case["R"] + 1


def _empty_store(case):
    """The cache's buffers, all zero: [units, or pages x heads][tokens ...] of the layout."""
    D, R, bits = case["D"], case["R"], case["bits"]
    dtype = torch.float32 if case["f32"] else torch.float16
    meta = torch.float16 if case["meta16"] else torch.float32
    E, WB = (32, 3) if bits == 3 else (32 // bits, 1)
    lead, Tq = ((case["B"] * _pages(case), case["Hkv"]), R) if case["store"] == "paged" else (
        (case["B"], case["Hkv"]), _pages(case) * R)
    z = lambda *s, t: torch.zeros(lead + s, dtype=t, device="cuda")  # noqa: E731
    w = lambda: torch.zeros(case["B"], case["Hkv"], R, D, dtype=dtype, device="cuda")  # noqa: E731
    return {"k_codes": z(Tq, D // E * WB, t=torch.int32), "k_scale": z(Tq // G, D, t=meta), "k_zero": z(Tq // G, D, t=meta),
            "v_codes": z(Tq // E * WB, D, t=torch.int32), "v_scale": z(Tq, D // G, t=meta), "v_zero": z(Tq, D // G, t=meta),
            "k_res": w(), "v_res": w()}


def prepare(case, seed):
    g = _gen(case, seed)
    dtype = torch.float32 if case["f32"] else torch.float16
    B, Hq, Hkv, D, N = (case[k] for k in ("B", "Hq", "Hkv", "D", "N"))
    s = {"case": case}
    if case["kind"] == "rope":
        rot, axes = case["rot"], case["axes"]
        s["qkv"] = _randn(g, dtype, B, N, (Hq + 2 * Hkv) * D, by=3.0)
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        at = case["start"] + torch.arange(N, device="cuda")
        # the first axis counts on; the others walk over rows and columns of patches, as in an image
        pos = [at] + [case["start"] + torch.arange(N, device="cuda") // 64 ** (axes - 1 - a) % 64 for a in range(1, axes)]
        s["positions"] = torch.stack([p + torch.zeros(B, 1, dtype=torch.int64, device="cuda") for p in pos])
        s["positions"] += torch.randint(0, 1000, (1, B, 1), generator=g, device="cuda")
        share = rot // 2 // axes
        s["sections"] = [rot // 2 - share * (axes - 1)] + [share] * (axes - 1)
        weight = lambda: (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dtype) if case["norm"] else None  # noqa: E731
        s["qw"], s["kw"] = weight(), weight()
        return s
    lens = _lens(case)
    K, V, big = _prompt(case, g)
    uniform, paged = case["store"] == "uniform", case["store"] == "paged"
    if paged:
        order = torch.randperm(B * _pages(case), generator=g, device="cuda").to(torch.int32)
        s["table"] = order.view(B, _pages(case))
    if own:
        import bit_asymmetric_kv_quantize_b200 as kivi

        meta = torch.float16 if case["meta16"] else torch.float32
        if paged:
            cache = kivi.PagedKiviCache(B, Hkv, D, case["bits"], _pages(case), B * _pages(case), s["table"], R=case["R"],
                                        dtype=dtype, meta=meta)
        else:
            cache = kivi.KiviCache(B, Hkv, D, case["bits"], (_pages(case) + 1) * case["R"], R=case["R"], dtype=dtype, meta=meta)
        for b in cache.buffers.values():
            b.zero_()
        s["cache"] = cache
        if uniform:
            cache.prefill(K, V)
        else:
            s["st"] = cache.ragged_prefill(K, V, torch.tensor(lens, device="cuda"))
            s["st0"] = s["st"].clone()
        s["buf"] = {n: cache.view(n) for n in BUFFERS}
    else:
        s["buf"] = _empty_store(case)
        _fill_store(s, K, V, torch.tensor(lens, device="cuda"))
    fills = torch.tensor([_fill(n, case["R"]) for n in lens], device="cuda")
    s["n_q"], s["r"] = fills[:, 0].clone(), fills[:, 1].clone()
    del K, V
    if case["kind"] == "read":
        s["K"] = torch.zeros(B, Hkv, case["n"], D, dtype=dtype, device="cuda")
        s["V"] = torch.zeros_like(s["K"])
        return s
    s["k"] = (torch.randn(B, Hkv, N, D, generator=g, device="cuda") * big[:, None, :]).to(dtype)
    s["v"] = _randn(g, dtype, B, Hkv, N, D)
    if case["kind"] == "tree":
        s["q"] = _randn(g, dtype, B, Hq, N, D)
        s["scale"] = 1 / math.sqrt(D)
        s["mask"] = _tree(case, seed)
    else:
        P = case["P"]
        s["count"] = torch.tensor(_counts(case), dtype=torch.int32, device="cuda")
        # accepted nodes come in the order of the tree; what stands behind the count is not read
        s["path"] = torch.rand(B, N, generator=g, device="cuda").argsort(1)[:, :P].sort(1).values.to(torch.int32).contiguous()
        s["n_q0"], s["r0"] = s["n_q"].clone(), s["r"].clone()
    return s


# ---- the quantizer in plain form -----------------------------------------------------------------


def _quantize(x, dim, bits, meta):
    """Codes, scales and zeros of groups along `dim`: s = (max - min) / top, z = min, code = round((x - z) / s)."""
    top = torch.full((1,), float(2 ** bits - 1), device=x.device)
    z, m = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    s, z = ((m - z) / top).to(meta).float(), z.to(meta).float()
    code = torch.where(s != 0, ((x - z) / torch.where(s != 0, s, torch.ones_like(s))).round().clamp(0, 2 ** bits - 1), torch.zeros_like(x))
    return code.to(torch.int32), s.squeeze(dim), z.squeeze(dim)


def _pack(codes, bits):
    """[..., E] codes -> [..., words]: 32 / bits codes in a word, or three words of one bit plane each."""
    if bits == 3:
        planes = (codes[..., None, :] >> torch.arange(3, device=codes.device, dtype=torch.int32)[:, None]) & 1
        return (planes << torch.arange(32, device=codes.device, dtype=torch.int32)).sum(-1, dtype=torch.int32)
    at = bits * torch.arange(32 // bits, device=codes.device, dtype=torch.int32)
    return (codes << at).sum(-1, dtype=torch.int32)[..., None]


def _unpack(words, bits):
    """The inverse: [..., words] -> [..., E]."""
    if bits == 3:
        planes = (words[..., :, None] >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1
        return (planes << torch.arange(3, device=words.device, dtype=torch.int32)[:, None]).sum(-2, dtype=torch.int32)
    at = bits * torch.arange(32 // bits, device=words.device, dtype=torch.int32)
    return (words >> at) & (2 ** bits - 1)


def _quantized_tokens(case, K, V):
    """The six arrays of [..., T, D] keys and values, T a multiple of 32."""
    bits, lead, T, D = case["bits"], K.shape[:-2], K.shape[-2], K.shape[-1]
    meta = torch.float16 if case["meta16"] else torch.float32
    E, WB = (32, 3) if bits == 3 else (32 // bits, 1)
    ck, sk, zk = _quantize(K.float().reshape(lead + (T // G, G, D)), -2, bits, meta)
    cv, sv, zv = _quantize(V.float().reshape(lead + (T, D // G, G)), -1, bits, meta)
    kw = _pack(ck.reshape(lead + (T, D // E, E)), bits).reshape(lead + (T, D // E * WB))
    vw = _pack(cv.reshape(lead + (T // E, E, D)).transpose(-1, -2), bits)  # [..., T / E, D, WB]
    vw = vw.transpose(-1, -2).reshape(lead + (T // E * WB, D))
    return {"k_codes": kw, "k_scale": sk.to(meta), "k_zero": zk.to(meta), "v_codes": vw, "v_scale": sv.to(meta), "v_zero": zv.to(meta)}


def _paged_view(s, name):
    """A contiguous store's array as pages [B][Hkv][pages][rows of a page][...], without a copy."""
    t = s["buf"][name]
    return t.view(t.shape[:2] + (_pages(s["case"]), -1) + t.shape[3:])


def _put_pages(s, at_b, at_l, new):
    """Writes [n][Hkv][rows][...] as page at_l of sequence at_b."""
    for name in STORE:
        if s["case"]["store"] == "paged":
            s["buf"][name][s["table"][at_b, at_l].long()] = new[name]
        else:
            _paged_view(s, name)[at_b, :, at_l] = new[name]


def _fill_store(s, K, V, lens):
    """A prompt in the cache: whole windows quantized, the rest in the window."""
    case, (B, Hkv, T, D) = s["case"], K.shape
    R = case["R"]
    r = (lens - 1) % R + 1
    pages = (lens - r) // R
    for l in range((T - 1) // R):
        b = (pages > l).nonzero()[:, 0]
        cut = slice(l * R, (l + 1) * R)
        _put_pages(s, b, torch.full_like(b, l), _quantized_tokens(case, K[b, :, cut], V[b, :, cut]))
    slot = torch.arange(R, device=K.device)
    at = (pages[:, None] * R + slot).clamp(max=T - 1)[:, None, :, None].expand(B, Hkv, R, D)
    for name, x in (("k_res", K), ("v_res", V)):
        s["buf"][name].copy_(x.gather(2, at) * (slot < r[:, None])[:, None, :, None])


# ---- the operators in plain form -----------------------------------------------------------------


def _store_values(s):
    """The quantized tokens as numbers: [B][Hkv][tokens][D] keys and values in 32 bits."""
    case, buf = s["case"], s["buf"]
    bits, D, B, Hkv = case["bits"], case["D"], case["B"], case["Hkv"]
    n = int((case["T"] - 1) // case["R"])  # pages that the longest sequence has filled
    E, WB = (32, 3) if bits == 3 else (32 // bits, 1)
    t = {}
    for name in STORE:
        if case["store"] == "paged":
            t[name] = buf[name][s["table"][:, :n].long()].transpose(1, 2)  # [B][Hkv][n][rows][...]
        else:
            t[name] = _paged_view(s, name)[:, :, :n]
    T = n * case["R"]
    ck = _unpack(t["k_codes"].reshape(B, Hkv, T, D // E, WB), bits).reshape(B, Hkv, T // G, G, D)
    K = ck * t["k_scale"].float().reshape(B, Hkv, T // G, 1, D) + t["k_zero"].float().reshape(B, Hkv, T // G, 1, D)
    del ck
    cv = _unpack(t["v_codes"].reshape(B, Hkv, T // E, WB, D).transpose(-1, -2), bits).transpose(-1, -2).reshape(B, Hkv, T, D // G, G)
    V = cv * t["v_scale"].float().reshape(B, Hkv, T, D // G, 1) + t["v_zero"].float().reshape(B, Hkv, T, D // G, 1)
    return K.reshape(B, Hkv, T, D), V.reshape(B, Hkv, T, D)


def _plain_tree(s):
    case = s["case"]
    B, Hq, Hkv, D, N, R = (case[k] for k in ("B", "Hq", "Hkv", "D", "N", "R"))
    K, V = _store_values(s)
    T = K.shape[2]
    q = s["q"].float().view(B, Hkv, Hq // Hkv * N, D) * s["scale"]
    at = torch.arange(T, device=q.device)
    slot = torch.arange(R, device=q.device)
    node = torch.arange(N, device=q.device)
    drafted = (s["mask"][:, :, node // 32] >> (node % 32).to(torch.int32)) & 1 == 1  # [B][N][N]
    sees = torch.cat([(at < s["n_q"][:, None])[:, None].expand(B, N, T), (slot < s["r"][:, None])[:, None].expand(B, N, R), drafted], -1)
    K = torch.cat([K, s["buf"]["k_res"].float(), s["k"].float()], 2)
    score = (q @ K.transpose(-1, -2)).view(B, Hkv, Hq // Hkv, N, T + R + N)
    del K
    score.masked_fill_(~sees[:, None, None], -math.inf)
    score -= score.amax(-1, keepdim=True)
    p = score.exp_()
    p /= p.sum(-1, keepdim=True)
    V = torch.cat([V, s["buf"]["v_res"].float(), s["v"].float()], 2)
    out = p.view(B, Hkv, Hq // Hkv * N, T + R + N) @ V
    return out.view(B, Hq, N, D).to(s["q"].dtype)


def _plain_commit(s):
    case = s["case"]
    B, Hkv, D, N, R, P = (case[k] for k in ("B", "Hkv", "D", "N", "R", "P"))
    s["n_q"].copy_(s["n_q0"])
    s["r"].copy_(s["r0"])
    n_q, r, count = s["n_q"], s["r"], s["count"].long()
    slot = torch.arange(R, device=r.device)

    def path_tokens(x, i):
        """Token i[b][slot] of each accepted path, and whether there is one."""
        at = s["path"].long().gather(1, i.clamp(0, P - 1))[:, None, :, None].expand(B, Hkv, R, D)
        return x.gather(2, at), ((i >= 0) & (i < count[:, None]))[:, None, :, None]

    full = {}
    for name, x in (("k_res", s["k"]), ("v_res", s["v"])):
        new, there = path_tokens(x, slot - r[:, None])
        full[name] = torch.where(there, new, s["buf"][name])
    flush = r + count > R
    b = flush.nonzero()[:, 0]
    _put_pages(s, b, n_q[b] // R, _quantized_tokens(case, full["k_res"][b], full["v_res"][b]))
    for name, x in (("k_res", s["k"]), ("v_res", s["v"])):
        new, there = path_tokens(x, slot + (R - r)[:, None])
        s["buf"][name].copy_(torch.where(there & flush[:, None, None, None], new, full[name]))
    n_q += torch.where(flush, R, 0)
    r += count - torch.where(flush, R, 0)
    return dict(s["buf"], n_q=n_q, r=r)


def _plain_rope(s):
    case = s["case"]
    B, Hq, Hkv, D, N, rot = (case[k] for k in ("B", "Hq", "Hkv", "D", "N", "rot"))
    x = s["qkv"].view(B, N, Hq + 2 * Hkv, D).transpose(1, 2)
    axis = torch.repeat_interleave(torch.arange(case["axes"], device=x.device), torch.tensor(s["sections"], device=x.device))
    angle = s["positions"].double().permute(1, 2, 0)[:, :, axis] * s["inv_freq"]  # [B][N][rot / 2]
    c, si = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * ((x * x).mean(-1, keepdim=True) + 1e-6).rsqrt() * w.float()
        y = x.clone()
        one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        y[..., one] = x[..., one] * c - x[..., two] * si
        y[..., two] = x[..., two] * c + x[..., one] * si
        return y.to(s["qkv"].dtype)

    return turned(x[:, :Hq], s["qw"]), turned(x[:, Hq : Hq + Hkv], s["kw"]), x[:, Hq + Hkv :].contiguous()


def _plain_read(s):
    case = s["case"]
    R, t0, n = case["R"], case["t0"], case["n"]
    K, V = _store_values(s)
    at = t0 + torch.arange(n, device=K.device)
    stored = (at < s["n_q"][:, None])[:, None, :, None]
    there = (at < (s["n_q"] + s["r"])[:, None])[:, None, :, None]
    slot = (at - s["n_q"][:, None]).clamp(0, R - 1)[:, None, :, None].expand(s["K"].shape)
    for out, x, res in ((s["K"], K, s["buf"]["k_res"]), (s["V"], V, s["buf"]["v_res"])):
        y = res.gather(2, slot).float()
        if x.shape[2]:
            y = torch.where(stored, x[:, :, at.clamp(max=x.shape[2] - 1)], y)
        out.copy_(torch.where(there, y.to(out.dtype), out))
    return s["K"], s["V"]


def run(state):
    s, case = state, state["case"]
    kind = case["kind"]
    if not own:
        return {"tree": _plain_tree, "commit": _plain_commit, "rope": _plain_rope, "read": _plain_read}[kind](s)
    if kind == "rope":
        import bit_asymmetric_kv_quantize_b200 as kivi

        return kivi.qk_norm_rope(s["qkv"], s["positions"], s["inv_freq"], case["Hq"], case["Hkv"], q_weight=s["qw"], k_weight=s["kw"],
                                 eps=1e-6, sections=s["sections"], interleaved=case["interleaved"])
    cache = s["cache"]
    if kind == "tree":
        if case["store"] == "uniform":
            return cache.tree_decode(s["q"], s["k"], s["v"], s["mask"], s["scale"])
        return cache.ragged_tree_decode(s["st"], s["q"], s["k"], s["v"], s["mask"], s["scale"])
    if kind == "read":
        if case["store"] == "uniform":
            return cache.read_tokens(case["t0"], case["n"], K=s["K"], V=s["V"])
        return cache.ragged_read_tokens(s["st"], case["t0"], case["n"], K=s["K"], V=s["V"])
    s["st"].copy_(s["st0"])
    cache.ragged_tree_commit(s["st"], s["k"], s["v"], s["path"], s["count"])
    lens = s["st"].view(torch.int64).view(-1, 2)  # {n_q, r, status} of each sequence
    return dict(s["buf"], n_q=lens[:, 0], r=lens[:, 1])


# ---- in 64 bits, from the definitions --------------------------------------------------------------


def _exact_tokens(s, b):
    """Keys and values of sequence b in 64 bits, token by token as the layout says: [Hkv][n][D]."""
    case, buf = s["case"], s["buf"]
    bits, D, R = case["bits"], case["D"], case["R"]
    n_q, r = int(s["n_q"][b]), int(s["r"][b])
    get = lambda name: (torch.cat([buf[name][p] for p in s["table"][b, : n_q // R].tolist()], 1) if n_q else buf[name][0][:, :0]) \
        if case["store"] == "paged" else buf[name][b]  # noqa: E731
    t, d = torch.arange(n_q, device="cuda"), torch.arange(D, device="cuda")
    kc, vc = get("k_codes").long() & 0xFFFFFFFF, get("v_codes").long() & 0xFFFFFFFF
    if bits == 3:
        ck = sum(((kc[:, :n_q][:, :, d // 32 * 3 + p] >> (d % 32)) & 1) << p for p in range(3))
        cv = sum(((vc[:, t // 32 * 3 + p] >> (t % 32)[:, None]) & 1) << p for p in range(3))
    else:
        E = 32 // bits
        ck = (kc[:, :n_q][:, :, d // E] >> (d % E * bits)) & (2 ** bits - 1)
        cv = (vc[:, t // E] >> (t % E * bits)[:, None]) & (2 ** bits - 1)
    K = ck.double() * get("k_scale").double()[:, t // G] + get("k_zero").double()[:, t // G]
    V = cv.double() * get("v_scale").double()[:, :n_q][:, :, d // G] + get("v_zero").double()[:, :n_q][:, :, d // G]
    return torch.cat([K, buf["k_res"][b, :, :r].double()], 1), torch.cat([V, buf["v_res"][b, :, :r].double()], 1)


def exact(case, seed):
    s = prepare(case, seed)
    B, Hq, Hkv, D, N = (case[k] for k in ("B", "Hq", "Hkv", "D", "N"))
    if case["kind"] == "tree":
        outs = []
        for b in range(B):
            K, V = _exact_tokens(s, b)
            K, V = torch.cat([K, s["k"][b].double()], 1), torch.cat([V, s["v"][b].double()], 1)
            words = s["mask"][b].long() & 0xFFFFFFFF
            sees = torch.stack([(words[:, j // 32] >> (j % 32)) & 1 for j in range(N)], 1) == 1
            sees = torch.cat([torch.ones(N, K.shape[1] - N, dtype=torch.bool, device="cuda"), sees], 1)
            rows = []
            for h in range(Hq):
                score = (s["q"][b, h].double() @ K[h * Hkv // Hq].T) * s["scale"]
                score = torch.where(sees, score, torch.full_like(score, -math.inf))
                rows.append(torch.softmax(score, -1) @ V[h * Hkv // Hq])
            outs.append(torch.stack(rows))
        return torch.stack(outs)
    if case["kind"] == "read":
        K, V = s["K"].double(), s["V"].double()
        for b in range(B):
            for out, x in zip((K, V), _exact_tokens(s, b)):
                x = x[:, case["t0"] : case["t0"] + case["n"]]
                out[b, :, : x.shape[1]] = x
        return K, V
    if case["kind"] == "rope":
        x = s["qkv"].double().view(B, N, Hq + 2 * Hkv, D)
        rot, axes = case["rot"], [a for a, n in enumerate(s["sections"]) for _ in range(n)]
        angle = torch.stack([s["positions"][a].double() * s["inv_freq"][i] for i, a in enumerate(axes)], -1)
        turn = torch.polar(torch.ones_like(angle), angle)[:, :, None]
        outs = []
        for y, w in ((x[:, :, :Hq], s["qw"]), (x[:, :, Hq : Hq + Hkv], s["kw"])):
            if w is not None:
                y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / D + 1e-6) * w.double()
            head, tail = y[..., :rot], y[..., rot:]
            if case["interleaved"]:
                head = torch.view_as_real(torch.view_as_complex(head.reshape(head.shape[:-1] + (rot // 2, 2)).contiguous()) * turn).flatten(-2)
            else:
                z = torch.complex(head[..., : rot // 2].contiguous(), head[..., rot // 2 :].contiguous()) * turn
                head = torch.cat([z.real, z.imag], -1)
            outs.append(torch.cat([head, tail], -1).transpose(1, 2).contiguous())
        return outs[0], outs[1], x[:, :, Hq + Hkv :].transpose(1, 2).contiguous()
    # commit: the windows and scales that the definition gives; codes are whole numbers and have to be equal as such
    R, top = case["R"], 2 ** case["bits"] - 1
    out = {n: s["buf"][n].double() for n in BUFFERS if "codes" not in n}
    for b, m in enumerate(s["count"].tolist()):
        n_q, r = int(s["n_q"][b]), int(s["r"][b])
        path = s["path"][b, :m].long()
        for x in ("k", "v"):
            win = torch.cat([s["buf"][x + "_res"][b, :, :r].double(), s[x][b][:, path].double()], 1)
            if r + m > R:
                full, win = win[:, :R], win[:, R:]
                groups = full.view(Hkv, R // G, G, D) if x == "k" else full.view(Hkv, R, D // G, G)
                dim = 2 if x == "k" else 3
                lo, hi = groups.min(dim).values, groups.max(dim).values
                for name, val in ((x + "_scale", (hi - lo) / top), (x + "_zero", lo)):
                    rows = val.shape[1]
                    if case["store"] == "paged":
                        out[name][int(s["table"][b, n_q // R])] = val
                    else:
                        out[name][b, :, n_q // R * rows : n_q // R * rows + rows] = val
                if r:  # slots that the new tokens do not reach keep what filled them
                    out[x + "_res"][b] = full
            out[x + "_res"][b, :, : win.shape[1]] = win
    return dict(out, k_codes=None, v_codes=None, n_q=None, r=None)
