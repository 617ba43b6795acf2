"""64-bit plain implementations for the operators around drafted tokens (not a test module).

They read the bytes of a cache by the layout that include/kivi.h states and share no code with
the library's kernels.

Tolerances (derived, not fitted).  With u = 2^-24 (half a step of binary32, relative):
  - a score s = scale * <q, K> of D products, formed in binary32 in any order, is off by at most
    e_s = scale * sum_d |q_d K_d| * (D + 8) u: D additions, and a few roundings for the product,
    the scale (folded with log2 e into q) and K = c s + z.  On matrix operands of binary16 a
    stored key c s + z is carried as c s_hi + c s_lo + z with a relative error of c s below
    2^-17 (s_hi has 7 bits, s_lo 11 more, their products are exact or rounded at 2^-18; codes about
    their center are smaller, and their zeros, two binary16 parts, are kept to 2^-22), so e_s
    grows by scale * sum_d |q_d| (|K_d| + |z_d|) 2^-17 <= scale * sum_d |q_d| 3 max|K_d| 2^-17.
  - a weight exp(s - max) is then off by a factor within exp(+-2 e_s) (its own score's error and the
    maximum's) times 1 + 8u (exp2 and its argument, |s - max| <= 128 before it underflows adds
    128 u); rounded to binary16 for the second product it is off by 2^-11 more, and weights
    below binary16's smallest normal by 2^-25 absolutely; V is carried like K (2^-17).
  - sums of n weights add n u.
  With A = sum p |V| the output is off by at most 2 eps A (numerator and denominator), eps the sum
  of the above, plus n 2^-25 max|V| for tiny weights, plus half a step of the output type.
"""
from __future__ import annotations

import math

import torch

import bit_asymmetric_kv_quantize_b200 as kivi

U = 2.0 ** -24


def fills(cache, st):
    """(n_q, r, status) of each sequence."""
    if st is None:
        return [(cache.n_q, cache.r, 0)] * cache.B
    return list(zip(*kivi.ragged_lengths(st)))


def tokens(cache, b, n_q, r):
    """Keys and values of sequence b in 64 bits: [Hkv][n_q + r][D], on the CPU."""
    bits, D, R = cache.bits, cache.D, cache.R
    paged = hasattr(cache, "block_table")
    get = {}
    for n in kivi.BUFFER_NAMES[:6]:
        x = cache.view(n)
        if paged:
            pages = cache.block_table[b, : n_q // R].tolist()
            x = torch.cat([x[p] for p in pages], 1) if pages else x[0][:, :0]
        else:
            x = x[b]
        get[n] = x.cpu()
    t, d = torch.arange(n_q), torch.arange(D)
    kc, vc = (get[n].long() & 0xFFFFFFFF for n in ("k_codes", "v_codes"))
    if bits == 3:
        ck = sum(((kc[:, :n_q][:, :, d // 32 * 3 + p] >> (d % 32)) & 1) << p for p in range(3))
        cv = sum(((vc[:, t // 32 * 3 + p] >> (t % 32)[:, None]) & 1) << p for p in range(3))
    else:
        E = 32 // bits
        ck = (kc[:, :n_q][:, :, d // E] >> (d % E * bits)) & (2 ** bits - 1)
        cv = (vc[:, t // E] >> (t % E * bits)[:, None]) & (2 ** bits - 1)
    K = ck.double() * get["k_scale"].double()[:, t // 32] + get["k_zero"].double()[:, t // 32]
    V = (cv.double() * get["v_scale"].double()[:, :n_q][:, :, d // 32]
         + get["v_zero"].double()[:, :n_q][:, :, d // 32])
    if cache.__dict__.get("outliers", (0, 0)) != (0, 0):
        ko, vo = cache.outliers
        for h in range(cache.Hkv):
            if ko:
                idx, val = (cache.view(n)[b, h, : n_q // 32].cpu() for n in ("k_out_idx", "k_out_val"))
                for m in range(ko):
                    at = idx[..., m].long() + 32 * torch.arange(n_q // 32)[:, None]
                    K[h][at, d] = val[..., m].double()
            if vo:
                idx, val = (cache.view(n)[b, h, :n_q].cpu() for n in ("v_out_idx", "v_out_val"))
                for m in range(vo):
                    at = idx[..., m].long() + 32 * torch.arange(D // 32)
                    V[h][t[:, None], at] = val[..., m].double()
    return (torch.cat([K, cache.view("k_res")[b, :, :r].cpu().double()], 1),
            torch.cat([V, cache.view("v_res")[b, :, :r].cpu().double()], 1))


def sees(mask, N):
    """bool [B][N][N] of int32 mask words."""
    w = mask.cpu().long() & 0xFFFFFFFF
    j = torch.arange(N)
    return ((w[:, :, j // 32] >> (j % 32)) & 1) == 1


def tree_reference(cache, st, q, k, v, mask, scale):
    """(out, tolerance) in 64 bits, [B][Hq][N][D]."""
    B, Hq, N, D = q.shape
    gq = Hq // cache.Hkv
    f16 = q.dtype == torch.float16
    out = torch.zeros(B, Hq, N, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    see = sees(mask, N)
    for b, (n_q, r, status) in enumerate(fills(cache, st)):
        if status:
            out[b] = math.nan
            continue
        K, V = tokens(cache, b, n_q, r)
        n = n_q + r
        K = torch.cat([K, k[b].cpu().double()], 1)
        V = torch.cat([V, v[b].cpu().double()], 1)
        m = torch.cat([torch.ones(N, n, dtype=torch.bool), see[b]], 1)
        for h in range(Hq):
            Kh, Vh, qh = K[h // gq], V[h // gq], q[b, h].cpu().double()
            s = torch.where(m, qh @ Kh.T * scale, torch.tensor(-math.inf, dtype=torch.float64))
            top = s.amax(1, keepdim=True)
            p = torch.where(m, torch.exp(s - torch.where(top == -math.inf, 0.0, top)), 0.0)
            l = p.sum(1, keepdim=True)
            p = torch.where(l > 0, p / l, 0.0)
            # a token without weight by its mask has no part, whatever its value is
            keep = m.any(0)
            Vk = torch.where(keep[:, None], Vh, 0.0)
            part = p[:, :, None] * torch.where(m[:, :, None], Vk[None], 0.0)
            out[b, h] = part.sum(1)
            if not torch.isfinite(out[b, h]).all():
                continue
            A = part.abs().sum(1)
            Kf = torch.where(keep[:, None], Kh, 0.0)
            qk = torch.where(m, qh.abs() @ Kf.abs().T, 0.0).amax(1, keepdim=True)
            e_s = abs(scale) * qk * (D + 8) * U
            if f16:
                e_s = e_s + abs(scale) * (qh.abs() @ Kf.abs().amax(0)[:, None]) * 3 * 2.0 ** -17
            eps = 2 * e_s + 140 * U + (n + N) * U + ((2.0 ** -11 + 2.0 ** -17) if f16 else 0.0)
            vmax = torch.where(m[:, :, None], Vk.abs()[None], 0.0).amax((1, 2))[:, None] if m.any() else 0.0
            half = torch.finfo(q.dtype).eps / 2
            tol[b, h] = 2 * eps * A + out[b, h].abs() * half + 2.0 ** -25 * half
            if f16:
                tol[b, h] += (n + N) * 2.0 ** -25 / l.clamp(min=1.0) * vmax + 2.0 ** -25 + vmax * 2.0 ** -17
    return out, tol


def assert_tree(got, want):
    ref, tol = want
    g = got.cpu().double()
    assert torch.equal(torch.isnan(g), torch.isnan(ref))
    fin = torch.isfinite(ref)
    assert torch.equal(g[~fin & ~torch.isnan(ref)], ref[~fin & ~torch.isnan(ref)])
    err = (g - ref).abs()
    bad = fin & (err > tol)
    assert not bad.any(), (int(bad.sum()), float((err / tol)[bad].max()), bad.nonzero()[0].tolist())


def rope_reference(qkv, positions, inv_freq, Hq, Hkv, qw, kw, eps, sections, interleaved):
    """(q, k, v) in 64 bits and the tolerance of q and k.  A head's norm is off by at most
    (D + 8) u relative (its sum of squares, of one sign, enters under a root; the root, two products,
    a quotient), cosine and sine by 4 u + pi 2^-24 absolutely (the fraction of a turn rounded to
    binary32, the function's own error), the two products and their sum by 3 u more, all against
    |y1| + |y2|; then half a step of the output type.  An angle a is a binary64 number on both sides:
    a = fl(pos f) here (half a step, |a| 2^-53, and its cosine taken of that number), and in the
    kernel turns = fl(fl(pos f) fl(1 / 2 pi)), three roundings of 2^-53 each, so the two angles
    differ by at most (1 + 3) |a| 2^-53, and cosine and sine by no more; at a = 2^40 that is 2^-11."""
    B, N, width = qkv.shape
    D = width // (Hq + 2 * Hkv)
    x = qkv.cpu().double().view(B, N, -1, D)
    rot = 2 * inv_freq.shape[0]
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    pos = positions.cpu().double().view(-1, B, N)
    ang = torch.stack([pos[a] * float(inv_freq[i]) for i, a in enumerate(axis)], -1)[:, :, None]
    half = torch.finfo(qkv.dtype).eps / 2
    res, tols = [], []
    for y, w in ((x[:, :, :Hq], qw), (x[:, :, Hq:Hq + Hkv], kw)):
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + eps) * w.cpu().double()
        one, two = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
                    else (slice(0, rot // 2), slice(rot // 2, rot)))
        z, t = y.clone(), (D + 8) * U * y.abs()
        z[..., one] = y[..., one] * ang.cos() - y[..., two] * ang.sin()
        z[..., two] = y[..., two] * ang.cos() + y[..., one] * ang.sin()
        both = (y[..., one].abs() + y[..., two].abs()) * ((D + 8 + 4 + 4 + 3) * U + 4 * ang.abs() * 2.0 ** -53)
        t[..., one] = both
        t[..., two] = both
        res.append(z.transpose(1, 2))
        tols.append((t + half * z.abs() + half * 2.0 ** -14).transpose(1, 2))
    return res + [x[:, :, Hq + Hkv:].transpose(1, 2)], tols
