"""Rotary positions and the cache in 4 or 8 bits from their definitions, in 64 bits, row by row and
head by head, with bounds of how far a correct kernel may be from them.

Quantising is defined operation by operation in fp32, so bytes are equal: `quantise` follows those
operations with numpy's fp32 (the FMA in fp64, where the product of two fp32 numbers is exact).

Bounds.  u: half a step of the tensors' type relative to the value, 2^-8 in bf16 and 2^-24 in fp32.
  rotary: u |y| + amp (|a| + |b|) (5 2^-24 + 2 pi 2^-29 + |t| 2^-50): fp32 roundings (the sines of two
      units, product, sum, and the rest of a turn: 2^-24 of an eighth), 32 bits of a turn, and the
      frequency's fp64 roundings, which the angle t multiplies (this reference's own too).
  read: u |x| + 2^-24 |x|, one FMA and one rounding.
  attention: a score is s (q . u) scale + m sum(q) scale, so its error is below
      e = (D + 16) 2^-23 scale sum |q| (|m| + s u) + 2^-21 |score| (2^-22 of q in fp32, exact in bf16;
      the tensor cores add 16 products at a time and may cut instead of rounding: a step, not half one)
      plus 2^-21 for the exponential; with A = sum p (|m| + s u) over the keys, n keys and
      w = 2^-11 (bf16) or 2^-20 (fp32), the weights' rounding in fp16 or as two of them,
      out: u |out| + A (w + 2 max e + (n / 16 + 40) 2^-23) + n 2^-30 max(p s) 2^bits
      lse: max e + (n / 16 + 40) 2^-23 + 2^-22 |lse|
"""
import math

import numpy as np
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def offsets(lens):
    o = [0]
    for n in lens:
        o.append(o[-1] + n)
    return o


def frequencies(width, theta=10000.0, scaling="none", factor=1.0, orig_len=0.0, low=1.0, high=32.0):
    out = []
    for i in range(width // 2):
        base = theta
        if scaling == "base" and width > 2:
            base = theta * factor ** (width / (width - 2))
        f = base ** (-2.0 * i / width)
        if scaling == "linear":
            f /= factor
        if scaling == "ramp":
            turns = orig_len * f / (2 * math.pi)
            g = min(max((turns - low) / (high - low), 0.0), 1.0)
            f = f * g + f / factor * (1 - g)
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def rotary(x, pos, freqs, layout, amp=1.0, inverse=False):
    """(y, tol) in fp64 on the CPU; x [N, H, D], pos [N], freqs in radians."""
    x = x.detach().cpu()
    xd, u = x.double(), HALF[x.dtype]
    R = 2 * len(freqs)
    t = torch.as_tensor(pos).double()[:, None] * freqs * (-1.0 if inverse else 1.0)
    c, s = (amp * torch.cos(t))[:, None], (amp * torch.sin(t))[:, None]
    y, tol = xd.clone(), torch.zeros_like(xd)
    for i in range(R // 2):
        j, k = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
        a, b = xd[..., j], xd[..., k]
        y[..., j] = a * c[..., i] - b * s[..., i]
        y[..., k] = a * s[..., i] + b * c[..., i]
        e = abs(amp) * (a.abs() + b.abs()) * (5 * 2.0 ** -24 + 2 * math.pi * 2.0 ** -29
                                              + t[:, None, i].abs() * 2.0 ** -50)
        for q in (j, k):
            tol[..., q] = u * y[..., q].abs() + e
    return y, tol


def quantise(x, bits):
    """(levels uint8 like x, par: bf16 values m and s as fp32 [..., 2]) of numpy fp32 rows."""
    f32, top = np.float32, 2 ** bits - 1
    with np.errstate(all="ignore"):
        lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
        b = lo.view(np.uint32).astype(np.int64)
        b = np.where(b >= 0x80000000, b + 0xffff, b) & 0xffff0000
        b = np.where(b == 0xff800000, 0xff7f0000, b)
        m = b.astype(np.uint32).view(f32)
        st = (hi * f32(0.5) - m * f32(0.5)) / f32(top / 2)
        s = ((st.view(np.uint32).astype(np.int64) + 0xffff) & 0xffff0000).astype(np.uint32).view(f32)
        s = np.where(s < f32(2.0 ** -126), f32(0), s).astype(f32)
        inv = np.where(s > 0, f32(1) / np.where(s > 0, s, f32(1)), f32(0)).astype(f32)
        c = (-m * inv).astype(f32)
        q = (x.astype(np.float64) * inv.astype(np.float64) + c.astype(np.float64)).astype(f32)
        q = np.rint(np.clip(q, 0, top))
        bad = ~np.isfinite(x).all(-1, keepdims=True)
        q = np.where(bad, 0, q).astype(np.uint8)
        par = np.concatenate([m, s], -1)
        par = np.where(bad, f32("nan"), par).astype(f32)
    return q, par


def pack(levels, bits):
    return levels if bits == 8 else levels[..., 0::2] | (levels[..., 1::2] << 4)


def unpack(b, bits):
    return b if bits == 8 else torch.stack([b & 15, b >> 4], -1).flatten(-2)


def values(cache, which):
    """fp64 [rows, Hkv, D] of what a cache's K (which = 0) or V (1) stands for: (m + s u, |m| + s u)."""
    lev = unpack((cache.v if which else cache.k).cpu(), cache.bits).double()
    m, s = cache.par.cpu().double()[..., 2 * which:2 * which + 2].unbind(-1)
    step = s[..., None] * lev
    return (m[..., None] + step).transpose(0, 1), (m[..., None].abs() + step).transpose(0, 1), \
        s.transpose(0, 1)


def filled(cache, K, V):
    """Fill a whole cache with rows of K and V [rows, Hkv, D], by the definition."""
    par = []
    for x, lev in ((K, cache.k), (V, cache.v)):
        q, p = quantise(x.float().cpu().numpy(), cache.bits)
        lev.copy_(torch.from_numpy(pack(q, cache.bits).copy()).transpose(0, 1))
        par.append(torch.from_numpy(p))
    cache.par.copy_(torch.cat(par, -1).transpose(0, 1).to(torch.bfloat16))
    return cache


def attention(Q, cache, sq, sk, lk, idx=None, block=64, scale=0.0, causal=False):
    """dict of out, lse and their bounds, fp64; rows of no sequence hold NaN."""
    N, H, D = Q.shape
    Hkv = cache.Hkv
    G = H // Hkv
    scale = scale or 1.0 / math.sqrt(D)
    u, w = HALF[Q.dtype], (2.0 ** -20 if Q.dtype == torch.float32 else 2.0 ** -11)
    k, ka, _ = values(cache, 0)
    v, va, vs = values(cache, 1)
    q = Q.cpu().double()
    r = {n: torch.full(s, float("nan"), dtype=torch.float64)
         for n, s in (("out", Q.shape), ("lse", (N, H)), ("out_tol", Q.shape), ("lse_tol", (N, H)))}
    for s in range(len(sq) - 1):
        a, n = sq[s + 1] - sq[s], lk[s]
        for i in range(a):
            row = sq[s] + i
            end = max(0, min(n, i + n - a + 1)) if causal else n
            for h in range(H):
                g = h // G
                see = torch.arange(end)
                if idx is not None:
                    on = set(int(b) for b in idx[row, g].tolist())
                    see = torch.tensor([j for j in range(end) if j // block in on], dtype=torch.long)
                if not len(see):
                    r["out"][row, h], r["lse"][row, h] = 0.0, -math.inf
                    r["out_tol"][row, h] = r["lse_tol"][row, h] = 0.0
                    continue
                at = sk[s] + see
                sc = k[at, g] @ q[row, h] * scale
                e = ((D + 16) * 2.0 ** -23 * scale * (ka[at, g] @ q[row, h].abs())
                     + 2.0 ** -21 * sc.abs() + 2.0 ** -21).max()
                z = torch.logsumexp(sc, 0)
                p = torch.exp(sc - z)
                o, A = p @ v[at, g], p @ va[at, g]
                c = (len(see) / 16 + 40) * 2.0 ** -23
                r["out"][row, h], r["lse"][row, h] = o, z
                r["out_tol"][row, h] = (u * o.abs() + A * (w + 2 * e + c)
                                        + len(see) * 2.0 ** -30 * (p * vs[at, g]).max() * 2 ** cache.bits)
                r["lse_tol"][row, h] = e + c + 2.0 ** -22 * z.abs()
    return r


def check(got, r, name, canary):
    """got against r[name] within its bound; rows of no sequence hold the canary."""
    got, want, tol = got.cpu().double(), r[name], r[name + "_tol"]
    none = torch.isnan(want)
    assert bool((got[none] == canary).all()), f"{name}: rows of no sequence were written"
    inf = torch.isinf(want)
    assert bool((got[inf] == want[inf]).all()), f"{name}: empty rows"
    some = ~none & ~inf
    err = (got[some] - want[some]).abs() - tol[some]
    assert bool((err <= 0).all()), (
        f"{name}: {int((err > 0).sum())} of {err.numel()} beyond the bound, worst "
        f"{float((got[some] - want[some]).abs().max()):.3g}")
