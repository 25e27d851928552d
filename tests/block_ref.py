"""The block-selection and block-attention operators from their definition, in
64 bits, sequence by sequence and head by head with dense masks; and bounds of
how far a correct kernel may be from it.

Bounds.  A rounding to bf16 is off by at most 2^-8 of the value, one to fp32 by
2^-24, and a sum of n fp32 terms by n 2^-24 of the sum of their magnitudes.
The kernels round each output once, the weights p before the product with V
(and dout), and ds before the products with K and Q -- to the tensors' type,
which for fp32 is no rounding beyond the sums' own.  With u the type's unit
(2^-8 or 2^-24), c = n 2^-24 for n the terms of the longest sum, and A = sum
p |v| etc. the sums of magnitudes:
  out    : u |out| + (u + c) A
  Delta  : sum |dout| (bound of out), because the kernels form it from the
           rounded out, plus c sum |dout| |out|
  dQ     : u |dQ| + scale sum_j ((u + c) |ds| + p (bound of Delta + c sum |dout| |v|)) |k|
  dK, dV : the same over the queries.
Scores carry c sum |q| |k| scale, which multiplies p by as much; it is added
to u where p enters.
"""
import math

import torch

UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def units(Nq, S, qb):
    return Nq // qb + (S if qb > 1 else 0)


def offsets(lens):
    o = [0]
    for n in lens:
        o.append(o[-1] + n)
    return o


def table_row(beg, s, per):
    return beg // per + (s if per > 1 else 0)


def allowed(idx, s, g, lq, lk, q0, block, qb, causal, dev):
    """bool [lq, lk]: which keys of sequence s its queries see under key head g."""
    nb = -(-lk // block)
    nu = -(-lq // qb)
    u0 = table_row(q0, s, qb)
    pick = torch.zeros(nu, nb + 1, dtype=torch.bool, device=dev)
    ids = idx[u0:u0 + nu, g].long()
    pick.scatter_(1, torch.where((ids < 0) | (ids >= nb), nb, ids), True)
    ok = pick[:, :nb].repeat_interleave(block, 1)[:, :lk].repeat_interleave(qb, 0)[:lq]
    if causal:
        pos = torch.arange(lq, device=dev)[:, None] + lk - lq
        ok = ok & (torch.arange(lk, device=dev) <= pos)
    return ok


def attention(Q, K, V, idx, sq, sk, block, qb, scale=0.0, causal=False, lk=None, dout=None):
    """dict of out, lse (and dQ, dK, dV) in fp64 with their bounds as ``name_tol``.

    Rows of no sequence hold NaN; sq, sk, lk are host lists."""
    H, Hkv, D = Q.shape[1], K.shape[1], Q.shape[2]
    G, S, dev = H // Hkv, len(sq) - 1, Q.device
    scale = scale or 1.0 / math.sqrt(D)
    u = UNIT[Q.dtype]
    nan = float("nan")
    f64 = {"dtype": torch.float64, "device": dev}
    r = {"out": torch.full(Q.shape, nan, **f64), "lse": torch.full(Q.shape[:2], nan, **f64)}
    names = ["out", "lse"]
    if dout is not None:
        r["dQ"] = torch.full(Q.shape, nan, **f64)
        r["dK"], r["dV"] = (torch.full(K.shape, nan, **f64) for _ in range(2))
        names += ["dQ", "dK", "dV"]
    for n in names:
        r[n + "_tol"] = torch.zeros_like(r[n])
    for s in range(S):
        q0, lq, k0 = sq[s], sq[s + 1] - sq[s], sk[s]
        n = (sk[s + 1] - sk[s]) if lk is None else lk[s]
        if dout is not None:
            for t in ("dK", "dV"):
                r[t][k0:k0 + n] = 0.0
        if lq == 0:
            continue
        c = (n + lq * G + D + 32) * 2.0 ** -24
        for g in range(Hkv):
            ok = (allowed(idx, s, g, lq, n, q0, block, qb, causal, dev) if n
                  else torch.zeros(lq, 0, dtype=torch.bool, device=dev))
            k, v = K[k0:k0 + n, g].double(), V[k0:k0 + n, g].double()
            for h in range(g * G, (g + 1) * G):
                q = Q[q0:q0 + lq, h].double()
                sc = (q @ k.T * scale).masked_fill(~ok, -math.inf)
                err = torch.where(ok, (q.abs() @ k.abs().T) * scale * c, 0.0)  # of a score
                z = torch.logsumexp(sc, 1) if n else torch.full((lq,), -math.inf, **f64)
                some = ok.any(1)
                p = torch.where(ok, torch.exp(sc - torch.where(some, z, 0.0)[:, None]), 0.0)
                perr = p * (u + c + 2 * err)
                vz = torch.where(ok.any(0)[:, None], v, 0.0)
                # values outside a row's view do not count, non-finite ones too
                o = torch.stack([p[i, ok[i]] @ v[ok[i]] for i in range(lq)]) \
                    if not torch.isfinite(v).all() else p @ v
                r["out"][q0:q0 + lq, h] = o
                otol = u * o.abs() + perr @ vz.abs()
                r["out_tol"][q0:q0 + lq, h] = otol
                r["lse"][q0:q0 + lq, h] = torch.where(some, z, -math.inf)
                r["lse_tol"][q0:q0 + lq, h] = torch.where(
                    some, 2.0 ** -20 * (1 + z.abs()) + err.amax(1) if n else z, 0.0)
                if dout is None:
                    continue
                do = dout[q0:q0 + lq, h].double()
                delta = (do * o).sum(1, keepdim=True)
                dtol = (do.abs() * (otol + c * o.abs())).sum(1, keepdim=True)
                dp = do @ v.T
                ds = p * (dp - delta)
                dstol = (u + c + 2 * err) * ds.abs() + p * (dtol + c * (do.abs() @ v.abs().T)) \
                    + p * c * (dp.abs() + delta.abs())
                dq, dk, dv = ds @ k * scale, ds.T @ q * scale, p.T @ do
                r["dQ"][q0:q0 + lq, h] = dq
                r["dQ_tol"][q0:q0 + lq, h] = u * dq.abs() + scale * (dstol + c * ds.abs()) @ k.abs()
                r["dK"][k0:k0 + n, g] += dk
                r["dK_tol"][k0:k0 + n, g] += scale * (dstol + c * ds.abs()).T @ q.abs()
                r["dV"][k0:k0 + n, g] += dv
                r["dV_tol"][k0:k0 + n, g] += (perr + c * p).T @ do.abs()
            if dout is not None:
                for t in ("dK", "dV"):
                    r[t + "_tol"][k0:k0 + n, g] += u * r[t][k0:k0 + n, g].abs()
    return r


def check(got, ref, name, untouched=None):
    """got within the bound of ref on every row of a sequence; the other rows still hold
    ``untouched`` (when given)."""
    want, tol = ref[name], ref[name + "_tol"]
    rest = torch.isnan(want) if name == "lse" else torch.isnan(want).all(-1)
    g = got.double()
    if untouched is not None:
        assert (got[rest] == untouched).all(), f"{name}: a row of no sequence was written"
    g, w, t = g[~rest], want[~rest], tol[~rest]
    fin = torch.isfinite(w)
    assert (torch.isfinite(g) == fin).all(), f"{name}: finite where it must not be, or not"
    assert (g[~fin & ~torch.isnan(w)] == w[~fin & ~torch.isnan(w)]).all(), name
    over = (g - w).abs() - t
    over = torch.where(fin, over, -1.0)
    worst = over.max().item() if over.numel() else -1.0
    assert worst <= 1e-30, (f"{name}: over its bound by {worst:.3e} at "
                            f"{(over == over.max()).nonzero()[0].tolist()}")


def block_sums(K, sk, block, lk=None):
    S = len(sk) - 1
    B = K.shape[0] // block + S
    out = torch.zeros(B, K.shape[1], K.shape[2], dtype=torch.float64, device=K.device)
    for s in range(S):
        n = (sk[s + 1] - sk[s]) if lk is None else lk[s]
        for b in range(-(-n // block)):
            rows = K[sk[s] + b * block:sk[s] + min(n, (b + 1) * block)]
            out[table_row(sk[s], s, block) + b] = rows.double().sum(0)
    return out


def select(Q, K, sq, sk, topk, block, qb, causal=False, lk=None, max_len=None):
    """int32 [units, Hkv, topk] by scores in 64 bits."""
    H, Hkv = Q.shape[1], K.shape[1]
    G, S = H // Hkv, len(sq) - 1
    idx = torch.full((units(Q.shape[0], S, qb), Hkv, topk), -1, dtype=torch.int32)
    sums = block_sums(K, sk, block, lk).cpu()
    q64 = Q.double().cpu()
    for s in range(S):
        lq = sq[s + 1] - sq[s]
        n = (sk[s + 1] - sk[s]) if lk is None else lk[s]
        nb = -(-n // block)
        if max_len is not None:
            nb = min(nb, -(-max_len // block))
        r0 = table_row(sk[s], s, block)
        for j in range(-(-lq // qb)):
            a, b = j * qb, min(lq, (j + 1) * qb)
            for g in range(Hkv):
                q = q64[sq[s] + a:sq[s] + b, g * G:(g + 1) * G].sum((0, 1))
                best = []
                for i in range(nb):
                    size = min(block, n - i * block)
                    v = float((q * sums[r0 + i, g]).sum()) / size
                    if causal:
                        if i * block + block > a + n - lq:
                            v = math.inf
                        if i * block > b - 1 + n - lq:
                            v = -math.inf
                    if v > -math.inf:
                        best.append((-v, i))
                ids = sorted(i for _, i in sorted(best)[:topk])
                idx[table_row(sq[s], s, qb) + j, g, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
    return idx
