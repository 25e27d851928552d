"""Workloads of rotary positions and of a key/value cache held in 4 or 8 bits: what is run, on which inputs, how much work it is.

Five operators, each with a plain form (elementary torch operations in fp32, fp64 for angles and wherever a rounding decides) and the
library's own calls:

* ``rotary``: pairs of a head's first elements turned by angles that grow with the row's position;
* ``write``: rows of K and V appended to a cache in 4 or 8 bits, and the same rows read back;
* ``read``: a whole cache back in bf16 or fp32, as for several queries at once;
* ``sums``: 64-bit sums of each block of cached keys, all or those that changed;
* ``attend``: single tokens' softmax attention over the cache, over chosen blocks or over all of it.

Positions.  Sequence s owns the rows [seq_q[s], seq_q[s+1]) of the new tokens and the cache rows [seq_k[s], seq_k[s] + len_k[s]); its
row i of lq stands at position i + len_k[s] - lq.

Cache.  Levels uint8 [Hkv, rows, D * bits / 8] for K and for V (element 2j of a row in the low half of byte j with 4 bits), and bf16
[Hkv, rows, 4]: K's least value m and step s, then V's.  An element stands for m + s * level.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"


# ---------------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------------
def _rotary(name, S, q, far, H, Hkv, D, width, layout, dtype=BF16, scaling="none", factor=1.0, packed=False, train=False):
    c = {"op": "rotary", "S": S, "q": q, "k": far, "H": H, "Hkv": Hkv, "D": D, "width": width, "layout": layout, "dtype": dtype,
         "scaling": scaling, "factor": factor, "packed": packed, "train": train}
    return {"name": name, **c} if name else c


def _cache(name, op, S, q, k, H, Hkv, D, bits, dtype=BF16, block=64, topk=0, causal=False, packed=False, renew=False):
    c = {"op": op, "S": S, "q": q, "k": k, "H": H, "Hkv": Hkv, "D": D, "bits": bits, "dtype": dtype, "block": block, "topk": topk,
         "causal": causal, "packed": packed, "renew": renew}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one new token for each of 16 requests, far into contexts stretched eightfold: latency
        _rotary("rotary-token-16", 16, 1, 60000, 32, 8, 128, 128, "half", scaling="ramp", factor=8.0),
        # a long prompt, Q and K taken as slices of one projection
        _rotary("rotary-prompt-32k", 1, 32768, 32768, 32, 8, 128, 128, "half", packed=True),
        # a training step on graphs of unlike sizes in fp32: half of each head turned, forward and backward
        _rotary("rotary-train-f32", 7, 2859, 2859, 8, 8, 64, 32, "interleaved", dtype=F32, train=True),
        # one new token for each of 64 requests goes into the cache
        _cache("write-token-64", "write", 64, 1, 4000, 32, 8, 128, 4),
        # a long prompt goes into the cache, K and V taken as slices of one projection
        _cache("write-prompt-32k", "write", 1, 32768, 32768, 32, 8, 128, 4, packed=True),
        # caches read back for the next chunk of four prompts
        _cache("read-chunk-4x8k", "read", 4, 1, 8000, 32, 8, 128, 4),
        # small caches in 8 bits read back in fp32
        _cache("read-8bit-f32", "read", 3, 1, 1237, 4, 4, 64, 8, dtype=F32),
        # after one new token for each of 8 requests: the sums of the last blocks
        _cache("sums-token-8", "sums", 8, 1, 4000, 32, 8, 128, 4, renew=True),
        # all block sums of a batch of graphs
        _cache("sums-graphs-64k", "sums", 24, 1, 2731, 8, 8, 64, 4),
        # the smallest serving call: one new token for each of 4 requests, 16 blocks for each of 8 key heads
        _cache("attend-token-4", "attend", 4, 1, 2000, 32, 8, 128, 4, topk=16),
        # a full serving batch with caches of about 8,000 tokens, of which each key head reads 32 blocks
        _cache("attend-token-128", "attend", 128, 1, 8000, 32, 8, 128, 4, topk=32),
        # a few requests with long caches that are read whole
        _cache("attend-whole-8x32k", "attend", 8, 1, 32000, 32, 8, 128, 4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "write", "read", "sums", "attend", "attend", "attend"])
    D = rng.choice([32, 64, 64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8, 16])
    bits = rng.choice([4, 4, 8])
    dtype = rng.choice([BF16, BF16, F32])
    S = _log(rng, 1, 64)
    if op == "rotary":
        D = rng.choice([16, D])
        width = rng.choice([w for w in (10, 16, 32, 64, 96, 128) if w <= D])
        G = min(G, 64 // Hkv)
        n = _log(rng, 1, max(1, min(32768, (1 << 25) // (Hkv * (G + 1) * D)) // S))
        scaling = rng.choice(["none", "linear", "base", "ramp"])
        return _rotary(None, S, n, n + _log(rng, 1, 200000), Hkv * G, Hkv, D, width, rng.choice(["half", "interleaved"]), dtype, scaling,
                       1.0 if scaling == "none" else rng.choice([2.0, 4.0, 16.0]), rng.random() < 0.4, rng.random() < 0.4)
    if op == "write":
        n = _log(rng, 1, max(1, 32768 // S))
        return _cache(None, op, S, n, n + _log(rng, 1, 3000), Hkv, Hkv, D, bits, dtype, packed=rng.random() < 0.5)
    if op == "read":
        return _cache(None, op, S, 1, _log(rng, 1, max(2, 32000 // S)), Hkv, Hkv, D, bits, dtype)
    block = rng.choice([16, 32, 64, 64, 128])
    if op == "sums":
        return _cache(None, op, S, 1, _log(rng, 1, max(2, 60000 // S)), Hkv, Hkv, D, bits, dtype, block, renew=rng.random() < 0.5)
    q = min(rng.choice([1, 1, 1, 2, 5]), max(1, 64 // S))
    if rng.random() < 0.4:  # the whole cache
        k = _log(rng, 1, max(2, 120000 // (S * q)))
        return _cache(None, op, S, q, k, Hkv * G, Hkv, D, bits, dtype, block, 0, rng.random() < 0.5)
    topk = rng.choice([1, 5, 16, 32]) if block <= 64 else rng.choice([1, 5, 16])
    return _cache(None, op, S, q, _log(rng, 1, min(16000, 1000000 // S)), Hkv * G, Hkv, D, bits, dtype, block, topk, rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------------
def _lengths(c):
    """New rows and cache lengths of each sequence: a function of the case alone."""
    r = random.Random(1000003 * c["S"] + 101 * c["k"] + c["q"])
    many = c["q"] > 8
    q = [max(1, int(c["q"] * r.uniform(0.6, 1.4))) if many and c["S"] > 1 else c["q"] for _ in range(c["S"])]
    k = [max(n, int((c["k"] - c["q"]) * r.uniform(0.6, 1.4)) + n) if c["S"] > 1 else max(n, c["k"]) for n in q]
    return q, k


def _offsets(v):
    o = [0]
    for x in v:
        o.append(o[-1] + x)
    return o


def _layout(c):
    """Offsets on the host: seq_q, seq_k, len_k.  A cache has room for more tokens than it holds."""
    q, k = _lengths(c)
    return _offsets(q), _offsets([max(k) + 37] * c["S"]), k


def _dt(c):
    return torch.bfloat16 if c["dtype"] == BF16 else torch.float32


def frequencies(c):
    """Radians per position of each pair, fp64, on the host."""
    R, theta = c["width"], 10000.0
    if c["scaling"] == "base" and R > 2:
        theta *= c["factor"] ** (R / (R - 2))
    f = theta ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    elif c["scaling"] == "ramp":  # many turns within the original length of 8,192: kept; less than one: stretched
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * (keep + (1 - keep) / c["factor"])
    return f


def _own_frequencies(c):
    from gnn_sparse_attention_gb300 import binding as gb
    return gb.gattn_rotary_freqs(c["width"], 10000.0, c["scaling"], c["factor"], orig_len=8192, low=1.0, high=32.0, device="cuda")


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(2000 + seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    sq, sk, lk = _layout(case)
    S, H, Hkv, D, dt = case["S"], case["H"], case["Hkv"], case["D"], _dt(case)
    N, Nk = sq[-1], sk[-1]
    i32 = {"dtype": torch.int32, "device": dev}
    st = {"case": case, "seq_q": torch.tensor(sq, **i32), "seq_k": torch.tensor(sk, **i32), "len_k": torch.tensor(lk, **i32),
          "max_len_k": max(lk)}
    if case["op"] == "rotary":
        st["freqs"] = _own_frequencies(case) if own else frequencies(case).to(dev)
        st["amp"] = 1.0 + 0.1 * math.log(case["factor"])
        if case["packed"]:  # Q, K and V side by side, as one projection leaves them
            qkv = randn(N, (H + 2 * Hkv) * D).to(dt)
            st["Q"], st["K"] = qkv[:, :H * D].unflatten(1, (H, D)), qkv[:, H * D:(H + Hkv) * D].unflatten(1, (Hkv, D))
        else:
            st["Q"], st["K"] = randn(N, H, D).to(dt), randn(N, Hkv, D).to(dt)
        if case["train"]:
            st["dQ"], st["dK"] = randn(N, H, D).to(dt), randn(N, Hkv, D).to(dt)
        return st

    def rows(n):
        """K with channels that stand out and neighbours that are alike, V with rows that do."""
        K = randn(n, Hkv, D) * (1 + 3 * (randn(Hkv, D) > 1.5))
        K += torch.repeat_interleave(0.7 * randn(n // 64 + 1, Hkv, D), 64, 0)[:n]
        return K.to(dt), (randn(n, Hkv, D) * torch.exp(0.5 * randn(n, Hkv, 1)) + 0.2).to(dt)

    if case["op"] == "write":
        st["K"], st["V"] = rows(N)
        if case["packed"]:
            kv = torch.cat([st["K"].flatten(1), st["V"].flatten(1)], 1)
            st["K"], st["V"] = (t.unflatten(1, (Hkv, D)) for t in kv.chunk(2, 1))
        st["cache"] = _empty(Nk, Hkv, D, case["bits"], dev)
        if own:
            st["own"] = _own_cache(st["cache"], case)
        return st
    K, V = rows(Nk)
    st["cache"] = _empty(Nk, Hkv, D, case["bits"], dev)
    for a in range(0, Nk, 1 << 16):
        _store(st["cache"], slice(a, a + (1 << 16)), K[a:a + (1 << 16)], V[a:a + (1 << 16)], case["bits"])
    del K, V
    if own:
        st["own"] = _own_cache(st["cache"], case)
    if case["op"] == "sums":
        if case["renew"]:
            st["since"] = st["len_k"] - 1
            st["sums"] = _block_sums(st["cache"], st["seq_k"], st["len_k"] - 1, case)
        return st
    if case["op"] == "read":
        st["since"] = torch.zeros(S, **i32)
        st["seq_out"] = torch.tensor(_offsets(lk), **i32)
        st["rows"] = sum(lk)
        return st
    Q = randn(N, H, D)
    Q += torch.repeat_interleave(0.7 * randn(N // 64 + 1, H, D), 64, 0)[:N]
    st["Q"] = Q.to(dt)
    if case["topk"]:  # some blocks of the sequence each, the last one always among them
        idx = torch.full((N, Hkv, case["topk"]), -1, dtype=torch.int32, device=dev)
        for s in range(S):
            nb = -(-lk[s] // case["block"])
            n = min(nb, case["topk"])
            a = torch.rand(sq[s + 1] - sq[s], Hkv, nb, generator=g, device=dev)
            a[..., -1] = 2.0
            idx[sq[s]:sq[s + 1], :, :n] = a.topk(n, -1).indices.sort(-1).values.int()
        st["idx"] = idx
    return st


def _empty(Nk, Hkv, D, bits, dev):
    lev = [torch.zeros(Hkv, Nk, D * bits // 8, dtype=torch.uint8, device=dev) for _ in range(2)]
    return {"k": lev[0], "v": lev[1], "par": torch.zeros(Hkv, Nk, 4, dtype=torch.bfloat16, device=dev)}


def _own_cache(cache, case):
    from gnn_sparse_attention_gb300 import binding as gb
    return gb.Cache(cache["k"], cache["v"], cache["par"], case["bits"])


# ---------------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------------
def _to_bf16(x, up):
    """fp32 to bf16 values (as fp32), towards +inf or -inf."""
    b = x.contiguous().view(torch.int32)
    cut = b & -65536
    away = (b != cut) & ((b >= 0) if up else (b < 0))
    return (cut + 65536 * away.int()).view(torch.float32)


def _quantise(x, bits):
    """Levels (int32, like x) and bf16 [..., 2] (least value, step) of rows along the last dimension."""
    top = 2 ** bits - 1
    x = x.float()
    m = _to_bf16(x.amin(-1, keepdim=True), False)
    s = (0.5 * x.amax(-1, keepdim=True) - 0.5 * m).double() / (top / 2)
    s = _to_bf16(s.float(), True)
    s = torch.where(s < 2.0 ** -126, 0.0, s)
    inv = torch.where(s > 0, (1.0 / s.double()).float(), 0.0)
    c = -m * inv
    u = (x.double() * inv.double() + c.double()).float().round().clamp(0, top)  # one rounding to fp32, as an FMA
    return u.int(), torch.cat([m, s], -1).bfloat16()


def _pack(u, bits):
    u = u.to(torch.uint8)
    return u if bits == 8 else u[..., 0::2] | (u[..., 1::2] << 4)


def _unpack(b, bits):
    return b if bits == 8 else torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _values(lev, par, bits):
    """fp32 elements of rows: lev [..., D * bits / 8], par [..., 2]."""
    p = par.float()
    return p[..., :1] + p[..., 1:] * _unpack(lev, bits).float()


def _store(cache, at, K, V, bits):
    """Rows of K and V into the rows `at` of the cache."""
    par = []
    for x, lev in ((K, cache["k"]), (V, cache["v"])):
        u, p = _quantise(x, bits)
        lev[:, at] = _pack(u, bits).transpose(0, 1)
        par.append(p)
    cache["par"][:, at] = torch.cat(par, -1).transpose(0, 1)


def _rows_of(seq, N):
    """Sequence of each of N rows and its number within."""
    r = torch.arange(N, device=seq.device)
    s = torch.searchsorted(seq[1:].long(), r, right=True).clamp(max=seq.numel() - 2)
    return s, r - seq[s].long()


def _turn(x, cos, sin, c):
    R = c["width"]
    y = x.float()
    r = y[..., :R]
    a, b = (r[..., :R // 2], r[..., R // 2:]) if c["layout"] == "half" else (r[..., 0::2], r[..., 1::2])
    p, q = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat([p, q], -1) if c["layout"] == "half" else torch.stack([p, q], -1).flatten(-2)
    return torch.cat([turned, y[..., R:]], -1).to(x.dtype)


def _rotary_plain(st):
    c = st["case"]
    s, i = _rows_of(st["seq_q"], st["Q"].shape[0])
    lq = (st["seq_q"][1:] - st["seq_q"][:-1]).long()
    pos = i + (st["len_k"].long() - lq)[s]
    t = pos.double()[:, None] * st["freqs"]
    cos, sin = ((st["amp"] * f(t)).float()[:, None] for f in (torch.cos, torch.sin))
    res = {"Q": _turn(st["Q"], cos, sin, c), "K": _turn(st["K"], cos, sin, c)}
    if c["train"]:
        res["dQ"], res["dK"] = _turn(st["dQ"], cos, -sin, c), _turn(st["dK"], cos, -sin, c)
    return res


def _write_plain(st):
    c, cache, N = st["case"], st["cache"], st["K"].shape[0]
    s, i = _rows_of(st["seq_q"], N)
    lq = (st["seq_q"][1:] - st["seq_q"][:-1]).long()
    at = (st["seq_k"][:-1].long() + st["len_k"].long() - lq)[s] + i
    _store(cache, at, st["K"], st["V"], c["bits"])
    return _read_rows(cache, at, c)


def _read_rows(cache, at, c):
    res = {}
    for n, j in (("k", 0), ("v", 2)):
        x = _values(cache[n][:, at], cache["par"][:, at, j:j + 2], c["bits"])
        res[n.upper()] = x.transpose(0, 1).to(_dt(c)).contiguous()
    return res


def _read_plain(st):
    s, i = _rows_of(st["seq_out"], st["rows"])
    return _read_rows(st["cache"], st["seq_k"][:-1].long()[s] + i, st["case"])


def _blocks(seq_k, len_k, block, Nk):
    """The table of blocks: sequence, first row, first position and rows present (0: unused) of each."""
    S = seq_k.numel() - 1
    beg = seq_k[:-1].long()
    base = beg // block + torch.arange(S, device=seq_k.device)
    u = torch.arange(Nk // block + S, device=seq_k.device)
    s = (torch.searchsorted(base, u, right=True) - 1).clamp(min=0)
    pos = (u - base[s]) * block
    return s, beg[s] + pos, pos, (len_k.long()[s] - pos).clamp(0, block)


def _block_sums(cache, seq_k, len_k, c):
    blk, bits = c["block"], c["bits"]
    Nk = cache["k"].shape[1]
    _, row, _, n = _blocks(seq_k, len_k, blk, Nk)
    t = torch.arange(blk, device=row.device)
    ok = t < n[:, None]
    r = torch.where(ok, row[:, None] + t, 0)
    p = cache["par"][:, r, :2].double()
    x = p[..., :1] + p[..., 1:] * _unpack(cache["k"][:, r], bits).double()
    return (x * ok[:, :, None]).sum(2).transpose(0, 1).contiguous()


def _sums_plain(st):
    c = st["case"]
    new = _block_sums(st["cache"], st["seq_k"], st["len_k"], c)
    if "since" in st:  # only the blocks that hold positions from `since` on
        s, _, pos, _ = _blocks(st["seq_k"], st["len_k"], c["block"], st["cache"]["k"].shape[1])
        new = torch.where((pos + c["block"] > st["since"][s])[:, None, None], new, st["sums"])
    return {"sums": new}


def _attend_plain(st):
    c, cache, Q = st["case"], st["cache"], st["Q"]
    N, H, D = Q.shape
    Hkv, blk = c["Hkv"], c["block"]
    s, i = _rows_of(st["seq_q"], N)
    lk = st["len_k"].long()[s]
    limit = lk
    if c["causal"]:
        limit = i + lk - (st["seq_q"][1:] - st["seq_q"][:-1]).long()[s] + 1
    if c["topk"]:
        idx = st["idx"].long()
        pos = (idx[..., None] * blk + torch.arange(blk, device=idx.device)).flatten(2)
        ok = (idx >= 0).repeat_interleave(blk, 2) & (pos < limit[:, None, None])
    else:
        pos = torch.arange(st["max_len_k"], device=Q.device).expand(N, Hkv, -1)
        ok = pos < limit[:, None, None]
    row = torch.where(ok, st["seq_k"][:-1].long()[s][:, None, None] + pos, 0)
    g = torch.arange(Hkv, device=Q.device)[None, :, None]
    q = Q.float().reshape(N, Hkv, H // Hkv, D)
    k = _values(cache["k"][g, row], cache["par"][g, row, :2], c["bits"])
    sc = torch.where(ok[:, :, None], (q @ k.transpose(-1, -2)) / math.sqrt(D), float("-inf"))
    del k
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(m == float("-inf"), 0.0, m))
    l = p.sum(-1, keepdim=True)
    v = _values(cache["v"][g, row], cache["par"][g, row, 2:], c["bits"])
    o = (p / torch.where(l > 0, l, 1.0)) @ v
    return {"out": o.reshape(N, H, D).to(Q.dtype), "lse": (m + torch.log(l)).reshape(N, H)}


# ---------------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------------
def _run_own(st):
    from gnn_sparse_attention_gb300 import binding as gb
    c = st["case"]
    seqs = {"seq_q": st["seq_q"], "seq_k": st["seq_k"], "len_k": st["len_k"]}
    if c["op"] == "rotary":
        par = {"layout": c["layout"], "amp": st["amp"], **seqs}
        res = dict(zip(("Q", "K"), gb.gattn_rotary(st["Q"], st["freqs"], K=st["K"], **par)))
        if c["train"]:
            res["dQ"], res["dK"] = gb.gattn_rotary(st["dQ"], st["freqs"], K=st["dK"], inverse=True, **par)
        return res
    if c["op"] == "write":
        gb.gattn_cache_write(st["own"], st["K"], st["V"], **seqs)
        K, V = gb.gattn_cache_read(st["own"], rows=st["K"].shape[0], dtype=st["K"].dtype, **seqs)
        return {"K": K, "V": V}
    if c["op"] == "read":
        K, V = gb.gattn_cache_read(st["own"], st["seq_out"], st["seq_k"], len_k=st["len_k"], since=st["since"], rows=st["rows"], dtype=_dt(c))
        return {"K": K, "V": V}
    if c["op"] == "sums":
        return {"sums": gb.gattn_cache_sums(st["own"], st["seq_k"], c["block"], lens=st["len_k"], since=st.get("since"), sums=st.get("sums"))}
    out, lse = gb.gattn_cache_fwd(st["Q"], st["own"], idx=st.get("idx"), block=c["block"], causal=c["causal"], max_len_k=st["max_len_k"], **seqs)
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _run_own(state)
    return {"rotary": _rotary_plain, "write": _write_plain, "read": _read_plain, "sums": _sums_plain,
            "attend": _attend_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------------------------------------
# work of one pass
# ---------------------------------------------------------------------------------------------------------------------------
def work(case):
    es = 2 if case["dtype"] == BF16 else 4
    sq, sk, lk = _layout(case)
    N, H, Hkv, D = sq[-1], case["H"], case["Hkv"], case["D"]
    if case["op"] == "rotary":
        n = N * (H + Hkv) * (2 if case["train"] else 1)
        return {"bytes": 2 * n * D * es, "flops": 3 * n * case["width"]}
    lev = D * case["bits"] // 8 + 4  # bytes of a cached row of K or of V
    if case["op"] == "write":
        return {"bytes": 2 * N * Hkv * (2 * D * es + lev), "flops": 8 * N * Hkv * D}
    if case["op"] == "read":
        return {"bytes": 2 * sum(lk) * Hkv * (D * es + lev), "flops": 4 * sum(lk) * Hkv * D}
    blk = case["block"]
    if case["op"] == "sums":
        new = [(n - 1) % blk + 1 for n in lk] if case["renew"] else lk
        blocks = sum(-(-n // blk) for n in new)
        return {"bytes": Hkv * (sum(new) * lev + 8 * blocks * D), "flops": 2 * sum(new) * Hkv * D}
    pairs = keys = 0
    for a, n in zip([b - a for a, b in zip(sq, sq[1:])], lk):
        most = min(n, case["topk"] * blk) if case["topk"] else n
        pairs += a * most
        keys += min(n, a * most)
    moved = 2 * keys * Hkv * lev + 2 * N * H * D * es + 4 * N * H + 4 * N * Hkv * case["topk"]
    return {"bytes": moved, "flops": 4 * pairs * H * D}


# ---------------------------------------------------------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    """Sequence by sequence from the definition.  A row's least value, step and factors are rounded where the format says so."""
    st = prepare(case, seed)
    sq, sk, lk = _layout(case)
    if case["op"] == "rotary":
        return _exact_rotary(st, sq, lk)
    if case["op"] == "write":
        return {n: _exact_rounded(st[n].double(), case["bits"]) for n in ("K", "V")}
    cached = {}
    for n, j in (("K", 0), ("V", 2)):
        b = st["cache"][n.lower()].long()
        lev = b if case["bits"] == 8 else torch.stack((b.remainder(16), b.div(16, rounding_mode="floor")), 3).reshape(b.shape[0], b.shape[1], -1)
        par = st["cache"]["par"].double()
        cached[n] = lev * par[:, :, j + 1, None] + par[:, :, j, None]  # [Hkv, rows, D]
    if case["op"] == "read":
        return {n: torch.cat([x[:, a:a + k] for a, k in zip(sk, lk)], 1).transpose(0, 1) for n, x in cached.items()}
    if case["op"] == "sums":
        return _exact_sums(st, cached["K"], sk, lk)
    return _exact_attend(st, cached, sq, sk, lk)


def _exact_rotary(st, sq, lk):
    c = st["case"]
    R = c["width"]
    f = frequencies(c).to(st["Q"].device)
    pos = torch.cat([torch.arange(n - (b - a), n, dtype=torch.float64) for a, b, n in zip(sq, sq[1:], lk)]).to(f.device)
    turn = torch.polar(torch.full_like(pos, st["amp"])[:, None].expand(-1, R // 2), pos[:, None] * f)[:, None]

    def rotated(x, t):
        x = x.double()
        y = x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2) if c["layout"] == "half" else x[..., :R].unflatten(-1, (R // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(y.contiguous()) * t)
        z = (z.transpose(-1, -2) if c["layout"] == "half" else z).flatten(-2)
        return torch.cat([z, x[..., R:]], -1)

    res = {n: rotated(st[n], turn) for n in ("Q", "K")}
    if c["train"]:
        res.update({n: rotated(st[n], turn.conj()) for n in ("dQ", "dK")})
    return res


def _exact_rounded(x, bits):
    top = 2.0 ** bits - 1

    def bf16(v, up):  # the next of 8 significant bits
        e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -126)))
        unit = torch.exp2(e - 7)
        return (torch.ceil(v / unit) if up else torch.floor(v / unit)) * unit

    def f32(v):
        return v.float().double()

    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    m = bf16(lo, False)
    s = bf16(f32(f32(hi / 2 - m / 2) / (top / 2)), True)
    flat = s < 2.0 ** -126
    inv = torch.where(flat, 0.0, f32(1 / torch.where(flat, 1.0, s)))
    u = torch.round(f32(x * inv + f32(-m * inv))).clamp(0.0, top)
    return torch.where(flat, m, m + s * u)


def _exact_sums(st, K, sk, lk):
    c = st["case"]
    blk = c["block"]
    out = torch.zeros(sk[-1] // blk + c["S"], c["Hkv"], c["D"], dtype=torch.float64, device=K.device)
    if c["renew"]:
        out.copy_(st["sums"])
    for s in range(c["S"]):
        b0, nb = sk[s] // blk + s, -(-lk[s] // blk)
        for j in range((lk[s] - 1) // blk if c["renew"] else 0, nb):
            out[b0 + j] = K[:, sk[s] + j * blk:sk[s] + min(lk[s], (j + 1) * blk)].sum(1)
    return {"sums": out}


def _exact_attend(st, cached, sq, sk, lk):
    c = st["case"]
    Hkv, G, D, blk = c["Hkv"], c["H"] // c["Hkv"], c["D"], c["block"]
    Q = st["Q"].double()
    out, lse = torch.zeros_like(Q), torch.zeros(Q.shape[:2], dtype=torch.float64, device=Q.device)
    for s in range(c["S"]):
        n, a = lk[s], sq[s + 1] - sq[s]
        for i in range(a):
            ok = torch.ones(Hkv, n, dtype=torch.bool, device=Q.device)
            if c["topk"]:
                ids = st["idx"][sq[s] + i].long()
                nb = -(-n // blk)
                on = torch.zeros(Hkv, nb + 1, dtype=torch.bool, device=Q.device).scatter_(1, torch.where(ids < 0, nb, ids), True)
                ok = on[:, :nb].repeat_interleave(blk, 1)[:, :n]
            if c["causal"]:
                ok = ok & (torch.arange(n, device=Q.device) < i + n - a + 1)
            q = Q[sq[s] + i].reshape(Hkv, G, D)
            sc = torch.einsum("hgd,hnd->hgn", q, cached["K"][:, sk[s]:sk[s] + n]) / math.sqrt(D)
            sc = sc.masked_fill(~ok[:, None], -math.inf)
            z = torch.logsumexp(sc, -1)
            w = torch.exp(sc - torch.where(z > -math.inf, z, 0.0)[..., None])
            out[sq[s] + i] = torch.einsum("hgn,hnd->hgd", w, cached["V"][:, sk[s]:sk[s] + n]).reshape(Hkv * G, D)
            lse[sq[s] + i] = z.reshape(-1)
    return {"out": out, "lse": lse}
