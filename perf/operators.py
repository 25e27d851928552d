"""Workloads of the block-attention and norm operators: what is run, on which inputs, and how much work it is.

Three operators, each with a plain form (elementary torch operations in fp32, fp64 where a choice hangs on the value) and the
library's own calls:

* ``select``: sums of each block of keys, a score of every block against each query block, and the ``topk`` best blocks;
* ``attend``: softmax attention of each query block over the tokens of the blocks chosen for it (forward alone, as when serving,
  or forward and backward, as when training), over packed sequences of any lengths;
* ``norm``: ``h = res + alpha * gate * norm(x)`` and ``y = norm(h)``, the step between two blocks of a transformer.

Units.  Sequence s holds the query rows [seq_q[s], seq_q[s+1]) and the key rows [seq_k[s], seq_k[s] + len_k[s]).  Its queries are
cut into units of ``q_block`` rows and its keys into blocks of ``block`` rows; unit j of sequence s has the table row
seq_q[s] // q_block + s + j (without the ``+ s`` for one-row units), and block j the row seq_k[s] // block + s + j of the sums.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"


# ---------------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------------
def _attn(name, op, S, q, k, H, Hkv, D, topk, block, q_block, dtype=BF16, causal=False, train=False, ragged=True):
    c = {"op": op, "S": S, "q": q, "k": k, "H": H, "Hkv": Hkv, "D": D, "topk": topk, "block": block, "q_block": q_block,
         "dtype": dtype, "causal": causal, "train": train, "ragged": ragged}
    return {"name": name, **c} if name else c


def _norm(name, N, F, kind, dtype=BF16, gate="token", post=True, bias=False, train=False):
    c = {"op": "norm", "N": N, "F": F, "kind": kind, "dtype": dtype, "gate": gate, "post": post, "bias": bias, "train": train}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a few requests, each with one new token: the last block's sum is renewed and 16 blocks are chosen per head group
        _attn("select-token-8", "select", 8, 1, 4000, 32, 8, 128, 16, 64, 1),
        # a batch of graphs of unlike sizes, 65,536 nodes in all, heads of the block-model workload (8 x 64)
        _attn("select-graphs-64k", "select", 24, 2731, 2731, 8, 8, 64, 16, 64, 128),
        # the smallest serving call: one new token for each of 4 requests, keys shared by groups of 4 heads
        _attn("token-4", "attend", 4, 1, 2000, 32, 8, 128, 16, 64, 1),
        # a full serving batch with caches of about 8,000 tokens, of which each head group reads 32 blocks
        _attn("token-128", "attend", 128, 1, 8000, 32, 8, 128, 32, 64, 1),
        # a long prompt read at once, causal, shared heads
        _attn("prompt-32k", "attend", 1, 32768, 32768, 32, 8, 128, 32, 64, 128, causal=True, ragged=False),
        # training on a batch of graphs of unlike sizes, 8 heads of 64
        _attn("train-graphs-64k", "attend", 24, 2731, 2731, 8, 8, 64, 16, 64, 128, train=True),
        # training on two packed causal sequences, shared heads of 128
        _attn("train-causal-16k", "attend", 2, 8191, 8191, 16, 4, 128, 16, 64, 128, causal=True, train=True),
        # training in fp32 on small graphs with an odd number of nodes and narrow heads (4 x 32)
        _attn("train-f32-3k", "attend", 7, 429, 429, 4, 4, 32, 8, 32, 64, dtype=F32, train=True),
        # between two blocks while serving: 16 rows, latency alone
        _norm("norm-token-16", 16, 1024, "rms"),
        # a long prompt's rows, wide
        _norm("norm-prompt-8k", 8192, 4096, "rms", gate="channel"),
        # a training step over 131,072 nodes, LayerNorm with biases and a gate per node
        _norm("norm-train-128k", 131072, 1024, "layer", bias=True, train=True),
        # a training step with rows that are no multiple of 16 bytes, in fp32
        _norm("norm-train-odd", 20011, 515, "rms", dtype=F32, gate="channel", train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "token", "train", "prompt", "norm", "norm"])
    if op == "norm":
        F = rng.choice([64, 129, 256, 515, 768, 1000, 1024, 2048, 4096])
        N = _log(rng, 1, max(2, min(131072, (1 << 27) // F)))
        return _norm(None, N, F, rng.choice(["rms", "layer"]), rng.choice([BF16, BF16, F32]), rng.choice(["token", "channel", "none"]),
                     rng.random() < 0.8, rng.random() < 0.5, rng.random() < 0.6)
    D = rng.choice([16, 32, 64, 64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    block = rng.choice([16, 32, 64, 64, 128])
    if op == "token":
        S, G = _log(rng, 1, 128), rng.choice([1, 2, 4, 8])
        k = _log(rng, 1, min(16000, 1000000 // S))
        topk = rng.choice([1, 5, 16, 32]) if block <= 64 else rng.choice([1, 5, 16])
        return _attn(None, "attend", S, 1, k, Hkv * G, Hkv, D, topk, block, 1)
    if op == "select":
        if rng.random() < 0.5:
            S = _log(rng, 1, 64)
            return _attn(None, "select", S, 1, _log(rng, 1, min(16000, 500000 // S)), Hkv * 4, Hkv, D, rng.choice([1, 7, 16]), block, 1)
        S = _log(rng, 1, 40)
        n = _log(rng, 1, 40000 // S)
        return _attn(None, "select", S, n, n, Hkv, Hkv, D, rng.choice([1, 7, 16]), block, rng.choice([32, 64, 128]), rng.choice([BF16, F32]),
                     rng.random() < 0.5)
    G = rng.choice([1, 2, 4])
    S = _log(rng, 1, 20)
    f32 = op == "train" and rng.random() < 0.25
    n = max(1, _log(rng, 16, 3000 if f32 else 16000) // S)
    keys = rng.choice([256, 512, 1024])
    Hkv = min(Hkv, 4)
    return _attn(None, "attend", S, n, n, Hkv * G, Hkv, min(D, 64) if f32 else D, max(1, keys // block), block, rng.choice([64, 128]),
                 F32 if f32 else BF16, rng.random() < 0.5, op == "train")


# ---------------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------------
def _lengths(c):
    """Query and key lengths of each sequence: a function of the case alone."""
    r = random.Random(1000003 * c["S"] + 101 * c["k"] + c["q"])
    if not c["ragged"]:
        return [c["q"]] * c["S"], [c["k"]] * c["S"]
    k = [max(1, int(c["k"] * r.uniform(0.6, 1.4))) for _ in range(c["S"])]
    return ([1] * c["S"], k) if c["q"] == 1 and c["q_block"] == 1 else (list(k), k)


def _offsets(v):
    o = [0]
    for x in v:
        o.append(o[-1] + x)
    return o


def _layout(c):
    """Offsets on the host: seq_q, seq_k, lengths of the keys.  Serving keeps a cache with room for more tokens."""
    lq, lk = _lengths(c)
    if c["q_block"] == 1:
        room = (max(lk) + 255) // 256 * 256
        return _offsets(lq), _offsets([room] * c["S"]), lk
    return _offsets(lq), _offsets(lk), lk


def _dt(c):
    return torch.bfloat16 if c["dtype"] == BF16 else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(1000 + seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    if case["op"] == "norm":
        N, F, dt = case["N"], case["F"], _dt(case)
        st = {"case": case, "res": (2 * randn(N, F)).to(dt), "x": (0.5 * randn(N, F) + 0.1).to(dt), "gate": None, "alpha": 0.7, "eps": 1e-5}
        if case["gate"] != "none":
            st["gate"] = torch.sigmoid(randn(N, F)).to(dt) if case["gate"] == "token" else 0.5 + 0.1 * randn(F)
        for w, on in (("w_post", case["post"]), ("w_pre", True)):
            st[w] = 1 + 0.1 * randn(F) if on else None
        for b, on in (("b_post", case["post"]), ("b_pre", True)):
            st[b] = 0.1 * randn(F) if on and case["bias"] else None
        if case["train"]:
            st["dh"], st["dy"] = randn(N, F).to(dt), randn(N, F).to(dt)
        return st

    sq, sk, lk = _layout(case)
    H, Hkv, D, dt = case["H"], case["Hkv"], case["D"], _dt(case)
    Nq, Nk, S = sq[-1], sk[-1], case["S"]
    i32 = {"dtype": torch.int32, "device": dev}
    st = {"case": case, "seq_q": torch.tensor(sq, **i32), "seq_k": torch.tensor(sk, **i32),
          "len_k": torch.tensor(lk, **i32) if case["q_block"] == 1 else None, "max_len_k": max(lk)}
    # neighbouring rows are alike, as features and hidden states are, so that some blocks matter more than others
    K = randn(Nk, Hkv, D)
    K += torch.repeat_interleave(0.7 * randn(Nk // 64 + 1, Hkv, D), 64, 0)[:Nk]
    Q = randn(Nq, H, D)
    Q += torch.repeat_interleave(0.7 * randn(Nq // 64 + 1, H, D), 64, 0)[:Nq]
    st["Q"], st["K"] = Q.to(dt), K.to(dt)
    if case["op"] == "select":
        if case["q_block"] == 1:  # the cache's sums, kept from token to token: all but the newest token's block are up to date
            st["since"] = st["len_k"] - 1
            st["sums"] = _sums(st["K"], st["seq_k"], st["len_k"] - 1, case["block"])
        return st
    st["V"] = randn(Nk, Hkv, D).to(dt)
    st["idx"] = _select(st["Q"], _sums(st["K"], st["seq_k"], st["len_k"], case["block"]), st)
    if case["train"]:
        st["dout"] = randn(Nq, H, D).to(dt)
    return st


# ---------------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------------
def _pieces(seq, lens, per, N):
    """The table of pieces of `per` rows: sequence, first row, first position in the sequence, rows present (0: unused)."""
    S = seq.numel() - 1
    one = 0 if per == 1 else 1
    beg = seq[:-1].long()
    ln = (seq[1:] - seq[:-1]).long() if lens is None else lens.long()
    base = beg // per + one * torch.arange(S, device=seq.device)
    u = torch.arange(N // per + one * S, device=seq.device)
    s = (torch.searchsorted(base, u, right=True) - 1).clamp(min=0)
    pos = (u - base[s]) * per
    return s, beg[s] + pos, pos, (ln[s] - pos).clamp(0, per)


def _sums(x, seq, lens, per):
    """fp64 sums of the rows of each piece: [pieces, heads, D]."""
    N = x.shape[0]
    s, row, pos, n = _pieces(seq, lens, per, N)
    r = row[:, None] + torch.arange(per, device=x.device)
    ok = torch.arange(per, device=x.device) < n[:, None]
    got = x[torch.where(ok, r, 0)].double()
    return (got * ok[:, :, None, None]).sum(1)


def _select(Q, sums, st):
    c = st["case"]
    G, qb, blk, topk = c["H"] // c["Hkv"], c["q_block"], c["block"], c["topk"]
    lens = (st["seq_k"][1:] - st["seq_k"][:-1]) if st["len_k"] is None else st["len_k"]
    us, _, upos, un = _pieces(st["seq_q"], None, qb, Q.shape[0])
    bs, _, bpos, bn = _pieces(st["seq_k"], lens, blk, st["K"].shape[0])
    q = _sums(Q, st["seq_q"], None, qb)
    q = q.reshape(q.shape[0], c["Hkv"], G, c["D"]).sum(2)
    score = torch.einsum("ugd,bgd->ugb", q, sums) / bn.clamp(min=1)
    ok = (us[:, None] == bs) & (un[:, None] > 0) & (bn > 0)
    if c["causal"]:
        lq = (st["seq_q"][1:] - st["seq_q"][:-1]).long()
        first = upos + (lens.long() - lq)[us]
        last = first + un - 1
        ok = ok & (bpos <= last[:, None])
        near = bpos + blk > first[:, None]
        score = torch.where(near[:, None], torch.full_like(score, float("inf")), score)
    score = torch.where(ok[:, None], score, torch.full_like(score, float("-inf")))
    best, at = torch.sort(score, dim=-1, descending=True, stable=True)
    best, at = best[..., :topk], at[..., :topk]
    none = torch.iinfo(torch.int32).max
    ids = torch.where(best > float("-inf"), (bpos // blk)[at], none)
    if ids.shape[-1] < topk:
        ids = torch.nn.functional.pad(ids, (0, topk - ids.shape[-1]), value=none)
    ids = torch.sort(ids, dim=-1).values
    return torch.where(ids == none, -1, ids).to(torch.int32)


def _gather(st):
    """Rows and masks of the attention: query rows [U, q_block], key rows and allowed pairs per unit and head group."""
    c = st["case"]
    Nq, Nk, blk = st["Q"].shape[0], st["K"].shape[0], c["block"]
    lens = ((st["seq_k"][1:] - st["seq_k"][:-1]) if st["len_k"] is None else st["len_k"]).long()
    us, urow, upos, un = _pieces(st["seq_q"], None, c["q_block"], Nq)
    t = torch.arange(c["q_block"], device=us.device)
    qok = t < un[:, None]
    qrow = torch.where(qok, urow[:, None] + t, Nq)                                   # row Nq: none
    idx = st["idx"].long()
    pos = (idx[..., None] * blk + torch.arange(blk, device=us.device)).flatten(2)       # [U, Hkv, keys]
    kok = (idx >= 0).repeat_interleave(blk, 2) & (pos < lens[us][:, None, None])
    krow = torch.where(kok, st["seq_k"][:-1].long()[us][:, None, None] + pos, Nk)
    ok = (kok[:, :, None, :] & qok[:, None, :, None])
    if c["causal"]:
        lq = (st["seq_q"][1:] - st["seq_q"][:-1]).long()
        qpos = upos[:, None] + t + (lens - lq)[us][:, None]
        ok = ok & (pos[:, :, None, :] <= qpos[:, None, :, None])
    return qrow, krow, ok


def _take_q(x, qrow, Hkv):
    """[Nq, H, ...] -> fp32 [U, Hkv, q_block * G, ...]"""
    U, qb = qrow.shape
    y = x[qrow.clamp(max=x.shape[0] - 1)].float()
    y = y.reshape(U, qb, Hkv, x.shape[1] // Hkv, -1).transpose(1, 2)
    return y.reshape(U, Hkv, qb * (x.shape[1] // Hkv), -1)


def _put_q(y, qrow, N, H, dtype):
    U, qb = qrow.shape
    Hkv, D = y.shape[1], y.shape[-1]
    out = torch.zeros(N + 1, H, D, device=y.device, dtype=torch.float32)
    out[qrow] = y.reshape(U, Hkv, qb, H // Hkv, D).transpose(1, 2).reshape(U, qb, H, D)
    return out[:N].to(dtype)


def _take_k(x, krow):
    g = torch.arange(x.shape[1], device=x.device)[None, :, None]
    return x[krow.clamp(max=x.shape[0] - 1), g].float()


def _put_k(y, krow, N, dtype):
    Hkv, D = y.shape[1], y.shape[-1]
    g = torch.arange(Hkv, device=y.device)[None, :, None]
    out = torch.zeros((N + 1) * Hkv, D, device=y.device, dtype=torch.float32)
    out.index_add_(0, (krow * Hkv + g).flatten(), y.reshape(-1, D))
    return out.reshape(N + 1, Hkv, D)[:N].to(dtype)


def _attend(st):
    c = st["case"]
    Q, K, V = st["Q"], st["K"], st["V"]
    H, Hkv, G = c["H"], c["Hkv"], c["H"] // c["Hkv"]
    scale = 1.0 / math.sqrt(c["D"])
    qrow, krow, ok = _gather(st)
    ok = ok.repeat_interleave(G, 2)
    q, k, v = _take_q(Q, qrow, Hkv), _take_k(K, krow), _take_k(V, krow)
    s = torch.where(ok, (q @ k.transpose(-1, -2)) * scale, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    del s
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l > 0, l, 1.0)
    o = p @ v
    lse = torch.where(l > 0, m + torch.log(l), float("-inf"))
    res = {"out": _put_q(o, qrow, Q.shape[0], H, Q.dtype), "lse": _put_q(lse, qrow, Q.shape[0], H, torch.float32)[..., 0]}
    if not c["train"]:
        return res
    do = _take_q(st["dout"], qrow, Hkv) * (qrow < Q.shape[0]).repeat_interleave(G, 1)[:, None, :, None]
    ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True)) * scale
    res["dQ"] = _put_q(ds @ k, qrow, Q.shape[0], H, Q.dtype)
    res["dK"] = _put_k(ds.transpose(-1, -2) @ q, krow, K.shape[0], K.dtype)
    res["dV"] = _put_k(p.transpose(-1, -2) @ do, krow, K.shape[0], K.dtype)
    return res


def _normed(x, w, b, kind, eps):
    """(norm(x), x-hat, 1 / deviation) of fp32 rows."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    y = x * r * w
    return (y if b is None else y + b), x * r, r


def _normed_bwd(dy, xh, r, w, kind):
    g = dy * w
    dx = g - xh * (g * xh).mean(-1, keepdim=True)
    if kind == "layer":
        dx = dx - g.mean(-1, keepdim=True)
    return dx * r


def _norm_plain(st):
    c = st["case"]
    kind, eps, alpha, dt = c["kind"], st["eps"], st["alpha"], st["res"].dtype
    x, gate = st["x"].float(), None if st["gate"] is None else st["gate"].float()
    u = x
    if c["post"]:
        u, xh, rx = _normed(x, st["w_post"], st["b_post"], kind, eps)
    h = st["res"].float() + alpha * (u if gate is None else gate * u)
    y, hh, rh = _normed(h, st["w_pre"], st["b_pre"], kind, eps)
    res = {"h": h.to(dt), "y": y.to(dt)}
    if not c["train"]:
        return res
    dy = st["dy"].float()
    dh = st["dh"].float() + _normed_bwd(dy, hh, rh, st["w_pre"], kind)
    res["dres"] = dh.to(dt)
    res["dw_pre"] = (dy * hh).sum(0)
    if c["bias"]:
        res["db_pre"] = dy.sum(0)
    du = alpha * (dh if gate is None else gate * dh)
    if c["gate"] == "token":
        res["dgate"] = (alpha * dh * u).to(dt)
    elif c["gate"] == "channel":
        res["dgate"] = (alpha * dh * u).sum(0)
    if c["post"]:
        res["dw_post"] = (du * xh).sum(0)
        if c["bias"]:
            res["db_post"] = du.sum(0)
        du = _normed_bwd(du, xh, rx, st["w_post"], kind)
    res["dx"] = du.to(dt)
    return res


def _select_plain(st):
    c = st["case"]
    if "since" not in st:
        sums = _sums(st["K"], st["seq_k"], st["len_k"], c["block"])
    else:  # only the blocks that hold positions from `since` on
        new = _sums(st["K"], st["seq_k"], st["len_k"], c["block"])
        s, _, pos, _ = _pieces(st["seq_k"], st["len_k"], c["block"], st["K"].shape[0])
        sums = torch.where((pos + c["block"] > st["since"][s])[:, None, None], new, st["sums"])
    return {"sums": sums, "idx": _select(st["Q"], sums, st)}


# ---------------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------------
def _run_own(st):
    from gnn_sparse_attention_gb300 import binding as gb
    c = st["case"]
    if c["op"] == "norm":
        par = {"w_post": st["w_post"], "b_post": st["b_post"], "w_pre": st["w_pre"], "b_pre": st["b_pre"], "alpha": st["alpha"],
               "kind": c["kind"]}
        h, y, stats = gb.gattn_norm_fwd(st["res"], st["x"], st["gate"], eps=st["eps"], **par)
        res = {"h": h, "y": y}
        if c["train"]:
            got = gb.gattn_norm_bwd(st["res"], stats, st["dh"], st["dy"], st["x"], st["gate"], **par)
            res.update({k: v for k, v in got.items() if v is not None})
        return res
    lay = {"block": c["block"], "q_block": c["q_block"], "len_k": st["len_k"], "causal": c["causal"]}
    if c["op"] == "select":
        sums = gb.gattn_block_sums(st["K"], st["seq_k"], c["block"], lens=st["len_k"], since=st.get("since"), sums=st.get("sums"))
        idx = gb.gattn_block_select(st["Q"], sums, st["seq_q"], st["seq_k"], c["topk"], nk=st["K"].shape[0], max_len_k=st["max_len_k"], **lay)
        return {"sums": sums, "idx": idx}
    out, lse = gb.gattn_block_fwd(st["Q"], st["K"], st["V"], st["idx"], st["seq_q"], st["seq_k"], **lay)
    res = {"out": out, "lse": lse}
    if c["train"]:
        res["dQ"], res["dK"], res["dV"] = gb.gattn_block_bwd(st["Q"], st["K"], st["V"], st["idx"], st["seq_q"], st["seq_k"], out,
                                                             st["dout"], lse, **lay)
    return res


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return _norm_plain(state) if op == "norm" else _select_plain(state) if op == "select" else _attend(state)


# ---------------------------------------------------------------------------------------------------------------------------
# work of one pass
# ---------------------------------------------------------------------------------------------------------------------------
def work(case):
    es = 2 if case["dtype"] == BF16 else 4
    if case["op"] == "norm":
        n = case["N"] * case["F"]
        tok = 1 if case["gate"] == "token" else 0
        moved = (4 + tok) * n * es                               # res, x, gate in; h, y out
        flops = 20 * n
        if case["train"]:
            moved += (4 + tok + 2 + tok) * n * es                # res, x, dh, dy, gate in; dres, dx, dgate out
            flops += 40 * n
        return {"bytes": moved, "flops": flops}
    sq, sk, lk = _layout(case)
    H, Hkv, D, blk, qb = case["H"], case["Hkv"], case["D"], case["block"], case["q_block"]
    lq = [b - a for a, b in zip(sq, sq[1:])]
    if case["op"] == "select":
        U = sum(-(-n // qb) for n in lq)
        B = sum(-(-n // blk) for n in lk)
        kin = Hkv * D * (es * blk * len(lk) + 8 * B) if qb == 1 else Hkv * D * (es * sum(lk) + 8 * B)
        pairs = sum(-(-a // qb) * -(-b // blk) for a, b in zip(lq, lk))
        return {"bytes": sq[-1] * H * D * es + kin + 4 * U * Hkv * case["topk"], "flops": 2 * pairs * Hkv * D}
    pairs, read = 0, 0
    for a, b in zip(lq, lk):
        most = min(case["topk"] * blk, b)
        read += min(b, most * -(-a // qb))
        if case["causal"]:
            pairs += sum(min(most, u * qb + b - a + qb // 2) * min(qb, a - u * qb) for u in range(-(-a // qb)))
        else:
            pairs += a * most
    qrows, krows = sq[-1] * H * D * es, read * Hkv * D * es
    moved, flops = 2 * qrows + 2 * krows + 4 * sq[-1] * H, 4 * pairs * H * D
    if case["train"]:
        moved += 4 * qrows + 4 * krows + 4 * sq[-1] * H          # Q, out, dout, K, V, lse in; dQ, dK, dV out
        flops += 10 * pairs * H * D
    return {"bytes": moved, "flops": flops}


# ---------------------------------------------------------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    """Sequence by sequence and head by head from the definition, with dense masks.  None where that takes too long."""
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(st)
    sq, sk, lk = _layout(case)
    if case["op"] == "select":
        return _exact_select(st, sq, sk, lk)
    cost = sum(a * b for a, b in zip([y - x for x, y in zip(sq, sq[1:])], lk)) * case["H"] * case["D"] * (14 if case["train"] else 4)
    if cost > 6e12:
        return None
    return _exact_attend(st, sq, sk, lk)


def _exact_attend(st, sq, sk, lk):
    c = st["case"]
    G, blk, qb, D = c["H"] // c["Hkv"], c["block"], c["q_block"], c["D"]
    dev = st["Q"].device
    f64 = {"dtype": torch.float64, "device": dev}
    out, dQ = torch.zeros(*st["Q"].shape, **f64), torch.zeros(*st["Q"].shape, **f64)
    lse = torch.full(st["Q"].shape[:2], 0.0, **f64)
    dK, dV = torch.zeros(*st["K"].shape, **f64), torch.zeros(*st["K"].shape, **f64)
    for s in range(c["S"]):
        q0, q1, k0, n = sq[s], sq[s + 1], sk[s], lk[s]
        if q1 == q0:
            continue
        units = -(-(q1 - q0) // qb)
        u0 = q0 // qb + (s if qb > 1 else 0)
        nb = -(-n // blk)
        for g in range(c["Hkv"]):
            chosen = torch.zeros(units, nb + 1, dtype=torch.bool, device=dev)
            ids = st["idx"][u0:u0 + units, g].long()
            chosen.scatter_(1, torch.where(ids < 0, nb, ids), True)
            ok = chosen[:, :nb].repeat_interleave(blk, 1)[:, :n].repeat_interleave(qb, 0)[:q1 - q0]
            if c["causal"]:
                i = torch.arange(q1 - q0, device=dev)[:, None] + n - (q1 - q0)
                ok = ok & (torch.arange(n, device=dev) <= i)
            some = ok.any(1)
            k, v = st["K"][k0:k0 + n, g].double(), st["V"][k0:k0 + n, g].double()
            for h in range(g * G, (g + 1) * G):
                q = st["Q"][q0:q1, h].double()
                sc = (q @ k.T / math.sqrt(D)).masked_fill_(~ok, -math.inf)
                z = torch.logsumexp(sc, 1)
                p = torch.exp(sc - torch.where(some, z, 0.0)[:, None])
                o = p @ v
                out[q0:q1, h], lse[q0:q1, h] = o, z
                if c["train"]:
                    do = st["dout"][q0:q1, h].double()
                    ds = p * (do @ v.T - (do * o).sum(1, keepdim=True)) / math.sqrt(D)
                    dQ[q0:q1, h] = ds @ k
                    dK[k0:k0 + n, g] += ds.T @ q
                    dV[k0:k0 + n, g] += p.T @ do
    res = {"out": out, "lse": lse}
    if c["train"]:
        res.update(dQ=dQ, dK=dK, dV=dV)
    return res


def _exact_select(st, sq, sk, lk):
    c = st["case"]
    G, blk, qb, topk = c["H"] // c["Hkv"], c["block"], c["q_block"], c["topk"]
    one = 1 if qb > 1 else 0
    dev = st["Q"].device
    B = st["K"].shape[0] // blk + c["S"]
    U = st["Q"].shape[0] // qb + one * c["S"]
    sums = torch.zeros(B, c["Hkv"], c["D"], dtype=torch.float64, device=dev)
    idx = torch.full((U, c["Hkv"], topk), -1, dtype=torch.int32, device=dev)
    for s in range(c["S"]):
        n, a = lk[s], sq[s + 1] - sq[s]
        nb, b0 = -(-n // blk), sk[s] // blk + s
        pad = torch.zeros(nb * blk, c["Hkv"], c["D"], dtype=torch.float64, device=dev)
        pad[:n] = st["K"][sk[s]:sk[s] + n].double()
        sums[b0:b0 + nb] = pad.view(nb, blk, c["Hkv"], c["D"]).sum(1)
        units = -(-a // qb)
        if not units:
            continue
        count = torch.full((nb,), float(blk), dtype=torch.float64, device=dev)
        count[-1] = n - (nb - 1) * blk
        q = torch.zeros(units * qb, c["H"], c["D"], dtype=torch.float64, device=dev)
        q[:a] = st["Q"][sq[s]:sq[s + 1]].double()
        q = q.view(units, qb, c["Hkv"], G, c["D"]).sum((1, 3))
        score = torch.einsum("ugd,bgd->ugb", q, sums[b0:b0 + nb] / count[:, None, None])
        rank = torch.arange(nb, device=dev)
        if c["causal"]:
            lo = torch.arange(units, device=dev) * qb + n - a
            hi = torch.minimum(lo + qb, torch.tensor(n, device=dev)) - 1
            score = score.masked_fill((rank * blk + blk > lo[:, None])[:, None], math.inf)
            score = score.masked_fill((rank * blk > hi[:, None])[:, None], -math.inf)
        order = torch.argsort(score, dim=-1, descending=True, stable=True)[..., :topk]
        kept = torch.gather(score, -1, order) > -math.inf
        order = torch.where(kept, order, nb).sort(-1).values
        idx[sq[s] // qb + one * s:][:units, :, :order.shape[-1]] = torch.where(order == nb, -1, order).int()
    return {"sums": sums, "idx": idx}


def _exact_norm(st):
    """Through autograd in fp64, from the two lines that define the operator."""
    c = st["case"]
    leaf = {k: st[k].double().requires_grad_() for k in ("res", "x", "gate", "w_post", "b_post", "w_pre", "b_pre") if st[k] is not None}

    def norm(x, w, b):
        z = x - x.mean(-1, keepdim=True) if c["kind"] == "layer" else x
        z = z / torch.sqrt(z.pow(2).mean(-1, keepdim=True) + st["eps"]) * w
        return z if b is None else z + b

    u = norm(leaf["x"], leaf["w_post"], leaf.get("b_post")) if c["post"] else leaf["x"]
    h = leaf["res"] + st["alpha"] * (leaf["gate"] * u if "gate" in leaf else u)
    y = norm(h, leaf["w_pre"], leaf.get("b_pre"))
    res = {"h": h.detach(), "y": y.detach()}
    if c["train"]:
        torch.autograd.backward([h, y], [st["dh"].double(), st["dy"].double()])
        res.update({"d" + k: v.grad for k, v in leaf.items()})
    return res
