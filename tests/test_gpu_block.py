"""Block selection and block attention on the GPU against their definition in
64 bits (tests/block_ref.py states the bounds)."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu

from gnn_sparse_attention_gb300 import binding as gb  # noqa: E402
from tests import block_ref as ref  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def random_idx(seed, sq, lk, qb, Hkv, topk, block):
    """Random lists: unsorted, with repeats, entries outside the sequence and empty units."""
    g = torch.Generator().manual_seed(seed)
    S = len(sq) - 1
    idx = torch.full((ref.units(sq[-1], S, qb), Hkv, topk), -1, dtype=torch.int32)
    for s in range(S):
        nb = -(-lk[s] // block)
        for j in range(-(-(sq[s + 1] - sq[s]) // qb)):
            ids = torch.randint(-2, nb + 2, (Hkv, topk), generator=g, dtype=torch.int32)
            if int(torch.randint(0, 6, (1,), generator=g)) == 0:
                ids.fill_(-1)
            idx[ref.table_row(sq[s], s, qb) + j] = ids
    return idx.to(DEV)


def run(seed, lq, lk, H, Hkv, D, dtype, block, qb, topk, causal=False, room=0, extra=0,
        train=True, idx=None, scale=0.0, edit=None):
    """One call of the forward (and backward) with canaries in every row of no sequence."""
    sq = ref.offsets(lq)
    sk = ref.offsets([n + room for n in lk])
    Nq, Nk = sq[-1] + extra, sk[-1] + extra
    dt = DT[dtype]
    Q, K, V = (randn(seed + i, n, h, D, dtype=dt) for i, (n, h) in
               enumerate([(Nq, H), (Nk, Hkv), (Nk, Hkv)]))
    nan = float("nan")
    for s in range(len(lk)):          # rows of no sequence must not matter
        K[sk[s] + lk[s]:sk[s + 1]] = nan
        V[sk[s] + lk[s]:sk[s + 1]] = nan
    Q[sq[-1]:], K[sk[-1]:], V[sk[-1]:] = nan, nan, nan
    if edit:
        edit(Q, K, V, sq, sk)
    if idx is None:
        idx = random_idx(seed, sq, lk, qb, Hkv, topk, block)
        if Nq // qb > sq[-1] // qb:
            idx = torch.cat([idx, torch.zeros(Nq // qb - sq[-1] // qb, Hkv, topk,
                                              dtype=torch.int32, device=DEV)])
    kw = {"block": block, "q_block": qb, "causal": causal, "scale": scale,
          "len_k": i32(lk) if room else None}
    out = torch.full((Nq, H, D), 7.0, device=DEV, dtype=dt)
    lse = torch.full((Nq, H), 7.0, device=DEV)
    gb.gattn_block_fwd(Q, K, V, idx, i32(sq), i32(sk), out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    gb.gattn_block_check_errors()
    dout = randn(seed + 9, Nq, H, D, dtype=dt)
    dout[sq[-1]:] = nan
    r = ref.attention(Q, K, V, idx, sq, sk, block, qb, scale, causal, lk,
                      dout if train else None)
    ref.check(out, r, "out", 7.0)
    ref.check(lse, r, "lse", 7.0)
    if not train:
        return Q, K, V, idx, out, lse, r
    grads = [torch.full(t.shape, 7.0, device=DEV, dtype=dt) for t in (Q, K, V)]
    gb.gattn_block_bwd(Q, K, V, idx, i32(sq), i32(sk), out, dout, lse, dQ=grads[0], dK=grads[1],
                       dV=grads[2], **kw)
    torch.cuda.synchronize()
    gb.gattn_block_check_errors()
    for t, n in zip(grads, ("dQ", "dK", "dV")):
        ref.check(t, r, n, 7.0)
    return Q, K, V, idx, out, lse, grads


HEADS = [("bf16", 64, 4, 4), ("bf16", 128, 8, 2), ("bf16", 32, 2, 2), ("bf16", 16, 2, 1),
         ("bf16", 8, 4, 4), ("f32", 32, 4, 4), ("f32", 128, 4, 1), ("f32", 4, 2, 2),
         ("f32", 64, 2, 1)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,D,H,Hkv", HEADS)
def test_head_layouts(dtype, D, H, Hkv, causal):
    run(1, [130, 1, 0, 257], [200, 1, 40, 257], H, Hkv, D, dtype, 64, 64, 3, causal, extra=5)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block,qb,topk", [(16, 128, 9), (32, 32, 7), (128, 128, 2), (64, 16, 1),
                                           (128, 64, 5), (64, 1, 4), (16, 2, 33), (32, 8, 128)])
def test_blocks_and_units(block, qb, topk, dtype, causal):
    run(2, [100, 3, 261], [333, 130, 261], 4, 2, 64, dtype, block, qb, topk, causal, room=13,
        extra=70)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 2, 8, 32, 128])
def test_shared_heads(G, dtype):
    run(3, [65, 130], [65, 130], 2 * G, 2, 16, dtype, 64, 16, 2, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lk", [[1], [63, 64, 65, 0], [5000, 1, 129], [2048] * 3])
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (4, 4, 64), (32, 1, 64)])
def test_one_token(lk, H, Hkv, D, dtype):
    run(4, [1] * len(lk), lk, H, Hkv, D, dtype, 64, 1, 16, True, room=100, train=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_token_backward(dtype):
    run(5, [1] * 5, [70, 1, 300, 64, 129], 8, 2, 64, dtype, 32, 1, 6, True, room=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lq,lk", [([0, 0], [0, 0]), ([0], [100]), ([100], [0]), ([1], [1]),
                                   ([300], [40]), ([7, 0, 9], [0, 5, 9])])
def test_small_and_empty(lq, lk, dtype):
    # more queries than keys: with causal the first ones see nothing
    run(6, lq, lk, 4, 2, 64, dtype, 64, 64, 2, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_units_of_one_block(dtype):
    """Every unit chooses block 0: its gradients are split over work items and joined."""
    lq = [6400]
    idx = torch.zeros(ref.units(6400, 1, 16), 1, 1, dtype=torch.int32, device=DEV)
    run(7, lq, [300], 2, 1, 64, dtype, 64, 16, 1, idx=idx)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,H,Hkv,D", [("bf16", 8, 8, 64), ("bf16", 16, 4, 128),
                                           ("bf16", 8, 2, 64), ("bf16", 16, 2, 32),
                                           ("f32", 4, 4, 32)])
def test_many_tiles(dtype, H, Hkv, D, causal):
    """Ten tiles and more per CTA, with empty sequences between: buffers are used in turn; the
    results of repeated calls are equal."""
    lens = [(137 * i) % 900 + 1 if i % 5 else 0 for i in range(24)]
    sq = ref.offsets(lens)
    idx = random_idx(12, sq, lens, 64, Hkv, 6, 32)
    first = run(12, lens, lens, H, Hkv, D, dtype, 32, 64, 6, causal, idx=idx)
    Q, K, V = first[:3]
    for _ in range(20):
        out, lse = gb.gattn_block_fwd(Q, K, V, idx, i32(sq), i32(sq), 32, 64, causal=causal)
        assert torch.equal(out, first[4]) and torch.equal(lse, first[5])
    gb.gattn_block_check_errors()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_unseen_values_do_not_matter(bad, dtype):
    """Non-finite keys and values in a chosen block, behind the causal mask of most rows."""
    def edit(Q, K, V, sq, sk):
        K[100] = bad
        V[100, :, 3] = bad
        V[90, :, 5] = bad

    idx = torch.arange(2, dtype=torch.int32, device=DEV).repeat(ref.units(128, 1, 64), 2, 1)
    sq, dt = [0, 128], DT[dtype]
    Q, K, V = (randn(8 + i, 128, 2 if i else 4, 64, dtype=dt) for i in range(3))
    edit(Q, K, V, sq, sq)
    out, lse = gb.gattn_block_fwd(Q, K, V, idx, i32(sq), i32(sq), 64, 64, causal=True)
    torch.cuda.synchronize()
    r = ref.attention(Q, K, V, idx, sq, sq, 64, 64, causal=True)
    o, w = out.double(), r["out"]
    seen = torch.isfinite(w[:100])
    assert (torch.isfinite(o[:100]) == seen).all()
    assert not seen[90:, :, 5].any() and seen[:90].all()
    # the bound of out with sum p |v| <= max |v| over the finite values (the weights sum to 1);
    # the reference's own bound is not finite here
    big = V.double()[torch.isfinite(V)].abs().max()
    c = (2 * 128 + 64 + 32) * 2.0 ** -24
    err = (Q.double().abs().sum(-1).max() * K.double()[:100].abs().max()) / 8 * c
    tol = ref.UNIT[dt] * w[:100].abs() + (ref.UNIT[dt] + c + 2 * err) * big
    assert ((o[:100] - w[:100]).abs()[seen] <= tol[seen]).all()
    if math.isinf(bad):
        assert (o[90:100, :, 5] == bad).all()
    assert not torch.isfinite(o[100:, :, 3]).any()


def test_results_do_not_vary():
    a = run(11, [300, 200], [300, 200], 4, 2, 64, "bf16", 64, 64, 4, True)
    b = run(11, [300, 200], [300, 200], 4, 2, 64, "bf16", 64, 64, 4, True)
    assert torch.equal(a[4], b[4]) and torch.equal(a[5], b[5])
    assert all(torch.equal(x, y) for x, y in zip(a[6], b[6]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_against_differences(dtype):
    """Directional derivative of sum(out * w) along random directions, by central differences
    of the fp64 definition at the kernel's own (rounded) inputs."""
    sq = [0, 70, 150]
    H, Hkv, D = 4, 2, 32
    dt = DT[dtype]
    Q, K, V = (randn(20 + i, 150, h, D, dtype=dt) for i, h in enumerate((H, Hkv, Hkv)))
    idx = random_idx(3, sq, [70, 80], 32, Hkv, 2, 32)
    kw = {"block": 32, "q_block": 32, "causal": True}
    out, lse = gb.gattn_block_fwd(Q, K, V, idx, i32(sq), i32(sq), **kw)
    w = randn(30, 150, H, D, dtype=dt)
    grads = gb.gattn_block_bwd(Q, K, V, idx, i32(sq), i32(sq), out, w, lse, **kw)
    r = ref.attention(Q, K, V, idx, sq, sq, 32, 32, causal=True, dout=w)
    h = 1e-5
    for n, (x, g) in enumerate(zip((Q, K, V), grads)):
        v = randn(40 + n, *x.shape).double()

        def loss(e):
            t = [y.double() + (e * v if y is x else 0) for y in (Q, K, V)]
            ref.UNIT[torch.float64] = 0.0
            return (ref.attention(*t, idx, sq, sq, 32, 32, causal=True)["out"] * w.double()).sum()

        diff = ((loss(h) - loss(-h)) / (2 * h)).item()
        name = ("dQ", "dK", "dV")[n]
        tol = (r[name + "_tol"] * v.abs()).sum().item()
        got = (g.double() * v).sum().item()
        # truncation of the difference: about h^2 times third derivatives of size |v|^3
        assert abs(got - diff) <= tol + 1e-6 * (1 + abs(diff)), (name, got, diff, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lists_kept_head_by_head_or_shared(dtype):
    """idx as [Hkv, units, topk] storage, with room behind each list, and one list for all heads."""
    sq, dt = [0, 150, 200], DT[dtype]
    Q, K, V, G = (randn(140 + i, 200, 4 if i in (0, 3) else 2, 64, dtype=dt) for i in range(4))
    kw = {"block": 32, "q_block": 32, "causal": True}
    idx = random_idx(9, sq, [150, 50], 32, 2, 4, 32)

    def both(ix):
        out, lse = gb.gattn_block_fwd(Q, K, V, ix, i32(sq), i32(sq), **kw)
        return out, lse, *gb.gattn_block_bwd(Q, K, V, ix, i32(sq), i32(sq), out, G, lse, **kw)

    wide = torch.full((2, idx.shape[0], 7), 1, dtype=torch.int32, device=DEV)
    wide[..., :4] = idx.transpose(0, 1)
    one = idx[:, :1].expand(-1, 2, -1)
    for a, b in ((idx, wide.transpose(0, 1)[..., :4]), (one.contiguous(), one)):
        assert not b.is_contiguous()
        assert all(torch.equal(x[:200], y[:200]) for x, y in zip(both(a), both(b)))
    with pytest.raises(ValueError, match="idx"):
        both(idx.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError, match="idx"):
        both(idx[:1, :1].expand(idx.shape[0], 2, -1))


# -- selection ----------------------------------------------------------------------------------
SELECT = [([1] * 5, [1, 63, 64, 700, 3000], 1), ([130, 0, 1, 400], [130, 9, 1, 400], 64),
          ([257], [1000], 16), ([33, 900], [33, 900], 128), ([50] * 3, [20] * 3, 32)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lq,lk,qb", SELECT)
@pytest.mark.parametrize("H,Hkv,D,block,topk", [(4, 2, 64, 16, 5), (8, 8, 16, 32, 1),
                                                (8, 1, 128, 64, 16), (2, 2, 8, 128, 3)])
def test_select(lq, lk, qb, H, Hkv, D, block, topk, dtype, causal):
    sq, sk = ref.offsets(lq), ref.offsets([n + 5 for n in lk])
    Q, K = randn(50, sq[-1] + 3, H, D, dtype=DT[dtype]), randn(51, sk[-1], Hkv, D, dtype=DT[dtype])
    for s, n in enumerate(lk):
        K[sk[s] + n:sk[s + 1]] = float("nan")
    sums = gb.gattn_block_sums(K, i32(sk), block, lens=i32(lk))
    want = ref.block_sums(K, sk, block, lk)
    assert (sums - want).abs().max() <= 2.0 ** -40 * block * K[:sk[-1]].nan_to_num().abs().max()
    idx = gb.gattn_block_select(Q, sums, i32(sq), i32(sk), topk, block, qb, K.shape[0],
                                len_k=i32(lk), causal=causal)
    exp = ref.select(Q, K, sq, sk, topk, block, qb, causal, lk)
    exp = torch.cat([exp, torch.full((idx.shape[0] - exp.shape[0], *exp.shape[1:]), -1,
                                     dtype=torch.int32)])[:idx.shape[0]]
    assert torch.equal(idx.cpu(), exp)


@pytest.mark.parametrize("qb", [1, 64])
def test_select_ties_go_to_the_lowest_block(qb):
    """Equal blocks, zero keys, and near-ties that fp32 cannot tell apart."""
    n, block = 640, 16
    sq = [0, 64]
    Q = torch.ones(64, 1, 16, device=DEV)
    for kind in range(3):
        K = torch.zeros(n, 1, 16, device=DEV)
        if kind == 1:
            K[:] = randn(60, 16, 1, 16).repeat(n // 16, 1, 1)
        if kind == 2:  # 1 + tiny in blocks 30 and 7: larger by 2^-30 of the score
            K[:] = 1.0
            K[30 * 16, 0, 0] = 1.0 + 2.0 ** -22
            K[7 * 16, 0, 0] = 1.0 + 2.0 ** -21
        sums = gb.gattn_block_sums(K, i32([0, n]), block)
        idx = gb.gattn_block_select(Q, sums, i32(sq), i32([0, n]), 3, block, qb, n)
        want = {0: [0, 1, 2], 1: [0, 1, 2], 2: [0, 7, 30]}[kind]
        rows = idx[:, 0][(idx[:, 0] >= 0).any(1)]
        assert rows.shape[0] == (64 if qb == 1 else 1) and (rows == i32(want)).all(), kind


def test_select_many_units_share_a_pass():
    """Enough units that eight of them share a pass over the sums."""
    lq, lk = [4000, 1, 3000, 2500], [3000, 64, 1, 2500]
    sq, sk = ref.offsets(lq), ref.offsets(lk)
    Q, K = randn(70, sq[-1], 8, 32, dtype=torch.bfloat16), randn(71, sk[-1], 8, 32, dtype=torch.bfloat16)
    sums = gb.gattn_block_sums(K, i32(sk), 64)
    for causal in (False, True):
        idx = gb.gattn_block_select(Q, sums, i32(sq), i32(sk), 4, 64, 16, sk[-1], causal=causal)
        assert torch.equal(idx.cpu(), ref.select(Q, K, sq, sk, 4, 64, 16, causal))


def test_select_is_cut_at_max_len():
    K, Q = randn(72, 1000, 1, 16), randn(73, 3, 1, 16)
    sums = gb.gattn_block_sums(K, i32([0, 1000]), 16)
    idx = gb.gattn_block_select(Q, sums, i32([0, 3]), i32([0, 1000]), 4, 16, 1, 1000, max_len_k=100)
    assert torch.equal(idx.cpu(), ref.select(Q, K, [0, 3], [0, 1000], 4, 16, 1, max_len=100))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("qb", [1, 64])
def test_select_non_finite_keys(qb, dtype):
    """Blocks whose score is not a number or -inf are never chosen, +inf comes first."""
    n, block, nan, inf = 400, 16, float("nan"), float("inf")
    K, Q = randn(75, n, 2, 32, dtype=DT[dtype]), randn(76, 128, 4, 32, dtype=DT[dtype]).abs()
    K[3 * block, 0, 5] = nan
    K[7 * block + 1, 0, 0] = inf           # q > 0: +inf
    K[9 * block + 2, 0, 0] = -inf
    K[11 * block, 0, 3], K[11 * block + 1, 0, 3] = inf, -inf
    sums = gb.gattn_block_sums(K, i32([0, n]), block)
    for topk in (1, 4, 30):
        idx = gb.gattn_block_select(Q, sums, i32([0, 128]), i32([0, n]), topk, block, qb, n)
        exp = ref.select(Q, K, [0, 128], [0, n], topk, block, qb)
        assert torch.equal(idx.cpu(), exp)
        first = idx[0, 0].tolist()
        assert 7 in first and not {3, 9, 11} & set(first)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("qb", [1, 32])
@pytest.mark.parametrize("q,k", [(1e20, 1e20), (1e-24, 1.0), (1.0, 1e-24), (1e-30, 1e-30), (1e30, 1e-30),
                                 (1e15, 1e30), (1e-38, 1e4), (0.0, 1.0), (1.0, 0.0)])
def test_select_at_the_ends_of_fp32(q, k, qb, causal):
    """Scores beyond the range of fp32, and norms whose squares it cannot hold: the choice is
    still that of the scores in 64 bits, with its near ties."""
    n, block = 640, 16
    # 64 bits see the difference of the last blocks, 32 do not
    Q, K = randn(77, 64, 2, 16), randn(78, n, 1, 16)
    K[320:] = K[:16].repeat(20, 1, 1)
    for i, at in enumerate((7, 3, 11, 2)):
        K[320 + 16 * at, 0, i] *= 1 + 2.0 ** (i - 22)
    Q, K = (Q.double() * q).float(), (K.double() * k).float()
    sums = gb.gattn_block_sums(K, i32([0, n]), block)
    for topk in (1, 5, 24, 60):
        idx = gb.gattn_block_select(Q, sums, i32([0, 64]), i32([0, n]), topk, block, qb, n, causal=causal)
        assert torch.equal(idx.cpu(), ref.select(Q, K, [0, 64], [0, n], topk, block, qb, causal)), topk


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("qb", [1, 64])
def test_sums_beyond_fp32(qb, dtype):
    """Keys and queries whose partial sums, or whole sums, are larger than fp32 can hold: the sums
    and the choice are those in 64 bits (some that cancel, some that do not)."""
    n, block, big = 300, 32, 2.0 ** 127
    Q, K = randn(83, 130, 8, 16, dtype=DT[dtype]), randn(84, n, 2, 16, dtype=DT[dtype])
    K[64:96, 0, 3] = big                       # 2^132
    K[96:112, 1, 5], K[112:128, 1, 5] = big, -big  # 0 in the end
    K[288:, :, 0] = -big                       # the last block is short
    Q[:, 0:4, 2], Q[0:64, 4:6, 7], Q[0:64, 6:8, 7] = 1.5 * big, big, -big
    sums = gb.gattn_block_sums(K, i32([0, n]), block)
    want = ref.block_sums(K, [0, n], block)
    mag = ref.block_sums(K.abs(), [0, n], block)
    assert ((sums - want).abs() <= 2.0 ** -40 * mag).all()
    part = torch.full_like(sums, 5.0)
    gb.gattn_block_sums(K, i32([0, n]), block, since=i32([70]), sums=part)
    assert ((part - want).abs()[2:] <= 2.0 ** -40 * mag[2:]).all() and (part[:2] == 5.0).all()
    for topk in (1, 4, 9):
        idx = gb.gattn_block_select(Q, sums, i32([0, 130]), i32([0, n]), topk, block, qb, n)
        assert torch.equal(idx.cpu(), ref.select(Q, K, [0, 130], [0, n], topk, block, qb))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_some_units_and_blocks_out_of_range(dtype):
    """Units and blocks of ordinary size beside huge, tiny, zero and non-finite ones, eight units
    to a pass over the sums."""
    lens, block, qb = [700, 40, 900], 16, 8
    sq = ref.offsets(lens)
    Q, K = randn(79, sq[-1], 16, 16, dtype=DT[dtype]), randn(80, sq[-1], 16, 16, dtype=DT[dtype])
    for s in range(3):
        Q[sq[s]:sq[s] + 8] *= 1e25
        Q[sq[s] + 8:sq[s] + 16] *= 1e-30
        Q[sq[s] + 16:sq[s] + 24] = 0
    K[100:116] *= 1e30
    K[740 + 64:740 + 80, 3] = 0
    K[740 + 80:740 + 96, 4] *= 1e-35
    K[740 + 100, 5, 7] = float("inf")
    K[740 + 130, 6, 7] = float("nan")
    sums = gb.gattn_block_sums(K, i32(sq), block)
    for causal in (False, True):
        idx = gb.gattn_block_select(Q, sums, i32(sq), i32(sq), 4, block, qb, sq[-1], causal=causal)
        assert torch.equal(idx.cpu(), ref.select(Q, K, sq, sq, 4, block, qb, causal))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_beyond_32_bits(dtype):
    """A sequence at the end of a cache of more than 2^31 elements."""
    Nk, n, H, Hkv, D = 2_200_000, 777, 8, 8, 128
    if torch.cuda.mem_get_info()[0] < 6 * Nk * Hkv * D * DT[dtype].itemsize:
        pytest.skip("needs more device memory")
    K, V = (torch.empty(Nk, Hkv, D, dtype=DT[dtype], device=DEV) for _ in range(2))
    K[-n:], V[-n:] = randn(77, n, Hkv, D, dtype=DT[dtype]), randn(78, n, Hkv, D, dtype=DT[dtype])
    sk = i32([Nk - n, Nk])
    for lq, qb in ((1, 1), (100, 64)):
        Q = randn(79, lq, H, D, dtype=DT[dtype])
        sums = gb.gattn_block_sums(K, sk, 64)
        idx = gb.gattn_block_select(Q, sums, i32([0, lq]), sk, 5, 64, qb, Nk, max_len_k=n)
        assert torch.equal(idx.cpu(), ref.select(Q, K[-n:], [0, lq], [0, n], 5, 64, qb))
        out, lse = gb.gattn_block_fwd(Q, K, V, idx, i32([0, lq]), sk, 64, qb)
        dout = randn(80, lq, H, D, dtype=DT[dtype])
        grads = gb.gattn_block_bwd(Q, K, V, idx, i32([0, lq]), sk, out, dout, lse, 64, qb)
        torch.cuda.synchronize()
        gb.gattn_block_check_errors()
        r = ref.attention(Q, K[-n:], V[-n:], idx, [0, lq], [0, n], 64, qb, dout=dout)
        for t, name in ((out, "out"), (lse, "lse"), (grads[0], "dQ"), (grads[1][-n:], "dK"),
                        (grads[2][-n:], "dV")):
            ref.check(t, r, name)
        del grads


def test_sums_are_renewed_from_a_position():
    sk, lens = [0, 300, 500], [290, 1]
    K = randn(74, 500, 2, 64, dtype=torch.bfloat16)
    sums = torch.full((gb.gattn_block_count(500, 2, 64), 2, 64), 5.0, dtype=torch.float64, device=DEV)
    gb.gattn_block_sums(K, i32(sk), 64, lens=i32(lens), since=i32([130, 0]), sums=sums)
    want = ref.block_sums(K, sk, 64, lens)
    for row, fresh in ((0, False), (1, False), (2, True), (3, True), (4, True), (5, True)):
        if fresh:
            assert (sums[row] - want[row]).abs().max() < 1e-9, row
        else:
            assert (sums[row] == 5.0).all(), row
    assert (sums[6:] == 5.0).all()


# -- together, captured, elsewhere ---------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_loop_in_one_graph(dtype):
    """Append a token, renew the sums, choose, attend: captured once, replayed while the device
    lengths grow across block borders."""
    S, room, H, Hkv, D, block, topk = 3, 256, 4, 2, 64, 16, 4
    dt = DT[dtype]
    lens = i32([14, 100, 31])
    sk, sq = i32([0, room, 2 * room, 3 * room]), i32([0, 1, 2, 3])
    K, V = (torch.zeros(S * room, Hkv, D, device=DEV, dtype=dt) for _ in range(2))
    for s, n in enumerate(lens.tolist()):
        K[s * room:s * room + n] = randn(80 + s, n, Hkv, D, dtype=dt)
        V[s * room:s * room + n] = randn(90 + s, n, Hkv, D, dtype=dt)
    Q, nk, nv = (torch.zeros(S, h, D, device=DEV, dtype=dt) for h in (H, Hkv, Hkv))
    sums = gb.gattn_block_sums(K, sk, block, lens=lens)
    base = sk[:-1].long()

    def step():
        at = base + lens
        K.index_copy_(0, at, nk)
        V.index_copy_(0, at, nv)
        old = lens.clone()
        lens.add_(1)
        gb.gattn_block_sums(K, sk, block, lens=lens, since=old, sums=sums)
        idx = gb.gattn_block_select(Q, sums, sq, sk, topk, block, 1, S * room, len_k=lens,
                                    causal=True, max_len_k=room)
        out, lse = gb.gattn_block_fwd(Q, K, V, idx, sq, sk, block, 1, causal=True, len_k=lens)
        return idx, out, lse

    keep = (K.clone(), V.clone(), lens.clone(), sums.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for t, k in zip((K, V, lens, sums), keep):
        t.copy_(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        idx, out, lse = step()
    for t in range(20):
        for i, x in enumerate((Q, nk, nv)):
            x.copy_(randn(100 + 3 * t + i, *x.shape, dtype=dt))
        graph.replay()
        torch.cuda.synchronize()
        ln = lens.tolist()
        assert torch.equal(idx.cpu(), ref.select(Q, K, sq.tolist(), sk.tolist(), topk, block, 1, True, ln))
        r = ref.attention(Q, K, V, idx, sq.tolist(), sk.tolist(), block, 1, causal=True, lk=ln)
        ref.check(out, r, "out")
        ref.check(lse, r, "lse")
    gb.gattn_block_check_errors()


def test_another_stream_and_shared_inputs():
    """Calls on two streams at once, each with its own workspace, on the same inputs."""
    sq = [0, 600]
    Q, K, V = (randn(110 + i, 600, 4, 64, dtype=torch.bfloat16) for i in range(3))
    idx = random_idx(5, sq, [600], 64, 4, 4, 64)
    G = randn(113, 600, 4, 64, dtype=torch.bfloat16)
    a = gb.gattn_block_fwd(Q, K, V, idx, i32(sq), i32(sq), 64, 64)
    ga = gb.gattn_block_bwd(Q, K, V, idx, i32(sq), i32(sq), a[0], G, a[1], 64, 64)
    off = i32(sq)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    res = []
    for st in streams:
        o, l = gb.gattn_block_fwd(Q, K, V, idx, off, off, 64, 64, stream=st)
        res.append((o, l, *gb.gattn_block_bwd(Q, K, V, idx, off, off, o, G, l, 64, 64, stream=st)))
    torch.cuda.synchronize()
    for r in res:
        assert all(torch.equal(x, y) for x, y in zip(r, (*a, *ga)))


def test_another_stream_allocates_for_itself():
    """Memory that the caller has released, but that work queued on the current stream still
    uses, is not handed to a call on another stream: neither for results nor for workspaces."""
    N, F, sq = 600, 256, [0, 600]
    off, one = i32(sq), i32([0, 1])
    Q, K, V, G = (randn(170 + i, N, 4, 64, dtype=torch.bfloat16) for i in range(4))
    idx = random_idx(7, sq, [N], 64, 4, 4, 64)
    x, res, dh = (randn(175 + i, N, F) for i in range(3))
    w = torch.ones(F, device=DEV)
    out, lse = gb.gattn_block_fwd(Q, K, V, idx, off, off, 64, 64)
    sums = gb.gattn_block_sums(K, off, 64)
    _, _, stats = gb.gattn_norm_fwd(res, x, w_post=w, w_pre=w)
    token = torch.zeros(1, 4, 2, dtype=torch.int32, device=DEV)
    calls = [
        lambda st: [gb.gattn_block_sums(K, off, 64, stream=st)],
        lambda st: [gb.gattn_block_select(Q, sums, off, off, 4, 64, 64, N, stream=st)],
        lambda st: gb.gattn_block_fwd(Q, K, V, idx, off, off, 64, 64, stream=st),
        lambda st: gb.gattn_block_fwd(Q[:1], K, V, token, one, off, 64, 1, stream=st),
        lambda st: gb.gattn_block_bwd(Q, K, V, idx, off, off, out, G, lse, 64, 64, stream=st),
        lambda st: gb.gattn_norm_fwd(res, x, w_post=w, w_pre=w, stream=st),
        lambda st: [t for t in gb.gattn_norm_bwd(res, stats, dh, x, x, w_post=w, w_pre=w,
                                                 stream=st).values() if t is not None],
    ]
    side = torch.cuda.Stream()
    for n, call in enumerate(calls):
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        # blocks of every size up to 64 MiB, in use by a copy behind a pause of a tenth of a second
        held = [torch.full((1 << b,), 3, dtype=torch.uint8, device=DEV)
                for b in range(9, 27) for _ in range(4)]
        spans = [(t.data_ptr(), t.numel()) for t in held]
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)
        copies = [t.clone() for t in held]
        del held
        got = call(side)
        side.synchronize()
        for t in got:
            a, e = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
            assert all(e <= p or a >= p + size for p, size in spans), n
        torch.cuda.synchronize()
        assert all((c == 3).all() for c in copies), n
        assert all(torch.equal(a, b) for a, b in zip(want, got)), n


def test_backward_in_a_graph():
    sq = i32([0, 200, 333])
    Q, K, V, G = (randn(120 + i, 333, 2, 64, dtype=torch.bfloat16) for i in range(4))
    idx = random_idx(6, [0, 200, 333], [200, 133], 64, 2, 2, 64)
    kw = {"block": 64, "q_block": 64, "causal": True}

    def step():
        out, lse = gb.gattn_block_fwd(Q, K, V, idx, sq, sq, **kw)
        return out, lse, *gb.gattn_block_bwd(Q, K, V, idx, sq, sq, out, G, lse, **kw)

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_outside_the_tensors_stay_inside():
    """Offsets and lengths that lie: the call returns and leaves canary rows of other buffers
    alone (every index is cut to the tensors)."""
    N = 256
    big = torch.full((3 * N, 2, 64), 7.0, device=DEV, dtype=torch.bfloat16)
    Q, K, V = (randn(130 + i, N, 2, 64, dtype=torch.bfloat16) for i in range(3))
    idx = torch.zeros(N // 64 + 2, 2, 3, dtype=torch.int32, device=DEV)
    idx[..., 1], idx[..., 2] = 1000000, -5
    out = big[N:2 * N]
    lse = torch.zeros(N, 2, device=DEV)
    for sq, sk in (([-5, 100, 5000], [0, 300, 200]), ([0, 256, 256], [-7, 9000, 3]),
                   ([300, 20, 256], [256, 256, 256])):
        gb.gattn_block_fwd(Q, K, V, idx, i32(sq), i32(sk), 64, 64, causal=True, out=out, lse=lse)
        gb.gattn_block_bwd(Q, K, V, idx, i32(sq), i32(sk), out, Q, lse, 64, 64, causal=True)
        s = gb.gattn_block_sums(K, i32(sk), 64)
        gb.gattn_block_select(Q, s, i32(sq), i32(sk), 3, 64, 64, N, causal=True)
        torch.cuda.synchronize()
    assert (big[:N] == 7.0).all() and (big[2 * N:] == 7.0).all()
    assert (idx[..., 1] == 1000000).all()


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 64), ("bf16", 128)])
def test_key_tiles_that_nobody_chose_between_others(dtype, D):
    """Most key tiles are in no list, so a CTA's work items are empty and not empty in turn, over
    several rounds: an empty item leaves nothing to the next one, and calls repeat bit by bit."""
    lens = [512 + 37 * (i % 3) for i in range(260)]
    sq = ref.offsets(lens)
    g = torch.Generator().manual_seed(21)
    idx = torch.randint(0, 16, (ref.units(sq[-1], len(lens), 128), 1, 1), generator=g, dtype=torch.int32)
    for s, n in enumerate(lens):  # (units behind a sequence's end belong to nothing)
        row = ref.table_row(sq[s], s, 128)
        idx[row + 1:row + -(-n // 128)] = idx[row]
    idx = idx.to(DEV)
    Q, K, V, _, out, lse, first = run(160, lens, lens, 1, 1, D, dtype, 32, 128, 1, idx=idx)
    G = randn(169, *Q.shape, dtype=DT[dtype])  # the dout of run()
    off = i32(sq)
    for _ in range(10):
        again = gb.gattn_block_bwd(Q, K, V, idx, off, off, out, G, lse, 32, 128)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    gb.gattn_block_check_errors()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", [9, 17, 40])
def test_offsets_out_of_order_that_want_more_items_than_there_are(S, dtype):
    """Offsets 0, N, 0, N, ...: tiles share blocks, and their work items would not fit the
    workspace.  Nothing outside the outputs and the workspace is written, and an ordinary call is
    right afterwards."""
    N, H, qb, block = 4096, 1, 16, 16
    Q, K, V, G = (randn(180 + i, N, H, 64, dtype=DT[dtype]) for i in range(4))
    off = i32([0 if i % 2 == 0 else N for i in range(S + 1)])
    units = gb.gattn_block_units(N, S, qb)
    idx = torch.zeros(units, 1, 1, dtype=torch.int32, device=DEV)
    lse = torch.zeros(N, H, device=DEV)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    desc, size = gb._block_attn(Q, K, V, idx, off, off, block, qb, 0.0, False, None)[1], ctypes.c_size_t()
    assert gb.load_library().gattn_block_bwd_workspace_size(desc, ctypes.byref(size)) == 0
    need = size.value
    ws[need:] = 7
    big = torch.full((5, N, H, 64), 7.0, device=DEV, dtype=DT[dtype])
    for _ in range(3):
        gb.gattn_block_bwd(Q, K, V, idx, off, off, Q, G, lse, block, qb, dQ=big[1], dK=big[2], dV=big[3],
                           workspace=ws[:need])
    torch.cuda.synchronize()
    gb.gattn_block_check_errors()
    assert (ws[need:] == 7).all() and (big[0] == 7.0).all() and (big[4] == 7.0).all()
    run(185, [N], [N], H, H, 64, dtype, block, qb, 1,
        idx=torch.zeros(ref.units(N, 1, qb), 1, 1, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D,G,qb", [(16, 2, 128), (64, 1, 64), (64, 4, 32), (128, 2, 64), (128, 1, 1)])
def test_gradients_of_rows_with_few_keys(D, G, qb, causal):
    """bf16 rows that see at most one step of 128 keys: ds = p (dP - Delta) is a small difference
    there, and Delta carries no rounding of out.

    Bounds, relative to |.|: a score is off by c |q||k| scale with c = (n + D + 32) 2^-24, lse by
    that and 2^-20 (1 + |lse|), so p by e_p, twice their sum and 2^-22 for the exponential; dP by
    c |dout||v|; Delta = sum p dP by the sum of p's and dP's errors and c for its own sum.  ds
    enters dQ as two bf16 (2^-16) and dK as one (2^-8); each result is rounded once (2^-8)."""
    lens, Hkv = [1, 2, 3, 7, 33, 64, 100, 128, 1, 5], 2
    H, block, sq = Hkv * G, 32, ref.offsets(lens)
    N = sq[-1]
    Q, K, V, W = (randn(190 + i, N, H if i in (0, 3) else Hkv, D, dtype=torch.bfloat16) for i in range(4))
    idx = torch.arange(4, dtype=torch.int32, device=DEV).repeat(gb.gattn_block_units(N, len(lens), qb), Hkv, 1)
    off, kw = i32(sq), {"block": block, "q_block": qb, "causal": causal}
    out, lse = gb.gattn_block_fwd(Q, K, V, idx, off, off, **kw)
    dQ, dK, dV = gb.gattn_block_bwd(Q, K, V, idx, off, off, out, W, lse, **kw)
    gb.gattn_block_check_errors()
    scale, u = 1 / math.sqrt(D), 2.0 ** -8
    for s, n in enumerate(lens):
        rows = slice(sq[s], sq[s + 1])
        c = (n * G + D + 32) * 2.0 ** -24
        ok = torch.ones(n, n, dtype=torch.bool, device=DEV)
        ok = ok.tril() if causal else ok
        for g in range(Hkv):
            k, v = K[rows, g].double(), V[rows, g].double()
            want, tol = torch.zeros(n, D, dtype=torch.float64, device=DEV), 0.0
            for h in range(g * G, (g + 1) * G):
                q, do = Q[rows, h].double(), W[rows, h].double()
                sc = (q @ k.T * scale).masked_fill(~ok, -math.inf)
                z = torch.logsumexp(sc, 1, keepdim=True)
                p = torch.exp(sc - z)
                err = torch.where(ok, q.abs() @ k.abs().T * scale * c, 0.0)
                ep = 2 * (err + err.amax(1, keepdim=True) + 2.0 ** -20 * (1 + z.abs())) + 2.0 ** -22
                dp, dpe = do @ v.T, c * (do.abs() @ v.abs().T)
                delta = (p * dp).sum(1, keepdim=True)
                de = (p * (ep * dp.abs() + dpe)).sum(1, keepdim=True) + c * (p * dp.abs()).sum(1, keepdim=True)
                ds = p * (dp - delta)
                dse = p * (ep * (dp - delta).abs() + dpe + de) + c * ds.abs()
                dq = ds @ k * scale
                t = u * dq.abs() + scale * ((dse + 2.0 ** -16 * ds.abs()) @ k.abs())
                over = ((dQ[rows, h].double() - dq).abs() - t).max().item()
                assert over <= 1e-30, (n, h, over)
                want += ds.T @ q * scale
                tol = tol + scale * ((dse + u * ds.abs()).T @ q.abs())
            over = ((dK[rows, g].double() - want).abs() - tol - u * want.abs()).max().item()
            assert over <= 1e-30, (n, g, over)


def test_items_that_take_long():
    """Eight million rows that all chose one block: the warps that write a work item's results wait
    more than 10 ms for them, which is no reason to give up.

    The rows repeat a period R times, so dK and dV are R times those of one period.  The bounds are R
    times the period's: these hold the weights' and ds' rounding, 2^-8 of the sum of magnitudes A.
    Adding up an item's 27,600 steps in fp32 is off by 27,700 2^-23 A at most, less than 2^-8 A, which
    is what twice the bounds leave for it."""
    n, R, D = 8192, 1024, 64
    if torch.cuda.mem_get_info()[0] < 12 * n * R * D * 2:
        pytest.skip("needs more device memory")
    Qs, Gs = (randn(200 + i, n, 1, D, dtype=torch.bfloat16) for i in range(2))
    K, V = (randn(202 + i, 128, 1, D, dtype=torch.bfloat16) for i in range(2))
    one = torch.zeros(ref.units(n, 1, 128), 1, 1, dtype=torch.int32, device=DEV)
    r = ref.attention(Qs, K, V, one, [0, n], [0, 128], 128, 128, dout=Gs)
    Q, G = (t.repeat(R, 1, 1) for t in (Qs, Gs))
    idx = torch.full((ref.units(n * R, 1, 128), 1, 128), -1, dtype=torch.int32, device=DEV)
    idx[..., 0] = 0
    sq, sk = i32([0, n * R]), i32([0, 128])
    out, lse = gb.gattn_block_fwd(Q, K, V, idx, sq, sk, 128, 128)
    got = gb.gattn_block_bwd(Q, K, V, idx, sq, sk, out, G, lse, 128, 128)
    gb.gattn_block_check_errors()
    for g, name in ((got[1], "dK"), (got[2], "dV")):
        over = (g.double() - R * r[name]).abs() - 2 * R * r[name + "_tol"]
        assert over.max() <= 0, (name, over.max().item())
    for k in (0, R // 2, R - 1):
        rows = slice(k * n, k * n + n)
        for t, name in ((out, "out"), (lse, "lse"), (got[0], "dQ")):
            ref.check(t[rows], r, name)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,D,H,Hkv", [("bf16", 32, 4, 4), ("bf16", 128, 4, 2), ("f32", 16, 2, 2)])
def test_many_small_graphs(dtype, D, H, Hkv, causal):
    """A batch of 600 graphs of 0 to 40 nodes: choice, attention and gradients."""
    g = torch.Generator().manual_seed(31)
    lens = torch.randint(0, 41, (600,), generator=g).tolist()
    sq = ref.offsets(lens)
    Q, K = randn(210, sq[-1], H, D, dtype=DT[dtype]), randn(211, sq[-1], Hkv, D, dtype=DT[dtype])
    sums = gb.gattn_block_sums(K, i32(sq), 16)
    idx = gb.gattn_block_select(Q, sums, i32(sq), i32(sq), 2, 16, 32, sq[-1], causal=causal, max_len_k=40)
    assert torch.equal(idx[:ref.units(sq[-1], 600, 32)].cpu(), ref.select(Q, K, sq, sq, 2, 16, 32, causal))

    def edit(q, k, v, *_):
        q.copy_(Q)
        k.copy_(K)

    run(212, lens, lens, H, Hkv, D, dtype, 16, 32, 2, causal, idx=idx, edit=edit)
