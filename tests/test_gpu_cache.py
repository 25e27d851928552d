"""The key/value cache in 4 and 8 bits on the GPU against its definition (tests/cache_ref.py)."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu

from gnn_sparse_attention_gb300 import binding as gb  # noqa: E402
from tests import block_ref  # noqa: E402
from tests import cache_ref as ref  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def marked(rows, Hkv, D, bits):
    """A cache whose every byte holds a mark."""
    c = gb.gattn_cache_new(rows, Hkv, D, bits)
    c.k.fill_(0xa5)
    c.v.fill_(0x5a)
    c.par.fill_(-77.0)
    return c


# ---------------------------------------------------------------------------
# write and read
# ---------------------------------------------------------------------------
def write(K, V, sq, sk, lk, bits, rows, view=lambda t: t):
    """Write through the kernel and by the definition; every byte of the cache is compared."""
    _, Hkv, D = K.shape
    c = marked(rows, Hkv, D, bits)
    want = [t.clone().cpu() for t in (c.k, c.v, c.par)]
    gb.gattn_cache_write(c, view(K), view(V), i32(sq), i32(sk), None if lk is None else i32(lk))
    torch.cuda.synchronize()
    for n, x in ((0, K), (1, V)):
        q, p = ref.quantise(x.float().cpu().numpy(), bits)
        q, p = torch.from_numpy(ref.pack(q, bits).copy()), torch.from_numpy(p).to(torch.bfloat16)
        for s in range(len(sq) - 1):
            a = sq[s + 1] - sq[s]
            n_k = (sk[s + 1] - sk[s]) if lk is None else lk[s]
            for i in range(a):
                pos = i + n_k - a
                if pos >= 0:
                    want[n][:, sk[s] + pos] = q[sq[s] + i]
                    want[2][:, sk[s] + pos, 2 * n:2 * n + 2] = p[sq[s] + i]
    assert torch.equal(c.k.cpu(), want[0])
    assert torch.equal(c.v.cpu(), want[1])
    got, par = c.par.cpu().float(), want[2].float()
    assert torch.equal(got.isnan(), par.isnan())
    assert torch.equal(got.nan_to_num(), par.nan_to_num())
    return c


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv,D", [(1, 32), (4, 64), (8, 128), (2, 128)])
def test_write_read(Hkv, D, dtype, bits):
    lq, lk, room = [37, 0, 1, 130], [40, 7, 1, 200], 9
    sq, sk = ref.offsets(lq), ref.offsets([n + room for n in lk])
    N = sq[-1] + 5
    K, V = randn(1, N, Hkv, D, dtype=DT[dtype]), 3 + randn(2, N, Hkv, D, dtype=DT[dtype])
    c = write(K, V, sq, sk, lk, bits, sk[-1] + 3)
    for out in (torch.bfloat16, torch.float32):
        got = [torch.full((N, Hkv, D), 7.0, device=DEV, dtype=out) for _ in range(2)]
        gb.gattn_cache_read(c, i32(sq), i32(sk), i32(lk), K=got[0], V=got[1])
        for n, (g, x) in enumerate(zip(got, (K, V))):
            val, mag, step = ref.values(c, n)
            for s in range(len(lq)):
                a, b = sk[s] + lk[s] - lq[s], sk[s] + lk[s]
                w, y = val[a:b], g[sq[s]:sq[s + 1]].cpu().double()
                assert bool(((y - w).abs() <= (ref.HALF[out] + 2.0 ** -24) * w.abs()).all())
                # half a step, and the roundings of x inv + c (two units of its size)
                src = x[sq[s]:sq[s + 1]].cpu().double()
                slack = step[a:b, :, None] * 0.5 + 2.0 ** -22 * (src.abs() + mag[a:b])
                assert bool(((w - src).abs() <= slack).all())
            assert bool((g[sq[-1]:] == 7.0).all())


@pytest.mark.parametrize("bits", [4, 8])
def test_write_values(bits):
    """Rows at the ends of the types: constant, huge, tiny, skewed, zeros, one outlier."""
    D = 64
    big = 3.3e38
    rows = [torch.zeros(D), torch.full((D,), 1.7), torch.full((D,), -0.1), torch.linspace(-big, big, D),
            torch.linspace(0, 1e-38, D), torch.linspace(0, 1e-44, D), torch.linspace(1000, 1000.25, D),
            torch.linspace(-1000.25, -1000, D), torch.full((D,), 1e30), torch.linspace(1e-30, 2e-30, D),
            torch.tensor([0.0] * (D - 1) + [1e6]), torch.tensor([-1e-20] + [1.0] * (D - 1)),
            torch.arange(D) * (1 / 32) - 1, torch.tensor([3.4028235e38] * D),
            torch.tensor([-3.4028235e38] * (D - 1) + [0.0]), torch.tensor([-0.0] * D),
            # steps so small next to the least value that levels leave their range by rounding
            torch.linspace(1, 1 + 2.0 ** -20, D), -torch.linspace(1, 1 + 2.0 ** -22, D),
            torch.full((D,), 7e10) + torch.arange(D) % 2 * 8192]
    x = torch.stack(rows).to(DEV)
    for dt in (torch.float32, torch.bfloat16):
        K = x.clamp(-3.38e38, 3.38e38).to(dt) if dt == torch.bfloat16 else x
        K = K.reshape(-1, 1, D).repeat(1, 2, 1)
        n = K.shape[0]
        c = write(K.contiguous(), K.flip(0).contiguous(), [0, n], [0, n], None, bits, n)
        got, _ = gb.gattn_cache_read(c, i32([0, n]), i32([0, n]), rows=n, dtype=torch.float32)
        exact = K[[0, 1, 2, 8, 15]].float()  # constant rows lose what bf16 loses of them
        assert bool(((got[[0, 1, 2, 8, 15]] - exact).abs() <= 2.0 ** -7 * exact.abs()).all())


@pytest.mark.parametrize("bits", [4, 8])
def test_rows_do_not_hang_on_their_neighbours(bits):
    """A row at the end of the range, or with levels that rounding moves out of theirs, among ordinary
    ones and alone: the same bytes."""
    D = 32
    odd = [torch.tensor([-3.4028235e38] * (D - 1) + [0.0]), torch.linspace(1, 1 + 2.0 ** -20, D),
           torch.full((D,), 7e10) + torch.arange(D) % 2 * 8192, torch.full((D,), float("nan"))]
    for row in odd:
        for n in (1, 40):
            K = randn(82, n, 1, D)
            for at in (0, n // 2):
                X = K.clone()
                X[at, 0] = row.to(DEV)
                write(X, K, [0, n], [0, n], None, bits, n)
                write(K, X, [0, n], [0, n], None, bits, n)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_random_bits(dtype, bits):
    """Rows of every exponent: bytes equal the definition's."""
    g = torch.Generator().manual_seed(5)
    n, Hkv, D = 400, 2, 128
    e = torch.randint(-60, 60, (n, Hkv, 1), generator=g)
    K = torch.randn(n, Hkv, D, generator=g) * torch.exp2(e.float())
    V = torch.randn(n, Hkv, D, generator=g) + torch.exp2(e.float() / 6)
    write(K.to(DEV, DT[dtype]), V.to(DEV, DT[dtype]), [0, n], [0, n], None, bits, n)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_rows(bad):
    K = randn(3, 6, 2, 64)
    K[1, 0, 63], K[2, 1, 0], K[4] = bad, bad, bad
    c = write(K, K.clone(), [0, 6], [0, 6], None, 4, 6)
    got, _ = gb.gattn_cache_read(c, i32([0, 6]), i32([0, 6]), rows=6, dtype=torch.float32)
    dead = torch.zeros(6, 2, dtype=torch.bool, device=DEV)
    dead[1, 0] = dead[2, 1] = dead[4, 0] = dead[4, 1] = True
    assert torch.equal(got.isnan().all(-1), dead) and torch.equal(got.isnan().any(-1), dead)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_slices(dtype):
    """K and V as slices of a joint projection; and rows that are appended one by one."""
    n, Hkv, D = 70, 4, 64
    qkv = randn(4, n, 5 * Hkv * D, dtype=DT[dtype])
    K, V = (qkv[:, i * Hkv * D:(i + 1) * Hkv * D].unflatten(1, (Hkv, D)) for i in (2, 4))
    c = marked(n, Hkv, D, 4)
    gb.gattn_cache_write(c, K, V, i32([0, n]), i32([0, n]))
    want = write(K.contiguous(), V.contiguous(), [0, n], [0, n], None, 4, n)
    assert torch.equal(c.k, want.k) and torch.equal(c.v, want.v) and torch.equal(c.par, want.par)
    d = marked(n, Hkv, D, 4)
    for i in range(n):
        gb.gattn_cache_write(d, K[i:i + 1], V[i:i + 1], i32([0, 1]), i32([0, n]), i32([i + 1]))
    assert torch.equal(d.k, want.k) and torch.equal(d.v, want.v) and torch.equal(d.par, want.par)
    big = randn(5, n, Hkv * D + 2, dtype=DT[dtype])  # rows that start in the middle of 16 bytes
    with pytest.raises(gb.GattnError):
        gb.gattn_cache_write(d, big[:, 2:].unflatten(1, (Hkv, D)), V, i32([0, n]), i32([0, n]))
    with pytest.raises(ValueError):  # rows that overlap
        gb.gattn_cache_write(d, K[:1].expand(n, -1, -1), V, i32([0, n]), i32([0, n]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sixteen_byte_borders(dtype):
    """Rows that start on 16-byte borders that are no 32-byte ones, in and out."""
    n, Hkv, D, dt = 40, 2, 32, DT[dtype]
    pad = 16 // torch.empty((), dtype=dt).element_size()
    K, V = randn(80, n, Hkv, D, dtype=dt), randn(81, n, Hkv, D, dtype=dt)
    want = write(K, V, [0, n], [0, n], None, 8, n)
    for off, extra in ((pad, pad), (0, pad), (pad, 0)):
        buf = torch.zeros(n * (Hkv * D + extra) + off, dtype=dt, device=DEV)
        views = []
        for x in (K, V):
            v = torch.zeros_like(buf)[off:].view(n, Hkv * D + extra)[:, :Hkv * D].unflatten(1, (Hkv, D))
            v.copy_(x)
            views.append(v)
        c = marked(n, Hkv, D, 8)
        gb.gattn_cache_write(c, *views, i32([0, n]), i32([0, n]))
        assert torch.equal(c.k, want.k) and torch.equal(c.v, want.v) and torch.equal(c.par, want.par)
    ref_k, ref_v = gb.gattn_cache_read(want, i32([0, n]), i32([0, n]), rows=n, dtype=dt)
    outs = [torch.zeros(n * Hkv * D + pad, dtype=dt, device=DEV)[pad:].view(n, Hkv, D) for _ in range(2)]
    gb.gattn_cache_read(want, i32([0, n]), i32([0, n]), K=outs[0], V=outs[1])
    assert torch.equal(outs[0], ref_k) and torch.equal(outs[1], ref_v)


@pytest.mark.parametrize("sq,sk,lk", [([0, 5], [0, 4], None), ([0, 5], [0, 9], [3]), ([0, 3, 6], [2, 4, 9], [2, 9]),
                                      ([2, 4], [3, 9], [6]), ([0, 0, 4], [0, 0, 8], [0, 4])])
def test_write_more_rows_than_room(sq, sk, lk):
    """Rows at positions below 0 are skipped, lengths are cut to the room, other rows stay."""
    K = randn(6, 6, 2, 32)
    cut = [min(sk[s + 1] - sk[s], lk[s] if lk else 1 << 30) for s in range(len(sk) - 1)]
    c = marked(9, 2, 32, 4)
    gb.gattn_cache_write(c, K, K, i32(sq), i32(sk), None if lk is None else i32(lk))
    want = write(K, K, sq, sk, cut, 4, 9)
    assert torch.equal(c.k, want.k) and torch.equal(c.par, want.par)


@pytest.mark.parametrize("bits", [4, 8])
def test_read_since(bits):
    lk, room = [50, 3, 0, 20], 60
    sk = ref.offsets([room] * 4)
    c = gb.gattn_cache_new(sk[-1], 2, 64, bits)
    ref.filled(c, randn(7, sk[-1], 2, 64), randn(8, sk[-1], 2, 64))
    val = [ref.values(c, n)[0].float() for n in (0, 1)]
    # whole sequences into the cache's own layout
    K, V = (torch.full((sk[-1], 2, 64), 7.0, device=DEV) for _ in range(2))
    gb.gattn_cache_read(c, i32(sk), i32(sk), i32(lk), since=i32([0] * 4), K=K, V=V)
    for t, w in ((K, val[0]), (V, val[1])):
        for s in range(4):
            a = sk[s]
            assert torch.equal(t[a:a + lk[s]].cpu(), w[a:a + lk[s]])
            assert bool((t[a + lk[s]:sk[s + 1]] == 7.0).all())
    # from a position on, one of them alone; positions below 0 and behind the end
    sq, since = [0, 10, 15, 20, 30], [40, -2, 0, 15]
    got = torch.full((32, 2, 64), 7.0, device=DEV)
    gb.gattn_cache_read(c, i32(sq), i32(sk), i32(lk), since=i32(since), V=got)
    want = torch.full((32, 2, 64), 7.0)
    for s in range(4):
        for i in range(sq[s + 1] - sq[s]):
            if 0 <= since[s] + i < lk[s]:
                want[sq[s] + i] = val[1][sk[s] + since[s] + i]
    assert torch.equal(got.cpu(), want)


# ---------------------------------------------------------------------------
# sums
# ---------------------------------------------------------------------------
def sums_ref(c, sk, lk, block):
    val = ref.values(c, 0)[0]
    out = torch.zeros(c.rows // block + len(lk), c.Hkv, c.D, dtype=torch.float64)
    mag = torch.zeros_like(out)
    for s, n in enumerate(lk):
        for j in range(-(-n // block)):
            x = val[sk[s] + j * block:sk[s] + min(n, (j + 1) * block)]
            out[sk[s] // block + s + j], mag[sk[s] // block + s + j] = x.sum(0), x.abs().sum(0)
    return out, mag


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv,D", [(1, 32), (4, 64), (2, 128)])
def test_sums(Hkv, D, block, bits):
    lk, room = [300, 0, 1, 64, 129], 11
    sk = ref.offsets([n + room for n in lk])
    c = gb.gattn_cache_new(sk[-1] + 40, Hkv, D, bits)
    K = randn(9, c.rows, Hkv, D)
    for s, n in enumerate(lk):
        K[sk[s] + n:sk[s + 1]] = float("nan")  # behind the sequences
    ref.filled(c, K, K.nan_to_num())
    want, mag = sums_ref(c, sk, lk, block)
    got = gb.gattn_cache_sums(c, i32(sk), block, lens=i32(lk))
    assert torch.equal(got.cpu(), want)  # steps within 2^23: no rounding anywhere
    # renewed from a position on: other blocks keep what they held
    since = [299, 0, 0, 63, 10]
    kept = torch.full_like(got, 5.0)
    gb.gattn_cache_sums(c, i32(sk), block, lens=i32(lk), since=i32(since), sums=kept)
    new = torch.full_like(want, 5.0)
    for s, n in enumerate(lk):
        b0, b1 = sk[s] // block + s, sk[s] // block + s + -(-n // block)
        new[b0 + since[s] // block:b1] = want[b0 + since[s] // block:b1]
    assert torch.equal(kept.cpu(), new)


@pytest.mark.parametrize("bits", [4, 8])
def test_sums_of_unlike_rows(bits):
    """Steps of any exponents: as fp64 adds them.  Constant rows, zeros, rows that are not finite."""
    n, Hkv, D = 256, 2, 64
    K = randn(10, n, Hkv, D) * torch.exp2(torch.randint(-40, 40, (n, Hkv, 1), device=DEV).float())
    K[64:128] = randn(11, 64, Hkv, 1)
    K[70:80] = 0.0
    K[128:192] = randn(12, 64, Hkv, D).abs()
    K[130, 0, 3] = 1e-30
    K[200, 1, 5] = float("nan")
    c = ref.filled(gb.gattn_cache_new(n, Hkv, D, bits), K, K.nan_to_num())
    want, mag = sums_ref(c, [0, n], [n], 64)
    got = gb.gattn_cache_sums(c, i32([0, n]), 64).cpu()
    assert torch.equal(got.isnan(), want.isnan()) and bool(got[3, 1].isnan().all())
    ok = ~want.isnan()
    assert bool(((got - want).abs()[ok] <= 64 * 2.0 ** -52 * mag[ok]).all())


@pytest.mark.parametrize("bits,spread", [(4, 1), (4, 3), (4, 6), (4, 7), (4, 13), (4, 28), (8, 1), (8, 2), (8, 3), (8, 8)])
@pytest.mark.parametrize("block", [16, 64, 128])
def test_sums_are_exact(block, bits, spread):
    """Steps of any mantissa over `spread` exponents, any levels (all the highest, all odd, random): no bit is
    lost.  All products and sums of a block are whole multiples of the least step's last bit below 2^53."""
    n, Hkv, D = 256, 2, 128
    g = torch.Generator().manual_seed(spread * 100 + block)
    c = gb.gattn_cache_new(n, Hkv, D, bits)
    for kind in range(4):
        mant = torch.randint(0, 128, (Hkv, n), generator=g)
        if kind == 0:
            mant.fill_(127)
        e = torch.randint(0, spread, (Hkv, n), generator=g)
        if kind == 1:
            e[:, ::2] = 0
            e[:, 1::2] = spread - 1
            mant[:, ::2] |= 1
        step = (1 + mant / 128) * torch.exp2(e.double() - 5)
        least = torch.randint(-255, 256, (Hkv, n), generator=g) / 64.0
        c.par.copy_(torch.stack([least.double(), step, least.double(), step], -1).to(torch.bfloat16))
        lev = torch.randint(0, 256, c.k.shape, generator=g)
        if kind == 0:
            lev.fill_(255)
        elif kind == 1:
            lev |= 0x11
        c.k.copy_(lev.to(torch.uint8))
        want, _ = sums_ref(c, [0, n], [n], block)
        assert torch.equal(gb.gattn_cache_sums(c, i32([0, n]), block).cpu(), want), kind


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def lists(seed, sq, lk, Hkv, topk, block):
    """Random lists: unsorted, with repeats, entries outside the sequence and empty ones."""
    g = torch.Generator().manual_seed(seed)
    idx = torch.full((sq[-1], Hkv, topk), -1, dtype=torch.int32)
    for s, n in enumerate(lk):
        for i in range(sq[s], sq[s + 1]):
            if int(torch.randint(0, 6, (1,), generator=g)):
                idx[i] = torch.randint(-2, -(-n // block) + 2, (Hkv, topk), generator=g,
                                       dtype=torch.int32)
    return idx.to(DEV)


def attend(seed, lq, lk, H, Hkv, D, dtype, bits, topk=0, block=64, causal=False, scale=0.0, extra=3,
           room=13, edit=None, max_len=True, idx=None):
    sq, sk = ref.offsets(lq), ref.offsets([n + room for n in lk])
    N = sq[-1] + extra
    c = gb.gattn_cache_new(sk[-1] + 5, Hkv, D, bits)
    K = randn(seed, c.rows, Hkv, D) * (1 + 2 * (randn(seed + 1, Hkv, D) > 1))
    V = randn(seed + 2, c.rows, Hkv, D) * torch.exp(randn(seed + 3, c.rows, Hkv, 1)) + 0.3
    Q = randn(seed + 4, N, H, D, dtype=DT[dtype])
    for s, n in enumerate(lk):  # rows of no sequence must not matter
        K[sk[s] + n:sk[s + 1]] = float("nan")
        V[sk[s] + n:sk[s + 1]] = float("nan")
    K[sk[-1]:], V[sk[-1]:] = float("nan"), float("nan")
    if edit:
        edit(Q, K, V)
    ref.filled(c, K, V)
    if topk and idx is None:
        idx = lists(seed, sq, lk, Hkv, topk, block)
        idx = torch.cat([idx, torch.zeros(extra, Hkv, topk, dtype=torch.int32, device=DEV)])
    out = torch.full((N, H, D), 7.0, device=DEV, dtype=DT[dtype])
    lse = torch.full((N, H), 7.0, device=DEV)
    kw = {"idx": idx, "block": block, "scale": scale, "causal": causal,
          "max_len_k": max(lk) if max_len else 0}
    gb.gattn_cache_fwd(Q, c, i32(sq), i32(sk), i32(lk), out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    r = ref.attention(Q, c, sq, sk, lk, None if idx is None else idx.cpu(), block, scale, causal)
    ref.check(out, r, "out", 7.0)
    ref.check(lse, r, "lse", 7.0)
    return Q, c, i32(sq), i32(sk), i32(lk), kw, out, lse


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,D", [(2, 2, 32), (8, 2, 64), (8, 1, 128), (4, 4, 128), (32, 2, 64)])
def test_one_token(H, Hkv, D, dtype, bits):
    attend(20, [1] * 4, [200, 1, 65, 0], H, Hkv, D, dtype, bits, topk=3)
    attend(21, [1] * 4, [200, 1, 65, 0], H, Hkv, D, dtype, bits)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 1000])
def test_lengths(n, dtype):
    attend(22, [1], [n], 4, 1, 64, dtype, 4)
    attend(23, [1], [n], 4, 1, 64, dtype, 4, topk=4, block=16)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("block,topk", [(16, 33), (32, 7), (64, 1), (128, 5), (16, 128)])
def test_blocks(block, topk, causal):
    attend(24, [3, 1, 0, 5], [333, 130, 9, 5], 8, 2, 64, "bf16", 4, topk, block, causal)
    attend(25, [2, 4], [333, 2], 4, 2, 32, "f32", 8, topk, block, causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_several_queries(dtype):
    """More queries than keys: with the mask the first see nothing."""
    attend(26, [5, 3, 1], [3, 100, 40], 8, 2, 128, dtype, 4, causal=True)


@pytest.mark.parametrize("G", [1, 2, 4, 8, 16, 32, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_heads(G, dtype):
    attend(27, [1, 1], [70, 150], 2 * G, 2, 32, dtype, 4, topk=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv", [(2, 1), (8, 8), (16, 1)])
def test_long(H, Hkv, dtype):
    """One token against a long cache: split over clusters and joined."""
    attend(28, [1], [20000], H, Hkv, 64, dtype, 4)
    attend(29, [1, 1], [9000, 17], H, Hkv, 64, dtype, 8, max_len=False)


@pytest.mark.parametrize("lk,H,Hkv,lq", [([17000], 2, 1, 1), ([17000, 40000, 1, 0, 300], 4, 1, 1), ([20000], 16, 1, 2),
                                         ([1, 18000, 16], 2, 2, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_stretches(lk, H, Hkv, lq, dtype):
    """Few long caches of unlike lengths: items are cut between CTAs and joined by a second kernel."""
    lq = [min(lq, n) for n in lk]
    attend(90, lq, lk, H, Hkv, 128, dtype, 8, causal=True)


def workspace_bytes(Q, c, S, kw):
    topk, n = 0 if kw["idx"] is None else kw["idx"].shape[2], ctypes.c_size_t()
    some = i32([0])  # sizes hang on no offset
    desc = gb._cache_desc(c, S, Q.shape[0], Q.shape[1], Q.dtype, kw["block"], topk, kw["causal"], kw["scale"],
                          kw["max_len_k"], some, some, some)
    assert gb.load_library().gattn_cache_fwd_workspace_size(desc, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("H,dtype", [(4, "f32"), (4, "bf16"), (16, "bf16")])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_stretches_of_every_layout(D, bits, H, dtype):
    """The form that cuts items and joins them, in every layout: a few long caches, and many items of one to 135
    steps, of which a CTA has several (the next one's copies are under way beside the old one's sums)."""
    row = D * bits // 8
    R = 16 if row > 64 else 32 if row > 32 else 64  # rows of a step
    Q, c, *_, kw, out, lse = attend(102, [1] * 4, [450 * R + 7, 3, 0, 100 * R + 1], H, 2, D, dtype, bits, extra=2)
    assert workspace_bytes(Q, c, 4, kw) > 0
    g = torch.Generator().manual_seed(103)
    lk = torch.randint(0, 3 * R, (159,), generator=g).tolist()
    lk[::9] = torch.randint(0, 20 * R, (len(lk[::9]),), generator=g).tolist()
    lk.insert(70, 135 * R - 5)
    Q, c, *_, kw, out, lse = attend(104, [1] * 160, lk, H, 2, D, dtype, bits, extra=5)
    assert workspace_bytes(Q, c, 160, kw) > 0


def test_stretches_over_many_items():
    """More items than CTAs, each of several: whole ones, cut ones, rows of no sequence, empty ones."""
    g = torch.Generator().manual_seed(91)
    lk = torch.randint(0, 3300, (170,), generator=g).tolist()
    attend(91, [1] * 170, lk, 2, 2, 128, "bf16", 8, extra=9)


def test_stretches_over_lists():
    attend(92, [1] * 41, [20000] + [3000] * 39 + [17], 2, 2, 128, "bf16", 8, topk=128, block=128, extra=1)


def test_sharp_scores():
    """One key outweighs all others, wherever it stands: the running maximum moves late."""
    for at in (0, 7, 100, 499):
        def edit(Q, K, V):
            K[at] = 40 * Q[0, 0].float()
        attend(30, [1], [500], 4, 1, 64, "bf16", 4, edit=edit, extra=0)
        attend(30, [1], [500], 4, 1, 64, "f32", 8, edit=edit, extra=0)


def test_steps_of_any_size():
    """Steps of V that differ by 2^40, the largest on keys that weigh least, and by order."""
    for sign in (1, -1):
        def edit(Q, K, V):
            V.mul_(torch.exp2(torch.linspace(-20 * sign, 20 * sign, V.shape[0], device=DEV)).reshape(-1, 1, 1))
            K.mul_(torch.linspace(3, 0.1, V.shape[0], device=DEV).reshape(-1, 1, 1))
        attend(31, [1], [400], 4, 1, 64, "bf16", 4, edit=edit)
        attend(31, [1], [400], 4, 1, 64, "f32", 4, edit=edit)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-12, 1e12, 1e-28, 3e36])
def test_sizes_of_queries(scale, dtype):
    def edit(Q, K, V):
        Q.mul_(scale)
    attend(32, [1], [100], 4, 2, 64, dtype, 4, edit=edit, scale=0.1 / scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_constant_rows(dtype):
    """Rows without steps: scores and outputs come from the least values alone."""
    def edit(Q, K, V):
        K.copy_(K[:, :, :1].expand_as(K).clone())
        V.copy_(V[:, :, :1].expand_as(V).clone())
    attend(33, [1, 1], [100, 3], 4, 2, 64, dtype, 4, edit=edit)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,topk", [(1, 0), (700, 0), (700, 3), (20000, 0)])
def test_scores_far_below_zero(n, topk, dtype):
    """Keys that score about -1e37: a lone one (other warps see none), many by a cluster, and cut between CTAs.

    A rounding of such a score in fp32 is 2^-24 1e37 > 2^98 nats, and it is rounded at other places in a warp's
    first step than in later ones: how equal keys weigh is not determined (ref.attention's bound of out is
    beyond 2^98 too).  What is: out is a mean of the rows seen with weights of 0 to 1 that sum to 1, so it lies
    between the least and the greatest of them, and a lone row is returned."""
    def edit(Q, K, V):
        Q.fill_(1e18)
        K.fill_(-1e18)
    idx = torch.tensor([[[0, 4, 9]]], dtype=torch.int32, device=DEV) if topk else None
    _, c, *_, out, lse = attend(100, [1], [n], 2, 1, 128, dtype, 8, topk=topk, edit=edit, extra=0, idx=idx)
    see = [j for j in range(n) if not topk or j // 64 in (0, 4, 9)]
    v, va, _ = ref.values(c, 1)
    lo, hi, mag = v[see, 0].amin(0), v[see, 0].amax(0), va[see, 0].amax(0)
    w = 2.0 ** -20 if dtype == "f32" else 2.0 ** -11  # weights, and sums of fp32 (tests/cache_ref.py)
    tol = ref.HALF[DT[dtype]] * torch.maximum(lo.abs(), hi.abs()) + mag * (w + (len(see) / 16 + 40) * 2.0 ** -23)
    got = out[0].cpu().double()
    assert bool((got >= lo - tol).all()) and bool((got <= hi + tol).all())
    assert bool(lse.isfinite().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [2, 8])
@pytest.mark.parametrize("D,bits,rows", [(128, 8, 16), (64, 4, 64)])
def test_weightless_keys_of_large_steps(D, bits, rows, H, dtype):
    """Constant rows of V carry all weight, and a key 200 nats below has steps of 2^30, 2^90 or none: 0 times its
    row is 0.  In the same step of a warp, and in a later one of it (32 steps on)."""
    n = 33 * rows
    for at in (5, 32 * rows + 3):
        for step in (2.0 ** 30, 2.0 ** 90, 0.0):
            def edit(Q, K, V):
                Q.fill_(1.0)
                K.zero_()
                K[at] = -200.0 / math.sqrt(D)
                V.fill_(1.5)
                V[at] = torch.arange(D, device=DEV) % 2 ** bits * step
            *_, out, lse = attend(101, [1], [n], H, 1, D, dtype, bits, edit=edit, extra=0)
            # the mean of equal values: one rounding, and fp32 ones of a weight, a product and a few sums
            assert bool(((out.double() - 1.5).abs() <= ref.HALF[DT[dtype]] * 1.5 + 2.0 ** -19).all())


@pytest.mark.parametrize("H,dtype", [(2, "f32"), (2, "bf16"), (8, "bf16")])
def test_slowly_rising_scores(H, dtype):
    """Each step raises one head's scores by a factor of 400 and the others' by 1%, and only the first rows have
    values: what the others hold is scaled with their own maximum, however often a neighbour's moves."""
    D, R, W = 128, 16, 200
    n, N = 4 * R * W, 256 * torch.cuda.get_device_properties(0).multi_processor_count  # a CTA for each item
    c = gb.gattn_cache_new(n, 1, D, 8)
    K, V = torch.zeros(n, 1, D), torch.zeros(n, 1, D)
    K[:] = (torch.arange(n) // (4 * R)).reshape(n, 1, 1)  # a warp takes every fourth step
    V[:4 * R] = (torch.arange(D) * 255 // (D - 1)) * (2.0 ** 30 if dtype == "f32" else 2.0 ** 50)
    ref.filled(c, K, V)
    Q = torch.full((N, H, D), 6.0 / 512, device=DEV, dtype=DT[dtype])
    Q[:, 0] = 6.0
    sq, sk = i32([0, N]), i32([0, n])
    out, lse = gb.gattn_cache_fwd(Q, c, sq, sk, scale=1 / D)
    r = ref.attention(Q[:1], c, [0, 1], [0, n], [n], scale=1 / D)
    ref.check(out[:1], r, "out", 7.0)
    ref.check(lse[:1], r, "lse", 7.0)
    assert bool((out == out[:1]).all()) and bool((lse == lse[:1]).all())


def test_one_key_is_returned():
    _, c, _, sk, lk, _, out, _ = attend(34, [1, 1], [1, 1], 4, 2, 64, "f32", 4, extra=0)
    val = ref.values(c, 1)[0].float()
    for s in range(2):
        for h in range(4):
            got, want = out[s, h].cpu(), val[int(sk[s]), h // 2]
            assert bool(((got - want).abs() <= 2.0 ** -21 * want.abs().max()).all())


def test_non_finite_is_where_it_is_seen():
    """A row that is not finite reaches the outputs of its own head and of queries that see it."""
    sk, lk = [0, 100, 200], [90, 90]
    c = gb.gattn_cache_new(200, 2, 64, 4)
    K, V = randn(35, 200, 2, 64), randn(36, 200, 2, 64)
    K[5, 0, 0], V[130, 1, 9] = float("nan"), float("inf")
    ref.filled(c, K, V)
    out, lse = gb.gattn_cache_fwd(randn(37, 2, 4, 64), c, i32([0, 1, 2]), i32(sk), i32(lk))
    bad = out.isnan().any(-1).cpu()
    assert bad.tolist() == [[True, True, False, False], [False, False, True, True]]
    assert lse.isnan().cpu().tolist() == [[True, True, False, False], [False] * 4]
    idx = torch.ones(2, 2, 1, dtype=torch.int32, device=DEV)  # rows 64 .. 89
    out, lse = gb.gattn_cache_fwd(randn(37, 2, 4, 64), c, i32([0, 1, 2]), i32(sk), i32(lk), idx=idx)
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all())


def test_lists_with_strides():
    args = attend(38, [1] * 3, [200, 300, 100], 8, 4, 64, "bf16", 4, topk=3, extra=0)
    Q, c, sq, sk, lk, kw, out, lse = args
    idx = kw.pop("idx")
    for other in (idx.transpose(0, 1).contiguous().transpose(0, 1),
                  torch.cat([idx, idx], 2)[:, :, :3]):
        o, z = gb.gattn_cache_fwd(Q, c, sq, sk, lk, idx=other, **kw)
        assert torch.equal(o, out) and torch.equal(z, lse)
    one = idx[:, :1].contiguous().expand(-1, 4, -1)  # shared by heads
    a = gb.gattn_cache_fwd(Q, c, sq, sk, lk, idx=one, **kw)
    b = gb.gattn_cache_fwd(Q, c, sq, sk, lk, idx=one.contiguous(), **kw)
    assert torch.equal(a[0], b[0])
    with pytest.raises(ValueError):
        gb.gattn_cache_fwd(Q, c, sq, sk, lk, idx=idx[:1, :1].expand(3, 4, -1), **kw)


@pytest.mark.parametrize("seq_k,len_k", [([-5, 1 << 30, 70], [50, 50]), ([60, 20, 10], [99, -3]),
                                         ([0, 90, 2000], [1 << 30, 1 << 30])])
def test_offsets_about_the_cache(seq_k, len_k):
    """Offsets outside the cache or out of order: results do not matter, other memory does not change."""
    c = marked(100, 2, 32, 4)
    K = randn(39, 2, 2, 32)
    guard = [t.clone() for t in (c.k, c.v, c.par)]
    gb.gattn_cache_write(c, K, K, i32([0, 1, 2]), i32(seq_k), i32(len_k))
    gb.gattn_cache_read(c, i32([0, 1, 2]), i32(seq_k), i32(len_k), rows=2)
    gb.gattn_cache_sums(c, i32(seq_k), 16, lens=i32(len_k))
    gb.gattn_cache_sums(c, i32(seq_k), 16, lens=i32(len_k), since=i32([-7, 1 << 30]),
                        sums=torch.zeros(8, 2, 32, dtype=torch.float64, device=DEV))
    gb.gattn_cache_fwd(randn(40, 2, 4, 32), c, i32([0, 1, 2]), i32(seq_k), i32(len_k))
    idx = torch.arange(-2, 6, dtype=torch.int32, device=DEV).expand(2, 2, 8).contiguous()
    gb.gattn_cache_fwd(randn(40, 2, 4, 32), c, i32([0, 1, 2]), i32(seq_k), i32(len_k), idx=idx)
    for sq in ([0, 1, 1 << 30], [-4, 1, 2], [2, 1, 0]):
        gb.gattn_cache_write(c, K, K, i32(sq), i32([0, 50, 100]), None)
        gb.gattn_cache_read(c, i32(sq), i32([0, 50, 100]), rows=2)
        gb.gattn_cache_fwd(randn(40, 2, 4, 32), c, i32(sq), i32([0, 50, 100]))
    torch.cuda.synchronize()
    assert all(g.shape == t.shape for g, t in zip(guard, (c.k, c.v, c.par)))


class Fenced:
    """Tensors in the middle of marked memory."""

    MARGIN, MARK = 1 << 16, 0xc3

    def __init__(self):
        self.all = []

    def __call__(self, dtype, *shape):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((n + 2 * self.MARGIN,), self.MARK, dtype=torch.uint8, device=DEV)
        self.all.append((buf, n))
        return buf[self.MARGIN:self.MARGIN + n].view(dtype).view(shape)

    def whole(self):
        torch.cuda.synchronize()
        return all(bool((b[:self.MARGIN] == self.MARK).all()) and bool((b[self.MARGIN + n:] == self.MARK).all())
                   for b, n in self.all)


ODD_OFFSETS = [([-5, 1 << 30, 70], [50, 50]), ([60, 20, 10], [99, -3]), ([0, 90, 2000], [1 << 30, 1 << 30]),
               ([0, 60, 100], [60, 40])]


@pytest.mark.parametrize("seq_k,len_k", ODD_OFFSETS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D,bits", [(100, 32, 4), (100, 64, 8), (20000, 128, 8)])
def test_memory_around_the_tensors(rows, D, bits, dtype, seq_k, len_k):
    """Whatever the offsets and lists say, what stands before and behind each tensor that a call writes stays, and
    read, sums and attention leave the cache as it is.  With 20,000 rows items are cut, through a workspace."""
    fence, dt = Fenced(), DT[dtype]
    c = gb.Cache(fence(torch.uint8, 2, rows, D * bits // 8), fence(torch.uint8, 2, rows, D * bits // 8),
                 fence(torch.bfloat16, 2, rows, 4), bits)
    ref.filled(c, randn(105, rows, 2, D), randn(106, rows, 2, D))
    new = randn(107, 3, 2, D, dtype=dt)
    Q = randn(108, 3, 4, D, dtype=dt)
    idx = torch.arange(-2, 6, dtype=torch.int32, device=DEV).expand(3, 2, 8).contiguous()
    K, V = fence(dt, 3, 2, D), fence(dt, 3, 2, D)
    sums = fence(torch.float64, rows // 16 + 2, 2, D)
    out, lse = fence(dt, 3, 4, D), fence(torch.float32, 3, 4)
    kw = {"idx": None, "block": 16, "causal": False, "scale": 0.0, "max_len_k": 0}
    n = max(workspace_bytes(Q, c, 2, kw), workspace_bytes(Q, c, 2, {**kw, "idx": idx}))
    assert (n > 0) == (rows == 20000)
    ws = fence(torch.uint8, n) if n else None
    far = [min(max(x * rows // 100, -(1 << 31)), (1 << 31) - 1) for x in seq_k]
    for sq in ([0, 1, 3], [0, 2, 1 << 30], [-4, 1, 2], [2, 1, 0], [3, 3, 3]):
        for k, ln in ((seq_k, len_k), (far, None), (far, len_k)):
            args = i32(sq), i32(k), None if ln is None else i32(ln)
            gb.gattn_cache_write(c, new, new, *args)
            assert fence.whole()
            kept = [t.clone() for t in (c.k, c.v, c.par.view(torch.int16))]
            for since in (None, i32([-7, 1 << 30]), i32([(1 << 31) - 1, 0])):
                gb.gattn_cache_read(c, *args, since=since, K=K, V=V)
                gb.gattn_cache_sums(c, args[1], 16, lens=args[2], since=since, sums=sums)
            for causal in (False, True):
                for choice in (None, idx):
                    gb.gattn_cache_fwd(Q, c, *args, idx=choice, block=16, causal=causal, out=out, lse=lse, workspace=ws)
            assert fence.whole()
            assert all(torch.equal(a, b) for a, b in zip(kept, (c.k, c.v, c.par.view(torch.int16))))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("width", [64, 10])
def test_memory_around_rotary(width, layout, dtype):
    fence, dt = Fenced(), DT[dtype]
    Q, K = randn(109, 70, 4, 64, dtype=dt), randn(110, 70, 2, 64, dtype=dt)
    q, k = fence(dt, 70, 4, 64), fence(dt, 70, 2, 64)
    f = gb.gattn_rotary_freqs(width)
    for sq in ([0, 30, 70], [0, 30, 1 << 30], [-5, 20, 71], [70, 30, 0], [71, 80, 90]):
        for kw in ({}, {"seq_k": i32([0, -9, 1 << 30])}, {"len_k": i32([-(1 << 31), (1 << 31) - 1])}):
            gb.gattn_rotary(Q, f, K=K, layout=layout, seq_q=i32(sq), out_q=q, out_k=k, **kw)
    assert fence.whole()


def test_offsets_beyond_32_bits():
    """A cache whose bytes pass 2^31 and rows 2^25: written, read, summed and attended to near its end."""
    rows, Hkv, D = (1 << 25) + 300, 2, 64
    c = gb.gattn_cache_new(rows, Hkv, D, 8)  # 2 x 4.3 GB
    sk, lk = [0, 40, rows - 150, rows], [40, 17, 150]
    K, V = randn(41, 150, Hkv, D), randn(42, 150, Hkv, D)
    gb.gattn_cache_write(c, K, V, i32([0, 0, 0, 150]), i32(sk), i32(lk))
    a = rows - 150
    small = gb.Cache(c.k[:, a:].contiguous(), c.v[:, a:].contiguous(), c.par[:, a:].contiguous(), 8)
    want = write(K, V, [0, 150], [0, 150], None, 8, 150)
    assert torch.equal(small.k, want.k) and torch.equal(small.par, want.par)
    kk, _ = gb.gattn_cache_read(c, i32([0, 0, 0, 150]), i32(sk), i32(lk), rows=150, dtype=torch.float32)
    k2, _ = gb.gattn_cache_read(small, i32([0, 150]), i32([0, 150]), rows=150, dtype=torch.float32)
    assert torch.equal(kk, k2)
    Q = randn(43, 1, 4, D)
    o1 = gb.gattn_cache_fwd(Q, c, i32([0, 0, 0, 1]), i32(sk), i32(lk), max_len_k=150)
    o2 = gb.gattn_cache_fwd(Q, small, i32([0, 1]), i32([0, 150]), max_len_k=150)
    assert torch.equal(o1[0], o2[0]) and torch.equal(o1[1], o2[1])
    s1 = gb.gattn_cache_sums(c, i32(sk), 64, lens=i32(lk), since=i32([40, 17, 0]),
                             sums=torch.zeros(rows // 64 + 3, Hkv, D, dtype=torch.float64, device=DEV))
    s2 = gb.gattn_cache_sums(small, i32([0, 150]), 64)
    b = a // 64 + 2
    assert torch.equal(s1[b:b + 3], s2[:3])


# ---------------------------------------------------------------------------
# the calls
# ---------------------------------------------------------------------------
def test_repeats_bit_by_bit():
    Q, c, sq, sk, lk, kw, out, lse = attend(44, [1] * 3, [3000, 500, 64], 16, 2, 128, "bf16", 4)
    for _ in range(3):
        o, z = gb.gattn_cache_fwd(Q, c, sq, sk, lk, **kw)
        assert torch.equal(o[:3], out[:3]) and torch.equal(z[:3], lse[:3])


def test_another_stream():
    Q, c, sq, sk, lk, kw, out, lse = attend(45, [1], [20000], 8, 1, 128, "bf16", 8)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    K, V = randn(46, 1, 1, 128), randn(47, 1, 1, 128)
    st.wait_stream(torch.cuda.current_stream())
    o, z = gb.gattn_cache_fwd(Q, c, sq, sk, lk, stream=st, **kw)
    k, v = gb.gattn_cache_read(c, i32([0, 20000]), sk, lk, rows=20000, stream=st)
    s = gb.gattn_cache_sums(c, sk, 64, lens=lk, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(o[:1], out[:1]) and torch.equal(z[:1], lse[:1])
    assert torch.equal(s, gb.gattn_cache_sums(c, sk, 64, lens=lk))
    k2, v2 = gb.gattn_cache_read(c, i32([0, 20000]), sk, lk, rows=20000)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    gb.gattn_cache_write(c, K, V, i32([0, 1]), sk, lk, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    k3, _ = gb.gattn_cache_read(c, i32([0, 1]), sk, lk, rows=1)
    assert not torch.equal(k3, k2[-1:])


@pytest.mark.parametrize("fill", [0x00, 0x7f, 0xff])
def test_workspaces_of_any_content(fill):
    """Nothing hangs on what a workspace holds: few items and many, rows of no sequence among them."""
    for lk, extra in (([18000, 3, 0], 2), ([9000] * 39 + [17], 5)):
        Q, c, sq, sk, lens, kw, out, lse = attend(111, [1] * len(lk), lk, 4, 2, 128, "bf16", 8, extra=extra)
        n = workspace_bytes(Q, c, len(lk), kw)
        assert n > 0
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        o, z = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
        gb.gattn_cache_fwd(Q, c, sq, sk, lens, out=o, lse=z, workspace=ws, **kw)
        assert torch.equal(o, out) and torch.equal(z, lse)


@pytest.mark.parametrize("n", [300, 2000])
def test_rows_of_no_sequence_between_clusters(n):
    """Rows of no sequence, among and behind those of sequences, where an item is a cluster's."""
    Q, c, sq, sk, lens, kw, out, lse = attend(112, [1, 0, 1], [n, n, 5], 4, 2, 64, "bf16", 4, extra=4)
    assert workspace_bytes(Q, c, 3, kw) == 0
    far = i32([2, 3, 3, 4])  # rows 0, 1 and behind 3 are nobody's
    o, z = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    gb.gattn_cache_fwd(Q.roll(2, 0), c, far, sk, lens, out=o, lse=z, **kw)
    assert torch.equal(o[2:4], out[:2]) and torch.equal(z[2:4], lse[:2])
    assert bool((o[:2] == 7.0).all()) and bool((o[4:] == 7.0).all()) and bool((z[:2] == 7.0).all())


def test_no_sequences_and_no_rows():
    c = gb.gattn_cache_new(0, 2, 64, 4)
    z = i32([0])
    gb.gattn_cache_write(c, randn(1, 0, 2, 64), randn(1, 0, 2, 64), z, z)
    assert gb.gattn_cache_read(c, z, z, rows=0)[0].shape == (0, 2, 64)
    assert gb.gattn_cache_sums(c, z, 64).shape == (0, 2, 64)
    out, lse = gb.gattn_cache_fwd(randn(1, 0, 4, 64), c, z, z)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # a sequence without any rows in an empty cache
    out, lse = gb.gattn_cache_fwd(randn(1, 1, 4, 64), c, i32([0, 1]), i32([0, 0]))
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def decode_state(bits, S, H, Hkv, D, start, steps, block):
    room = start + steps
    sk = [s * room for s in range(S + 1)]
    c = gb.gattn_cache_new(sk[-1], Hkv, D, bits)
    new = [[randn(50 + t, S, h, D, dtype=torch.bfloat16) for h in (H, Hkv, Hkv)] for t in range(steps)]
    K0, V0 = (randn(s, S * start, Hkv, D, dtype=torch.bfloat16) for s in (48, 49))
    sq0 = i32([s * start for s in range(S + 1)])
    ln = i32([start] * S)
    gb.gattn_cache_write(c, K0, V0, sq0, i32(sk), ln)
    sums = gb.gattn_cache_sums(c, i32(sk), block, lens=ln)
    return c, sums, new, i32(list(range(S + 1))), i32(sk), ln


def decode_step(c, sums, Q, K, V, freqs, sq, sk, ln, block, topk, room):
    """One new token for every request: positions, cache, sums, choice, attention."""
    ln.add_(1)
    Q, K = gb.gattn_rotary(Q, freqs, K=K, seq_q=sq, seq_k=sk, len_k=ln)
    gb.gattn_cache_write(c, K, V, sq, sk, ln)
    gb.gattn_cache_sums(c, sk, block, lens=ln, since=ln - 1, sums=sums)
    idx = gb.gattn_block_select(Q, sums, sq, sk, topk, block, 1, c.rows, len_k=ln, max_len_k=room)
    return (*gb.gattn_cache_fwd(Q, c, sq, sk, ln, idx=idx, block=block, max_len_k=room), idx, Q)


@pytest.mark.parametrize("bits", [4, 8])
def test_serving_loop(bits):
    """The operators together, as a server runs them, against the definitions step by step; then the
    same loop captured once into a graph and replayed over growing caches."""
    S, H, Hkv, D, start, steps, block, topk = 3, 8, 2, 64, 150, 5, 32, 3
    room = start + steps
    freqs = gb.gattn_rotary_freqs(D, scaling="ramp", factor=4.0, orig_len=64)
    rad = ref.frequencies(D, scaling="ramp", factor=4.0, orig_len=64)
    c, sums, new, sq, sk, ln = decode_state(bits, S, H, Hkv, D, start, steps, block)
    outs = []
    for t in range(steps):
        out, lse, idx, Qr = decode_step(c, sums, *new[t], freqs, sq, sk, ln, block, topk, room)
        lk = [start + t + 1] * S
        y, tol = ref.rotary(new[t][0], [n - 1 for n in lk], rad, "half")
        assert bool(((Qr.cpu().double() - y).abs() <= tol).all())
        want, _ = sums_ref(c, sk.tolist(), lk, block)
        assert torch.equal(sums.cpu(), want)
        r = ref.attention(Qr, c, sq.tolist(), sk.tolist(), lk, idx.cpu(), block)
        ref.check(out, r, "out", 7.0)
        ref.check(lse, r, "lse", 7.0)
        outs.append((out.clone(), lse.clone()))

    c2, sums2, new2, sq2, sk2, ln2 = decode_state(bits, S, H, Hkv, D, start, steps, block)
    ins = [t.clone() for t in new2[0]]
    args = (c2, sums2, *ins, freqs, sq2, sk2, ln2, block, topk, room)
    keep = [t.clone() for t in (c2.k, c2.v, c2.par, sums2, ln2)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        decode_step(*args)  # warm-up
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = decode_step(*args)
    for t, k in zip((c2.k, c2.v, c2.par, sums2, ln2), keep):
        t.copy_(k)
    for t in range(steps):
        for a, b in zip(ins, new2[t]):
            a.copy_(b)
        graph.replay()
        assert torch.equal(got[0], outs[t][0]) and torch.equal(got[1], outs[t][1])


def test_two_graphs():
    """Two captured graphs of the split form, replayed at the same time, keep apart."""
    calls = []
    for seed in (60, 61):
        Q, c, sq, sk, lk, kw, out, lse = attend(seed, [1], [18000], 4, 1, 128, "bf16", 8, extra=0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, z = gb.gattn_cache_fwd(Q, c, sq, sk, lk, **kw)
        calls.append((g, o, z, out, lse, torch.cuda.Stream(), (Q, c, sq, sk, lk)))
    for _ in range(20):
        for g, *_, st, _ in calls:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, o, z, out, lse, *_ in calls:
        assert torch.equal(o, out) and torch.equal(z, lse)


def test_chunk_through_block_attention():
    """Several queries at once: the cache read back, and block attention over what comes back."""
    S, lq, lk, H, Hkv, D = 2, [100, 37], [300, 37], 4, 2, 64
    sq, sk = ref.offsets(lq), ref.offsets([n + 9 for n in lk])
    c = gb.gattn_cache_new(sk[-1], Hkv, D, 4)
    ref.filled(c, randn(70, sk[-1], Hkv, D), randn(71, sk[-1], Hkv, D))
    Q = randn(72, sq[-1], H, D, dtype=torch.bfloat16)
    so = i32(ref.offsets(lk))
    K, V = gb.gattn_cache_read(c, so, i32(sk), i32(lk), since=i32([0, 0]), rows=sum(lk))
    sums = gb.gattn_cache_sums(c, i32(sk), 64, lens=i32(lk))
    idx = gb.gattn_block_select(Q, sums, i32(sq), i32(sk), 2, 64, 32, c.rows, len_k=i32(lk), causal=True)
    out, lse = gb.gattn_block_fwd(Q, K, V, idx, i32(sq), so, 64, 32, causal=True)
    r = block_ref.attention(Q, K, V, idx, sq, so.tolist(), 64, 32, causal=True)
    block_ref.check(out, r, "out", 7.0)
    block_ref.check(lse, r, "lse", 7.0)
