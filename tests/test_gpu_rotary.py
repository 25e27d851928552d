"""Rotary positions on the GPU against their definition (tests/cache_ref.py)."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu

from gnn_sparse_attention_gb300 import binding as gb  # noqa: E402
from tests import cache_ref as ref  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def near(got, x, pos, rad, layout, amp=1.0, inverse=False):
    y, tol = ref.rotary(x, pos, rad, layout, amp, inverse)
    err = (got.cpu().double() - y).abs() - tol
    assert bool((err <= 0).all()), f"{int((err > 0).sum())} beyond the bound, worst {float(err.max()):.3g}"


WIDTHS = [(128, 128), (128, 64), (64, 64), (64, 16), (32, 32), (16, 16), (128, 96), (64, 10), (10, 6), (7, 2),
          (256, 128), (1024, 1024), (64, 62), (128, 100), (72, 34), (8, 4)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,width", WIDTHS)
def test_widths(D, width, layout, dtype):
    pos = [0, 1, 2, 77, 4095, 131071, 1000003, 2 ** 31 - 1, -1, -500]
    Q, K = randn(1, 10, 4, D, dtype=DT[dtype]), randn(2, 10, 3, D, dtype=DT[dtype])
    f = gb.gattn_rotary_freqs(width)
    rad = ref.frequencies(width)
    for inverse in (False, True):
        q, k = gb.gattn_rotary(Q, f, K=K, layout=layout, pos=i32(pos), amp=1.25, inverse=inverse)
        near(q, Q, pos, rad, layout, 1.25, inverse)
        near(k, K, pos, rad, layout, 1.25, inverse)
    alone, none = gb.gattn_rotary(K, f, layout=layout, pos=i32(pos), amp=1.25, inverse=True)
    assert none is None and torch.equal(alone, k)


@pytest.mark.parametrize("kind", ["none", "linear", "base", "ramp"])
@pytest.mark.parametrize("width", [2, 4, 64, 128])
def test_scalings(kind, width):
    kw = {"scaling": kind, "factor": 8.0, "orig_len": 4096.0, "low": 1.0, "high": 16.0}
    f = gb.gattn_rotary_freqs(width, 500000.0, device="cpu", **kw)
    rad = ref.frequencies(width, 500000.0, **kw)
    turns = f.numpy().view("uint64").astype("float64") / 2.0 ** 64 * 6.283185307179586
    assert abs(turns - rad.numpy()).max() <= 2.0 ** -50
    x = randn(3, 5, 2, 128)
    pos = [0, 5, 8191, 100000, 16777217]
    near(gb.gattn_rotary(x, f.to(DEV), pos=i32(pos))[0], x, pos, rad, "half")


@pytest.mark.parametrize("N", [1, 3, 40, 1000, 9001])
@pytest.mark.parametrize("H,Hkv", [(1, 0), (32, 8), (3, 5)])
def test_rows_and_heads(N, H, Hkv):
    pos = torch.arange(N) * 3 + 11
    Q = randn(4, N, H, 64, dtype=torch.bfloat16)
    K = randn(5, N, Hkv, 64, dtype=torch.bfloat16) if Hkv else None
    f, rad = gb.gattn_rotary_freqs(64), ref.frequencies(64)
    q, k = gb.gattn_rotary(Q, f, K=K, pos=pos.int().to(DEV))
    near(q, Q, pos, rad, "half")
    if Hkv:
        near(k, K, pos, rad, "half")


@pytest.mark.parametrize("width", [64, 10])
@pytest.mark.parametrize("cached", [False, True])
def test_sequences(cached, width):
    """Positions of sequences; rows of none keep what they hold."""
    lq = [5, 0, 1, 30]
    lk = [5, 4, 900, 29] if cached else lq
    sq = [2 + x for x in ref.offsets(lq)]
    sk = ref.offsets([n + 3 for n in lk])
    N = sq[-1] + 4
    x = randn(6, N, 2, 64)
    kw = {"seq_q": i32(sq)}
    if cached:
        kw.update(seq_k=i32(sk), len_k=i32(lk))
    f, rad = gb.gattn_rotary_freqs(width), ref.frequencies(width)
    out = torch.full_like(x, 7.0)
    gb.gattn_rotary(x, f, out_q=out, **kw)
    assert bool((out[:2] == 7.0).all()) and bool((out[sq[-1]:] == 7.0).all())
    pos = [i + lk[s] - lq[s] for s in range(4) for i in range(lq[s])]
    near(out[2:sq[-1]], x[2:sq[-1]], pos, rad, "half")
    if cached:  # lengths by room
        y = torch.full_like(x, 7.0)
        gb.gattn_rotary(x, f, out_q=y, seq_q=i32(sq), seq_k=i32(ref.offsets(lk)))
        assert torch.equal(y, out)


@pytest.mark.parametrize("width", [64, 10])
def test_lengths_beyond_the_room(width):
    """The position is that of the attention, which cuts lengths to the room that seq_k leaves."""
    sq, sk, lk, cut = [0, 3, 5, 6], [0, 40, 45, 45], [41, 1000, 7], [40, 5, 0]
    x = randn(14, 6, 2, 64)
    f, rad = gb.gattn_rotary_freqs(width), ref.frequencies(width)
    pos = [i + cut[s] - (sq[s + 1] - sq[s]) for s in range(3) for i in range(sq[s + 1] - sq[s])]
    got, _ = gb.gattn_rotary(x, f, seq_q=i32(sq), seq_k=i32(sk), len_k=i32(lk))
    near(got, x, pos, rad, "half")
    same, _ = gb.gattn_rotary(x, f, seq_q=i32(sq), seq_k=i32(sk), len_k=i32(cut))
    assert torch.equal(got, same)
    less, _ = gb.gattn_rotary(x, f, seq_q=i32(sq), seq_k=i32(sk), len_k=i32([-1, -5, 0]))
    none, _ = gb.gattn_rotary(x, f, seq_q=i32(sq), seq_k=i32(sk), len_k=i32([0, 0, 0]))
    assert torch.equal(less, none)
    # without the room there is nothing to cut by
    pos = [i + lk[s] - (sq[s + 1] - sq[s]) for s in range(3) for i in range(sq[s + 1] - sq[s])]
    near(gb.gattn_rotary(x, f, seq_q=i32(sq), len_k=i32(lk))[0], x, pos, rad, "half")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_slices_and_in_place(layout, dtype):
    """Q and K as slices of a joint projection, aligned or not, into others and in place."""
    N, H, Hkv, D = 50, 4, 2, 64
    pos = torch.randint(0, 10000, (N,), generator=torch.Generator().manual_seed(1))
    f, rad = gb.gattn_rotary_freqs(32), ref.frequencies(32)
    for pad in (0, 1):
        qkv = randn(7, N, (H + 2 * Hkv) * D + pad, dtype=DT[dtype])
        Q = qkv[:, pad:pad + H * D].unflatten(1, (H, D))
        K = qkv[:, pad + H * D:pad + (H + Hkv) * D].unflatten(1, (Hkv, D))
        want = gb.gattn_rotary(Q.contiguous(), f, K=K.contiguous(), layout=layout, pos=pos.int().to(DEV))
        near(want[0], Q, pos, rad, layout)
        got = gb.gattn_rotary(Q, f, K=K, layout=layout, pos=pos.int().to(DEV))
        # other paths may form a product in another order of fused operations
        near(got[0], Q, pos, rad, layout)
        near(got[1], K, pos, rad, layout)
        q0, k0, rest = Q.clone(), K.clone(), qkv[:, pad + (H + Hkv) * D:].clone()
        gb.gattn_rotary(Q, f, K=K, layout=layout, pos=pos.int().to(DEV), out_q=Q, out_k=K)
        near(Q, q0, pos, rad, layout)
        near(K, k0, pos, rad, layout)
        assert torch.equal(qkv[:, pad + (H + Hkv) * D:], rest)


def test_gradient_is_the_inverse():
    """<rotary(x), y> = <x, inverse(y)>, and turning back returns the row."""
    f = gb.gattn_rotary_freqs(64)
    x, y = randn(8, 20, 4, 64), randn(9, 20, 4, 64)
    pos = i32(list(range(0, 200, 10)))
    a, b = gb.gattn_rotary(x, f, pos=pos)[0], gb.gattn_rotary(y, f, pos=pos, inverse=True)[0]
    lhs, rhs = (a.double() * y.double()).sum(), (x.double() * b.double()).sum()
    assert abs(lhs - rhs) <= 2.0 ** -20 * (x.double().norm() * y.double().norm())
    back = gb.gattn_rotary(a, f, pos=pos, inverse=True)[0]
    assert bool(((back - x).abs() <= 2.0 ** -19 * (1 + x.abs().max())).all())


def test_offsets_beyond_32_bits():
    N, H, D = 70000, 256, 128  # 2.3 G elements
    x = torch.zeros(N, H, D, dtype=torch.bfloat16, device=DEV)
    x[-2:] = randn(10, 2, H, D, dtype=torch.bfloat16)
    tail = x[-2:].clone()
    f, rad = gb.gattn_rotary_freqs(128), ref.frequencies(128)
    gb.gattn_rotary(x, f, seq_q=i32([0, N]), out_q=x)
    near(x[-2:], tail, [N - 2, N - 1], rad, "half")
    assert bool((x[:1000] == 0).all())


def test_another_stream_and_graph():
    f = gb.gattn_rotary_freqs(64)
    Q, K = randn(11, 16, 8, 64, dtype=torch.bfloat16), randn(12, 16, 2, 64, dtype=torch.bfloat16)
    pos = i32(list(range(16)))
    want = gb.gattn_rotary(Q, f, K=K, pos=pos)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = gb.gattn_rotary(Q, f, K=K, pos=pos, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = gb.gattn_rotary(Q, f, K=K, pos=pos)
    pos.add_(100)
    g.replay()
    want = gb.gattn_rotary(Q, f, K=K, pos=pos)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals():
    x, f = randn(13, 4, 2, 64), gb.gattn_rotary_freqs(64)
    pos = i32([0, 1, 2, 3])
    with pytest.raises(ValueError):
        gb.gattn_rotary(x, f)
    with pytest.raises(ValueError):
        gb.gattn_rotary(x, f, pos=pos, seq_q=i32([0, 4]))
    with pytest.raises(ValueError):
        gb.gattn_rotary(x, f, pos=pos, layout="other")
    with pytest.raises(ValueError):
        gb.gattn_rotary(x, f, K=x[:3], pos=pos)
    with pytest.raises(ValueError):
        gb.gattn_rotary(x, f.cpu(), pos=pos)
    with pytest.raises(ValueError):
        gb.gattn_rotary(x.transpose(0, 1), f, pos=pos[:2])
    with pytest.raises(ValueError):
        gb.gattn_rotary(x[:1].expand(4, -1, -1), f, pos=pos)
    with pytest.raises(gb.GattnError):
        gb.gattn_rotary(x, gb.gattn_rotary_freqs(66), pos=pos)
    with pytest.raises(gb.GattnError):
        gb.gattn_rotary(x.double(), f, pos=pos)
