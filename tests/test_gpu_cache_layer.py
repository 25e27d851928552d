"""rotary, GraphTransformerBlock with positions, and BlockCache on the GPU."""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu

from gnn_sparse_attention_gb300 import binding as gb, layer  # noqa: E402
from tests import cache_ref as ref  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def turned(x, pos, rad, layout, amp=1.0):
    """Rotary positions in torch operations, differentiable, in x's type."""
    R = 2 * len(rad)
    t = pos.double()[:, None] * rad.to(x.device)
    c, s = (amp * t.cos()).to(x.dtype)[:, None], (amp * t.sin()).to(x.dtype)[:, None]
    r = x[..., :R]
    a, b = (r[..., :R // 2], r[..., R // 2:]) if layout == "half" else (r[..., 0::2], r[..., 1::2])
    p, q = a * c - b * s, a * s + b * c
    y = torch.cat([p, q], -1) if layout == "half" else torch.stack([p, q], -1).flatten(-2)
    return torch.cat([y, x[..., R:]], -1)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rotary_autograd(dtype, layout):
    """Gradients of slices of a joint projection against autograd in 64 bits and the formula's bound."""
    N, H, Hkv, D, R = 37, 4, 2, 64, 32
    qkv = randn(1, N, (H + 2 * Hkv) * D, dtype=DT[dtype]).requires_grad_()
    Q, K, _ = qkv.split([H * D, Hkv * D, Hkv * D], 1)
    f, rad = gb.gattn_rotary_freqs(R), ref.frequencies(R)
    seq = i32([0, 20, 20, 37])
    pos = torch.cat([torch.arange(20), torch.arange(17)])
    q, k = layer.rotary(Q.unflatten(1, (H, D)), K.unflatten(1, (Hkv, D)), f, layout, seq=seq, amp=1.1)
    gq, gk = randn(2, N, H, D, dtype=DT[dtype]), randn(3, N, Hkv, D, dtype=DT[dtype])
    grad, = torch.autograd.grad([q, k], [qkv], [gq, gk])
    for g, w, h in ((gq, grad[:, :H * D], H), (gk, grad[:, H * D:(H + Hkv) * D], Hkv)):
        y, tol = ref.rotary(g, pos, rad, layout, 1.1, inverse=True)
        assert bool(((w.reshape(N, h, D).cpu().double() - y).abs() <= tol).all())
    assert bool((grad[:, (H + Hkv) * D:] == 0).all())
    x = qkv.detach().double().requires_grad_()
    q64 = turned(x[:, :H * D].unflatten(1, (H, D)), pos.to(DEV), rad, layout, 1.1)
    k64 = turned(x[:, H * D:(H + Hkv) * D].unflatten(1, (Hkv, D)), pos.to(DEV), rad, layout, 1.1)
    want, = torch.autograd.grad([q64, k64], [x], [gq.double(), gk.double()])
    # one rounding to the type of values of up to amp (|a| + |b|)
    assert bool(((grad.double() - want).abs() <= ref.HALF[DT[dtype]] * 1.01 * want.abs() + 2.0 ** -19).all())


def test_rotary_against_differences():
    x = randn(4, 5, 2, 16).requires_grad_()
    f = gb.gattn_rotary_freqs(16)
    pos = i32([0, 3, 10, 500, 70000])
    w = randn(5, 5, 2, 16)
    y, none = layer.rotary(x, None, f, pos=pos)
    assert none is None
    grad, = torch.autograd.grad((y * w).sum(), x)
    for i in range(0, 160, 13):  # the map is linear: a step of one is as good as any
        d = torch.zeros(160, device=DEV)
        d[i] = 1.0
        d = d.view(5, 2, 16)
        diff = ((gb.gattn_rotary(d, f, pos=pos)[0] * w).sum()).item()
        assert abs(diff - grad.view(-1)[i].item()) <= 2.0 ** -20 * 8


def test_rotary_twice_differentiable():
    x = randn(6, 7, 2, 32).requires_grad_()
    f = gb.gattn_rotary_freqs(32)
    pos = i32(list(range(7)))
    y, _ = layer.rotary(x, None, f, pos=pos)
    g, = torch.autograd.grad((y ** 3).sum(), x, create_graph=True)
    h, = torch.autograd.grad((g * randn(7, 7, 2, 32)).sum(), x)
    z = x.detach().double().requires_grad_()
    y64 = turned(z, pos, ref.frequencies(32), "half")
    g64, = torch.autograd.grad((y64 ** 3).sum(), z, create_graph=True)
    h64, = torch.autograd.grad((g64 * randn(7, 7, 2, 32).double()).sum(), z)
    # sums of two products of values below 6 ** 2 * 6 in fp32, a few roundings each
    assert float((h.double() - h64).abs().max()) <= 2.0 ** -23 * 20 * 6 ** 3


def test_rotary_rows_of_no_sequence_and_copies():
    x = randn(8, 12, 2, 32)
    f = gb.gattn_rotary_freqs(32)
    y, k = layer.rotary(x, x[:, :1], f, seq=i32([3, 8]))
    assert bool((y[:3] == 0).all()) and bool((y[8:] == 0).all()) and bool((k[8:] == 0).all())
    t = x.transpose(1, 2).contiguous().transpose(1, 2)  # heads do not lie side by side
    z, _ = layer.rotary(t, None, f, seq=i32([3, 8]))
    assert torch.equal(z, y)
    e = x[:1].expand(12, -1, -1)
    z, _ = layer.rotary(e, None, f, pos=i32(list(range(12))))
    assert torch.equal(z, layer.rotary(e.contiguous(), None, f, pos=i32(list(range(12))))[0])
    with pytest.raises(ValueError):
        layer.rotary(x, x.bfloat16(), f, seq=i32([3, 8]))


@pytest.mark.parametrize("rotary", [0, 32, 64])
def test_transformer_block_positions(rotary):
    """The block is the composition of its parts, with Q and K turned within their graphs."""
    torch.manual_seed(1)
    seq = i32([0, 70, 150])
    m = layer.GraphTransformerBlock(64, 2, 64, topk=8, block=32, causal=True, dtype=torch.float32, device=DEV,
                                    rotary=rotary)
    assert "freqs" not in m.state_dict()
    h = randn(9, 150, 64).requires_grad_()
    out = m(h, seq)
    pos = torch.cat([torch.arange(70), torch.arange(80)]).to(DEV)
    p = {n: v.detach().double() for n, v in m.named_parameters()}
    x = h.detach().double().requires_grad_()

    def norm(v, w):
        return v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + 1e-6) * w

    y = norm(x, p["w_in"])
    q, k, v = (t.unflatten(1, (2, 64)) for t in (y @ p["qkv.weight"].T).chunk(3, -1))
    if rotary:
        q, k = (turned(t, pos, ref.frequencies(rotary), "half") for t in (q, k))
    a = torch.zeros_like(q)
    for s, e in ((0, 70), (70, 150)):  # 8 blocks of 32: everything is chosen
        sc = torch.einsum("ihd,jhd->hij", q[s:e], k[s:e]) / 8
        sc = sc.masked_fill(torch.triu(torch.ones(e - s, e - s, dtype=torch.bool, device=DEV), 1), -math.inf)
        a[s:e] = torch.einsum("hij,jhd->ihd", sc.softmax(-1), v[s:e])
    g = x + p["gate_attn"] * norm(a.flatten(1) @ p["o.weight"].T, p["w_attn"])
    mlp = torch.nn.functional.gelu(norm(g, p["w_mid"]) @ p["up.weight"].T) @ p["down.weight"].T
    want = g + p["gate_mlp"] * norm(mlp, p["w_mlp"])
    w = randn(10, 150, 64)
    grad, = torch.autograd.grad(out, h, w)
    grad64, = torch.autograd.grad(want, x, w.double())
    # dense fp32 products and norms of a layer: about 1e-6 of the largest value each
    out, want = out.detach(), want.detach()
    assert float((out.double() - want).abs().max()) <= 1e-4 * float(want.abs().max())
    assert float((grad.double() - grad64).abs().max()) <= 1e-4 * float(grad64.abs().max())


def test_training_step_with_positions_in_a_graph():
    torch.manual_seed(2)
    seq = i32([0, 100, 180])
    m = layer.GraphTransformerBlock(64, 2, 64, topk=2, causal=True, device=DEV, rotary=64)
    h, g = randn(11, 180, 64, dtype=torch.bfloat16), randn(12, 180, 64, dtype=torch.bfloat16)

    def step():
        return torch.autograd.grad(m(h, seq), list(m.parameters()), g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            want = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert float((a.double() - b.double()).norm()) <= 1e-2 * float(a.double().norm())


@pytest.mark.parametrize("topk", [0, 3])
@pytest.mark.parametrize("bits", [4, 8])
def test_block_cache(bits, topk):
    """A prompt appended, then steps of one and of several rows, against the definitions."""
    S, H, Hkv, D, room = 2, 4, 2, 64, 200
    c = layer.BlockCache(S, room, Hkv, D, bits, topk=topk, block=32)
    f, rad = gb.gattn_rotary_freqs(D), ref.frequencies(D)
    prompt = [100, 37]
    n = sum(prompt)
    K, V = randn(13, n, Hkv, D, dtype=torch.bfloat16), randn(14, n, Hkv, D, dtype=torch.bfloat16)
    sq = i32(ref.offsets(prompt))
    c.append(gb.gattn_rotary(K, f, seq_q=sq)[0], V, sq)
    lens = list(prompt)
    for t, rows in enumerate(([1, 1], [1, 1], [3, 0], [1, 2])):
        o = ref.offsets(rows)
        qkv = randn(20 + t, o[-1], (H + 2 * Hkv) * D, dtype=torch.bfloat16)  # one projection's slices
        Q, K, V = (x.unflatten(1, (-1, D)) for x in qkv.split([H * D, Hkv * D, Hkv * D], 1))
        out, lse = c.step(Q, K, V, i32(o), freqs=f)
        lens = [a + b for a, b in zip(lens, rows)]
        assert c.length.tolist() == lens
        pos = [lens[s] - rows[s] + i for s in range(S) for i in range(rows[s])]
        y, tol = ref.rotary(Q, pos, rad, "half")
        q = gb.gattn_rotary(Q, f, pos=i32(pos))[0]
        assert bool(((q.cpu().double() - y).abs() <= tol).all())
        idx = None
        if topk:
            idx = gb.gattn_block_select(q, c.sums, i32(o), c.seq_k, topk, 32, 1, S * room,
                                        len_k=c.length, causal=True).cpu()
        r = ref.attention(q, c.cache, o, c.seq_k.tolist(), lens, idx, 32, causal=True)
        ref.check(out, r, "out", 7.0)
        ref.check(lse, r, "lse", 7.0)
    fresh = gb.gattn_cache_sums(c.cache, c.seq_k, 32, lens=c.length)
    for s in range(S):
        b = s * room // 32 + s
        nb = -(-lens[s] // 32)
        assert torch.equal(c.sums[b:b + nb], fresh[b:b + nb])


def test_block_cache_step_in_a_graph():
    S, H, Hkv, D, room = 3, 4, 2, 128, 128
    f = gb.gattn_rotary_freqs(D)
    seq = i32([0, 1, 2, 3])
    ins = [[randn(30 + 3 * t + i, S, h, D, dtype=torch.bfloat16) for i, h in enumerate((H, Hkv, Hkv))]
           for t in range(6)]

    def fresh():
        c = layer.BlockCache(S, room, Hkv, D, topk=2, block=16)
        K, V = randn(50, 90, Hkv, D, dtype=torch.bfloat16), randn(51, 90, Hkv, D, dtype=torch.bfloat16)
        c.append(K, V, i32([0, 30, 60, 90]))
        return c

    c = fresh()
    want = [tuple(t.clone() for t in c.step(*x, seq, freqs=f)) for x in ins]
    c = fresh()
    x = [t.clone() for t in ins[0]]
    keep = [t.clone() for t in (c.cache.k, c.cache.v, c.cache.par, c.sums, c.length)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        c.step(*x, seq, freqs=f)
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = c.step(*x, seq, freqs=f)
    for t, k in zip((c.cache.k, c.cache.v, c.cache.par, c.sums, c.length), keep):
        t.copy_(k)
    for t in range(6):
        for a, b in zip(x, ins[t]):
            a.copy_(b)
        g.replay()
        assert torch.equal(out, want[t][0]) and torch.equal(lse, want[t][1])


def test_block_cache_refused_calls_leave_it():
    """A call that is refused, early or late in its chain, leaves lengths as they were, and the call put right gives
    what it gives without the refused one."""
    S, H, Hkv, D, room = 2, 4, 2, 64, 64
    f = gb.gattn_rotary_freqs(D)
    seq = i32([0, 1, 2])
    K0, V0 = randn(60, 40, Hkv, D, dtype=torch.bfloat16), randn(61, 40, Hkv, D, dtype=torch.bfloat16)
    Q, K, V = (randn(62 + i, S, h, D, dtype=torch.bfloat16) for i, h in enumerate((H, Hkv, Hkv)))
    outs = []
    for refused in (False, True):
        c = layer.BlockCache(S, room, Hkv, D, topk=2, block=16)
        c.append(K0, V0, i32([0, 20, 40]))
        if refused:
            for q, k, v, s, kw in ((Q, K[:, :1], V, seq, {}), (Q, K, V.float(), seq, {}), (Q, K, V, seq.long(), {}),
                                   (Q, K, V, i32([0, 2]), {}), (Q[:, :3], K, V, seq, {}), (Q, K, V, seq, {"scale": -1.0}),
                                   (Q.half(), K.half(), V.half(), seq, {}), (Q, K, V, seq, {"layout": "other"})):
                with pytest.raises((ValueError, gb.GattnError)):
                    c.step(q, k, v, s, freqs=f, **kw)
                assert c.length.dtype == torch.int32 and c.length.tolist() == [20, 20]
            for k, v, s in ((K[:, :1], V, seq), (K, V, seq.long()), (K, V, i32([0, 2])), (K, V[:1], seq)):
                with pytest.raises((ValueError, gb.GattnError)):
                    c.append(k, v, s)
                assert c.length.tolist() == [20, 20]
        outs.append((*c.step(Q, K, V, seq, freqs=f), c.length.clone(), c.sums.clone()))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_block_cache_says_when_it_is_full():
    """A sequence that outgrows its room is told, and its neighbours keep their rows."""
    S, Hkv, D, room = 3, 2, 64, 32
    c = layer.BlockCache(S, room, Hkv, D, topk=0, block=16)
    K, V = randn(65, 96, Hkv, D), randn(66, 96, Hkv, D)
    c.append(K, V, i32([0, 32, 63, 95]))  # the first and the last are full
    c.check_errors()
    kept = [t.clone() for t in (c.cache.k, c.cache.v)]
    q = randn(67, 3, 4, D)
    c.step(q, K[:3], V[:3], i32([0, 0, 1, 1]))
    c.check_errors()
    c.step(q, K[:3], V[:3], i32([0, 1, 1, 1]))
    with pytest.raises(RuntimeError, match="0"):
        c.check_errors()
    for t, was in zip((c.cache.k, c.cache.v), kept):
        assert torch.equal(t[:, 2 * room:], was[:, 2 * room:])
        assert torch.equal(t[:, room:2 * room - 1], was[:, room:2 * room - 1])
