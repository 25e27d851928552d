"""The block-attention and norm operators through autograd, and a transformer layer that runs
them together with the attention over edges, against compositions in 64 bits."""
import math

import pytest

from gnn_sparse_attention_gb300 import synth
from tests.helpers import TOL, relerr

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu

from gnn_sparse_attention_gb300 import binding as gb  # noqa: E402
from gnn_sparse_attention_gb300 import layer  # noqa: E402
from tests import block_ref as ref  # noqa: E402

DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def np64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_block_attention_autograd(dtype, causal):
    torch.manual_seed(0)
    sq = [0, 150, 150, 231]
    H, Hkv, D = 4, 2, 64
    # ten more rows than the sequences hold: they get zeros, also as gradients
    Q, K, V = (torch.randn(241, h, D, device=DEV).to(dtype).requires_grad_() for h in (H, Hkv, Hkv))
    G = torch.randn(241, H, D, device=DEV).to(dtype)
    out, lse, idx = layer.block_attention(Q, K, V, i32(sq), topk=2, block=32, q_block=32, causal=causal)
    want = ref.select(Q.detach(), K.detach(), sq, sq, 2, 32, 32, causal)
    assert torch.equal(idx[:want.shape[0]].cpu(), want)
    out.backward(G)
    r = ref.attention(Q.detach(), K.detach(), V.detach(), idx, sq, sq, 32, 32, causal=causal, dout=G)
    ref.check(out.detach(), r, "out", 0.0)
    ref.check(lse, r, "lse", 0.0)
    for t, n in ((Q, "dQ"), (K, "dK"), (V, "dV")):
        ref.check(t.grad, r, n, 0.0)


def test_block_attention_serves_a_cache():
    """One new token per sequence against keys with room behind them, through the layer call."""
    torch.manual_seed(1)
    S, room, H, Hkv, D = 3, 128, 8, 2, 64
    Q = torch.randn(S, H, D, device=DEV).to(torch.bfloat16)
    K, V = (torch.randn(S * room, Hkv, D, device=DEV).to(torch.bfloat16) for _ in range(2))
    lens, sk, sq = [100, 1, 128], [0, room, 2 * room, 3 * room], [0, 1, 2, 3]
    out, lse, idx = layer.block_attention(Q, K, V, i32(sq), topk=3, block=16, q_block=1, causal=True,
                                          seq_k=i32(sk), len_k=i32(lens))
    assert torch.equal(idx.cpu(), ref.select(Q, K, sq, sk, 3, 16, 1, True, lens))
    r = ref.attention(Q, K, V, idx, sq, sk, 16, 1, causal=True, lk=lens)
    ref.check(out, r, "out")
    ref.check(lse, r, "lse")


def test_block_attention_told_the_longest_sequence():
    """The most keys of a sequence bound the work of the choice, not its result."""
    torch.manual_seed(2)
    Q, K, V = (torch.randn(600, 2, 32, device=DEV) for _ in range(3))
    seq = i32([0, 250, 251, 600])
    a = layer.block_attention(Q, K, V, seq, topk=3, block=16, q_block=32)
    b = layer.block_attention(Q, K, V, seq, topk=3, block=16, q_block=32, max_len_k=349)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gated_residual_norm_autograd(kind):
    torch.manual_seed(2)
    N, F = 50, 96
    leaf = {k: torch.randn(N, F, device=DEV, requires_grad=True) for k in ("res", "x", "gate")}
    leaf.update({k: (torch.randn(F, device=DEV) * 0.2 + 1).requires_grad_() for k in
                 ("w_post", "b_post", "w_pre", "b_pre")})
    gh, gy = torch.randn(N, F, device=DEV), torch.randn(N, F, device=DEV)
    h, y = layer.gated_residual_norm(**leaf, alpha=0.5, kind=kind, eps=1e-5)
    torch.autograd.backward([h, y], [gh, gy])
    d = {k: v.detach().double().requires_grad_() for k, v in leaf.items()}

    def norm(v, w, b):
        v = v - v.mean(-1, keepdim=True) if kind == "layer" else v
        return v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + 1e-5) * w + b

    h64 = d["res"] + 0.5 * d["gate"] * norm(d["x"], d["w_post"], d["b_post"])
    y64 = norm(h64, d["w_pre"], d["b_pre"])
    torch.autograd.backward([h64, y64], [gh.double(), gy.double()])
    assert relerr(np64(h), np64(h64)) < TOL["f32"] and relerr(np64(y), np64(y64)) < TOL["f32"]
    for k in leaf:
        assert relerr(np64(leaf[k].grad), np64(d[k].grad)) < TOL["f32"], k


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_slices_and_gradients_of_slices(dtype):
    """Columns of a wider tensor, rows and vectors that start off a 16-byte border, and gradients
    that arrive as such slices: the results of packed copies."""
    torch.manual_seed(7)
    N, F = 40, 33
    # what a network has in hand: two parts of one projection, rows behind the first, a vector's tail
    both = torch.randn(N + 1, 3 * F, device=DEV).to(dtype).requires_grad_()
    rows = torch.randn(N + 1, F, device=DEV).to(dtype).requires_grad_()
    vec = (1 + 0.1 * torch.randn(F + 1, device=DEV)).requires_grad_()
    gy, gh = torch.randn(2 * N, F, device=DEV).to(dtype), torch.randn(2 * N, F, device=DEV).to(dtype)

    def step(same):
        x, gate, more = (same(t) for t in both[1:].chunk(3, -1))
        w = same(vec[1:])
        h, y = layer.gated_residual_norm(same(rows[1:]), x, gate, w, None, w, None)
        # (their gradients are slices that begin off a border)
        top = torch.cat([more[:-1], h[:-1], y[:1]]), torch.cat([more[:1], y[:-1], more[1:]])
        loss = (top[0] * gh[:2 * N - 1]).sum() + (top[1] * gy[:2 * N - 1]).sum()
        return (h, y, *torch.autograd.grad(loss, (both, rows, vec)))

    assert rows[1:].data_ptr() % 16 and vec[1:].data_ptr() % 16
    for a, b in zip(step(lambda t: t), step(lambda t: t.clone(memory_format=torch.contiguous_format))):
        assert torch.equal(a, b)
    # attention: a flat buffer's views, off a border
    sq, n = [0, 70], 70 * 2 * 16
    flat = torch.randn(3 * n + 1, device=DEV).to(dtype).requires_grad_()
    wide = torch.randn(n + 1, device=DEV).to(dtype)

    def attend(same):
        Q, K, V = (same(t).view(70, 2, 16) for t in flat[1:].split(n))
        out, lse, _ = layer.block_attention(Q, K, V, i32(sq), topk=2, block=16, q_block=16)
        # (the cut's gradient is a view of the flat gradient)
        all_ = torch.cat([flat[:1], out.reshape(-1)])
        return out, lse, *torch.autograd.grad((all_ * wide).sum(), flat)

    for a, b in zip(attend(lambda t: t), attend(lambda t: t.clone())):
        assert torch.equal(a, b)


def test_second_derivatives_are_refused():
    """A gradient penalty would silently lose the part that goes through these operators."""
    torch.manual_seed(8)
    Q, K, V = (torch.randn(40, 2, 16, device=DEV, requires_grad=True) for _ in range(3))
    out = layer.block_attention(Q, K, V, i32([0, 40]), topk=1, block=16, q_block=16)[0]
    r, x, w = (torch.randn(*s, device=DEV, requires_grad=True) for s in ((20, 64), (20, 64), (64,)))
    h, y = layer.gated_residual_norm(r, x, w_pre=w)
    for res, leaf in ((out, Q), (out.pow(2), V), (y, x), (h + y.pow(2), w)):
        plain = torch.autograd.grad(res.sum(), leaf, retain_graph=True)[0]
        g = torch.autograd.grad(res.sum(), leaf, create_graph=True)[0]
        assert torch.equal(plain, g)
        with pytest.raises(RuntimeError, match="once"):
            (g.pow(2).sum() + leaf.sum()).backward()


def test_create_graph_alone_changes_nothing():
    """backward(create_graph=True) without a second derivative: gradients that an optimiser can
    detach, zero and add to."""
    torch.manual_seed(10)
    m = layer.GraphTransformerBlock(64, 2, 32, topk=2, dtype=torch.float32, device=DEV)
    h, seq = torch.randn(50, 64, device=DEV), i32([0, 50])
    opt = torch.optim.SGD(m.parameters(), lr=0.0)
    (m(h, seq).pow(2)).sum().backward()
    want = [p.grad.clone() for p in m.parameters()]
    opt.zero_grad(set_to_none=True)
    for _ in range(2):
        m(h, seq).pow(2).sum().backward(create_graph=True)
        assert all(torch.equal(p.grad, w) for p, w in zip(m.parameters(), want))
        opt.zero_grad(set_to_none=False)
    assert not any(p.grad.any() for p in m.parameters())


def test_gated_residual_norm_parts_without_a_gradient():
    """Only one of the two results is used; a gate or a norm is left out."""
    torch.manual_seed(3)
    x, r = (torch.randn(20, 64, device=DEV, requires_grad=True) for _ in range(2))
    w = torch.ones(64, device=DEV, requires_grad=True)
    h, y = layer.gated_residual_norm(r, x, w_pre=w)
    h.sum().backward()
    assert torch.equal(r.grad, torch.ones_like(r)) and torch.equal(x.grad, torch.ones_like(x))
    assert torch.equal(w.grad, torch.zeros_like(w))
    x.grad = r.grad = w.grad = None
    h, y = layer.gated_residual_norm(r, w_pre=w)
    y.sum().backward()
    assert r.grad is not None and w.grad is not None and torch.isfinite(r.grad).all()
    h, y = layer.gated_residual_norm(r, x, alpha=2.0)
    assert y is None and relerr(np64(h), np64(r) + 2 * np64(x)) < 1e-6


def _dense_block(m, h, seq, idx, ip, ix, block, q_block, causal):
    """GraphTransformerBlock in fp64 on the CPU: dense masks for the edges and for the blocks."""
    P = {n: p.detach().double().cpu().requires_grad_() for n, p in m.named_parameters()}
    h = h.detach().double().cpu().requires_grad_()
    N, H, D = h.shape[0], m.heads, m.head_dim
    edges = torch.zeros(N, N, dtype=torch.bool)
    for i in range(N):
        edges[i, ix[ip[i]:ip[i + 1]].tolist()] = True
    blocks = torch.zeros(H, N, N, dtype=torch.bool)
    for s in range(len(seq) - 1):
        a, n = seq[s], seq[s + 1] - seq[s]
        for k in range(H):
            blocks[k, a:a + n, a:a + n] = ref.allowed(idx.cpu(), s, k, n, n, a, block, q_block, causal, "cpu")

    def norm(v, name):
        v2 = v - v.mean(-1, keepdim=True) if m.kind == "layer" else v
        v2 = v2 / torch.sqrt(v2.pow(2).mean(-1, keepdim=True) + 1e-6) * P[f"w_{name}"]
        return v2 + P[f"b_{name}"] if m.kind == "layer" else v2

    def attend(q, k, v, ok):
        sc = (q @ k.T / math.sqrt(D)).masked_fill(~ok, -math.inf)
        p = torch.softmax(sc, -1)
        return torch.where(ok.any(1, keepdim=True), torch.nan_to_num(p), 0.0) @ v

    q, k, v = (t.reshape(N, H, D) for t in (norm(h, "in") @ P["qkv.weight"].T).chunk(3, -1))
    a = torch.stack([attend(q[:, i], k[:, i], v[:, i], blocks[i]) + attend(q[:, i], k[:, i], v[:, i], edges)
                     for i in range(H)], 1)
    h1 = h + P["gate_attn"] * norm(a.reshape(N, -1) @ P["o.weight"].T, "attn")
    mlp = torch.nn.functional.gelu(norm(h1, "mid") @ P["up.weight"].T) @ P["down.weight"].T
    return h1 + P["gate_mlp"] * norm(mlp, "mlp"), h, P


@pytest.mark.parametrize("kind,causal", [("rms", False), ("layer", True)])
def test_transformer_block_matches_a_dense_composition(kind, causal):
    """All operators in one layer, forward and gradients, fp32 (bar 1e-4 of the largest value)."""
    torch.manual_seed(4)
    seq = [0, 90, 90, 161]
    N, dim, H, D = seq[-1], 48, 2, 16
    ip, ix = synth.small_graph(5, N, 4.0, isolated=0.1)
    m = layer.GraphTransformerBlock(dim, H, D, mlp_dim=64, topk=2, block=16, q_block=16, causal=causal,
                                    kind=kind, gate_init=0.5, dtype=torch.float32, device=DEV)
    with torch.no_grad():
        for n, p in m.named_parameters():
            if n.startswith(("w_", "b_", "gate")):
                p.add_(0.1 * torch.randn_like(p))
    h = torch.randn(N, dim, device=DEV, requires_grad=True)
    plan = gb.gattn_plan_create(torch.from_numpy(ip).cuda(), torch.from_numpy(ix).cuda())
    try:
        # the choice, fixed for both sides
        with torch.no_grad():
            _, y = layer.gated_residual_norm(h, w_pre=m.w_in, b_pre=m.b_in, kind=kind)
            Q, K, _ = (t.reshape(N, H, D).contiguous() for t in m.qkv(y).chunk(3, -1))
            sums = gb.gattn_block_sums(K, i32(seq), 16)
            idx = gb.gattn_block_select(Q, sums, i32(seq), i32(seq), 2, 16, 16, N, causal=causal)
        out = m(h, i32(seq), plan)
        assert torch.equal(out, m(h, i32(seq), plan, idx=idx))
        g = torch.randn_like(out)
        out.backward(g)
        want, h64, P = _dense_block(m, h, seq, idx, ip, ix, 16, 16, causal)
        want.backward(g.double().cpu())
        assert relerr(np64(out), want.detach().numpy()) < TOL["f32"]
        assert relerr(np64(h.grad), h64.grad.numpy()) < TOL["f32"]
        for n, p in m.named_parameters():
            assert relerr(np64(p.grad), P[n].grad.numpy()) < TOL["f32"], n
    finally:
        plan.close()


def test_transformer_block_trains_in_bf16():
    """Two layers, a step of training on ragged graphs: runs, and every gradient is finite."""
    torch.manual_seed(5)
    seq = [0, 700, 701, 1300]
    ip, ix = synth.small_graph(6, seq[-1], 6.0)
    plan = gb.gattn_plan_create(torch.from_numpy(ip).cuda(), torch.from_numpy(ix).cuda())
    ms = [layer.GraphTransformerBlock(256, 4, 64, topk=4, kind=k, device=DEV) for k in ("rms", "layer")]
    h = torch.randn(seq[-1], 256, device=DEV).to(torch.bfloat16).requires_grad_()
    try:
        x = h
        for m in ms:
            x = m(x, i32(seq), plan)
        x.float().pow(2).mean().backward()
        torch.cuda.synchronize()
        gb.gattn_block_check_errors()
        assert torch.isfinite(x).all() and torch.isfinite(h.grad).all()
        for m in ms:
            for n, p in m.named_parameters():
                assert p.grad is not None and torch.isfinite(p.grad).all(), n
    finally:
        plan.close()


def test_training_step_in_a_graph():
    """A layer's forward and backward captured and replayed (its leaves used in no eager graph
    that is still alive)."""
    torch.manual_seed(6)
    seq = i32([0, 300, 420])
    m = layer.GraphTransformerBlock(128, 2, 64, topk=2, device=DEV)
    h = torch.randn(420, 128, device=DEV).to(torch.bfloat16)
    g = torch.randn(420, 128, device=DEV).to(torch.bfloat16)

    def step():
        grads = torch.autograd.grad(m(h, seq), list(m.parameters()), g)
        return [t.clone() for t in grads]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            want = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert relerr(np64(b), np64(a)) < 1e-2


def test_transformer_block_cast_whole():
    """module.to(bfloat16) casts the norms' weights and gates too: the layer still runs, with the
    results of the same values kept in fp32, and gradients in the parameters' type."""
    torch.manual_seed(9)
    seq = i32([0, 100, 180])
    m = layer.GraphTransformerBlock(64, 2, 32, topk=2, kind="layer", dtype=torch.float32, device=DEV)
    with torch.no_grad():
        for p in m.parameters():
            p.add_(0.1 * torch.randn_like(p))
    m = m.to(torch.bfloat16)
    h, g = (torch.randn(180, 64, device=DEV).to(torch.bfloat16) for _ in range(2))
    out = m(h, seq)
    got = torch.autograd.grad(out, list(m.parameters()), g)
    for n, p in list(m.named_parameters()):
        if p.dim() == 1:
            setattr(m, n, torch.nn.Parameter(p.detach().float()))
    want = m(h, seq)
    assert torch.equal(out, want)
    for p, a, b in zip(m.parameters(), got, torch.autograd.grad(want, list(m.parameters()), g)):
        assert a.dtype == torch.bfloat16 and torch.equal(a, b.to(torch.bfloat16))


@pytest.mark.parametrize("seq", [[0], [0, 0, 0]])
def test_transformer_block_without_nodes(seq):
    """An empty batch: no rows out, and gradients that are zeros."""
    m = layer.GraphTransformerBlock(64, 2, 32, topk=2, dtype=torch.float32, device=DEV)
    h = torch.zeros(0, 64, device=DEV, requires_grad=True)
    out = m(h, i32(seq))
    assert out.shape == (0, 64)
    out.sum().backward()
    assert h.grad.shape == h.shape
    assert all(p.grad is not None and not p.grad.any() for p in m.parameters())
