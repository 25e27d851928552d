"""The gated residual norm on the GPU against its definition in 64 bits.

Bounds: u = 2^-8 (bf16) or 2^-24 (fp32) for the one rounding of each output; c =
(F + 64) 2^-24 for the fp32 row sums and c_n = (N + 64) 2^-24 for column sums,
each times the sum of magnitudes.  The error of a normalised row (its
statistics' c) goes through the formulas below to first order, doubled for what
is beyond.
"""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu

from gnn_sparse_attention_gb300 import binding as gb  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def inputs(N, F, dtype, gate, post, pre, bias, seed=0):
    dt = DT[dtype]
    a = {"res": randn(seed, N, F, dtype=dt), "x": (0.5 * randn(seed + 1, N, F) + 0.3).to(dt)}
    a["gate"] = {"none": None, "channel": randn(seed + 2, F), "token": randn(seed + 2, N, F, dtype=dt)}[gate]
    for n, on, k in (("w_post", post, 3), ("b_post", post and bias, 4), ("w_pre", pre, 5),
                     ("b_pre", pre and bias, 6)):
        a[n] = (1 + 0.3 * randn(seed + k, F)) if on else None
    return a


def norm64(v, w, b, kind, eps):
    m = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
    r = 1 / torch.sqrt((v - m).pow(2).mean(-1, keepdim=True) + eps)
    vh = (v - m) * r
    y = vh * w
    return (y if b is None else y + b), vh, r, m


def within(got, want, tol, name):
    over = ((got.double() - want).abs() - tol).max().item() if got.numel() else -1.0
    assert over <= 0, f"{name}: over its bound by {over:.3e} (bound there about {tol.mean():.3e})"


def check(N, F, dtype, kind="rms", gate="token", post=True, pre=True, bias=True, alpha=0.7,
          with_dh=True, eps=1e-5, a=None):
    a = a or inputs(N, F, dtype, gate, post, pre, bias)
    u, c, cn = UNIT[dtype], (F + 64) * 2.0 ** -24, (N + 64) * 2.0 ** -24
    par = {k: a[k] for k in ("w_post", "b_post", "w_pre", "b_pre")}
    h, y, stats = gb.gattn_norm_fwd(a["res"], a["x"], a["gate"], alpha=alpha, kind=kind, eps=eps, **par)
    d = {k: None if v is None else v.double() for k, v in a.items()}
    g = 1.0 if d["gate"] is None else d["gate"]
    un, xh, rx, mx = norm64(d["x"], d["w_post"], d["b_post"], kind, eps) if post else (d["x"], None, None, None)
    h64 = d["res"] + alpha * g * un
    # a normalised row: its statistics carry c of the row's size
    xe = 4 * c * (xh.abs() + (d["x"].abs().mean(-1, keepdim=True) + mx.abs()) * rx) if post else 0 * un
    ue = xe * (d["w_post"].abs() if post else 1) + 4 * 2.0 ** -24 * (un.abs() + (d["b_post"].abs() if d["b_post"] is not None else 0))
    he = alpha * abs(g) * ue + 4 * 2.0 ** -24 * (d["res"].abs() + (alpha * g * un).abs())
    within(h, h64, u * h64.abs() + he, "h")
    if pre:
        y64, hh, rh, mh = norm64(h64, d["w_pre"], d["b_pre"], kind, eps)
        hhe = 4 * c * (hh.abs() + (h64.abs().mean(-1, keepdim=True) + mh.abs()) * rh) + 2 * rh * (
            he + he.mean(-1, keepdim=True) * (1 + hh.abs() * (hh.abs().amax(-1, keepdim=True))))
        within(y, y64, u * y64.abs() + hhe * d["w_pre"].abs() + 4 * 2.0 ** -24 * (y64.abs() + hh.abs() * d["w_pre"].abs()), "y")
    else:
        assert y is None
    dh = randn(20, N, F, dtype=DT[dtype]) if with_dh else None
    dy = randn(21, N, F, dtype=DT[dtype]) if pre else None
    got = gb.gattn_norm_bwd(a["res"], stats, dh, dy, a["x"], a["gate"], alpha=alpha, kind=kind, **par)

    def back(gp, vh, r):
        m = (gp * vh).mean(-1, keepdim=True)
        m2 = gp.mean(-1, keepdim=True) if kind == "layer" else 0.0
        return r * (gp - vh * m - m2)

    dd = dh.double() if with_dh else torch.zeros_like(h64)
    de = 4 * 2.0 ** -24 * dd.abs()
    if pre:
        gp = dy.double() * d["w_pre"]
        e = hhe
        add = back(gp, hh, rh)
        mean = (gp * hh).abs().mean(-1, keepdim=True)
        de = de + 2 * rh * (e * mean + hh.abs() * (gp.abs() * e).mean(-1, keepdim=True)) + 8 * c * rh * (
            gp.abs() + hh.abs() * mean + gp.abs().mean(-1, keepdim=True))
        dd = dd + add
        within(got["dw_pre"], (dy.double() * hh).sum(0), 2 * (dy.double().abs() * e).sum(0) + 2 * cn * (dy.double() * hh).abs().sum(0), "dw_pre")
        if a["b_pre"] is not None:
            within(got["db_pre"], dy.double().sum(0), 2 * cn * dy.double().abs().sum(0), "db_pre")
        assert (got["db_pre"] is None) == (a["b_pre"] is None)
    else:
        assert got["dw_pre"] is None and got["db_pre"] is None
    within(got["dres"], dd, u * dd.abs() + de, "dres")
    du, due = alpha * g * dd, abs(alpha) * abs(g) * de + 4 * 2.0 ** -24 * (alpha * g * dd).abs()
    dg, dge = alpha * dd * un, abs(alpha) * (de * un.abs() + dd.abs() * ue) + 4 * 2.0 ** -24 * (alpha * dd * un).abs()
    if a["gate"] is None:
        assert got["dgate"] is None
    elif a["gate"].dim() == 1:
        within(got["dgate"], dg.sum(0), dge.sum(0) + 2 * cn * dg.abs().sum(0), "dgate")
    else:
        within(got["dgate"], dg, u * dg.abs() + dge, "dgate")
    if post:
        within(got["dw_post"], (du * xh).sum(0), (due * xh.abs() + du.abs() * xe).sum(0) + 2 * cn * (du * xh).abs().sum(0), "dw_post")
        if a["b_post"] is not None:
            within(got["db_post"], du.sum(0), due.sum(0) + 2 * cn * du.abs().sum(0), "db_post")
        gp, gpe = du * d["w_post"], due * d["w_post"].abs()
        dx = back(gp, xh, rx)
        mean = (gp * xh).abs().mean(-1, keepdim=True)
        dxe = rx * (gpe + xh.abs() * (gpe * xh.abs()).mean(-1, keepdim=True) + gpe.mean(-1, keepdim=True)) + 8 * c * rx * (
            gp.abs() + xh.abs() * mean + gp.abs().mean(-1, keepdim=True)) + 2 * rx * (
            xe * mean + xh.abs() * (gp.abs() * xe).mean(-1, keepdim=True))
    else:
        dx, dxe = du, due
    within(got["dx"], dx, u * dx.abs() + dxe, "dx")
    return a, h, y, got


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("F", [1, 7, 8, 64, 129, 256, 257, 515, 1000, 1024, 1032, 4096, 4100, 8200, 16384])
def test_row_sizes(F, dtype, kind):
    check(37, F, dtype, kind)


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post,pre,bias,with_dh", [(True, True, False, True), (True, True, True, False),
                                                   (False, True, True, True), (True, False, True, True),
                                                   (False, False, False, True)])
@pytest.mark.parametrize("kind,dtype,F", [("rms", "bf16", 512), ("layer", "f32", 130)])
def test_parts(kind, dtype, F, gate, post, pre, bias, with_dh):
    check(65, F, dtype, kind, gate, post, pre, bias, with_dh=with_dh)


@pytest.mark.parametrize("N", [0, 1, 2, 3, 5, 5000])
@pytest.mark.parametrize("dtype,F", [("bf16", 128), ("f32", 1024), ("bf16", 2049)])
def test_row_counts(N, dtype, F):
    check(N, F, dtype, "layer", "channel")


@pytest.mark.parametrize("gate", ["channel", "token"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,F", [(12000, 257), (9000, 520), (6000, 777), (5000, 1026), (3000, 2048), (2000, 2056),
                                 (1500, 4095), (1000, 5120), (800, 8191), (800, 8192), (600, 8200), (600, 16384)])
def test_many_rows_of_every_shape(N, F, dtype, gate):
    """Rows enough that every CTA walks four and more, at each way that a row is laid out."""
    check(N, F, dtype, "layer", gate)


@pytest.mark.parametrize("F", [64, 1024])
def test_first_norm_of_a_model(F):
    """Without x: h is res, y its norm; the gradient of res is that of y plus dh."""
    res, w, dy, dh = randn(1, 50, F), randn(2, F), randn(3, 50, F), randn(4, 50, F)
    h, y, stats = gb.gattn_norm_fwd(res, w_pre=w, eps=1e-6)
    assert h is res
    r = res.double().requires_grad_()
    w64 = w.double().requires_grad_()
    y64 = r / torch.sqrt(r.pow(2).mean(-1, keepdim=True) + 1e-6) * w64
    c = (F + 64) * 2.0 ** -24
    within(y, y64.detach(), 4 * c * y64.detach().abs(), "y")
    torch.autograd.backward([y64, r], [dy.double(), dh.double()])
    g = gb.gattn_norm_bwd(res, stats, dh, dy, w_pre=w)
    assert g["dx"] is None and g["dgate"] is None
    scale = 16 * c * (dh.double().abs() + (dy * w).double().abs() + (dy * w).double().abs().mean(-1, keepdim=True) * (1 + 4 * res.double().abs()))
    within(g["dres"], r.grad, scale, "dres")
    within(g["dw_pre"], w64.grad, 16 * c * (dy.double() * y64.detach() / w.double()).abs().sum(0), "dw_pre")


def test_constant_and_large_rows():
    """Rows without deviation, and a mean that is large against the deviation."""
    a = inputs(6, 1024, "f32", "none", True, True, True)
    a["x"][0] = 3.0
    a["x"][1] = 0.0
    a["x"][2] += 1000.0
    check(6, 1024, "f32", "layer", "none", a=a, eps=1e-3)


def test_h_may_be_res():
    a = inputs(33, 1000, "bf16", "token", True, True, True)
    par = {k: a[k] for k in ("w_post", "b_post", "w_pre", "b_pre")}
    h, y, _ = gb.gattn_norm_fwd(a["res"], a["x"], a["gate"], **par)
    r = a["res"].clone()
    h2, y2, _ = gb.gattn_norm_fwd(r, a["x"], a["gate"], h=r, **par)
    assert h2 is r and torch.equal(h, h2) and torch.equal(y, y2)


def test_gradients_against_differences():
    a = inputs(9, 70, "f32", "token", True, True, True)
    dh, dy = randn(20, 9, 70), randn(21, 9, 70)
    par = {k: a[k] for k in ("w_post", "b_post", "w_pre", "b_pre")}
    for kind in ("rms", "layer"):
        h, y, st = gb.gattn_norm_fwd(a["res"], a["x"], a["gate"], alpha=0.7, kind=kind, eps=1e-5, **par)
        got = gb.gattn_norm_bwd(a["res"], st, dh, dy, a["x"], a["gate"], alpha=0.7, kind=kind, **par)

        def loss(t):
            u = norm64(t["x"], t["w_post"], t["b_post"], kind, 1e-5)[0]
            hh = t["res"] + 0.7 * t["gate"] * u
            return ((hh * dh.double()).sum() + (norm64(hh, t["w_pre"], t["b_pre"], kind, 1e-5)[0] * dy.double()).sum()).item()

        for i, n in enumerate(a):
            t = {k: v.double() for k, v in a.items()}
            v = randn(40 + i, *a[n].shape).double()
            e = 1e-5
            diff = (loss({**t, n: t[n] + e * v}) - loss({**t, n: t[n] - e * v})) / (2 * e)
            dot = (got["d" + n].double() * v).sum().item()
            # fp32 sums of 630 products (2^-24 x 700 of their magnitudes) and e^2 of the difference
            size = (got["d" + n].double() * v).abs().sum().item()
            assert abs(dot - diff) <= 2.0 ** -24 * 700 * 4 * size + 1e-5, (kind, n, dot, diff)


def test_captured_and_repeated():
    a = inputs(3000, 1024, "bf16", "channel", True, True, True)
    par = {k: a[k] for k in ("w_post", "b_post", "w_pre", "b_pre")}
    dh, dy = randn(20, 3000, 1024, dtype=torch.bfloat16), randn(21, 3000, 1024, dtype=torch.bfloat16)

    def step():
        h, y, st = gb.gattn_norm_fwd(a["res"], a["x"], a["gate"], kind="layer", **par)
        return [h, y, *gb.gattn_norm_bwd(a["res"], st, dh, dy, a["x"], a["gate"], kind="layer", **par).values()]

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for t in got:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_offsets_beyond_32_bits():
    """The last rows of tensors of more than 2^31 elements are those of a call on them alone."""
    N, F, n = 2_200_000, 1000, 37
    if torch.cuda.mem_get_info()[0] < 10 * N * F * 2:
        pytest.skip("needs more device memory")
    res, x, dy = (torch.zeros(N, F, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    for i, t in enumerate((res, x, dy)):
        t[-n:] = randn(30 + i, n, F, dtype=torch.bfloat16)
    w = 1 + 0.3 * randn(33, F)
    whole = gb.gattn_norm_fwd(res, x, None, w_post=w, w_pre=w)
    tail = gb.gattn_norm_fwd(res[-n:].clone(), x[-n:].clone(), None, w_post=w, w_pre=w)
    assert all(torch.equal(a[-n:], b) for a, b in zip(whole, tail))
    a = gb.gattn_norm_bwd(res, whole[2], None, dy, x, w_post=w, w_pre=w)
    b = gb.gattn_norm_bwd(res[-n:].clone(), tail[2], None, dy[-n:].clone(), x[-n:].clone(),
                          w_post=w, w_pre=w)
    assert torch.equal(a["dres"][-n:], b["dres"]) and torch.equal(a["dx"][-n:], b["dx"])
