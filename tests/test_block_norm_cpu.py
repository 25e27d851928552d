"""Refusals of the block-attention and norm entry points, on a machine without a GPU: every
check that the host makes answers before CUDA is touched."""
import ctypes

import pytest
import torch

from gnn_sparse_attention_gb300 import binding as gb
from gnn_sparse_attention_gb300 import build as gbuild

OK, INVALID, UNSUPPORTED = 0, 1, 3


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gb.load_library()


def block(**kw):
    d = dict(S=1, Nq=64, Nk=64, H=4, Hkv=2, D=64, dtype=1, block=64, q_block=64, topk=2, causal=0,
             scale=0.0, max_len_k=0, seq_q=4096, seq_k=4096, len_k=None, idx_stride=(0, 0))
    d.update(kw)
    d["idx_stride"] = (ctypes.c_int64 * 2)(*d["idx_stride"])
    return gb._BlockDesc(**d)


def size(lib, name, d):
    n = ctypes.c_size_t(77)
    return getattr(lib, name)(ctypes.byref(d), ctypes.byref(n)), n.value


SIZES = ("gattn_block_select_workspace_size", "gattn_block_fwd_workspace_size",
         "gattn_block_bwd_workspace_size")


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), INVALID), (dict(S=-1), INVALID), (dict(Nq=-1), INVALID), (dict(Nk=-1), INVALID),
    (dict(H=0), INVALID), (dict(topk=0), INVALID), (dict(D=-64), INVALID),
    (dict(D=48), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(D=4), UNSUPPORTED),
    (dict(D=2, dtype=0), UNSUPPORTED), (dict(H=6), UNSUPPORTED), (dict(Hkv=3), UNSUPPORTED),
    (dict(H=2, Hkv=4), UNSUPPORTED), (dict(H=256, Hkv=1, D=8), UNSUPPORTED),
    (dict(H=1024, Hkv=1024, D=128), UNSUPPORTED), (dict(block=8), UNSUPPORTED),
    (dict(block=48), UNSUPPORTED), (dict(block=256), UNSUPPORTED), (dict(q_block=3), UNSUPPORTED),
    (dict(q_block=256), UNSUPPORTED), (dict(q_block=0), UNSUPPORTED), (dict(topk=129), UNSUPPORTED),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(seq_q=None), INVALID), (dict(seq_k=None), INVALID),
    (dict(seq_k=4097), INVALID), (dict(max_len_k=-1), INVALID),
    (dict(Nk=2 ** 31 - 1), UNSUPPORTED),
    (dict(idx_stride=(-1, 2)), INVALID)])
def test_descriptors(lib, bad, status):
    d = block(**bad)
    for name in SIZES:
        assert size(lib, name, d)[0] == status, name
    assert b"gattn_block" in lib.gattn_last_error()
    p = ctypes.c_void_p(4096)
    assert lib.gattn_block_sums(ctypes.byref(d), p, None, p, None) == status
    assert lib.gattn_block_select(ctypes.byref(d), p, p, p, p, 1 << 30, None) == status
    assert lib.gattn_block_fwd(ctypes.byref(d), p, p, p, p, p, p, p, 1 << 40, None) == status
    assert lib.gattn_block_bwd(ctypes.byref(d), *[p] * 10, p, 1 << 40, None) == status


def test_null_descriptor_and_size(lib):
    for name in SIZES:
        assert getattr(lib, name)(None, None) == INVALID
        assert getattr(lib, name)(ctypes.byref(block()), None) == INVALID
    assert lib.gattn_block_fwd(None, *[None] * 7, 0, None) == INVALID


def test_pointers_and_workspaces(lib):
    d, p, odd = block(), ctypes.c_void_p(4096), ctypes.c_void_p(4100)
    for k in range(4):
        a = [p, p, p, p]
        for v in (None, odd):
            b = list(a)
            b[k] = v
            # Q, K, V misaligned or missing; idx and lse may be 4-byte aligned
            if k < 3:
                assert lib.gattn_block_fwd(ctypes.byref(d), *b[:3], p, p, p, p, 1 << 40, None) == INVALID
    assert lib.gattn_block_fwd(ctypes.byref(d), p, p, p, None, p, p, p, 1 << 40, None) == INVALID
    assert lib.gattn_block_fwd(ctypes.byref(d), p, p, p, p, None, p, p, 1 << 40, None) == INVALID
    assert lib.gattn_block_fwd(ctypes.byref(d), p, p, p, p, p, None, p, 1 << 40, None) == INVALID
    st, need = size(lib, "gattn_block_bwd_workspace_size", d)
    assert st == OK and need > 0
    for ws, n in ((None, need), (p, need - 1), (odd, need)):
        assert lib.gattn_block_bwd(ctypes.byref(d), *[p] * 10, ws, n, None) == INVALID
        assert b"workspace" in lib.gattn_last_error()
    st, need = size(lib, "gattn_block_select_workspace_size", d)
    assert st == OK and need > 0
    assert lib.gattn_block_select(ctypes.byref(d), p, p, p, p, need - 1, None) == INVALID
    assert size(lib, "gattn_block_select_workspace_size", block(q_block=1)) == (OK, 0)


def test_nothing_to_do_is_fine(lib):
    p = ctypes.c_void_p(4096)
    empty = block(S=0, Nq=0, Nk=0, seq_q=None, seq_k=None)
    assert lib.gattn_block_sums(ctypes.byref(empty), None, None, None, None) == OK
    assert lib.gattn_block_select(ctypes.byref(empty), None, None, None, None, 0, None) == OK
    assert lib.gattn_block_fwd(ctypes.byref(empty), *[None] * 7, 0, None) == OK
    assert lib.gattn_block_bwd(ctypes.byref(empty), *[None] * 11, 0, None) == OK
    norm_empty = norm(N=0)
    assert lib.gattn_norm_fwd(ctypes.byref(norm_empty), p, p, None, p, p, p, None) == OK


def norm(**kw):
    d = dict(N=4, F=64, dtype=1, kind=0, gate=0, alpha=1.0, eps=1e-5, w_post=4096, b_post=None,
             w_pre=4096, b_pre=None)
    d.update(kw)
    return gb._NormDesc(**d)


@pytest.mark.parametrize("bad,status", [
    (dict(N=-1), INVALID), (dict(N=2 ** 31), INVALID), (dict(F=0), INVALID), (dict(F=16385), UNSUPPORTED),
    (dict(dtype=5), INVALID), (dict(kind=2), INVALID), (dict(gate=3), INVALID),
    (dict(w_post=None, b_post=4096), INVALID), (dict(w_pre=None, b_pre=4096), INVALID),
    (dict(w_pre=4100), INVALID), (dict(b_post=4097), INVALID)])
def test_norm_descriptors(lib, bad, status):
    d, p = norm(**bad), ctypes.c_void_p(4096)
    n = ctypes.c_size_t()
    assert lib.gattn_norm_workspace_size(ctypes.byref(d), ctypes.byref(n)) == status
    assert lib.gattn_norm_fwd(ctypes.byref(d), p, p, None, p, p, p, None) == status
    assert lib.gattn_norm_bwd(ctypes.byref(d), *[p] * 13, p, 1 << 40, None) == status
    assert b"gattn_norm" in lib.gattn_last_error()


def test_norm_pointers(lib):
    p, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4104)

    def fwd(d, *a):
        return lib.gattn_norm_fwd(ctypes.byref(d), *a, None)

    assert fwd(norm(), p, None, None, p, p, p) == INVALID                     # w_post without x
    assert fwd(norm(w_post=None, w_pre=None), p, None, None, p, p, p) == INVALID   # nothing to do
    assert fwd(norm(gate=2), p, p, None, p, p, p) == INVALID                  # no gate
    for k in (0, 1, 3, 4, 5):
        for bad in (odd, None):
            if k == 1 and bad is None:
                continue
            a = [p, p, None, p, p, p]
            a[k] = bad
            assert fwd(norm(), *a) == INVALID, k

    def bwd(d, ws=p, n=1 << 40, **kw):
        a = dict(res=p, stats=p, dh=p, dy=p, x=p, gate=None, dres=p, dx=p, dgate=None, dw_post=p,
                 db_post=None, dw_pre=p, db_pre=None)
        a.update(kw)
        return lib.gattn_norm_bwd(ctypes.byref(d), *a.values(), ws, n, None)

    assert bwd(norm(), dy=None) == INVALID
    assert bwd(norm(w_pre=None), dw_pre=None, dy=None, dh=None) == INVALID
    assert bwd(norm(w_pre=None), dw_pre=p) == INVALID
    assert bwd(norm(w_post=None), dw_post=p) == INVALID
    assert bwd(norm(), dgate=p) == INVALID
    assert bwd(norm(), x=None) == INVALID
    assert bwd(norm(), res=None) == INVALID and bwd(norm(), stats=odd) == INVALID
    assert bwd(norm(), ws=None) == INVALID and bwd(norm(), n=16) == INVALID


def test_binding_refuses_host_tensors_and_shapes(lib):
    K, seq = torch.zeros(64, 2, 16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gb.gattn_block_sums(K, seq, 16)
    with pytest.raises(ValueError, match="CUDA"):
        gb.gattn_block_fwd(K, K, K, torch.zeros(1, 2, 1, dtype=torch.int32), seq, seq, 16, 64)
    with pytest.raises(ValueError, match="dimensions"):
        gb.gattn_block_sums(K[0], seq, 16)
    with pytest.raises(ValueError):
        gb.gattn_block_fwd(K, K, K[1:], torch.zeros(1, 2, 1, dtype=torch.int32), seq, seq, 16, 64)
    with pytest.raises(ValueError, match="CUDA"):
        gb.gattn_norm_fwd(K[0], K[0])
    with pytest.raises(ValueError, match="CUDA"):
        gb.gattn_norm_bwd(K[0], K[0])


def test_table_rows():
    """Every unit and block of any offsets has a table row of its own, inside the tables."""
    import random
    r = random.Random(0)
    for _ in range(300):
        S, per = r.randint(1, 9), 2 ** r.randint(0, 7)
        lens = [r.choice([0, 1, per - 1, per, per + 1, r.randint(0, 5 * per)]) for _ in range(S)]
        off = [r.randint(0, 3)]
        for n in lens:
            off.append(off[-1] + max(n, 0))
        N = off[-1] + r.randint(0, 300)
        rows = gb.gattn_block_units(N, S, per)
        assert gb.gattn_block_count(N, S, per) == N // per + S
        seen = set()
        for s in range(S):
            for j in range(-(-(off[s + 1] - off[s]) // per)):
                row = off[s] // per + (s if per > 1 else 0) + j
                assert 0 <= row < rows and row not in seen
                seen.add(row)
