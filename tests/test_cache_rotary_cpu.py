"""Refusals of the cache and rotary entry points, and the frequencies, on a machine without a GPU:
every check that the host makes answers before CUDA is touched."""
import ctypes
import math

import numpy as np
import pytest
import torch

from gnn_sparse_attention_gb300 import binding as gb
from gnn_sparse_attention_gb300 import build as gbuild
from tests import cache_ref as ref

OK, INVALID, UNSUPPORTED = 0, 1, 3
P = 4096  # stands for a device pointer that is never followed


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gb.load_library()


def cache(**kw):
    d = dict(S=1, N=4, Nk=64, H=4, Hkv=2, D=64, dtype=1, bits=4, block=64, topk=2, causal=0, scale=0.0,
             max_len_k=0, seq_q=P, seq_k=P, len_k=None, idx_stride=(0, 0), row_stride=(0, 0), k=P, v=P,
             par=P)
    d.update(kw)
    for n in ("idx_stride", "row_stride"):
        d[n] = (ctypes.c_int64 * 2)(*d[n])
    return ctypes.byref(gb._CacheDesc(**d))


def calls(lib, d):
    p, n = ctypes.c_void_p(P), ctypes.c_size_t(77)
    return {"write": lambda: lib.gattn_cache_write(d, p, p, None),
            "read": lambda: lib.gattn_cache_read(d, None, p, p, None),
            "sums": lambda: lib.gattn_cache_sums(d, None, p, None),
            "size": lambda: lib.gattn_cache_fwd_workspace_size(d, ctypes.byref(n)),
            "fwd": lambda: lib.gattn_cache_fwd(d, p, p, p, p, p, 1 << 40, None)}


ALL = ("write", "read", "sums", "size", "fwd")


@pytest.mark.parametrize("bad,status,where", [
    (dict(dtype=2), INVALID, ALL), (dict(S=-1), INVALID, ALL), (dict(N=-1), INVALID, ALL),
    (dict(Nk=-1), INVALID, ALL), (dict(bits=2), UNSUPPORTED, ALL), (dict(bits=0), UNSUPPORTED, ALL),
    (dict(D=16), UNSUPPORTED, ALL), (dict(D=96), UNSUPPORTED, ALL), (dict(D=256), UNSUPPORTED, ALL),
    (dict(Hkv=0), UNSUPPORTED, ALL), (dict(Hkv=3), UNSUPPORTED, ALL), (dict(Hkv=2048), UNSUPPORTED, ALL),
    (dict(Nk=2 ** 31 - 1), UNSUPPORTED, ALL), (dict(Nk=2 ** 31 - 65537, Hkv=1), UNSUPPORTED, ALL), (dict(seq_k=None), INVALID, ALL),
    (dict(seq_q=None), INVALID, ("write", "read", "size", "fwd")), (dict(seq_k=P + 1), INVALID, ALL),
    (dict(k=None), INVALID, ALL), (dict(v=P + 8), INVALID, ALL), (dict(par=None), INVALID, ALL),
    (dict(block=8), UNSUPPORTED, ("sums", "size", "fwd")), (dict(block=48), UNSUPPORTED, ("sums", "size", "fwd")),
    (dict(H=6), UNSUPPORTED, ("size", "fwd")), (dict(H=1), UNSUPPORTED, ("size", "fwd")),
    (dict(H=512), UNSUPPORTED, ("size", "fwd")), (dict(topk=129), UNSUPPORTED, ("size", "fwd")),
    (dict(topk=-1), UNSUPPORTED, ("size", "fwd")), (dict(scale=-1.0), INVALID, ("size", "fwd")),
    (dict(scale=float("nan")), INVALID, ("size", "fwd")), (dict(max_len_k=-1), INVALID, ("size", "fwd")),
    (dict(idx_stride=(-1, 2)), INVALID, ("size", "fwd")), (dict(topk=0), INVALID, ("fwd",)),
    (dict(N=1 << 29), UNSUPPORTED, ("size", "fwd")),
    (dict(row_stride=(64, 0)), INVALID, ("write",)), (dict(row_stride=(0, 131)), INVALID, ("write",)),
    (dict(row_stride=(-128, 0)), INVALID, ("write",))])
def test_cache_descriptors(lib, bad, status, where):
    c = calls(lib, cache(**bad))
    for name in where:
        assert c[name]() == status, name
        assert b"gattn_cache" in lib.gattn_last_error()


def test_cache_pointers(lib):
    d, p = cache(), ctypes.c_void_p(P)
    odd = ctypes.c_void_p(P + 8)
    assert lib.gattn_cache_write(None, p, p, None) == INVALID
    assert lib.gattn_cache_write(d, None, p, None) == INVALID
    assert lib.gattn_cache_write(d, p, odd, None) == INVALID
    assert lib.gattn_cache_read(d, None, odd, None, None) == INVALID
    assert lib.gattn_cache_read(d, ctypes.c_void_p(P + 2), p, p, None) == INVALID
    assert lib.gattn_cache_sums(d, None, None, None) == INVALID
    assert lib.gattn_cache_fwd(d, None, None, p, p, None, 0, None) == INVALID
    assert lib.gattn_cache_fwd(d, p, ctypes.c_void_p(P + 1), p, p, None, 0, None) == INVALID
    assert lib.gattn_cache_fwd(d, p, None, p, None, None, 0, None) == INVALID
    assert lib.gattn_cache_fwd_workspace_size(d, None) == INVALID
    # nothing to do: no pointer is needed
    for empty in (dict(S=0, seq_q=None, seq_k=None), dict(N=0), ):
        d = cache(**empty)
        assert lib.gattn_cache_write(d, None, None, None) == OK
        assert lib.gattn_cache_read(d, None, None, None, None) == OK
        assert lib.gattn_cache_fwd(d, None, None, None, None, None, 0, None) == OK
    assert lib.gattn_cache_read(cache(), None, None, None, None) == OK


def test_long_caches_need_a_workspace(lib):
    n = ctypes.c_size_t()
    d = cache(N=1, H=2, Hkv=1, Nk=1 << 20, topk=0)
    assert lib.gattn_cache_fwd_workspace_size(d, ctypes.byref(n)) == OK and n.value > 0
    p = ctypes.c_void_p(P)
    for ws, size in ((None, n.value), (p, n.value - 1), (ctypes.c_void_p(P + 4), n.value)):
        assert lib.gattn_cache_fwd(d, p, None, p, p, ws, size, None) == INVALID
    d = cache(N=1, H=2, Hkv=1, Nk=64)
    assert lib.gattn_cache_fwd_workspace_size(d, ctypes.byref(n)) == OK and n.value == 0


def rotary(**kw):
    d = dict(N=4, H=4, Hkv=2, D=64, dtype=1, width=64, layout=0, inverse=0, S=1, amp=1.0, freqs=P, pos=P,
             seq_q=None, seq_k=None, len_k=None)
    d.update(kw)
    return ctypes.byref(gb._RotaryDesc(**d))


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=7), INVALID), (dict(N=-1), INVALID), (dict(H=0), INVALID), (dict(Hkv=-1), INVALID),
    (dict(D=0), INVALID), (dict(S=-2), INVALID), (dict(D=1026), UNSUPPORTED), (dict(H=65536), UNSUPPORTED),
    (dict(width=0), INVALID), (dict(width=63), INVALID), (dict(width=66), INVALID), (dict(layout=2), INVALID),
    (dict(amp=float("inf")), INVALID), (dict(pos=None), INVALID), (dict(pos=P + 2), INVALID),
    (dict(freqs=None), INVALID), (dict(freqs=P + 4), INVALID), (dict(q_stride=255), INVALID),
    (dict(k_out_stride=64), INVALID), (dict(q_stride=512), INVALID)])
def test_rotary_descriptors(lib, bad, status):
    p = ctypes.c_void_p(P)  # q_stride=512: in place with another stride than the output's
    assert lib.gattn_rotary(rotary(**bad), p, p, p, p, None) == status
    assert b"gattn_rotary" in lib.gattn_last_error()


def test_rotary_pointers(lib):
    p, odd = ctypes.c_void_p(P), ctypes.c_void_p(P + 1)
    assert lib.gattn_rotary(None, p, p, p, p, None) == INVALID
    for args in ((None, p, p, p), (p, None, p, p), (p, p, None, p), (p, p, p, None), (odd, p, p, p)):
        assert lib.gattn_rotary(rotary(), *args, None) == INVALID
    assert lib.gattn_rotary(rotary(N=0), None, None, None, None, None) == OK


@pytest.mark.parametrize("kind", ["none", "linear", "base", "ramp"])
@pytest.mark.parametrize("width,theta", [(2, 10000.0), (10, 1.0), (64, 10000.0), (128, 500000.0), (1024, 1e8)])
def test_frequencies(lib, width, theta, kind):
    kw = {"scaling": kind, "factor": 4.0, "orig_len": 4096.0}
    got = gb.gattn_rotary_freqs(width, theta, device="cpu", **kw)
    want = ref.frequencies(width, theta, **kw)
    turns = got.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    # fp64 through a power and a few products, then units of 2^-62
    assert np.abs(turns - want.numpy() / (2 * math.pi)).max() <= 2.0 ** -51


def test_frequency_refusals(lib):
    for kw in (dict(width=3), dict(width=0), dict(width=2048), dict(theta=0.5), dict(theta=float("nan")),
               dict(scaling="linear", factor=0.5), dict(scaling="ramp", factor=2.0, orig_len=0.0),
               dict(scaling="ramp", factor=2.0, orig_len=4096.0, low=4.0, high=4.0)):
        with pytest.raises(gb.GattnError):
            gb.gattn_rotary_freqs(**{"width": 64, "device": "cpu", **kw})
    with pytest.raises(ValueError):
        gb.gattn_rotary_freqs(64, scaling="other", device="cpu")


def test_python_refusals():
    with pytest.raises(ValueError):
        gb.gattn_cache_new(10, 2, 48, device="cpu")
    with pytest.raises(ValueError):
        gb.gattn_cache_new(10, 2, 64, bits=2, device="cpu")
    with pytest.raises(ValueError):
        gb.gattn_cache_new(10, 2, 64, device="cpu")  # no cache on the host
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        gb.gattn_rotary(x, torch.zeros(32, dtype=torch.int64), pos=torch.zeros(4, dtype=torch.int32))


@pytest.mark.parametrize("bits", [4, 8])
def test_reference_quantiser(bits):
    """The definition itself: every element within half a step (and its roundings) of its value."""
    x = np.random.default_rng(1).standard_normal((500, 64)).astype(np.float32)
    q, p = ref.quantise(x, bits)
    m, s = p[:, :1].astype(np.float64), p[:, 1:].astype(np.float64)
    assert (np.abs(m + s * q - x) <= s * 0.5 + 2.0 ** -22 * (np.abs(x) + np.abs(m) + s * q)).all()
    assert q.max() == 2 ** bits - 1 or q.max() == 2 ** bits - 2
    assert (m <= x.min(1, keepdims=True)).all()
