"""The backward's work items, counted without a GPU: the kernels' own arithmetic (block_items.cuh,
compiled for the host) behind an emulation of the marks and counts, for offsets in order and for
offsets that are not, where tiles share blocks and the items may want more room than there is."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from gnn_sparse_attention_gb300 import build as gbuild

TILE, SMS = 128, 152

DRIVER = r"""
#include "block_items.cuh"
struct Item { int x, y, z, w; };
extern "C" int units_of(int64_t entries, int rows, int sms, int f32) {
  return gattn::item_units(entries, rows, sms, f32 != 0);
}
extern "C" int64_t slots_of(int64_t entries, int chunk) { return gattn::item_slots(entries, chunk); }
// what items_kernel does, tile after tile instead of by a scan: returns the items to walk
extern "C" int64_t cut(int n, int chunk, int64_t slots, int64_t max_items, int32_t* cnt, Item* items) {
  int64_t item = 0, slot = 0;
  for (int i = 0; i < n; ++i) {
    const int k = gattn::tile_items(cnt[2 * i], chunk);
    gattn::put_items(i, k, item, slot, chunk, slots, max_items, cnt + 2 * i, items);
    item += k;
    slot += k > 1 ? k : 0;
  }
  return item < max_items ? item : max_items;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("items")
    src, so = d / "items.cpp", d / "items.so"
    src.write_text(DRIVER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{gbuild.CSRC}", str(src), "-o", str(so)],
                   check=True)
    lib = ctypes.CDLL(os.fspath(so))
    i64, i32, P = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    lib.slots_of.argtypes, lib.slots_of.restype = [i64, i32], i64
    lib.units_of.argtypes = [i64, i32, i32, i32]
    lib.cut.argtypes, lib.cut.restype = [i32, i32, i64, i64, P, P], i64
    return lib


def clamp(x, lo, hi):
    return min(max(x, lo), hi)


class Case:
    """Sequences, lists and what the mark and count kernels make of them."""

    def __init__(self, lib, sq, sk, Nq, Nk, Hkv, G, block, qb, topk, seed, f32, pick=None):
        self.S = S = len(sq) - 1
        self.U = Nq // qb + (S if qb > 1 else 0)
        B, self.KT = Nk // block + S, Nk // TILE + S
        self.Hkv, self.entries = Hkv, self.U * Hkv * topk
        self.chunk = lib.units_of(self.entries, qb * G, SMS, f32)

        def base(beg, s, per):
            return max(beg[s], 0) // per + (s if per > 1 else 0)

        def span(o, s, N):
            b = clamp(o[s], 0, N)
            return b, clamp(o[s + 1], b, N) - b

        rng = np.random.default_rng(seed)
        bits = np.zeros((B, Hkv, self.U), bool)
        bq = [base(sq, s, qb) for s in range(S)]
        for u in range(self.U):
            s = piece_seq(bq, u)
            n = span(sq, s, Nq)[1]
            off = (u - bq[s]) * qb
            if not 0 <= off < n:
                continue
            nb, b0 = -(-span(sk, s, Nk)[1] // block), base(sk, s, block)
            for kh in range(Hkv):
                for b in (rng.integers(0, max(nb, 1), topk) if pick is None else [pick] * topk):
                    if b < nb and b0 + b < B:
                        bits[b0 + b, kh, u] = True
        words = (self.U + 31) // 32
        wide = np.zeros((B, Hkv, words * 32), bool)
        wide[..., :self.U] = bits
        bk = [base(sk, s, TILE) for s in range(S)]
        self.counts = np.full((self.KT, Hkv), -1, np.int64)
        for kt in range(self.KT):
            s = piece_seq(bk, kt)
            kl, ql = span(sk, s, Nk)[1], span(sq, s, Nq)[1]
            pos = (kt - bk[s]) * TILE
            if not 0 <= pos < kl:
                continue
            nb = min(TILE // block, -(-kl // block) - pos // block)
            row = min(base(sk, s, block) + pos // block, B - nb)
            assert 0 <= row and row + nb <= B
            nu = -(-ql // qb)
            lo, hi = bq[s] // 32 * 32, min((bq[s] + nu - 1) // 32, words - 1) * 32 + 32
            for kh in range(Hkv):
                any_ = wide[row:row + nb, kh].any(0)
                self.counts[kt, kh] = any_[lo:hi].sum() if nu > 0 and hi > lo else 0


def piece_seq(base, row):
    """The warp's search of 32 probes a step, as it runs, for bases in any order."""
    lo, n = 0, len(base)
    while n > 1:
        step = (n + 31) // 32
        m = [lane for lane in range(32) if lo + lane * step < lo + n and base[lo + lane * step] <= row]
        hi = max(m) if m else 0
        n = min(step, n - hi * step)
        lo += hi * step
    return lo


def cut(lib, counts, chunk, entries, Hkv):
    """(items to walk, cnt) after the checks that hold for any counts: every item that is walked was
    written and names units of a tile that exists, and no slot lies outside the partial sums."""
    counts = np.asarray(counts).reshape(-1)
    n = counts.size
    slots = lib.slots_of(entries, chunk)
    most = n + slots
    cnt = np.full((n, 2), 99999999, np.int32)
    cnt[:, 0] = counts
    items = np.full((most + 64, 4), -77, np.int32)
    head = lib.cut(n, chunk, slots, most, cnt.ctypes.data, items.ctypes.data)
    assert 0 <= head <= most
    assert (items[most:] == -77).all(), "written past the items"
    walked = items[:head]
    assert (walked[:, 0] >= 0).all() and (walked[:, 0] < n).all(), "an item that nobody wrote is walked"
    assert (walked[:, 2] >= 0).all() and (walked[:, 2] <= chunk).all()
    assert (walked[:, 3] >= -1).all() and (walked[:, 3] < slots).all(), "a slot past the partial sums"
    used = walked[:, 3][walked[:, 3] >= 0]
    assert len(set(used.tolist())) == used.size, "two items share a slot"
    for i in range(n):  # what the join reads
        c, first = cnt[i]
        if c > chunk:
            k = -(-c // chunk)
            assert 0 <= first and first + k <= slots, "the join reads past the partial sums"
            mine = walked[walked[:, 0] == i]
            assert sorted(mine[:, 3].tolist()) == list(range(first, first + k))
    return walked, cnt, slots


def whole(walked, counts, chunk):
    """With room enough every tile's units are covered once, in pieces of at most `chunk`."""
    for i, c in enumerate(np.asarray(counts).reshape(-1)):
        mine = walked[walked[:, 0] == i]
        if c < 0:
            assert len(mine) == 0
            continue
        at = 0
        for x in mine[np.argsort(mine[:, 1])]:
            assert x[1] == at and (x[3] >= 0) == (c > chunk)
            at += x[2]
        assert at == c and len(mine) >= 1


@pytest.mark.parametrize("seed", range(40))
def test_offsets_in_order_have_room(lib, seed):
    r = random.Random(seed)
    S, block, qb = r.randint(1, 9), r.choice([16, 32, 64, 128]), r.choice([1, 16, 64, 128])
    lq = [r.choice([0, 1, r.randint(0, 900)]) for _ in range(S)]
    lk = [r.choice([0, 1, r.randint(0, 900)]) for _ in range(S)]
    sq, sk = [r.randint(0, 40)], [r.randint(0, 40)]
    for a, b in zip(lq, lk):
        sq.append(sq[-1] + a)
        sk.append(sk[-1] + b)
    pick = r.choice([None, None, 0])
    c = Case(lib, sq, sk, sq[-1] + r.randint(0, 200), sk[-1] + r.randint(0, 200), r.choice([1, 2]),
             r.choice([1, 4]), block, qb, r.choice([1, 5, 16]), seed, r.random() < 0.7, pick)
    assert c.counts[c.counts > 0].sum() <= c.entries
    for chunk in {c.chunk, 1, 7}:  # (1 and 7: more tiles of several items)
        walked, cnt, _ = cut(lib, c.counts, chunk, c.entries, c.Hkv)
        whole(walked, c.counts, chunk)
        assert (cnt[:, 0] == c.counts.reshape(-1)).all()


@pytest.mark.parametrize("S", [3, 17, 40])
@pytest.mark.parametrize("pick", [None, 0])
@pytest.mark.parametrize("f32", [True, False])
def test_offsets_out_of_order_stay_inside(lib, S, pick, f32):
    """Offsets 0, N, 0, N, ...: neighbouring tiles count the same bits."""
    N = 4096
    o = [0 if i % 2 == 0 else N for i in range(S + 1)]
    c = Case(lib, o, o, N, N, 1, 1, 16, 128, 1, 5, f32, pick)
    walked, _, slots = cut(lib, c.counts, c.chunk, c.entries, 1)
    wanted = sum(-(-x // c.chunk) for x in c.counts.reshape(-1).tolist() if x > c.chunk)
    if f32 and S > 3 and pick == 0:
        assert wanted > slots  # the case is one that asks for more than there is
    if wanted <= slots:
        whole(walked, c.counts, c.chunk)


@pytest.mark.parametrize("seed", range(20))
def test_any_counts_stay_inside(lib, seed):
    r = random.Random(seed)
    n, chunk, entries = r.randint(1, 400), r.choice([1, 2, 33]), r.randint(0, 3000)
    counts = [r.choice([-1, 0, 1, chunk, chunk + 1, r.randint(0, 500)]) for _ in range(n)]
    cut(lib, counts, chunk, entries, 1)


@pytest.mark.parametrize("f32", [0, 1])
@pytest.mark.parametrize("rows", [1, 16, 128, 16384])
def test_units_of_an_item(lib, rows, f32):
    """Four items an SM of large problems, none of them of more than 2^23 rows or 2^18 units."""
    for entries in (0, 1, 607, 100000, 10 ** 7, 10 ** 9, 10 ** 12):
        n = lib.units_of(entries, rows, SMS, f32)
        assert 1 <= n <= 2 ** 18 and n * rows <= 2 ** 23
        if 32 <= entries // (SMS * 4) < 2 ** 23 // max(rows, 32):
            assert n == -(-entries // (SMS * 4))
