// block_tc_bwd.cu -- backward of block attention on the tensor cores (bf16).
//
// Two kernels, both with the forward's division of labour (compute warps, one or
// two warps that issue products, one that resolves lists, one that issues TMA;
// every hand-over an mbarrier, every wait bounded):
//
// dQ: a tile of up to 128 (query row, head) pairs walks its unit's block list
//   in steps of 128 keys,
//     S = Q K^T, dP = dO V^T                          -> TMEM (two S buffers)
//     ds = 2^(S scale log2e - lse log2e) (dP - Delta)  -> TMEM, over S
//     dQ += ds K                                       -> TMEM
//   The next step's S and dP run while ds of this one is formed, and four warps
//   write a finished tile while the others are at the next.  ds enters the
//   product as the sum of two bf16: rounded once it would add as much error to
//   dQ as dQ's own rounding, on top of that of Delta (formed from the rounded
//   out), and dQ would be half again as far off as the rounding of the result
//   alone; the second product costs a quarter of the kernel's tensor work.
//   With few keys a row's ds is a small difference of dP and Delta, and the rounding
//   of out left dQ and dK two to three times as far off as their own.  A tile
//   whose rows see one step of keys at most (those of short sequences, and the
//   first of causal ones) has every p and dP of a row at hand, so it forms Delta =
//   sum p dP of them and leaves it for the key side.  Rows of several steps keep
//   the Delta of the rounded out: 1.1 to 1.3 times the result's own rounding for
//   dQ, where a pass of S and dP before the first ds would cost half the kernel.
//
// dK, dV: a work item is a tile of 128 keys and up to `chunk` of the units that
//   chose one of its blocks (block_api.cu builds the items), walked in steps
//   of 64 (query row, head) pairs,
//     S^T = K Q^T, dP^T = V dO^T                       -> TMEM, two buffers
//     p, ds as bf16                 -> TMEM, over S^T and dP^T (D <= 64: beside them)
//     dV += p dO, dK += ds Q                           -> TMEM
//   64 rather than 128 queries a step leave room for several stages of Q and
//   dO and a second score buffer next to the two accumulators; two groups of
//   eight warps take the steps in turn, so that one forms p and ds while the other
//   waits for its products.  p and ds enter these products as one bf16 each, which
//   leaves dV and dK 1.4 times as far off as their own rounding (0.0024 against
//   0.0017); ds as two would be a fifth product of four, and at D <= 64 TMEM has no
//   64 columns left for it.  (A third group at D <= 64 left 72 registers a thread:
//   its spills filled what shared memory leaves of L1, 532 us against 471.)  Four
//   more warps write a finished item.  Units of fewer than 64 pairs share a step,
//   each in a box of its own; a box knows which of the tile's blocks its unit
//   chose.  A key is a TMEM lane, so its mask within a box is a range of columns.
//
//   Measured (as the forward's cases): 24 graphs of 2,731 nodes, 8 heads of 64: dQ
//   233 us, dK and dV 402 us; two causal sequences of 8,191, 16 heads of 128 on 4:
//   173 and 300 us.  A unit seldom chose all blocks of a key tile: with blocks of
//   64 and one choice in three, 1.6 times the useful products run (1.9 with one
//   in eight).  Tiles of 64 keys would run at half the tensor cores' rate.
//
// Rows that must not count but sit in an operand of the last products (keys
// behind the list's end, queries behind a unit's end) are zeroed in shared
// memory, because 0 * NaN is NaN there.
#include <algorithm>
#include <type_traits>

#include "attn_launch.cuh"
#include "attn_pipe.cuh"
#include "block_tc.cuh"

namespace gattn {

namespace {

__device__ int g_err;  // a bounded wait gave up

constexpr int kT = kBlkTile;
constexpr int kPiece = kT * 128;  // 128 rows x 64 bf16 columns

struct DqParams {
  CUtensorMap mq, mo, mk, mv;  // Q, dO, K, V
  BlockBwdParams b;
  int ht, hs, rows;
  int64_t n_tiles;
};

struct DqInfo {
  int steps, n, total;
  int row, rows, pos;
  int kbeg, len, kh, h0;
};

template <int DP>
struct DqSm {
  static constexpr int KB = DP / 64;
  static constexpr int NQ = DP == 64 ? 2 : 1;   // Q and dO buffers
  // K and V stages.  A stage of K is free after dQ, right before the scores that
  // want it next where there are two: a third hides the load (D = 128: 231 -> 174 us)
  static constexpr int NK = DP == 64 ? 4 : 3, NV = DP == 64 ? 4 : 2;
  static constexpr int NG = DP == 64 ? 2 : 1;   // dQ buffers (tiles in turn)
  static constexpr int OP = KB * kPiece;
  static constexpr int Q = 0;
  static constexpr int O = Q + NQ * OP;
  static constexpr int K = O + NQ * OP;
  static constexpr int V = K + NK * OP;
  static constexpr int IDS = V + NV * OP;
  static constexpr int INFO = IDS + 2 * kBlkMaxTopk * 4;
  static constexpr int BAR = INFO + 2 * int(sizeof(DqInfo));
  static constexpr int NBAR = 4 + 2 * NQ + 2 * NK + 2 * NV + 2 + 1 + 2 + 2 * NG + 4;
  static constexpr int END = BAR + NBAR * 8 + 8;
  static constexpr int BYTES = END + 1024;
  static_assert(BYTES <= 227 * 1024, "shared memory of one CTA");
  // TMEM: S [0, 256) in two buffers, dP [256, 384), dQ from 384 on
  static_assert(384 + NG * DP <= 512, "TMEM columns");
};

constexpr int kDqWarps = 16, kDqOut = 4;
constexpr int kDqThr = (kDqWarps + 3 + kDqOut) * 32;

}  // namespace

template <int DP>
__global__ void __launch_bounds__(kDqThr, 1) block_dq_tc(const __grid_constant__ DqParams p) {
  using namespace tc;
  using M = DqSm<DP>;
  constexpr int KB = M::KB, NQ = M::NQ, NK = M::NK, NV = M::NV, NG = M::NG, OP = M::OP;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + M::BAR);
  uint64_t *tile_full = bar, *tile_empty = tile_full + 2, *q_full = tile_empty + 2,
           *q_empty = q_full + NQ, *k_full = q_empty + NQ, *k_empty = k_full + NK,
           *v_full = k_empty + NK, *v_empty = v_full + NV, *s_full = v_empty + NV,
           *dp_empty = s_full + 2, *d_full = dp_empty + 1, *g_full = d_full + 2,
           *g_empty = g_full + NG, *row_sum = g_empty + NG;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bar + M::NBAR);
  DqInfo* info = reinterpret_cast<DqInfo*>(sm + M::INFO);
  int* ids = reinterpret_cast<int*>(sm + M::IDS);
  const BlockGeom& g = p.b.g;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(tile_full + i, 1);
      mbar_init(tile_empty + i, kDqWarps + kDqOut + 2);
      mbar_init(s_full + i, 1);
      mbar_init(d_full + i, kDqWarps);
    }
    mbar_init(dp_empty, kDqWarps);
    for (int i = 0; i < 4; ++i) mbar_init(row_sum + i, kDqWarps / 4);
    for (int i = 0; i < NG; ++i) {
      mbar_init(g_full + i, 1);
      mbar_init(g_empty + i, kDqOut);
    }
    for (int i = 0; i < NQ; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
    }
    for (int i = 0; i < NK; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(v_full + i, 1);
      mbar_init(v_empty + i, 1);
    }
    mbar_init_fence();
  }
  if (warp == kDqWarps) tmem_alloc512(s_tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  bool ok = !(p.b.fail && warp < kDqWarps);  // false: a wait gave up, leave

  if (warp == kDqWarps + 2) {
    // ---------------------------------------------------------------- lists
    int ti = 0;
    for (int64_t t = blockIdx.x; t < p.n_tiles && ok; t += gridDim.x, ++ti) {
      const int slot = ti & 1;
      const int hsub = int(t % p.hs), u = int((t / p.hs) % g.U), kh = int(t / p.hs / g.U);
      const Unit un = unit_at(g, u);
      const Span ks = span_k(g, un.s);
      if (ti >= 2) ok = warp_wait(tile_empty + slot, ((ti >> 1) - 1) & 1);
      if (!ok) break;
      int* list = ids + slot * kBlkMaxTopk;
      int n = 0;
      if (un.n > 0)
        n = block_list(p.b.idx + u * g.is_u + kh * g.is_h, g.topk,
                       (ks.len + g.block - 1) / g.block, list);
      const int total = list_keys(list, n, g.block, ks.len);
      const int seen =
          g.causal ? list_keys(list, n, g.block, min(un.pos + un.n, ks.len)) : total;
      if (lane == 0) {
        DqInfo& f = info[slot];
        f.steps = (seen + kT - 1) / kT;
        f.n = n;
        f.total = total;
        f.row = un.row;
        f.rows = un.n;
        f.pos = un.pos;
        f.kbeg = ks.beg;
        f.len = ks.len;
        f.kh = kh;
        f.h0 = kh * g.G + hsub * p.ht;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(tile_full + slot);
    }
  } else if (warp == kDqWarps + 1) {
    // ---------------------------------------------------------------- copies
    const int per = kT / g.block;
    const uint32_t blk_bytes = uint32_t(g.block) * 128;
    int gi = 0, ti = 0, tq = 0;
    int nk = 0, nv = 0;  // steps whose K, V have been asked for
    for (int64_t t = blockIdx.x; t < p.n_tiles && ok; t += gridDim.x, ++ti) {
      const int slot = ti & 1;
      ok = warp_wait(tile_full + slot, (ti >> 1) & 1);
      if (!ok) break;
      const DqInfo& f = info[slot];
      const int* list = ids + slot * kBlkMaxTopk;
      const int steps = f.steps, n = f.n, kbeg = f.kbeg, kh = f.kh;
      if (steps > 0) {
        const int qs = tq % NQ;
        if (tq >= NQ) ok = warp_wait(q_empty + qs, ((tq / NQ) - 1) & 1);
        if (!ok) break;
        ++tq;
        if (lane == 0) {
          mbar_expect_tx(q_full + qs, uint32_t(p.rows) * 256 * KB);
          for (int kb = 0; kb < KB; ++kb) {
            tma_tile3d(sm + M::Q + qs * OP + kb * kPiece, &p.mq, kb * 64, f.h0, f.row, q_full + qs);
            tma_tile3d(sm + M::O + qs * OP + kb * kPiece, &p.mo, kb * 64, f.h0, f.row, q_full + qs);
          }
        }
      }
      for (int st = 0; st < steps; ++st, ++gi) {
        const int nb = min(per, n - st * per);
        for (int kv = 0; kv < 2; ++kv) {
          const int ns = kv ? NV : NK, si = gi % ns;
          uint64_t* full = (kv ? v_full : k_full) + si;
          if (gi >= ns) ok = ok && warp_wait((kv ? v_empty : k_empty) + si, ((gi / ns) - 1) & 1);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(full, nb * blk_bytes * KB);
          __syncwarp();
          if (lane < nb * KB) {
            const int b = lane / KB, kb = lane % KB;
            tma_tile3d(sm + (kv ? M::V : M::K) + si * OP + kb * kPiece + b * blk_bytes,
                       kv ? &p.mv : &p.mk, kb * 64, kh, kbeg + list[st * per + b] * g.block,
                       full);
          }
          if (kv) ++nv;
          else ++nk;
        }
        if (!ok) break;
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(tile_empty + slot);
    }
    if (!ok) {  // the copies in flight must land before the CTA's memory is given up
      for (int c = tq - 1; c >= max(0, tq - NQ); --c)  // the newest use of each stage
        warp_wait(q_full + c % NQ, (c / NQ) & 1, kDrainLimit);
      for (int c = nk - 1; c >= max(0, nk - NK); --c)
        warp_wait(k_full + c % NK, (c / NK) & 1, kDrainLimit);
      for (int c = nv - 1; c >= max(0, nv - NV); --c)
        warp_wait(v_full + c % NV, (c / NV) & 1, kDrainLimit);
    }
  } else if (warp == kDqWarps) {
    // ---------------------------------------------------------------- products
    constexpr uint32_t IDESC_S = f16_idesc(kT, kT, false), IDESC_G = f16_idesc(kT, DP, true);
    const uint64_t dQ = desc_k(sm + M::Q), dO = desc_k(sm + M::O), dK = desc_k(sm + M::K),
                   dV = desc_k(sm + M::V), dKm = desc_mn(sm + M::K, kPiece);
    const uint32_t tm = uniform(tmem);
    int gi = 0, ti = 0, tq = 0, done = 0;  // steps with scores, tiles, with dQ products
    int due_tile = 0, due_i = 0;            // of step `done`
    bool due_last = false;
    auto product_dq = [&]() {
      const int si = done % NK, b = done & 1, buf = due_tile % NG;
      ok = ok && warp_wait(d_full + b, (done >> 1) & 1);
      if (due_i == 0 && due_tile >= NG)
        ok = ok && warp_wait(g_empty + buf, (due_tile / NG - 1) & 1);
      if (!ok) return;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t out = tm + 384 + buf * DP, ds = tm + b * kT;
        mma_tm<kT>(out, ds, 16, 16, desc_at(dKm, si * OP), IDESC_G, due_i > 0);
        mma_tm<kT>(out, ds + 8, 16, 16, desc_at(dKm, si * OP), IDESC_G, true);
        mma_commit(k_empty + si);
        if (due_last) mma_commit(g_full + buf);
      }
      __syncwarp();
      ++done;
    };
    for (int64_t t = blockIdx.x; t < p.n_tiles && ok; t += gridDim.x, ++ti) {
      const int slot = ti & 1;
      if (!__all_sync(0xffffffffu, mbar_test(tile_full + slot, (ti >> 1) & 1))) {
        if (ok && done < gi) product_dq();  // the lists may wait for that tile to be written
        ok = ok && warp_wait(tile_full + slot, (ti >> 1) & 1);
      }
      if (!ok) break;
      const int n = uniform(info[slot].steps);
      __syncwarp();
      if (lane == 0) mbar_arrive(tile_empty + slot);
      if (n <= 0) continue;
      const int qs = tq % NQ;
      ok = warp_wait(q_full + qs, (tq / NQ) & 1);
      for (int i = 0; i < n && ok; ++i, ++gi) {
        const int sk = gi % NK, sv = gi % NV, b = gi & 1;
        ok = ok && warp_wait(k_full + sk, (gi / NK) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one())  // over the ds of step gi - 2, whose product was issued before
          mma_kk<KB>(tm + b * kT, desc_at(dQ, qs * OP), kPiece, desc_at(dK, sk * OP), kPiece,
                     IDESC_S);
        __syncwarp();
        ok = warp_wait(v_full + sv, (gi / NV) & 1);
        if (gi >= 1) ok = ok && warp_wait(dp_empty, (gi - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          mma_kk<KB>(tm + 2 * kT, desc_at(dO, qs * OP), kPiece, desc_at(dV, sv * OP), kPiece,
                     IDESC_S);
          mma_commit(s_full + b);
          mma_commit(v_empty + sv);
          if (i == n - 1) mma_commit(q_empty + qs);
        }
        __syncwarp();
        if (done < gi) product_dq();
        due_tile = tq;
        due_i = i;
        due_last = i == n - 1;
      }
      ++tq;
    }
    if (ok && done < gi) product_dq();
    if (ok && tq > 0) ok = warp_wait(g_full + (tq - 1) % NG, ((tq - 1) / NG) & 1);
    if (!ok) {  // whatever was issued has completed before TMEM is given up
      for (int k = 0; k <= 2 && k <= gi; ++k) {
        const int c = gi - k;
        warp_wait(s_full + (c & 1), (c >> 1) & 1, kDrainLimit);
        warp_wait(k_empty + c % NK, (c / NK) & 1, kDrainLimit);
      }
    }
  } else if (warp >= kDqWarps + 3) {
    // ---------------------------------------------------------------- output
    const int quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lanes = uint32_t(quad * 32) << 16;
    const int th = r % p.ht, tt = r / p.ht;
    const bool wide = wide_rows(p.b.dQ, g.D);
    int ti = 0, to = 0;  // tiles, tiles with steps
    for (int64_t t = blockIdx.x; t < p.n_tiles; t += gridDim.x, ++ti) {
      const int slot = ti & 1, buf = to % NG;
      ok = ok && warp_wait(tile_full + slot, (ti >> 1) & 1);
      if (!ok) break;
      const DqInfo& f = info[slot];
      const bool some = f.steps > 0, valid = r < p.rows && tt < f.rows;
      const int64_t qrow = int64_t(f.row + tt) * g.H + f.h0 + th;
      if (some) {
        ok = warp_wait(g_full + buf, (to / NG) & 1);
        if (!ok) break;
        tc_fence_after();
      }
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) {
        float o[32];
        __syncwarp();
        if (some) {
          tmem_ld32(tmem + lanes + 384 + buf * DP + c * 32, o);
          tmem_wait_ld();
        }
        if (c == DP / 32 - 1) {  // the buffer is free before the row's end is written
          tc_fence_before();
          __syncwarp();
          if (lane == 0 && some) mbar_arrive(g_empty + buf);
        }
        if (valid) {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = some ? o[i] * g.scale : 0.f;
          store_row(static_cast<__nv_bfloat16*>(p.b.dQ) + qrow * g.D, c * 32, g.D, o, wide);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(tile_empty + slot);
      to += some;
    }
  } else {
    // ---------------------------------------------------------------- ds
    const int r = (warp & 3) * 32 + lane, cc = warp >> 2;  // row, 32-column chunk
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const int th = r % p.ht, tt = r / p.ht;
    int gi = 0, ti = 0, singles = 0;  // steps, tiles, tiles of one step
    for (int64_t t = blockIdx.x; t < p.n_tiles; t += gridDim.x, ++ti) {
      const int slot = ti & 1;
      ok = ok && warp_wait(tile_full + slot, (ti >> 1) & 1);
      if (!ok) break;
      const DqInfo& f = info[slot];
      const int steps = f.steps, total = f.total;
      const bool valid = r < p.rows && tt < f.rows;
      const int lim = !valid ? 0
                      : g.causal ? list_keys(ids + slot * kBlkMaxTopk, f.n, g.block,
                                             min(f.pos + tt + 1, f.len))
                                 : total;
      const int64_t qrow = int64_t(f.row + tt) * g.H + f.h0 + th;
      float2 stat = make_float2(0.f, 0.f);
      if (lim > 0) stat = p.b.stat[qrow];  // a row that sees nothing has lse = -inf
      for (int st = 0; st < steps; ++st, ++gi) {
        const int b = gi & 1;
        ok = ok && warp_wait(s_full + b, (gi >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tS = tmem + lanes + b * kT + cc * 32;
        float dv[32];
        tmem_ld32(tmem + lanes + 2 * kT + cc * 32, dv);
        tmem_wait_ld();
        const int mine = lim - st * kT - cc * 32;
        const bool cut = __any_sync(0xffffffffu, mine < 32);
        const float2 qm = f2s(g.qmul), nl = f2s(-stat.x);
        if (steps == 1) {  // Delta from the row's own p and dP
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float sv[16];
            tmem_ld16(tS + h * 16, sv);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int c0 = h * 16 + 2 * j;
              const float2 z = f2fma(make_float2(sv[2 * j], sv[2 * j + 1]), qm, nl);
              sum.x = c0 < mine ? fmaf(ex2(z.x), dv[c0], sum.x) : sum.x;
              sum.y = c0 + 1 < mine ? fmaf(ex2(z.y), dv[c0 + 1], sum.y) : sum.y;
            }
          }
          // the four warps of these rows meet in the dP that they have read
          const uint32_t tR = tmem + lanes + 2 * kT;
          tmem_st1(tR + cc * 32, sum.x + sum.y);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(row_sum + (warp & 3));
          ok = warp_wait(row_sum + (warp & 3), singles & 1);
          if (!ok) break;
          ++singles;
          tc_fence_after();
          const float d0 = tmem_ld1(tR), d1 = tmem_ld1(tR + 32), d2 = tmem_ld1(tR + 64),
                      d3 = tmem_ld1(tR + 96);
          tmem_wait_ld();
          stat.y = (d0 + d1) + (d2 + d3);
          if (cc == 0 && lim > 0) p.b.stat[qrow].y = stat.y;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(dp_empty);
        if (total < (st + 1) * kT) {  // keys behind the list's end: zeros in K
          const int nv = total - st * kT;
          for (int kb = 0; kb < KB; ++kb) {
            uint4* k = reinterpret_cast<uint4*>(sm + M::K + gi % NK * OP + kb * kPiece);
            for (int i = nv * 8 + threadIdx.x; i < kT * 8; i += kDqWarps * 32)
              k[i] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
          __syncwarp();
        }
        const float2 nd = f2s(-stat.y);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 16 columns: ds rounded, and what the rounding left
          float sv[16], w[16];
          tmem_ld16(tS + h * 16, sv);
          tmem_wait_ld();
          if (cut) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {  // p = 0, and nothing of dP
              sv[j] = h * 16 + j < mine ? sv[j] : neg_inf();
              dv[h * 16 + j] = h * 16 + j < mine ? dv[h * 16 + j] : stat.y;
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 z = f2fma(make_float2(sv[2 * j], sv[2 * j + 1]), qm, nl);
            const float2 y =
                f2mul(make_float2(ex2(z.x), ex2(z.y)),
                      f2add(make_float2(dv[h * 16 + 2 * j], dv[h * 16 + 2 * j + 1]), nd));
            const uint32_t hi = bf16x2_bits(y.x, y.y);
            const float2 lo = f2fma(make_float2(__uint_as_float(hi << 16),
                                                __uint_as_float(hi & 0xffff0000u)),
                                    f2s(-1.f), y);
            w[j] = __uint_as_float(hi);
            w[8 + j] = __uint_as_float(bf16x2_bits(lo.x, lo.y));
          }
          tmem_st16(tS + h * 16, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_full + b);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(tile_empty + slot);
    }
  }
  if (!ok) atomicOr(&g_err, 2);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kDqWarps) tmem_free512(tmem);
}

namespace {

constexpr int kNR = 64;               // query pairs per step
constexpr int kQPiece = kNR * 128;    // 64 rows x 64 bf16 columns
constexpr int kKvWarps = 16, kKvOut = 4;  // two groups of eight, steps in turn
constexpr int kKvThr = (kKvWarps + 4 + kKvOut) * 32;
constexpr int kList = 256;            // units resolved at a time (8 bitmap words)

struct DkvParams {
  CUtensorMap mq, mo, mk, mv;
  BlockBwdParams b;
  int bh, bt;      // heads and query rows of a box
  int br, boxes;   // pairs of a box, boxes of a step
  int ub;          // boxes of a unit
  int l_bh, l_br, l_hn, l_qb;  // log2 of bh, br, of a unit's head groups, of q_block
};

struct Box {
  int mask;        // blocks of the key tile that the unit chose
  int end;         // first position that the box's first query does not see
  int rows;        // pairs of the box that exist
  int row, h0;     // first query row, first head
};

struct KvInfo {
  int item;        // -1: no more items
  int steps;
  int kbeg, pos, n;  // first key row, its position, keys of the tile
  int kh, slot;
};

template <int DP>
struct KvSm {
  static constexpr int KB = DP / 64;
  static constexpr int NS = DP == 64 ? 8 : 4;  // Q and dO stages (64k nodes, 6: 420 us)
  static constexpr int NB = DP == 64 ? 2 : 1;  // K and V buffers (items in turn)
  // p and ds beside S^T and dP^T, where TMEM has room: the scores of a group's next
  // step are then computed while it forms these (64k nodes: 438 -> 420 us)
  static constexpr bool SEP = DP == 64;
  static_assert(NS % 2 == 0, "a stage belongs to one group, which waits for each of its phases");
  static constexpr int OP = KB * kPiece, QP = KB * kQPiece;
  static constexpr int K = 0;
  static constexpr int V = NB * OP;
  static constexpr int Q = 2 * NB * OP;
  static constexpr int O = Q + NS * QP;
  static constexpr int STAT = O + NS * QP;       // [NS][64] (lse log2e, Delta)
  static constexpr int BOX = STAT + NS * kNR * 8;
  static constexpr int LIST = BOX + NS * kNR * int(sizeof(Box));
  static constexpr int INFO = LIST + kList * 8;
  static constexpr int BAR = (INFO + 2 * int(sizeof(KvInfo)) + 7) / 8 * 8;
  static constexpr int NBAR = 4 + 2 * NB + 3 * NS + 6 + 2;
  static constexpr int END = BAR + NBAR * 8 + 8;
  static constexpr int BYTES = END + 1024;
  static_assert(BYTES <= 227 * 1024, "shared memory of one CTA");
  // TMEM: S^T [0, 128) and dP^T [128, 256) of the groups; p and ds; dV, dK.  16 queries
  // of p take P16 columns (8, or 16 where they overwrite scores).
  static constexpr int T_P = SEP ? 256 : 0, T_DS = SEP ? 320 : 128, P16 = SEP ? 8 : 16;
  static constexpr int T_ACC = SEP ? 384 : 256;
  static_assert(T_ACC + 2 * DP <= 512, "TMEM columns");
};

// arrive once this thread's cp.async copies so far have landed
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(bar))
               : "memory");
}

}  // namespace

template <int DP>
__global__ void __launch_bounds__(kKvThr, 1) block_dkv_tc(const __grid_constant__ DkvParams p) {
  using namespace tc;
  using M = KvSm<DP>;
  constexpr int KB = M::KB, NS = M::NS, NB = M::NB, OP = M::OP, QP = M::QP;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + M::BAR);
  uint64_t *item_full = bar, *item_empty = item_full + 2, *kv_full = item_empty + 2,
           *kv_empty = kv_full + NB, *q_full = kv_empty + NB, *q_empty = q_full + NS,
           *box_full = q_empty + NS, *s_full = box_full + NS, *s_empty = s_full + 2,
           *p_full = s_empty + 2, *g_full = p_full + 2, *g_empty = g_full + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bar + M::NBAR);
  KvInfo* info = reinterpret_cast<KvInfo*>(sm + M::INFO);
  int2* list = reinterpret_cast<int2*>(sm + M::LIST);
  const BlockGeom& g = p.b.g;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(item_full + i, 1);
      mbar_init(item_empty + i, kKvWarps + kKvOut + 3);
      mbar_init(s_full + i, 1);
      mbar_init(s_empty + i, 8);
      mbar_init(p_full + i, 8);
    }
    mbar_init(g_full, 1);
    mbar_init(g_empty, kKvOut);
    for (int i = 0; i < NB; ++i) {
      mbar_init(kv_full + i, 1);
      mbar_init(kv_empty + i, 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(q_full + i, 1 + 32);  // the copies' bytes, and each lane's statistics
      mbar_init(q_empty + i, 1);
      mbar_init(box_full + i, 1);
    }
    mbar_init_fence();
  }
  if (warp == kKvWarps) tmem_alloc512(s_tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  bool ok = !(p.b.fail && warp < kKvWarps);

  if (warp == kKvWarps + 2) {
    // ---------------------------------------------------------------- lists
    const int64_t n_items = p.b.head[0];
    int gi = 0;
    for (int ti = 0;; ++ti) {
      int it = 0;
      if (lane == 0) it = atomicAdd(p.b.head + 1, 1);
      it = uniform(it);
      const int slot = ti & 1;
      if (it >= n_items) {
        if (ti >= 2) ok = warp_wait(item_empty + slot, ((ti >> 1) - 1) & 1);
        if (ok && lane == 0) {
          info[slot].item = -1;
          mbar_arrive(item_full + slot);
        }
        break;
      }
      const int4 q = p.b.items[it];
      const int kt = q.x / g.Hkv, kh = q.x - kt * g.Hkv;
      const int s = piece_seq(g.seq_k, g.S, kT, kt);
      const Span ks = span_k(g, s), qs = span_q(g, s);
      const int pos = (kt - piece_base(g.seq_k, s, kT)) * kT;
      const int nb = min(kT / g.block, (ks.len + g.block - 1) / g.block - pos / g.block);
      const int brow = min(piece_base(g.seq_k, s, g.block) + pos / g.block, g.B - nb);
      const int ub = piece_base(g.seq_q, s, g.qb), nu = (qs.len + g.qb - 1) / g.qb;
      const int steps = int((int64_t(q.z) * p.ub + p.boxes - 1) / p.boxes);
      if (ti >= 2) ok = warp_wait(item_empty + slot, ((ti >> 1) - 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        KvInfo& f = info[slot];
        f.item = it;
        f.steps = steps;
        f.kbeg = ks.beg + pos;
        f.pos = pos;
        f.n = min(kT, ks.len - pos);
        f.kh = kh;
        f.slot = q.w;
        mbar_arrive(item_full + slot);
      }
      // units in ascending order: the set bits of the blocks' rows, 8 words at a time
      int w0 = ub / 32, seen = 0;   // next word, units before it
      int have = 0, next = 0;       // resolved units, the next one of them
      int sub = 0;                  // boxes of that unit already issued
      for (int st = 0; st < steps && ok; ++st, ++gi) {
        const int si = gi % NS;
        if (gi >= NS) ok = warp_wait(q_empty + si, ((gi / NS) - 1) & 1);
        if (!ok) break;
        Box* box = reinterpret_cast<Box*>(sm + M::BOX) + si * kNR;
        for (int j = 0; j < p.boxes; ++j) {
          while (next >= have && seen < q.y + q.z && w0 <= (ub + nu - 1) / 32) {
            // resolve the next 8 words: lanes 0-7
            const int w = w0 + lane;
            uint32_t bits[8], any = 0;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              bits[b] = lane < 8 && b < nb && w < p.b.words
                            ? p.b.bits[(int64_t(brow + b) * g.Hkv + kh) * p.b.words + w] : 0u;
              any |= bits[b];
            }
            const int c = __popc(any);
            int before = c;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
              const int x = __shfl_up_sync(0xffffffffu, before, o);
              if (lane >= o) before += x;
            }
            const int all = __shfl_sync(0xffffffffu, before, 7);
            const int lo = max(seen, q.y), hi = min(seen + all, q.y + q.z);
            __syncwarp();
            for (int k = 0; k < 8; ++k) {  // a lane takes a bit of each word
              const uint32_t a = __shfl_sync(0xffffffffu, any, k);
              const int at = seen + __shfl_sync(0xffffffffu, before - c, k) +
                             __popc(a & ((1u << lane) - 1));
              if (a == 0) continue;
              int mk = 0;
#pragma unroll
              for (int b = 0; b < 8; ++b)
                mk |= int((__shfl_sync(0xffffffffu, bits[b], k) >> lane) & 1u) << b;
              if (((a >> lane) & 1u) && at >= lo && at < hi)
                list[at - lo] = make_int2((w0 + k) * 32 + lane, mk);
            }
            __syncwarp();
            have = max(0, hi - lo);
            next = 0;
            seen += all;
            w0 += 8;
          }
          Box x{0, 0, 0, 0, 0};
          if (next < have) {
            const int2 e = list[next];
            const int unit = e.x - ub;                       // of the sequence
            const int off = unit << p.l_qb;
            const int t0 = (sub >> p.l_hn) * p.bt;
            // (a unit outside the sequence: only where offsets lie about the tables)
            const int n =
                unit >= 0 && unit < nu ? clampi(min(g.qb, qs.len - off) - t0, 0, p.bt) : 0;
            x.mask = e.y;
            x.rows = n << p.l_bh;
            x.end = g.causal ? off + t0 + ks.len - qs.len + 1 : INT32_MAX / 2;
            x.row = qs.beg + off + t0;
            x.h0 = kh * g.G + ((sub & ((1 << p.l_hn) - 1)) << p.l_bh);
            if (++sub == p.ub) {
              sub = 0;
              ++next;
            }
          }
          if (lane == 0) box[j] = x;
        }
        if (lane == 0) mbar_arrive(box_full + si);
        __syncwarp();
      }
      if (!ok) break;
    }
  } else if (warp == kKvWarps + 1) {
    // ---------------------------------------------------------------- copies
    int gi = 0, tk = 0;
    for (int ti = 0;; ++ti) {
      const int slot = ti & 1;
      ok = warp_wait(item_full + slot, (ti >> 1) & 1);
      if (!ok) break;
      const KvInfo f = info[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(item_empty + slot);
      if (f.item < 0) break;
      if (f.steps == 0) continue;
      const int kb2 = tk % NB;
      if (tk >= NB) ok = warp_wait(kv_empty + kb2, (tk / NB - 1) & 1);
      if (!ok) break;
      ++tk;
      if (lane == 0) mbar_expect_tx(kv_full + kb2, 2 * OP);
      __syncwarp();
      if (lane < 2 * KB)
        tma_tile3d(sm + (lane & 1 ? M::V : M::K) + kb2 * OP + (lane >> 1) * kPiece,
                   lane & 1 ? &p.mv : &p.mk, (lane >> 1) * 64, f.kh, f.kbeg, kv_full + kb2);
      for (int st = 0; st < f.steps; ++st, ++gi) {
        const int si = gi % NS;
        ok = warp_wait(box_full + si, (gi / NS) & 1);  // it waited for the stage to be free
        if (!ok) break;
        const Box* box = reinterpret_cast<const Box*>(sm + M::BOX) + si * kNR;
        if (p.boxes == 1) {  // uniform operands: a copy is one instruction
          const int row = uniform(box[0].row), h0 = uniform(box[0].h0);
          const bool some = uniform(box[0].rows) > 0;
          if (elect_one()) {
            mbar_expect_tx(q_full + si, some ? kNR * 256 * KB : 0);
            for (int kb = 0; kb < KB && some; ++kb) {
              tma_tile3d(sm + M::Q + si * QP + kb * kQPiece, &p.mq, kb * 64, h0, row, q_full + si);
              tma_tile3d(sm + M::O + si * QP + kb * kQPiece, &p.mo, kb * 64, h0, row, q_full + si);
            }
          }
        } else {
          int full = 0;  // boxes with pairs: all of them but at an item's end
          for (int j = lane; j < p.boxes; j += 32) full += box[j].rows > 0;
          full = __reduce_add_sync(0xffffffffu, full);
          if (lane == 0) mbar_expect_tx(q_full + si, uint32_t(full * p.br) * 256 * KB);
          __syncwarp();
          for (int e = lane; e < p.boxes * 2 * KB; e += 32) {
            const int j = e / (2 * KB), o = e & 1, kb = (e >> 1) % KB;
            const Box x = box[j];
            if (x.rows > 0)
              tma_tile3d(sm + (o ? M::O : M::Q) + si * QP + kb * kQPiece + j * p.br * 128,
                         o ? &p.mo : &p.mq, kb * 64, x.h0, x.row, q_full + si);
          }
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < kNR / 32; ++e) {  // the statistics
          const int c = e * 32 + lane, i = c & (p.br - 1);
          const Box& x = box[c >> p.l_br];
          if (i < x.rows)
            cp_async8(sm + M::STAT + (si * kNR + c) * 8,
                      p.b.stat + int64_t(x.row + (i >> p.l_bh)) * g.H + x.h0 + (i & (p.bh - 1)));
        }
        cp_async_arrive(q_full + si);
        __syncwarp();
      }
      if (!ok) break;
    }
    cp_async_wait<0>();
    if (!ok) {  // the copies in flight must land before the CTA's memory is given up
      for (int c = tk - 1; c >= max(0, tk - NB); --c)
        warp_wait(kv_full + c % NB, (c / NB) & 1, kDrainLimit);
      for (int c = gi - 1; c >= max(0, gi - NS); --c)
        warp_wait(q_full + c % NS, (c / NS) & 1, kDrainLimit);
    }
  } else if (warp == kKvWarps) {
    // ---------------------------------------------------------------- scores
    // A warp for S and dP, another for dV and dK: at D <= 64 one warp alone is busy
    // for 890 clocks a step with issuing what the tensor cores do in 480.
    constexpr uint32_t IDESC_S = f16_idesc(kT, kNR, false);
    const uint64_t dK = desc_k(sm + M::K), dV = desc_k(sm + M::V), dQ = desc_k(sm + M::Q),
                   dO = desc_k(sm + M::O);
    const uint32_t tm = uniform(tmem);
    int gi = 0, tk = 0;  // steps, items
    for (int ti = 0; ok; ++ti) {
      const int slot = ti & 1;
      ok = warp_wait(item_full + slot, (ti >> 1) & 1);
      if (!ok) break;
      const int it = uniform(info[slot].item), n = uniform(info[slot].steps);
      __syncwarp();
      if (lane == 0) mbar_arrive(item_empty + slot);
      if (it < 0) break;
      if (n <= 0) continue;
      const int kb2 = tk % NB;
      ok = warp_wait(kv_full + kb2, (tk / NB) & 1);
      for (int i = 0; i < n && ok; ++i, ++gi) {
        const int si = gi % NS, x = gi & 1, c = gi - 2;
        // over the scores of step gi - 2, which have been read, or p and ds of it,
        // whose products have run
        if (c >= 0)
          ok = M::SEP ? warp_wait(s_empty + x, (c >> 1) & 1)
                      : warp_wait(q_empty + c % NS, (c / NS) & 1);
        ok = ok && warp_wait(q_full + si, (gi / NS) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          mma_kk<KB>(tm + x * kNR, desc_at(dK, kb2 * OP), kPiece, desc_at(dQ, si * QP), kQPiece,
                     IDESC_S);
          mma_kk<KB>(tm + 128 + x * kNR, desc_at(dV, kb2 * OP), kPiece, desc_at(dO, si * QP),
                     kQPiece, IDESC_S);
          mma_commit(s_full + x);
          if (i == n - 1) mma_commit(kv_empty + kb2);
        }
        __syncwarp();
      }
      ++tk;
    }
    if (!ok)  // what was issued completes before TMEM is given up
      for (int c = gi; c >= 0 && c > gi - 3; --c) warp_wait(s_full + (c & 1), (c >> 1) & 1, kDrainLimit);
  } else if (warp == kKvWarps + 3) {
    // ---------------------------------------------------------------- gradients
    constexpr uint32_t IDESC_G = f16_idesc(kT, DP, true);
    const uint64_t dQm = desc_mn(sm + M::Q, kQPiece), dOm = desc_mn(sm + M::O, kQPiece);
    const uint32_t tm = uniform(tmem);
    int gi = 0, tk = 0;
    for (int ti = 0; ok; ++ti) {
      const int slot = ti & 1;
      ok = warp_wait(item_full + slot, (ti >> 1) & 1);
      if (!ok) break;
      const int it = uniform(info[slot].item), n = uniform(info[slot].steps);
      __syncwarp();
      if (lane == 0) mbar_arrive(item_empty + slot);
      if (it < 0) break;
      if (n <= 0) continue;
      if (tk >= 1) ok = warp_wait(g_empty, (tk - 1) & 1);
      for (int i = 0; i < n && ok; ++i, ++gi) {
        const int si = gi % NS, x = gi & 1;
        ok = warp_wait(q_full + si, (gi / NS) & 1) && warp_wait(p_full + x, (gi >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t pt = tm + x * (4 * M::P16);
          mma_tm<kNR>(tm + M::T_ACC, pt + M::T_P, 16, M::P16, desc_at(dOm, si * QP), IDESC_G,
                      i > 0);
          mma_tm<kNR>(tm + M::T_ACC + DP, pt + M::T_DS, 16, M::P16, desc_at(dQm, si * QP), IDESC_G,
                      i > 0);
          mma_commit(q_empty + si);
          if (i == n - 1) mma_commit(g_full);
        }
        __syncwarp();
      }
      ++tk;
    }
    // every product has completed before TMEM is given up
    if (ok && tk > 0) ok = warp_wait(g_full, (tk - 1) & 1);
    if (!ok)
      for (int c = gi; c >= 0 && c > gi - 3; --c) warp_wait(q_empty + c % NS, (c / NS) & 1, kDrainLimit);
  } else if (warp >= kKvWarps + 4) {
    // ---------------------------------------------------------------- output
    const int quad = warp & 3, r = quad * 32 + lane;  // key
    const uint32_t lanes = uint32_t(quad * 32) << 16;
    const bool wide_k = wide_rows(p.b.dK, g.D), wide_v = wide_rows(p.b.dV, g.D);
    int to = 0;  // items with steps
    for (int ti = 0;; ++ti) {
      const int slot = ti & 1;
      ok = ok && warp_wait(item_full + slot, (ti >> 1) & 1);
      if (!ok) break;
      const KvInfo f = info[slot];
      if (f.item < 0) break;
      const bool some = f.steps > 0, valid = r < f.n;
      if (some) {
        ok = warp_wait(g_full, to & 1);
        if (!ok) break;
        tc_fence_after();
      }
      const int64_t krow = (int64_t(f.kbeg + r) * g.Hkv + f.kh) * g.D;
#pragma unroll 1
      for (int c = 0; c < 2 * DP / 32; ++c) {  // dV, then dK
        const bool k = c >= DP / 32;
        const int col = c * 32 - (k ? DP : 0);
        float o[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0.f;
        __syncwarp();
        if (some) {
          tmem_ld32(tmem + lanes + M::T_ACC + c * 32, o);
          tmem_wait_ld();
        }
        if (c == 2 * DP / 32 - 1) {  // the buffer is free before the row's end is written
          tc_fence_before();
          __syncwarp();
          if (lane == 0 && some) mbar_arrive(g_empty);
        }
        if (valid && f.slot < 0) {
          const float mul = k ? g.scale : 1.f;
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= mul;
          store_row(static_cast<__nv_bfloat16*>(k ? p.b.dK : p.b.dV) + krow, col, g.D, o,
                    k ? wide_k : wide_v);
        } else if (valid) {
          float* out = p.b.part + (int64_t(f.slot) * 2 + (k ? 0 : 1)) * kT * g.D +
                       int64_t(r) * g.D + col;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (col + q * 4 < g.D)
              *reinterpret_cast<float4*>(out + q * 4) =
                  make_float4(o[q * 4], o[q * 4 + 1], o[q * 4 + 2], o[q * 4 + 3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(item_empty + slot);
      to += some;
    }
  } else {
    // ---------------------------------------------------------------- p and ds
    const int r = (warp & 3) * 32 + lane, part = (warp >> 2) & 1;  // key, 32 of 64 columns
    const int x = warp >> 3;                                       // group
    const int tid = threadIdx.x & 255;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + x * kNR + part * 32, tD = tS + 128;
    const uint32_t wP = tmem + lanes + (x * 4 + part * 2) * M::P16 + M::T_P,
                   wS = wP - M::T_P + M::T_DS;
    const int blk = r / g.block;
    int gi = 0;
    for (int ti = 0;; ++ti) {
      const int slot = ti & 1;
      ok = ok && warp_wait(item_full + slot, (ti >> 1) & 1);
      if (!ok) break;
      const KvInfo f = info[slot];
      if (f.item < 0) break;
      const int pos = f.pos + r;
      const bool valid = r < f.n;
      for (int i = (gi ^ x) & 1; i < f.steps; i += 2) {
        const int c = gi + i, si = c % NS;
        // what the statistics and boxes say, while the scores are on their way
        ok = ok && warp_wait(q_full + si, (c / NS) & 1);
        if (!ok) break;
        const Box* box = reinterpret_cast<const Box*>(sm + M::BOX) + si * kNR;
        // this key's columns of the step; pairs that do not exist: zeros in Q and dO
        uint32_t see = 0;
        bool zeros = false;
        for (int j = 0; j < p.boxes; ++j) {
          const Box y = box[j];
          zeros = zeros || y.rows < p.br;
          const int c0 = j * p.br - part * 32;
          if (c0 >= 32 || c0 + p.br <= 0) continue;
          if (!valid || !((y.mask >> blk) & 1)) continue;
          // query t of the box sees positions below end + t
          const int t0 = max(0, pos - y.end + 1);
          const int lo = max(c0 + (t0 < p.bt ? t0 * p.bh : p.br), 0), hi = min(c0 + y.rows, 32);
          if (hi > lo) see |= (hi - lo == 32 ? 0xffffffffu : ((1u << (hi - lo)) - 1) << lo);
        }
        if (zeros) {
          for (int j = 0; j < p.boxes; ++j) {
            const int n = box[j].rows;
            for (int o = 0; o < 2 * KB; ++o) {
              uint4* q = reinterpret_cast<uint4*>(sm + (o < KB ? M::Q : M::O) + si * QP +
                                                  (o % KB) * kQPiece + j * p.br * 128);
              for (int k = n * 8 + tid; k < p.br * 8; k += 256) q[k] = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async();
        }
        ok = warp_wait(s_full + x, (c >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const float4* stat =
            reinterpret_cast<const float4*>(sm + M::STAT + (si * kNR + part * 32) * 8);
        const float2 qm = f2s(g.qmul);
        auto form = [&](auto all) {  // all: the warp's keys see every column
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 16 columns
            float sv[16], dv[16], wp[8], wd[8];
            tmem_ld16(tS + h * 16, sv);
            tmem_ld16(tD + h * 16, dv);
            tmem_wait_ld();
            if (M::SEP && h == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(s_empty + x);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 a = stat[h * 8 + j];  // (lse, Delta) of columns 2 j, 2 j + 1
              const float2 z =
                  f2fma(make_float2(sv[2 * j], sv[2 * j + 1]), qm, make_float2(-a.x, -a.z));
              float2 y = make_float2(ex2(z.x), ex2(z.y));
              float2 ds =
                  f2mul(y, f2add(make_float2(dv[2 * j], dv[2 * j + 1]), make_float2(-a.y, -a.w)));
              if (!decltype(all)::value) {
                const bool s0 = (see >> (h * 16 + 2 * j)) & 1u,
                           s1 = (see >> (h * 16 + 2 * j + 1)) & 1u;
                y.x = s0 ? y.x : 0.f;
                y.y = s1 ? y.y : 0.f;
                ds.x = s0 ? ds.x : 0.f;
                ds.y = s1 ? ds.y : 0.f;
              }
              wp[j] = __uint_as_float(bf16x2_bits(y.x, y.y));
              wd[j] = __uint_as_float(bf16x2_bits(ds.x, ds.y));
            }
            tmem_st8(wP + h * M::P16, wp);
            tmem_st8(wS + h * M::P16, wd);
          }
        };
        if (M::SEP && c >= 2) {  // the products with the group's last p and ds have run
          ok = warp_wait(q_empty + (c - 2) % NS, ((c - 2) / NS) & 1);
          if (!ok) break;
          tc_fence_after();
        }
        if (__all_sync(0xffffffffu, see == 0xffffffffu)) {
          form(std::true_type{});
        } else if (__any_sync(0xffffffffu, see)) {
          form(std::false_type{});
        } else {  // keys of a block that the unit did not choose
          const float none[8] = {};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tmem_st8(wP + h * M::P16, none);
            tmem_st8(wS + h * M::P16, none);
          }
          if (M::SEP && lane == 0) mbar_arrive(s_empty + x);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + x);
      }
      if (!ok) break;
      gi += f.steps;
      __syncwarp();
      if (lane == 0) mbar_arrive(item_empty + slot);
    }
  }
  if (!ok) atomicOr(&g_err, 2);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kKvWarps) tmem_free512(tmem);
}

gattn_status launch_block_bwd_tc(const BlockBwdParams& b, cudaStream_t st) {
  const BlockGeom& g = b.g;
  auto go = [&](auto kern, unsigned grid, int threads, int bytes, const auto& p) -> gattn_status {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) {
      kern<<<grid, threads, bytes, st>>>(p);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
      set_error("gattn_block_bwd launch failed: %s", cudaGetErrorString(e));
      return GATTN_ERR_CUDA;
    }
    return GATTN_OK;
  };
  const void *K = g.Nk ? b.K : b.Q, *V = g.Nk ? b.V : b.Q;  // never read when Nk is 0
  const void *Q = g.Nq ? b.Q : b.K, *dO = g.Nq ? b.dO : b.K;
  gattn_status s = GATTN_OK;
  if (g.U > 0 && g.Nq > 0) {
    DqParams p{};
    p.b = b;
    p.ht = tile_heads(g);
    p.hs = g.G / p.ht;
    p.rows = p.ht * g.qb;
    p.n_tiles = int64_t(g.U) * g.Hkv * p.hs;
    if (!encode_heads_map(&p.mq, Q, g.Nq, g.H, g.D, p.ht, g.qb) ||
        !encode_heads_map(&p.mo, dO, g.Nq, g.H, g.D, p.ht, g.qb) ||
        !encode_heads_map(&p.mk, K, g.Nk, g.Hkv, g.D, 1, g.block) ||
        !encode_heads_map(&p.mv, V, g.Nk, g.Hkv, g.D, 1, g.block))
      return GATTN_ERR_CUDA;
    const unsigned grid = unsigned(std::min<int64_t>(p.n_tiles, sm_count()));
    s = g.D <= 64 ? go(block_dq_tc<64>, grid, kDqThr, DqSm<64>::BYTES, p)
                  : go(block_dq_tc<128>, grid, kDqThr, DqSm<128>::BYTES, p);
    if (s != GATTN_OK) return s;
  }
  if (g.Nk > 0) {
    DkvParams p{};
    p.b = b;
    p.bt = std::min(g.qb, kNR);
    p.bh = std::min(g.G, kNR / p.bt);
    p.br = p.bt * p.bh;
    p.boxes = kNR / p.br;
    p.ub = (g.qb / p.bt) * (g.G / p.bh);
    const auto log2i = [](int x) { return 31 - __builtin_clz(x); };
    p.l_bh = log2i(p.bh);
    p.l_br = log2i(p.br);
    p.l_hn = log2i(g.G / p.bh);
    p.l_qb = log2i(g.qb);
    if (!encode_heads_map(&p.mq, Q, g.Nq, g.H, g.D, p.bh, p.bt) ||
        !encode_heads_map(&p.mo, dO, g.Nq, g.H, g.D, p.bh, p.bt) ||
        !encode_heads_map(&p.mk, K, g.Nk, g.Hkv, g.D, 1, kT) ||
        !encode_heads_map(&p.mv, V, g.Nk, g.Hkv, g.D, 1, kT))
      return GATTN_ERR_CUDA;
    const unsigned grid = unsigned(std::min<int64_t>(b.max_items, sm_count()));
    s = g.D <= 64 ? go(block_dkv_tc<64>, grid, kKvThr, KvSm<64>::BYTES, p)
                  : go(block_dkv_tc<128>, grid, kKvThr, KvSm<128>::BYTES, p);
  }
  return s;
}

cudaError_t block_bwd_tc_take_error(int* err) {
  cudaError_t e = cudaMemcpyFromSymbol(err, g_err, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && *err) e = cudaMemcpyToSymbol(g_err, &zero, sizeof(int));
  return e;
}

}  // namespace gattn
