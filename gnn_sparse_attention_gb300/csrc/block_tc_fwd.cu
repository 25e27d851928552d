// block_tc_fwd.cu -- forward of block attention on the tensor cores
// (bf16, D = 8 .. 128; heads narrower than 64 are padded with zeros by TMA).
//
// A tile is up to 128 (query row, head) pairs of one unit and key head: they
// share the unit's block list.  A step is 128 keys, i.e. 128 / block blocks
// of the list, each fetched by a TMA box of its own rows:
//   S = Q K^T  (128 x 128 x D)      -> TMEM
//   p = 2^(s - m) as bf16           -> TMEM, over the scores it came from
//   O += P V   (128 x D x 128)      -> TMEM, P as the left operand
// p is rounded to bf16 because the product takes bf16; its sum l is fp32.  out is
// then 0.0019 to 0.0024 off (2-norm), where its own rounding alone is 0.0017.  p as
// two bf16, the second in the scores' other columns, was measured: 128 tokens
// against caches of 8,000 170 -> 185 us, a prompt of 32,768 769 -> 1,083 us.
// A softmax step is a chain of latencies (TMEM, maximum, exponentials, TMEM)
// longer than the step's products, so two streams share the work, each with its
// own 256 threads (thread = row and half of its 128 columns; the halves exchange
// their maxima in shared memory), score buffer, running maximum and sum, and
// output.  Where a key head's queries fill two tiles or
// more (PAIR), the streams are two tiles of the same unit on the same steps, and
// every K and V that is fetched serves both: at D = 128 a tile alone asks for
// 64 KB a step, 18 TB/s of L2 at the tensor cores' rate, about twice what L2
// gives.  Otherwise they take one tile's steps in turn and are merged when the
// tile is written.  While one stream is in its softmax, the tensor core runs the other's
// P V and next scores.  P in TMEM instead of shared memory takes 64 KB of the
// step's 160 KB of shared-memory traffic away (128 bytes a clock would
// otherwise be the bound at D = 128) and leaves room for a third stage.
// Roles: warps 0-15 softmax, warps 16-19 merge a finished tile's streams and write
// it while the softmax is at the next one, warp 20 issues the products, warp 21
// issues TMA, warp 22 resolves the next tile's block list meanwhile (a chain of
// dependent loads of two microseconds); every hand-over is an mbarrier, every
// wait is bounded.
//
// With the list ascending, the keys that a row sees are the first columns of
// its steps (list_keys), so the mask is one number per row and only the
// steps around it compare.  O is rescaled only when the maximum grew by more
// than 2^8 (p stays below 2^8, far from overflow).
//
// Rows of V that no row may see (behind the sequence's end, or of no block)
// are zeroed in shared memory, because 0 * NaN is NaN in the product.  Under
// the causal mask some rows see a value that others must not: in those steps
// non-finite values are taken out of V and added back to the rows that see
// them when the tile is written.
//
// When there are fewer tiles than SMs (one new token per sequence), each
// tile's steps are split over several CTAs and a second kernel joins them.
//
// Measured (bf16, blocks of 64): a causal prompt of 32,768 tokens, 32 heads of 128
// on 8 key heads, 32 blocks a unit: 0.76 ms, 1.40 PFLOP/s; two causal sequences
// of 8,191, 16 heads of 128 on 4, 16 blocks: 120 us, 1.04; 24 graphs of 2,731
// nodes, 8 heads of 64, 16 blocks: 187 us, 0.75; 128 tokens against caches of 8,000
// (32 heads on 8): 167 us, 6.4 TB/s.  What bounds the first three is the
// softmax's latency: two streams keep the tensor cores busy half of the time (a
// third at D = 64), and TMEM has no room for a third or, at D = 128, for a second
// score buffer of each.
#include <algorithm>

#include "attn_launch.cuh"
#include "attn_pipe.cuh"
#include "block_tc.cuh"

namespace gattn {

namespace {

__device__ int g_err;  // a bounded wait gave up

constexpr int kT = kBlkTile;
constexpr int kPiece = kT * 128;       // 128 rows x 64 bf16 columns
constexpr int kSoftWarps = 16;          // two streams of eight
constexpr int kOutWarps = 4;
constexpr int kMma = kSoftWarps + kOutWarps, kCopy = kMma + 1, kLists = kMma + 2;
constexpr int kThr = (kLists + 1) * 32;

struct TcFwdParams {
  CUtensorMap mq, mk, mv;
  BlockGeom g;
  const int32_t* idx;
  const __nv_bfloat16* V;
  __nv_bfloat16* out;
  float* lse;
  float *part_o, *part_l;  // nsplit > 1: [tile][split][rows][D], [tile][split][rows]
  int ht, hs, rows;        // heads per tile, tiles (PAIR: pairs of them) per unit and key head,
                           // rows per tile
  int nsplit;
  int fail;                // failure-path test: the softmax warps give up their first wait
  int64_t n_tiles;         // splits counted
};

// What the producer tells the other warps about a tile.
struct TileInfo {
  int s0, s1;          // steps [s0, s1) of the list
  int n, total;        // blocks in the list, keys in them
  int least;           // keys that the tile's first row sees
  int row, rows;       // first query row, query rows
  int pos;             // position of the first query row
  int kbeg, len;       // the sequence's keys
  int kh, h0;          // key head, first query head
  int poison;          // a non-finite value was taken out of V
  int64_t part;        // index of its partial result
};

template <int DP, bool PAIR>
struct Sm {
  static constexpr int KB = DP / 64;
  static constexpr int QT = PAIR ? 2 : 1;       // Q tiles of a buffer
  static constexpr int NQ = 2 / QT;             // Q buffers
  static constexpr int NS = DP == 64 ? 4 : 2;   // K stages
  static constexpr int NV = DP == 64 ? 4 : 2;   // V stages
  static constexpr int NO = DP == 64 ? 2 : 1;   // output buffers of a stream (tiles in turn)
  static constexpr int OP = KB * kPiece;         // one operand tile
  static constexpr int Q = 0;
  static constexpr int K = Q + NQ * QT * OP;
  static constexpr int V = K + NS * OP;
  static constexpr int ML = V + NV * OP;         // [2 tiles][2 streams][2 halves][128] (m, l)
  static constexpr int RED = ML + 8192;          // [2 streams][2 halves][128] maxima
  static constexpr int LIM = RED + 2048;         // [2 tiles][128] keys that a row sees
  static constexpr int IDS = LIM + 2 * kT * 2;
  static constexpr int INFO = IDS + 2 * kBlkMaxTopk * 4;
  static constexpr int BAR = INFO + 2 * int(sizeof(TileInfo));
  static constexpr int NBAR = 4 + 2 * NQ + 2 * NS + 2 * NV + 6 + 3 * NO + 4 + 8;
  static constexpr int END = BAR + NBAR * 8 + 8;
  static constexpr int BYTES = END + 1024;
  static_assert(BYTES <= 227 * 1024, "shared memory of one CTA");
  // TMEM: scores of the streams [0, 256), outputs from 256 on
  static constexpr int out_col(int stream, int buf) { return 2 * kT + (buf * 2 + stream) * DP; }
  static_assert(out_col(1, NO - 1) + DP <= 512, "TMEM columns");
};

}  // namespace

template <int DP, bool PAIR>
__global__ void __launch_bounds__(kThr, 1) block_fwd_tc(const __grid_constant__ TcFwdParams p) {
  using namespace tc;
  using M = Sm<DP, PAIR>;
  constexpr int KB = M::KB, QT = M::QT, NQ = M::NQ, NS = M::NS, NV = M::NV, NO = M::NO, OP = M::OP;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + M::BAR);
  uint64_t *tile_full = bar, *tile_empty = tile_full + 2, *q_full = tile_empty + 2,
           *q_empty = q_full + NQ, *k_full = q_empty + NQ, *k_empty = k_full + NS,
           *v_full = k_empty + NS, *v_empty = v_full + NV, *s_full = v_empty + NV,
           *p_full = s_full + 2, *pv_done = p_full + 2, *o_full = pv_done + 2,
           *o_empty = o_full + NO, *ml_full = o_empty + 2 * NO, *ml_empty = ml_full + 2,
           *pair = ml_empty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bar + M::NBAR);
  TileInfo* info = reinterpret_cast<TileInfo*>(sm + M::INFO);
  int* ids = reinterpret_cast<int*>(sm + M::IDS);
  int16_t* lims = reinterpret_cast<int16_t*>(sm + M::LIM);
  float2* ml = reinterpret_cast<float2*>(sm + M::ML);
  float* red = reinterpret_cast<float*>(sm + M::RED);
  const BlockGeom& g = p.g;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(tile_full + i, 1);
      mbar_init(tile_empty + i, kSoftWarps + kOutWarps + 2);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, kSoftWarps / 2);
      mbar_init(pv_done + i, 1);
      mbar_init(ml_full + i, kSoftWarps);
      mbar_init(ml_empty + i, kOutWarps);
    }
    for (int i = 0; i < NO; ++i) {
      mbar_init(o_full + i, 1);
      mbar_init(o_empty + 2 * i, kOutWarps);  // PAIR: by stream
      mbar_init(o_empty + 2 * i + 1, kOutWarps);
    }
    for (int i = 0; i < 8; ++i) mbar_init(pair + i, 2);
    for (int i = 0; i < NQ; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(v_full + i, 1);
      mbar_init(v_empty + i, 1);
    }
    mbar_init_fence();
  }
  if (warp == kMma) tmem_alloc512(s_tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  // false: a wait gave up, leave
  bool ok = !(p.fail && warp < kSoftWarps);

  if (warp == kLists) {
    // ---------------------------------------------------------------- lists
    int ti = 0;
    for (int64_t t = blockIdx.x; t < p.n_tiles && ok; t += gridDim.x, ++ti) {
      const int slot = ti & 1;
      int64_t x = t;
      const int sp = int(x % p.nsplit);
      x /= p.nsplit;
      const int hsub = int(x % p.hs);
      x /= p.hs;
      const int u = int(x % g.U), kh = int(x / g.U);
      const Unit un = unit_at(g, u);
      const Span ks = span_k(g, un.s);
      if (ti >= 2) ok = warp_wait(tile_empty + slot, ((ti >> 1) - 1) & 1);
      if (!ok) break;
      int* list = ids + slot * kBlkMaxTopk;
      int n = 0;
      if (un.n > 0)
        n = block_list(p.idx + u * g.is_u + kh * g.is_h, g.topk,
                       (ks.len + g.block - 1) / g.block, list);
      const int total = list_keys(list, n, g.block, ks.len);
      // keys that the tile's last row sees bound its steps
      const int seen =
          g.causal ? list_keys(list, n, g.block, min(un.pos + un.n, ks.len)) : total;
      const int steps = (seen + kT - 1) / kT;
      const int each = (steps + p.nsplit - 1) / p.nsplit;
      const int s0 = min(sp * each, steps), s1 = min(s0 + each, steps);
      if (lane == 0) {
        TileInfo& f = info[slot];
        f.s0 = s0;
        f.s1 = s1;
        f.n = n;
        f.total = total;
        f.least = g.causal ? list_keys(list, n, g.block, min(un.pos + 1, ks.len)) : total;
        f.row = un.row;
        f.rows = un.n;
        f.pos = un.pos;
        f.kbeg = ks.beg;
        f.len = ks.len;
        f.kh = kh;
        f.h0 = kh * g.G + hsub * QT * p.ht;
        f.poison = 0;
        f.part = t;
      }
      for (int r = lane; r < kT; r += 32) {
        const int tt = r / p.ht;
        lims[slot * kT + r] = int16_t(
            r >= p.rows || tt >= un.n ? 0
            : g.causal ? list_keys(list, n, g.block, min(un.pos + tt + 1, ks.len)) : total);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(tile_full + slot);
    }
  } else if (warp == kCopy) {
    // ---------------------------------------------------------------- copies
    const int per = kT / g.block;  // blocks per step
    const uint32_t blk_bytes = uint32_t(g.block) * 128;
    int gi = 0, ti = 0, tq = 0;
    int nk = 0, nv = 0;  // steps whose K, V have been asked for
    for (int64_t t = blockIdx.x; t < p.n_tiles && ok; t += gridDim.x, ++ti) {
      const int slot = ti & 1;
      ok = warp_wait(tile_full + slot, (ti >> 1) & 1);
      if (!ok) break;
      const TileInfo& f = info[slot];
      const int* list = ids + slot * kBlkMaxTopk;
      const int s0 = f.s0, s1 = f.s1, n = f.n, kbeg = f.kbeg, kh = f.kh;
      if (s1 > s0) {
        const int qs = tq % NQ;
        if (tq >= NQ) ok = warp_wait(q_empty + qs, ((tq / NQ) - 1) & 1);
        if (!ok) break;
        ++tq;
        if (lane == 0) {
          mbar_expect_tx(q_full + qs, uint32_t(p.rows) * 128 * KB * QT);
          for (int x = 0; x < QT; ++x)
            for (int kb = 0; kb < KB; ++kb)
              tma_tile3d(sm + M::Q + (qs * QT + x) * OP + kb * kPiece, &p.mq, kb * 64,
                         f.h0 + x * p.ht, f.row, q_full + qs);
        }
      }
      for (int st = s0; st < s1; ++st, ++gi) {
        const int nb = min(per, n - st * per);  // blocks of this step
        for (int kv = 0; kv < 2; ++kv) {
          const int ns = kv ? NV : NS, si = gi % ns;
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
      for (int c = nk - 1; c >= max(0, nk - NS); --c)
        warp_wait(k_full + c % NS, (c / NS) & 1, kDrainLimit);
      for (int c = nv - 1; c >= max(0, nv - NV); --c)
        warp_wait(v_full + c % NV, (c / NV) & 1, kDrainLimit);
    }
  } else if (warp == kMma) {
    // ---------------------------------------------------------------- products
    constexpr uint32_t IDESC_S = f16_idesc(kT, kT, false), IDESC_O = f16_idesc(kT, DP, true);
    const uint64_t dQ = desc_k(sm + M::Q), dK = desc_k(sm + M::K), dV = desc_mn(sm + M::V, kPiece);
    const uint32_t tm = uniform(tmem);
    // Step gi belongs to stream gi & 1 (PAIR: a step of the list is two of these, one
    // per stream, on the same K and V).  Its scores are issued after the P V
    // of step gi - 2 (products run in the order of their issue), so the
    // stream's P is no longer needed when they overwrite it.  The last two steps'
    // P V are due: step gi - 1 and gi - 2, in tiles of `tile` steps.
    int gi = 0, ti = 0, tq = 0, done = 0;       // steps with scores, tiles, with P V
    int due_tile[2] = {0, 0}, due_i[2] = {0, 0};  // by stream: the tile, the step in it
    bool due_last[2] = {false, false};
    auto product_pv = [&]() {                   // of step `done`
      const int x = done & 1, kv = PAIR ? done >> 1 : done, si = kv % NV;
      const int tile = x ? due_tile[1] : due_tile[0];
      const int i = x ? due_i[1] : due_i[0], buf = tile % NO;
      ok = ok && warp_wait(p_full + x, (done >> 1) & 1) && warp_wait(v_full + si, (kv / NV) & 1);
      // the stream's first step of the tile overwrites its output
      if (i < 2 && tile >= NO)
        ok = ok && warp_wait(o_empty + 2 * buf + (PAIR ? x : 0), (tile / NO - 1) & 1);
      if (!ok) return;
      tc_fence_after();
      if (elect_one()) {
        mma_tm<kT>(tm + M::out_col(x, buf), tm + x * kT, 32, 32, desc_at(dV, si * OP), IDESC_O,
                   i >= 2);
        mma_commit(pv_done + x);
        if (!PAIR || x) mma_commit(v_empty + si);
        if (x ? due_last[1] : due_last[0]) mma_commit(o_full + buf);
      }
      __syncwarp();
      ++done;
    };
    for (int64_t t = blockIdx.x; t < p.n_tiles && ok; t += gridDim.x, ++ti) {
      const int slot = ti & 1;
      if (!__all_sync(0xffffffffu, mbar_test(tile_full + slot, (ti >> 1) & 1))) {
        while (ok && done < gi) product_pv();  // the lists may wait for these tiles to be written
        ok = ok && warp_wait(tile_full + slot, (ti >> 1) & 1);
      }
      if (!ok) break;
      const int n = uniform(info[slot].s1 - info[slot].s0) * QT;
      __syncwarp();
      if (lane == 0) mbar_arrive(tile_empty + slot);
      if (n <= 0) continue;
      const int qs = tq % NQ;
      ok = warp_wait(q_full + qs, (tq / NQ) & 1);
      for (int i = 0; i < n && ok; ++i, ++gi) {
        const int x = gi & 1, kv = PAIR ? gi >> 1 : gi, si = kv % NS;
        if (gi - done == 2) product_pv();
        ok = ok && warp_wait(k_full + si, (kv / NS) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          mma_kk<KB>(tm + x * kT, desc_at(dQ, PAIR ? x * OP : qs * OP), kPiece,
                     desc_at(dK, si * OP), kPiece, IDESC_S);
          mma_commit(s_full + x);
          if (!PAIR || x) mma_commit(k_empty + si);
          if (i == n - 1) mma_commit(q_empty + qs);
        }
        __syncwarp();
        if (x) {
          due_tile[1] = tq;
          due_i[1] = i;
          due_last[1] = i == n - 1;
        } else {
          due_tile[0] = tq;
          due_i[0] = i;
          due_last[0] = i == n - 1;
        }
      }
      ++tq;
    }
    while (ok && done < gi) product_pv();
    // every product has completed before TMEM is given up
    for (int k = 1; k <= 2 && k <= gi; ++k) {
      const int c = gi - k;
      if (ok) ok = warp_wait(pv_done + (c & 1), (c >> 1) & 1);
      if (!ok) {
        warp_wait(s_full + (c & 1), (c >> 1) & 1, kDrainLimit);
        warp_wait(pv_done + (c & 1), (c >> 1) & 1, kDrainLimit);
      }
    }
  } else if (warp < kSoftWarps) {
    // ---------------------------------------------------------------- softmax
    const int quad = warp & 3, half = (warp >> 2) & 1, x = warp >> 3;  // lanes, columns, stream
    const int r = quad * 32 + lane;
    const uint32_t lanes = uint32_t(quad * 32) << 16;
    const uint32_t tS = tmem + lanes + x * kT + half * 64;
    int gi = 0, ti = 0, to = 0;  // steps, tiles, tiles with steps
    for (int64_t t = blockIdx.x; t < p.n_tiles; t += gridDim.x, ++ti) {
      const int slot = ti & 1;
      ok = ok && warp_wait(tile_full + slot, (ti >> 1) & 1);
      if (!ok) break;
      const int s0 = info[slot].s0, steps = (info[slot].s1 - s0) * QT;
      const int total = info[slot].total, least = info[slot].least;
      const int lim = lims[slot * kT + r];
      const int buf = to % NO;
      const int head = (gi ^ x) & 1;  // the stream's first step of the tile
      float m = neg_inf(), l = 0.f;
      for (int i = head; i < steps; i += 2) {
        const int c = gi + i, st = s0 + (PAIR ? i >> 1 : i);
        ok = ok && warp_wait(s_full + x, (c >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const int mine = lim - st * kT - half * 64;  // of these 64 columns the row sees
        const bool cut = __any_sync(0xffffffffu, mine < 64);
        // the maximum over columns [0, 32), then [32, 64), which stay in registers
        float sv[32];
        float c0 = neg_inf(), c1 = c0, c2 = c0, c3 = c0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tmem_ld32(tS + h * 32, sv);
          tmem_wait_ld();
          if (cut) {
#pragma unroll
            for (int j = 0; j < 32; ++j) sv[j] = j < mine - h * 32 ? sv[j] : neg_inf();
          }
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            c0 = fmaxf(c0, sv[j]);
            c1 = fmaxf(c1, sv[j + 1]);
            c2 = fmaxf(c2, sv[j + 2]);
            c3 = fmaxf(c3, sv[j + 3]);
          }
        }
        const float cm = fmaxf(fmaxf(c0, c1), fmaxf(c2, c3));
        red[(x * 2 + half) * kT + r] = cm;
        __syncwarp();
        if (lane == 0) mbar_arrive(pair + x * 4 + quad);
        ok = warp_wait(pair + x * 4 + quad, (c >> 1) & 1);
        if (!ok) break;
        // (the word is written again in the stream's next step, whose scores
        // wait for the P of every warp that reads it here)
        const float mx = fmaxf(m, fmaxf(cm, red[(x * 2 + (half ^ 1)) * kT + r]));
        // keep the old scale while p stays below 2^8
        const bool grow = !((mx - m) * g.qmul <= 8.f) && mx != m;
        const float old = m;
        if (grow) m = mx;
        const float mq = m == neg_inf() ? 0.f : m * g.qmul;
        const int end = (st + 1) * kT;
        const bool tail = total < end, mixed = least < min(total, end);
        if ((tail || mixed) && (!PAIR || x == 0)) {  // (the other stream's P V comes after)
          const int kv = PAIR ? c >> 1 : c, si = kv % NV;
          ok = warp_wait(v_full + si, (kv / NV) & 1);
          if (!ok) break;
          const int nv = min(total - st * kT, kT), tid = threadIdx.x & 255;
          for (int kb = 0; kb < KB; ++kb) {
            uint4* v = reinterpret_cast<uint4*>(sm + M::V + si * OP + kb * kPiece);
            for (int k = nv * 8 + tid; k < kT * 8; k += 256) v[k] = make_uint4(0, 0, 0, 0);
            if (!mixed) continue;
#pragma unroll
            for (int e = 0; e < kT * 8 / 256; ++e) {
              const int k = e * 256 + tid;
              if (k >= nv * 8) break;
              const uint4 y = v[k];
              const uint32_t big =
                  __vmaxu2(__vmaxu2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu),
                           __vmaxu2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu));
              if ((big & 0xffffu) < 0x7f80u && big < 0x7f800000u) continue;  // all finite
              uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                if ((w[z] & 0x7f80u) == 0x7f80u) w[z] &= 0xffff0000u;
                if ((w[z] & 0x7f800000u) == 0x7f800000u) w[z] &= 0xffffu;
              }
              v[k] = make_uint4(w[0], w[1], w[2], w[3]);
              *const_cast<volatile int*>(&info[slot].poison) = 1;
            }
          }
          fence_proxy_async();  // -> visible to the tensor cores
          __syncwarp();
        }
        if (i > head && __any_sync(0xffffffffu, grow)) {
          // O holds the stream's steps before this one at the old scale
          ok = warp_wait(pv_done + x, ((c >> 1) - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const float corr = grow ? ex2((old - m) * g.qmul) : 1.f;  // 0 from -inf
          l *= corr;
          const uint32_t tO = tmem + lanes + M::out_col(x, buf) + half * (DP / 2);
#pragma unroll 1
          for (int k = 0; k < DP / 32; ++k) {
            float o[16];
            tmem_ld16(tO + k * 16, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] *= corr;
            tmem_st16(tO + k * 16, o);
          }
        }
        float2 sum = make_float2(0.f, 0.f);
        const float2 qm = f2s(g.qmul), nm = f2s(-mq);
#pragma unroll
        for (int h = 1; h >= 0; --h) {
          if (h == 0) {
            tmem_ld32(tS, sv);
            tmem_wait_ld();
            if (cut) {
#pragma unroll
              for (int j = 0; j < 32; ++j) sv[j] = j < mine ? sv[j] : neg_inf();
            }
          }
          float w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 z = f2fma(make_float2(sv[2 * j], sv[2 * j + 1]), qm, nm);
            const float2 y = make_float2(ex2(z.x), ex2(z.y));
            sum = f2add(sum, y);
            w[j] = __uint_as_float(bf16x2_bits(y.x, y.y));
          }
          tmem_st16(tS + h * 32, w);
        }
        l += sum.x + sum.y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + x);
      }
      if (!ok) break;
      gi += steps;
      if (steps > 0) {  // the row's scale and sum, for the warps that write the tile
        const int par = to & 1;
        if (to >= 2) ok = warp_wait(ml_empty + par, ((to >> 1) - 1) & 1);
        if (!ok) break;
        ml[((par * 2 + x) * 2 + half) * kT + r] = make_float2(m * g.qmul, l);
        ++to;
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_full + par);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(tile_empty + slot);
    }
  } else {
    // ---------------------------------------------------------------- output
    const int quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lanes = uint32_t(quad * 32) << 16;
    const int th = r % p.ht, tt = r / p.ht;
    const bool wide = wide_rows(p.out, g.D);
    int gi = 0, ti = 0, to = 0;
    for (int64_t t = blockIdx.x; t < p.n_tiles; t += gridDim.x, ++ti) {
      const int slot = ti & 1;
      ok = ok && warp_wait(tile_full + slot, (ti >> 1) & 1);
      if (!ok) break;
      const TileInfo f = info[slot];
      const bool valid = r < p.rows && tt < f.rows;
      const int steps = (f.s1 - f.s0) * QT, buf = to % NO, par = to & 1;
      const bool some = steps > 0;
      // which streams had a step
      const bool has0 = steps > 1 || (some && (gi & 1) == 0);
      const bool has1 = steps > 1 || (some && (gi & 1) == 1);
      gi += steps;
      float La = neg_inf(), Lb = neg_inf(), w0 = 0.f, w1 = 0.f;
      if (some) {
        ok = warp_wait(ml_full + par, (to >> 1) & 1);
        if (!ok) break;
        float2 a = ml[par * 4 * kT + r], b = ml[(par * 4 + 2) * kT + r];
        a.y += ml[(par * 4 + 1) * kT + r].y;  // the halves of a row share m
        b.y += ml[(par * 4 + 3) * kT + r].y;
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_empty + par);
        // log2-sum-exp; O of a stream is scaled by its own 2^-m
        if (a.y != 0.f) La = a.x + lg2(a.y);
        if (b.y != 0.f) Lb = b.x + lg2(b.y);
        if (!PAIR) {  // of both together
          const float big = fmaxf(La, Lb);
          float L = neg_inf();
          if (big != neg_inf()) L = big + lg2(ex2(La - big) + ex2(Lb - big));
          if (La != La || Lb != Lb) L = La + Lb;  // not a number
          La = Lb = L;
        }
        if (a.y != 0.f) w0 = ex2(a.x - La);
        if (b.y != 0.f) w1 = ex2(b.x - Lb);
        ok = warp_wait(o_full + buf, (to / NO) & 1);
        if (!ok) break;
        tc_fence_after();
        ++to;
      }
      const bool poison = some && *const_cast<volatile int*>(&info[slot].poison);
#pragma unroll 1
      for (int x = 0; x < QT; ++x) {  // the tiles of this unit (one, of both streams)
        const float L = x ? Lb : La;
        const int64_t qrow = int64_t(f.row + tt) * g.H + f.h0 + x * p.ht + th;
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) {
          const int col = c * 32;
          float o[32], v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
          __syncwarp();
          if (PAIR ? some : has0) {
            tmem_ld32(tmem + lanes + M::out_col(PAIR ? x : 0, buf) + col, v);
            tmem_wait_ld();
            const float s = x ? w1 : w0;
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = v[i] * s;
          }
          if (!PAIR && has1) {
            tmem_ld32(tmem + lanes + M::out_col(1, buf) + col, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = fmaf(v[i], w1, o[i]);
          }
          if (poison && valid && L != neg_inf()) {  // values that were taken out of V
            const int* list = ids + slot * kBlkMaxTopk;
            const int lim = lims[slot * kT + r];
            for (int k = f.s0 * kT; k < min(lim, f.s1 * kT); ++k) {
              const __nv_bfloat16* vr =
                  p.V +
                  (int64_t(f.kbeg + list[k / g.block] * g.block + k % g.block) * g.Hkv + f.kh) *
                      g.D;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float y = col + i < g.D ? __bfloat162float(vr[col + i]) : 0.f;
                if (!(fabsf(y) <= 3.4e38f)) o[i] += y;
              }
            }
          }
          if (!PAIR && p.nsplit > 1) {
            float* d = p.part_o + (f.part * p.rows + r) * g.D + col;
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (valid && col + q * 4 < g.D)
                *reinterpret_cast<float4*>(d + q * 4) =
                    make_float4(o[q * 4], o[q * 4 + 1], o[q * 4 + 2], o[q * 4 + 3]);
          }
          if (c == DP / 32 - 1) {  // the buffer is free before the row's end is written
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && some) mbar_arrive(o_empty + 2 * buf + x);
          }
          if (valid && (PAIR || p.nsplit == 1))
            store_row(p.out + qrow * g.D, col, g.D, o, wide);
        }
        if (valid && (PAIR || p.nsplit == 1)) p.lse[qrow] = L * kLn2;
        else if (valid) p.part_l[f.part * p.rows + r] = L;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(tile_empty + slot);
    }
  }
  if (!ok) atomicOr(&g_err, 2);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_free512(tmem);
}

namespace {

// Splits of a tile joined: out = sum_i 2^(L_i - L) o_i, L = log2 sum_i 2^L_i.
__global__ void __launch_bounds__(128) block_join(const TcFwdParams p) {
  const BlockGeom& g = p.g;
  const int64_t tile = blockIdx.x;  // (key head, unit, head group)
  const int hsub = int(tile % p.hs), u = int((tile / p.hs) % g.U), kh = int(tile / p.hs / g.U);
  const Unit un = unit_at(g, u);
  const int vec = g.D / 4;
  for (int i = threadIdx.x; i < p.rows * vec; i += 128) {
    const int r = i / vec, c = i - r * vec, t = r / p.ht;
    if (t >= un.n) continue;
    const float* L = p.part_l + tile * p.nsplit * p.rows + r;
    float mx = neg_inf();
    for (int s = 0; s < p.nsplit; ++s) mx = fmaxf(mx, L[s * p.rows]);
    const float base = mx == neg_inf() ? 0.f : mx;
    float sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < p.nsplit; ++s) {
      const float w = ex2(L[s * p.rows] - base);
      if (w == 0.f) continue;  // a split that saw nothing
      const float4 x = reinterpret_cast<const float4*>(
          p.part_o + ((tile * p.nsplit + s) * p.rows + r) * g.D)[c];
      sum += w;
      o.x = fmaf(w, x.x, o.x);
      o.y = fmaf(w, x.y, o.y);
      o.z = fmaf(w, x.z, o.z);
      o.w = fmaf(w, x.w, o.w);
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    const int64_t row = int64_t(un.row + t) * g.H + kh * g.G + hsub * p.ht + r % p.ht;
    *reinterpret_cast<uint2*>(p.out + row * g.D + c * 4) =
        make_uint2(tc::bf16x2_bits(o.x * inv, o.y * inv), tc::bf16x2_bits(o.z * inv, o.w * inv));
    if (c == 0) p.lse[row] = sum != 0.f ? (base + lg2(sum)) * kLn2 : neg_inf();
  }
}

struct Shape {
  int ht, hs, rows, nsplit;
  int64_t tiles;
  bool pair;
};
Shape shape(const BlockGeom& g) {
  Shape s{};
  s.ht = tile_heads(g);
  s.hs = g.G / s.ht;
  s.rows = s.ht * g.qb;
  s.tiles = int64_t(g.U) * g.Hkv * s.hs;
  s.nsplit = 1;
  // Two tiles of one unit at a time where there are two, and pairs enough for
  // every SM (prompt of 32,768, 4 heads of 128 a key head: 0.89 -> 0.81 ms)
  s.pair = s.hs > 1 && s.tiles / 2 >= sm_count();
  if (s.pair) {
    s.hs /= 2;
    s.tiles /= 2;
    return s;
  }
  // Fewer tiles than SMs: split each over its steps so that most SMs work.
  // One step a split at least; never more CTAs than SMs (a second round of
  // one CTA costs as much as the first).
  const int64_t steps = (int64_t(g.topk) * g.block + kT - 1) / kT;
  const int64_t fit = sm_count() / std::max<int64_t>(1, s.tiles);
  s.nsplit = int(std::max<int64_t>(1, std::min(steps, fit)));
  return s;
}

}  // namespace

size_t block_fwd_tc_workspace(const BlockGeom& g) {
  const Shape s = shape(g);
  return s.nsplit > 1 ? size_t(s.tiles) * s.nsplit * s.rows * (g.D + 1) * 4 : 0;
}

gattn_status launch_block_fwd_tc(const BlockGeom& g, const void* Q, const void* K, const void* V,
                                 const int32_t* idx, void* out, float* lse, void* ws,
                                 cudaStream_t st) {
  const Shape s = shape(g);
  TcFwdParams p{};
  p.g = g;
  if (!encode_heads_map(&p.mq, Q, g.Nq, g.H, g.D, s.ht, g.qb) ||
      !encode_heads_map(&p.mk, g.Nk ? K : Q, g.Nk, g.Hkv, g.D, 1, g.block) ||
      !encode_heads_map(&p.mv, g.Nk ? V : Q, g.Nk, g.Hkv, g.D, 1, g.block))
    return GATTN_ERR_CUDA;
  p.idx = idx;
  p.V = static_cast<const __nv_bfloat16*>(V);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.ht = s.ht;
  p.hs = s.hs;
  p.rows = s.rows;
  p.nsplit = s.nsplit;
  p.fail = block_wait_test();
  p.n_tiles = s.tiles * s.nsplit;
  p.part_o = static_cast<float*>(ws);
  p.part_l = p.part_o + (s.nsplit > 1 ? s.tiles * s.nsplit * s.rows * g.D : 0);
  const unsigned grid = unsigned(std::min<int64_t>(p.n_tiles, sm_count()));
  auto go = [&](auto kern, int bytes) -> gattn_status {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) {
      kern<<<grid, kThr, bytes, st>>>(p);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
      set_error("gattn_block_fwd launch failed: %s", cudaGetErrorString(e));
      return GATTN_ERR_CUDA;
    }
    return GATTN_OK;
  };
  gattn_status r;
  if (s.pair)
    r = g.D <= 64 ? go(block_fwd_tc<64, true>, Sm<64, true>::BYTES)
                  : go(block_fwd_tc<128, true>, Sm<128, true>::BYTES);
  else
    r = g.D <= 64 ? go(block_fwd_tc<64, false>, Sm<64, false>::BYTES)
                  : go(block_fwd_tc<128, false>, Sm<128, false>::BYTES);
  if (r != GATTN_OK || s.nsplit == 1) return r;
  block_join<<<unsigned(s.tiles), 128, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("gattn_block_fwd (join) launch failed: %s", cudaGetErrorString(e));
    return GATTN_ERR_CUDA;
  }
  return GATTN_OK;
}

cudaError_t block_fwd_tc_take_error(int* err) {
  cudaError_t e = cudaMemcpyFromSymbol(err, g_err, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && *err) e = cudaMemcpyToSymbol(g_err, &zero, sizeof(int));
  return e;
}

}  // namespace gattn
