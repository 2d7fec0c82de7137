// Attention over the 8-bit key/value cache, for the few newest tokens of each
// sequence.
//
//   s_rj = scale * ks_j (q_r . kc_j),  o_r = sum_j p_rj vs_j vc_j,
//   p_rj = exp(s_rj) / sum_j' exp(s_rj')
// with kc, vc the E4M3 codes and ks, vs the scales of token j's block. The rows
// r of a key head are its new tokens times its query heads, 16 to a tile.
//
// Bound by memory: 2 d bytes of cache for each token and key head against
// 4 d flops for each of its rows. So codes are read once (16 rows at a time),
// converted to fp16 in registers (exact) and multiplied by mma.sync
// m16n8k16: the tensor work of 16 rows is far below its limit.
//
// Work is split over the tokens: a CTA takes one piece of one sequence's
// tokens for one row tile of a key head; each of its warps walks 32-token
// tiles on its own, with its own ring of TMA loads, running maximum, sum and
// output (no barrier between warps), merged at the CTA's end. Pieces are
// joined by a second kernel, which also turns the scores of the first into the
// tokens' weights (a probability needs the sum over all pieces).
//
// Scales differ from block to block. K's multiplies the scores. V's goes into
// the exponent: with lv = log2 vs, the operand of P V is 2^(s + lv - mv) <= 1
// with mv a running maximum of s + lv, so that fp16 holds it whatever the
// scales are, while the sum takes 2^(s - m).
//
// The order of channels and tokens inside an MMA is free (sums), so it is
// chosen for the loads: a lane reads 16 contiguous bytes of a token at a time
// and 8 lanes hit 8 different 16-byte bank groups of the swizzled tile.
//
// Tokens that a row must not see get a score of -inf; V codes of tokens behind
// the sequence (free slots, holding anything) are cleared before use.

#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "e4m3.cuh"
#include "serving.h"
#include "tc.cuh"

namespace sda {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTok = 32;       // tokens of a warp's tile
constexpr int kStages = 2;     // tiles in flight per warp
constexpr int kCtasPerSm = 3;
constexpr int kSms = 148;

template <int D>
struct Smem {
  static constexpr int kHalf = kTok * D;           // K or V codes of a tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kRing = kWarps * kStages * kStage;
  // merge at the end, over the ring: per warp 16 rows of output and (m, l, mv)
  static constexpr int kMerge = kWarps * 16 * (D + 4) * 4;
  static constexpr int kBars = kRing > kMerge ? kRing : kMerge;
  static constexpr int kTotal = kBars + 8 * kWarps * kStages + 16;
};

struct Args {
  const uint16_t* q;
  const int32_t* seq;
  const int32_t* lens;
  const int32_t* table;
  const float* k_scale;
  const float* v_scale;
  uint16_t* o;
  float* part_o;   // [B, H_kv, n_split, rows_pad, d]
  float* part_ml;  // [B, H_kv, n_split, rows_pad, 4]: m, l, mv
  float* scores;   // [B, H_kv, tokens, rows_pad], log2 units; NULL: weights are not kept
  unsigned* status;
  int n_split, row_tiles, rows_pad;
  uint64_t wait_ns;
};

// Order of the 8 tokens of an n-tile and of the 8 channel groups of a row
// (d = 128: rows of 8 16-byte chunks): neighbours differ in the bit that the
// swizzle needs.
__device__ __forceinline__ int spread(int i) { return (i >> 1) | ((i & 1) << 2); }

__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.f : m; }

// 16-byte chunk `ch` of token row `row` in a swizzled tile of D-byte rows.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int row, int ch) {
  if constexpr (D == 128) return row * 128 + ((ch ^ (row & 7)) << 4);
  else return row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
cache_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, Cache c, Args a) {
  using S = Smem<D>;
  constexpr int KS = D / 16;     // k16 steps of a score
  constexpr int NT = D / 8;      // n-tiles of the output
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + kWarps * kStages);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g4 = lane >> 2, cq = lane & 3;

  // piece slowest: the empty pieces of short sequences come last
  const int per_piece = c.B * c.H_kv * a.row_tiles;
  const int piece = blockIdx.x / per_piece;
  const int rest = blockIdx.x % per_piece;
  const int rt = rest % a.row_tiles;
  const int hk = (rest / a.row_tiles) % c.H_kv;
  const int b = rest / (a.row_tiles * c.H_kv);
  const int g = c.H / c.H_kv;

  bool bad = false;
  const NewRows nr = new_rows(c, a.seq, a.lens, b, bad);
  if (bad && threadIdx.x == 0) report_status(a.status, kStatusBadIndex);
  const int rows = nr.n * g;          // rows of this sequence and key head
  const int r0 = rt * 16;
  if (r0 >= rows) return;
  // tokens seen by row r: below first + r / g + 1, and no more than the table holds
  const int last_row = min(r0 + 15, rows - 1);
  const int seen = min(nr.len, max(0, nr.first + last_row / g + 1));
  const int n_tiles = (seen + kTok - 1) / kTok;
  const int tile0 = static_cast<int>(static_cast<long long>(n_tiles) * piece / a.n_split);
  const int tile1 = static_cast<int>(static_cast<long long>(n_tiles) * (piece + 1) / a.n_split);
  const bool whole = a.n_split == 1;
  const size_t part = (static_cast<size_t>(b) * c.H_kv + hk) * a.n_split + piece;
  if (tile0 >= tile1 && !whole) {     // nothing in this piece: an empty sum
    if (threadIdx.x < 16 && r0 + threadIdx.x < rows)
      *reinterpret_cast<float4*>(a.part_ml + (part * a.rows_pad + r0 + threadIdx.x) * 4) =
          make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    return;
  }
  if (threadIdx.x < kWarps * kStages) tc::mbar_init(&bars[threadIdx.x], 1);
  if (threadIdx.x == 0) *abort_flag = 0;
  tc::fence_mbar_init();
  __syncthreads();

  const int32_t* blocks = a.table + static_cast<size_t>(b) * c.max_blocks;
  const int shift = 31 - __clz(c.block);
  unsigned char* ring = smem + warp * kStages * S::kStage;
  uint64_t* full = bars + warp * kStages;

  // block of a 16-token half tile, -1 where the number is not one of the pool
  auto block_of = [&](int t16) {
    const int tok = t16 * 16;
    if (tok >= seen) return -1;
    const int blk = __ldg(blocks + (tok >> shift));
    return blk >= 0 && blk < c.n_blocks ? blk : -1;
  };
  const int my_tiles = tile1 - tile0 > warp ? (tile1 - tile0 - warp + kWarps - 1) / kWarps : 0;
  // This warp's blocks and scales, a batch of 16 tiles per register: lane l holds half l % 2 of tile
  // base + l / 2. The next batch is read a batch ahead of its use.
  struct Held {
    int blk;
    float ks, vs;
  };
  auto hold = [&](int base) {
    Held x{-1, 0.f, 0.f};
    const int i = base + lane / 2;
    if (i < my_tiles) {
      const int t = tile0 + warp + i * kWarps;
      x.blk = block_of(t * 2 + (lane & 1));
      if (x.blk < 0 && t * kTok + 16 * (lane & 1) < seen) report_status(a.status, kStatusBadIndex);
      if (x.blk >= 0) {
        const size_t head = static_cast<size_t>(x.blk) * c.H_kv + hk;
        x.ks = __ldg(a.k_scale + head);
        x.vs = __ldg(a.v_scale + head);
      }
    }
    return x;
  };
  // one lane: the loads of tile i into its stage (absent blocks: nothing, their tokens are not seen)
  auto load_tile = [&](int i, int blk0, int blk1) {
    const int st = i % kStages;
    const int tok = (tile0 + warp + i * kWarps) * kTok;
    unsigned char* dst = ring + st * S::kStage;
    if (c.block >= kTok) {
      tc::mbar_arrive_expect_tx(&full[st], blk0 >= 0 ? S::kStage : 0);
      if (blk0 >= 0) {
        const int y = (blk0 * c.H_kv + hk) * c.block + (tok & (c.block - 1));
        tc::tma_load_2d(dst, &tm_k, &full[st], 0, y);
        tc::tma_load_2d(dst + S::kHalf, &tm_v, &full[st], 0, y);
      }
    } else {
      tc::mbar_arrive_expect_tx(&full[st], (blk0 >= 0 ? S::kHalf : 0) + (blk1 >= 0 ? S::kHalf : 0));
      for (int u = 0; u < 2; ++u) {
        const int blk = u ? blk1 : blk0;
        if (blk < 0) continue;
        const int y = (blk * c.H_kv + hk) * c.block;
        tc::tma_load_2d(dst + u * 16 * D, &tm_k, &full[st], 0, y);
        tc::tma_load_2d(dst + S::kHalf + u * 16 * D, &tm_v, &full[st], 0, y);
      }
    }
  };

  Held now = hold(0);
  int issued = 0;
  for (; issued < kStages && issued < my_tiles; ++issued) {
    const int b0 = __shfl_sync(0xffffffffu, now.blk, 2 * issued), b1 = __shfl_sync(0xffffffffu, now.blk, 2 * issued + 1);
    if (lane == 0) load_tile(issued, b0, b1);
  }
  Held next = hold(16);

  // Q fragments in fp16: row r times 2^(14 - e), e its exponent, undone in the score's factor
  uint32_t qf[KS][4];
  float factor[2];
  int lim[2];                         // tokens that rows g4 and g4 + 8 of the tile see
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = r0 + g4 + 8 * u;
    const bool there = r < rows;
    const int i = there ? r / g : 0, qh = there ? r % g : 0;
    lim[u] = there ? min(nr.len, max(0, nr.first + i + 1)) : seen;  // rows that are not there: computed, not kept
    const uint16_t* src = a.q + static_cast<size_t>(nr.row0 + i) * c.ld_q + (hk * g + qh) * D;
    uint4 x[D / 32];                  // this lane's channels: 16 at 16 cq (and 16 at 64 + 16 cq)
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
      x[e] = there ? __ldg(reinterpret_cast<const uint4*>(src + 64 * (e / 2) + 16 * cq + 8 * (e % 2)))
                   : make_uint4(0u, 0u, 0u, 0u);
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      const uint32_t in[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
      for (int f = 0; f < 4; ++f) top = fmaxf(top, fmaxf(fabsf(bf16_lo(in[f])), fabsf(bf16_hi(in[f]))));
    }
    top = quad_max(top);
    const int e2 = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -110);
    const float up = __uint_as_float(static_cast<uint32_t>(14 - e2 + 127) << 23);
    factor[u] = __uint_as_float(static_cast<uint32_t>(e2 - 14 + 127) << 23) * c.scale_log2;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      const uint32_t in[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
      for (int f = 0; f < 4; ++f) {   // channels 8 e' + 2 f, + 1 of the lane's 16
        const int kk = 4 * (e / 2) + 2 * (e % 2) + f / 2;
        qf[kk][u + 2 * (f % 2)] = pack_f16(bf16_lo(in[f]) * up, bf16_hi(in[f]) * up);
      }
    }
  }

  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, mv[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float* my_scores = a.scores == nullptr
                         ? nullptr
                         : a.scores + (static_cast<size_t>(b) * c.H_kv + hk) * c.max_blocks * c.block * a.rows_pad;
  bool ok = true;

  for (int i = 0; i < my_tiles; ++i) {
    const int st = i % kStages;
    const int tok0 = (tile0 + warp + i * kWarps) * kTok;
    if (i % 16 == 0 && i > 0) {
      now = next;
      next = hold(i + 16);
    }
    const int la = 2 * (i % 16), lb = la + 1;
    const int blk_a = __shfl_sync(0xffffffffu, now.blk, la), blk_b = __shfl_sync(0xffffffffu, now.blk, lb);
    const float ks_a = __shfl_sync(0xffffffffu, now.ks, la), ks_b = __shfl_sync(0xffffffffu, now.ks, lb);
    const float vs_a = __shfl_sync(0xffffffffu, now.vs, la), vs_b = __shfl_sync(0xffffffffu, now.vs, lb);
    ok = tc::wait_warp(&full[st], (i / kStages) & 1, abort_flag, a.wait_ns);
    if (!ok) break;
    const unsigned char* kt = ring + st * S::kStage;
    const unsigned char* vt = kt + S::kHalf;

    // scores of the 32 tokens: n-tile n holds tokens 8 n + order(2 cq), 8 n + order(2 cq + 1) of this lane
    float s[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int row = 8 * n + (D == 128 ? spread(g4) : g4);
      s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int half = 0; half < KS / 4; ++half) {
        const uint4 x = *reinterpret_cast<const uint4*>(kt + chunk_at<D>(row, cq + 4 * half));
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mma_f16(s[n], qf[4 * half + e], e4m3x2_to_f16x2(static_cast<uint16_t>(in[e])),
                  e4m3x2_to_f16x2(static_cast<uint16_t>(in[e] >> 16)));
      }
    }
    const int t_lo = D == 128 ? cq : 2 * cq, t_hi = D == 128 ? cq + 4 : 2 * cq + 1;  // the lane's tokens of an n-tile
    const bool edge = tok0 + kTok > min(lim[0], lim[1]) || blk_a < 0 || blk_b < 0;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] *= factor[e / 2] * (n < 2 ? ks_a : ks_b);
    if (__any_sync(0xffffffffu, edge)) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = tok0 + 8 * n + (e % 2 ? t_hi : t_lo);
          if (tok >= lim[e / 2] || (n < 2 ? blk_a : blk_b) < 0) s[n][e] = -INFINITY;
        }
    }
    if (my_scores != nullptr) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = r0 + g4 + 8 * u;
        if (r < rows) {
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int tok = tok0 + 8 * n + (e ? t_hi : t_lo);
              if (tok < seen) my_scores[static_cast<size_t>(tok) * a.rows_pad + r] = s[n][2 * u + e];
            }
        }
      }
    }
    // running maxima; lv = log2 of V's scale
    const float lv_a = __log2f(vs_a), lv_b = __log2f(vs_b);
    uint32_t pf[2][4];                // P fragments of the two k16 steps
    float alpha_v[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float ma = quad_max(fmaxf(fmaxf(s[0][2 * u], s[0][2 * u + 1]), fmaxf(s[1][2 * u], s[1][2 * u + 1])));
      const float mb = quad_max(fmaxf(fmaxf(s[2][2 * u], s[2][2 * u + 1]), fmaxf(s[3][2 * u], s[3][2 * u + 1])));
      const float m_new = fmaxf(m[u], fmaxf(ma, mb));
      const float mv_new = fmaxf(mv[u], fmaxf(ma + lv_a, mb + lv_b));
      const float mr = finite_or_0(m_new), mvr = finite_or_0(mv_new);
      l[u] *= tc::ex2(m[u] - mr);
      alpha_v[u] = tc::ex2(mv[u] - mvr);
      m[u] = m_new;
      mv[u] = mv_new;
      // 2^(s + lv - mv) = 2^(s - m) 2^(m + lv - mv)
      const float fa = tc::ex2(fminf(mr + lv_a - mvr, 127.f)), fb = tc::ex2(fminf(mr + lv_b - mvr, 127.f));
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float p0 = tc::ex2(s[n][2 * u] - mr), p1 = tc::ex2(s[n][2 * u + 1] - mr);
        sum += p0 + p1;
        const float f = n < 2 ? fa : fb;
        pf[n / 2][u + 2 * (n % 2)] = pack_f16(p0 * f, p1 * f);
      }
      l[u] += sum;
    }
    if (__any_sync(0xffffffffu, alpha_v[0] != 1.f || alpha_v[1] != 1.f)) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] *= alpha_v[e / 2];
    }
    // O += P V: this lane's n-tiles j are its channel group g4, its tokens those of P
    const bool clear = tok0 + kTok > seen || blk_a < 0 || blk_b < 0;  // V rows of no token of the sequence
#pragma unroll
    for (int n2 = 0; n2 < 2; ++n2) {
      uint32_t w[4][D / 32];          // 4 tokens, d / 8 channels of the lane's group
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 16 * n2 + 8 * (e / 2) + (e % 2 ? t_hi : t_lo);
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(vt + chunk_at<D>(row, spread(g4)));
          w[e][0] = x.x;
          w[e][1] = x.y;
          w[e][2] = x.z;
          w[e][3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(vt + chunk_at<D>(row, g4 >> 1) + 8 * (g4 & 1));
          w[e][0] = x.x;
          w[e][1] = x.y;
        }
        if (clear && (tok0 + row >= seen || (n2 == 0 ? blk_a : blk_b) < 0)) {
#pragma unroll
          for (int f = 0; f < D / 32; ++f) w[e][f] = 0u;
        }
      }
#pragma unroll
      for (int f = 0; f < D / 32; ++f) {
        // channels 4 f .. 4 f + 3 of the group, tokens paired byte by byte
        const uint32_t a01 = __byte_perm(w[0][f], w[1][f], 0x5140), a23 = __byte_perm(w[0][f], w[1][f], 0x7362);
        const uint32_t b01 = __byte_perm(w[2][f], w[3][f], 0x5140), b23 = __byte_perm(w[2][f], w[3][f], 0x7362);
        mma_f16(acc[4 * f], pf[n2], e4m3x2_to_f16x2(static_cast<uint16_t>(a01)), e4m3x2_to_f16x2(static_cast<uint16_t>(b01)));
        mma_f16(acc[4 * f + 1], pf[n2], e4m3x2_to_f16x2(static_cast<uint16_t>(a01 >> 16)), e4m3x2_to_f16x2(static_cast<uint16_t>(b01 >> 16)));
        mma_f16(acc[4 * f + 2], pf[n2], e4m3x2_to_f16x2(static_cast<uint16_t>(a23)), e4m3x2_to_f16x2(static_cast<uint16_t>(b23)));
        mma_f16(acc[4 * f + 3], pf[n2], e4m3x2_to_f16x2(static_cast<uint16_t>(a23 >> 16)), e4m3x2_to_f16x2(static_cast<uint16_t>(b23 >> 16)));
      }
    }
    __syncwarp();                     // every lane has read the stage
    if (issued < my_tiles) {
      const int from = issued / 16 == i / 16 ? now.blk : next.blk;
      const int b0 = __shfl_sync(0xffffffffu, from, 2 * (issued % 16)), b1 = __shfl_sync(0xffffffffu, from, 2 * (issued % 16) + 1);
      if (lane == 0) load_tile(issued, b0, b1);
      ++issued;
    }
  }
  if (!ok) {                          // given up: no load is in flight when the CTA ends
    volatile int never = 0;
    for (int i = max(0, issued - kStages); i < issued; ++i) tc::wait_warp(&full[i % kStages], (i / kStages) & 1, &never);
  }

  // ---------------------------------------------------------------- merge of the warps
  __syncthreads();                    // the ring is free
  if (*abort_flag) {
    if (threadIdx.x == 0) report_status(a.status, kStatusTimeout);
    return;
  }
  float* mo = reinterpret_cast<float*>(smem);                 // [warp][16][D + 4]: a row's output, then (m, l, mv)
  constexpr int LD = D + 4;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    l[u] = quad_sum(l[u]);
    float* row = mo + (warp * 16 + g4 + 8 * u) * LD;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      // n index 2 cq and 2 cq + 1 of n-tile j: channel j of their groups
      const int grp0 = D == 128 ? cq : 2 * cq, grp1 = D == 128 ? cq + 4 : 2 * cq + 1;
      row[(D / 8) * grp0 + j] = acc[j][2 * u];
      row[(D / 8) * grp1 + j] = acc[j][2 * u + 1];
    }
    if (cq == 0) {
      row[D] = m[u];
      row[D + 1] = l[u];
      row[D + 2] = mv[u];
    }
  }
  __syncthreads();
  // 8 threads a row
  const int r = threadIdx.x / 8, part8 = threadIdx.x % 8;
  if (r0 + r >= rows) return;
  float M = -INFINITY, MV = -INFINITY;
#pragma unroll
  for (int u = 0; u < kWarps; ++u) {
    M = fmaxf(M, mo[(u * 16 + r) * LD + D]);
    MV = fmaxf(MV, mo[(u * 16 + r) * LD + D + 2]);
  }
  const float Mr = finite_or_0(M), MVr = finite_or_0(MV);
  float L = 0.f, fac[kWarps];
#pragma unroll
  for (int u = 0; u < kWarps; ++u) {
    L += mo[(u * 16 + r) * LD + D + 1] * tc::ex2(mo[(u * 16 + r) * LD + D] - Mr);
    fac[u] = tc::ex2(mo[(u * 16 + r) * LD + D + 2] - MVr);
  }
  const float fin = L > 0.f ? tc::ex2(MVr - Mr) / L : (L == 0.f ? 0.f : L);
  const size_t prow = part * a.rows_pad + r0 + r;
  if ((!whole || a.scores != nullptr) && part8 == 0) *reinterpret_cast<float4*>(a.part_ml + prow * 4) = make_float4(M, L, MV, 0.f);
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {  // 4 channels at a time, 8 threads side by side
    const int ch = 32 * e + 4 * part8;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < kWarps; ++u) {
      const float4 y = *reinterpret_cast<const float4*>(mo + (u * 16 + r) * LD + ch);
      x.x = fmaf(y.x, fac[u], x.x);
      x.y = fmaf(y.y, fac[u], x.y);
      x.z = fmaf(y.z, fac[u], x.z);
      x.w = fmaf(y.w, fac[u], x.w);
    }
    if (whole) {
      const int rr = r0 + r;
      uint16_t* dst = a.o + static_cast<size_t>(nr.row0 + rr / g) * c.ld_o + (hk * g + rr % g) * D + ch;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(x.x * fin, x.y * fin), pack_bf16(x.z * fin, x.w * fin));
    } else {
      *reinterpret_cast<float4*>(a.part_o + prow * D + ch) = x;
    }
  }
}

// ---------------------------------------------------------------------------
// second kernel: the pieces' outputs joined, and the weights. CTAs
// [0, n_join) join 8 rows each (a warp per row); the others take kSpan tokens
// of one sequence and key head.
// ---------------------------------------------------------------------------

constexpr int kJoinThreads = 256;
constexpr int kSpan = 1024;
constexpr int kMaxRowsHeld = 1024;

template <int D>
__global__ void __launch_bounds__(kJoinThreads)
cache_join_kernel(Cache c, Args a, int n_join, int row_groups, int spans, const float* w_in, float* w_out) {
  __shared__ float lse2[kMaxRowsHeld];
  const int g = c.H / c.H_kv;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  bool bad = false;
  if (static_cast<int>(blockIdx.x) < n_join) {
    const int rg = blockIdx.x % row_groups, hk = (blockIdx.x / row_groups) % c.H_kv, b = blockIdx.x / (row_groups * c.H_kv);
    const NewRows nr = new_rows(c, a.seq, a.lens, b, bad);
    const int r = rg * 8 + warp;
    if (r >= nr.n * g) return;
    const size_t part0 = (static_cast<size_t>(b) * c.H_kv + hk) * a.n_split;
    float M = -INFINITY, MV = -INFINITY;
    for (int s = lane; s < a.n_split; s += 32) {
      const float4 x = *reinterpret_cast<const float4*>(a.part_ml + ((part0 + s) * a.rows_pad + r) * 4);
      M = fmaxf(M, x.x);
      MV = fmaxf(MV, x.z);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      MV = fmaxf(MV, __shfl_xor_sync(0xffffffffu, MV, o));
    }
    const float Mr = finite_or_0(M), MVr = finite_or_0(MV);
    float L = 0.f, x[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) x[e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.n_split; ++s) {
      const float4 st = *reinterpret_cast<const float4*>(a.part_ml + ((part0 + s) * a.rows_pad + r) * 4);
      if (st.x == -INFINITY) continue;  // an empty piece wrote no output
      L = fmaf(st.y, tc::ex2(st.x - Mr), L);
      const float f = tc::ex2(st.z - MVr);
      const float* po = a.part_o + ((part0 + s) * a.rows_pad + r) * D;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) x[e] = fmaf(po[lane * (D / 32) + e], f, x[e]);
    }
    const float fin = L > 0.f ? tc::ex2(MVr - Mr) / L : (L == 0.f ? 0.f : L);
    uint16_t* dst = a.o + static_cast<size_t>(nr.row0 + r / g) * c.ld_o + (hk * g + r % g) * D + lane * (D / 32);
    if constexpr (D == 128) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(x[0] * fin, x[1] * fin), pack_bf16(x[2] * fin, x[3] * fin));
    else *reinterpret_cast<uint32_t*>(dst) = pack_bf16(x[0] * fin, x[1] * fin);
    return;
  }
  const int id = blockIdx.x - n_join;
  const int sp = id / (c.B * c.H_kv), hk = id % c.H_kv, b = (id / c.H_kv) % c.B;
  const NewRows nr = new_rows(c, a.seq, a.lens, b, bad);
  const int rows = nr.n * g;
  const int tok0 = sp * kSpan, tok1 = min(tok0 + kSpan, nr.len);
  if (tok0 >= tok1) return;
  const size_t part0 = (static_cast<size_t>(b) * c.H_kv + hk) * a.n_split;
  const float* sc = a.scores + (static_cast<size_t>(b) * c.H_kv + hk) * c.max_blocks * c.block * a.rows_pad;
  float sum[kSpan / kJoinThreads];
#pragma unroll
  for (int e = 0; e < kSpan / kJoinThreads; ++e) sum[e] = 0.f;
  for (int base = 0; base < rows; base += kMaxRowsHeld) {
    const int n = min(kMaxRowsHeld, rows - base);
    if (base > 0) __syncthreads();
    for (int r = warp; r < n; r += kJoinThreads / 32) {  // log2 of the row's sum over all pieces
      float M = -INFINITY, L = 0.f;
      for (int s = lane; s < a.n_split; s += 32) {
        const float4 x = *reinterpret_cast<const float4*>(a.part_ml + ((part0 + s) * a.rows_pad + base + r) * 4);
        const float Mn = fmaxf(M, x.x);
        if (Mn != -INFINITY) L = L * tc::ex2(M - Mn) + x.y * tc::ex2(x.x - Mn);
        M = Mn;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float M2 = __shfl_xor_sync(0xffffffffu, M, o), L2 = __shfl_xor_sync(0xffffffffu, L, o);
        const float Mn = fmaxf(M, M2);
        if (Mn != -INFINITY) L = L * tc::ex2(M - Mn) + L2 * tc::ex2(M2 - Mn);
        M = Mn;
      }
      if (lane == 0) lse2[r] = M == -INFINITY ? INFINITY : M + log2f(L);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kSpan / kJoinThreads; ++e) {
      const int tok = tok0 + e * kJoinThreads + threadIdx.x;
      if (tok >= tok1) continue;
      const float* row = sc + static_cast<size_t>(tok) * a.rows_pad + base;
      for (int r = 0; r < n; ++r) {
        // rows that end before this token left no score behind
        if (tok < min(nr.len, nr.first + (base + r) / g + 1)) sum[e] += tc::ex2(row[r] - lse2[r]);
      }
    }
  }
  const int shift = 31 - __clz(c.block);
#pragma unroll
  for (int e = 0; e < kSpan / kJoinThreads; ++e) {
    const int tok = tok0 + e * kJoinThreads + threadIdx.x;
    if (tok >= tok1) continue;
    const int blk = __ldg(a.table + static_cast<size_t>(b) * c.max_blocks + (tok >> shift));
    if (blk < 0 || blk >= c.n_blocks) continue;
    const size_t at = (static_cast<size_t>(blk) * c.H_kv + hk) * c.block + (tok & (c.block - 1));
    w_out[at] = (w_in != nullptr ? w_in[at] : 0.f) + sum[e];
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

// The pool's codes as rows of d bytes; box = a tile's tokens of one block and head.
bool make_map(CUtensorMap* map, const void* base, const Cache& c) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.d), static_cast<cuuint64_t>(c.n_blocks) * c.H_kv * c.block};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.d)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(c.d), static_cast<cuuint32_t>(c.block < kTok ? c.block : kTok)};
  const cuuint32_t estr[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, c.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t run(const Cache& c, const Args& a, const uint8_t* k_codes, const uint8_t* v_codes, const float* w_in,
                float* w_out, cudaStream_t stream) {
  if (encode_fn() == nullptr) return cudaErrorNotSupported;
  CUtensorMap mk, mv;
  if (!make_map(&mk, k_codes, c) || !make_map(&mv, v_codes, c)) return cudaErrorInvalidValue;
  const int smem = Smem<D>::kTotal + 1024;
  cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long heads = static_cast<long long>(c.B) * c.H_kv;
  const long long blocks = heads * a.row_tiles * a.n_split;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  cache_attn_kernel<D><<<static_cast<unsigned>(blocks), kThreads, smem, stream>>>(mk, mv, c, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || (a.n_split == 1 && a.scores == nullptr)) return e;
  const int row_groups = a.rows_pad / 8 + (a.rows_pad % 8 != 0);
  const long long n_join = a.n_split > 1 ? heads * row_groups : 0;
  const int spans = a.scores == nullptr ? 0 : (c.max_blocks * c.block + kSpan - 1) / kSpan;
  const long long all = n_join + heads * spans;
  if (all >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  cache_join_kernel<D><<<static_cast<unsigned>(all), kJoinThreads, 0, stream>>>(c, a, static_cast<int>(n_join), row_groups,
                                                                               spans, w_in, w_out);
  return cudaGetLastError();
}

}  // namespace

CacheLayout make_cache_layout(const Cache& c) {
  CacheLayout y{};
  const long long heads = static_cast<long long>(c.B) * c.H_kv;
  const int most = c.max_new < c.rows ? c.max_new : c.rows;  // rows of one sequence
  const int rows = (most > 0 ? most : 1) * (c.H / c.H_kv);
  y.row_tiles = (rows + 15) / 16;
  y.rows_pad = (rows + 3) / 4 * 4;
  // Pieces: one wave of resident CTAs where the batch leaves room for it, of 512 tokens at least;
  // for batches above half a wave pieces of 2048 tokens, so that sequences of unequal length spread;
  // one piece where there are many row tiles.
  const long long tokens = static_cast<long long>(c.max_blocks) * c.block;
  const long long slots = static_cast<long long>(kSms) * kCtasPerSm, base = heads * y.row_tiles;
  long long n = base * 2 <= slots ? slots / base : base >= 16 * slots ? 1 : (tokens + 2047) / 2048;
  const long long most_pieces = (tokens + 511) / 512;
  if (n > most_pieces) n = most_pieces;
  y.n_split = static_cast<int>(n < 1 ? 1 : n);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  size_t off = 256;
  const size_t slots_rows = static_cast<size_t>(heads) * y.n_split * y.rows_pad;
  y.part_o = off;   off = up(off + (y.n_split > 1 ? slots_rows * c.d * 4 : 0));
  y.part_ml = off;  off = up(off + (y.n_split > 1 || c.weights ? slots_rows * 16 : 0));
  y.scores = off;   off = up(off + (c.weights ? static_cast<size_t>(heads) * tokens * y.rows_pad * 4 : 0));
  y.total = off;
  return y;
}

cudaError_t launch_cache_attn(const Cache& c, const CacheLayout& y, void* ws, const uint16_t* q, const int32_t* seq,
                              const int32_t* lens, const int32_t* table, const uint8_t* k_codes,
                              const uint8_t* v_codes, const float* k_scale, const float* v_scale, const float* w_in,
                              float* w_out, uint16_t* o, cudaStream_t stream) {
  unsigned char* base = static_cast<unsigned char*>(ws);
  Args a{};
  a.q = q;
  a.seq = seq;
  a.lens = lens;
  a.table = table;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.o = o;
  a.part_o = reinterpret_cast<float*>(base + y.part_o);
  a.part_ml = reinterpret_cast<float*>(base + y.part_ml);
  a.scores = w_out != nullptr ? reinterpret_cast<float*>(base + y.scores) : nullptr;
  a.status = reinterpret_cast<unsigned*>(base);
  a.n_split = y.n_split;
  a.row_tiles = y.row_tiles;
  a.rows_pad = y.rows_pad;
  a.wait_ns = attention_wait_limit();
  if (c.d == 128) return run<128>(c, a, k_codes, v_codes, w_in, w_out, stream);
  if (c.d == 64) return run<64>(c, a, k_codes, v_codes, w_in, w_out, stream);
  return cudaErrorInvalidValue;
}

}  // namespace sda
