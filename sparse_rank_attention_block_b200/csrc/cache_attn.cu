// Attention over the 8-bit key/value cache, for the newest tokens of each
// sequence: made for a few of them. Any number is right, but every 16 query rows
// of a key head read and convert the cache anew (a chunk of 1,560 tokens over
// 32,768, 32 heads over 8: 4.4 ms, 186 TFLOP/s).
//
//   s_rj = scale * ks_j (q_r . kc_j),  o_r = sum_j p_rj vs_j vc_j,
//   p_rj = exp(s_rj) / sum_j' exp(s_rj')
// with kc, vc the E4M3 codes and ks, vs the scales of token j's block. The rows
// r of a key head are its new tokens times its query heads, 8 or 16 to a tile.
//
// Bound by memory: 2 d bytes of cache for each token and key head against
// 4 d flops for each of its rows. So codes are read once for a tile of rows,
// converted to fp16 in registers (exact) and multiplied by mma.sync
// m16n8k16, with the tokens (S^T = K Q^T) and the channels (O^T = V^T P^T) as
// its 16 rows and the few query rows as its 8 columns: nothing is padded, and
// the output takes d / 4 registers for 8 query rows.
//
// Work is split over the tokens of all sequences as one line: sequence by
// sequence, in it unit by unit (key heads times row tiles), in that the 32-token
// tiles in order. Every CTA of the one wave of resident CTAs takes an equal
// stretch of that line, whatever the sequences' lengths. In a unit its warps
// take the tiles in turn, each with its own ring of TMA loads and its own running
// maximum, sum and output (no barrier between warps), merged where the unit or
// the stretch ends. Where a stretch holds all tiles of a unit the CTA writes the
// output; where it holds a part, a partial sum, which a second kernel joins in
// the order of the line. A third turns the scores of the first into the tokens'
// weights (a probability needs the sum over all tokens). Where no
// sequence can have more than kWholeTiles tiles, a CTA takes one whole unit.
//
// Scales differ from block to block. K's multiplies the scores. V's goes into
// the exponent: with lv = log2 vs, the operand of P V is 2^(s + lv - mv) with
// mv a running maximum of s + lv, while the sum takes 2^(s - m).
//
// That operand is fp16, the MMA's type with the most digits that E4M3 converts
// to exactly. Taken 2^7 up it has full precision down to 2^-21 of the maximum.
// Smaller terms decide an output whose largest term has a V near zero (a token
// that draws attention and holds nothing, a block scaled for another channel),
// so a tile that holds some takes P V in up to three passes over 2^28 each: the
// precision is 2^-11 of every term down to 2^-77 of the maximum, and what is
// below 2^-88 counts as zero. The passes cost such a tile its conversions and
// MMAs again (131,072 tokens, 4 rows to a key head, every tile of this kind: 69
// against 62.5 us); elsewhere they are a test of the least operand and code to
// fetch (one sequence of 300 tokens 6.2 against 5.5 us, 16 sequences of 1 to 4
// new tokens 33.6 against 32.9 us, long ones within the noise).
// The first pass stands apart from the rare ones: in one loop with them it costs
// the loads their head start (131,072 tokens 54.4 against 52.1 us).
//
// The order of channels and tokens inside an MMA is free (sums), so it is
// chosen for the loads: a lane reads 16 contiguous bytes of a token at a time
// and 8 lanes hit 8 different 16-byte bank groups of the swizzled tile.
//
// References move, and the output is rescaled, only when a maximum grows by
// more than 2^8 (exact: every term shares the reference).
//
// Measured (32 heads over 8, d = 128): one sequence of 131,072 tokens 52 us
// (5.2 TB/s; 41 us at the measured copy rate), 64 sequences of 500 to 16,000
// tokens with weights 137 us (97 us), of which the first kernel takes 115, the
// join 6, the weights 16. Two CTAs of three stages an SM against three of two:
// 52.6 and 54.3 us (long), 33.0 and 37.9 us (16 sequences, 1 to 4 new tokens).
//
// Tokens that a row must not see get a score of -inf; V codes of tokens behind
// the sequence (free slots, holding anything) are cleared before use.

#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "e4m3.cuh"
#include "launch.cuh"
#include "serving.h"
#include "serving_tc.cuh"

namespace sda {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTok = 32;       // tokens of a tile
constexpr int kStages = 3;     // tiles in flight per warp
constexpr int kCtasPerSm = 2;
constexpr int kSms = 148;
constexpr int kLeast = 8;      // places of a stretch, at least
// What a unit costs before its first tile (block numbers, scales, Q, the merge at its end: each a chain of
// reads), in tiles: places without a tile at its start. 16 sequences of 33 to 6,000 tokens, 1 to 4 new ones each:
// 40.9, 37.9, 36.6 and 41.0 us with 4, 8, 16 and 32; 64 sequences of 500 to 16,000: 139.9, 137.7, 140.0, 141.9 us.
constexpr int kLead = 8;
constexpr int kWholeTiles = 16;
constexpr int kMaxSeq = 65536;
// fp16 operands of P: 2^kUp times their value, at most 2^15 (a reference may lag by 2^8), in full precision from
// kLeastP on; two further passes, 2^kBand each, below that. The outputs then stay below 2^(15 + 9 + 24 + 56).
constexpr int kUp = 7, kBand = 28;
constexpr float kLeastP = 0x1p-14f;
// 2^(s - m) is zero below 2^-126: no loss where P is at most 2^kFarUp times it, and the least that counts 2^-81.
constexpr float kFarUp = 40.f;

template <int D>
struct Smem {
  static constexpr int kHalf = kTok * D;           // K or V codes of a tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kMerge = kWarps * 16 * (D + 4) * 4;  // at a unit's end, over the ring: outputs and (m, l, mv)
  static constexpr int kBars = kRing > kMerge ? kRing : kMerge;
  static constexpr int kTotal = kBars + 8 * kWarps * kStages + 16;
  static_assert(kBars >= kMaxSeq / 32 * 4, "the sums over 32 sequences each fit into the ring before its first load");
};

struct Args {
  const uint16_t* q;
  const int32_t* seq;
  const int32_t* lens;
  const int32_t* table;
  const float* k_scale;
  const float* v_scale;
  uint16_t* o;
  float* part_o;       // [2 * workers, tile_rows, d]: partial outputs
  float4* part_ml;     // [2 * workers, tile_rows]: their m, l, mv
  int* line;           // [B + 1]: where each sequence begins on the line; the last: its length
  float* lse2;         // [rows, H], log2 of the sum: rows that one stretch holds whole (weights kept)
  float* scores;       // [B, H_kv, tokens, rows_pad], log2 units; NULL: weights are not kept
  unsigned* status;
  int workers, tile_rows, rows_pad;
  int whole_row_tiles;  // > 0: CTA i takes unit i, sequences having that many row tiles of room; no line
  uint64_t wait_ns;
};

// Places of a CTA's stretch of a line of W: CTA i takes [i S, (i + 1) S).
__device__ __forceinline__ int stretch_size(int W, int workers) { return max(kLeast, (W + workers - 1) / workers); }

// Sequence b on the line: units (row tiles x key heads) of kLead + n_tiles places each. A sequence with rows
// has one tile at least, so that its rows are written. (The host has checked that the line fits an int.)
struct SeqLine {
  NewRows nr;
  int rows, row_tiles, n_tiles;
  __device__ __forceinline__ int places(const Cache& c) const { return c.H_kv * row_tiles * (kLead + n_tiles); }
};
__device__ __forceinline__ SeqLine seq_line(const Cache& c, const Args& a, int b, bool& bad) {
  SeqLine s;
  s.nr = new_rows(c, a.seq, a.lens, b, bad);
  s.rows = s.nr.n * c.g;
  s.row_tiles = (s.rows + a.tile_rows - 1) >> (a.tile_rows == 8 ? 3 : 4);  // 8 or 16
  s.n_tiles = max(1, (s.nr.len + kTok - 1) / kTok);
  return s;
}

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
// Over the 8 lanes that share lane % 4: the tokens of a column of S^T.
__device__ __forceinline__ float column_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float column_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}
// Transpose of an 8 x 8 matrix of 16-bit values held as an MMA fragment.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ constexpr float exp2_of(int e) {  // -126 <= e <= 127
  return __builtin_bit_cast(float, static_cast<uint32_t>(e + 127) << 23);
}
__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.f : m; }

// 16-byte chunk `ch` of token row `row` in a swizzled tile of D-byte rows.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int row, int ch) {
  if constexpr (D == 128) return row * 128 + ((ch ^ (row & 7)) << 4);
  else return row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
}

// NR: groups of 8 query rows. HALVES: a tile's two 16-token halves may lie in different blocks (block = 16).
template <int D, int NR, bool HALVES>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
cache_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, Cache c, Args a) {
  using S = Smem<D>;
  constexpr int KS = D / 16;     // k16 steps of a score
  constexpr int MT = D / 16;     // 16-channel tiles of the output
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + kWarps * kStages);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g4 = lane >> 2, cq = lane & 3;
  const int g = c.g;

  if (threadIdx.x < kWarps * kStages) tc::mbar_init(&bars[threadIdx.x], 1);
  if (threadIdx.x == 0) *abort_flag = 0;
  tc::fence_mbar_init();
  pdl_wait();

  // ------------------------------------------------------------ this CTA's stretch of the line
  bool bad = false;
  int b = 0, unit = 0, tile = 0;
  int pos = 0, end = 0;  // places on the line: of the next tile, and of the stretch's end
  SeqLine sl;
  if (a.whole_row_tiles > 0) {
    const int per_seq = c.H_kv * a.whole_row_tiles, u = blockIdx.x % per_seq;
    b = blockIdx.x / per_seq;
    sl = seq_line(c, a, b, bad);
    if (bad && threadIdx.x == 0 && u == 0) report_status(a.status, kStatusBadIndex);
    unit = u / a.whole_row_tiles * sl.row_tiles + u % a.whole_row_tiles;
    end = u % a.whole_row_tiles < sl.row_tiles ? sl.n_tiles : 0;
    __syncthreads();
  } else {
    int* sums = reinterpret_cast<int*>(smem);  // places of 32 sequences each (the ring is not in use yet)
    const int groups = (c.B + 31) / 32;
    for (int u = warp; u < groups; u += kWarps) {
      const int i = 32 * u + lane;
      const int n = __reduce_add_sync(0xffffffffu, i < c.B ? seq_line(c, a, i, bad).places(c) : 0);
      if (lane == 0) sums[u] = n;
    }
    if (blockIdx.x == 0 && bad) report_status(a.status, kStatusBadIndex);
    __syncthreads();
    int W = 0;
    for (int u = lane; u < groups; u += 32) W += sums[u];
    W = __reduce_add_sync(0xffffffffu, W);
    const int S_ = stretch_size(W, a.workers);
    pos = min(static_cast<long long>(blockIdx.x) * S_, static_cast<long long>(W));
    end = min(static_cast<long long>(pos) + S_, static_cast<long long>(W));
    // the group of sequences that holds pos, then the sequence: `before` is where it begins
    int before = 0;
    auto find = [&](int n) {  // lane that holds pos among the lanes' n places each, -1: behind them
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      const uint32_t at = __ballot_sync(0xffffffffu, pos >= before + incl - n && pos < before + incl);
      const int found = __ffs(at) - 1;
      before += found >= 0 ? __shfl_sync(0xffffffffu, incl - n, found) : __shfl_sync(0xffffffffu, incl, 31);
      return found;
    };
    int group = 0;
    for (int base = 0; base < groups; base += 32) {
      const int at = find(base + lane < groups ? sums[base + lane] : 0);
      if (at >= 0) {
        group = base + at;
        break;
      }
    }
    const int at = find(32 * group + lane < c.B ? seq_line(c, a, 32 * group + lane, bad).places(c) : 0);
    if (at >= 0) b = 32 * group + at;
    if (blockIdx.x == 0) {  // the line for the second kernel
      int start = 0;
      for (int u = 0; u < groups; ++u) {
        if (u % kWarps == warp) {
          const int n = 32 * u + lane < c.B ? seq_line(c, a, 32 * u + lane, bad).places(c) : 0;
          int incl = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
          }
          if (32 * u + lane < c.B) a.line[32 * u + lane] = start + incl - n;
        }
        start += sums[u];
      }
      if (threadIdx.x == 0) a.line[c.B] = W;
    }
    tc::fence_proxy_async_smem();
    __syncthreads();  // the sums have been read: the ring may be filled
    sl = seq_line(c, a, b, bad);
    if (pos < end) {
      unit = (pos - before) / (kLead + sl.n_tiles);
      tile = (pos - before) % (kLead + sl.n_tiles) - kLead;
      if (tile < 0) {     // on the places before the unit's first tile
        pos -= tile;
        tile = 0;
      }
    }
  }
  pdl_launch();

  // codes are read once (and again by a unit's other row tiles, soon after): L2 is for the scores
  const uint64_t once = tc::l2_evict_first();
  const int shift = 31 - __clz(c.block);
  unsigned char* ring = smem + warp * kStages * S::kStage;
  uint64_t* full = bars + warp * kStages;
  int done = 0;       // tiles of this warp so far: their places in the ring go on from segment to segment
  bool ok = true;

  while (pos < end) {
    // ---------------------------------------------------------- a segment: tiles [tile, tile + seg_all) of one unit
    const int hk = unit / sl.row_tiles, r0 = 8 * NR * (unit % sl.row_tiles);
    const int seg_all = min(sl.n_tiles - tile, end - pos);
    // this warp's tiles: tile0 + kWarps i, i < seg
    const int tile0 = tile + warp, seg = seg_all > warp ? (seg_all - warp + kWarps - 1) / kWarps : 0;
    // tokens that the tile's last row sees
    const int seen = min(sl.nr.len, max(0, sl.nr.first + min(r0 + 8 * NR - 1, sl.rows - 1) / g + 1));
    const int32_t* blocks = a.table + static_cast<size_t>(b) * c.max_blocks;

    // This segment's blocks and scales, a batch of 16 tiles per register: lane l holds half l % 2 of tile
    // base + l / 2. The next batch is read a batch ahead of its use.
    struct Held {
      int blk;
      float ks, vs;
    };
    auto hold = [&](int base) {
      Held x{-1, 0.f, 0.f};
      const int i = base + lane / 2, tok = (tile0 + kWarps * i) * kTok + 16 * (lane & 1);
      if (i < seg && tok < seen) {
        x.blk = __ldg(blocks + (tok >> shift));
        if (x.blk < 0 || x.blk >= c.n_blocks) {
          report_status(a.status, kStatusBadIndex);
          x.blk = -1;
        } else {
          const size_t head = static_cast<size_t>(x.blk) * c.H_kv + hk;
          x.ks = __ldg(a.k_scale + head);
          x.vs = __ldg(a.v_scale + head);
        }
      }
      return x;
    };
    // one lane: the loads of the segment's tile i (absent blocks: nothing, their tokens are not seen)
    auto load_tile = [&](int i, int blk0, int blk1) {
      const int st = (done + i) % kStages;
      const int tok = (tile0 + kWarps * i) * kTok;
      unsigned char* dst = ring + st * S::kStage;
      if constexpr (!HALVES) {
        tc::mbar_arrive_expect_tx(&full[st], blk0 >= 0 ? S::kStage : 0);
        if (blk0 >= 0) {
          const int y = (blk0 * c.H_kv + hk) * c.block + (tok & (c.block - 1));
          tc::tma_load_2d(dst, &tm_k, &full[st], 0, y, once);
          tc::tma_load_2d(dst + S::kHalf, &tm_v, &full[st], 0, y, once);
        }
      } else {
        tc::mbar_arrive_expect_tx(&full[st], (blk0 >= 0 ? S::kHalf : 0) + (blk1 >= 0 ? S::kHalf : 0));
        for (int u = 0; u < 2; ++u) {
          const int blk = u ? blk1 : blk0;
          if (blk < 0) continue;
          const int y = (blk * c.H_kv + hk) * c.block;
          tc::tma_load_2d(dst + u * 16 * D, &tm_k, &full[st], 0, y, once);
          tc::tma_load_2d(dst + S::kHalf + u * 16 * D, &tm_v, &full[st], 0, y, once);
        }
      }
    };
    Held now = hold(0);
    int issued = 0;
    for (; issued < kStages && issued < seg; ++issued) {
      const int b0 = __shfl_sync(0xffffffffu, now.blk, 2 * issued), b1 = __shfl_sync(0xffffffffu, now.blk, 2 * issued + 1);
      if (lane == 0) load_tile(issued, b0, b1);
    }
    Held next = hold(16);

    // Q fragments in fp16: row r times 2^(14 - e), e its exponent, undone in the score's factor
    uint32_t qf[NR][KS][2];
    float factor[NR][2];              // of this lane's columns: rows 2 cq and 2 cq + 1 of each group of 8
    int lim[NR][2];                   // tokens that they see
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      const int r = r0 + 8 * nr + g4;
      const bool there = r < sl.rows;
      const int i = there ? r / g : 0, qh = there ? r % g : 0;
      const int my_lim = there ? min(sl.nr.len, max(0, sl.nr.first + i + 1)) : seen;  // rows not there: computed, not kept
      const uint16_t* src = a.q + static_cast<size_t>(sl.nr.row0 + i) * c.ld_q + (hk * g + qh) * D;
      uint4 x[D / 32];                // this lane's channels: 16 at 16 cq (and 16 at 64 + 16 cq)
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
      const float my_factor = __uint_as_float(static_cast<uint32_t>(e2 - 14 + 127) << 23) * c.scale_log2;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        const uint32_t in[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
        for (int f = 0; f < 4; ++f)   // channels 8 e' + 2 f, + 1 of the lane's 16
          qf[nr][4 * (e / 2) + 2 * (e % 2) + f / 2][f % 2] = pack_f16(bf16_lo(in[f]) * up, bf16_hi(in[f]) * up);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        factor[nr][u] = __shfl_sync(0xffffffffu, my_factor, 4 * (2 * cq + u));
        lim[nr][u] = __shfl_sync(0xffffffffu, my_lim, 4 * (2 * cq + u));
      }
    }
    int lim_least = lim[0][0];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) lim_least = min(lim_least, min(lim[nr][0], lim[nr][1]));

    float acc[NR][MT][4];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nr][j][e] = 0.f;
    float m[NR][2], mv[NR][2], l[NR][2];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        m[nr][u] = mv[nr][u] = -INFINITY;
        l[nr][u] = 0.f;
      }
    float* my_scores = a.scores == nullptr ? nullptr
                                           : a.scores +
                                                 (static_cast<size_t>(b) * c.H_kv + hk) * c.max_blocks * c.block * a.rows_pad +
                                                 r0 + 2 * cq;
    // the MMA's row i stands for token (D == 128: spread(i)) of each 8
    const int row_k = D == 128 ? spread(g4) : g4;
    const int t_lo = D == 128 ? cq : 2 * cq, t_hi = D == 128 ? cq + 4 : 2 * cq + 1;  // the tokens of MMA rows 2 cq, 2 cq + 1

    for (int i = 0; i < seg; ++i) {
      const int st = (done + i) % kStages;
      const int tok0 = (tile0 + kWarps * i) * kTok;
      if (i % 16 == 0 && i > 0) {
        now = next;
        next = hold(i + 16);
      }
      int blk[2];
      float ks[2], lv[2];             // lv = log2 of V's scale
#pragma unroll
      for (int hf = 0; hf < (HALVES ? 2 : 1); ++hf) {
        const int from = 2 * (i % 16) + hf;
        blk[hf] = __shfl_sync(0xffffffffu, now.blk, from);
        ks[hf] = __shfl_sync(0xffffffffu, now.ks, from);
        lv[hf] = __log2f(__shfl_sync(0xffffffffu, now.vs, from));
      }
      if constexpr (!HALVES) {
        blk[1] = blk[0];
        ks[1] = ks[0];
        lv[1] = lv[0];
      }
      ok = tc::wait_warp(&full[st], ((done + i) / kStages) & 1, abort_flag, a.wait_ns);
      if (!ok) break;                 // the load stays counted as issued
      if (i % 16 == 0 && !(is_scale(now.ks) && is_scale(now.vs))) report_status(a.status, kStatusBadIndex);
      const unsigned char* kt = ring + st * S::kStage;
      const unsigned char* vt = kt + S::kHalf;

      // S^T of the 32 tokens: s[hf]: tokens 16 hf + row_k (e < 2) and 16 hf + 8 + row_k, columns 2 cq + e % 2
      float s[NR][2][4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) s[nr][hf][0] = s[nr][hf][1] = s[nr][hf][2] = s[nr][hf][3] = 0.f;
#pragma unroll
        for (int half = 0; half < KS / 4; ++half) {
          const uint4 x = *reinterpret_cast<const uint4*>(kt + chunk_at<D>(16 * hf + row_k, cq + 4 * half));
          const uint4 y = *reinterpret_cast<const uint4*>(kt + chunk_at<D>(16 * hf + 8 + row_k, cq + 4 * half));
          const uint32_t in_x[4] = {x.x, x.y, x.z, x.w}, in_y[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t kf[4] = {e4m3x2_to_f16x2(static_cast<uint16_t>(in_x[e])),
                                    e4m3x2_to_f16x2(static_cast<uint16_t>(in_y[e])),
                                    e4m3x2_to_f16x2(static_cast<uint16_t>(in_x[e] >> 16)),
                                    e4m3x2_to_f16x2(static_cast<uint16_t>(in_y[e] >> 16))};
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) mma_f16(s[nr][hf], kf, qf[nr][4 * half + e][0], qf[nr][4 * half + e][1]);
          }
        }
      }
      const bool edge = tok0 + kTok > lim_least || blk[0] < 0 || blk[1] < 0;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float f0 = factor[nr][u] * ks[0], f1 = factor[nr][u] * ks[1];
          s[nr][0][u] *= f0;
          s[nr][0][2 + u] *= f0;
          s[nr][1][u] *= f1;
          s[nr][1][2 + u] *= f1;
        }
      if (__any_sync(0xffffffffu, edge)) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (tok0 + 16 * hf + 8 * (e / 2) + row_k >= lim[nr][e % 2] || blk[hf] < 0) s[nr][hf][e] = -INFINITY;
      }
      if (my_scores != nullptr) {     // two rows at a time; the second may be a free slot
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
          if (r0 + 8 * nr + 2 * cq < sl.rows) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int tok = tok0 + 16 * hf + 8 * e + row_k;
                if (tok < seen)
                  *reinterpret_cast<float2*>(my_scores + static_cast<size_t>(tok) * a.rows_pad + 8 * nr) =
                      make_float2(s[nr][hf][2 * e], s[nr][hf][2 * e + 1]);
              }
          }
      }
      float top[NR][2], top_v[NR][2];
      bool grow = false;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if constexpr (HALVES) {
            const float ma = column_max(fmaxf(s[nr][0][u], s[nr][0][2 + u]));
            const float mb = column_max(fmaxf(s[nr][1][u], s[nr][1][2 + u]));
            top[nr][u] = fmaxf(ma, mb);
            top_v[nr][u] = fmaxf(ma + lv[0], mb + lv[1]);
          } else {
            top[nr][u] = column_max(fmaxf(fmaxf(s[nr][0][u], s[nr][0][2 + u]), fmaxf(s[nr][1][u], s[nr][1][2 + u])));
            top_v[nr][u] = top[nr][u] + lv[0];
          }
          grow = grow || top[nr][u] > m[nr][u] + 8.f || top_v[nr][u] > mv[nr][u] + 8.f;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float m_new = fmaxf(m[nr][u], top[nr][u]), mv_new = fmaxf(mv[nr][u], top_v[nr][u]);
            l[nr][u] *= tc::ex2(m[nr][u] - finite_or_0(m_new));
            const float alpha = tc::ex2(mv[nr][u] - finite_or_0(mv_new));
            m[nr][u] = m_new;
            mv[nr][u] = mv_new;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              acc[nr][j][u] *= alpha;
              acc[nr][j][2 + u] *= alpha;
            }
          }
      }
      float p[NR][2][4];              // 2^(s + lv - mv + kUp)
      uint32_t pf[NR][2][2];          // P^T fragments of the two 16-token steps
      bool small = false;             // some p below kLeastP, but not zero
      bool far = false;               // some p too far above its 2^(s - m)
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float mr = finite_or_0(m[nr][u]), mvr = finite_or_0(mv[nr][u]);
          // 2^(s + lv - mv) = 2^(s - m) 2^(m + lv - mv)
          const float up_a = mr + lv[0] - mvr + kUp, up_b = mr + lv[HALVES ? 1 : 0] - mvr + kUp;
          const float fa = tc::ex2(up_a), fb = HALVES ? tc::ex2(up_b) : fa;
          far = far || fmaxf(up_a, up_b) > kFarUp;
          const float a0 = tc::ex2(s[nr][0][u] - mr), a1 = tc::ex2(s[nr][0][2 + u] - mr);
          const float b0 = tc::ex2(s[nr][1][u] - mr), b1 = tc::ex2(s[nr][1][2 + u] - mr);
          l[nr][u] += (a0 + a1) + (b0 + b1);
          p[nr][0][u] = a0 * fa;
          p[nr][0][2 + u] = a1 * fa;
          p[nr][1][u] = b0 * fb;
          p[nr][1][2 + u] = b1 * fb;
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          pf[nr][hf][0] = pack_f16(p[nr][hf][0], p[nr][hf][1]);
          pf[nr][hf][1] = pack_f16(p[nr][hf][2], p[nr][hf][3]);
        }
        uint32_t least = ~0u;         // of the bits less one: what is zero (a token not seen) comes last
#pragma unroll
        for (int e = 0; e < 8; ++e) least = min(least, __float_as_uint(p[nr][e / 4][e % 4]) - 1u);
        small = small || far || least < __float_as_uint(kLeastP) - 1u;
      }
      // Terms that fp16 does not hold in full are left to further passes, each 2^kBand up (exactly, the output so far
      // with them): a dominant token whose V is small leaves the output to them.
      auto take = [&](float least) {  // operands: what is not below `least`; the rest stays in p, 2^kBand up
        bool rest = false;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool now = !(p[nr][hf][e] < least);  // a NaN is taken, too
              x[e] = now ? p[nr][hf][e] : 0.f;
              p[nr][hf][e] = now ? 0.f : p[nr][hf][e] * exp2_of(kBand);
              rest = rest || p[nr][hf][e] > 0.f;
            }
            pf[nr][hf][0] = pack_f16(x[0], x[1]);
            pf[nr][hf][1] = pack_f16(x[2], x[3]);
          }
        return __any_sync(0xffffffffu, rest) != 0;
      };
      const bool clear = tok0 + kTok > seen || blk[0] < 0 || blk[1] < 0;  // V rows of no token of the sequence
      // O^T += V^T P^T: this lane's channels are those of group g4, two to an MMA; its tokens those of P
      auto add_pv = [&] {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            pf[nr][hf][0] = transpose8(pf[nr][hf][0]);
            pf[nr][hf][1] = transpose8(pf[nr][hf][1]);
          }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t w[4][D / 32];      // 4 tokens, d / 8 channels of the lane's group
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = 16 * hf + 8 * (e / 2) + (e % 2 ? t_hi : t_lo);
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
            if (clear && (tok0 + row >= seen || blk[hf] < 0)) {
#pragma unroll
              for (int f = 0; f < D / 32; ++f) w[e][f] = 0u;
            }
          }
#pragma unroll
          for (int f = 0; f < D / 32; ++f) {
            // channels 4 f .. 4 f + 3 of the group, tokens paired byte by byte
            const uint32_t a01 = __byte_perm(w[0][f], w[1][f], 0x5140), a23 = __byte_perm(w[0][f], w[1][f], 0x7362);
            const uint32_t b01 = __byte_perm(w[2][f], w[3][f], 0x5140), b23 = __byte_perm(w[2][f], w[3][f], 0x7362);
            const uint32_t v0[4] = {e4m3x2_to_f16x2(static_cast<uint16_t>(a01)), e4m3x2_to_f16x2(static_cast<uint16_t>(a01 >> 16)),
                                    e4m3x2_to_f16x2(static_cast<uint16_t>(b01)), e4m3x2_to_f16x2(static_cast<uint16_t>(b01 >> 16))};
            const uint32_t v1[4] = {e4m3x2_to_f16x2(static_cast<uint16_t>(a23)), e4m3x2_to_f16x2(static_cast<uint16_t>(a23 >> 16)),
                                    e4m3x2_to_f16x2(static_cast<uint16_t>(b23)), e4m3x2_to_f16x2(static_cast<uint16_t>(b23 >> 16))};
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
              mma_f16(acc[nr][2 * f], v0, pf[nr][hf][0], pf[nr][hf][1]);
              mma_f16(acc[nr][2 * f + 1], v1, pf[nr][hf][0], pf[nr][hf][1]);
            }
          }
        }
      };
      auto scale_acc = [&](float by) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nr][j][e] *= by;
      };
      bool bands = false;
      if (__any_sync(0xffffffffu, small)) {
        if (__any_sync(0xffffffffu, far)) {  // in one step: 2^(s - m) would be zero where its V's scale makes up for it
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                p[nr][hf][e] = tc::ex2(s[nr][hf][e] + (lv[hf] - finite_or_0(mv[nr][e % 2]) + kUp));
        }
        bands = take(kLeastP);
      }
      add_pv();
      if (bands) {
        scale_acc(exp2_of(kBand));
        if (take(kLeastP)) {
          add_pv();
          scale_acc(exp2_of(kBand));
          take(0.f);
          add_pv();
          scale_acc(exp2_of(-2 * kBand));
        } else {
          add_pv();
          scale_acc(exp2_of(-kBand));
        }
      }
      __syncwarp();                   // every lane has read the stage
      if (issued < seg) {
        const int from = issued / 16 == i / 16 ? now.blk : next.blk;
        const int b0 = __shfl_sync(0xffffffffu, from, 2 * (issued % 16)), b1 = __shfl_sync(0xffffffffu, from, 2 * (issued % 16) + 1);
        if (lane == 0) load_tile(issued, b0, b1);
        ++issued;
      }
    }
    if (!ok) {                        // given up: no load is in flight when the CTA ends
      volatile int never = 0;
      for (int i = max(0, issued - kStages); i < issued; ++i)
        tc::wait_warp(&full[(done + i) % kStages], ((done + i) / kStages) & 1, &never);
    }
    done += seg;

    // ---------------------------------------------------------- the warps' outputs merged
    constexpr int LD = D + 4, ROWS = 8 * NR;
    float* merge = reinterpret_cast<float*>(smem);              // [warp][ROWS][LD]: a row's output, then (m, l, mv)
    __syncthreads();                                            // the ring is free
    if (*abort_flag) break;                                     // uniform
    const int ch0 = D == 128 ? 16 * spread(g4) : 8 * g4;        // this lane's channels: d / 8 from here
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float L = column_sum(l[nr][u]);
        float* row = merge + (warp * ROWS + 8 * nr + 2 * cq + u) * LD;
#pragma unroll
        for (int j = 0; j < MT; j += 2)
          *reinterpret_cast<float4*>(row + ch0 + 2 * j) =
              make_float4(acc[nr][j][u], acc[nr][j][2 + u], acc[nr][j + 1][u], acc[nr][j + 1][2 + u]);
        if (g4 == 0) *reinterpret_cast<float4*>(row + D) = make_float4(m[nr][u], L, mv[nr][u], 0.f);
      }
    __syncthreads();
    {
      constexpr int PER = kThreads / ROWS;                      // threads of a row, 4 channels each at a time
      const int r = threadIdx.x / PER, t = threadIdx.x % PER, rr = r0 + r;
      if (rr < sl.rows) {
        float4 st[kWarps];
        float M = -INFINITY, MV = -INFINITY;
#pragma unroll
        for (int u = 0; u < kWarps; ++u) {
          st[u] = *reinterpret_cast<const float4*>(merge + (u * ROWS + r) * LD + D);
          M = fmaxf(M, st[u].x);
          MV = fmaxf(MV, st[u].z);
        }
        const float Mr = finite_or_0(M), MVr = finite_or_0(MV);
        float L = 0.f, f[kWarps];
#pragma unroll
        for (int u = 0; u < kWarps; ++u) {
          L = fmaf(st[u].y, tc::ex2(st[u].x - Mr), L);
          f[u] = tc::ex2(st[u].z - MVr) * exp2_of(-kUp);
        }
        const bool whole = tile == 0 && seg_all == sl.n_tiles;
        const int row = sl.nr.row0 + rr / g, head = hk * g + rr % g;
        const size_t slot = (2 * static_cast<size_t>(blockIdx.x) + (tile == 0 ? 1 : 0)) * ROWS + r;  // a unit's first part, or a later one
        const float fin = L > 0.f ? tc::ex2(MVr - Mr) / L : (L == 0.f ? 0.f : L);
        if (t == 0) {
          if (!whole) a.part_ml[slot] = make_float4(M, L, MV, 0.f);
          else if (a.scores != nullptr) a.lse2[static_cast<size_t>(row) * c.H + head] = M == -INFINITY ? INFINITY : M + log2f(L);
        }
#pragma unroll
        for (int ch = 4 * t; ch < D; ch += 4 * PER) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int u = 0; u < kWarps; ++u) {
            const float4 y = *reinterpret_cast<const float4*>(merge + (u * ROWS + r) * LD + ch);
            x.x = fmaf(y.x, f[u], x.x);
            x.y = fmaf(y.y, f[u], x.y);
            x.z = fmaf(y.z, f[u], x.z);
            x.w = fmaf(y.w, f[u], x.w);
          }
          if (whole)
            *reinterpret_cast<uint2*>(a.o + static_cast<size_t>(row) * c.ld_o + head * D + ch) =
                make_uint2(pack_bf16(x.x * fin, x.y * fin), pack_bf16(x.z * fin, x.w * fin));
          else
            *reinterpret_cast<float4*>(a.part_o + slot * D + ch) = x;
        }
      }
    }
    // ---------------------------------------------------------- the next unit
    pos += seg_all + kLead;
    tile = 0;
    if (pos < end) {
      tc::fence_proxy_async_smem();
      __syncthreads();                // the merge has been read: the ring may be filled
      if (++unit >= c.H_kv * sl.row_tiles) {
        unit = 0;
        do {
          sl = seq_line(c, a, ++b, bad);
        } while (sl.rows == 0);
      }
    }
  }
  if (*abort_flag && threadIdx.x == 0) report_status(a.status, kStatusTimeout);
}

// ---------------------------------------------------------------------------
// second kernel: the parts' outputs joined, and each row's sum. Bound by the
// latency of a few dependent reads.
// ---------------------------------------------------------------------------

constexpr int kJoinThreads = 256;
constexpr int kMaxParts = kSms * kCtasPerSm;

// The slots of a unit's parts: 2 first + 1, then 2 (first + 1), 2 (first + 2) .. 2 last.
struct Parts {
  int first, n;
  __device__ __forceinline__ size_t slot(int i) const { return 2 * static_cast<size_t>(first + i) + (i == 0 ? 1 : 0); }
};
// Of a unit that begins at place `start` of a line of stretches of `size` places.
__device__ __forceinline__ Parts parts_of(int start, int n_tiles, int size) {
  const int first = (start + kLead) / size;
  return Parts{first, (start + kLead + n_tiles - 1) / size - first + 1};
}

// WIDE: a CTA per row (many parts); otherwise a warp per row.
template <int D, bool WIDE>
__global__ void __launch_bounds__(kJoinThreads)
cache_join_kernel(Cache c, Args a) {
  constexpr int V = D / 32;      // channels of a lane
  constexpr int NW = kJoinThreads / 32;
  const int g = c.g;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  bool bad = false;
  pdl_wait();
  pdl_launch();
  const int size = stretch_size(a.line[c.B], a.workers);
  auto keep_sum = [&](const SeqLine& sl, int hk, int r, float M, float L) {
    if (a.scores != nullptr)
      a.lse2[static_cast<size_t>(sl.nr.row0 + r / g) * c.H + hk * g + r % g] = M == -INFINITY ? INFINITY : M + log2f(L);
  };
  if constexpr (!WIDE) {
    const int id = blockIdx.x * NW + warp;
    const int r = id % a.rows_pad, hk = (id / a.rows_pad) % c.H_kv, b = id / (a.rows_pad * c.H_kv);
    if (b >= c.B) return;
    const SeqLine sl = seq_line(c, a, b, bad);
    if (r >= sl.rows) return;
    const Parts ps =
        parts_of(a.line[b] + (hk * sl.row_tiles + r / a.tile_rows) * (kLead + sl.n_tiles), sl.n_tiles, size);
    const int n = ps.n, r_in = r % a.tile_rows;
    if (n == 1) return;          // written by the first kernel
    float M = -INFINITY, MV = -INFINITY, L = 0.f, x[V];
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const float4 st = i0 + lane < n ? a.part_ml[ps.slot(i0 + lane) * a.tile_rows + r_in]
                                      : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
      float Mn = st.x, MVn = st.z;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        Mn = fmaxf(Mn, __shfl_xor_sync(0xffffffffu, Mn, o));
        MVn = fmaxf(MVn, __shfl_xor_sync(0xffffffffu, MVn, o));
      }
      Mn = fmaxf(M, Mn);
      MVn = fmaxf(MV, MVn);
      const float Mr = finite_or_0(Mn), MVr = finite_or_0(MVn);
      L = L * tc::ex2(M - Mr) + warp_sum(st.y * tc::ex2(st.x - Mr));
      const float f0 = tc::ex2(MV - MVr), f = tc::ex2(st.z - MVr);
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] *= f0;
      M = Mn;
      MV = MVn;
      const int m = min(32, n - i0);
#pragma unroll 8
      for (int i = 0; i < m; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, i);
        const float* po = a.part_o + (ps.slot(i0 + i) * a.tile_rows + r_in) * D + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = fmaf(po[e], fi, x[e]);  // one 8- or 16-byte read
      }
    }
    const float fin = L > 0.f ? tc::ex2(finite_or_0(MV) - finite_or_0(M)) / L : (L == 0.f ? 0.f : L);
    uint16_t* dst = a.o + static_cast<size_t>(sl.nr.row0 + r / g) * c.ld_o + (hk * g + r % g) * D + lane * V;
    if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(x[0] * fin, x[1] * fin), pack_bf16(x[2] * fin, x[3] * fin));
    else *reinterpret_cast<uint32_t*>(dst) = pack_bf16(x[0] * fin, x[1] * fin);
    if (lane == 0) keep_sum(sl, hk, r, M, L);
  } else {
    __shared__ float held[kMaxParts];
    __shared__ float part[NW][D];
    __shared__ float red[3][NW];
    const int r = blockIdx.x % a.rows_pad, hk = (blockIdx.x / a.rows_pad) % c.H_kv, b = blockIdx.x / (a.rows_pad * c.H_kv);
    const SeqLine sl = seq_line(c, a, b, bad);
    if (r >= sl.rows) return;
    const Parts ps =
        parts_of(a.line[b] + (hk * sl.row_tiles + r / a.tile_rows) * (kLead + sl.n_tiles), sl.n_tiles, size);
    const int n = ps.n, r_in = r % a.tile_rows;
    if (n == 1) return;          // written by the first kernel
    float M = -INFINITY, MV = -INFINITY;
    for (int i = threadIdx.x; i < n; i += kJoinThreads) {
      const float4 st = a.part_ml[ps.slot(i) * a.tile_rows + r_in];
      M = fmaxf(M, st.x);
      MV = fmaxf(MV, st.z);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      MV = fmaxf(MV, __shfl_xor_sync(0xffffffffu, MV, o));
    }
    if (lane == 0) {
      red[0][warp] = M;
      red[1][warp] = MV;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NW; ++u) {
      M = fmaxf(M, red[0][u]);
      MV = fmaxf(MV, red[1][u]);
    }
    const float Mr = finite_or_0(M), MVr = finite_or_0(MV);
    float L = 0.f;
    for (int i = threadIdx.x; i < n; i += kJoinThreads) {
      const float4 st = a.part_ml[ps.slot(i) * a.tile_rows + r_in];
      L = fmaf(st.y, tc::ex2(st.x - Mr), L);
      held[i] = tc::ex2(st.z - MVr);
    }
    L = warp_sum(L);
    if (lane == 0) red[2][warp] = L;
    __syncthreads();
    float x[V];
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = 0.f;
#pragma unroll 8
    for (int i = warp; i < n; i += NW) {
      const float f = held[i];
      const float* po = a.part_o + (ps.slot(i) * a.tile_rows + r_in) * D + lane * V;
      if constexpr (V == 4) {
        const float4 y = *reinterpret_cast<const float4*>(po);
        x[0] = fmaf(y.x, f, x[0]);
        x[1] = fmaf(y.y, f, x[1]);
        x[2] = fmaf(y.z, f, x[2]);
        x[3] = fmaf(y.w, f, x[3]);
      } else {
        const float2 y = *reinterpret_cast<const float2*>(po);
        x[0] = fmaf(y.x, f, x[0]);
        x[1] = fmaf(y.y, f, x[1]);
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) part[warp][lane * V + e] = x[e];
    __syncthreads();
    if (warp != 0) return;
    L = 0.f;
#pragma unroll
    for (int u = 0; u < NW; ++u) L += red[2][u];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      x[e] = 0.f;
#pragma unroll
      for (int u = 0; u < NW; ++u) x[e] += part[u][lane * V + e];
    }
    const float fin = L > 0.f ? tc::ex2(MVr - Mr) / L : (L == 0.f ? 0.f : L);
    uint16_t* dst = a.o + static_cast<size_t>(sl.nr.row0 + r / g) * c.ld_o + (hk * g + r % g) * D + lane * V;
    if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(x[0] * fin, x[1] * fin), pack_bf16(x[2] * fin, x[3] * fin));
    else *reinterpret_cast<uint32_t*>(dst) = pack_bf16(x[0] * fin, x[1] * fin);
    if (lane == 0) keep_sum(sl, hk, r, M, L);
  }
}

// ---------------------------------------------------------------------------
// third kernel: the weights, from the scores (most still in L2) and the rows'
// sums. A thread takes a token, or SIDE threads side by side one token of many
// rows, four rows each at a time.
// ---------------------------------------------------------------------------

constexpr int kWeightThreads = 256;
constexpr int kWeightTokens = 8;    // per thread
constexpr int kMaxRowsHeld = 512;

template <int SIDE>
__global__ void __launch_bounds__(kWeightThreads)
cache_weights_kernel(Cache c, Args a, const float* w_in, float* w_out) {
  constexpr int T = kWeightTokens, STEP = kWeightThreads / SIDE;
  __shared__ __align__(16) float held[kMaxRowsHeld];
  pdl_wait();
  const int hk = blockIdx.z, b = blockIdx.y, tok0 = blockIdx.x * (T * STEP);
  bool bad = false;
  const NewRows nr = new_rows(c, a.seq, a.lens, b, bad);
  const int tok1 = nr.len, g = c.g, rows = nr.n * g;
  if (tok0 >= tok1) return;
  const int shift = 31 - __clz(c.block), q = threadIdx.x % SIDE, t0 = tok0 + threadIdx.x / SIDE;
  float sum[T];
#pragma unroll
  for (int e = 0; e < T; ++e) sum[e] = 0.f;
  const float* sc = a.scores + (static_cast<size_t>(b) * c.H_kv + hk) * c.max_blocks * c.block * a.rows_pad;
  for (int base = 0; base < rows; base += kMaxRowsHeld) {
    const int n = min(kMaxRowsHeld, rows - base), n4 = (n + 3) / 4 * 4;
    // the first four rows' scores and the rows' sums are on their way together
    float4 x[T];
    auto read = [&](int r) {
#pragma unroll
      for (int e = 0; e < T; ++e)
        x[e] = r < n && t0 + e * STEP < tok1
                   ? __ldcs(reinterpret_cast<const float4*>(sc + static_cast<size_t>(t0 + e * STEP) * a.rows_pad + base + r))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    read(4 * q);
    if (base > 0) __syncthreads();
    for (int rr = threadIdx.x; rr < n4; rr += kWeightThreads) {
      const int r = base + rr;
      held[rr] = rr < n ? a.lse2[static_cast<size_t>(nr.row0 + r / g) * c.H + hk * g + r % g] : INFINITY;
    }
    __syncthreads();
    const bool all_seen = tok0 + T * STEP <= nr.first + 1 && n % 4 == 0;
    for (int r = 4 * q; r < n; r += 4 * SIDE) {
      const float4 h4 = *reinterpret_cast<const float4*>(held + r);
      if (r >= 4 * SIDE) read(r);
#pragma unroll
      for (int e = 0; e < T; ++e) {
        float p0 = tc::ex2(x[e].x - h4.x), p1 = tc::ex2(x[e].y - h4.y), p2 = tc::ex2(x[e].z - h4.z), p3 = tc::ex2(x[e].w - h4.w);
        if (!all_seen) {
          // rows that end before a token left no score for it: the first that sees it is row (tok - first) g
          const int from = min(max(t0 + e * STEP - nr.first, 0), nr.n) * g - base - r;
          p0 = from <= 0 ? p0 : 0.f;
          p1 = from <= 1 && r + 1 < n ? p1 : 0.f;
          p2 = from <= 2 && r + 2 < n ? p2 : 0.f;
          p3 = from <= 3 && r + 3 < n ? p3 : 0.f;
        }
        sum[e] += (p0 + p1) + (p2 + p3);
      }
    }
  }
  int at[T];                          // the tokens' places in w, -1: none
  const int32_t* blocks = a.table + static_cast<size_t>(b) * c.max_blocks;
#pragma unroll
  for (int e = 0; e < T; ++e) {
    const int tok = t0 + e * STEP;
    at[e] = q == 0 && tok < tok1 ? __ldg(blocks + (tok >> shift)) : -1;
  }
#pragma unroll
  for (int e = 0; e < T; ++e) {
    at[e] = at[e] >= 0 && at[e] < c.n_blocks ? (at[e] * c.H_kv + hk) * c.block + ((t0 + e * STEP) & (c.block - 1)) : -1;
#pragma unroll
    for (int o = 1; o < SIDE; o <<= 1) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], o);
  }
  if (w_in != nullptr) {
    float old[T];
#pragma unroll
    for (int e = 0; e < T; ++e) old[e] = at[e] >= 0 ? w_in[at[e]] : 0.f;
#pragma unroll
    for (int e = 0; e < T; ++e) sum[e] += old[e];
  }
#pragma unroll
  for (int e = 0; e < T; ++e)
    if (at[e] >= 0) w_out[at[e]] = sum[e];
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

template <int D, int NR, bool HALVES>
cudaError_t run_attn(const Cache& c, const Args& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
  const int smem = Smem<D>::kTotal + 1024;
  cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<D, NR, HALVES>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_after(cache_attn_kernel<D, NR, HALVES>, dim3(a.workers), dim3(kThreads), smem, stream, mk, mv, c, a);
}

template <int D>
cudaError_t run(const Cache& c, const Args& a, const uint8_t* k_codes, const uint8_t* v_codes, const float* w_in,
                float* w_out, bool wide_join, cudaStream_t stream) {
  if (encode_fn() == nullptr) return cudaErrorNotSupported;
  CUtensorMap mk, mv;
  if (!make_map(&mk, k_codes, c) || !make_map(&mv, v_codes, c)) return cudaErrorInvalidValue;
  const bool halves = c.block < kTok, one = a.tile_rows == 8;
  cudaError_t e = halves ? (one ? run_attn<D, 1, true>(c, a, mk, mv, stream) : run_attn<D, 2, true>(c, a, mk, mv, stream))
                               : (one ? run_attn<D, 1, false>(c, a, mk, mv, stream) : run_attn<D, 2, false>(c, a, mk, mv, stream));
  if (e != cudaSuccess) return e;
  if (a.whole_row_tiles == 0) {
    const unsigned rows = static_cast<unsigned>(c.B * c.H_kv * a.rows_pad);  // below 2^31
    e = wide_join ? launch_after(cache_join_kernel<D, true>, dim3(rows), dim3(kJoinThreads), 0, stream, c, a)
                  : launch_after(cache_join_kernel<D, false>, dim3((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32)),
                                 dim3(kJoinThreads), 0, stream, c, a);
    if (e != cudaSuccess) return e;
  }
  if (a.scores == nullptr) return cudaSuccess;
  auto weights = [&](auto side) {
    constexpr int SIDE = decltype(side)::value, SPAN = kWeightTokens * kWeightThreads / SIDE;
    const int spans = (c.max_blocks * c.block + SPAN - 1) / SPAN;
    return launch_after(cache_weights_kernel<SIDE>, dim3(spans, c.B, c.H_kv), dim3(kWeightThreads), 0, stream, c, a, w_in,
                        w_out);
  };
  return a.rows_pad >= 16 ? weights(std::integral_constant<int, 4>{}) : weights(std::integral_constant<int, 1>{});
}

}  // namespace

CacheLayout make_cache_layout(const Cache& c) {
  CacheLayout y{};
  const long long heads = static_cast<long long>(c.B) * c.H_kv;
  const int most = c.max_new < c.rows ? c.max_new : c.rows;  // rows of one sequence
  const int rows = (most > 0 ? most : 1) * (c.g);
  y.rows_pad = (rows + 3) / 4 * 4;
  y.tile_rows = rows <= 8 ? 8 : 16;
  const long long tokens = static_cast<long long>(c.max_blocks) * c.block;
  // one wave of resident CTAs, or as many as the longest possible line fills
  const long long row_tiles = (rows + y.tile_rows - 1) / y.tile_rows, most_tiles = (tokens + kTok - 1) / kTok;
  y.line_places = heads * row_tiles * (kLead + most_tiles);
  long long ctas = (y.line_places + kLeast - 1) / kLeast;
  if (ctas > kSms * kCtasPerSm) ctas = kSms * kCtasPerSm;
  y.whole_row_tiles = most_tiles <= kWholeTiles && heads * row_tiles < (1ll << 31) ? static_cast<int>(row_tiles) : 0;
  y.workers = static_cast<int>(y.whole_row_tiles > 0 ? heads * row_tiles : ctas);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  size_t off = 256;
  const size_t slots = y.whole_row_tiles > 0 ? 0 : 2 * static_cast<size_t>(y.workers) * y.tile_rows;
  y.line = off;     off = up(off + (static_cast<size_t>(c.B) + 1) * 4);
  y.part_o = off;   off = up(off + slots * c.d * 4);
  y.part_ml = off;  off = up(off + slots * 16);
  y.lse2 = off;     off = up(off + (c.weights ? static_cast<size_t>(c.rows) * c.H * 4 : 0));
  y.scores = off;   off = up(off + (c.weights ? static_cast<size_t>(heads) * tokens * y.rows_pad * 4 : 0));
  y.total = off;
  y.join_ctas = heads * y.rows_pad;
  // A row's parts number about workers / units. A CTA per row costs many rows of few parts several waves, a
  // warp per row costs few rows of many parts a chain of reads: the CTA from 16 parts on.
  y.wide_join = y.workers >= 16 * heads * row_tiles;
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
  a.part_ml = reinterpret_cast<float4*>(base + y.part_ml);
  a.line = reinterpret_cast<int*>(base + y.line);
  a.lse2 = reinterpret_cast<float*>(base + y.lse2);
  a.scores = w_out != nullptr ? reinterpret_cast<float*>(base + y.scores) : nullptr;
  a.status = reinterpret_cast<unsigned*>(base);
  a.workers = y.workers;
  a.tile_rows = y.tile_rows;
  a.whole_row_tiles = y.whole_row_tiles;
  a.rows_pad = y.rows_pad;
  a.wait_ns = serving_wait_limit();
  if (c.d == 128) return run<128>(c, a, k_codes, v_codes, w_in, w_out, y.wide_join != 0, stream);
  if (c.d == 64) return run<64>(c, a, k_codes, v_codes, w_in, w_out, y.wide_join != 0, stream);
  return cudaErrorInvalidValue;
}

}  // namespace sda
