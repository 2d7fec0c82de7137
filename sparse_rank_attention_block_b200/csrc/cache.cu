// The 8-bit key/value cache: append and eviction.
//
// Values are E4M3 codes times a scale for each block of tokens and key head.
// Append picks the scale as a power of two, so that scaling neither rounds a
// code nor, when a later token makes a block's scale grow, the older ones
// (only values that become subnormal are rounded again).
//
// Both are bound by memory: append reads the new rows (bf16) and writes their
// codes, eviction reads the weights of every token and moves the kept rows.
// Measured: 9,076 tokens, 9,001 of them to one of 6 sequences, 8 heads: 20 us
// (2.8 TB/s; 8.5 us at the measured copy rate); from inputs in L2: 6 whole
// prompts of 1,500 tokens 13.4 us, 4 tokens for each of 64 sequences 7.7 us, one
// for each 6.7 us, a launch and a chain of four reads. Eviction of 32 sequences
// of 6,000 to 16,384 tokens to 4,096, 8 heads: 134 us (85 us at the copy rate),
// 31 us of it the selection, whose instructions bound it, and 106 us the move
// (5.2 TB/s).

#include "common.cuh"
#include "e4m3.cuh"
#include "launch.cuh"
#include "serving.h"

namespace sda {

namespace {

// ---------------------------------------------------------------------------
// append: a CTA takes one touched block and some of its units (a head's K or V);
// a unit's new rows stay in registers between their maximum and their encoding. A
// thread holds a 16-byte chunk (8 channels) of up to kPasses rows.
// ---------------------------------------------------------------------------

constexpr int kPasses = 4;

// Smallest power of two s in [2^-126, 2^120] with amax <= 448 s, for the bits of a bf16 amax >= 0.
__device__ __forceinline__ float wanted_scale(uint32_t amax_bf16) {
  const int e = static_cast<int>(amax_bf16 >> 7), frac = amax_bf16 & 0x7f;
  // amax = (1 + frac / 128) 2^(e - 127) and 448 = 1.75 * 2^8
  const int biased = e - 8 + (frac > 96 ? 1 : 0);  // exponent field of s
  return __uint_as_float(static_cast<uint32_t>(max(biased, 1)) << 23);
}

template <int D>
__global__ void cache_append_kernel(Cache c, int touched, int units, const uint16_t* __restrict__ k,
                                    const uint16_t* __restrict__ v, const int32_t* __restrict__ seq,
                                    const int32_t* __restrict__ lens, const int32_t* __restrict__ table,
                                    uint8_t* __restrict__ k_codes, uint8_t* __restrict__ v_codes,
                                    float* __restrict__ k_scale, float* __restrict__ v_scale, float* __restrict__ w,
                                    unsigned* status) {
  constexpr int CH = D / 8;  // chunks of a row
  __shared__ uint32_t warp_max[2][32];
  const int b = blockIdx.y, i = blockIdx.x % touched, u0 = blockIdx.x / touched * units;
  bool bad = false;
  pdl_wait();
  const NewRows r = new_rows(c, seq, lens, b, bad);
  bad = bad || r.first < 0;
  const int start = max(r.first, 0);
  const int bi = (start >> (31 - __clz(c.block))) + i;        // block of the sequence
  const int lo = max(bi * c.block, start);                    // its new positions [lo, hi)
  const int hi = min(min((bi + 1) * c.block, r.first + r.n), c.max_blocks * c.block);
  if (threadIdx.x == 0 && blockIdx.x == 0 && bad) report_status(status, kStatusBadIndex);
  if (lo >= hi || bi >= c.max_blocks) return;
  const int blk = __ldg(table + static_cast<size_t>(b) * c.max_blocks + bi);
  if (blk < 0 || blk >= c.n_blocks) {
    if (threadIdx.x == 0) report_status(status, kStatusBadIndex);
    return;
  }
  const int slot0 = lo - bi * c.block, n = hi - lo;           // slots [slot0, slot0 + n); older tokens before them
  const int ch = threadIdx.x % CH, row0 = threadIdx.x / CH, step = blockDim.x / CH;
  const size_t first_row = static_cast<size_t>(r.row0) + (lo - r.first);
  const int u1 = min(u0 + units, 2 * c.H_kv);
  // unit u: head u / 2, K or V; the next unit's rows are on their way while one is encoded
  uint4 x[kPasses];
  auto read = [&](int u) {
    const uint16_t* src = u & 1 ? v : k;
    const long long ld = u & 1 ? c.ld_v : c.ld_k;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int row = row0 + p * step;
      x[p] = row < n ? __ldcs(reinterpret_cast<const uint4*>(src + (first_row + row) * ld + (u >> 1) * D) + ch)
                     : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  // |x| of a bf16 orders like its bits without the sign; infinities and NaN (>= 0x7f80) do not count
  auto magnitude = [](uint32_t two) {
    const uint32_t lo16 = two & 0x7fffu, hi16 = (two >> 16) & 0x7fffu;
    return (lo16 < 0x7f80u ? lo16 : 0u) | (hi16 < 0x7f80u ? hi16 : 0u) << 16;
  };
  read(u0);
  for (int u = u0; u < u1; ++u) {
    const size_t head = static_cast<size_t>(blk) * c.H_kv + (u >> 1);
    uint8_t* codes = (u & 1 ? v_codes : k_codes) + head * c.block * D;
    float* scale = (u & 1 ? v_scale : k_scale) + head;
    const float before = slot0 > 0 ? *scale : 0.f;
    uint32_t m2 = 0u;  // two 16-bit magnitudes
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      m2 = __vmaxu2(m2, __vmaxu2(magnitude(x[p].x), magnitude(x[p].y)));
      m2 = __vmaxu2(m2, __vmaxu2(magnitude(x[p].z), magnitude(x[p].w)));
    }
    uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
    const int warps = blockDim.x / 32;
    uint32_t* tops = warp_max[u & 1];  // two in turn: one barrier a unit is enough
    if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = m;
    __syncthreads();                   // every thread has read the old scale, too
    for (int g = 0; g < warps; ++g) m = max(m, tops[g]);
    const float want = wanted_scale(m);
    const float after = slot0 > 0 ? fmaxf(before, want) : want;
    if (threadIdx.x == 0) {
      *scale = after;
      if (!is_scale(before)) report_status(status, kStatusBadIndex);
    }
    if (slot0 > 0 && before != after) {
      const Rescale again(before / after);
      for (int row = row0; row < slot0; row += step) {
        uint2* at = reinterpret_cast<uint2*>(codes + row * D) + ch;
        const uint2 old = *at;
        *at = make_uint2(again(old.x), again(old.y));
      }
    }
    // x / scale: for a power of two (every scale that append chose) the product with its inverse is the quotient
    const bool pow2 = (__float_as_uint(after) & 0x7fffffu) == 0u;
    const float inv = 1.f / after;
    uint2 out[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const uint32_t in[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
      uint32_t two[4];
      if (pow2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) two[e] = f32x2_to_e4m3x2(bf16_lo(in[e]) * inv, bf16_hi(in[e]) * inv);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) two[e] = f32x2_to_e4m3x2(bf16_lo(in[e]) / after, bf16_hi(in[e]) / after);
      }
      out[p] = make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
    }
    if (u + 1 < u1) read(u + 1);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int row = row0 + p * step;
      if (row < n) *(reinterpret_cast<uint2*>(codes + (slot0 + row) * D) + ch) = out[p];
    }
    if (w != nullptr && !(u & 1))
      for (int row = threadIdx.x; row < n; row += blockDim.x) w[head * c.block + slot0 + row] = 0.f;
  }
}

// ---------------------------------------------------------------------------
// eviction, first kernel: which tokens stay. One CTA per sequence and head: a
// radix selection of the n-th largest weight (8 bits a pass, keys in shared
// memory where they fit), then the kept positions in order.
// ---------------------------------------------------------------------------

constexpr int kSelThreads = 1024;
constexpr int kSelKeys = 49152;  // keys held in shared memory (192 KB); longer sequences read them again each pass

// Order of the floats as unsigned integers; -0 equals +0, NaN is the largest.
__device__ __forceinline__ uint32_t weight_key(float x) {
  uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads)
cache_select_kernel(Cache c, int cap, const int32_t* __restrict__ lens, const int32_t* __restrict__ table,
                    const float* __restrict__ w, int32_t* __restrict__ kept, int32_t* __restrict__ rows,
                    int32_t* __restrict__ dst_lens, unsigned* status) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ uint32_t hist[256];
  __shared__ uint32_t found[2];  // digit, tokens above it
  __shared__ int warp_gt[32], warp_eq[32];
  const int h = blockIdx.x % c.H_kv, b = blockIdx.x / c.H_kv;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int shift_b = 31 - __clz(c.block);
  const int32_t* blocks = table + static_cast<size_t>(b) * c.max_blocks;
  pdl_wait();
  const int given = __ldg(lens + b);
  const int len = min(max(given, 0), c.max_blocks * c.block);
  const int n = min(len, c.keep), last = min(c.recent, n);
  const int older = len - last, need = n - last;  // `need` of the `older` first tokens stay
  if (threadIdx.x == 0 && h == 0) {
    dst_lens[b] = n;
    if (len != given) report_status(status, kStatusBadIndex);
  }
  // row of the pool that holds token t, -1 where its block is none of the pool's
  auto row_of = [&](int t) {
    const int blk = __ldg(blocks + (t >> shift_b));
    if (blk >= 0 && blk < c.n_blocks) return (blk * c.H_kv + h) * c.block + (t & (c.block - 1));
    report_status(status, kStatusBadIndex);
    return -1;
  };
  // keys of tokens t .. t + 3 (t a multiple of 4: one block), 0 in a block that is none of the pool's
  auto load_keys = [&](int t) {
    const int row = row_of(t);
    const float4 x = row >= 0 ? __ldg(reinterpret_cast<const float4*>(w + row)) : make_float4(0.f, 0.f, 0.f, 0.f);
    return row >= 0 ? make_uint4(weight_key(x.x), weight_key(x.y), weight_key(x.z), weight_key(x.w)) : make_uint4(0u, 0u, 0u, 0u);
  };
  const size_t out0 = (static_cast<size_t>(b) * c.H_kv + h) * c.keep;
  auto stay = [&](int i, int t) {
    kept[out0 + i] = t;
    if (t >= 0) rows[out0 + i] = row_of(t);
  };
  pdl_launch();
  for (int t = threadIdx.x; t < c.keep - need; t += kSelThreads) stay(need + t, t < last ? older + t : -1);
  if (need == 0) return;
  if (need == older) {
    for (int t = threadIdx.x; t < need; t += kSelThreads) stay(t, t);
    return;
  }
  const bool held = older <= cap;
  if (held)
    for (int t = 4 * threadIdx.x; t < older; t += 4 * kSelThreads) *reinterpret_cast<uint4*>(keys + t) = load_keys(t);
  // A lane takes four tokens at a time, warps contiguous pieces, so that the order of the positions is the
  // order of the lanes and warps.
  const int per_warp = (older + 32 * 128 - 1) / (32 * 128) * 128;
  const int t0 = min(warp * per_warp, older), t1 = min(t0 + per_warp, older);
  auto keys_at = [&](int t, uint32_t (&k)[4]) {  // 0 behind the piece: below every key but the smallest, and not counted
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (t < t1) x = held ? *reinterpret_cast<const uint4*>(keys + t) : load_keys(t);
    k[0] = x.x;
    k[1] = x.y;
    k[2] = x.z;
    k[3] = x.w;
    return min(4, t1 - t);                       // how many of them count
  };

  uint32_t prefix = 0u, mask = 0u;
  int rank = need;  // the rank-th largest among the keys that match the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) hist[threadIdx.x] = 0u;
    __syncthreads();
    for (int t = t0 + 4 * lane; t < t1; t += 128) {
      uint32_t k[4];
      const int n_k = keys_at(t, k);
#pragma unroll
      for (int e = 0; e < 4; ++e)                // counts: the order does not matter
        if (e < n_k && (k[e] & mask) == prefix) atomicAdd(&hist[(k[e] >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      // digits from the top: lane l holds digits 255 - 8 l .. 248 - 8 l
      uint32_t cnt[8], sum = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        cnt[e] = hist[255 - 8 * lane - e];
        sum += cnt[e];
      }
      uint32_t above = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, above, o);
        if (lane >= o) above += u;
      }
      above -= sum;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (above < static_cast<uint32_t>(rank) && static_cast<uint32_t>(rank) <= above + cnt[e]) {
          found[0] = 255 - 8 * lane - e;
          found[1] = above;
        }
        above += cnt[e];
      }
    }
    __syncthreads();
    prefix |= found[0] << shift;
    mask |= 255u << shift;
    rank -= static_cast<int>(found[1]);
  }
  // keys above `prefix` stay, and the first `rank` of those equal to it
  int gt = 0, eq = 0;
  for (int t = t0 + 4 * lane; t < t1; t += 128) {
    uint32_t k[4];
    const int n_k = keys_at(t, k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gt += e < n_k && k[e] > prefix;
      eq += e < n_k && k[e] == prefix;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    warp_gt[warp] = gt;
    warp_eq[warp] = eq;
  }
  __syncthreads();
  int gt_before = 0, eq_before = 0;
  for (int u = 0; u < warp; ++u) {
    gt_before += warp_gt[u];
    eq_before += warp_eq[u];
  }
  for (int base = t0; base < t1; base += 128) {
    const int t = base + 4 * lane;
    uint32_t k[4];
    const int n_k = keys_at(t, k);
    uint32_t mine = 0u;                          // (equal, above) of this lane's four, 16 bits each
#pragma unroll
    for (int e = 0; e < 4; ++e) mine += e < n_k ? (k[e] > prefix ? 1u : k[e] == prefix ? 0x10000u : 0u) : 0u;
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    int my_gt = gt_before + static_cast<int>((incl - mine) & 0xffffu), my_eq = eq_before + static_cast<int>((incl - mine) >> 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e >= n_k) continue;
      if (k[e] > prefix || (k[e] == prefix && my_eq < rank)) stay(my_gt + min(my_eq, rank), t + e);
      my_gt += k[e] > prefix;
      my_eq += k[e] == prefix;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
    gt_before += static_cast<int>(all & 0xffffu);
    eq_before += static_cast<int>(all >> 16);
  }
}

// ---------------------------------------------------------------------------
// eviction, second kernel: the kept rows move. One CTA per target block and
// head. A thread's rows are on their way while the target's scales are found.
// ---------------------------------------------------------------------------

constexpr int kChunks = 4;  // 16-byte chunks of K and V a thread moves

template <int D>
__global__ void cache_move_kernel(Cache c, const int32_t* __restrict__ lens, uint8_t* k_codes, uint8_t* v_codes,
                                  float* k_scale, float* v_scale, float* w, const int32_t* __restrict__ dst_table,
                                  const int32_t* __restrict__ rows, unsigned* status) {
  constexpr int CH = D / 16;  // chunks of a row
  __shared__ float scale[2][128];
  __shared__ float ratio[2][128];
  const int b = blockIdx.y, h = blockIdx.x % c.H_kv, i = blockIdx.x / c.H_kv;
  const int shift = 31 - __clz(c.block), t = threadIdx.x;
  pdl_wait();
  const int len = min(max(__ldg(lens + b), 0), c.max_blocks * c.block);
  const int dst = __ldg(dst_table + static_cast<size_t>(b) * c.dst_blocks + i);
  const int first = i * c.block, count = min(c.block, min(len, c.keep) - first);
  if (count <= 0) return;
  if (dst < 0 || dst >= c.n_blocks) {
    if (t == 0) report_status(status, kStatusBadIndex);
    return;
  }
  const int32_t* src = rows + (static_cast<size_t>(b) * c.H_kv + h) * c.keep + first;
  const int dst_head = dst * c.H_kv + h;
  // chunk e of the block's K rows, then of its V rows; threads: a quarter of both
  uint4 x[kChunks];
  int row[kChunks];
#pragma unroll
  for (int u = 0; u < kChunks; ++u) {
    const int e = t + (u % 2) * blockDim.x, r = e / CH;
    row[u] = r < count ? src[r] : -1;
  }
#pragma unroll
  for (int u = 0; u < kChunks; ++u)
    if (row[u] >= 0)
      x[u] = *(reinterpret_cast<const uint4*>((u < 2 ? k_codes : v_codes) + static_cast<size_t>(row[u]) * D) +
               (t + (u % 2) * blockDim.x) % CH);
  for (int r = t; r < c.block; r += blockDim.x) {  // blocks of 64-channel rows: two rows a thread
    const int from = r < count ? src[r] : -1;
    float a = 0.f, bb = 0.f;
    if (from >= 0) {
      a = k_scale[from >> shift];
      bb = v_scale[from >> shift];
      w[static_cast<size_t>(dst_head) * c.block + r] = w[from];
    }
    scale[0][r] = a;
    scale[1][r] = bb;
  }
  __syncthreads();
  // scales are not negative: their bits order like their values
  uint32_t k_top = 0u, v_top = 0u;
  for (int r = t % 32; r < c.block; r += 32) {
    k_top = max(k_top, __float_as_uint(scale[0][r]));
    v_top = max(v_top, __float_as_uint(scale[1][r]));
  }
  const float ks = __uint_as_float(__reduce_max_sync(0xffffffffu, k_top));
  const float vs = __uint_as_float(__reduce_max_sync(0xffffffffu, v_top));
  if (t == 0) {
    k_scale[dst_head] = ks;
    v_scale[dst_head] = vs;
    if (!(is_scale(ks) && is_scale(vs))) report_status(status, kStatusBadIndex);  // the largest bits: all are or it is not
  }
  for (int r = t; r < c.block; r += blockDim.x) {
    ratio[0][r] = ks > 0.f ? scale[0][r] / ks : 1.f;
    ratio[1][r] = vs > 0.f ? scale[1][r] / vs : 1.f;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kChunks; ++u) {
    if (row[u] < 0) continue;
    const int e = t + (u % 2) * blockDim.x, r = e / CH;
    const float f = ratio[u < 2 ? 0 : 1][r];
    uint4 y = x[u];
    if (f != 1.f) {
      const Rescale again(f);
      y = make_uint4(again(y.x), again(y.y), again(y.z), again(y.w));
    }
    *(reinterpret_cast<uint4*>((u < 2 ? k_codes : v_codes) + (static_cast<size_t>(dst_head) * c.block + r) * D) + e % CH) = y;
  }
}

}  // namespace

cudaError_t launch_cache_append(const Cache& c, const uint16_t* k, const uint16_t* v, const int32_t* seq,
                                const int32_t* lens, const int32_t* table, uint8_t* k_codes, uint8_t* v_codes,
                                float* k_scale, float* v_scale, float* w, unsigned* status, cudaStream_t stream) {
  const int most = min(c.max_new, c.rows);
  const int touched = (most + c.block - 2) / c.block + 1;  // blocks that `most` tokens can lie in
  // Single tokens: a CTA per unit, for latency. More tokens can touch a block more than they do, so that half of the
  // CTAs or more find nothing to do: two units a CTA (8 heads; us with one, two and four units: 64 sequences of 4 new
  // tokens 8.6, 7.8, 12.2; of 17: 10.2, 10.0, 12.9; of 200: 26.1, 23.9, 24.5; 6 of 1,500: 14.3, 13.3, 13.4; one of
  // 9,001 beside five of 5 to 25: 24.4, 20.3, 19.9; and 64 of one token: 6.7, 6.8 with two).
  const int units = touched > 1 ? 2 : 1;
  const dim3 grid(static_cast<unsigned>(touched) * ((2 * c.H_kv + units - 1) / units), c.B);
  const int threads = c.block * c.d / 8 / kPasses;
  return launch_after(c.d == 128 ? cache_append_kernel<128> : cache_append_kernel<64>, grid, dim3(threads), 0, stream, c,
                      touched, units, k, v, seq, lens, table, k_codes, v_codes, k_scale, v_scale, w, status);
}

cudaError_t launch_cache_evict(const Cache& c, const int32_t* lens, const int32_t* table, uint8_t* k_codes,
                               uint8_t* v_codes, float* k_scale, float* v_scale, float* w, const int32_t* dst_table,
                               int32_t* kept, int32_t* dst_lens, int32_t* rows, unsigned* status, cudaStream_t stream) {
  const int cap = min(c.max_blocks * c.block, kSelKeys);
  cudaError_t e = cudaFuncSetAttribute(cache_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4);
  if (e != cudaSuccess) return e;
  e = launch_after(cache_select_kernel, dim3(c.B * c.H_kv), dim3(kSelThreads), cap * 4, stream, c, cap, lens, table, w,
                   kept, rows, dst_lens, status);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(c.dst_blocks) * c.H_kv, c.B);
  const int threads = c.block * c.d / 16 * 2 / kChunks;
  return launch_after(c.d == 128 ? cache_move_kernel<128> : cache_move_kernel<64>, grid, dim3(threads), 0, stream, c, lens,
                      k_codes, v_codes, k_scale, v_scale, w, dst_table, rows, status);
}

}  // namespace sda
