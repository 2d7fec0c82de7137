// The 8-bit key/value cache: append and eviction.
//
// Values are E4M3 codes times a scale for each block of tokens and key head.
// Append picks the scale as a power of two, so that scaling neither rounds a
// code nor, when a later token makes a block's scale grow, the older ones
// (only values that become subnormal are rounded again).
//
// Both are bound by memory: append reads the new rows (bf16) and writes their
// codes, eviction reads the weights of every token and moves the kept rows.

#include "common.cuh"
#include "e4m3.cuh"
#include "serving.h"

namespace sda {

namespace {

// ---------------------------------------------------------------------------
// append: one CTA per touched block, head and K or V; the block's new rows stay
// in registers between their maximum and their encoding. A thread holds a
// 16-byte chunk (8 channels) of up to kPasses rows.
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
__global__ void cache_append_kernel(Cache c, int touched, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                                    const int32_t* __restrict__ seq, const int32_t* __restrict__ lens,
                                    const int32_t* __restrict__ table, uint8_t* __restrict__ k_codes,
                                    uint8_t* __restrict__ v_codes, float* __restrict__ k_scale,
                                    float* __restrict__ v_scale, float* __restrict__ w, unsigned* status) {
  constexpr int CH = D / 8;  // chunks of a row
  __shared__ uint32_t warp_max[32];
  const int b = blockIdx.y;
  const int is_v = blockIdx.x & 1, h = (blockIdx.x >> 1) % c.H_kv, i = (blockIdx.x >> 1) / c.H_kv;
  bool bad = false;
  const NewRows r = new_rows(c, seq, lens, b, bad);
  bad = bad || r.first < 0;
  const int start = max(r.first, 0);
  const int bi = start / c.block + i;                         // block of the sequence
  const int lo = max(bi * c.block, start);                    // its new positions [lo, hi)
  const int hi = min(min((bi + 1) * c.block, r.first + r.n), c.max_blocks * c.block);
  if (threadIdx.x == 0 && blockIdx.x == 0 && bad) report_status(status, kStatusBadIndex);
  if (i >= touched || lo >= hi || bi >= c.max_blocks) return;
  const int blk = __ldg(table + static_cast<size_t>(b) * c.max_blocks + bi);
  if (blk < 0 || blk >= c.n_blocks) {
    if (threadIdx.x == 0) report_status(status, kStatusBadIndex);
    return;
  }
  const uint16_t* src = is_v ? v : k;
  const long long ld = is_v ? c.ld_v : c.ld_k;
  const size_t head = static_cast<size_t>(blk) * c.H_kv + h;
  uint8_t* codes = (is_v ? v_codes : k_codes) + head * c.block * D;
  float* scale = (is_v ? v_scale : k_scale) + head;
  const int slot0 = lo - bi * c.block, n = hi - lo;           // slots [slot0, slot0 + n); older tokens before them
  const int ch = threadIdx.x % CH, row0 = threadIdx.x / CH, step = blockDim.x / CH;
  const float before = slot0 > 0 ? *scale : 0.f;

  uint4 x[kPasses];
  uint32_t m2 = 0u;  // two 16-bit magnitudes
  const size_t first_row = static_cast<size_t>(r.row0) + (lo - r.first);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int row = row0 + p * step;
    x[p] = row < n ? __ldcs(reinterpret_cast<const uint4*>(src + (first_row + row) * ld + h * D) + ch)
                   : make_uint4(0u, 0u, 0u, 0u);
  }
  // |x| of a bf16 orders like its bits without the sign; infinities and NaN (>= 0x7f80) do not count
  auto magnitude = [](uint32_t two) {
    const uint32_t a = two & 0x7fffu, bb = (two >> 16) & 0x7fffu;
    return (a < 0x7f80u ? a : 0u) | (bb < 0x7f80u ? bb : 0u) << 16;
  };
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    m2 = __vmaxu2(m2, __vmaxu2(magnitude(x[p].x), magnitude(x[p].y)));
    m2 = __vmaxu2(m2, __vmaxu2(magnitude(x[p].z), magnitude(x[p].w)));
  }
  uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
  const int warps = blockDim.x / 32;
  if (warps > 1) {
    if (threadIdx.x % 32 == 0) warp_max[threadIdx.x / 32] = m;
    __syncthreads();
    m = warp_max[0];
    for (int u = 1; u < warps; ++u) m = max(m, warp_max[u]);
  }
  const float want = wanted_scale(m);
  const float after = slot0 > 0 ? fmaxf(before, want) : want;
  // every thread has read the old scale before it changes (the barrier above; one warp: program order)
  if (warps == 1) __syncwarp();
  if (threadIdx.x == 0) *scale = after;
  if (slot0 > 0) {
    const float ratio = before / after;
    if (ratio != 1.f)
      for (int row = row0; row < slot0; row += step) {
        uint2* at = reinterpret_cast<uint2*>(codes + row * D) + ch;
        const uint2 old = *at;
        *at = make_uint2(e4m3x4_rescale(old.x, ratio), e4m3x4_rescale(old.y, ratio));
      }
  }
  // x / scale: for a power of two (every scale that append chose) the product with its inverse is the quotient
  const bool pow2 = (__float_as_uint(after) & 0x7fffffu) == 0u;
  const float inv = 1.f / after;
  auto scaled = [&](float f) { return pow2 ? f * inv : f / after; };
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int row = row0 + p * step;
    if (row < n) {
      const uint32_t in[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
      uint32_t two[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) two[e] = f32x2_to_e4m3x2(scaled(bf16_lo(in[e])), scaled(bf16_hi(in[e])));
      *(reinterpret_cast<uint2*>(codes + (slot0 + row) * D) + ch) = make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
    }
  }
  if (w != nullptr && !is_v)
    for (int row = threadIdx.x; row < n; row += blockDim.x) w[head * c.block + slot0 + row] = 0.f;
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
                    const float* __restrict__ w, int32_t* __restrict__ kept, int32_t* __restrict__ dst_lens,
                    unsigned* status) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[256];
  __shared__ uint32_t found[2];  // digit, tokens above it
  __shared__ int warp_gt[32], warp_eq[32];
  const int h = blockIdx.x % c.H_kv, b = blockIdx.x / c.H_kv;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int32_t* blocks = table + static_cast<size_t>(b) * c.max_blocks;
  const int given = __ldg(lens + b);
  const int len = min(max(given, 0), c.max_blocks * c.block);
  const int n = min(len, c.keep), last = min(c.recent, n);
  const int older = len - last, need = n - last;  // `need` of the `older` first tokens stay
  if (threadIdx.x == 0 && h == 0) {
    dst_lens[b] = n;
    if (len != given) report_status(status, kStatusBadIndex);
  }
  auto load_key = [&](int t) -> uint32_t {
    const int blk = __ldg(blocks + t / c.block);
    if (blk < 0 || blk >= c.n_blocks) {
      report_status(status, kStatusBadIndex);
      return 0u;
    }
    return weight_key(__ldg(w + (static_cast<size_t>(blk) * c.H_kv + h) * c.block + t % c.block));
  };
  int32_t* out = kept + (static_cast<size_t>(b) * c.H_kv + h) * c.keep;
  for (int t = threadIdx.x; t < c.keep - need; t += kSelThreads) out[need + t] = t < last ? older + t : -1;
  if (need == 0) return;
  if (need == older) {
    for (int t = threadIdx.x; t < need; t += kSelThreads) out[t] = t;
    return;
  }
  const bool held = older <= cap;
  if (held)
    for (int t = threadIdx.x; t < older; t += kSelThreads) keys[t] = load_key(t);
  // warp-contiguous pieces, so that the order of the positions is the order of the warps
  const int per_warp = ((older + 32 * 32 - 1) / (32 * 32)) * 32;
  const int t0 = min(warp * per_warp, older), t1 = min(t0 + per_warp, older);
  auto key_at = [&](int t) { return held ? keys[t] : load_key(t); };

  uint32_t prefix = 0u, mask = 0u;
  int rank = need;  // the rank-th largest among the keys that match the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) hist[threadIdx.x] = 0u;
    __syncthreads();
    for (int base = t0; base < t1; base += 32) {
      const int t = base + lane;
      const uint32_t key = t < t1 ? key_at(t) : 0u;
      const bool in = t < t1 && (key & mask) == prefix;
      const uint32_t digit = in ? (key >> shift) & 255u : 256u;
      // equal weights are common (zeros above all): one addition per digit and warp
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      if (in && lane == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
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
  for (int base = t0; base < t1; base += 32) {
    const int t = base + lane;
    const uint32_t key = t < t1 ? key_at(t) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, t < t1 && key > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, t < t1 && key == prefix));
  }
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
  const uint32_t below = (1u << lane) - 1u;
  for (int base = t0; base < t1; base += 32) {
    const int t = base + lane;
    const uint32_t key = t < t1 ? key_at(t) : 0u;
    const uint32_t g = __ballot_sync(0xffffffffu, t < t1 && key > prefix);
    const uint32_t e = __ballot_sync(0xffffffffu, t < t1 && key == prefix);
    const int my_eq = eq_before + __popc(e & below);
    if (t < t1 && (key > prefix || (key == prefix && my_eq < rank)))
      out[gt_before + __popc(g & below) + min(my_eq, rank)] = t;
    gt_before += __popc(g);
    eq_before += __popc(e);
  }
}

// ---------------------------------------------------------------------------
// eviction, second kernel: the kept rows move. One CTA per target block and
// head: the sources' places and the target's scales in shared memory first,
// then K and V rows in 16-byte chunks.
// ---------------------------------------------------------------------------

constexpr int kMoveThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMoveThreads)
cache_move_kernel(Cache c, const int32_t* __restrict__ lens, const int32_t* __restrict__ table, uint8_t* k_codes,
                  uint8_t* v_codes, float* k_scale, float* v_scale, float* w, const int32_t* __restrict__ dst_table,
                  const int32_t* __restrict__ kept, unsigned* status) {
  constexpr int CH = D / 16;  // chunks of a row
  __shared__ int src_row[128];            // row of the pool, -1: none
  __shared__ float ratio[2][128];
  __shared__ float warp_top[2][4];
  const int b = blockIdx.y, h = blockIdx.x % c.H_kv, i = blockIdx.x / c.H_kv;
  const int len = min(max(__ldg(lens + b), 0), c.max_blocks * c.block);
  const int n = min(len, c.keep);
  const int first = i * c.block, count = min(c.block, n - first);
  if (count <= 0) return;
  const int dst = __ldg(dst_table + static_cast<size_t>(b) * c.dst_blocks + i);
  if (dst < 0 || dst >= c.n_blocks) {
    if (threadIdx.x == 0) report_status(status, kStatusBadIndex);
    return;
  }
  const size_t dst_head = static_cast<size_t>(dst) * c.H_kv + h;
  float ks = 0.f, vs = 0.f;
  const int t = threadIdx.x;
  if (t < 128) {
    int row = -1;
    if (t < count) {
      const int pos = __ldg(kept + (static_cast<size_t>(b) * c.H_kv + h) * c.keep + first + t);
      const int blk = __ldg(table + static_cast<size_t>(b) * c.max_blocks + pos / c.block);
      if (blk >= 0 && blk < c.n_blocks) {
        const size_t head = static_cast<size_t>(blk) * c.H_kv + h;
        row = static_cast<int>(head) * c.block + pos % c.block;
        ks = k_scale[head];
        vs = v_scale[head];
        w[dst_head * c.block + t] = w[row];
      }
    }
    src_row[t] = row;
    float kt = ks, vt = vs;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      kt = fmaxf(kt, __shfl_xor_sync(0xffffffffu, kt, o));
      vt = fmaxf(vt, __shfl_xor_sync(0xffffffffu, vt, o));
    }
    if (t % 32 == 0) {
      warp_top[0][t / 32] = kt;
      warp_top[1][t / 32] = vt;
    }
  }
  __syncthreads();
  if (t < 128) {
    const float kt = fmaxf(fmaxf(warp_top[0][0], warp_top[0][1]), fmaxf(warp_top[0][2], warp_top[0][3]));
    const float vt = fmaxf(fmaxf(warp_top[1][0], warp_top[1][1]), fmaxf(warp_top[1][2], warp_top[1][3]));
    ratio[0][t] = kt > 0.f ? ks / kt : 1.f;
    ratio[1][t] = vt > 0.f ? vs / vt : 1.f;
    if (t == 0) {
      k_scale[dst_head] = kt;
      v_scale[dst_head] = vt;
    }
  }
  __syncthreads();
  constexpr int U = 4;  // chunks in flight per thread
  const int total = 2 * count * CH;
  for (int e0 = t; e0 < total; e0 += U * kMoveThreads) {
    uint4 x[U];
    int row[U], kv[U], ch[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = e0 + u * kMoveThreads;
      kv[u] = e >= count * CH;
      const int rest = e - kv[u] * count * CH;
      row[u] = rest / CH;
      ch[u] = rest % CH;
      if (e >= total || src_row[row[u]] < 0) row[u] = -1;
      if (row[u] >= 0) x[u] = *(reinterpret_cast<const uint4*>((kv[u] ? v_codes : k_codes) + static_cast<size_t>(src_row[row[u]]) * D) + ch[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (row[u] < 0) continue;
      const float f = ratio[kv[u]][row[u]];
      uint4 y = x[u];
      if (f != 1.f)
        y = make_uint4(e4m3x4_rescale(y.x, f), e4m3x4_rescale(y.y, f), e4m3x4_rescale(y.z, f), e4m3x4_rescale(y.w, f));
      *(reinterpret_cast<uint4*>((kv[u] ? v_codes : k_codes) + (dst_head * c.block + row[u]) * D) + ch[u]) = y;
    }
  }
}

}  // namespace

cudaError_t launch_cache_append(const Cache& c, const uint16_t* k, const uint16_t* v, const int32_t* seq,
                                const int32_t* lens, const int32_t* table, uint8_t* k_codes, uint8_t* v_codes,
                                float* k_scale, float* v_scale, float* w, unsigned* status, cudaStream_t stream) {
  const int most = min(c.max_new, c.rows);
  const int touched = (most + c.block - 2) / c.block + 1;  // blocks that `most` tokens can lie in
  const dim3 grid(static_cast<unsigned>(touched) * c.H_kv * 2, c.B);
  const int threads = c.block * c.d / 8 / kPasses;
  if (c.d == 128)
    cache_append_kernel<128><<<grid, threads, 0, stream>>>(c, touched, k, v, seq, lens, table, k_codes, v_codes,
                                                           k_scale, v_scale, w, status);
  else
    cache_append_kernel<64><<<grid, threads, 0, stream>>>(c, touched, k, v, seq, lens, table, k_codes, v_codes,
                                                          k_scale, v_scale, w, status);
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const Cache& c, const int32_t* lens, const int32_t* table, uint8_t* k_codes,
                               uint8_t* v_codes, float* k_scale, float* v_scale, float* w, const int32_t* dst_table,
                               int32_t* kept, int32_t* dst_lens, unsigned* status, cudaStream_t stream) {
  const int cap = min(c.max_blocks * c.block, kSelKeys);
  cudaError_t e = cudaFuncSetAttribute(cache_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4);
  if (e != cudaSuccess) return e;
  cache_select_kernel<<<c.B * c.H_kv, kSelThreads, cap * 4, stream>>>(c, cap, lens, table, w, kept, dst_lens, status);
  const dim3 grid(static_cast<unsigned>(c.dst_blocks) * c.H_kv, c.B);
  if (c.d == 128)
    cache_move_kernel<128><<<grid, kMoveThreads, 0, stream>>>(c, lens, table, k_codes, v_codes, k_scale, v_scale, w,
                                                              dst_table, kept, status);
  else
    cache_move_kernel<64><<<grid, kMoveThreads, 0, stream>>>(c, lens, table, k_codes, v_codes, k_scale, v_scale, w,
                                                             dst_table, kept, status);
  return cudaGetLastError();
}

}  // namespace sda
