// Attention over whole prompts on the 5th-generation tensor cores (tcgen05):
// packed sequences of different lengths, shared key heads, causal or all to
// all. For query row i of a sequence with n_q queries and n_k keys
//   o_i = sum_j p_ij v_j,  p_ij = exp(scale q_i . k_j) / sum_j' exp(scale q_i . k_j')
// over the keys j <= i + n_k - n_q (causal) or all n_k keys; a row that sees
// no key gives zeros and lse = -inf.
//
// Bound by the tensor pipe and, as closely, by the exponential unit: a
// 128 x 128 tile at d = 128 takes 1024 cycles of MMA (S = Q K^T and O += P V)
// and 1024 cycles of MUFU. One CTA per SM therefore carries TWO 128-row tiles
// that share every K and V tile: the tensor pipe works on one while the
// softmax warps work on the other. The two tiles are two query heads of the
// same key head (equal work under the causal mask) or, where the heads of a
// key head are odd in number, two adjacent row tiles of one head.
//
// Warps: 0 loads (TMA: Q tiles, then a ring of K and V tiles), 1 issues every
// MMA and clears V rows behind the sequence, 2 finds the next tiles to work on, 3
// owns TMEM; 4..7 and 8..11 softmax and epilogue of tile 0 and 1, a thread per row.
//
// A CTA takes its share of the (row tile, head group) items one after another, at
// most one CTA per SM: the search for an item, its loads and its first scores run
// under the end of the one before (9 prompts of 1 to 2,900 tokens 135 us against
// 145 us with a CTA per item, 4,680 rows on 512 keys 60 against 70 us; one long
// sequence loses 3 %, 100 tokens 1.3 us). Items go out heaviest first, in rounds.
//
// The MMAs of one thread execute in order, so the issue order
//   PV_0(j), QK_0(j+1), PV_1(j), QK_1(j+1)
// lets P_w overlay S_w in TMEM (bf16, half the columns): QK_w(j+1) comes
// after PV_w(j) has read P_w, and S_w(j+1) ready implies PV_w(j) done, so the
// softmax may rescale O_w without another wait. It does so only when a row's
// maximum grows by more than 2^8 (exact: numerator and denominator share the
// reference). P is rounded to bf16 (the type of V, as the MMA asks); the sum
// takes the unrounded fp32 values. One issuer also keeps the two tiles in
// opposite phase; an issuer for each tile let them fall into step, both in the
// exponentials and then both in the MMAs (4,230 cycles for a pair of steps).
// Handing P over in two halves cost more in waits than it overlapped (+4 %), and
// taking a share of the exponentials on the FMA pipe lost 4 to 8 % (d = 128).
//
// Measured: one sequence of 16,384 tokens, 16 heads over 4, causal: 1.04 ms,
// 1,055 TFLOP/s (0.65 of the measured burst peak; clocks fall to 1.53 GHz
// under it), about 3,450 cycles for a pair of steps where the tensor pipe alone
// needs 2,048: each tile's chain of softmax, P V and Q K^T is what remains.
//
// TMEM: S_0 [0,128), S_1 [128,256), O_0 [256,256+d), O_1 [384,384+d).
// Shared memory: Q_0, Q_1, kStages tiles of K or V, 4 KB of output per softmax warp.
//
// Rows of K and V behind the sequence belong to other sequences or to nobody:
// their scores are replaced before use and their V rows are cleared in shared
// memory, so nothing there (infinities, NaN) reaches an output. Rows of O
// behind the sequence are not written.
//
// Every wait is bounded; a CTA that gives up reports through the status word,
// drains its loads and MMAs, frees TMEM and exits.

#include <cudaTypedefs.h>

#include <climits>
#include <mutex>

#include "common.cuh"
#include "ex2_fma.cuh"
#include "launch.cuh"
#include "serving.h"
#include "serving_tc.cuh"

namespace sda {

namespace {

constexpr int kThreads = 384;
constexpr int kTile = 128;  // query rows of a tile, keys of a step
constexpr int kSms = 148;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 * tile
constexpr int kRegsLaunch = 168, kRegsLow = 56, kRegsHigh = 224;
static_assert(kRegsLow * 128 + kRegsHigh * 256 <= kRegsLaunch * kThreads, "register split exceeds the launch");

template <int D>
struct Smem {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kTile * 128;  // [half][128 rows][128 B]
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + 2 * kTileBytes;
  static constexpr int kOut = kRing + kStages * kTileBytes;  // 32 rows x 128 B for each softmax warp
  static constexpr int kBars = kOut + 8 * 4096;
  static constexpr int kTotal = kBars + 512;
};

enum {  // w: tile (two each); an item's barriers two each, by its number
  B_QFULL = 0, B_QFREE = 2, B_SFULL = 4, B_PFULL = 6, B_ODONE = 8, B_OFREE = 10, B_ITEM = 12, B_TAKEN = 14, B_DRAIN = 16,
  B_FULL = 17  // ring full, then ring empty
};
constexpr int kManyTiles = 1 << 24;  // a lane's count of tiles, at most: more than ascending offsets can have
constexpr int kConsumers = 10;  // of an item: loader, MMA warp, 8 softmax warps

// What the CTA works on, found by one warp.
struct Item {
  int valid;
  int q0, nq, k0, nk;  // the sequence's rows of q and of k
  int t;               // row tile within the sequence
};

struct Span {
  int q0, nq, k0, nk;
};

// Sequence s with offsets clamped into the tensors; `bad` when they were not.
__device__ __forceinline__ Span span_of(const Prompt& p, const int32_t* seq_q, const int32_t* seq_k, int s, bool& bad) {
  const int qa = __ldg(seq_q + s), qb = __ldg(seq_q + s + 1), ka = __ldg(seq_k + s), kb = __ldg(seq_k + s + 1);
  Span r;
  r.q0 = min(max(qa, 0), p.rows_q);
  r.nq = min(max(qb, r.q0), p.rows_q) - r.q0;
  r.k0 = min(max(ka, 0), p.rows_k);
  r.nk = min(max(kb, r.k0), p.rows_k) - r.k0;
  bad = bad || r.q0 != qa || r.q0 + r.nq != qb || r.k0 != ka || r.k0 + r.nk != kb;
  return r;
}

// Keys that the rows below `end` of a sequence may see.
__device__ __forceinline__ int keys_below(const Prompt& p, const Span& s, int end) {
  return p.causal ? max(0, min(s.nk, end + s.nk - s.nq)) : s.nk;
}

// Row tiles (of R = 2^lr rows) of a sequence whose key steps number more than x.
__device__ __forceinline__ int tiles_over(const Prompt& p, const Span& s, int lr, int x) {
  const int T = (s.nq + (1 << lr) - 1) >> lr;
  if (x < 0 || T == 0) return T;
  if (!p.causal) return s.nk > kTile * x ? T : 0;
  if (s.nk <= kTile * x) return 0;  // the last tile sees all nk keys, none sees more
  // tile t (not the last) sees (t + 1) R + nk - nq keys
  const int need = kTile * x - (s.nk - s.nq);
  const int first = need < 0 ? 0 : need >> lr;
  return T - min(first, T - 1);
}

// The CTA's row tiles. Tiles go out heaviest first (most key steps), so that
// the last ones to start are short: tile i of the order has the step count x
// with over(x) <= i < over(x - 1), over(x) the number of tiles of more than x
// steps, found by bisection; among equals, sequences in order. A CTA asks for
// ascending i, so the count x and the place among the sequences go on from the
// tile before: the offsets are read a few times for each count that occurs,
// not for each tile (4,096 prompts of 100 tokens, 32 heads over 8, d = 128:
// 2.9 ms, 33.7 with a search of its own for each tile).
struct Search {
  int x, lo, hi;      // the count of tiles lo .. hi - 1 of the order; hi = 0 before the first
  int base, before;   // of them, `before` belong to the sequences before `base`
};
__device__ void find_item(const Prompt& p, const int32_t* seq_q, const int32_t* seq_k, int lr, int i, Search& at, Item* out,
                          bool& bad) {
  const int lane = threadIdx.x & 31;
  Span mine{0, 0, 0, 0};  // of the first 32 sequences
  if (lane < p.n_seq) mine = span_of(p, seq_q, seq_k, lane, bad);
  auto over = [&](int x) {
    int n = lane < p.n_seq ? tiles_over(p, mine, lr, x) : 0;
    for (int s = 32 + lane; s < p.n_seq; s += 32)
      n = min(n + tiles_over(p, span_of(p, seq_q, seq_k, s, bad), lr, x), kManyTiles);
    return __reduce_add_sync(0xffffffffu, n);
  };
  // one lane says that there is none, in order before the lane that finds it: the warp need not be converged
  if (lane == 0) out->valid = 0;
  __syncwarp();
  if (p.n_seq == 1) {  // one sequence: its tiles from the last
    const int T = (mine.nq + (1 << lr) - 1) >> lr;
    if (lane == 0 && i < T) *out = Item{1, mine.q0, mine.nq, mine.k0, mine.nk, T - 1 - i};
    return;
  }
  if (i >= at.hi) {
    int least = 0, most = at.x;  // the next count is one of these
    if (at.hi == 0) {            // the first tile
      int top = lane < p.n_seq ? (mine.nk + kTile - 1) / kTile : 0, sum = top;
      for (int s = 32 + lane; s < p.n_seq; s += 32) {
        const int n = (span_of(p, seq_q, seq_k, s, bad).nk + kTile - 1) / kTile;
        top = max(top, n);
        sum = min(sum + n, kManyTiles);
      }
      most = __reduce_max_sync(0xffffffffu, top);  // over(most) = 0 <= i
      // Ascending offsets leave no more tiles than this. Others are reported by then, and whatever they hold, they do
      // not make the work a multiple of what the tensors have.
      if (__reduce_add_sync(0xffffffffu, sum) > p.rows_k / kTile + p.n_seq || over(-1) > (p.rows_q >> lr) + p.n_seq) return;
    }
    at.hi = over(-1);
    if (i >= at.hi) return;      // behind the last
    while (least < most) {
      const int mid = (least + most) / 2;
      if (over(mid) <= i) most = mid;
      else least = mid + 1;
    }
    at = Search{least, over(least), over(least - 1), 0, 0};
  }
  while (at.base < p.n_seq) {
    const int s = at.base + lane;
    Span sp = at.base == 0 ? mine : Span{0, 0, 0, 0};
    if (at.base > 0 && s < p.n_seq) sp = span_of(p, seq_q, seq_k, s, bad);
    const int above = s < p.n_seq ? tiles_over(p, sp, lr, at.x) : 0;
    const int n = s < p.n_seq ? tiles_over(p, sp, lr, at.x - 1) - above : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    const int rest = i - at.lo - at.before;  // number among the tiles of this count from `base` on
    if (rest >= sum - n && rest < sum) {
      out->q0 = sp.q0;
      out->nq = sp.nq;
      out->k0 = sp.k0;
      out->nk = sp.nk;
      out->t = ((sp.nq + (1 << lr) - 1) >> lr) - 1 - above - (rest - (sum - n));
      out->valid = 1;
    }
    const int all = __shfl_sync(0xffffffffu, sum, 31);
    if (rest < all) break;
    at.before += all;
    at.base += 32;
  }
}

__device__ __forceinline__ uint32_t sw(uint32_t row, uint32_t chunk) { return tc::sw128_offset(row, chunk); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prompt_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, Prompt p, int pair_heads,
                   const int32_t* __restrict__ seq_q, const int32_t* __restrict__ seq_k, uint16_t* __restrict__ o,
                   float* __restrict__ lse, unsigned* status, uint64_t wait_ns) {
  using S = Smem<D>;
  constexpr int NS = S::kStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* full = bars + B_FULL;
  uint64_t* empty = full + NS;
  unsigned char* tail = smem + S::kBars + 8 * (B_FULL + 2 * NS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 4);
  Item* items = reinterpret_cast<Item*>(tail + 16);  // two

  // through a shuffle, so that the compiler knows it to be the same for the warp
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int groups = pair_heads ? p.H / 2 : p.H;  // head groups, fastest: they share the tile's K and V through L2

  if (threadIdx.x == 0) {
    for (int w = 0; w < 2; ++w) {
      tc::mbar_init(&bars[B_QFULL + w], 1);
      tc::mbar_init(&bars[B_QFREE + w], 1);
      tc::mbar_init(&bars[B_SFULL + w], 1);
      tc::mbar_init(&bars[B_PFULL + w], 4);  // a warp each
      tc::mbar_init(&bars[B_ODONE + w], 1);
      tc::mbar_init(&bars[B_OFREE + w], 4);
      tc::mbar_init(&bars[B_ITEM + w], 1);
      tc::mbar_init(&bars[B_TAKEN + w], kConsumers);
    }
    tc::mbar_init(&bars[B_DRAIN], 1);
    for (int s = 0; s < NS; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::fence_mbar_init();
    tc::tma_prefetch(&tm_q);
    tc::tma_prefetch(&tm_k);
    tc::tma_prefetch(&tm_v);
  }
  if (warp == 3) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::fence_before_sync();
  }
  pdl_wait();
  if (threadIdx.x == 0) *abort_flag = (*reinterpret_cast<volatile unsigned*>(status) & kStatusTimeout) ? 1 : 0;
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  if (*abort_flag) {  // uniform
    if (warp == 3) tc::tmem_dealloc(tmem, kTmemCols);
    return;
  }

  // Item r of this CTA: the items go out in rounds, every second one in reverse, so that each CTA's share is even.
  auto number = [&](int r) {
    const int c = (r & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
    return static_cast<long long>(r) * gridDim.x + c;
  };
  // What a role needs to know of item r: waits for it, copies it, hands its place back.
  struct Work {
    Span seq;
    int row0, row_1, n0, n1, n, h0;
    bool live_1;
  };
  bool ok = true;
  auto take = [&](int r, Work& k) {  // a whole warp
    ok = tc::wait_warp(&bars[B_ITEM + (r & 1)], (r >> 1) & 1, abort_flag, wait_ns);
    if (!ok) return false;
    const Item it = items[r & 1];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&bars[B_TAKEN + (r & 1)]);
    if (!it.valid) return false;
    const int hg = static_cast<int>(number(r) % groups);
    k.seq = Span{it.q0, it.nq, it.k0, it.nk};
    k.row0 = it.t * (pair_heads ? kTile : 2 * kTile);
    k.h0 = pair_heads ? 2 * hg : hg;
    // tile w: rows [row_w, end_w) of the sequence, head h_w, steps n_w (0: nothing visible)
    k.row_1 = pair_heads ? k.row0 : k.row0 + kTile;
    k.live_1 = k.row_1 < it.nq;
    k.n0 = (keys_below(p, k.seq, min(k.row0 + kTile, it.nq)) + kTile - 1) / kTile;
    k.n1 = k.live_1 ? (keys_below(p, k.seq, min(k.row_1 + kTile, it.nq)) + kTile - 1) / kTile : 0;
    k.n = max(k.n0, k.n1);
    return true;
  };
  const int g = p.H / p.H_kv;
  Work k;

  if (warp < 4) {
    tc::setmaxnreg_dec<kRegsLow>();
    volatile int never = 0;
    if (warp == 0) {
      // ------------------------------------------------------------ loads
      int cnt = 0;                  // ring tiles so far
      int q_cnt[2] = {0, 0};        // Q tiles so far
      for (int r = 0; take(r, k); ++r) {
        if (lane == 0) {
          for (int w = 0; w < 2 && ok; ++w) {
            if ((w ? k.n1 : k.n0) == 0) continue;
            if (q_cnt[w] > 0) ok = tc::wait1(&bars[B_QFREE + w], (q_cnt[w] - 1) & 1, abort_flag, wait_ns);
            if (!ok) break;
            tc::mbar_arrive_expect_tx(&bars[B_QFULL + w], S::kTileBytes);
            for (int hf = 0; hf < S::kHalves; ++hf)
              tc::tma_load_3d(smem + S::kQ + w * S::kTileBytes + hf * kTile * 128, &tm_q, &bars[B_QFULL + w], 64 * hf,
                              pair_heads ? k.h0 + w : k.h0, k.seq.q0 + (w ? k.row_1 : k.row0));
            ++q_cnt[w];
          }
          // ring order K_0, V_0, K_1, V_1, ...: the order in which the MMAs release them
          for (int c = 0; c < 2 * k.n && ok; ++c) {
            const int st = cnt % NS;
            if (cnt >= NS) ok = tc::wait1(&empty[st], (cnt / NS - 1) & 1, abort_flag, wait_ns);
            if (!ok) break;
            tc::mbar_arrive_expect_tx(&full[st], S::kTileBytes);
            for (int hf = 0; hf < S::kHalves; ++hf)
              tc::tma_load_3d(smem + S::kRing + st * S::kTileBytes + hf * kTile * 128, c % 2 == 0 ? &tm_k : &tm_v, &full[st],
                              64 * hf, k.h0 / g, k.seq.k0 + c / 2 * kTile);
            ++cnt;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0);
        if (!ok) break;
      }
      // no load is in flight when the CTA ends, whatever the others did
      if (lane == 0) {
        for (int w = 0; w < 2; ++w)
          if (q_cnt[w] > 0) tc::wait1(&bars[B_QFULL + w], (q_cnt[w] - 1) & 1, &never);
        for (int b = cnt > NS ? cnt - NS : 0; b < cnt; ++b) tc::wait1(&full[b % NS], (b / NS) & 1, &never);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issue
      // The whole warp walks the loop, so that descriptors and addresses are uniform values; one lane issues. With
      // one lane in a branch of its own they were moved between register files for every MMA, and the pipe waited
      // for them (a pair of steps took 3,880 cycles, 3,350 like this).
      constexpr uint32_t idesc_qk = tc::idesc_bf16(128, 128, false);
      constexpr uint32_t idesc_pv = tc::idesc_bf16(128, D, true);  // B = V, MN-major
      const uint32_t leader = lane == 0;
      const uint64_t desc_k0 = tc::smem_desc_sw128(smem + S::kRing, 16, 1024);           // K: K-major
      const uint64_t desc_v0 = tc::smem_desc_sw128(smem + S::kRing, kTile * 128, 1024);  // V: MN-major
      const uint64_t desc_q0 = tc::smem_desc_sw128(smem + S::kQ, 16, 1024);
      constexpr uint32_t kTile16 = S::kTileBytes / 16, kHalf16 = kTile * 128 / 16;       // descriptors count in 16 bytes
      auto wait = [&](uint64_t* bar, uint32_t parity) { return tc::wait_warp(bar, parity, abort_flag, wait_ns); };
      auto qk = [&](int w, int st) {
        const uint64_t da = desc_q0 + w * kTile16, db = desc_k0 + st * kTile16;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t at = kk / 4 * kHalf16 + kk % 4 * 2;
          tc::mma_ss_by(leader, tmem + kColS + 128 * w, da + at, db + at, idesc_qk, kk > 0 ? 1u : 0u);
        }
        tc::commit_by(leader, &bars[B_SFULL + w]);
      };
      auto pv = [&](int w, int st, uint32_t acc) {
        const uint64_t db = desc_v0 + st * kTile16;
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          tc::mma_ts_by(leader, tmem + kColO + 128 * w, tmem + kColS + 128 * w + kk * 8, db + kk * 128, idesc_pv,
                        kk > 0 ? 1u : acc);
      };
      // place in the ring of the next tile, its stage and parity; counts of each tile's items and steps so far
      int st = 0, par = 0;
      uint32_t q_par[2] = {0, 0}, p_par[2] = {0, 0}, o_cnt[2] = {0, 0};
      auto advance = [&](int& s_, int& p_, int by) {
        s_ += by;
        if (s_ >= NS) s_ -= NS, p_ ^= 1;
      };
      for (int r = 0; take(r, k); ++r) {
        const int n = __shfl_sync(0xffffffffu, k.n, 0), m0 = __shfl_sync(0xffffffffu, k.n0, 0),
                  m1 = __shfl_sync(0xffffffffu, k.n1, 0), nk = __shfl_sync(0xffffffffu, k.seq.nk, 0);
        if (n == 0) continue;
        ok = wait(&full[st], par);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (!ok || (w ? m1 : m0) == 0) continue;
          ok = wait(&bars[B_QFULL + w], q_par[w]);
          q_par[w] ^= 1;
          tc::fence_after_sync();
          if (ok) {
            qk(w, st);
            if ((w ? m1 : m0) == 1) tc::commit_by(leader, &bars[B_QFREE + w]);
          }
        }
        if (!ok) break;
        tc::commit_by(leader, &empty[st]);
        advance(st, par, 1);
        int sv = st, v_par = par, sk = st, k_par = par;  // V_j and K_{j+1}
        advance(sk, k_par, 1);
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
          ok = wait(&full[sv], v_par);
          if (ok && j + 1 < n) ok = wait(&full[sk], k_par);
          if (!ok) break;
          const int there = nk - j * kTile;
          if (j == n - 1 && there < kTile) {  // the last tile: clear the V rows behind the sequence
            unsigned char* vst = smem + S::kRing + sv * S::kTileBytes;
            for (int e = there * 8 * S::kHalves + lane; e < kTile * 8 * S::kHalves; e += 32) {
              const int row = e / (8 * S::kHalves), ch = e % (8 * S::kHalves);
              *reinterpret_cast<uint4*>(vst + (ch / 8) * kTile * 128 + row * 128 + (ch % 8) * 16) = make_uint4(0, 0, 0, 0);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
          }
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int nw = w ? m1 : m0;
            if (j >= nw) continue;
            if (j == 0 && o_cnt[w] > 0) ok = wait(&bars[B_OFREE + w], (o_cnt[w] - 1) & 1);  // the last item's output is out
            if (ok) ok = wait(&bars[B_PFULL + w], p_par[w]);
            if (!ok) break;
            p_par[w] ^= 1;
            tc::fence_after_sync();
            pv(w, sv, j > 0);
            if (j == nw - 1) {
              tc::commit_by(leader, &bars[B_ODONE + w]);
              ++o_cnt[w];
            } else {
              qk(w, sk);
              if (j + 1 == nw - 1) tc::commit_by(leader, &bars[B_QFREE + w]);
            }
          }
          if (!ok) break;
          tc::commit_by(leader, &empty[sv]);
          if (j + 1 < n) tc::commit_by(leader, &empty[sk]);
          advance(sv, v_par, 2);
          advance(sk, k_par, 2);
        }
        if (!ok) break;
        // 2 n tiles of the item, one of them taken above
        for (int left = 2 * n - 1; left > 0; left -= NS) advance(st, par, left < NS ? left : NS);
      }
      // drain: every MMA this warp issued
      tc::commit_by(leader, &bars[B_DRAIN]);
      tc::wait_warp(&bars[B_DRAIN], 0, &never);
    } else if (warp == 2) {
      // ------------------------------------------------------------ items, one ahead of their use
      Search at{0, 0, 0, 0, 0};
      for (int r = 0;; ++r) {
        if (r >= 2) ok = tc::wait_warp(&bars[B_TAKEN + (r & 1)], ((r >> 1) - 1) & 1, abort_flag, wait_ns);
        if (!ok) break;
        bool bad = false;
        const long long tile = number(r) / groups;
        find_item(p, seq_q, seq_k, pair_heads ? 7 : 8, static_cast<int>(min(tile, static_cast<long long>(INT_MAX))),
                  at, &items[r & 1], bad);
        if (r == 0 && blockIdx.x == 0 && __any_sync(0xffffffffu, bad) && lane == 0) report_status(status, kStatusBadIndex);
        __syncwarp();
        const int valid = *reinterpret_cast<volatile int*>(&items[r & 1].valid);
        if (lane == 0) tc::mbar_arrive(&bars[B_ITEM + (r & 1)]);
        if (!valid) break;
      }
    }
  } else {
    tc::setmaxnreg_inc<kRegsHigh>();
    // ------------------------------------------------------------ softmax of tile w, epilogue
    const int w = warp < 8 ? 0 : 1;
    const int quarter = warp & 3;
    const int row = 32 * quarter + lane;
    const uint32_t lane_base = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t t_s = tmem + lane_base + kColS + 128 * w;
    const uint32_t t_o = tmem + lane_base + kColO + 128 * w;
    uint32_t s_par = 0, o_par = 0;  // parities of S and O
    for (int r = 0; take(r, k); ++r) {
    const Span seq = k.seq;
    const int nw = w ? k.n1 : k.n0;
    const int tile_row = w ? k.row_1 : k.row0;
    const int my_row = tile_row + row;               // row of the sequence
    const int lim = keys_below(p, seq, my_row + 1);  // keys this row sees (rows behind the sequence: all)
    const int lim_first = keys_below(p, seq, tile_row + 1);
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < nw; ++j) {
      ok = tc::wait_warp(&bars[B_SFULL + w], s_par, abort_flag, wait_ns);
      if (!ok) break;
      s_par ^= 1;
      tc::fence_after_sync();
      float s[128];
      {
        uint32_t sr[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_ld32p(t_s + 32 * c, sr + 32 * c);
        tc::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = __uint_as_float(sr[c]);
      }
      if ((j + 1) * kTile > lim_first) {  // some row of the tile does not see all of the step's keys
        const int vis = lim - j * kTile;
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = c < vis ? s[c] : -INFINITY;
      }
      auto row_max = [&] {
        float a0 = fmaxf(s[0], s[1]), a1 = fmaxf(s[2], s[3]), a2 = fmaxf(s[4], s[5]), a3 = fmaxf(s[6], s[7]);
#pragma unroll
        for (int c = 8; c < 128; c += 8) {
          a0 = max3(a0, s[c], s[c + 1]);
          a1 = max3(a1, s[c + 2], s[c + 3]);
          a2 = max3(a2, s[c + 4], s[c + 5]);
          a3 = max3(a3, s[c + 6], s[c + 7]);
        }
        return max3(a0, a1, fmaxf(a2, a3)) * p.scale_log2;
      };
      if (j == 0) m = row_max();
      // The exponentials begin with the reference so far; whether the step's maximum is within 2^8 of it is seen
      // under their latency, and if it is not (rarely) they are taken again.
      const uint64_t sc2 = f2(p.scale_log2, p.scale_log2);
      for (;;) {
        const float mref = (m == -INFINITY) ? 0.f : m;
        const uint64_t nm2 = f2(-mref, -mref);
        uint64_t acc0 = f2(0.f, 0.f), acc1 = f2(0.f, 0.f);
        float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int c = 16 * ch + e;  // key pair 2c, 2c + 1
            float x0, x1;
            f2_split(fma2(f2(s[2 * c], s[2 * c + 1]), sc2, nm2), x0, x1);
            const float p0 = tc::ex2(x0), p1 = tc::ex2(x1);  // 2^-inf = 0 on hidden keys
            if (e & 1) {
              acc1 = add2(acc1, f2(p0, p1));
              a1 = max3(a1, s[2 * c], s[2 * c + 1]);
            } else {
              acc0 = add2(acc0, f2(p0, p1));
              a0 = max3(a0, s[2 * c], s[2 * c + 1]);
            }
            pk[e] = pack_bf16(p0, p1);
          }
          tc::tmem_st16p(t_s + 16 * ch, pk);
        }
        const float mx = fmaxf(a0, a1) * p.scale_log2;
        const bool grow = mx > m + 8.0f;
        if (__any_sync(0xffffffffu, grow)) {
          // S_w(j) ready: PV_w(j - 1) is done and O_w rests (there is none yet at j = 0, and no growth)
          const float alpha = !grow ? 1.f : (m == -INFINITY ? 0.f : tc::ex2(m - mx));
          if (grow) {
            l *= alpha;
            m = mx;
          }
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t r[16];
            tc::tmem_ld16p(t_o + 16 * c, r);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tc::tmem_st16p(t_o + 16 * c, r);
          }
          continue;
        }
        float r0, r1;
        f2_split(add2(acc0, acc1), r0, r1);
        l += r0 + r1;
        break;
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars[B_PFULL + w]);
    }
    if (!ok) break;
    const bool live = w == 0 || k.live_1;
    if (nw > 0) {
      ok = tc::wait_warp(&bars[B_ODONE + w], o_par, abort_flag, wait_ns);
      if (!ok) break;
      o_par ^= 1;
    }
    if (live) {
      tc::fence_after_sync();
      const int head = pair_heads ? k.h0 + w : k.h0;
      const bool mine = my_row < seq.nq;
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // a NaN sum stays NaN
      if (lse != nullptr && mine)
        lse[static_cast<size_t>(seq.q0 + my_row) * p.H + head] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      // O / l as bf16, 64 channels at a time, through this warp's 32 x 128 B, then whole rows out
      unsigned char* out = smem + S::kOut + (warp - 4) * 4096;
#pragma unroll
      for (int hf = 0; hf < S::kHalves; ++hf) {
        uint32_t x[64];
        if (nw > 0) {
          tc::tmem_ld32p(t_o + 64 * hf, x);
          tc::tmem_ld32p(t_o + 64 * hf + 32, x + 32);
          tc::tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 64; ++e) x[e] = 0u;
        }
        if (hf == S::kHalves - 1 && nw > 0) {  // O_w is in registers: the next item may overwrite it
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bars[B_OFREE + w]);
        }
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = pack_bf16(__uint_as_float(x[8 * ch + 2 * e]) * inv, __uint_as_float(x[8 * ch + 2 * e + 1]) * inv);
          *reinterpret_cast<uint4*>(out + sw(lane, ch)) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        __syncwarp();
        const int ch = lane % 8;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const int rr = i + lane / 8, at = tile_row + 32 * quarter + rr;
          if (at < seq.nq) {
            const uint4 v = *reinterpret_cast<const uint4*>(out + sw(rr, ch));
            *reinterpret_cast<uint4*>(o + static_cast<size_t>(seq.q0 + at) * p.ld_o + head * D + 64 * hf + 8 * ch) = v;
          }
        }
        __syncwarp();
      }
    }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) report_status(status, kStatusTimeout);
  if (warp == 3) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
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

// [rows, heads, d] bf16, rows `ld` elements apart, as (d, heads, rows); box = 64 channels x 128 rows of one head.
bool make_map(CUtensorMap* map, const void* base, int d, int heads, int rows, long long ld) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[3] = {64, 1, kTile};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t run(const Prompt& p, const uint16_t* q, const uint16_t* k, const uint16_t* v, const int32_t* seq_q,
                const int32_t* seq_k, uint16_t* o, float* lse, unsigned* status, cudaStream_t stream) {
  if (encode_fn() == nullptr) return cudaErrorNotSupported;
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, q, D, p.H, p.rows_q, p.ld_q) || !make_map(&mk, k, D, p.H_kv, p.rows_k, p.ld_k) ||
      !make_map(&mv, v, D, p.H_kv, p.rows_k, p.ld_v))
    return cudaErrorInvalidValue;
  const int smem = Smem<D>::kTotal + 1024;
  cudaError_t e = cudaFuncSetAttribute(prompt_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // setmaxnreg.inc waits until the block's registers can serve it: refuse a build that would leave it short
  static int regs = -1;
  if (regs < 0) {
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, prompt_attn_kernel<D>);
    if (e != cudaSuccess) return e;
    regs = attr.numRegs;
  }
  if (regs * kThreads < kRegsLow * 128 + kRegsHigh * 256) return cudaErrorInvalidConfiguration;
  const int pair_heads = (p.H / p.H_kv) % 2 == 0 ? 1 : 0;
  const int R = pair_heads ? kTile : 2 * kTile;
  const long long tiles = static_cast<long long>(p.rows_q) / R + p.n_seq;  // at least the sequences' row tiles
  const long long most = tiles * (pair_heads ? p.H / 2 : p.H), blocks = min(most, static_cast<long long>(kSms));
  return launch_after(prompt_attn_kernel<D>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), smem, stream, mq, mk, mv, p,
                      pair_heads, seq_q, seq_k, o, lse, status, serving_wait_limit());
}

}  // namespace

cudaError_t launch_prompt_attn(const Prompt& p, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                               const int32_t* seq_q, const int32_t* seq_k, uint16_t* o, float* lse, unsigned* status,
                               cudaStream_t stream) {
  if (p.d == 128) return run<128>(p, q, k, v, seq_q, seq_k, o, lse, status, stream);
  if (p.d == 64) return run<64>(p, q, k, v, seq_q, seq_k, o, lse, status, stream);
  return cudaErrorInvalidValue;
}

}  // namespace sda
