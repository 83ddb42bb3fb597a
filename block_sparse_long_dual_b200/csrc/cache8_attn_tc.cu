// Attention of a few query rows over the whole 8-bit KV cache on the sm_100a
// tensor cores (the first of the two steps: pieces; cache8_attn.cu joins them).
//
// The codes go to the tensor core as they are (kind::f8f6f4), so no cached value
// is converted by a thread.  Per 128 tokens:
//   S^T [128 tokens, 2 NC] = K [128, D] . Q^T     Q: NC query rows (the group's heads x query tokens)
//   O^T [D, 2 NC]          = V^T [D, 128] . P^T
// A bf16 query row or a float32 probability does not fit 4 significant bits, so
// each takes two columns: x = hi + lo / 2^k, hi = e4m3(x), lo = e4m3((x - hi) 2^k).
// A query row is scaled so that its largest element lies in (224, 448]; with k = 4 the
// two parts end at steps of 2^-13, so a bf16 element of at least 2^-6 (2^-13 of the
// largest is always enough) is exact and a smaller one off by 2^-14 at most, under
// 2^-21 of the largest.  Probabilities are scaled to 256 for their block's largest; with
// k = 5 the parts are off by 2^-9 of the value at most (the width of bf16), or by half a
// step of 2^-22 of the block's largest where that is more.  The rounding is unbiased and
// only O sees it: the sum that divides O, lse and the weights take the probabilities as
// computed.  It brings O's error against 64 bits from 1.67e-3 (the bf16 output's own
// rounding) to 1.73e-3, over 32768 tokens of normal values.  (A third part would take a
// stage of the rings at d 64.)  The products' sums, scores, maxima, sums and O are float32.
//
// Each scale block has its own reference maximum and, in TMEM, its own O^T, so
// scales that lie far apart between blocks lose nothing: the block's factor
// 2^(max - running max) * v_scale is applied when O^T is added to the registers.
//
//   warps 0 .. 3  thread i = token i of the tile for S (TMEM lane i; i and i + 128 in
//                 tiles of 256): scores, block maxima (warp maxima through shared
//                 memory), probabilities as e4m3 into shared memory; thread r = dim r
//                 for O^T: the running O of the piece in registers.  O^T of tile j - 1
//                 is added after the probabilities of tile j are on their way.
//   warp 4        O's factors of each tile, out of the way of the softmax warps, and the
//                 producer: TMA tiles of K and V (a ring each)
//   warp 5        MMA issuer
// A tile is 32 KB (128 tokens of d = 128, 256 of d = 64: with 128 tokens the softmax
// warps, a chain of latencies, set the pace of the smaller rows) and 8 to 12 MMAs of
// N = 2 NC; the tensor core is idle most of the time and the kernel's bound is the
// cache's bytes: 16 x 8 heads x 32768 tokens, d 128, 4 rows: 160 us for 1074 MB, 6.7
// TB/s (102% of the measured copy rate, which writes half its bytes); d 64 with 8 rows
// 5.0 - 5.3 TB/s and with 16 rows 3.8, bound by the softmax warps.  144 to 168 registers;
// 16 rows of d 64 over 64-token blocks spill 12 bytes a thread.  Work split, pieces and
// their slots: cache8.cuh.  Every wait is bounded; one that runs out sets
// SFA_ERR_TIMEOUT and an abort flag, after which waits return at once and the CTA runs
// to its end (the copies and MMAs it issued are drained).
#include <cuda.h>
#include <float.h>
#include <math.h>

#include "cache8.cuh"
#include "tc_ptx8.cuh"

namespace sfa {

namespace {

using namespace c8;

constexpr int kTileThreads = 192;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kEdge = kMaxCols - 1;  // tokens that not every query sees: nq - 1 at most
constexpr float kLoQ = 16.f, kLoP = 32.f, kTopP = 256.f;

template <int D, int NC, int T>
struct Lay {
  static constexpr int N = 2 * NC;                   // MMA columns
  static constexpr int TILE_T = tile_tokens(D, NC);  // tokens of a tile
  static constexpr int H = TILE_T / 128;             // tokens per softmax thread
  static constexpr int SUBH = 128 / T;               // scale blocks of 128 tokens
  static constexpr int SUB = H * SUBH;               // and of a tile
  static constexpr uint32_t TILE = TILE_T * D;       // bytes of a K or V tile
  static constexpr int STAGES = 49152 / TILE;        // 48 KB each for K and V
  static constexpr int NK = STAGES, NV = NC == 8 ? STAGES : STAGES - STAGES / 3;  // 16 rows leave less room
  static constexpr uint32_t QB = N * D, PB = TILE_T * N;
  static constexpr uint32_t OFF_K = 0, OFF_V = NK * TILE;
  static constexpr uint32_t OFF_Q = (NK + NV) * TILE;                // two buffers
  static constexpr uint32_t OFF_P = OFF_Q + 2 * QB;                  // two buffers
  static constexpr uint32_t OFF_EV = OFF_P + 2 * PB;                 // edge tokens' V rows, two buffers
  static constexpr uint32_t OFF_EE = OFF_EV + 2 * kEdge * D;         // their probabilities [2][kEdge][NC]
  static constexpr uint32_t OFF_MAX = OFF_EE + 2 * kEdge * NC * 4;   // warp maxima [2][H][4][NC]
  static constexpr uint32_t OFF_FAC = OFF_MAX + 2 * H * 4 * NC * 4;  // [2][NC] keep, [2][SUB][NC] f,
                                                                     // [2][SUB][NC] f v, [NC] running maxima
  static constexpr uint32_t OFF_QF = OFF_FAC + NC * (3 + 4 * SUB) * 4;  // row factors [2][NC]
  static constexpr uint32_t OFF_BACK = OFF_QF + 2 * NC * 4;          // newest tokens that a row does not see [NC]
  static constexpr uint32_t OFF_BAR = OFF_BACK + NC * 4;
  static constexpr int B0 = NK + NV, NBAR = B0 + 9;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr uint32_t BYTES = OFF_MISC + 128 + 1024;
  // TMEM columns: S two buffers of H parts, O two buffers of SUB parts
  static constexpr uint32_t COL_O = 2 * H * N, COLS_USED = COL_O + 2 * SUB * N;
  static constexpr uint32_t TMEM = COLS_USED <= 64 ? 64 : (COLS_USED <= 128 ? 128 : 256);
  __host__ __device__ static constexpr int kf(int s) { return s; }
  __host__ __device__ static constexpr int vf(int s) { return NK + s; }
  __host__ __device__ static constexpr int sf(int b) { return B0 + b; }
  __host__ __device__ static constexpr int pf(int b) { return B0 + 2 + b; }
  __host__ __device__ static constexpr int of(int b) { return B0 + 4 + b; }
  __host__ __device__ static constexpr int qf(int b) { return B0 + 6 + b; }
  static constexpr int DRAIN = B0 + 8;
};

struct Ctx {
  uint32_t bars;
  volatile int* abort_flag;
  int* status;
  __device__ __forceinline__ uint32_t bar(int k) const { return bars + 8u * k; }
};

__device__ __noinline__ bool wait_slow(const Ctx& c, uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (*c.abort_flag) return false;
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0 && globaltimer_ns() - t0 > kTimeoutNs) {
      *c.abort_flag = 1;
      report(c.status, SFA_ERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(const Ctx& c, uint32_t bar, uint32_t parity) {
  return tc::mbar_try_wait(bar, parity) || wait_slow(c, bar, parity);
}
__device__ void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!tc::mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > kTimeoutNs) return;
}

// The pieces of a CTA's share, in order.
template <int TILE_T>
struct Pieces {
  int left;                   // tiles of the share after the present piece
  int b, g, nv, first, last;  // unit (b, g), its visible tokens, the piece's tiles [first, last)

  // `skip`: tiles of sequence b0 before the share; nv0: its visible tokens.
  __device__ void begin(int b0, int skip, int nv0, int n) {
    b = b0;
    nv = nv0;
    const int tiles = (nv + TILE_T - 1) / TILE_T;
    g = skip / tiles;
    first = skip % tiles;
    last = min(tiles, first + n);
    left = n - (last - first);
  }
  __device__ bool next(const Cache8Attn& p) {
    if (left <= 0) return false;
    int tiles = (nv + TILE_T - 1) / TILE_T;
    if (++g == p.Hkv) {
      g = 0;
      do {
        if (++b >= p.B) {  // only if the lengths changed under the call
          left = 0;
          return false;
        }
        nv = visible(p.lens, b, p.L, p.back, nullptr);
        tiles = (nv + TILE_T - 1) / TILE_T;
      } while (tiles == 0);
    }
    first = 0;
    last = min(tiles, left);
    left -= last;
    return true;
  }
};

// NC consecutive floats of shared memory, 16 bytes a load.
template <int NC>
__device__ __forceinline__ void load_row(const float* p, float (&v)[NC]) {
#pragma unroll
  for (int c = 0; c < NC; c += 4) {
    const float4 u = *reinterpret_cast<const float4*>(p + c);
    v[c] = u.x; v[c + 1] = u.y; v[c + 2] = u.z; v[c + 3] = u.w;
  }
}

// The same as packed pairs (float32 pair arithmetic: half the instructions of the tile loop's sums and products).
template <int NC>
__device__ __forceinline__ void load_pairs(const float* p, uint64_t (&v)[NC / 2]) {
#pragma unroll
  for (int c = 0; c < NC; c += 4) {
    const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(p + c);
    v[c / 2] = u.x;
    v[c / 2 + 1] = u.y;
  }
}
__device__ __forceinline__ uint64_t pair(float x) { return tc::f2_pack(x, x); }
__device__ __forceinline__ uint64_t pair_bits(uint32_t a, uint32_t b) {
  return tc::f2_pack(__uint_as_float(a), __uint_as_float(b));
}

// Sums of NC values over the warp, each lane left with the sum of one row (*row): halves are exchanged, then quarters...
template <int NC>
__device__ __forceinline__ float warp_row_sums(float (&x)[NC], int* row) {
  const int lane = threadIdx.x & 31;
  int r = 0, m = 16;
#pragma unroll
  for (int w = NC / 2; w >= 1; w /= 2, m /= 2) {
    const bool up = (lane & m) != 0;
#pragma unroll
    for (int c = 0; c < w; ++c) {
      const float give = up ? x[c] : x[c + w], own = up ? x[c + w] : x[c];
      x[c] = own + __shfl_xor_sync(0xffffffffu, give, m);
    }
    r += up ? w : 0;
  }
#pragma unroll
  for (; m >= 1; m /= 2) x[0] += __shfl_xor_sync(0xffffffffu, x[0], m);
  *row = r;
  return x[0];
}

template <int N>
__device__ __forceinline__ void tmem_row(uint32_t at, uint32_t (&v)[N]) {
  static_assert(N == 16 || N == 32, "two columns a query row");
  if constexpr (N == 16) tc::tmem_ld16(at, v);
  else tc::tmem_ld32(at, v);
}

// The softmax warps; and with the factor warp: once a tile, and once at a piece's end.
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ void tile_sync() { asm volatile("bar.sync 2, 160;" ::: "memory"); }

// The share's tiles one by one: first row of each in the code arrays.
template <int TILE_T>
struct TileRows {
  Pieces<TILE_T> pc;
  int tile;
  __device__ int take(const Cache8Attn& p) {
    if (tile == pc.last) {
      pc.next(p);
      tile = pc.first;
    }
    return (pc.b * p.Hkv + pc.g) * p.L + TILE_T * tile++;
  }
};

// Query rows of one unit as two e4m3 parts: B operand, K-major, no swizzle (8 rows x 16 bytes contiguous).
template <int D, int NC, int T>
__device__ __forceinline__ void write_q(const Cache8Attn& p, unsigned char* sm, int buf, int unit, int tid) {
  using L = Lay<D, NC, T>;
  constexpr int TPR = 128 / NC, DPT = D / TPR;  // threads per row, dims per thread
  const int c = tid / TPR, part = tid % TPR;
  float x[DPT];
#pragma unroll
  for (int e = 0; e < DPT; ++e) x[e] = 0.f;
  if (c < p.cols) {
    const uint2* src = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                      ((size_t)unit * p.cols + c) * D + part * DPT);
#pragma unroll
    for (int e = 0; e < DPT / 4; ++e) {
      const uint2 u = __ldg(src + e);
      x[4 * e] = __uint_as_float(u.x << 16);
      x[4 * e + 1] = __uint_as_float(u.x & 0xFFFF0000u);
      x[4 * e + 2] = __uint_as_float(u.y << 16);
      x[4 * e + 3] = __uint_as_float(u.y & 0xFFFF0000u);
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < DPT; ++e) {
    if (isfinite(x[e])) top = max(top, __float_as_uint(fabsf(x[e])));
    else x[e] = NAN;
  }
#pragma unroll
  for (int o = TPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int ex = need_exp(top);
  const float inv = pow2i(-ex);
  unsigned char* q = sm + L::OFF_Q + buf * L::QB;
#pragma unroll
  for (int e = 0; e < DPT; e += 2) {
    const float a = x[e] * inv, b = x[e + 1] * inv;
    const uint32_t hi = to_e4m3x2(a, b);
    const float2 h = __half22float2(from_e4m3x2(hi));
    const uint32_t lo = to_e4m3x2((a - h.x) * kLoQ, (b - h.y) * kLoQ);
    const int k = part * DPT + e;
    auto at = [&](int r) { return (r >> 3) * (D * 8) + (k >> 4) * 128 + (r & 7) * 16 + (k & 15); };
    *reinterpret_cast<uint16_t*>(q + at(c)) = (uint16_t)hi;
    *reinterpret_cast<uint16_t*>(q + at(NC + c)) = (uint16_t)lo;
  }
  if (part == 0) reinterpret_cast<float*>(sm + L::OFF_QF)[buf * NC + c] = pow2i(ex) * p.sl2;
}

template <int D, int NC, int T>
__global__ void __launch_bounds__(kTileThreads, kCtasPerSm)
    attn_tile_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ Cache8Attn p) {
  using L = Lay<D, NC, T>;
  constexpr int N = L::N, H = L::H, SUB = L::SUB, SUBH = L::SUBH, NK = L::NK, NV = L::NV, TILE_T = L::TILE_T;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = tc::smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  unsigned char* sm = smem_raw + pad;
  const uint32_t sb = raw + pad;
  int* sched = reinterpret_cast<int*>(sm + L::OFF_MISC);  // first sequence, its tiles before the share, the
                                                          // share's tiles, the sequence's visible tokens
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::OFF_MISC + 28);
  // The piece after the present one, [2][6]: whether there is one, b, g, nv, first, last.  Warp 4 alone reads the
  // lengths for it: the warps that meet at tile_sync have to agree on the pieces even if the lengths changed under
  // the call.
  int* follow = reinterpret_cast<int*>(sm + L::OFF_MISC + 64);
  Ctx cx;
  cx.bars = sb + L::OFF_BAR;
  cx.abort_flag = reinterpret_cast<volatile int*>(sm + L::OFF_MISC + 32);
  cx.status = p.status;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining step waits for this grid's end itself
  if (warp == 0) {
    int b, skip;
    const int n = warp_share(p.lens, p.B, p.Hkv, p.L, p.back, TILE_T, p.G, blockIdx.x, &b, &skip,
                             blockIdx.x == 0 ? p.status : nullptr);
    if (lane == 0) {
      sched[0] = b;
      sched[1] = skip;
      sched[2] = n;
      sched[3] = visible(p.lens, b, p.L, p.back, nullptr);
    }
  } else if (warp == 4 && lane == 0) {
    *cx.abort_flag = 0;
    for (int k = 0; k < L::NBAR; ++k)
      tc::mbar_init(cx.bar(k), k == L::pf(0) || k == L::pf(1) || k == L::qf(0) || k == L::qf(1) ? 128 : 1);
    tc::fence_mbar_init();
    tc::prefetch_tmap(&tmK);
    tc::prefetch_tmap(&tmV);
  } else if (warp == 1) {
    if (lane < NC) reinterpret_cast<int*>(sm + L::OFF_BACK)[lane] = p.nq - 1 - lane % p.nq;
  } else if (warp == 5) {
    tc::tmem_alloc(tc::smem_u32(tmem_slot), L::TMEM);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n = sched[2];

  if (n > 0) {
    Pieces<TILE_T> pc;
    pc.begin(sched[0], sched[1], sched[3], n);
    if (warp == 4) {
      // ------------------------ factors and copies --------------------------
      const float* smax = reinterpret_cast<const float*>(sm + L::OFF_MAX);
      float* fkeep = reinterpret_cast<float*>(sm + L::OFF_FAC);
      float* ff = fkeep + 2 * NC;
      float* ffv = ff + 2 * SUB * NC;
      float* fmax_row = ffv + 2 * SUB * NC;
      constexpr int WPS = T / 32;  // warps per scale block
      const int fc = lane % NC, fs = lane / NC;  // this lane: row fc, scale block fs of the tile
      const bool mine = fs < SUB;
      TileRows<TILE_T> kr{pc, pc.first}, vr{pc, pc.first};
      const uint64_t once = tc::policy_evict_first();  // leaves L2 to the scores, queries and pieces (2%)
      const uint32_t tiles = (uint32_t)n;
      uint32_t nk = 0, nv = 0;  // K and V tiles whose copy has been started (lane 0)
      auto load_k = [&] {
        const uint32_t s = nk % NK;
        tc::mbar_arrive_expect_tx(cx.bar(L::kf(s)), L::TILE);
        tc::tma_load_2d_hint(sb + L::OFF_K + s * L::TILE, &tmK, cx.bar(L::kf(s)), 0, kr.take(p), once);
        ++nk;
      };
      auto load_v = [&] {
        const uint32_t s = nv % NV;
        tc::mbar_arrive_expect_tx(cx.bar(L::vf(s)), L::TILE);
        tc::tma_load_2d_hint(sb + L::OFF_V + s * L::TILE, &tmV, cx.bar(L::vf(s)), 0, vr.take(p), once);
        ++nv;
      };
      if (lane == 0) {
        for (uint32_t i = 0; i < NK && i < tiles; ++i) {
          load_k();
          if (i < NV) load_v();
        }
      }
      uint32_t j = 0, piece = 0;
      for (;;) {
        const int blk0 = (pc.b * p.Hkv + pc.g) * p.nblk;
        Pieces<TILE_T> nx = pc;
        const bool more = nx.next(p);
        if (lane == 0) {
          int* f = follow + (piece & 1) * 6;
          f[0] = more;
          f[1] = nx.b;
          f[2] = nx.g;
          f[3] = nx.nv;
          f[4] = nx.first;
          f[5] = nx.last;
        }
        float vs_next = 0.f, M = -INFINITY;  // M: running maximum of row fc
        auto load_scale = [&](int tile) {
          const int t = tile * TILE_T + fs * T;
          vs_next = mine && t < pc.nv ? __ldg(p.vs + blk0 + t / T) * (1.f / kTopP) : 0.f;
        };
        load_scale(pc.first);
        for (int tile = pc.first; tile < pc.last; ++tile, ++j) {
          const float vs = vs_next;
          if (tile + 1 < pc.last) load_scale(tile + 1);
          tile_sync();
          const float* wm = smax + (j & 1) * H * 4 * NC;
          float mt = -INFINITY;
          if (mine) {
#pragma unroll
            for (int w = 0; w < WPS; ++w) mt = fmaxf(mt, wm[(fs * WPS + w) * NC + fc]);
          }
          float mn = fmaxf(M, mt);
#pragma unroll
          for (int o = NC; o < NC * SUB; o <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
          if (mine) {
            const float f = mt == -INFINITY ? 0.f : tc::ex2_approx(mt - mn);
            if (fs == 0) {
              fkeep[(j & 1) * NC + fc] = M == -INFINITY ? 0.f : tc::ex2_approx(M - mn);
              fmax_row[fc] = mn;
            }
            ff[((j & 1) * SUB + fs) * NC + fc] = f;
            ffv[((j & 1) * SUB + fs) * NC + fc] = f * vs;
          }
          M = mn;
          if (lane == 0) {
            // Every softmax thread has S(j): its MMAs are done with K(j)'s stage.  O(j - 1) complete: so is V(j - 1)'s.
            if (nk < tiles) load_k();
            if (j > 0 && nv < tiles && wait(cx, cx.bar(L::of((j - 1) & 1)), ((j - 1) >> 1) & 1)) load_v();
          }
          __syncwarp();
        }
        tile_sync();
        if (!more) break;
        pc = nx;
        ++piece;
      }
      if (lane == 0 && *cx.abort_flag) {  // every copy that was started lands before the CTA exits
        for (uint32_t i = nk > NK ? nk - NK : 0; i < nk; ++i) drain(cx.bar(L::kf(i % NK)), (i / NK) & 1);
        for (uint32_t i = nv > NV ? nv - NV : 0; i < nv; ++i) drain(cx.bar(L::vf(i % NV)), (i / NV) & 1);
      }
    } else if (warp == 5) {
      // ------------------------------ MMA issuer ----------------------------
      if (lane == 0) {
        constexpr uint32_t id_qk = tc::idesc_e4m3_f32(128, N, false, false);
        constexpr uint32_t id_pv = tc::idesc_e4m3_f32(128, N, true, true);
        constexpr uint32_t SWZ = D == 128 ? 2 : 4, ROWS8 = 8 * D;
        uint32_t piece = 0;
        int in_piece = pc.last - pc.first;  // tiles of this piece whose S is not issued yet
        uint32_t qbuf = 0;
        bool q_ready = false;
        auto issue_s = [&](uint32_t j) -> bool {
          if (in_piece == 0) {
            if (!pc.next(p)) return true;
            in_piece = pc.last - pc.first;
            ++piece;
            qbuf = piece & 1;
            q_ready = false;
          }
          --in_piece;
          if (!q_ready && !wait(cx, cx.bar(L::qf(qbuf)), (piece >> 1) & 1)) return false;
          q_ready = true;
          const int s = j % NK;
          if (!wait(cx, cx.bar(L::kf(s)), (j / NK) & 1)) return false;
          tc::tc_fence_after();
          const uint32_t k = sb + L::OFF_K + s * L::TILE, q = sb + L::OFF_Q + qbuf * L::QB;
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              tc::mma_e4m3_ss(tmem + ((j & 1) * H + h) * N, tc::smem_desc(k + h * 128 * D + i * 32, 16, ROWS8, SWZ),
                              tc::smem_desc(q + i * 256, 128, D * 8, 0), id_qk, i > 0);
          tc::mma_commit(cx.bar(L::sf(j & 1)));
          return true;
        };
        const uint32_t tiles = (uint32_t)n;
        bool ok = issue_s(0);
        if (ok && tiles > 1) ok = issue_s(1);
        for (uint32_t j = 0; ok && j < tiles; ++j) {
          const int s = j % NV;
          if (!wait(cx, cx.bar(L::pf(j & 1)), (j >> 1) & 1) || !wait(cx, cx.bar(L::vf(s)), (j / NV) & 1)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint32_t v = sb + L::OFF_V + s * L::TILE, pp = sb + L::OFF_P + (j & 1) * L::PB;
#pragma unroll
          for (int i = 0; i < TILE_T / 32; ++i)
            tc::mma_e4m3_ss(tmem + L::COL_O + ((j & 1) * SUB + i / (T / 32)) * N,
                            tc::smem_desc(v + i * 4 * ROWS8, ROWS8, ROWS8, SWZ),
                            tc::smem_desc(pp + i * 512, 128, TILE_T * 16, 0), id_pv, i % (T / 32) > 0);
          tc::mma_commit(cx.bar(L::of(j & 1)));
          if (j + 2 < tiles) ok = issue_s(j + 2);
        }
        tc::mma_commit(cx.bar(L::DRAIN));  // everything issued completes before teardown
        drain(cx.bar(L::DRAIN), 0);
      }
    } else {
      // ------------------------- softmax and O ------------------------------
      float* smax = reinterpret_cast<float*>(sm + L::OFF_MAX);    // [2][H][4][NC]
      const float* fkeep = reinterpret_cast<const float*>(sm + L::OFF_FAC);  // [2][NC]
      const float* ff = fkeep + 2 * NC;                           // [2][SUB][NC]
      const float* ffv = ff + 2 * SUB * NC;                       // [2][SUB][NC]
      const float* fmax_row = ffv + 2 * SUB * NC;                 // [NC]
      float* ee = reinterpret_cast<float*>(sm + L::OFF_EE);       // [2][kEdge][NC]
      const float* qfac = reinterpret_cast<const float*>(sm + L::OFF_QF);
      const int* unseen = reinterpret_cast<const int*>(sm + L::OFF_BACK);
      const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
      constexpr int WPS = T / 32;  // warps per scale block
      const int my_sub = tid / T;  // scale block of this thread's token within its 128
      uint32_t j = 0, piece = 0;

      write_q<D, NC, T>(p, sm, 0, pc.b * p.Hkv + pc.g, tid);
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(cx.bar(L::qf(0)));
      bool more = false;
      for (;;) {
        const int unit = pc.b * p.Hkv + pc.g;
        const int blk0 = unit * p.nblk;  // B Hkv blocks stay under 2^31
        // The scales of a tile are loaded a tile ahead.
        float ks_next[H];
        auto load_scales = [&](int tile) {
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const int t = tile * TILE_T + h * 128 + tid;
            ks_next[h] = t < pc.nv ? __ldg(p.ks + blk0 + t / T) : 0.f;
          }
        };
        load_scales(pc.first);
        softmax_sync();  // this piece's row factors, written by other warps
        constexpr int NP = NC / 2;
        uint64_t l[NP], acc[NP], e_prev[H][NP];  // pairs of rows
#pragma unroll
        for (int c = 0; c < NP; ++c) {
          l[c] = acc[c] = 0;
#pragma unroll
          for (int h = 0; h < H; ++h) e_prev[h][c] = 0;
        }
        int edge_prev = TILE_T;  // first edge token of the previous tile
        int edge_n = 0;          // and how many
        // Adds O^T of tile i to the registers, and the tile's probabilities to l.
        auto absorb = [&](uint32_t i) {
          wait(cx, cx.bar(L::of(i & 1)), (i >> 1) & 1);
          __syncwarp();
          tc::tc_fence_after();
          constexpr int BOTH = NC == 8 && SUB > 1 ? 2 : 1;  // blocks loaded at once (16 rows: registers for one)
          uint32_t o[BOTH][N];
          const uint32_t at = tmem + lane_base + L::COL_O + (i & 1) * SUB * N;
#pragma unroll
          for (int s = 0; s < BOTH; ++s) tmem_row<N>(at + s * N, o[s]);
          {
            uint64_t kp[NP];
            load_pairs<NC>(fkeep + (i & 1) * NC, kp);
#pragma unroll
            for (int c = 0; c < NP; ++c) {
              acc[c] = tc::f2_mul(acc[c], kp[c]);
              l[c] = tc::f2_mul(l[c], kp[c]);
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
              uint64_t fp[NP];
              load_pairs<NC>(ff + ((i & 1) * SUB + h * SUBH + my_sub) * NC, fp);
#pragma unroll
              for (int c = 0; c < NP; ++c) l[c] = tc::f2_fma(e_prev[h][c], fp[c], l[c]);
            }
          }
          const float* vp = ffv + (i & 1) * SUB * NC;
          // d = 64: lanes 64 .. 127 hold copies of other rows (the MMA has 128) that are never written out.
#pragma unroll
          for (int s0 = 0; s0 < SUB; s0 += BOTH) {
            if (s0 > 0) {
#pragma unroll
              for (int s = 0; s < BOTH; ++s) tmem_row<N>(at + (s0 + s) * N, o[s]);
            }
            tc::tmem_wait_ld();
#pragma unroll
            for (int s = 0; s < BOTH; ++s) {
              uint64_t fv[NP];
              load_pairs<NC>(vp + (s0 + s) * NC, fv);
#pragma unroll
              for (int c = 0; c < NP; ++c) {
                const uint64_t x = tc::f2_fma(pair_bits(o[s][NC + 2 * c], o[s][NC + 2 * c + 1]), pair(1.f / kLoP),
                                              pair_bits(o[s][2 * c], o[s][2 * c + 1]));
                acc[c] = tc::f2_fma(x, fv[c], acc[c]);
              }
            }
          }
          for (int r = 0; r < edge_n; ++r) {
            const float v = __low2float(from_e4m3x2(sm[L::OFF_EV + ((i & 1) * kEdge + r) * D + tid % D])) * kTopP;
            float er[NC], vr[NC];
            load_row<NC>(ee + ((i & 1) * kEdge + r) * NC, er);
            load_row<NC>(vp + ((edge_prev + r) / T) * NC, vr);
#pragma unroll
            for (int c = 0; c < NP; ++c) {
              float a0, a1;
              tc::f2_unpack(acc[c], a0, a1);
              if (!(er[2 * c] < 0.f)) a0 = fmaf(er[2 * c] * vr[2 * c], v, a0);  // < 0: the row does not see it
              if (!(er[2 * c + 1] < 0.f)) a1 = fmaf(er[2 * c + 1] * vr[2 * c + 1], v, a1);
              acc[c] = tc::f2_pack(a0, a1);
            }
          }
          tc::tc_fence_before();
        };

        for (int tile = pc.first; tile < pc.last; ++tile, ++j) {
          const int t0 = tile * TILE_T;
          const int edge = max(pc.nv - p.nq + 1 - t0, 0);  // tokens from here on: not seen by every row
          float ks[H];
#pragma unroll
          for (int h = 0; h < H; ++h) ks[h] = ks_next[h];
          if (tile + 1 < pc.last) load_scales(tile + 1);
          wait(cx, cx.bar(L::sf(j & 1)), (j >> 1) & 1);
          __syncwarp();
          tc::tc_fence_after();
          float e[H][NC];  // scores in log2 units, then probabilities against the block's maximum
          {
            uint64_t qf[NP];
            load_pairs<NC>(qfac + (piece & 1) * NC, qf);
#pragma unroll
            for (int h = 0; h < H; ++h) {
              uint32_t r[N];
              tmem_row<N>(tmem + lane_base + ((j & 1) * H + h) * N, r);
              tc::tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < NP; ++c) {
                const uint64_t x = tc::f2_fma(pair_bits(r[NC + 2 * c], r[NC + 2 * c + 1]), pair(1.f / kLoQ),
                                              pair_bits(r[2 * c], r[2 * c + 1]));
                tc::f2_unpack(tc::f2_mul(x, tc::f2_mul(pair(ks[h]), qf[c])), e[h][2 * c], e[h][2 * c + 1]);
              }
            }
          }
          if (edge < TILE_T) {  // only here some row does not see some token; rows from cols on are never used
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const int last = pc.nv - unseen[c] - t0;
#pragma unroll
              for (int h = 0; h < H; ++h)
                if (h * 128 + tid >= last) e[h][c] = -INFINITY;
            }
          }
          float* wm = smax + (j & 1) * H * 4 * NC;
#pragma unroll
          for (int h = 0; h < H; ++h) {
            float m[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) m[c] = tc::warp_max(e[h][c]);
            if (lane == 0) {
#pragma unroll
              for (int c = 0; c < NC; c += 4)
                *reinterpret_cast<float4*>(wm + (h * 4 + warp) * NC + c) = make_float4(m[c], m[c + 1], m[c + 2], m[c + 3]);
            }
          }
          if (p.scores != nullptr) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
              const int t = t0 + h * 128 + tid;
              if (t >= pc.nv) continue;
              float* sc = p.scores + ((size_t)unit * p.Lp + t) * p.cpad;
              if (p.cpad >= 4) {
#pragma unroll
                for (int c = 0; c < NC; c += 4)
                  if (c < p.cpad)
                    *reinterpret_cast<float4*>(sc + c) = make_float4(e[h][c], e[h][c + 1], e[h][c + 2], e[h][c + 3]);
              } else if (p.cpad == 2) {
                *reinterpret_cast<float2*>(sc) = make_float2(e[h][0], e[h][1]);
              } else {
                *sc = e[h][0];
              }
            }
          }
          tile_sync();
          // Probabilities as two e4m3 parts: B operand, MN-major, no swizzle (8 tokens x 16 rows contiguous).
#pragma unroll
          for (int h = 0; h < H; ++h) {
            float m[WPS][NC];
#pragma unroll
            for (int w = 0; w < WPS; ++w) load_row<NC>(wm + (h * 4 + my_sub * WPS + w) * NC, m[w]);
            uint32_t hi[NC / 4], lo[NC / 4];
#pragma unroll
            for (int c = 0; c < NC; c += 4) {
              uint32_t h2[2], l2[2];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                // A block without a score: against the lowest float, exp2(-inf) = 0.
                float mx = tc::max3(m[0][c + u], m[1][c + u], -FLT_MAX);
                if (WPS == 4) mx = tc::max3(mx, m[WPS - 2][c + u], m[WPS - 1][c + u]);
                e[h][c + u] = tc::ex2_approx(e[h][c + u] - mx);
              }
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const uint64_t x = tc::f2_pack(e[h][c + 2 * u], e[h][c + 2 * u + 1]);
                float a, b;
                tc::f2_unpack(tc::f2_mul(x, pair(kTopP)), a, b);
                h2[u] = to_e4m3x2(a, b);
                const float2 f = __half22float2(from_e4m3x2(h2[u]));
                // (a - f) kLoP, exact up to the last rounding
                tc::f2_unpack(tc::f2_fma(tc::f2_pack(f.x, f.y), pair(-kLoP), tc::f2_mul(x, pair(kTopP * kLoP))), a, b);
                l2[u] = to_e4m3x2(a, b);
              }
              hi[c / 4] = h2[0] | (h2[1] << 16);
              lo[c / 4] = l2[0] | (l2[1] << 16);
            }
            unsigned char* pp = sm + L::OFF_P + (j & 1) * L::PB + (h * 128 + tid) * 16;
            if constexpr (NC == 8) {
              *reinterpret_cast<uint4*>(pp) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
            } else {
              *reinterpret_cast<uint4*>(pp) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4*>(pp + TILE_T * 16) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
          }
          if (edge < TILE_T) {
            // Rows of V that some query must not see: a NaN there would pass through a zero probability.  Rows behind
            // the last token become 0; the few that only the later queries see move aside and are added by hand.
            wait(cx, cx.bar(L::vf(j % NV)), (j / NV) & 1);
            __syncwarp();
#pragma unroll
            for (int h = 0; h < H; ++h) {
              const int i = h * 128 + tid, t = t0 + i;
              if (i < edge) continue;
              uint4* row = reinterpret_cast<uint4*>(sm + L::OFF_V + (j % NV) * L::TILE + i * D);
              if (t < pc.nv) {
                uint4* ev = reinterpret_cast<uint4*>(sm + L::OFF_EV + ((j & 1) * kEdge + i - edge) * D);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) ev[k] = row[k ^ (D == 128 ? (i & 7) : ((i >> 1) & 3))];
                float* er = ee + ((j & 1) * kEdge + i - edge) * NC;
#pragma unroll
                for (int c = 0; c < NC; ++c) er[c] = t < pc.nv - unseen[c] ? e[h][c] : -1.f;
              }
#pragma unroll
              for (int k = 0; k < D / 16; ++k) row[k] = make_uint4(0, 0, 0, 0);
            }
          }
          tc::fence_proxy_async_smem();
          tc::tc_fence_before();
          tc::mbar_arrive(cx.bar(L::pf(j & 1)));
          if (tile == pc.first) {  // the next piece's query rows, ahead of their first use
            const int* f = follow + (piece & 1) * 6;
            more = f[0] != 0;
            if (more) {
              write_q<D, NC, T>(p, sm, (piece + 1) & 1, f[1] * p.Hkv + f[2], tid);
              tc::fence_proxy_async_smem();
              tc::mbar_arrive(cx.bar(L::qf((piece + 1) & 1)));
            }
          } else {
            absorb(j - 1);
          }
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int c = 0; c < NP; ++c) e_prev[h][c] = tc::f2_pack(e[h][2 * c], e[h][2 * c + 1]);
          edge_prev = edge;
          edge_n = max(min(pc.nv - t0, TILE_T) - edge, 0);
        }
        tile_sync();
        absorb(j - 1);

        // A piece that is its whole unit gives the outputs at once; others go to the joining step.
        const bool whole = pc.first == 0 && pc.last == (pc.nv + TILE_T - 1) / TILE_T;
        const size_t slot = (size_t)blockIdx.x + unit;
        float o[NC];
        {
          float v[NC];
#pragma unroll
          for (int c = 0; c < NP; ++c) {
            tc::f2_unpack(l[c], v[2 * c], v[2 * c + 1]);
            tc::f2_unpack(acc[c], o[2 * c], o[2 * c + 1]);
          }
          int row;
          const float sum = warp_row_sums<NC>(v, &row);
          smax[warp * NC + row] = sum;  // (the lanes of one row write the same)
        }
        if (!whole && tid < D) {
          float* to = p.part_o + slot * p.cols * D + tid;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (c < p.cols) to[c * D] = o[c];
        }
        softmax_sync();
        if (tid < p.cols) {
          const float m = fmax_row[tid];
          const float sum = ((smax[tid] + smax[NC + tid]) + smax[2 * NC + tid]) + smax[3 * NC + tid];
          reinterpret_cast<float2*>(p.part_ml)[slot * p.cols + tid] = make_float2(m, sum);
          if (whole && p.lse != nullptr)
            p.lse[(size_t)unit * p.cols + tid] =
                sum == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(sum)) * 0.6931471805599453f;
        }
        if (whole && tid < D) {
          float sum[NC], u[NC];
          load_row<NC>(smax, sum);
#pragma unroll
          for (int w = 1; w < 4; ++w) {
            load_row<NC>(smax + w * NC, u);
#pragma unroll
            for (int c = 0; c < NC; ++c) sum[c] += u[c];
          }
          __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.o) + (size_t)unit * p.cols * D + tid;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (c < p.cols)  // sum = 0 exactly when the row sees no token (a NaN score makes it NaN, and the row's o);
                             // the division is 2 ulp of float32 off at most, for sums under 2^31
              to[c * D] = __float2bfloat16_rn(sum[c] == 0.f ? 0.f : __fdividef(o[c], sum[c]));
        }
        if (!more) break;
        const int* f = follow + (piece & 1) * 6;
        pc.b = f[1];
        pc.g = f[2];
        pc.nv = f[3];
        pc.first = f[4];
        pc.last = f[5];
        ++piece;
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, L::TMEM);
  }
}

template <int D, int NC, int T>
cudaError_t launch_t(const Cache8Attn& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  using L = Lay<D, NC, T>;
  static_assert(kCtasPerSm * (L::BYTES + 1024) <= 228 * 1024, "shared memory of an SM");
  static_assert(kCtasPerSm * L::TMEM <= 512, "tensor memory of an SM");
  static_assert(L::SUB * NC <= 32, "a lane of warp 4 for each factor");
  auto kern = attn_tile_kernel<D, NC, T>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem_once(kern, L::BYTES, true, done);
  if (e != cudaSuccess) return e;
  kern<<<p.G, kTileThreads, L::BYTES, st>>>(tk, tv, p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const Cache8Attn& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  if (p.cols <= 8)
    return p.T == 128 ? launch_t<D, 8, 128>(p, tk, tv, st) : launch_t<D, 8, 64>(p, tk, tv, st);
  return p.T == 128 ? launch_t<D, 16, 128>(p, tk, tv, st) : launch_t<D, 16, 64>(p, tk, tv, st);
}

}  // namespace

cudaError_t launch_cache8_tiles(const Cache8Attn& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  return p.D == 128 ? launch_d<128>(p, tk, tv, st) : launch_d<64>(p, tk, tv, st);
}

}  // namespace sfa
