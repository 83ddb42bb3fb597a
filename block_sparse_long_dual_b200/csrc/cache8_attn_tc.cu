// Attention of a few query rows over the whole 8-bit KV cache on the sm_100a
// tensor cores (the first of the two steps: pieces; cache8_attn.cu joins them).
//
// The codes go to the tensor core as they are (kind::f8f6f4), so no cached value
// is converted by a thread.  Per tile of 128 tokens:
//   S^T [128 tokens, 2 NC] = K [128, D] . Q^T     Q: NC query rows (the group's heads x query tokens)
//   O^T [D, 2 NC]          = V^T [D, 128] . P^T
// A bf16 query row or a float32 probability does not fit 4 significant bits, so
// each takes two columns: x = hi + lo / 2^k, hi = e4m3(x), lo = e4m3((x - hi) 2^k).
// For a query row scaled to its largest element, hi and lo together hold every
// bf16 significand exactly down to 2^-21 of the largest; for probabilities scaled
// to their block's largest, 8 significant bits down to 2^-14 and an absolute step
// of 2^-23.  The products' sums, scores, maxima, sums and O are float32.
//
// Each scale block has its own reference maximum and, in TMEM, its own O^T, so
// scales that lie far apart between blocks lose nothing: the block's factor
// 2^(max - running max) * v_scale is applied when O^T is added to the registers.
//
//   warps 0 .. 3  thread t = token t of the tile for S (TMEM lane t): scores, block
//                 maximum (warp maxima through shared memory), probabilities as
//                 e4m3 into shared memory; thread r = dim r for O^T: the running
//                 O of the piece in registers.  O^T of tile j - 1 is added after
//                 the probabilities of tile j are on their way.
//   warp 4        producer: TMA tiles of K and V (a ring each)
//   warp 5        MMA issuer
// A tile of 128 tokens is 32 KB (d = 128) and 8 MMAs of N = 2 NC; the tensor core
// is idle most of the time and the kernel's bound is the cache's bytes.
// Work split, pieces and their slots: cache8.cuh.  Every wait is bounded; one that
// runs out sets SFA_ERR_TIMEOUT and an abort flag, after which waits return at
// once and the CTA runs to its end (the copies and MMAs it issued are drained).
#include <cuda.h>
#include <math.h>

#include "cache8.cuh"
#include "tc_ptx.cuh"

namespace sfa {

namespace {

using namespace c8;

constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kEdge = kMaxCols - 1;   // tokens that not every query sees: nq - 1 at most
constexpr float kLoQ = 16.f, kLoP = 32.f, kTopP = 256.f;

template <int D, int NC, int T>
struct Lay {
  static constexpr int N = 2 * NC;                // MMA columns
  static constexpr int SUB = kTile / T;           // scale blocks of a tile
  static constexpr uint32_t TILE = kTile * D;     // bytes of a K or V tile
  static constexpr int NK = D == 128 ? 3 : 6;     // ring stages of K, of V (16 rows leave less room)
  static constexpr int NV = NC == 8 ? NK : NK - NK / 3;
  static constexpr uint32_t QB = N * D, PB = kTile * N;
  static constexpr uint32_t OFF_K = 0, OFF_V = NK * TILE;
  static constexpr uint32_t OFF_Q = (NK + NV) * TILE;            // two buffers
  static constexpr uint32_t OFF_P = OFF_Q + 2 * QB;              // two buffers
  static constexpr uint32_t OFF_EV = OFF_P + 2 * PB;             // edge tokens' V rows, two buffers
  static constexpr uint32_t OFF_EE = OFF_EV + 2 * kEdge * D;     // their probabilities [2][kEdge][NC]
  static constexpr uint32_t OFF_MAX = OFF_EE + 2 * kEdge * NC * 4;   // warp maxima [2][4][NC]
  static constexpr uint32_t OFF_FAC = OFF_MAX + 2 * 4 * NC * 4;      // [2][NC] keep, [2][SUB][NC] f, [2][SUB][NC] f v
  static constexpr uint32_t OFF_QF = OFF_FAC + 2 * NC * (1 + 2 * SUB) * 4;  // row factors [2][NC]
  static constexpr uint32_t OFF_BAR = OFF_QF + 2 * NC * 4;
  static constexpr int NBAR = 2 * NK + 2 * NV + 9;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr uint32_t BYTES = OFF_MISC + 64 + 1024;
  // TMEM columns: S two buffers, O two buffers x SUB
  static constexpr uint32_t COL_O = 2 * N, COLS_USED = 2 * N + 2 * SUB * N;
  static constexpr uint32_t TMEM = COLS_USED <= 64 ? 64 : (COLS_USED <= 128 ? 128 : 256);
  static constexpr int B0 = 2 * NK + 2 * NV;
  __host__ __device__ static constexpr int kf(int s) { return s; }
  __host__ __device__ static constexpr int ke(int s) { return NK + s; }
  __host__ __device__ static constexpr int vf(int s) { return 2 * NK + s; }
  __host__ __device__ static constexpr int ve(int s) { return 2 * NK + NV + s; }
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
struct Pieces {
  long long left;  // tiles of the share after the present piece
  int b, g, nv, first, last;  // unit (b, g), its visible tokens, the piece's tiles [first, last)

  __device__ void begin(const Cache8Attn& p, int b0, long long x0, long long before, long long n) {
    b = b0;
    nv = visible(p.lens, b, p.L, p.back, nullptr);
    const int tiles = (nv + kTile - 1) / kTile;
    g = (int)((x0 - before) / tiles);
    first = (int)((x0 - before) % tiles);
    last = (int)min((long long)tiles, first + n);
    left = n - (last - first);
  }
  __device__ bool next(const Cache8Attn& p) {
    if (left <= 0) return false;
    int tiles = (nv + kTile - 1) / kTile;
    if (++g == p.Hkv) {
      g = 0;
      do {
        if (++b >= p.B) {  // only if the lengths changed under the call
          left = 0;
          return false;
        }
        nv = visible(p.lens, b, p.L, p.back, nullptr);
        tiles = (nv + kTile - 1) / kTile;
      } while (tiles == 0);  // `left` tiles follow, so a sequence with tiles does
    }
    first = 0;
    last = (int)min((long long)tiles, left);
    left -= last;
    return true;
  }
};

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

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
__global__ void __launch_bounds__(192, 2)
    attn_tile_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ Cache8Attn p) {
  using L = Lay<D, NC, T>;
  constexpr int N = L::N, SUB = L::SUB, NK = L::NK, NV = L::NV;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = tc::smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  unsigned char* sm = smem_raw + pad;
  const uint32_t sb = raw + pad;
  long long* sched = reinterpret_cast<long long*>(sm + L::OFF_MISC);  // before, x0, tiles of the share
  int* sched_b = reinterpret_cast<int*>(sm + L::OFF_MISC + 24);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::OFF_MISC + 28);
  Ctx cx;
  cx.bars = sb + L::OFF_BAR;
  cx.abort_flag = reinterpret_cast<volatile int*>(sm + L::OFF_MISC + 32);
  cx.status = p.status;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == 0) {
    long long dummy, before = 0;
    const long long total = warp_count_tiles(p.lens, p.B, p.Hkv, p.L, p.back, 0, &dummy,
                                             blockIdx.x == 0 ? p.status : nullptr);
    const Split s(total, p.G);
    const long long x0 = s.start(blockIdx.x), n = s.start(blockIdx.x + 1) - x0;
    int b = -1;
    if (n > 0) b = warp_find_seq(p.lens, p.B, p.Hkv, p.L, p.back, x0, &before);
    if (lane == 0) {
      sched[0] = before;
      sched[1] = x0;
      sched[2] = b < 0 ? 0 : n;
      *sched_b = b;
    }
  } else if (warp == 4 && lane == 0) {
    *cx.abort_flag = 0;
    for (int k = 0; k < L::NBAR; ++k)
      tc::mbar_init(cx.bar(k), k == L::pf(0) || k == L::pf(1) || k == L::qf(0) || k == L::qf(1) ? 128 : 1);
    tc::fence_mbar_init();
    tc::prefetch_tmap(&tmK);
    tc::prefetch_tmap(&tmV);
  } else if (warp == 5) {
    tc::tmem_alloc(tc::smem_u32(tmem_slot), L::TMEM);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const long long n = sched[2];

  if (n > 0) {
    Pieces pc;
    pc.begin(p, *sched_b, sched[1], sched[0], n);
    if (warp == 4) {
      // ------------------------------ producer ------------------------------
      if (lane == 0) {
        uint32_t j = 0;
        bool ok = true;
        do {
          const int row0 = (pc.b * p.Hkv + pc.g) * p.L;
          for (int t = pc.first; ok && t < pc.last; ++t, ++j) {
            const uint32_t sk = j % NK, sv = j % NV;
            if (j >= NK && !wait(cx, cx.bar(L::ke(sk)), ((j / NK) & 1) ^ 1)) { ok = false; break; }
            tc::mbar_arrive_expect_tx(cx.bar(L::kf(sk)), L::TILE);
            tc::tma_load_2d(sb + L::OFF_K + sk * L::TILE, &tmK, cx.bar(L::kf(sk)), 0, row0 + t * kTile);
            if (j >= NV && !wait(cx, cx.bar(L::ve(sv)), ((j / NV) & 1) ^ 1)) {
              drain(cx.bar(L::kf(sk)), (j / NK) & 1);
              ok = false;
              break;
            }
            tc::mbar_arrive_expect_tx(cx.bar(L::vf(sv)), L::TILE);
            tc::tma_load_2d(sb + L::OFF_V + sv * L::TILE, &tmV, cx.bar(L::vf(sv)), 0, row0 + t * kTile);
          }
        } while (ok && pc.next(p));
        if (*cx.abort_flag) {  // every copy that was started lands before the CTA exits
          for (uint32_t i = j > NK ? j - NK : 0; i < j; ++i) drain(cx.bar(L::kf(i % NK)), (i / NK) & 1);
          for (uint32_t i = j > NV ? j - NV : 0; i < j; ++i) drain(cx.bar(L::vf(i % NV)), (i / NV) & 1);
        }
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
          for (int i = 0; i < D / 32; ++i)
            tc::mma_e4m3_ss(tmem + (j & 1) * N, tc::smem_desc(k + i * 32, 16, ROWS8, SWZ),
                            tc::smem_desc(q + i * 256, 128, D * 8, 0), id_qk, i > 0);
          tc::mma_commit(cx.bar(L::ke(s)));
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
          for (int i = 0; i < kTile / 32; ++i) {
            const int sub = i / (T / 32);
            tc::mma_e4m3_ss(tmem + L::COL_O + ((j & 1) * SUB + sub) * N,
                            tc::smem_desc(v + i * 4 * ROWS8, ROWS8, ROWS8, SWZ),
                            tc::smem_desc(pp + i * 512, 128, 2048, 0), id_pv, i % (T / 32) > 0);
          }
          tc::mma_commit(cx.bar(L::ve(s)));
          tc::mma_commit(cx.bar(L::of(j & 1)));
          if (j + 2 < tiles) ok = issue_s(j + 2);
        }
        tc::mma_commit(cx.bar(L::DRAIN));  // everything issued completes before teardown
        drain(cx.bar(L::DRAIN), 0);
      }
    } else {
      // ------------------------- softmax and O ------------------------------
      float* smax = reinterpret_cast<float*>(sm + L::OFF_MAX);    // [2][4][NC]
      float* fkeep = reinterpret_cast<float*>(sm + L::OFF_FAC);   // [2][NC]
      float* ff = fkeep + 2 * NC;                                 // [2][SUB][NC]
      float* ffv = ff + 2 * SUB * NC;                             // [2][SUB][NC]
      float* ee = reinterpret_cast<float*>(sm + L::OFF_EE);       // [2][kEdge][NC]
      const float* qfac = reinterpret_cast<const float*>(sm + L::OFF_QF);
      const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
      const int sub = tid / T;
      constexpr int WPS = T / 32;  // warps per scale block
      uint32_t j = 0, piece = 0;

      write_q<D, NC, T>(p, sm, 0, pc.b * p.Hkv + pc.g, tid);
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(cx.bar(L::qf(0)));
      Pieces nx = pc;
      bool more = nx.next(p);
      for (;;) {
        const int unit = pc.b * p.Hkv + pc.g;
        if (more) {  // the next piece's query rows, a piece ahead of their first use
          write_q<D, NC, T>(p, sm, (piece + 1) & 1, nx.b * p.Hkv + nx.g, tid);
          tc::fence_proxy_async_smem();
          tc::mbar_arrive(cx.bar(L::qf((piece + 1) & 1)));
        }
        softmax_sync();  // this piece's row factors, written by other warps
        float qf[NC], l[NC], acc[NC], e_prev[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          qf[c] = qfac[(piece & 1) * NC + c];
          l[c] = acc[c] = e_prev[c] = 0.f;
        }
        float M = -INFINITY;  // threads 0 .. NC - 1: running maximum of row tid
        int edge_prev = kTile;  // first edge token of the previous tile
        int edge_n = 0;         // and how many
        // Adds O^T of tile i to the registers, and the tile's probabilities to l.
        auto absorb = [&](uint32_t i) {
          wait(cx, cx.bar(L::of(i & 1)), (i >> 1) & 1);
          __syncwarp();
          tc::tc_fence_after();
          const float* kp = fkeep + (i & 1) * NC;
          const float* fp = ff + ((i & 1) * SUB + sub) * NC;
          const float* vp = ffv + (i & 1) * SUB * NC;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float k = kp[c];
            acc[c] *= k;
            l[c] = fmaf(e_prev[c], fp[c], l[c] * k);
          }
          if (D == 128 || warp < 2) {
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
              uint32_t o[N];
              const uint32_t at = tmem + lane_base + L::COL_O + ((i & 1) * SUB + s) * N;
              if constexpr (N == 16) tc::tmem_ld16(at, o); else tc::tmem_ld32(at, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < NC; ++c)
                acc[c] = fmaf(fmaf(__uint_as_float(o[NC + c]), 1.f / kLoP, __uint_as_float(o[c])), vp[s * NC + c],
                              acc[c]);
            }
            for (int r = 0; r < edge_n; ++r) {
              const float v = __low2float(from_e4m3x2(sm[L::OFF_EV + ((i & 1) * kEdge + r) * D + tid])) * kTopP;
              const float* er = ee + ((i & 1) * kEdge + r) * NC;
              const float* vr = vp + ((edge_prev + r) / T) * NC;
#pragma unroll
              for (int c = 0; c < NC; ++c)
                if (!(er[c] < 0.f)) acc[c] = fmaf(er[c] * vr[c], v, acc[c]);  // < 0: the row does not see it
            }
          }
          tc::tc_fence_before();
        };

        for (int tile = pc.first; tile < pc.last; ++tile, ++j) {
          const int t = tile * kTile + tid;
          const bool live = t < pc.nv;
          const float ks = live ? __ldg(p.ks + (size_t)unit * p.nblk + t / T) : 0.f;
          float vs[SUB];
          if (tid < NC) {
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
              const int t0 = tile * kTile + s * T;
              vs[s] = t0 < pc.nv ? __ldg(p.vs + (size_t)unit * p.nblk + t0 / T) * (1.f / kTopP) : 0.f;
            }
          }
          wait(cx, cx.bar(L::sf(j & 1)), (j >> 1) & 1);
          __syncwarp();
          tc::tc_fence_after();
          float e[NC];
          {
            uint32_t r[N];
            if constexpr (N == 16) tc::tmem_ld16(tmem + lane_base + (j & 1) * N, r);
            else tc::tmem_ld32(tmem + lane_base + (j & 1) * N, r);
            tc::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const float s = fmaf(__uint_as_float(r[NC + c]), 1.f / kLoQ, __uint_as_float(r[c])) * (ks * qf[c]);
              const bool sees = c < p.cols && t < pc.nv - (p.nq - 1 - c % p.nq);
              e[c] = sees ? s : -INFINITY;
            }
          }
          float* wm = smax + (j & 1) * 4 * NC;
          {
            float mine = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const float m = tc::warp_max(e[c]);
              if (lane == c) mine = m;
            }
            if (lane < NC) wm[warp * NC + lane] = mine;
          }
          if (p.scores != nullptr && live) {
            float* sc = p.scores + (size_t)unit * p.cols * p.Lp + t;
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (c < p.cols) sc[(size_t)c * p.Lp] = e[c];
          }
          softmax_sync();
          const int edge = max(pc.nv - p.nq + 1 - tile * kTile, 0);  // tokens from here on: not seen by every row
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < WPS; ++w) m = fmaxf(m, wm[(sub * WPS + w) * NC + c]);
            const float x = e[c];
            e[c] = tc::ex2_approx(x - (m == -INFINITY ? 0.f : m));
          }
          if (tid < NC) {  // factors of row tid: running maximum, this tile's blocks against it
            float mt[SUB], mn = M;
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
              mt[s] = -INFINITY;
#pragma unroll
              for (int w = 0; w < WPS; ++w) mt[s] = fmaxf(mt[s], wm[(s * WPS + w) * NC + tid]);
              mn = fmaxf(mn, mt[s]);
            }
            fkeep[(j & 1) * NC + tid] = M == -INFINITY ? 0.f : exp2f(M - mn);
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
              const float f = mt[s] == -INFINITY ? 0.f : exp2f(mt[s] - mn);
              ff[((j & 1) * SUB + s) * NC + tid] = f;
              ffv[((j & 1) * SUB + s) * NC + tid] = f * vs[s];
            }
            M = mn;
          }
          // Probabilities as two e4m3 parts: B operand, MN-major, no swizzle (8 tokens x 16 rows contiguous).
          {
            uint32_t hi[NC / 4], lo[NC / 4];
#pragma unroll
            for (int c = 0; c < NC; c += 4) {
              uint32_t h2[2], l2[2];
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const float a = e[c + 2 * u] * kTopP, b = e[c + 2 * u + 1] * kTopP;
                h2[u] = to_e4m3x2(a, b);
                const float2 h = __half22float2(from_e4m3x2(h2[u]));
                l2[u] = to_e4m3x2((a - h.x) * kLoP, (b - h.y) * kLoP);
              }
              hi[c / 4] = h2[0] | (h2[1] << 16);
              lo[c / 4] = l2[0] | (l2[1] << 16);
            }
            unsigned char* pp = sm + L::OFF_P + (j & 1) * L::PB + tid * 16;
            if constexpr (NC == 8) {
              *reinterpret_cast<uint4*>(pp) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
            } else {
              *reinterpret_cast<uint4*>(pp) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4*>(pp + 2048) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
          }
          if (edge < kTile) {
            // Rows of V that some query must not see: a NaN there would pass through a zero probability.  Rows behind
            // the last token become 0; the few that only the later queries see move aside and are added by hand.
            wait(cx, cx.bar(L::vf(j % NV)), (j / NV) & 1);
            __syncwarp();
            if (tid >= edge) {
              uint4* row = reinterpret_cast<uint4*>(sm + L::OFF_V + (j % NV) * L::TILE + tid * D);
              if (live) {
                uint4* ev = reinterpret_cast<uint4*>(sm + L::OFF_EV + ((j & 1) * kEdge + tid - edge) * D);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) ev[i] = row[i ^ (D == 128 ? (tid & 7) : ((tid >> 1) & 3))];
                float* er = ee + ((j & 1) * kEdge + tid - edge) * NC;
#pragma unroll
                for (int c = 0; c < NC; ++c)
                  er[c] = c < p.cols && t < pc.nv - (p.nq - 1 - c % p.nq) ? e[c] : -1.f;
              }
#pragma unroll
              for (int i = 0; i < D / 16; ++i) row[i] = make_uint4(0, 0, 0, 0);
            }
          }
          tc::fence_proxy_async_smem();
          tc::tc_fence_before();
          tc::mbar_arrive(cx.bar(L::pf(j & 1)));
          if (tile > pc.first) absorb(j - 1);
#pragma unroll
          for (int c = 0; c < NC; ++c) e_prev[c] = e[c];
          edge_prev = edge;
          edge_n = max(min(pc.nv - tile * kTile, kTile) - edge, 0);
        }
        softmax_sync();
        absorb(j - 1);

        const size_t slot = (size_t)blockIdx.x + unit;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          float v = l[c];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if (lane == 0) smax[warp * NC + c] = v;
          if (c < p.cols && tid < D) p.part_o[(slot * p.cols + c) * D + tid] = acc[c];
        }
        softmax_sync();
        if (tid < p.cols)
          reinterpret_cast<float2*>(p.part_ml)[slot * p.cols + tid] =
              make_float2(M, (smax[tid] + smax[NC + tid]) + (smax[2 * NC + tid] + smax[3 * NC + tid]));
        if (!more) break;
        pc = nx;
        more = nx.next(p);
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
  static_assert(2 * (L::BYTES + 1024) <= 227 * 1024, "two CTAs per SM");
  auto kern = attn_tile_kernel<D, NC, T>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::BYTES);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e != cudaSuccess) return e;
  kern<<<p.G, 192, L::BYTES, st>>>(tk, tv, p);
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
