// 8-bit KV cache: e4m3 codes, power-of-two block scales, and how a call's work
// is split over CTAs.  Shared by cache8_store.cu, cache8_attn.cu, cache8_attn_tc.cu and
// api.cu.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"

namespace sfa {
namespace c8 {

// Two floats -> two e4m3 codes (lo in the low byte), to nearest even; NaN -> 0x7F.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes -> half2 (exact: every e4m3 value is a half).
__device__ __forceinline__ __half2 from_e4m3x2(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)c));
  return *reinterpret_cast<const __half2*>(&r);
}
// Four codes -> four floats.
__device__ __forceinline__ void from_e4m3x4(uint32_t c, float (&v)[4]) {
  const float2 a = __half22float2(from_e4m3x2(c & 0xFFFFu)), b = __half22float2(from_e4m3x2(c >> 16));
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

constexpr int kMinExp = -126;

// The smallest e >= -126 with a <= 448 * 2^e, from the bits of a finite a >= 0: 448 = 1.75 * 2^8, so
// a = 1.f * 2^x needs x - 8 while 1.f <= 1.75, else x - 7.
__device__ __forceinline__ int need_exp(uint32_t abits) {
  const int e = (int)(abits >> 23) - 127 - 8 + ((abits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < kMinExp ? kMinExp : e;
}
__device__ __forceinline__ int scale_exp(float scale) { return (int)(__float_as_uint(scale) >> 23) - 127; }
// 2^e for e clamped to [-126, 127].
__device__ __forceinline__ float pow2i(int e) {
  e = e < -126 ? -126 : (e > 127 ? 127 : e);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Order-preserving unsigned key of an accumulated weight: NaN above everything, -0 equal to +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// ---------------------------------------------------------------------------
// Work split of the whole-cache attention.  The tiles (`tile` tokens of one
// (b, KV head)) of all sequences form one list, ordered (b, head, tile); the G
// working CTAs take consecutive shares of it, equal to within one tile whatever
// the lengths.  A share that crosses a head's end is cut there; the piece of
// unit u = b Hkv + g in CTA i has the partial-result slot i + u (both only grow
// along the list, and one grows at every cut, so no two pieces share a slot).
// A piece costs about as much as two tiles of 128 tokens (start, last O^T,
// results), so every unit counts for unit_cost more tiles than it has, in front:
// shares are equal in cost, and a CTA of many short units gets fewer tiles (64
// sequences x 8 heads of 0 .. 500 tokens: 19.8 us, 24.7 with shares equal in
// tiles, 20.9 with one tile a piece; long contexts the same).
// The list is indexed in 32 bits: B Hkv L is under 2^31, B Hkv under 2^27.
// ---------------------------------------------------------------------------
constexpr int kSms = 148, kCtasPerSm = 2;
constexpr int kMaxCols = 16;  // query rows (heads of the group x query tokens) of a unit

// Tokens of a tile: a softmax thread holds one token's row of scores, and two where the row is short
// and the token's bytes are few (cache8_attn_tc.cu).
__host__ __device__ constexpr int tile_tokens(int D, int cols) { return D == 64 && cols <= 8 ? 256 : 128; }

struct Split {
  int total;  // cost of all units, in tiles
  int G;      // CTAs with a share: as many as launched, or one per tile of cost where that is less,
              // so that no share between two others is empty
  int q, r;   // the first r CTAs take q + 1, the others q
  __device__ Split(int t, int launched) : total(t), G(t < launched ? t : launched), q(1), r(0) {
    if (t > launched) {
      q = total / G;
      r = total - q * G;
    }
  }
  __device__ bool one_each() const { return total == G; }
  __device__ int start(int i) const { return i < G ? i * q + min(i, r) : total; }
  __device__ int owner(int t) const {
    if (one_each()) return t;
    return t < r * (q + 1) ? t / (q + 1) : r + (t - r * (q + 1)) / q;
  }
};

__device__ __forceinline__ int visible(const int* lens, int b, int L, int back, int* status) {
  const int n = lens[b];
  if (n < 0 || n > L) {
    report(status, SFA_ERR_INDEX);
    return 0;
  }
  return n > back ? n - back : 0;
}

// Tiles of a head of sequence b (0: none visible).
__device__ __forceinline__ int head_tiles(const int* lens, int b, int B, int L, int back, int tile, int* status) {
  return b < B ? (visible(lens, b, L, back, status) + tile - 1) / tile : 0;
}

__device__ __forceinline__ int warp_inclusive(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += u;
  }
  return x;
}

// What a unit costs beside its tiles: nothing where every tile has a CTA to itself.
__device__ __forceinline__ int unit_cost(int tiles, int launched, int tile) {
  return tiles <= launched ? 0 : tile == 128 ? 2 : 1;
}

// One warp: cost of the whole batch (*total), the cost that each unit of it has beside its tiles, and (returned) the
// cost of the sequences before b_at.
__device__ __forceinline__ int warp_count_cost(const int* lens, int B, int Hkv, int L, int back, int tile, int launched,
                                               int b_at, int* total, int* per_unit) {
  const int lane = threadIdx.x & 31;
  int all = 0, seqs = 0, pre = 0, pre_seqs = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int t = head_tiles(lens, b0 + lane, B, L, back, tile, nullptr);
    const unsigned some = __ballot_sync(0xffffffffu, t > 0);
    const bool in_front = b0 + lane < b_at;
    pre += (int)__reduce_add_sync(0xffffffffu, (unsigned)(in_front ? t : 0));
    all += (int)__reduce_add_sync(0xffffffffu, (unsigned)t);
    pre_seqs += __popc(some & __ballot_sync(0xffffffffu, in_front));
    seqs += __popc(some);
  }
  *per_unit = unit_cost(all * Hkv, launched, tile);
  *total = (all + *per_unit * seqs) * Hkv;
  return (pre + *per_unit * pre_seqs) * Hkv;
}

// One warp: the share of CTA i of `launched`: its tiles (0: none), its first sequence, and that sequence's tiles
// before the share.
__device__ __forceinline__ int warp_share(const int* lens, int B, int Hkv, int L, int back, int tile, int launched,
                                          int i, int* b_first, int* skip, int* status) {
  const int lane = threadIdx.x & 31;
  const unsigned upto = 0xffffffffu >> (31 - lane);
  const int t0 = head_tiles(lens, lane, B, L, back, tile, status);
  const int tin0 = warp_inclusive(t0);
  int all = __shfl_sync(0xffffffffu, tin0, 31), seqs = __popc(__ballot_sync(0xffffffffu, t0 > 0));
  for (int b0 = 32; b0 < B; b0 += 32) {
    const int t = head_tiles(lens, b0 + lane, B, L, back, tile, status);
    all += (int)__reduce_add_sync(0xffffffffu, (unsigned)t);
    seqs += __popc(__ballot_sync(0xffffffffu, t > 0));
  }
  const int extra = unit_cost(all * Hkv, launched, tile);
  const Split s((all + extra * seqs) * Hkv, launched);
  const int x1 = s.start(i + 1);
  int x = s.start(i);
  *b_first = *skip = 0;
  if (x1 <= x) return 0;
  // Tiles of the list before the costs x0 and x1.
  int cost_in_front = 0, tiles_in_front = 0, from = -1;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int t = b0 == 0 ? t0 : head_tiles(lens, b0 + lane, B, L, back, tile, nullptr);
    const int tin = b0 == 0 ? tin0 : warp_inclusive(t);
    const unsigned some = __ballot_sync(0xffffffffu, t > 0);
    const int inc = cost_in_front + (tin + extra * __popc(some & upto)) * Hkv;
#pragma unroll 1
    for (;;) {
      const unsigned in = __ballot_sync(0xffffffffu, x < inc);
      if (in == 0) break;
      const int l = __ffs(in) - 1;
      const int tl = __shfl_sync(0xffffffffu, t, l), cost = tl + extra;
      const int y = x - __shfl_sync(0xffffffffu, inc, l) + cost * Hkv;  // cost into the sequence
      int g = (int)__fdividef((float)y, (float)cost);                  // off by one at most for Hkv < 2^20
      while (g * cost > y) --g;
      while (y - g * cost >= cost) ++g;
      const int here = g * tl + max(y - g * cost - extra, 0);
      const int at = tiles_in_front + __shfl_sync(0xffffffffu, tin - t, l) * Hkv + here;
      if (from >= 0) return at - from;
      from = at;
      *b_first = b0 + l;
      *skip = here;
      if (s.one_each()) return 1;
      x = x1;
    }
    cost_in_front = __shfl_sync(0xffffffffu, inc, 31);
    tiles_in_front += __shfl_sync(0xffffffffu, tin, 31) * Hkv;
  }
  return from < 0 ? 0 : tiles_in_front - from;  // to the end; 0 only if the lengths changed under the call
}

}  // namespace c8

// ---------------------------------------------------------------------------
// Launch interface (api.cu -> kernels)
// ---------------------------------------------------------------------------
struct Cache8Append {
  const void* K;
  const void* V;
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  float* weight;      // nullable
  const int* at;      // read
  const int* counts;  // nullable
  int* lens;          // written
  int* status;
  int B, Hkv, L, D, T, n, nblk;
  bool in_place;      // at == lens: the lengths advance in a kernel of their own
};

struct Cache8Attn {
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  const int* lens;
  const void* q;      // [B, Hq, nq, D]
  void* o;
  float* lse;         // nullable
  const float* w_in;  // nullable
  float* w_out;       // nullable
  int* status;
  // workspace
  float* part_ml;     // [G + U, cols, 2] running maximum (log2 units) and sum of each piece
  float* part_o;      // [G + U, cols, D]
  float* scores;      // [U, Lp, cpad] log2-unit scores (only with w_out); cpad: cols rounded up to 1, 2 or 4 n
  // list attention
  const int* idx;
  int k_list;
  int B, Hq, Hkv, L, D, T, nblk, nq, cols, cpad, back, tile, G, Lp;
  float sl2;          // softmax scale * log2(e)
};

struct Cache8Evict {
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  const int* lens;
  const float* weight;
  uint8_t* dk;
  uint8_t* dv;
  float* dks;
  float* dvs;
  int* dlens;
  float* dweight;     // nullable
  int* idx;
  int* status;
  int B, Hkv, L, D, T, nblk, dL, dnblk, keep, recent;
};

struct Cache8Gather {
  const uint8_t* k;
  const float* ks;
  void* out;
  int B, Hkv, L, D, T, nblk, nfc, pos0, npos;
  uint8_t fc[1024];
};

// Sets a kernel's dynamic shared memory (and, for kernels that live off it, the largest carve-out) once per device:
// `done` is the kernel's own word, a bit per device ordinal.  Two threads that race set the same values twice.
template <typename K>
inline cudaError_t allow_smem_once(K kern, size_t bytes, bool carveout, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && carveout) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

cudaError_t launch_cache8_append(const Cache8Append& p, cudaStream_t st);
cudaError_t launch_cache8_evict(const Cache8Evict& p, cudaStream_t st);
cudaError_t launch_cache8_gather(const Cache8Gather& p, cudaStream_t st);
// tk, tv: the code arrays as 2-D tensors of D-byte rows, boxes of D x tile, swizzle as wide as a row.
cudaError_t launch_cache8_tiles(const Cache8Attn& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st);
cudaError_t launch_cache8_attn(const Cache8Attn& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st);
cudaError_t launch_cache8_attn_list(const Cache8Attn& p, cudaStream_t st);

}  // namespace sfa
