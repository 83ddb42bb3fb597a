// 8-bit KV cache: e4m3 codes, power-of-two block scales, and how a call's work
// is split over CTAs.  Shared by cache8_store.cu and cache8_attn.cu.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

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
// Work split of the whole-cache attention.  The tiles (kTile tokens of one
// (b, KV head)) of all sequences form one list, ordered (b, head, tile); CTA i
// of the G working ones takes tiles [i T / G, (i + 1) T / G): equal shares whatever the lengths.
// A share that crosses a head's end is cut there; the piece of unit u = b Hkv + g
// in CTA i has the partial-result slot i + u (both only grow along the list, and
// one grows at every cut, so no two pieces share a slot).
// ---------------------------------------------------------------------------
constexpr int kTile = 128;
constexpr int kMaxCtas = 2 * 148;  // two per SM
constexpr int kMaxCols = 16;       // query rows (heads of the group x query tokens) of a unit

struct Split {
  long long total;  // tiles of all units
  int G;            // CTAs with a share: as many as launched, or one per tile where there are fewer
                    // tiles, so that no share between two others is empty
  __device__ Split(long long t, int launched) : total(t), G(t < launched ? (int)t : launched) {}
  __device__ long long start(int i) const { return i < G ? total * i / G : total; }
  __device__ int owner(long long t) const { return (int)(((t + 1) * G + total - 1) / total) - 1; }
};

__device__ __forceinline__ int visible(const int* lens, int b, int L, int back, int* status) {
  const int n = lens[b];
  if (n < 0 || n > L) {
    report(status, SFA_ERR_INDEX);
    return 0;
  }
  return n > back ? n - back : 0;
}

// One warp: total tiles of the batch (all heads), and the tiles before sequence b_at.
__device__ __forceinline__ long long warp_count_tiles(const int* lens, int B, int Hkv, int L, int back, int b_at,
                                                      long long* before, int* status) {
  const int lane = threadIdx.x & 31;
  long long all = 0, pre = 0;
  for (int b = lane; b < B; b += 32) {
    const long long t = (long long)((visible(lens, b, L, back, status) + kTile - 1) / kTile) * Hkv;
    all += t;
    if (b < b_at) pre += t;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    pre += __shfl_xor_sync(0xffffffffu, pre, o);
  }
  *before = pre;
  return all;
}

// One warp: the sequence that tile x of the list belongs to, and the tiles before it (x < total).
__device__ __forceinline__ int warp_find_seq(const int* lens, int B, int Hkv, int L, int back, long long x,
                                             long long* before) {
  const int lane = threadIdx.x & 31;
  long long base = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int b = b0 + lane;
    const long long t = b < B ? (long long)((visible(lens, b, L, back, nullptr) + kTile - 1) / kTile) * Hkv : 0;
    long long inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    const unsigned in = __ballot_sync(0xffffffffu, x < base + inc);
    if (in != 0) {
      const int l = __ffs(in) - 1;
      *before = base + __shfl_sync(0xffffffffu, inc - t, l);
      return b0 + l;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  *before = 0;
  return -1;
}

}  // namespace c8

// ---------------------------------------------------------------------------
// Launch interface (cache8_api.cu -> kernels)
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
  float* lse2;        // [U, cols] log2 of the sum of 2^score
  float* scores;      // [U, cols, Lp] log2-unit scores (only with w_out)
  // list attention
  const int* idx;
  int k_list;
  int B, Hq, Hkv, L, D, T, nblk, nq, cols, back, G, Lp;
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

cudaError_t launch_cache8_append(const Cache8Append& p, cudaStream_t st);
cudaError_t launch_cache8_evict(const Cache8Evict& p, cudaStream_t st);
cudaError_t launch_cache8_gather(const Cache8Gather& p, cudaStream_t st);
// tk, tv: the code arrays as 2-D tensors of D-byte rows, boxes of D x 128, swizzle as wide as a row.
cudaError_t launch_cache8_tiles(const Cache8Attn& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st);
cudaError_t launch_cache8_attn(const Cache8Attn& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st);
cudaError_t launch_cache8_attn_list(const Cache8Attn& p, cudaStream_t st);

}  // namespace sfa
