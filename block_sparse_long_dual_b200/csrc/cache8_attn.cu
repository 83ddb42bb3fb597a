// Attention over the 8-bit KV cache: joining the pieces of the whole-cache attention
// (cache8_attn_tc.cu), the accumulated weights, and index lists.
#include <math.h>

#include "cache8.cuh"

namespace sfa {

namespace {

using namespace c8;

constexpr float kLn2 = 0.6931471805599453f;

// Joins the pieces of one (unit, query row): CTA per (row, unit), a thread per dim.
template <int D>
__global__ void __launch_bounds__(D) attn_join_kernel(Cache8Attn p) {
  __shared__ long long sh_total, sh_t0;
  const int unit = blockIdx.x / p.cols, c = blockIdx.x % p.cols, b = unit / p.Hkv, g = unit % p.Hkv;
  const int tid = threadIdx.x;
  const int nv = visible(p.lens, b, p.L, p.back, nullptr);
  const int tiles = (nv + kTile - 1) / kTile;
  if (tid < 32) {
    long long before;
    const long long total = warp_count_tiles(p.lens, p.B, p.Hkv, p.L, p.back, b, &before, nullptr);
    if (tid == 0) { sh_total = total; sh_t0 = before + (long long)g * tiles; }
  }
  __syncthreads();
  float M = -INFINITY, L = 0.f, o = 0.f;
  if (tiles > 0) {
    const Split s(sh_total, p.G);
    const int i0 = s.owner(sh_t0), i1 = s.owner(sh_t0 + tiles - 1);
    for (int i = i0; i <= i1; ++i) M = fmaxf(M, p.part_ml[(((size_t)i + unit) * p.cols + c) * 2]);
    const float base = M == -INFINITY ? 0.f : M;
    for (int i = i0; i <= i1; ++i) {
      const size_t slot = ((size_t)i + unit) * p.cols + c;
      const float f = exp2f(p.part_ml[slot * 2] - base);
      L += p.part_ml[slot * 2 + 1] * f;
      o = fmaf(p.part_o[slot * D + tid], f, o);
    }
  }
  // L = 0 exactly when the row sees no token (a NaN score makes L NaN, and the row's o)
  const size_t row = (size_t)unit * p.cols + c;
  static_cast<__nv_bfloat16*>(p.o)[row * D + tid] = __float2bfloat16_rn(L == 0.f ? 0.f : o / L);
  if (tid == 0) {
    const float l2 = L == 0.f ? -INFINITY : (M == -INFINITY ? 0.f : M) + log2f(L);
    if (p.lse != nullptr) p.lse[row] = l2 * kLn2;
    if (p.w_out != nullptr) p.lse2[row] = l2;
  }
}

// Adds each token's attention weight, summed over the unit's query rows in order.
__global__ void __launch_bounds__(256) attn_weight_kernel(Cache8Attn p, int chunks) {
  const int unit = blockIdx.x / chunks, b = unit / p.Hkv;
  const int nv = visible(p.lens, b, p.L, p.back, nullptr);
  const int t = (blockIdx.x % chunks) * 256 + threadIdx.x;
  if (t >= nv) return;
  const float* s = p.scores + (size_t)unit * p.cols * p.Lp + t;
  float w = 0.f;
  for (int c = 0; c < p.cols; ++c) {
    const float x = s[(size_t)c * p.Lp];
    if (x != -INFINITY) w += exp2f(x - p.lse2[unit * p.cols + c]);
  }
  const size_t at = (size_t)unit * p.L + t;
  p.w_out[at] = p.w_in != nullptr ? p.w_in[at] + w : w;
}

// ---------------------------------------------------------------------------
// Index lists: CTA per (b, q head).  A row of d codes is read by d / 16 lanes,
// 16 bytes each; each such lane group runs its own online softmax over its
// tokens, kListBatch of them with both loads in flight, and the groups are
// joined at the end.
// ---------------------------------------------------------------------------
constexpr int kListBatch = 4;

template <int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) attn_list_kernel(Cache8Attn p) {
  constexpr int LPT = D / 16, GROUPS = WARPS * 32 / LPT;
  __shared__ float gm[GROUPS], gl[GROUPS];
  __shared__ float go[GROUPS][D + 4];
  __shared__ int bad;
  const int row = blockIdx.x, b = row / p.Hq, h = row % p.Hq, g = h / (p.Hq / p.Hkv);
  const int unit = b * p.Hkv + g;
  const int tid = threadIdx.x, grp = tid / LPT, part = tid % LPT;
  const int* list = p.idx + (size_t)row * p.k_list;
  if (tid == 0) bad = 0;
  __syncthreads();
  const int n = visible(p.lens, b, p.L, 0, tid == 0 ? p.status : nullptr);
  float q[16];
  {
    const uint4* qr = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (size_t)row * D + part * 16);
    const uint4 u[2] = {__ldg(qr), __ldg(qr + 1)};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q[j * 8 + 2 * e] = __uint_as_float(w[e] << 16);
        q[j * 8 + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
      }
    }
  }
  float m = -INFINITY, l = 0.f, acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  // the warp's groups walk the list together (a group past the end has no token): the shuffles need all lanes
  for (int base = 0; base < p.k_list; base += GROUPS * kListBatch) {
    int tok[kListBatch];
    uint4 ku[kListBatch], vu[kListBatch];
    float ks[kListBatch], vs[kListBatch];
#pragma unroll
    for (int u = 0; u < kListBatch; ++u) {
      const int j = base + u * GROUPS + grp;
      int t = j < p.k_list ? __ldg(list + j) : -1;
      if (t >= n || t < -1) {
        bad = 1;
        t = -1;
      }
      tok[u] = t;
    }
#pragma unroll
    for (int u = 0; u < kListBatch; ++u) {
      ku[u] = vu[u] = make_uint4(0, 0, 0, 0);
      ks[u] = vs[u] = 0.f;
      if (tok[u] >= 0) {
        const size_t at = ((size_t)unit * p.L + tok[u]) * D + part * 16;
        ku[u] = __ldg(reinterpret_cast<const uint4*>(p.k + at));
        vu[u] = __ldg(reinterpret_cast<const uint4*>(p.v + at));
        ks[u] = __ldg(p.ks + (size_t)unit * p.nblk + tok[u] / p.T);
        vs[u] = __ldg(p.vs + (size_t)unit * p.nblk + tok[u] / p.T);
      }
    }
#pragma unroll
    for (int u = 0; u < kListBatch; ++u) {
      const uint32_t kw[4] = {ku[u].x, ku[u].y, ku[u].z, ku[u].w};
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float kv[4];
        from_e4m3x4(kw[e], kv);
#pragma unroll
        for (int z = 0; z < 4; ++z) s = fmaf(q[e * 4 + z], kv[z], s);
      }
#pragma unroll
      for (int o = LPT / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (tok[u] < 0) continue;
      s *= ks[u] * p.sl2;
      const float mn = fmaxf(m, s), mb = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m - mb), e = exp2f(s - mb);
      l = l * f + e;
      const float ev = e * vs[u];
      const uint32_t vw[4] = {vu[u].x, vu[u].y, vu[u].z, vu[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float vv[4];
        from_e4m3x4(vw[i], vv);
#pragma unroll
        for (int z = 0; z < 4; ++z) acc[i * 4 + z] = fmaf(acc[i * 4 + z], f, ev * vv[z]);
      }
      m = mn;
    }
  }
  if (part == 0) { gm[grp] = m; gl[grp] = l; }
#pragma unroll
  for (int e = 0; e < 16; ++e) go[grp][part * 16 + e] = acc[e];
  __syncthreads();
  if (bad && tid == 0) report(p.status, SFA_ERR_INDEX);
  if (tid < D) {
    float M = -INFINITY, L = 0.f, o = 0.f;
    for (int i = 0; i < GROUPS; ++i) M = fmaxf(M, gm[i]);
    const float base = M == -INFINITY ? 0.f : M;
    for (int i = 0; i < GROUPS; ++i) {
      const float f = exp2f(gm[i] - base);
      L += gl[i] * f;
      o = fmaf(go[i][tid], f, o);
    }
    const bool none = bad || L == 0.f;
    static_cast<__nv_bfloat16*>(p.o)[(size_t)row * D + tid] = __float2bfloat16_rn(none ? 0.f : o / L);
    if (tid == 0 && p.lse != nullptr) p.lse[row] = none ? -INFINITY : (base + log2f(L)) * kLn2;
  }
}

}  // namespace

cudaError_t launch_cache8_attn(const Cache8Attn& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  cudaError_t e = launch_cache8_tiles(p, tk, tv, st);
  if (e != cudaSuccess) return e;
  const unsigned rows = (unsigned)(p.B * p.Hkv * p.cols);
  if (p.D == 128) attn_join_kernel<128><<<rows, 128, 0, st>>>(p);
  else attn_join_kernel<64><<<rows, 64, 0, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.w_out == nullptr) return e;
  const int chunks = (p.L + 255) / 256;
  attn_weight_kernel<<<(unsigned)(chunks * p.B * p.Hkv), 256, 0, st>>>(p, chunks);
  return cudaGetLastError();
}

cudaError_t launch_cache8_attn_list(const Cache8Attn& p, cudaStream_t st) {
  const unsigned rows = (unsigned)(p.B * p.Hq);
  if (p.D == 128) attn_list_kernel<128, 8><<<rows, 256, 0, st>>>(p);
  else attn_list_kernel<64, 8><<<rows, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace sfa
