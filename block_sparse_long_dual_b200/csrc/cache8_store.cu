// 8-bit KV cache: quantising rows into it, eviction by accumulated weight, and
// the compact dominant-pair copy of its keys.
#include "cache8.cuh"

namespace sfa {

namespace {

using namespace c8;

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t block_max(uint32_t x, uint32_t* sh) {
  x = __reduce_max_sync(0xffffffffu, x);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  uint32_t m = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = max(m, sh[w]);
  return m;
}

// ---------------------------------------------------------------------------
// append: a CTA per (touched block of T tokens, (b, KV head), K or V).  The new
// rows of the block are read once into registers (16 bytes = 8 elements a
// load), their largest magnitude gives the scale, and the codes leave from the
// same registers.
// ---------------------------------------------------------------------------
template <int D, int T>
__global__ void __launch_bounds__(kThreads) append_kernel(Cache8Append p, int touched) {
  constexpr int CPR = D / 8;                  // chunks of 8 elements per row
  constexpr int CH = T * CPR / kThreads;      // chunks per thread
  __shared__ uint32_t sh[kThreads / 32];
  const int unit = blockIdx.x / touched, bi = blockIdx.x % touched;
  const int b = unit / p.Hkv, kv = blockIdx.y, tid = threadIdx.x;
  const int at = p.at[b], cnt = p.counts ? p.counts[b] : p.n;
  if (at < 0 || cnt < 0 || cnt > p.n || at > p.L - cnt) {
    if (tid == 0) report(p.status, SFA_ERR_INDEX);
    return;
  }
  const int end = at + cnt;
  if (!p.in_place && bi == 0 && kv == 0 && unit % p.Hkv == 0 && tid == 0) p.lens[b] = end;
  const int blk = at / T + bi, row0 = blk * T;
  if (cnt == 0 || row0 >= end) return;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(kv ? p.V : p.K) + (size_t)unit * p.n * D;
  uint8_t* dst = (kv ? p.v : p.k) + ((size_t)unit * p.L + row0) * D;
  float* scale = (kv ? p.vs : p.ks) + (size_t)unit * p.nblk + blk;
  const int was = row0 < at ? scale_exp(*scale) : kMinExp;

  uint4 x[CH];
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = tid + c * kThreads, row = row0 + i / CPR;
    x[c] = make_uint4(0, 0, 0, 0);
    if (row >= at && row < end)
      x[c] = __ldg(reinterpret_cast<const uint4*>(src + (size_t)(row - at) * D + (i % CPR) * 8));
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = (w[e] & 0x7FFFu) << 16, hi = w[e] & 0x7FFF0000u;
      if (lo < 0x7F800000u) top = max(top, lo);
      if (hi < 0x7F800000u) top = max(top, hi);
    }
  }
  top = block_max(top, sh);
  int ex = need_exp(top);
  const bool grown = row0 < at && ex > was;
  if (row0 < at && was > ex) ex = was;
  const float inv = pow2i(-ex);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = tid + c * kThreads, row = row0 + i / CPR;
    if (row >= at && row < end) {
      const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xFFFF0000u);
        o[e] = to_e4m3x2(isfinite(lo) ? lo * inv : NAN, isfinite(hi) ? hi * inv : NAN);
      }
      *reinterpret_cast<uint2*>(dst + (size_t)i * 8) = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
    } else if (grown && row < at) {  // earlier rows of the block move to the larger scale
      uint2* cp = reinterpret_cast<uint2*>(dst + (size_t)i * 8);
      const uint2 u = *cp;
      const float f = pow2i(was - ex);
      float a[4], d[4];
      from_e4m3x4(u.x, a);
      from_e4m3x4(u.y, d);
      *cp = make_uint2(to_e4m3x2(a[0] * f, a[1] * f) | (to_e4m3x2(a[2] * f, a[3] * f) << 16),
                       to_e4m3x2(d[0] * f, d[1] * f) | (to_e4m3x2(d[2] * f, d[3] * f) << 16));
    }
  }
  if (tid == 0) *scale = pow2i(ex);
  if (kv == 0 && p.weight != nullptr && tid < T) {
    const int row = row0 + tid;
    if (row >= at && row < end) p.weight[(size_t)unit * p.L + row] = 0.f;
  }
}

// Lengths after an append at the lengths themselves (every CTA above reads them first).
__global__ void advance_kernel(Cache8Append p) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= p.B) return;
  const int at = p.lens[b], cnt = p.counts ? p.counts[b] : p.n;
  if (at < 0 || cnt < 0 || cnt > p.n || at > p.L - cnt) return;
  p.lens[b] = at + cnt;
}

// ---------------------------------------------------------------------------
// evict, selection: a CTA per (b, KV head).  Radix select (11 + 11 + 10 bits)
// of the order-preserving weight keys, then the kept rows written in order.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(Cache8Evict p) {
  __shared__ int hist[2048];
  __shared__ int wsum[32];
  __shared__ int sh_digit, sh_above;
  const int unit = blockIdx.x, b = unit / p.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int n = p.lens[b];
  if (n < 0 || n > p.L) {
    if (tid == 0) report(p.status, SFA_ERR_INDEX);
    n = 0;
  }
  int* out = p.idx + (size_t)unit * p.keep;
  const int kept = n < p.keep ? n : p.keep;
  if (unit % p.Hkv == 0 && tid == 0) p.dlens[b] = kept;
  if (n <= p.keep) {
    for (int i = tid; i < p.keep; i += kSelThreads) out[i] = i < n ? i : -1;
    return;
  }
  const int old = n - p.recent, want = p.keep - p.recent;
  const float* w = p.weight + (size_t)unit * p.L;
  for (int i = tid; i < p.recent; i += kSelThreads) out[want + i] = old + i;
  if (want == 0) return;

  uint32_t prefix = 0;
  int need = want;  // how many of the keys that match the prefix are kept
  const int shift[4] = {21, 10, 0, 0}, bits[3] = {11, 11, 10};
  for (int pass = 0; pass < 3; ++pass) {
    const int nb = 1 << bits[pass];
    for (int i = tid; i < nb; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < old; i += kSelThreads) {
      const uint32_t key = weight_key(w[i]);
      if (pass == 0 || (key >> shift[pass - 1]) == prefix) atomicAdd(&hist[(key >> shift[pass]) & (nb - 1)], 1);
    }
    __syncthreads();
    // suffix sums: thread t owns the bins [nb - per (t + 1), nb - per t), from the top down
    const int per = nb / kSelThreads;  // 2 or 1
    int c[2] = {0, 0}, mine = 0;
    for (int j = 0; j < per; ++j) { c[j] = hist[nb - 1 - (tid * per + j)]; mine += c[j]; }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int before = inc - mine;
    for (int q = 0; q < warp; ++q) before += wsum[q];
    for (int j = 0; j < per; ++j) {
      if (before < need && before + c[j] >= need) {
        sh_digit = nb - 1 - (tid * per + j);
        sh_above = before;
      }
      before += c[j];
    }
    __syncthreads();
    prefix = (prefix << bits[pass]) | (uint32_t)sh_digit;
    need -= sh_above;
    __syncthreads();
  }
  // key > prefix: kept; key == prefix: the first `need` of them.  4096 rows at a time, in order.
  int gt_done = 0, eq_done = 0;
  for (int base = 0; base < old; base += 4 * kSelThreads) {
    uint32_t key[4];
    uint32_t pk = 0;  // (greater << 16) | equal, over this thread's four rows
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = base + tid * 4 + j;
      key[j] = i < old ? weight_key(w[i]) : 0u;
      if (i < old) pk += key[j] > prefix ? 65536u : (key[j] == prefix ? 1u : 0u);
    }
    uint32_t inc = pk;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) wsum[warp] = (int)inc;
    __syncthreads();
    uint32_t before = inc - pk, all = 0;
    for (int q = 0; q < kSelThreads / 32; ++q) {
      const uint32_t v = (uint32_t)wsum[q];
      if (q < warp) before += v;
      all += v;
    }
    int gt = gt_done + (int)(before >> 16), eq = eq_done + (int)(before & 0xFFFFu);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = base + tid * 4 + j;
      if (i >= old) break;
      if (key[j] > prefix) {
        out[gt + min(eq, need)] = i;
        ++gt;
      } else if (key[j] == prefix) {
        if (eq < need) out[gt + eq] = i;
        ++eq;
      }
    }
    gt_done += (int)(all >> 16);
    eq_done += (int)(all & 0xFFFFu);
    __syncthreads();
  }
}

// evict, move: a CTA per (dst block, (b, KV head), K or V).  e4m3 magnitudes order like their 7-bit
// codes, so the scale a row needs comes from its largest code and its old exponent, in integers.
template <int D, int T>
__global__ void __launch_bounds__(kThreads) evict_move_kernel(Cache8Evict p, int nblocks) {
  constexpr int CPR = D / 16;             // 16-byte chunks per row
  constexpr int CH = T * CPR / kThreads;  // chunks per thread
  __shared__ uint32_t sh[kThreads / 32];
  const int unit = blockIdx.x / nblocks, blk = blockIdx.x % nblocks;
  const int kv = blockIdx.y, tid = threadIdx.x;
  const int* list = p.idx + (size_t)unit * p.keep + (size_t)blk * T;
  const int rows = min(T, p.keep - blk * T);
  if (list[0] < 0) return;  // nothing was kept here (the list is padded at its end)
  const uint8_t* src = (kv ? p.v : p.k) + (size_t)unit * p.L * D;
  const float* scale = (kv ? p.vs : p.ks) + (size_t)unit * p.nblk;
  uint8_t* dst = (kv ? p.dv : p.dk) + ((size_t)unit * p.dL + (size_t)blk * T) * D;
  uint4 x[CH];
  int ex[CH], at[CH];
  int need = kMinExp;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = tid + c * kThreads, r = i / CPR;
    at[c] = r < rows ? list[r] : -1;
    x[c] = make_uint4(0, 0, 0, 0);
    ex[c] = kMinExp;
    if (at[c] >= 0) {
      x[c] = __ldg(reinterpret_cast<const uint4*>(src + (size_t)at[c] * D + (i % CPR) * 16));
      ex[c] = scale_exp(__ldg(scale + at[c] / T));
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t a = w[e] & 0x7F7F7F7Fu;
      m = __vmaxu4(m, a & ~__vcmpeq4(a, 0x7F7F7F7Fu));  // NaN codes do not count
    }
    m = __vmaxu4(m, m >> 16);
    m = __vmaxu4(m, m >> 8) & 0x7Fu;
    if (m != 0) need = max(need, need_exp(__float_as_uint(__half2float(__low2half(from_e4m3x2(m))))) + ex[c]);
  }
  need = (int)block_max((uint32_t)(need - kMinExp), sh) + kMinExp;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (at[c] < 0) continue;
    uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
    if (ex[c] != need) {
      const float f = pow2i(ex[c] - need);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v[4];
        from_e4m3x4(w[e], v);
        w[e] = to_e4m3x2(v[0] * f, v[1] * f) | (to_e4m3x2(v[2] * f, v[3] * f) << 16);
      }
    }
    *reinterpret_cast<uint4*>(dst + (size_t)(tid + c * kThreads) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (tid == 0) (kv ? p.dvs : p.dks)[(size_t)unit * p.dnblk + blk] = pow2i(need);
  if (kv == 0 && p.dweight != nullptr && tid < rows && list[tid] >= 0)
    p.dweight[(size_t)unit * p.dL + blk * T + tid] = p.weight[(size_t)unit * p.L + list[tid]];
}

// ---------------------------------------------------------------------------
// gather: a thread per (token, pair of adjacent output columns)
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ Cache8Gather p) {
  const size_t items = (size_t)p.B * p.Hkv * p.npos * p.nfc;  // bf16 pairs
  for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < items; i += (size_t)gridDim.x * kThreads) {
    const int c = (int)(i % p.nfc) * 2;  // column pair (c, c + 1); nfc is even, so both lie in one half
    size_t r = i / p.nfc;
    const int t = p.pos0 + (int)(r % p.npos);
    const size_t unit = r / p.npos;
    const int g = (int)(unit % p.Hkv);
    const int hi = c >= p.nfc ? p.D / 2 : 0, cc = c >= p.nfc ? c - p.nfc : c;
    const uint8_t* row = p.k + (unit * p.L + t) * p.D + hi;
    const uint32_t a = row[p.fc[g * p.nfc + cc]], d = row[p.fc[g * p.nfc + cc + 1]];
    const float f = p.ks[unit * p.nblk + t / p.T];
    const float2 v = __half22float2(from_e4m3x2(a | (d << 8)));
    reinterpret_cast<uint32_t*>(p.out)[(unit * p.L + t) * p.nfc + c / 2] = pack_bf16x2(v.x * f, v.y * f);
  }
}

}  // namespace

cudaError_t launch_cache8_append(const Cache8Append& p, cudaStream_t st) {
  const int touched = (int)(((long long)p.n + p.T - 2) / p.T) + 1;  // blocks n rows can touch
  const int most = (p.L + p.T - 1) / p.T;
  const int nb = touched < most ? touched : most;
  const long long gx = (long long)nb * p.B * p.Hkv;
  if (gx > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)gx, 2);
  if (p.D == 128) {
    if (p.T == 128) append_kernel<128, 128><<<grid, kThreads, 0, st>>>(p, nb);
    else append_kernel<128, 64><<<grid, kThreads, 0, st>>>(p, nb);
  } else {
    if (p.T == 128) append_kernel<64, 128><<<grid, kThreads, 0, st>>>(p, nb);
    else append_kernel<64, 64><<<grid, kThreads, 0, st>>>(p, nb);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.in_place) return e;
  advance_kernel<<<(p.B + 127) / 128, 128, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_cache8_evict(const Cache8Evict& p, cudaStream_t st) {
  evict_select_kernel<<<p.B * p.Hkv, kSelThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int most = p.keep < p.L ? p.keep : p.L;
  const int nb = (most + p.T - 1) / p.T;
  const long long gx = (long long)nb * p.B * p.Hkv;
  if (gx > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)gx, 2);
  if (p.D == 128) {
    if (p.T == 128) evict_move_kernel<128, 128><<<grid, kThreads, 0, st>>>(p, nb);
    else evict_move_kernel<128, 64><<<grid, kThreads, 0, st>>>(p, nb);
  } else {
    if (p.T == 128) evict_move_kernel<64, 128><<<grid, kThreads, 0, st>>>(p, nb);
    else evict_move_kernel<64, 64><<<grid, kThreads, 0, st>>>(p, nb);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache8_gather(const Cache8Gather& p, cudaStream_t st) {
  const size_t items = (size_t)p.B * p.Hkv * p.npos * p.nfc;
  if (items == 0) return cudaSuccess;
  size_t blocks = (items + kThreads - 1) / kThreads;
  if (blocks > (size_t)148 * 32) blocks = (size_t)148 * 32;
  gather_kernel<<<(unsigned)blocks, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace sfa
