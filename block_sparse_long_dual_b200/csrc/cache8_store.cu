// 8-bit KV cache: quantising rows into it, eviction by accumulated weight, and
// the compact dominant-pair copy of its keys.
#include <cooperative_groups.h>

#include "cache8.cuh"
#include "tc_ptx8.cuh"

namespace sfa {

namespace {

using namespace c8;
namespace cg = cooperative_groups;

constexpr int kThreads = 256;

template <int THREADS>
__device__ __forceinline__ uint32_t block_max(uint32_t x, uint32_t* sh) {
  x = __reduce_max_sync(0xffffffffu, x);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  uint32_t m = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) m = max(m, sh[w]);
  return m;
}

// ---------------------------------------------------------------------------
// append: a CTA per (touched block of T tokens, (b, KV head), K or V).  The new
// rows of the block are read once into registers (16 bytes = 8 elements a
// load), their largest magnitude gives the scale, and the codes leave from the
// same registers.  Bound by the bytes of the rows.  Load, reduce and store of one
// CTA do not overlap, so the CTAs of an SM have to: 64 registers a thread, four CTAs
// (a 131072-token prompt of 8 heads, 810 MB: 115 us, 7.0 TB/s, above the measured
// copy rate, which writes half its bytes; 149 us with two, 122 with three, 151 with
// five, which spill).
// ---------------------------------------------------------------------------
constexpr int kAppend = 256;

template <int D, int T>
__global__ void __launch_bounds__(kAppend, 4) append_kernel(Cache8Append p, int touched) {
  constexpr int CPR = D / 8;                  // chunks of 8 elements per row
  constexpr int CH = T * CPR / kAppend;      // chunks per thread
  __shared__ uint32_t sh[kAppend / 32];
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
    const int i = tid + c * kAppend, row = row0 + i / CPR;
    x[c] = make_uint4(0, 0, 0, 0);
    if (row >= at && row < end)
      x[c] = __ldg(reinterpret_cast<const uint4*>(src + (size_t)(row - at) * D + (i % CPR) * 8));
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {  // bf16 magnitudes order like their bits: two at a time
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[c].x & 0x7FFF7FFFu, x[c].y & 0x7FFF7FFFu),
                                 __vmaxu2(x[c].z & 0x7FFF7FFFu, x[c].w & 0x7FFF7FFFu)));
  }
  top = block_max<kAppend>(max(top & 0xFFFFu, top >> 16), sh);
  const bool finite = top < 0x7F80u;
  if (!finite) {  // an infinity or NaN somewhere in the block: the largest of the others
    top = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = w[e] & 0x7FFFu, hi = (w[e] >> 16) & 0x7FFFu;
        top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
      }
    }
    __syncthreads();  // sh has been read
    top = block_max<kAppend>(top, sh);
  }
  top <<= 16;
  int ex = need_exp(top);
  const bool grown = row0 < at && ex > was;
  if (row0 < at && was > ex) ex = was;
  const float inv = pow2i(-ex);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = tid + c * kAppend, row = row0 + i / CPR;
    if (row >= at && row < end) {
      uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint64_t v = tc::f2_mul(tc::f2_pack(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u)),
                                tc::f2_pack(inv, inv));
        float lo, hi;
        tc::f2_unpack(v, lo, hi);
        o[e] = to_e4m3x2(lo, hi);
      }
      if (!finite) {  // infinities (that the conversion would saturate) become NaN like NaN itself
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if ((w[e] & 0x7FFFu) >= 0x7F80u) o[e] = (o[e] & 0xFF00u) | 0x7Fu;
          if ((w[e] & 0x7FFF0000u) >= 0x7F800000u) o[e] = (o[e] & 0xFFu) | 0x7F00u;
        }
      }
      *reinterpret_cast<uint2*>(dst + (size_t)i * 8) =
          make_uint2(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410));
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
// evict, selection: a cluster of CS CTAs per (b, KV head), each over a contiguous
// slice of the tokens.  Radix select (11 + 11 + 10 bits) of the order-preserving
// weight keys.  The slices' histograms are summed through distributed shared
// memory, each CTA an eighth of the bins (all bins in every CTA: 59 against 54.8
// us); every CTA then finds the eighth and the bin of the threshold.  A slice's
// own histogram also tells how many kept rows lie before the next slice's.  The
// slice stays in shared memory through all passes (a longer one is read again in
// each pass): copied there asynchronously, all of it on its way at once, 16 bytes a
// copy where the slice starts on 16 bytes (51.4 us, 52.7 with 4 bytes each); the
// first pass puts the keys in place.  The loops are short code: unrolled code
// that runs once waits for its instructions (keys in registers: 7 us more).
// One histogram serves: with two or four copies, lanes apart, 53.5 and 55.5 us
// against 53.3, with equal weights everywhere 57.5 against 57.2.
// 131072 -> 8192 tokens of 4 x 8 heads (the times above are this whole eviction's,
// now 52 us): the selection takes 25 us for 17 MB, bound by the latencies of its steps
// (histograms 6 us, meetings and sums 9, the copy 3, the list 2).
// ---------------------------------------------------------------------------
constexpr int kSlice = 16384;  // keys in shared memory
constexpr int kBins = 2048;
constexpr size_t kSelSmem = ((size_t)kSlice + kBins) * sizeof(uint32_t);

// Exclusive sum over the block of a 32-bit value.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* wsum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();  // wsum may still be read from the call before
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane] : 0u) + inc - x;
}

template <int CS, int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const __grid_constant__ Cache8Evict p) {
  constexpr int kBpt = kBins / kSelThreads;  // bins per thread
  extern __shared__ __align__(16) uint32_t sel_smem[];
  uint32_t* key = sel_smem;             // [kSlice]
  uint32_t* hist = sel_smem + kSlice;   // [kBins]
  __shared__ uint32_t part[CS > 1 ? kBins / CS : 1];  // this CTA's share of the bins, over all slices
  __shared__ uint32_t ptotal[2];  // and their sum (two: the next pass begins while others read)
  __shared__ uint32_t wsum[kSelThreads / 32];
  __shared__ uint32_t share[2];  // this slice's keys above and at the threshold
  __shared__ uint32_t sh_digit, sh_above;
  // The moving CTAs may start (they wait for this grid's end).  Beside clusters they have no room and gain nothing.
  if (CS == 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = CS == 1 ? 0 : (int)cluster.block_rank();
  const int unit = blockIdx.x / CS, b = unit / p.Hkv, tid = threadIdx.x, lane = tid & 31;
  int n = p.lens[b];
  if (n < 0 || n > p.L) {
    if (tid == 0) report(p.status, SFA_ERR_INDEX);
    n = 0;
  }
  int* out = p.idx + (size_t)unit * p.keep;
  if (unit % p.Hkv == 0 && rank == 0 && tid == 0) p.dlens[b] = n < p.keep ? n : p.keep;
  if (n <= p.keep) {
    for (int i = rank * kSelThreads + tid; i < p.keep; i += CS * kSelThreads) out[i] = i < n ? i : -1;
    return;
  }
  const int old = n - p.recent, want = p.keep - p.recent;
  for (int i = rank * kSelThreads + tid; i < p.recent; i += CS * kSelThreads) out[want + i] = old + i;
  if (want == 0) return;

  const int per = ((old + CS - 1) / CS + 3) & ~3, lo = min(rank * per, old), hi = min(lo + per, old);
  const float* w = p.weight + (size_t)unit * p.L;
  int first = lo, cnt = 0;  // the keys in shared memory: rows [first, first + cnt)
  auto load = [&](int from) {
    __syncthreads();  // everyone is done with the keys before
    first = from;
    cnt = min(kSlice, hi - from);
    const int quads = (reinterpret_cast<uintptr_t>(w + from) & 15) == 0 ? cnt / 4 : 0;
#pragma unroll 2
    for (int i = tid; i < quads; i += kSelThreads)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(key + 4 * i)), "l"(w + from + 4 * i)
                   : "memory");
#pragma unroll 4
    for (int i = 4 * quads + tid; i < cnt; i += kSelThreads)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::smem_u32(key + i)), "l"(w + from + i) : "memory");
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
  };
  const bool whole = hi - lo <= kSlice;
  if (tid < 2) share[tid] = 0;
  for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
  if (whole) load(lo);
  else __syncthreads();

  uint32_t prefix = 0, need = (uint32_t)want;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), up = pass == 1 ? 21 : 10;
    const uint32_t mask = pass == 2 ? 1023u : 2047u;  // (the last pass leaves the upper bins empty)
    for (int from = lo; from < hi; from += kSlice) {
      if (!whole) load(from);
#pragma unroll 2
      for (int i = 4 * tid; i < cnt; i += 4 * kSelThreads) {
        uint4* at = reinterpret_cast<uint4*>(key + i);
        uint4 x = *at;
        if (pass == 0 || !whole) {
          x = make_uint4(weight_key(__uint_as_float(x.x)), weight_key(__uint_as_float(x.y)),
                         weight_key(__uint_as_float(x.z)), weight_key(__uint_as_float(x.w)));
          if (whole) *at = x;
        }
        const uint32_t k[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j < cnt && (pass == 0 || (k[j] >> up) == prefix)) atomicAdd(hist + ((k[j] >> shift) & mask), 1u);
      }
    }
    __syncthreads();
    // Thread t owns the kBpt bins from bin0 on, the first thread the top ones: an exclusive sum over t runs from the
    // top bin down.
    const int bin0 = kBins - kBpt * (tid + 1);
    uint32_t own[kBpt];
#pragma unroll
    for (int j = 0; j < kBpt; j += 2) {
      const uint2 u = *reinterpret_cast<const uint2*>(hist + bin0 + j);
      own[j] = u.x;
      own[j + 1] = u.y;
    }
    if (CS > 1) {
      constexpr int PB = kBins / CS;
      if (tid == 0) ptotal[pass & 1] = 0;
      cluster.sync();
      if (tid < PB) {
        uint32_t v = 0;
#pragma unroll
        for (int q = 0; q < CS; ++q) v += cluster.map_shared_rank(hist, q)[rank * PB + tid];
        part[tid] = v;
        v = __reduce_add_sync(0xffffffffu, v);
        if (lane == 0 && v != 0) atomicAdd(&ptotal[pass & 1], v);
      }
      cluster.sync();
      // The eighth that holds the threshold (from the top down), and the keys above it.
      const uint32_t t = lane < CS ? *cluster.map_shared_rank(&ptotal[pass & 1], CS - 1 - lane) : 0u;
      uint32_t run = 0, skipped = 0;
      int e = -1;
#pragma unroll
      for (int q = 0; q < CS; ++q) {
        const uint32_t v = __shfl_sync(0xffffffffu, t, q);
        if (e < 0 && run + v >= need) {
          e = CS - 1 - q;
          skipped = run;
        }
        run += v;
      }
      const uint32_t v = tid < PB ? cluster.map_shared_rank(part, e)[PB - 1 - tid] : 0u;
      const uint32_t before = skipped + block_scan(v, wsum);
      if (tid < PB && before < need && before + v >= need) {
        sh_digit = (uint32_t)(e * PB + PB - 1 - tid);
        sh_above = before;
      }
    } else {
      uint32_t all = 0;
#pragma unroll
      for (int j = 0; j < kBpt; ++j) all += own[j];
      uint32_t before = block_scan(all, wsum);
#pragma unroll
      for (int j = kBpt - 1; j >= 0; --j) {
        if (before < need && before + own[j] >= need) {
          sh_digit = (uint32_t)(bin0 + j);
          sh_above = before;
        }
        before += own[j];
      }
    }
#pragma unroll
    for (int j = 0; j < kBpt; j += 2) *reinterpret_cast<uint2*>(hist + bin0 + j) = make_uint2(0, 0);
    __syncthreads();
    const uint32_t digit = sh_digit;
    uint32_t above = 0;
#pragma unroll
    for (int j = 0; j < kBpt; ++j) {
      const uint32_t bin = (uint32_t)(bin0 + j);
      if (bin > digit) above += own[j];
      if (pass == 2 && bin == digit) share[1] = own[j];
    }
    above = __reduce_add_sync(0xffffffffu, above);
    if (lane == 0 && above != 0) atomicAdd(&share[0], above);
    prefix = pass == 0 ? digit : (prefix << (pass == 1 ? 11 : 10)) | digit;
    need -= sh_above;
    __syncthreads();  // sh_digit, sh_above are written again in the next pass
  }
  // key > prefix: kept; key == prefix: the first `need` of them over the whole head.
  uint32_t gt = 0, eq = 0;
  if (CS > 1) {
    cluster.sync();
    for (int q = 0; q < rank; ++q) {
      const uint32_t* o = cluster.map_shared_rank(share, q);
      gt += o[0];
      eq += o[1];
    }
  }
  for (int from = lo; from < hi; from += kSlice) {
    if (!whole) load(from);
    // Rows of 32 keys, a warp's one after the other, each lane with the votes of one of them.
    const int rows = (cnt + 31) / 32, per_warp = (rows + kSelThreads / 32 - 1) / (kSelThreads / 32);
    const int row0 = (tid >> 5) * per_warp;
    uint32_t vg = 0, ve = 0;
#pragma unroll 4
    for (int r = 0; r < per_warp; ++r) {
      const int i = (row0 + r) * 32 + lane;
      uint32_t k = i < cnt ? key[i] : 0u;
      if (!whole) k = weight_key(__uint_as_float(k));
      const uint32_t g = __ballot_sync(0xffffffffu, i < cnt && k > prefix);
      const uint32_t e = __ballot_sync(0xffffffffu, i < cnt && k == prefix);
      if (lane == r) { vg = g; ve = e; }
    }
    const uint32_t before = block_scan(((uint32_t)__popc(vg) << 16) | (uint32_t)__popc(ve), wsum);  // 16384 keys at most
    uint32_t g = gt + (before >> 16), e = eq + (before & 0xFFFFu);
    uint32_t v = vg | ve;
    if ((int)__reduce_max_sync(0xffffffffu, (unsigned)__popc(v)) <= per_warp) {  // a lane a row
      const int row = first + (row0 + lane) * 32;
      for (; v != 0; v &= v - 1) {
        const int at = __ffs(v) - 1;
        const bool more = (vg >> at) & 1u;
        if (more || e < need) out[g + min(e, need)] = row + at;
        g += more;
        e += !more;
      }
    } else {  // a lane a key
      const uint32_t under = (1u << lane) - 1u;
#pragma unroll 1
      for (int r = 0; r < per_warp; ++r) {
        const uint32_t rg = __shfl_sync(0xffffffffu, vg, r), re = __shfl_sync(0xffffffffu, ve, r);
        const uint32_t kg = __shfl_sync(0xffffffffu, g, r) + __popc(rg & under);
        const uint32_t ke = __shfl_sync(0xffffffffu, e, r) + __popc(re & under);
        const bool more = (rg >> lane) & 1u;
        if (more || (((re >> lane) & 1u) && ke < need)) out[kg + min(ke, need)] = first + (row0 + r) * 32 + lane;
      }
    }
    if (!whole) {  // wsum still holds the warps' totals
      const uint32_t all = __reduce_add_sync(0xffffffffu, lane < kSelThreads / 32 ? wsum[lane] : 0u);
      gt += all >> 16;
      eq += all & 0xFFFFu;
    }
  }
  if (CS > 1) cluster.sync();  // the other CTAs have read this one's shared memory
}

template <int CS, int kSelThreads>
static cudaError_t launch_select(const Cache8Evict& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem_once(evict_select_kernel<CS, kSelThreads>, kSelSmem, false, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = kSelSmem;
  cfg.gridDim = dim3((unsigned)(p.B * p.Hkv * CS));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CS;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CS > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<CS, kSelThreads>, p);
}

// evict, move: a CTA per (dst block, (b, KV head), K or V), eight to an SM (two dependent loads, a reduction and a
// store have to overlap between CTAs: 137 MB of rows read and written in 23 us, 91% of the measured copy rate; the
// whole eviction of 131072 -> 8192 tokens of 4 x 8 heads 52.7 us when it was tried, 53.4 with six CTAs, 57.2 with four).
// Eight CTAs leave 32 registers a thread: d 128 with 128-token blocks spills 16 bytes of them.  e4m3 magnitudes order
// like their 7-bit codes, so the scale a row needs comes from its largest code and its old exponent, in integers.
template <int D, int T>
__global__ void __launch_bounds__(kThreads, 8) evict_move_kernel(const __grid_constant__ Cache8Evict p, int nblocks) {
  constexpr int CPR = D / 16;             // 16-byte chunks per row
  constexpr int CH = T * CPR / kThreads;  // chunks per thread
  __shared__ uint32_t sh[kThreads / 32];
  const int unit = blockIdx.x / nblocks, blk = blockIdx.x % nblocks;
  const int kv = blockIdx.y, tid = threadIdx.x;
  const int* list = p.idx + (size_t)unit * p.keep + (size_t)blk * T;
  const int rows = min(T, p.keep - blk * T);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched beside the selection: its lists are complete
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
  // The largest magnitude of the chunk's 16 codes, two bytes a word at a time; 0x7F is NaN, which does not count.
  auto top_code = [](const uint4& u, bool skip_nan) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t a = w[e] & 0x007F007Fu, d = (w[e] >> 8) & 0x007F007Fu;
      if (skip_nan) {
        a &= ~__vcmpeq2(a, 0x007F007Fu);
        d &= ~__vcmpeq2(d, 0x007F007Fu);
      }
      m = __vmaxu2(m, __vmaxu2(a, d));
    }
    return max(m & 0xFFFFu, m >> 16);
  };
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    uint32_t m = top_code(x[c], false);
    if (m == 0x7Fu) m = top_code(x[c], true);
    if (m != 0) need = max(need, need_exp(__float_as_uint(__half2float(__low2half(from_e4m3x2(m))))) + ex[c]);
  }
  need = (int)block_max<kThreads>((uint32_t)(need - kMinExp), sh) + kMinExp;
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
// gather: a CTA per 128 tokens of one (b, KV head).  The dominant dims touch nearly every 32-byte
// sector of a row, so whole rows are read, 16 bytes a lane, and staged in shared memory (row stride
// D + 4 bytes: the byte reads of neighbouring tokens fall into different banks); the output leaves
// four bytes (two columns) a thread, contiguous over the CTA's tokens.  131072 tokens x 4 x 8 heads, 12 pairs, d 128:
// 537 MB read and 201 MB written in 124 us replayed in a graph, 5.9 TB/s (91% of the measured copy rate), in 126 to 140
// us called from Python: bound by those bytes, and by 74% of the issue slots beside them.
// ---------------------------------------------------------------------------
constexpr int kGatherTokens = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ Cache8Gather p, int tiles) {
  constexpr int STRIDE = D + 4, CPR = D / 16;
  __shared__ uint32_t rows[kGatherTokens * STRIDE / 4];
  __shared__ float sc[kGatherTokens];
  __shared__ uint16_t pair[128];  // byte offsets of the two dims of an output word
  const int tid = threadIdx.x;
  const int unit = blockIdx.x / tiles, g = unit % p.Hkv;
  const int t0 = p.pos0 + (blockIdx.x % tiles) * kGatherTokens;
  const int n = min(kGatherTokens, p.pos0 + p.npos - t0);
  const uint4* src = reinterpret_cast<const uint4*>(p.k + ((size_t)unit * p.L + t0) * D);
#pragma unroll
  for (int i = 0; i < kGatherTokens * CPR / kThreads; ++i) {
    const int c = tid + i * kThreads, r = c / CPR;
    if (r < n) {
      const uint4 u = __ldg(src + c);
      uint32_t* d = rows + r * (STRIDE / 4) + (c % CPR) * 4;
      d[0] = u.x; d[1] = u.y; d[2] = u.z; d[3] = u.w;
    }
  }
  if (tid < n) sc[tid] = __ldg(p.ks + (size_t)unit * p.nblk + (t0 + tid) / p.T);
  for (int w = tid; w < p.nfc; w += kThreads) {  // word w: columns 2 w and 2 w + 1 (nfc is even: one half)
    const int hi = 2 * w >= p.nfc, c = 2 * w - (hi ? p.nfc : 0);
    const uint8_t* f = p.fc + g * p.nfc + c;
    pair[w] = (uint16_t)((f[0] + (hi ? D / 2 : 0)) | ((f[1] + (hi ? D / 2 : 0)) << 8));
  }
  __syncthreads();
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out) + ((size_t)unit * p.L + t0) * p.nfc;
  const int per = kThreads / p.nfc;  // tokens the CTA writes at a time; a thread keeps its column pair
  const int r0 = tid / p.nfc, w = tid % p.nfc;
  if (r0 >= per) return;
  const uint8_t* lo = reinterpret_cast<const uint8_t*>(rows) + (pair[w] & 255u);
  const uint8_t* hi = reinterpret_cast<const uint8_t*>(rows) + (pair[w] >> 8);
#pragma unroll 4
  for (int r = r0; r < n; r += per) {
    const float2 v = __half22float2(from_e4m3x2(lo[r * STRIDE] | ((uint32_t)hi[r * STRIDE] << 8)));
    const float f = sc[r];
    out[r * p.nfc + w] = pack_bf16x2(v.x * f, v.y * f);
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
    if (p.T == 128) append_kernel<128, 128><<<grid, kAppend, 0, st>>>(p, nb);
    else append_kernel<128, 64><<<grid, kAppend, 0, st>>>(p, nb);
  } else {
    if (p.T == 128) append_kernel<64, 128><<<grid, kAppend, 0, st>>>(p, nb);
    else append_kernel<64, 64><<<grid, kAppend, 0, st>>>(p, nb);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.in_place) return e;
  advance_kernel<<<(p.B + 127) / 128, 128, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_cache8_evict(const Cache8Evict& p, cudaStream_t st) {
  if ((long long)p.B * p.Hkv * 8 >= (1LL << 31)) return cudaErrorInvalidValue;
  // One CTA's shared memory holds 16384 keys; longer caches are spread over eight CTAs a head, of half the threads
  // (two share an SM, and every warp pays for the meetings: 131072 tokens 32 against 40 us).  The host knows the
  // capacity, not the lengths, so the rule is on the capacity.  Whole evictions to 8192 tokens of 4 x 8 heads, one CTA
  // a head against eight: 16384 tokens 36.1, 40.4 us; 32768 55.1, 43.6; 131072 126.7, 52.5.  It costs a long cache
  // that holds little: 2175 -> 2048 tokens of 16 x 8 heads 29.8 us in a cache of 2304 rows, 78.7 in one of 131072
  // (30.6 with one CTA a head).
  cudaError_t e = p.L > kSlice ? launch_select<8, 512>(p, st) : launch_select<1, 1024>(p, st);
  if (e != cudaSuccess) return e;
  const int most = p.keep < p.L ? p.keep : p.L;
  const int nb = (most + p.T - 1) / p.T;
  const long long gx = (long long)nb * p.B * p.Hkv;
  if (gx > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)gx, 2);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.L > kSlice ? 0 : 1;
  if (p.D == 128)
    return p.T == 128 ? cudaLaunchKernelEx(&cfg, evict_move_kernel<128, 128>, p, nb)
                      : cudaLaunchKernelEx(&cfg, evict_move_kernel<128, 64>, p, nb);
  return p.T == 128 ? cudaLaunchKernelEx(&cfg, evict_move_kernel<64, 128>, p, nb)
                    : cudaLaunchKernelEx(&cfg, evict_move_kernel<64, 64>, p, nb);
}

cudaError_t launch_cache8_gather(const Cache8Gather& p, cudaStream_t st) {
  if (p.npos == 0) return cudaSuccess;
  const int tiles = (p.npos + kGatherTokens - 1) / kGatherTokens;
  const unsigned grid = (unsigned)tiles * p.B * p.Hkv;
  if (p.D == 128) gather_kernel<128><<<grid, kThreads, 0, st>>>(p, tiles);
  else gather_kernel<64><<<grid, kThreads, 0, st>>>(p, tiles);
  return cudaGetLastError();
}

}  // namespace sfa
