// Attention over the 8-bit KV cache: joining the pieces of the whole-cache attention
// (cache8_attn_tc.cu), the accumulated weights, and index lists.
#include <cooperative_groups.h>
#include <math.h>

#include "cache8.cuh"
#include "tc_ptx8.cuh"

namespace sfa {

namespace {

using namespace c8;
namespace cg = cooperative_groups;

constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------------------
// Joining the pieces.  The first CTAs each join one query row of one unit (a
// thread per dim, the row's pieces shared among the thread groups) or, where there
// are rows enough to fill the SMs without that, all rows of a unit, a thread group
// a row; the others, with weights, each add the attention weights of some chunks of tokens
// of one unit: the rows' log-sum-exps again from the pieces' maxima and sums (a few
// numbers), then exp2 of the scores that the first step left, summed over the
// rows in order.  A unit of one piece has its outputs from the first step already.
// Launched while the first step still runs: everything up to pieces_ready() needs
// only the lengths.  At 16 x 8 units of 4 rows over 32768 tokens it adds 4 us to the
// 160 of the first step; with weights, 4 x 8 units over 131072 tokens, 21 us for
// 67 MB of scores, 17 of weights read and 17 written: 4.8 TB/s.  With 16 rows the
// scores are 128 bytes a token, written and read: 16 x 8 units over 16384 tokens cost
// 58 us more than without weights at d = 128 (151 against 93), 51 at d = 64 (122, 71).
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

__device__ __forceinline__ void pieces_ready() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Tokens per thread of the weights part: about four 16-byte loads of scores in flight (128K x 4 with weights: the
// whole call 201.5 us, 204.5 with eight, which spill; of the four, 4 to 8 bytes a thread spill where CTAs join by rows).
constexpr int weight_tokens(int CP) { return CP <= 4 ? 4 : (CP == 8 ? 2 : 1); }

template <int D, int CP, bool UNIT>  // CP = p.cpad; UNIT: a joining CTA takes all rows of a unit
__global__ void __launch_bounds__(kJoinThreads, 4) attn_join_kernel(const __grid_constant__ Cache8Attn p, int parts,
                                                                   int per_part) {
  constexpr int GR = kJoinThreads / D;  // thread groups
  constexpr int TPT = weight_tokens(CP);
  __shared__ int sh_total, sh_t0;
  __shared__ float so[GR][D], sl[GR];
  __shared__ __align__(16) float slse[kMaxCols];
  const int tid = threadIdx.x;
  const unsigned rows = (unsigned)(p.B * p.Hkv * (UNIT ? 1 : p.cols));  // joining CTAs
  const bool join = blockIdx.x < rows;
  const int unit = join ? blockIdx.x / (UNIT ? 1 : p.cols) : (blockIdx.x - rows) / parts;
  const int b = unit / p.Hkv, g = unit % p.Hkv;
  const int nv = visible(p.lens, b, p.L, p.back, nullptr);
  const int tiles = (nv + p.tile - 1) / p.tile;
  constexpr int CHUNK = TPT * kJoinThreads;
  const int part0 = join ? 0 : (int)((blockIdx.x - rows) % parts) * per_part;  // this CTA's tokens
  if (!join && part0 >= nv) return;
  if (tid < 32) {
    int total, extra;
    const int before = warp_count_cost(p.lens, p.B, p.Hkv, p.L, p.back, p.tile, p.G, b, &total, &extra);
    if (tid == 0) { sh_total = total; sh_t0 = before + g * (tiles + extra) + extra; }
  }
  __syncthreads();
  size_t s0 = 0;  // the unit's pieces have the slots [s0, s0 + np)
  int np = 0;
  if (tiles > 0) {
    const Split s(sh_total, p.G);
    const int i0 = s.owner(sh_t0);
    np = s.owner(sh_t0 + tiles - 1) - i0 + 1;
    s0 = (size_t)i0 + unit;
  }
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  pieces_ready();
  if (join && np == 1) return;  // one piece: the first step has written the outputs
  if (join && UNIT) {
    const int grp = tid / D, r = tid % D;
    for (int c = grp; c < p.cols; c += GR) {
      float M = -INFINITY, l = 0.f, o = 0.f;
      for (int i = 0; i < np; ++i) {
        const size_t at = (s0 + i) * p.cols + c;
        const float2 x = ml[at];
        const float v = p.part_o[at * D + r], mn = fmaxf(M, x.x), base = mn == -INFINITY ? 0.f : mn;
        const float keep = exp2f(M - base), f = exp2f(x.x - base);
        l = fmaf(x.y, f, l * keep);
        o = fmaf(v, f, o * keep);
        M = mn;
      }
      // l = 0 exactly when the row sees no token (a NaN score makes l NaN, and the row's o)
      const size_t row = (size_t)unit * p.cols + c;
      static_cast<__nv_bfloat16*>(p.o)[row * D + r] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
      if (r == 0 && p.lse != nullptr) p.lse[row] = l == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) + log2f(l)) * kLn2;
    }
    return;
  }
  if (join) {
    const int c = blockIdx.x % p.cols, grp = tid / D, r = tid % D;
    float M = -INFINITY;
    for (int i = 0; i < np; ++i) M = fmaxf(M, ml[(s0 + i) * p.cols + c].x);
    const float base = M == -INFINITY ? 0.f : M;
    float l = 0.f, o = 0.f;
#pragma unroll 4
    for (int i = grp; i < np; i += GR) {
      const size_t at = (s0 + i) * p.cols + c;
      const float2 x = ml[at];
      const float f = exp2f(x.x - base);
      l = fmaf(x.y, f, l);
      o = fmaf(p.part_o[at * D + r], f, o);
    }
    so[grp][r] = o;
    if (r == 0) sl[grp] = l;
    __syncthreads();
    if (tid >= D) return;
    l = sl[0];
    o = so[0][tid];
#pragma unroll
    for (int i = 1; i < GR; ++i) {
      l += sl[i];
      o += so[i][tid];
    }
    // l = 0 exactly when the row sees no token (a NaN score makes l NaN, and the row's o)
    static_cast<__nv_bfloat16*>(p.o)[(size_t)blockIdx.x * D + tid] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
    if (tid == 0 && p.lse != nullptr) p.lse[blockIdx.x] = l == 0.f ? -INFINITY : (base + log2f(l)) * kLn2;
    return;
  }
  // A chunk's scores and weights; the first chunk's go out before the log-sum-exps are worked out.
  float s[TPT][CP], w_in[TPT];
  const int part1 = min(part0 + per_part, nv);
  const float* sp = p.scores + ((size_t)unit * p.Lp + part0 + tid) * CP;
  const size_t w0 = (size_t)unit * p.L + part0 + tid;
  const float* wi = p.w_in != nullptr ? p.w_in + w0 : nullptr;
  float* wo = p.w_out + w0;
  auto load_chunk = [&](int n) {  // n: tokens of this thread's stride that are there
#pragma unroll
    for (int k = 0; k < TPT; ++k) {
      w_in[k] = 0.f;
      if (k * kJoinThreads < n) {
        const float* q = sp + k * kJoinThreads * CP;
        if constexpr (CP >= 4) {
#pragma unroll
          for (int c = 0; c < CP; c += 4) {
            const float4 u = __ldcs(reinterpret_cast<const float4*>(q + c));
            s[k][c] = u.x; s[k][c + 1] = u.y; s[k][c + 2] = u.z; s[k][c + 3] = u.w;
          }
        } else {
#pragma unroll
          for (int c = 0; c < CP; ++c) s[k][c] = q[c];
        }
        if (wi != nullptr) w_in[k] = wi[k * kJoinThreads];
      }
    }
  };
  int left = part1 - part0 - tid;
  load_chunk(left);
  for (int c = tid >> 5; c < CP; c += kJoinThreads / 32) {  // a warp per row
    const int lane = tid & 31;
    float M = -INFINITY, l = 0.f;
    if (c < p.cols) {
      for (int i = lane; i < np; i += 32) M = fmaxf(M, ml[(s0 + i) * p.cols + c].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    }
    const float base = M == -INFINITY ? 0.f : M;
    if (c < p.cols) {
      for (int i = lane; i < np; i += 32) {
        const float2 x = ml[(s0 + i) * p.cols + c];
        l = fmaf(x.y, exp2f(x.x - base), l);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    }
    // Rows that see nothing have scores of -inf only, and rows past cols (whose scores mean nothing) add none.
    if (lane == 0) slse[c] = c >= p.cols ? INFINITY : (l == 0.f ? 0.f : base + log2f(l));
  }
  __syncthreads();
  float sub[CP];
#pragma unroll
  for (int c = 0; c < CP; ++c) sub[c] = slse[c];
  for (;;) {
#pragma unroll
    for (int k = 0; k < TPT; ++k) {
      float w = 0.f;
#pragma unroll
      for (int c = 0; c < CP; ++c)
        if (CP < 4 || c < p.cols) w += tc::ex2_approx(s[k][c] - sub[c]);  // below 2^-126: 0
      if (k * kJoinThreads < left) wo[k * kJoinThreads] = w_in[k] + w;
    }
    left -= CHUNK;
    if (left + tid <= 0) break;
    sp += CHUNK * CP;
    if (wi != nullptr) wi += CHUNK;
    wo += CHUNK;
    load_chunk(left);
  }
}

template <int D, int CP, bool UNIT>
static cudaError_t launch_join(const Cache8Attn& p, cudaStream_t st) {
  // The weights part: CTAs of whole chunks, as many as are resident beside the joining ones (each pays its start once).
  const int chunk = weight_tokens(CP) * kJoinThreads, chunks = (p.L + chunk - 1) / chunk;
  const long long units = (long long)p.B * p.Hkv, joining = units * (UNIT ? 1 : p.cols);
  const long long room = 4 * kSms - joining > kSms ? 4 * kSms - joining : kSms;
  long long each = (units * chunks + room - 1) / room;
  each = each > chunks ? chunks : each;
  const int parts = (int)((chunks + each - 1) / each);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.B * p.Hkv * ((UNIT ? 1 : p.cols) + (p.w_out != nullptr ? parts : 0)));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_join_kernel<D, CP, UNIT>, p, parts, (int)each * chunk);
}

template <int D, int CP>
static cudaError_t launch_join_u(const Cache8Attn& p, cudaStream_t st) {
  // A CTA a row while they are resident at once, four to an SM; more rows: a CTA a unit (24 sequences x 8 heads of 8
  // rows with weights: the whole call 48.8 against 54.5 us; 16 x 8 of 4 rows: 166 against 164.6).
  return (long long)p.B * p.Hkv * p.cols > 4 * kSms ? launch_join<D, CP, true>(p, st) : launch_join<D, CP, false>(p, st);
}

template <int D>
static cudaError_t launch_join_d(const Cache8Attn& p, cudaStream_t st) {
  switch (p.cpad) {
    case 1: return launch_join_u<D, 1>(p, st);
    case 2: return launch_join_u<D, 2>(p, st);
    case 4: return launch_join_u<D, 4>(p, st);
    case 8: return launch_join_u<D, 8>(p, st);
    case 12: return launch_join_u<D, 12>(p, st);
    default: return launch_join_u<D, 16>(p, st);
  }
}

// ---------------------------------------------------------------------------
// Index lists: a CTA, or two that join their halves, per (b, q head).  A row of d codes is read by d / 16 lanes,
// 16 bytes each; each such lane group runs its own online softmax over its
// tokens, BATCH of them with both loads in flight, and the groups are
// joined at the end.  The list is checked and staged in shared memory first
// (kListPart entries at a time), so that a row's address waits for no second load.
// 512 rows of 1023 of up to 16383 tokens, d 128: 31.7 us for 139 MB of rows, 4.4 TB/s:
// bound by rows of 128 bytes at random addresses, the chain from a row to its
// probability, and the instructions that widen the codes (issue 63%).  Rows through a
// ring of asynchronous copies: 37.4 us; o rescaled only where the maximum grows: 32.6.
// ---------------------------------------------------------------------------
constexpr int kListPart = 2048;

template <int D, int WARPS, int BATCH, int CTAS, int CL>
__global__ void __launch_bounds__(WARPS * 32, CTAS) attn_list_kernel(const __grid_constant__ Cache8Attn p) {
  constexpr int LPT = D / 16, GROUPS = WARPS * 32 / LPT;
  __shared__ int list[kListPart];
  __shared__ float gm[GROUPS], gl[GROUPS];
  __shared__ __align__(16) float go[GROUPS][D + 4];
  __shared__ int bad;
  __shared__ float other[D + 2];  // CL = 2: the second CTA's o, maximum and sum
  __shared__ int other_bad;
  cg::cluster_group cluster = cg::this_cluster();
  if (CL > 1) cluster.barrier_arrive();  // waited for before the first access to the other CTA
  const int rank = CL > 1 ? (int)cluster.block_rank() : 0;
  const int row = blockIdx.x / CL, b = row / p.Hq, h = row % p.Hq, g = h / (p.Hq / p.Hkv);
  const int unit = b * p.Hkv + g;
  const int tid = threadIdx.x, grp = tid / LPT, part = tid % LPT;
  const int* src = p.idx + (size_t)row * p.k_list;
  if (tid == 0) bad = 0;
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
  const int n = visible(p.lens, b, p.L, 0, tid == 0 ? p.status : nullptr);
  const uint8_t* kbase = p.k + (size_t)unit * p.L * D + part * 16;
  const uint8_t* vbase = p.v + (size_t)unit * p.L * D + part * 16;
  const float* ksp = p.ks + (size_t)unit * p.nblk;
  const float* vsp = p.vs + (size_t)unit * p.nblk;
  const int tshift = p.T == 128 ? 7 : 6;
  float m = -INFINITY, l = 0.f, acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  const int half = (p.k_list + CL - 1) / CL, end = min(rank * half + half, p.k_list);
  for (int from = rank * half; from < end; from += kListPart) {
    const int have = min(kListPart, end - from);
    __syncthreads();
    for (int i = tid; i < have; i += WARPS * 32) {
      int t = __ldg(src + from + i);
      if (t >= n || t < -1) {
        bad = 1;
        t = -1;
      }
      list[i] = t;
    }
    __syncthreads();
    // the warp's groups walk the list together (a group past the end has no token): the shuffles need all lanes
    for (int base = 0; base < have; base += GROUPS * BATCH) {
      int tok[BATCH];
      uint4 ku[BATCH], vu[BATCH];
      float ks[BATCH], vs[BATCH];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const int j = base + u * GROUPS + grp;
        tok[u] = j < have ? list[j] : -1;
        ku[u] = vu[u] = make_uint4(0, 0, 0, 0);
        ks[u] = vs[u] = 0.f;
        if (tok[u] >= 0) {
          const size_t at = (size_t)tok[u] * D;
          ku[u] = __ldg(reinterpret_cast<const uint4*>(kbase + at));
          vu[u] = __ldg(reinterpret_cast<const uint4*>(vbase + at));
          ks[u] = __ldg(ksp + (tok[u] >> tshift));
          vs[u] = __ldg(vsp + (tok[u] >> tshift));
        }
      }
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
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
        const float f = tc::ex2_approx(m - mb), e = tc::ex2_approx(s - mb);
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
  }
  if (part == 0) { gm[grp] = m; gl[grp] = l; }
#pragma unroll
  for (int e = 0; e < 16; e += 4)
    *reinterpret_cast<float4*>(&go[grp][part * 16 + e]) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
  __syncthreads();
  if (bad && tid == 0) report(p.status, SFA_ERR_INDEX);
  float M = -INFINITY, L = 0.f, o = 0.f;
  if (tid < D) {
#pragma unroll 8
    for (int i = 0; i < GROUPS; ++i) M = fmaxf(M, gm[i]);
    const float base = M == -INFINITY ? 0.f : M;
#pragma unroll 8
    for (int i = 0; i < GROUPS; ++i) {
      const float f = exp2f(gm[i] - base);
      L += gl[i] * f;
      o = fmaf(go[i][tid], f, o);
    }
  }
  bool broken = bad;
  if (CL > 1) {
    cluster.barrier_wait();
    if (rank == 1) {
      float* to = cluster.map_shared_rank(other, 0);
      if (tid < D) to[tid] = o;
      if (tid == 0) {
        to[D] = M;
        to[D + 1] = L;
        *cluster.map_shared_rank(&other_bad, 0) = bad;
      }
    }
    cluster.sync();
    if (rank == 1) return;
    broken |= other_bad != 0;
    const float m1 = other[D], mn = fmaxf(M, m1), base = mn == -INFINITY ? 0.f : mn;
    const float f0 = exp2f(M - base), f1 = exp2f(m1 - base);
    L = L * f0 + other[D + 1] * f1;
    if (tid < D) o = o * f0 + other[tid] * f1;
    M = mn;
  }
  if (tid < D) {
    const bool none = broken || L == 0.f;
    static_cast<__nv_bfloat16*>(p.o)[(size_t)row * D + tid] = __float2bfloat16_rn(none ? 0.f : o / L);
    if (tid == 0 && p.lse != nullptr) p.lse[row] = none ? -INFINITY : ((M == -INFINITY ? 0.f : M) + log2f(L)) * kLn2;
  }
}

template <int D>
cudaError_t launch_list(const Cache8Attn& p, cudaStream_t st) {
  const unsigned rows = (unsigned)(p.B * p.Hq);
  // Up to two rows an SM: four tokens in flight a lane group (128 x 256 tokens: 5.4 us, 6.1 with two); more rows:
  // two tokens and twice the warps an SM (512 x 1023 tokens: 33.5 us, 37.8 with four), in CTAs of half a row, whose
  // number an SM comes out evener (31.7 us).
  if (rows <= 2u * kSms) {
    attn_list_kernel<D, 8, 4, 2, 1><<<rows, 256, 0, st>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows * 2);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_list_kernel<D, 4, 2, 8, 2>, p);
}

}  // namespace

cudaError_t launch_cache8_attn(const Cache8Attn& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  cudaError_t e = launch_cache8_tiles(p, tk, tv, st);
  if (e != cudaSuccess) return e;
  return p.D == 128 ? launch_join_d<128>(p, st) : launch_join_d<64>(p, st);
}

cudaError_t launch_cache8_attn_list(const Cache8Attn& p, cudaStream_t st) {
  return p.D == 128 ? launch_list<128>(p, st) : launch_list<64>(p, st);
}

}  // namespace sfa
