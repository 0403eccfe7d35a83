// norms.cu -- the norms around a block (sm_100a): the gated group norm between
// a scan and out_proj, and the residual norm between two blocks.
//
// Both are bound by their streams (every input read once, every output
// written once): a team of threads holds one group of channels (one row, for
// the residual norm) in registers from its load to its store, VEC elements at
// a time, so the second and third use of a value costs no traffic. The sums
// are fp32, and each output is rounded once.
//
// The block-wide forms may have 1024 threads, so 64 registers each, and the
// longest rows do not fit them: gated groups above 16384 channels spill 0.4-2
// KB a thread (24576 channels, bf16: 3.1 TB/s, gate first 1.0; fp32 1.1), fp32
// ones above 8192 200 bytes (4.6 TB/s), residual rows above 16384 60-220 bytes
// (5.5-6.1 TB/s). Rows without vector loads are slower at every length (5001
// channels, bf16: 1.5 and 4.1 TB/s; 20001: 0.5 and 1.6). The blocks of this
// library have 2560 and 7680 channels.
//
// Teams. A gated group of up to 1024 channels is one team of 8, 16 or 32
// lanes, and a block of 256 threads holds several; larger groups, and the rows
// of the residual norm, are one block each (65536 x 2560 with a fp32 residual,
// 2.01 GB: 293 us, 6.9 TB/s). VEC is 8 (16-byte loads at bf16,
// two at fp32) where pointers, strides and channel counts allow it, else 1.
#include <cuda_bf16.h>

#include "ssm.h"
#include "ssm_internal.h"
#include "ssm_math.cuh"

namespace ssm {
namespace {

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = IO<T>::load(p);
  } else if constexpr (sizeof(T) == 2) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(u[i] << 16), f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    *p = IO<T>::from_f(f[0]);
  } else if constexpr (sizeof(T) == 2) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// Sum over a team: `width` lanes of a warp (a power of two), or the whole block.
__device__ __forceinline__ float lanes_sum(float x, int width) {
  for (int m = width >> 1; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}
__device__ __forceinline__ float block_sum(float x, float* part) {
  x = lanes_sum(x, 32);
  if (blockDim.x == 32) return x;
  __syncthreads();  // the last sum's readers are done with `part`
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
  return lanes_sum(lane < nw ? part[lane] : 0.0f, 32);
}

// n / d for 0 <= n < 2^31 without a division, by a multiplication with d's rounded-up reciprocal, made once on the
// host (Granlund and Montgomery, Division by Invariant Integers using Multiplication, 1994).
struct Divider {
  uint32_t d, mul, shift;
  explicit Divider(uint32_t div = 1) : d(div), mul(0), shift(0) {
    while ((uint64_t{1} << shift) < d) ++shift;
    mul = static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{1} << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n, uint32_t& rest) const {
    const uint32_t q = (__umulhi(n, mul) + n) >> shift;
    rest = n - q * d;
    return q;
  }
};

struct GatedArgs {
  const void *x, *z;
  const float* w;
  void* y;
  Divider seqlen, groups;
  uint32_t rows;
  uint32_t active, row_step;  // teams at work, a multiple of the groups; rows from one of a team's units to its next
  int group;
  float eps;
  int64_t x_tok, x_seq, z_tok, z_seq, y_tok, y_seq;
  int flat;  // rows at one stride: no sequence strides
  int shared_weight;
  int team, team_shift;  // lanes of a team and their log2; team 0 = the block
};

// VEC elements as they lie in memory.
template <typename T, int VEC>
struct Raw {
  static constexpr int kWords = sizeof(T) * VEC >= 4 ? sizeof(T) * VEC / 4 : 1;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 1) {
      if constexpr (sizeof(T) == 2) w[0] = *reinterpret_cast<const uint16_t*>(p);
      else w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
  }
};

// A team keeps its group and walks the rows `row_step` apart, so that its
// weights stay in registers and a row costs no division, and the next row's
// loads are in flight while one is summed and stored. x and z are kept as they
// lie in memory; with the gate first x SiLU(z) is formed twice, for the sum and
// for the output. Bound by instructions next to the streams (two SFU
// operations an element): 16384 x 7680 in groups of 128, bf16 (755 MB), takes
// 122 us, and 143 us with a
// block per 16 groups of a row and divisions.
template <typename T, int VEC, int NV, bool FIRST, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 256) gated_norm_kernel(const GatedArgs a) {
  __shared__ float part[32];
  constexpr bool kKeepW = NV <= 2;
  const int team = BLOCK ? static_cast<int>(blockDim.x) : a.team;
  const int i0 = BLOCK ? threadIdx.x : threadIdx.x & (team - 1);
  // the block's first team: counted in teams, since a row may have more threads than 32 bits count
  const uint32_t team0 = BLOCK ? blockIdx.x : blockIdx.x * (blockDim.x >> a.team_shift);
  const uint32_t tid = BLOCK ? team0 : team0 + (threadIdx.x >> a.team_shift);
  uint32_t grp, first_grp;
  uint32_t row = a.groups(tid, grp);
  const bool has = tid < a.active;
  // the block's threads make the same number of rounds: its first team's, whose rows come first
  uint32_t round = BLOCK ? row : a.groups(team0, first_grp);
  const float inv_n = 1.0f / static_cast<float>(a.group);
  const int64_t c0 = static_cast<int64_t>(grp) * a.group + i0 * VEC;
  const T* x = static_cast<const T*>(a.x) + c0;
  const T* z = static_cast<const T*>(a.z) + c0;
  T* y = static_cast<T*>(a.y) + c0;
  const float* w = a.w + (a.shared_weight ? i0 * VEC : c0);
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = has && (i0 + i * team) * VEC < a.group;
  float wk[kKeepW ? NV : 1][VEC];
  if constexpr (kKeepW) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) load_vec<float, VEC>(w + i * team * VEC, wk[i]);
  }
  Raw<T, VEC> xr[NV], zr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < Raw<T, VEC>::kWords; ++j) xr[i].w[j] = 0u, zr[i].w[j] = 0u;
  int64_t yo = 0;
  auto fetch = [&]() {
    if (row >= a.rows) return;
    uint32_t t = row, s = 0;
    if (!a.flat) s = a.seqlen(row, t);
    const T* xp = x + s * a.x_seq + t * a.x_tok;
    const T* zp = z + s * a.z_seq + t * a.z_tok;
    yo = s * a.y_seq + t * a.y_tok;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) {
        xr[i].load(xp + i * team * VEC);
        if (a.z) zr[i].load(zp + i * team * VEC);
      }
  };
  fetch();
  for (; round < a.rows; round += a.row_step) {
    const bool live = row < a.rows;
    T* yp = y + yo;
    Raw<T, VEC> xc[NV], zc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) xc[i] = xr[i], zc[i] = zr[i];
    row += a.row_step;
    fetch();
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[VEC];
      xc[i].get(f);
      if constexpr (FIRST) {
        float g[VEC];
        zc[i].get(g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] *= silu(g[j]);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum = fmaf(f[j], f[j], sum);
    }
    sum = BLOCK ? block_sum(sum, part) : lanes_sum(sum, team);
    const float r = rsqrtf(fmaf(sum, inv_n, a.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!live || !in[i]) continue;
      float f[VEC], g[VEC], wv[VEC];
      xc[i].get(f);
      if constexpr (kKeepW) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) wv[j] = wk[i][j];
      } else {
        load_vec<float, VEC>(w + i * team * VEC, wv);
      }
      if (a.z) {
        zc[i].get(g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] *= silu(g[j]);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] *= r * wv[j];
      store_vec<T, VEC>(yp + i * team * VEC, f);
    }
  }
}

struct ResidualArgs {
  const void *x, *rin;
  const float *w, *post;
  void *y, *rout;
  int64_t x_st, rin_st, y_st, rout_st;
  int64_t rows;
  int dim;
  float eps, alpha;
  int team, team_shift;  // lanes of a team and their log2 where a block holds several rows
};

template <typename T, typename R, int VEC, int NV, bool POST, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 256) residual_norm_kernel(const ResidualArgs a) {
  __shared__ float part[32];
  const int team = BLOCK ? static_cast<int>(blockDim.x) : a.team;
  const int i0 = BLOCK ? threadIdx.x : threadIdx.x & (team - 1);
  const int64_t row = BLOCK ? blockIdx.x : (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> a.team_shift;
  const bool live = BLOCK || row < a.rows;
  const T* x = static_cast<const T*>(a.x) + row * a.x_st;
  const R* rin = a.rin ? static_cast<const R*>(a.rin) + row * a.rin_st : nullptr;
  auto sum_of = [&](float s) { return BLOCK ? block_sum(s, part) : lanes_sum(s, team); };
  float v[NV][VEC], res[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i0 + i * team) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[i][j] = 0.0f, res[i][j] = 0.0f;
    if (live && e < a.dim) {
      load_vec<T, VEC>(x + e, v[i]);
      if (rin) load_vec<R, VEC>(rin + e, res[i]);
    }
  }
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  if constexpr (POST) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum = fmaf(v[i][j], v[i][j], sum);
    const float r = rsqrtf(fmaf(sum_of(sum), inv_dim, a.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i0 + i * team) * VEC;
      if (e >= a.dim) continue;
      float wv[VEC];
      load_vec<float, VEC>(a.post + e, wv);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] *= r * wv[j];
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      res[i][j] = fmaf(a.alpha, v[i][j], res[i][j]);
      sum = fmaf(res[i][j], res[i][j], sum);
    }
  if (a.rout) {
    R* rout = static_cast<R*>(a.rout) + row * a.rout_st;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i0 + i * team) * VEC;
      if (live && e < a.dim) store_vec<R, VEC>(rout + e, res[i]);
    }
  }
  const float r = rsqrtf(fmaf(sum_of(sum), inv_dim, a.eps));
  T* y = static_cast<T*>(a.y) + row * a.y_st;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i0 + i * team) * VEC;
    if (!live || e >= a.dim) continue;
    float wv[VEC];
    load_vec<float, VEC>(a.w + e, wv);
#pragma unroll
    for (int j = 0; j < VEC; ++j) wv[j] *= res[i][j] * r;
    store_vec<T, VEC>(y + e, wv);
  }
}

// Threads and values per thread that cover n channels of a block's team:
// vectors of 8 from one per thread up to four, single elements from eight up.
constexpr int kMaxGroup = 32768;

// Blocks of a kernel that one SM holds, asked once, times the SMs.
template <typename K>
unsigned resident_blocks(K kernel, int threads) {
  int dev = 0, sms = 148, per_sm = 1;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0) != cudaSuccess || per_sm < 1) per_sm = 1;
  return static_cast<unsigned>(sms * per_sm);
}

template <typename T, int VEC, int NV, bool FIRST, bool BLOCK>
cudaError_t launch_gated_as(GatedArgs a, int threads, cudaStream_t st) {
  const uint32_t per_block = BLOCK ? 1 : threads >> a.team_shift, groups = a.groups.d, units = a.rows * groups;
  uint32_t grid = (units + per_block - 1) / per_block;
  auto kernel = gated_norm_kernel<T, VEC, NV, FIRST, BLOCK>;
  if (grid > 512) {  // the occupancy query costs 1 us: not for the small calls
    uint32_t most = resident_blocks(kernel, threads);
    if (most * per_block < groups) most = (groups + per_block - 1) / per_block;  // a team for each group at least
    if (grid > most) grid = most;
  }
  const uint32_t teams = grid * per_block;
  a.row_step = teams / groups, a.active = a.row_step * groups;
  kernel<<<grid, threads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, bool FIRST>
cudaError_t launch_gated(GatedArgs a, bool vec, cudaStream_t st) {
  const int n = vec ? a.group / 8 : a.group;  // vectors or elements of a group
  if (a.group <= 1024) {
    a.team = 32;
    while (vec && a.team > 8 && n <= a.team / 2) a.team >>= 1;
    a.team_shift = a.team == 32 ? 5 : a.team == 16 ? 4 : 3;
    const int nv = (n + a.team - 1) / a.team;
    if (vec)
      return nv <= 1   ? launch_gated_as<T, 8, 1, FIRST, false>(a, 256, st)
             : nv <= 2 ? launch_gated_as<T, 8, 2, FIRST, false>(a, 256, st)
                       : launch_gated_as<T, 8, 4, FIRST, false>(a, 256, st);
    return nv <= 4    ? launch_gated_as<T, 1, 4, FIRST, false>(a, 256, st)
           : nv <= 12 ? launch_gated_as<T, 1, 12, FIRST, false>(a, 256, st)
                      : launch_gated_as<T, 1, 32, FIRST, false>(a, 256, st);
  }
  a.team = 0;
  auto threads = [n](int nv) { return ((n + nv - 1) / nv + 31) / 32 * 32; };
  // Two vectors a thread at bf16 (39062 rows of 5120: 209 us, one: 273 us), one at fp32 (404 us, two: 456 us).
  if (vec)
    return n <= 1024 && sizeof(T) == 4 ? launch_gated_as<T, 8, 1, FIRST, true>(a, threads(1), st)
           : n <= 2048                 ? launch_gated_as<T, 8, 2, FIRST, true>(a, threads(2), st)
                                       : launch_gated_as<T, 8, 4, FIRST, true>(a, threads(4), st);
  return n <= 4096   ? launch_gated_as<T, 1, 4, FIRST, true>(a, threads(4), st)
         : n <= 8192 ? launch_gated_as<T, 1, 8, FIRST, true>(a, threads(8), st)
                     : launch_gated_as<T, 1, 32, FIRST, true>(a, threads(32), st);
}

template <typename T, typename R, bool POST>
cudaError_t launch_residual(ResidualArgs a, bool vec, cudaStream_t st) {
  const int n = vec ? a.dim / 8 : a.dim;
  if (vec && n <= 32) {  // short rows: a block of 256 threads holds several
    a.team = n <= 8 ? 8 : n <= 16 ? 16 : 32, a.team_shift = n <= 8 ? 3 : n <= 16 ? 4 : 5;
    const int64_t per_block = 256 >> a.team_shift;
    residual_norm_kernel<T, R, 8, 1, POST, false>
        <<<static_cast<unsigned>((a.rows + per_block - 1) / per_block), 256, 0, st>>>(a);
    return cudaGetLastError();
  }
  const unsigned grid = static_cast<unsigned>(a.rows);
  auto threads = [n](int nv) { return ((n + nv - 1) / nv + 31) / 32 * 32; };
  if (vec) {
    if (n <= 1024) residual_norm_kernel<T, R, 8, 1, POST, true><<<grid, threads(1), 0, st>>>(a);
    else if (n <= 2048) residual_norm_kernel<T, R, 8, 2, POST, true><<<grid, threads(2), 0, st>>>(a);
    else residual_norm_kernel<T, R, 8, 4, POST, true><<<grid, threads(4), 0, st>>>(a);
  } else {
    if (n <= 4096) residual_norm_kernel<T, R, 1, 4, POST, true><<<grid, threads(4), 0, st>>>(a);
    else if (n <= 8192) residual_norm_kernel<T, R, 1, 8, POST, true><<<grid, threads(8), 0, st>>>(a);
    else residual_norm_kernel<T, R, 1, 32, POST, true><<<grid, threads(32), 0, st>>>(a);
  }
  return cudaGetLastError();
}

template <typename T, typename R>
cudaError_t launch_residual_post(const ResidualArgs& a, bool vec, cudaStream_t st) {
  return a.post ? launch_residual<T, R, true>(a, vec, st) : launch_residual<T, R, false>(a, vec, st);
}

size_t dtype_bytes(int32_t t) { return t == SSM_BF16 ? 2 : 4; }
bool known_dtype(int32_t t) { return t == SSM_F32 || t == SSM_BF16; }

}  // namespace
}  // namespace ssm

extern "C" {

ssm_status ssm_gated_norm(const ssm_gated_norm_dims* d, const void* x, const void* z, const float* w, void* y,
                          void* stream) {
  using ssm::aligned;
  using ssm::fail;
  if (!d) return fail(SSM_ERR_INVALID_ARG, "dims is NULL");
  if (d->batch < 0 || d->seqlen < 0 || d->dim <= 0 || d->group <= 0 || d->dim % d->group != 0)
    return fail(SSM_ERR_INVALID_ARG, "need batch, seqlen >= 0 and dim=%lld a positive multiple of group=%lld",
                (long long)d->dim, (long long)d->group);
  if (d->group > ssm::kMaxGroup) return fail(SSM_ERR_UNSUPPORTED, "group=%lld: at most 32768", (long long)d->group);
  if (!ssm::known_dtype(d->io_dtype)) return fail(SSM_ERR_INVALID_ARG, "io_dtype=%d unknown", d->io_dtype);
  if (!(d->eps >= 0.0f)) return fail(SSM_ERR_INVALID_ARG, "eps=%g must be >= 0", d->eps);
  if ((d->gate_first & ~1) || (d->shared_weight & ~1))
    return fail(SSM_ERR_INVALID_ARG, "gate_first and shared_weight must be 0 or 1");
  const int64_t groups = d->dim / d->group;
  if (d->batch > 0 && d->seqlen > 0 && d->batch > 0x7fffffff / d->seqlen / groups)
    return fail(SSM_ERR_INVALID_ARG, "batch * seqlen * groups must be below 2^31");
  ssm::GatedArgs a{};
  a.x_tok = d->x_tok_stride ? d->x_tok_stride : d->dim, a.x_seq = d->x_seq_stride ? d->x_seq_stride : d->seqlen * a.x_tok;
  a.z_tok = d->z_tok_stride ? d->z_tok_stride : d->dim, a.z_seq = d->z_seq_stride ? d->z_seq_stride : d->seqlen * a.z_tok;
  a.y_tok = d->y_tok_stride ? d->y_tok_stride : d->dim, a.y_seq = d->y_seq_stride ? d->y_seq_stride : d->seqlen * a.y_tok;
  if (a.x_tok < d->dim || a.z_tok < d->dim || a.y_tok < d->dim || a.x_seq < 0 || a.z_seq < 0 || a.y_seq < 0)
    return fail(SSM_ERR_INVALID_ARG, "token strides must be >= dim and sequence strides >= 0");
  if (d->batch == 0 || d->seqlen == 0) return fail(SSM_OK, "");
  const size_t e = ssm::dtype_bytes(d->io_dtype);
  if (!x || !w || !y) return fail(SSM_ERR_INVALID_ARG, "x, w or y is NULL");
  if (!aligned(x, e) || (z && !aligned(z, e)) || !aligned(y, e) || !aligned(w, 4))
    return fail(SSM_ERR_INVALID_ARG, "x, z, w or y is not aligned to its element");
  // y may lie over x or z where each element is over its own; a stride of one token or sequence says nothing
  auto apart = [&](const void* in, int64_t tok, int64_t seq) {
    return in == y && ((d->seqlen > 1 && tok != a.y_tok) || (d->batch > 1 && seq != a.y_seq));
  };
  if (apart(x, a.x_tok, a.x_seq) || apart(z, a.z_tok, a.z_seq))
    return fail(SSM_ERR_INVALID_ARG, "y over x or z must have its strides");
  a.x = x, a.z = z, a.w = w, a.y = y;
  a.seqlen = ssm::Divider(static_cast<uint32_t>(d->seqlen)), a.groups = ssm::Divider(static_cast<uint32_t>(groups));
  a.rows = static_cast<uint32_t>(d->batch * d->seqlen), a.group = static_cast<int>(d->group);
  a.flat = d->batch == 1 || (a.x_seq == d->seqlen * a.x_tok && (!z || a.z_seq == d->seqlen * a.z_tok) &&
                             a.y_seq == d->seqlen * a.y_tok);
  a.eps = d->eps, a.shared_weight = d->shared_weight;
  const int64_t st8 = a.x_tok | a.x_seq | a.y_tok | a.y_seq | (z ? a.z_tok | a.z_seq : 0) | d->group;
  const bool vec = st8 % 8 == 0 && aligned(x, 16) && (!z || aligned(z, 16)) && aligned(y, 16) && aligned(w, 16);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool first = d->gate_first && z;
  cudaError_t err;
  if (d->io_dtype == SSM_BF16)
    err = first ? ssm::launch_gated<__nv_bfloat16, true>(a, vec, st) : ssm::launch_gated<__nv_bfloat16, false>(a, vec, st);
  else
    err = first ? ssm::launch_gated<float, true>(a, vec, st) : ssm::launch_gated<float, false>(a, vec, st);
  if (err != cudaSuccess) return fail(SSM_ERR_CUDA, "gated-norm launch: %s", cudaGetErrorString(err));
  return fail(SSM_OK, "");
}

ssm_status ssm_residual_norm(const ssm_residual_norm_dims* d, const void* x, const void* residual_in, const float* w,
                             const float* post_w, void* y, void* residual_out, void* stream) {
  using ssm::aligned;
  using ssm::fail;
  if (!d) return fail(SSM_ERR_INVALID_ARG, "dims is NULL");
  if (d->rows < 0 || d->rows > 0x7fffffff || d->dim <= 0)
    return fail(SSM_ERR_INVALID_ARG, "need 0 <= rows=%lld < 2^31 and dim=%lld > 0", (long long)d->rows,
                (long long)d->dim);
  if (d->dim > ssm::kMaxGroup) return fail(SSM_ERR_UNSUPPORTED, "dim=%lld: at most 32768", (long long)d->dim);
  if (!ssm::known_dtype(d->io_dtype) || !ssm::known_dtype(d->residual_dtype))
    return fail(SSM_ERR_INVALID_ARG, "io_dtype=%d or residual_dtype=%d unknown", d->io_dtype, d->residual_dtype);
  if (!(d->eps >= 0.0f)) return fail(SSM_ERR_INVALID_ARG, "eps=%g must be >= 0", d->eps);
  ssm::ResidualArgs a{};
  a.x_st = d->x_stride ? d->x_stride : d->dim, a.y_st = d->y_stride ? d->y_stride : d->dim;
  a.rin_st = d->residual_in_stride ? d->residual_in_stride : d->dim;
  a.rout_st = d->residual_out_stride ? d->residual_out_stride : d->dim;
  if (a.x_st < d->dim || a.y_st < d->dim || a.rin_st < d->dim || a.rout_st < d->dim)
    return fail(SSM_ERR_INVALID_ARG, "row strides must be >= dim");
  if (d->rows == 0) return fail(SSM_OK, "");
  const size_t e = ssm::dtype_bytes(d->io_dtype), er = ssm::dtype_bytes(d->residual_dtype);
  if (!x || !w || !y) return fail(SSM_ERR_INVALID_ARG, "x, w or y is NULL");
  if (y == residual_out) return fail(SSM_ERR_INVALID_ARG, "y and residual_out are the same buffer");
  // a result may lie over an input where each element is over its own
  auto apart = [&](const void* out, size_t eo, int64_t so, const void* in, size_t ei, int64_t si) {
    return out && out == in && (eo != ei || (d->rows > 1 && so != si));
  };
  if (apart(y, e, a.y_st, x, e, a.x_st) || apart(y, e, a.y_st, residual_in, er, a.rin_st) ||
      apart(residual_out, er, a.rout_st, x, e, a.x_st) || apart(residual_out, er, a.rout_st, residual_in, er, a.rin_st))
    return fail(SSM_ERR_INVALID_ARG, "a result over an input must have its type and stride");
  if (!aligned(x, e) || !aligned(y, e) || !aligned(w, 4) || (post_w && !aligned(post_w, 4)) ||
      (residual_in && !aligned(residual_in, er)) || (residual_out && !aligned(residual_out, er)))
    return fail(SSM_ERR_INVALID_ARG, "a pointer is not aligned to its element");
  a.x = x, a.rin = residual_in, a.w = w, a.post = post_w, a.y = y, a.rout = residual_out;
  a.rows = d->rows, a.dim = static_cast<int>(d->dim), a.eps = d->eps, a.alpha = d->residual_scale;
  const int64_t st8 = a.x_st | a.y_st | (residual_in ? a.rin_st : 0) | (residual_out ? a.rout_st : 0) | d->dim;
  const bool vec = st8 % 8 == 0 && aligned(x, 16) && aligned(y, 16) && aligned(w, 16) && (!post_w || aligned(post_w, 16)) &&
                   (!residual_in || aligned(residual_in, 16)) && (!residual_out || aligned(residual_out, 16));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (d->io_dtype == SSM_BF16)
    err = d->residual_dtype == SSM_BF16 ? ssm::launch_residual_post<__nv_bfloat16, __nv_bfloat16>(a, vec, st)
                                        : ssm::launch_residual_post<__nv_bfloat16, float>(a, vec, st);
  else
    err = d->residual_dtype == SSM_BF16 ? ssm::launch_residual_post<float, __nv_bfloat16>(a, vec, st)
                                        : ssm::launch_residual_post<float, float>(a, vec, st);
  if (err != cudaSuccess) return fail(SSM_ERR_CUDA, "residual-norm launch: %s", cudaGetErrorString(err));
  return fail(SSM_OK, "");
}

}  // extern "C"
