// norms.cu -- the norms around a block (sm_100a): the gated group norm between
// a scan and out_proj, and the residual norm between two blocks.
//
// Both are bound by their streams (every input read once, every output
// written once): a team of threads holds one group of channels (one row, for
// the residual norm) in registers from its load to its store, VEC elements at
// a time, so the second and third use of a value costs no traffic. The sums
// are fp32, and each output is rounded once.
//
// Teams. A gated group of up to 1024 channels is one team of 8, 16 or 32
// lanes, and a block of 256 threads holds several; larger groups, and the rows
// of the residual norm, are one block each. VEC is 8 (16-byte loads at bf16,
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

struct GatedArgs {
  const void *x, *z;
  const float* w;
  void* y;
  int64_t seqlen, groups, units;  // units = rows * groups
  int group;
  float eps;
  int64_t x_tok, x_seq, z_tok, z_seq, y_tok, y_seq;
  int shared_weight;
  int team;  // lanes of a team; 0 = the block
};

template <typename T, int VEC, int NV, bool FIRST>
__global__ void __launch_bounds__(1024) gated_norm_kernel(const GatedArgs a) {
  __shared__ float part[32];
  const int team = a.team ? a.team : static_cast<int>(blockDim.x);
  const int i0 = a.team ? (threadIdx.x & (team - 1)) : threadIdx.x;
  const int64_t unit = a.team ? blockIdx.x * static_cast<int64_t>(blockDim.x / team) + threadIdx.x / team : blockIdx.x;
  const bool live = unit < a.units;
  const int64_t row = live ? unit / a.groups : 0, grp = live ? unit % a.groups : 0;
  const int64_t s = row / a.seqlen, t = row % a.seqlen, c0 = grp * a.group;
  const T* x = static_cast<const T*>(a.x) + s * a.x_seq + t * a.x_tok + c0;
  const T* z = a.z ? static_cast<const T*>(a.z) + s * a.z_seq + t * a.z_tok + c0 : nullptr;
  const float* w = a.w + (a.shared_weight ? 0 : c0);
  float v[NV][VEC], gate[NV][VEC];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i0 + i * team) * VEC;
    const bool in = live && e < a.group;
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[i][j] = 0.0f, gate[i][j] = 1.0f;
    if (in) {
      load_vec<T, VEC>(x + e, v[i]);
      if (z) load_vec<T, VEC>(z + e, gate[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if (z) gate[i][j] = silu(gate[i][j]);
      if (FIRST) v[i][j] *= gate[i][j];
      sum = fmaf(v[i][j], v[i][j], sum);
    }
  sum = a.team ? lanes_sum(sum, team) : block_sum(sum, part);
  const float r = rsqrtf(sum / static_cast<float>(a.group) + a.eps);
  T* y = static_cast<T*>(a.y) + s * a.y_seq + t * a.y_tok + c0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i0 + i * team) * VEC;
    if (!(live && e < a.group)) continue;
    float wv[VEC];
    load_vec<float, VEC>(w + e, wv);
#pragma unroll
    for (int j = 0; j < VEC; ++j) wv[j] = FIRST ? v[i][j] * r * wv[j] : v[i][j] * r * wv[j] * gate[i][j];
    store_vec<T, VEC>(y + e, wv);
  }
}

struct ResidualArgs {
  const void *x, *rin;
  const float *w, *post;
  void *y, *rout;
  int64_t x_st, rin_st, y_st, rout_st;
  int dim;
  float eps, alpha;
};

template <typename T, typename R, int VEC, int NV, bool POST>
__global__ void __launch_bounds__(1024) residual_norm_kernel(const ResidualArgs a) {
  __shared__ float part[32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.x_st;
  const R* rin = a.rin ? static_cast<const R*>(a.rin) + row * a.rin_st : nullptr;
  float v[NV][VEC], res[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (threadIdx.x + i * blockDim.x) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[i][j] = 0.0f, res[i][j] = 0.0f;
    if (e < a.dim) {
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
    const float r = rsqrtf(block_sum(sum, part) * inv_dim + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (threadIdx.x + i * blockDim.x) * VEC;
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
  R* rout = a.rout ? static_cast<R*>(a.rout) + row * a.rout_st : nullptr;
  if (rout) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (threadIdx.x + i * blockDim.x) * VEC;
      if (e < a.dim) store_vec<R, VEC>(rout + e, res[i]);
    }
  }
  const float r = rsqrtf(block_sum(sum, part) * inv_dim + a.eps);
  T* y = static_cast<T*>(a.y) + row * a.y_st;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (threadIdx.x + i * blockDim.x) * VEC;
    if (e >= a.dim) continue;
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

template <typename T, bool FIRST>
cudaError_t launch_gated(GatedArgs a, bool vec, cudaStream_t st) {
  const int n = vec ? a.group / 8 : a.group;  // vectors or elements of a group
  if (a.group <= 1024) {
    // up to 8 vectors of 8 ... one team of lanes; several teams a block of 256 threads
    a.team = 32;
    while (vec && a.team > 8 && n <= a.team / 2) a.team >>= 1;
    const int64_t per_block = 256 / a.team;
    const unsigned grid = static_cast<unsigned>((a.units + per_block - 1) / per_block);
    const int nv = (n + a.team - 1) / a.team;
    if (vec) {
      if (nv <= 1) gated_norm_kernel<T, 8, 1, FIRST><<<grid, 256, 0, st>>>(a);
      else if (nv <= 2) gated_norm_kernel<T, 8, 2, FIRST><<<grid, 256, 0, st>>>(a);
      else gated_norm_kernel<T, 8, 4, FIRST><<<grid, 256, 0, st>>>(a);
    } else {
      if (nv <= 4) gated_norm_kernel<T, 1, 4, FIRST><<<grid, 256, 0, st>>>(a);
      else gated_norm_kernel<T, 1, 32, FIRST><<<grid, 256, 0, st>>>(a);
    }
    return cudaGetLastError();
  }
  a.team = 0;
  const unsigned grid = static_cast<unsigned>(a.units);
  auto threads = [n](int nv) { return ((n + nv - 1) / nv + 31) / 32 * 32; };
  if (vec) {
    if (n <= 1024) gated_norm_kernel<T, 8, 1, FIRST><<<grid, threads(1), 0, st>>>(a);
    else gated_norm_kernel<T, 8, 4, FIRST><<<grid, threads(4), 0, st>>>(a);
  } else {
    if (n <= 4096) gated_norm_kernel<T, 1, 4, FIRST><<<grid, threads(4), 0, st>>>(a);
    else gated_norm_kernel<T, 1, 32, FIRST><<<grid, threads(32), 0, st>>>(a);
  }
  return cudaGetLastError();
}

template <typename T, typename R, bool POST>
cudaError_t launch_residual(const ResidualArgs& a, int64_t rows, bool vec, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(rows);
  const int n = vec ? a.dim / 8 : a.dim;
  auto threads = [n](int nv) { return ((n + nv - 1) / nv + 31) / 32 * 32; };
  if (vec) {
    if (n <= 1024) residual_norm_kernel<T, R, 8, 1, POST><<<grid, threads(1), 0, st>>>(a);
    else residual_norm_kernel<T, R, 8, 4, POST><<<grid, threads(4), 0, st>>>(a);
  } else {
    if (n <= 4096) residual_norm_kernel<T, R, 1, 4, POST><<<grid, threads(4), 0, st>>>(a);
    else residual_norm_kernel<T, R, 1, 32, POST><<<grid, threads(32), 0, st>>>(a);
  }
  return cudaGetLastError();
}

template <typename T, typename R>
cudaError_t launch_residual_post(const ResidualArgs& a, int64_t rows, bool vec, cudaStream_t st) {
  return a.post ? launch_residual<T, R, true>(a, rows, vec, st) : launch_residual<T, R, false>(a, rows, vec, st);
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
  a.x = x, a.z = z, a.w = w, a.y = y;
  a.seqlen = d->seqlen, a.groups = groups, a.units = d->batch * d->seqlen * groups, a.group = static_cast<int>(d->group);
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
  if (!aligned(x, e) || !aligned(y, e) || !aligned(w, 4) || (post_w && !aligned(post_w, 4)) ||
      (residual_in && !aligned(residual_in, er)) || (residual_out && !aligned(residual_out, er)))
    return fail(SSM_ERR_INVALID_ARG, "a pointer is not aligned to its element");
  a.x = x, a.rin = residual_in, a.w = w, a.post = post_w, a.y = y, a.rout = residual_out;
  a.dim = static_cast<int>(d->dim), a.eps = d->eps, a.alpha = d->residual_scale;
  const int64_t st8 = a.x_st | a.y_st | (residual_in ? a.rin_st : 0) | (residual_out ? a.rout_st : 0) | d->dim;
  const bool vec = st8 % 8 == 0 && aligned(x, 16) && aligned(y, 16) && aligned(w, 16) && (!post_w || aligned(post_w, 16)) &&
                   (!residual_in || aligned(residual_in, 16)) && (!residual_out || aligned(residual_out, 16));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (d->io_dtype == SSM_BF16)
    err = d->residual_dtype == SSM_BF16 ? ssm::launch_residual_post<__nv_bfloat16, __nv_bfloat16>(a, d->rows, vec, st)
                                        : ssm::launch_residual_post<__nv_bfloat16, float>(a, d->rows, vec, st);
  else
    err = d->residual_dtype == SSM_BF16 ? ssm::launch_residual_post<float, __nv_bfloat16>(a, d->rows, vec, st)
                                        : ssm::launch_residual_post<float, float>(a, d->rows, vec, st);
  if (err != cudaSuccess) return fail(SSM_ERR_CUDA, "residual-norm launch: %s", cudaGetErrorString(err));
  return fail(SSM_OK, "");
}

}  // extern "C"
