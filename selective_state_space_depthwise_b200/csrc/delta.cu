// delta.cu -- the gated delta rule's entry points and its recurrent kernel
// (sm_100a). Per sequence and head, with S in R^{dv x dk} and a = exp(g):
//
//   u = beta (v - a S k),   S <- a S + u k^T,   o = scale S q.
//
// The rows of S do not meet: row r needs only its own dot products p = S_r.k
// and w = S_r.q, since u_r = beta (v_r - a p) and, with S taken before the
// update, o_r = scale (a w + u_r (k.q)). Both products come from one pass over
// the old row, so a token costs one reduction, not two in turn.
//
// A warp owns 8 steps of rows: with d_key in (64, 128] a row spans the 32
// lanes (four channels a lane), up to 64 it spans 16 lanes and a step covers
// two rows. The 16 partial products of the 8 steps are reduced together, each
// exchange halving the values a lane still carries (16 shuffles instead of
// 80), and end with one product per lane.
//
// The state stays in registers over the tokens of the call; a decode step is
// the same kernel with one token, bound by the state's stream (4 dv dk bytes
// in and out per row and head).
#include <cuda_bf16.h>

#include "delta_internal.h"
#include "sm100_ptx.cuh"
#include "ssm.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

constexpr int kRecWarps = 4;
constexpr int kRecSteps = 8;  // row steps of a warp

// Sums v[N] over the LPR lanes of a group. Lane i of the group returns entry i / (LPR / N).
template <int LPR, int N>
__device__ __forceinline__ float reduce_all(float (&v)[N], int lane) {
  int m = LPR / 2;
#pragma unroll
  for (int n = N; n > 1; n >>= 1, m >>= 1) {
    const bool hi = lane & m;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float give = hi ? v[i] : v[i + n / 2], keep = hi ? v[i + n / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
    }
  }
#pragma unroll
  for (; m > 0; m >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
  return v[0];
}

template <int LPR>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int m = LPR / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

__device__ __forceinline__ float4 load_bf16x4(const __nv_bfloat16* p, bool in) {
  if (!in) return make_float4(0.f, 0.f, 0.f, 0.f);
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}

__device__ __forceinline__ float dot4(float4 a, float4 b) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, a.x * b.x)));
}

// One block: kRecWarps * kRecSteps * 32 / LPR rows of one (sequence, head). Never with packed tokens (takes_chunks).
// One token: seven blocks an SM. A decode step of 256 x 60 heads of 128 x 128
// (2.03 GB) takes 301-325 us between boxes, 6.2-6.7 TB/s (on the best 301,
// with six blocks 311, five 338, eight 306). Its 72 registers hold it all; with
// up to 64 key channels 16 bytes spill.
template <int LPR, int BLOCKS>
__global__ void __launch_bounds__(32 * kRecWarps, BLOCKS) delta_recurrent_kernel(const DeltaArgs a, int row_blocks) {
  constexpr int kPar = 32 / LPR;           // rows of one step
  constexpr int kLanes = LPR / (2 * kRecSteps);  // lanes that hold one product
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t unit = blockIdx.x / row_blocks;
  const int64_t s = unit / a.H, h = unit % a.H;
  const int64_t grp = h / (a.H / a.G);
  const int row0 = (static_cast<int>(blockIdx.x % row_blocks) * kRecWarps + warp) * kRecSteps * kPar;
  if (row0 >= a.dv) return;

  int64_t slot = s;
  if (a.index) {
    slot = a.index[s];
    if (slot < 0 || slot >= a.num_states) return;  // padding
  }
  const int part = lane / LPR, c = (lane % LPR) * 4;
  const bool in = c < a.dk;
  const __nv_bfloat16* qp = a.q + s * a.q_seq + grp * a.dk + c;
  const __nv_bfloat16* kp = a.k + s * a.k_seq + grp * a.dk + c;
  const float* gp = a.g + s * a.gb_seq + h;
  const float* bp = a.beta + s * a.gb_seq + h;
  // The reduction leaves product `mine` here: p of step mine (< kRecSteps) or w of step mine - kRecSteps.
  const int mine = lane % LPR / kLanes, step = mine % kRecSteps;
  const int my_row = row0 + step * kPar + part;
  const bool row_in = my_row < a.dv;
  const __nv_bfloat16* vp = a.v + s * a.v_seq + h * a.dv + (row_in ? my_row : 0);
  __nv_bfloat16* op = a.out + s * a.o_seq + h * a.dv + my_row;
  const bool stores = row_in && mine >= kRecSteps && lane % kLanes == 0;

  float4 S[kRecSteps];
  const int64_t sbase = (slot * a.H + h) * a.dv;
#pragma unroll
  for (int i = 0; i < kRecSteps; ++i) {
    const int r = row0 + i * kPar + part;
    S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.state_in && in && r < a.dv)
      S[i] = __ldcs(reinterpret_cast<const float4*>(a.state_in + (sbase + r) * a.dk + c));
  }
  float4 q{}, k{};
  float g = 0.f, b = 0.f, v = 0.f;
  const int n = static_cast<int>(a.L);
  if (n > 0) q = load_bf16x4(qp, in), k = load_bf16x4(kp, in), g = *gp, b = *bp, v = __bfloat162float(*vp);
  for (int t = 0; t < n; ++t) {
    float4 qn{}, kn{};
    float gn = 0.f, bn = 0.f, vn = 0.f;
    if (t + 1 < n) {
      qp += a.q_tok, kp += a.k_tok, vp += a.v_tok, gp += a.gb_tok, bp += a.gb_tok;
      qn = load_bf16x4(qp, in), kn = load_bf16x4(kp, in), gn = *gp, bn = *bp, vn = __bfloat162float(*vp);
    }
    // The norms scale the products, not k and q: their sums are on the way while the products' are.
    // A key whose squares overflow makes rk NaN, and with it the update, as in the chunk kernels; without norms its
    // sum is looked at where a lane's part is large. Of a query with norms, rq.
    float rq = a.scale, rk = 1.0f;
    if (a.l2norm) {
      const float kk = group_sum<LPR>(dot4(k, k));
      rk = fmaf(kk, 0.0f, rsqrtf(kk + kL2Eps));
      const float qq = group_sum<LPR>(dot4(q, q));
      rq *= fmaf(qq, 0.0f, rsqrtf(qq + kL2Eps));
    } else if (__any_sync(0xffffffffu, !(dot4(k, k) <= 1e37f))) {
      rk = fmaf(group_sum<LPR>(dot4(k, k)), 0.0f, 1.0f);
    }
    const float kq = group_sum<LPR>(dot4(k, q)) * rk;
    const float decay = expf(g);
    float pw[2 * kRecSteps];
#pragma unroll
    for (int i = 0; i < kRecSteps; ++i) pw[i] = dot4(S[i], k), pw[kRecSteps + i] = dot4(S[i], q);
    const float mine_sum = reduce_all<LPR>(pw, lane);
    const float u = b * (v - decay * (mine_sum * rk));  // meant by the lanes that hold a p
#pragma unroll
    for (int i = 0; i < kRecSteps; ++i) {
      const float ui = __shfl_sync(0xffffffffu, u, part * LPR + kLanes * i) * rk;
      S[i].x = fmaf(decay, S[i].x, ui * k.x);
      S[i].y = fmaf(decay, S[i].y, ui * k.y);
      S[i].z = fmaf(decay, S[i].z, ui * k.z);
      S[i].w = fmaf(decay, S[i].w, ui * k.w);
    }
    const float um = __shfl_sync(0xffffffffu, u, part * LPR + kLanes * step);
    if (stores) *op = __float2bfloat16_rn(rq * fmaf(decay, mine_sum, um * kq));
    op += a.o_tok;
    q = qn, k = kn, g = gn, b = bn, v = vn;
  }
#pragma unroll
  for (int i = 0; i < kRecSteps; ++i) {
    const int r = row0 + i * kPar + part;
    if (in && r < a.dv) __stcs(reinterpret_cast<float4*>(a.state_out + (sbase + r) * a.dk + c), S[i]);
  }
}

// Blocks of a (sequence, head).
int64_t recurrent_blocks(int64_t dk, int64_t dv) {
  const int64_t rows = kRecWarps * kRecSteps * (dk > 64 ? 1 : 2);
  return (dv + rows - 1) / rows;
}

template <int LPR, int BLOCKS>
cudaError_t launch_recurrent_as(const DeltaArgs& a, cudaStream_t st) {
  const int rb = static_cast<int>(recurrent_blocks(a.dk, a.dv));
  delta_recurrent_kernel<LPR, BLOCKS>
      <<<static_cast<unsigned>(a.batch * a.H * rb), 32 * kRecWarps, 0, st>>>(a, rb);
  return cudaGetLastError();
}

// Over several tokens a block waits for its own sums, not for memory: four blocks an SM, whose registers hold it all
// (16 tokens of 32 heads of 128 x 128 take 10.1 us, with seven 13.8; of 64 sequences 229 us against 233).
cudaError_t launch_delta_recurrent(const DeltaArgs& a, cudaStream_t st) {
  if (a.L > 1) return a.dk > 64 ? launch_recurrent_as<32, 4>(a, st) : launch_recurrent_as<16, 4>(a, st);
  return a.dk > 64 ? launch_recurrent_as<32, 7>(a, st) : launch_recurrent_as<16, 7>(a, st);
}

ssm_status delta_shape(const ssm_delta_dims* d, bool prefill) {
  if (!d) return fail(SSM_ERR_INVALID_ARG, "dims is NULL");
  if (d->batch <= 0) return fail(SSM_ERR_INVALID_ARG, "batch=%lld must be > 0", (long long)d->batch);
  if (prefill && (d->seqlen < 0 || d->seqlen > 0x7fffff00))
    return fail(SSM_ERR_INVALID_ARG, "seqlen=%lld must be in 0..2^31-256", (long long)d->seqlen);
  if (d->nheads <= 0 || d->ngroups <= 0 || d->nheads % d->ngroups != 0)
    return fail(SSM_ERR_INVALID_ARG, "nheads=%lld must be a positive multiple of ngroups=%lld", (long long)d->nheads,
                (long long)d->ngroups);
  if (d->d_key < 8 || d->d_key > 128 || d->d_key % 8 != 0)
    return fail(SSM_ERR_UNSUPPORTED, "d_key=%lld: built for multiples of 8 up to 128", (long long)d->d_key);
  if (d->d_value < 8 || d->d_value > 4096 || d->d_value % 8 != 0)
    return fail(SSM_ERR_UNSUPPORTED, "d_value=%lld: built for multiples of 8 up to 4096", (long long)d->d_value);
  if (d->nheads > 0x7fffff || d->batch > 0x7fffff / d->nheads)
    return fail(SSM_ERR_INVALID_ARG, "batch * nheads must be below 2^23");
  if (prefill && d->seqlen > 0 && d->seqlen / 64 + 1 > 0x7fffffff / (d->batch * d->nheads))
    return fail(SSM_ERR_INVALID_ARG, "batch * nheads * seqlen / 64 must be below 2^31");
  if (!(d->scale >= 0.0f)) return fail(SSM_ERR_INVALID_ARG, "scale=%g must be > 0, or 0 for the default", d->scale);
  if (d->qk_l2norm != 0 && d->qk_l2norm != 1) return fail(SSM_ERR_INVALID_ARG, "qk_l2norm must be 0 or 1");
  return SSM_OK;
}

// Whether a prefill takes the chunk kernels. Packed lengths are known on the device alone. Below 64 tokens token by
// token may be faster, by these fits (us, within 15%) to 1 to 64 sequences of 8 to 80 heads: L tokens take 2.3 + L
// (0.47 + 0.00145 for each block beyond one an SM); one chunk 17.5 (3 less up to 64 key channels, 2.5 more in pairs)
// and 13 (16.5) for each further round of walks over the SMs, and 2 are added for its second launch. (32 heads of 128
// x 128: 24 tokens 13.9, 33 18.3, in chunks 17.7, but 21.8 and 26.3 call after call from the host; 64 sequences of
// them: 8 tokens 131, 16 228, in chunks 180.)
bool takes_chunks(const ssm_delta_dims& d, bool packed) {
  if (d.seqlen <= 0) return false;
  if (packed || d.seqlen >= kDeltaChunk) return true;
  const int64_t sms = device_sms();
  const int64_t blocks = d.batch * d.nheads * recurrent_blocks(d.d_key, d.d_value);
  const int64_t rounds = (d.batch * delta_walkers(d.nheads, d.ngroups, d.d_value) + sms - 1) / sms;
  const bool pair = delta_pairs(d.nheads, d.ngroups, d.d_value);
  const double token = 0.47 + (blocks > sms ? 0.00145 * static_cast<double>(blocks - sms) : 0.0);
  const double chunk = (pair ? 22.0 : 19.5) - (d.d_key <= 64 ? 3.0 : 0.0) +
                       (pair ? 16.5 : 13.0) * static_cast<double>(rounds - 1);
  return 2.3 + static_cast<double>(d.seqlen) * token > chunk;
}

// Shape, stride and pointer checks shared by both entry points.
ssm_status delta_args(const ssm_delta_dims* d, bool prefill, const void* q, const void* k, const void* v,
                      const float* g, const float* beta, void* out, const float* state_in, float* state_out,
                      DeltaArgs* a) {
  const ssm_status shape = delta_shape(d, prefill);
  if (shape != SSM_OK) return shape;
  const int64_t L = prefill ? d->seqlen : 1, nk = d->ngroups * d->d_key, nv = d->nheads * d->d_value;
  a->batch = d->batch, a->L = L, a->H = d->nheads, a->G = d->ngroups, a->dk = d->d_key, a->dv = d->d_value;
  auto tok = [](int64_t given, int64_t dense) { return given ? given : dense; };
  a->q_tok = tok(d->q_tok_stride, nk), a->k_tok = tok(d->k_tok_stride, nk), a->v_tok = tok(d->v_tok_stride, nv);
  a->o_tok = tok(d->out_tok_stride, nv), a->gb_tok = tok(d->gb_tok_stride, d->nheads);
  // Rows of a decode step are dense by default whatever the token strides, which it does not use.
  auto seq = [&](int64_t given, int64_t token, int64_t row) { return given ? given : prefill ? L * token : row; };
  a->q_seq = seq(d->q_seq_stride, a->q_tok, nk), a->k_seq = seq(d->k_seq_stride, a->k_tok, nk);
  a->v_seq = seq(d->v_seq_stride, a->v_tok, nv), a->o_seq = seq(d->out_seq_stride, a->o_tok, nv);
  a->gb_seq = seq(d->gb_seq_stride, a->gb_tok, d->nheads);
  const int64_t toks[4] = {a->q_tok, a->k_tok, a->v_tok, a->o_tok}, least[4] = {nk, nk, nv, nv};
  const int64_t seqs[4] = {a->q_seq, a->k_seq, a->v_seq, a->o_seq};
  for (int i = 0; i < 4; ++i) {
    if (toks[i] % 8 != 0 || seqs[i] < 0 || seqs[i] % 8 != 0)
      return fail(SSM_ERR_INVALID_ARG, "q/k/v/out strides must be non-negative multiples of 8 elements");
    if (toks[i] < least[i])
      return fail(SSM_ERR_INVALID_ARG, "q/k/v/out token strides must cover a token's heads");
  }
  if (a->gb_tok < d->nheads || a->gb_seq < 0)
    return fail(SSM_ERR_INVALID_ARG, "g/beta strides: token stride >= nheads, sequence stride >= 0");
  if (!state_out || !aligned(state_out, 16))
    return fail(SSM_ERR_INVALID_ARG, "state_out is NULL or not 16-byte aligned");
  if (state_in && !aligned(state_in, 16)) return fail(SSM_ERR_INVALID_ARG, "state_in is not 16-byte aligned");
  if (L > 0) {
    const void* io[4] = {q, k, v, out};
    const char* names[4] = {"q", "k", "v", "out"};
    for (int i = 0; i < 4; ++i) {
      if (!io[i]) return fail(SSM_ERR_INVALID_ARG, "%s is NULL", names[i]);
      if (!aligned(io[i], 16)) return fail(SSM_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
    }
    if (out == q || out == k || out == v) return fail(SSM_ERR_INVALID_ARG, "out must not overlap q, k or v");
    if (!g || !beta || !aligned(g, 4) || !aligned(beta, 4))
      return fail(SSM_ERR_INVALID_ARG, "g or beta is NULL or not 4-byte aligned");
  }
  a->q = static_cast<const __nv_bfloat16*>(q), a->k = static_cast<const __nv_bfloat16*>(k);
  a->v = static_cast<const __nv_bfloat16*>(v), a->out = static_cast<__nv_bfloat16*>(out);
  a->g = g, a->beta = beta, a->state_in = state_in, a->state_out = state_out;
  a->cu = nullptr, a->index = nullptr, a->num_states = d->batch;
  a->scale = d->scale != 0.0f ? d->scale : 1.0f / sqrtf(static_cast<float>(d->d_key));
  a->l2norm = d->qk_l2norm;
  a->two16 = 65536u;
  a->err = nullptr;
  return SSM_OK;
}

}  // namespace
}  // namespace ssm

extern "C" {

size_t ssm_delta_prefill_workspace_bytes(const ssm_delta_dims* dims, int32_t packed) {
  if (ssm::delta_shape(dims, true) != SSM_OK || !ssm::takes_chunks(*dims, packed)) return 0;
  return ssm::delta_chunk_workspace(dims->batch, dims->seqlen, dims->nheads, dims->ngroups, dims->d_key, dims->d_value, packed);
}

ssm_status ssm_delta_prefill(const ssm_delta_dims* dims, const void* q, const void* k, const void* v, const float* g,
                             const float* beta, const int32_t* cu_seqlens, const float* state_in, void* out,
                             float* state_out, void* workspace, size_t workspace_bytes, void* stream) {
  using ssm::fail;
  ssm::DeltaArgs a{};
  const ssm_status st = ssm::delta_args(dims, true, q, k, v, g, beta, out, state_in, state_out, &a);
  if (st != SSM_OK) return st;
  if (cu_seqlens && !ssm::aligned(cu_seqlens, 4)) return fail(SSM_ERR_INVALID_ARG, "cu_seqlens is not 4-byte aligned");
  a.cu = cu_seqlens;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (ssm::takes_chunks(*dims, a.cu)) {
    const size_t need = ssm::delta_chunk_workspace(a.batch, a.L, a.H, a.G, a.dk, a.dv, a.cu);
    if (!workspace || !ssm::aligned(workspace, 256))
      return fail(SSM_ERR_INVALID_ARG, "workspace is NULL or not 256-byte aligned");
    if (workspace_bytes < need)
      return fail(SSM_ERR_INVALID_ARG, "workspace of %zu bytes, need %zu", workspace_bytes, need);
    a.err = ssm::device_error_ptr();
    if (!a.err) return fail(SSM_ERR_CUDA, "device error word: %s", cudaGetErrorString(cudaGetLastError()));
    err = ssm::launch_delta_chunk(a, workspace, cs);
  } else {
    err = ssm::launch_delta_recurrent(a, cs);
  }
  if (err != cudaSuccess) return fail(SSM_ERR_CUDA, "delta-rule launch: %s", cudaGetErrorString(err));
  return fail(SSM_OK, "");
}

ssm_status ssm_delta_decode_step(const ssm_delta_dims* dims, const void* q, const void* k, const void* v,
                                 const float* g, const float* beta, const int32_t* state_index, int64_t num_states,
                                 const float* state_in, void* out, float* state_out, void* stream) {
  using ssm::fail;
  ssm::DeltaArgs a{};
  const ssm_status st = ssm::delta_args(dims, false, q, k, v, g, beta, out, state_in, state_out, &a);
  if (st != SSM_OK) return st;
  if (!state_in) return fail(SSM_ERR_INVALID_ARG, "state_in is NULL");
  if (num_states <= 0 || (!state_index && num_states < dims->batch))
    return fail(SSM_ERR_INVALID_ARG, "num_states=%lld: must be > 0, and >= batch without state_index",
                (long long)num_states);
  if (state_index && !ssm::aligned(state_index, 4))
    return fail(SSM_ERR_INVALID_ARG, "state_index is not 4-byte aligned");
  a.index = state_index, a.num_states = num_states;
  const cudaError_t err = ssm::launch_delta_recurrent(a, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return fail(SSM_ERR_CUDA, "delta-rule decode launch: %s", cudaGetErrorString(err));
  return fail(SSM_OK, "");
}

}  // extern "C"
