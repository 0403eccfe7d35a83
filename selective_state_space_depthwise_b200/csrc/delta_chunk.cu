// delta_chunk.cu -- the gated delta rule over whole sequences, 64 tokens at a
// time on the tensor cores (sm_100a).
//
// With G_i the running sum of g within a chunk, S the state before it and the
// keys k_i as rows of K, the chunk's updates u_i (rows of U) satisfy
//
//   (I + A) U = diag(beta) (V - diag(e^G) K S^T),
//   A_ij = beta_i e^{G_i - G_j} k_i.k_j   (j < i),
//
// so with T = (I + A)^-1 diag(beta), a unit triangular inverse that does not
// depend on S, a chunk is four products around the state:
//
//   Y = K S^T,  R = V - diag(e^G) Y,  U = T R,
//   O = scale (diag(e^G) Q S^T + (Q K^T * e^{G_i - G_j}, j <= i) U),
//   S <- e^{G_C} S + sum_j e^{G_C - G_j} u_j k_j^T.
//
// Transposed, with the 128 rows of S (a slice of d_value) as the 128 lanes of
// tensor memory, every left operand (S, R, U) is an accumulator read back,
// scaled and split in registers, and stored to tensor memory as the next
// product's A operand: the state never leaves the SM, and shared memory holds
// only the right operands (K, Q by TMA; T and the masked scores).
//
// Precision. q, k and v are bf16 and enter exactly; the key norms, decays and
// beta are fp32 factors of rows and columns, never folded into a bf16 operand.
// S, R, U and T are fp32 and go to the tensor cores as three bf16 terms (the
// top 8 bits, the next 8, the last 8 of the significand: exact), as many
// products as pairs of terms above 2^-24. Only the output's own product takes
// two terms (2^-16, against its rounding to bf16). The tensor core adds into
// fp32 accumulators with truncation, so the state itself is added up in fp32
// registers, and the accumulators hold one chunk's contribution at a time.
//
// One CTA per (sequence, head, 128 rows of d_value), 20 warps:
//   warps 0-7   state: hold S (a thread: one row, half of the key channels),
//               form the A operands between the products;
//   warps 8-11  prep, one chunk ahead: running decays, key norms, A and the
//               masked scores from one 128 x 64 product [K; Q] K^T, the inverse;
//   warps 12-15 output: both terms of O from tensor memory, rounded and stored;
//   warp 16     one thread issues the TMA loads (three chunks ahead) and every MMA
//               (warps 17-19 only complete its warpgroup).
// Values that are not finite: a product with a zero would spread them to tokens
// before theirs, so the state warps take them out of the operands, mark the
// first such token of each row, and the output warps write NaN from there on.
#include <cuda.h>
#include <cuda_bf16.h>

#include "delta_internal.h"
#include "sm100_ptx.cuh"
#include "ssm.h"
#include "ssm_internal.h"
#include "ssm_math.cuh"
#include "tma_map.cuh"

namespace ssm {
namespace {

constexpr int kC = 64;  // tokens of a chunk
constexpr int kStateWarps = 8, kPrepWarp = 8, kOutWarp = 12, kCtlWarp = 16;
constexpr int kChunkThreads = 32 * 20;
// Registers. 20 warps launch with 96 a thread (five warps on each quarter of
// an SM); the state warps, which hold half a row of S, take what the output
// and control warps give up: 2 x 120 + 96 + 88 + 56 = 5 x 96.
constexpr int kLaunchRegs = 96, kStateRegs = 120, kOutRegs = 88, kCtlRegs = 56;
static_assert(2 * kStateRegs + kLaunchRegs + kOutRegs + kCtlRegs <= 5 * kLaunchRegs, "register split");
constexpr int kStages = 3;
constexpr int kALd = 68;  // floats between rows of A (16-byte rows, conflict-free columns)

// Tensor memory, 512 columns.
constexpr uint32_t kTmDelta = 0;    // the chunk's contribution to S; before it, R's three terms
constexpr uint32_t kTmS = 128;      // S's three terms: half h at 96 h; then U's scaled terms in the second half
constexpr uint32_t kTmY = 320;      // Y, then U
constexpr uint32_t kTmO = 384;      // Q S^T, then the scores times U
constexpr uint32_t kTmG = 448;      // [K; Q] K^T of the next chunk; then U's two output terms

struct Coef {
  float eg[kC];   // e^{G_j} |k_j|^-1: scales Y
  float ec[kC];   // e^{G_C - G_j} |k_j|^-1, 0 behind the sequence: scales U into the state
  float oq[kC];   // scale e^{G_i} |q_i|^-1: scales Q S^T
  float decay;    // e^{G_C}
  float pad[3];
};

template <int KA>  // 64-column atoms of d_key
struct ChunkSmem {
  static constexpr int kAtom = kC * 128;          // 64 rows of 128 bytes
  static constexpr int kKQ = KA * 2 * kAtom;      // per atom: K, then Q
  static constexpr int kV = kC * 256;             // [token][128]
  static constexpr int kStage = kKQ + kV;
  static constexpr int kT = kStages * kStage;     // three terms [i][j]
  static constexpr int kP = kT + 3 * kAtom;       // two buffers of two terms [i][j]
  static constexpr int kA = kP + 4 * kAtom;       // fp32 [64][kALd]
  static constexpr int kCoef = kA + kC * kALd * 4;
  static constexpr int kVec = kCoef + 4 * static_cast<int>(sizeof(Coef));  // Ghi, Glo, rk [64], beta [2][64]
  static constexpr int kBad = kVec + 5 * kC * 4;  // int [2][128]
  static constexpr int kBar = kBad + 2 * 128 * 4;
  static constexpr int kNumBars = kStages + 15;
  static constexpr int kMisc = kBar + kNumBars * 8;  // TMEM address, abort flag
  static constexpr int kTotal = kMisc + 16;
  static_assert(kBar % 8 == 0 && kCoef % 16 == 0 && kVec % 16 == 0, "alignment");
  static_assert(kTotal + 1024 <= 232448, "227 KB of shared memory");
  static constexpr uint32_t kTx = static_cast<uint32_t>(kStage);
};

enum Bar {  // after the stages' full barriers; each completes once a chunk
  kGDone, kGFree, kTPReady, kSReady0, kSReady1, kYDone, kOiDone, kRReady, kUDone, kUsReady, kSDone0, kSDone1, kUoReady,
  kOiRead, kOaDone,  // kOFree follows
  kNumNamed
};
static_assert(kNumNamed == 15, "barrier count");

struct ChunkMaps {
  CUtensorMap q, k, v;
};

__host__ __device__ constexpr uint32_t chunk_idesc(int n, bool b_mn_major) {  // bf16 x bf16 -> fp32, M = 128
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn_major ? (1u << 16) : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (8u << 24);
}

// A wait that all threads of a warp make together. Once any wait of the CTA
// has run out, the flag lets the others through: every loop ends, on memory
// of its own, and the error word tells the host.
struct Waiter {
  volatile int* abort;
  int* err;
  __device__ __forceinline__ void slow(uint32_t bar, uint32_t parity, int code) const {
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
#pragma unroll 1
      for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return;
      if (*abort) return;
      if (globaltimer_ns() - t0 > 2000000000ull) {
        *abort = 1;
        if (err) atomicExch(err, code);
        return;
      }
    }
  }
  __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity, int code) const {
    if (!mbar_try_wait(bar, parity)) slow(bar, parity, code);
  }
};

// x0, x1 as three packed bf16 pairs whose sum is exact: 8 bits of the significand each.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t& h, uint32_t& m, uint32_t& l) {
  const uint32_t a0 = __float_as_uint(x0), a1 = __float_as_uint(x1);
  h = __byte_perm(a0, a1, 0x7632);
  const float r0 = x0 - __uint_as_float(a0 & 0xffff0000u), r1 = x1 - __uint_as_float(a1 & 0xffff0000u);
  const uint32_t b0 = __float_as_uint(r0), b1 = __float_as_uint(r1);
  m = __byte_perm(b0, b1, 0x7632);
  const float s0 = r0 - __uint_as_float(b0 & 0xffff0000u), s1 = r1 - __uint_as_float(b1 & 0xffff0000u);
  l = __byte_perm(__float_as_uint(s0), __float_as_uint(s1), 0x7632);
}
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& h, uint32_t& m) {
  const uint32_t a0 = __float_as_uint(x0), a1 = __float_as_uint(x1);
  h = __byte_perm(a0, a1, 0x7632);
  const float r0 = x0 - __uint_as_float(a0 & 0xffff0000u), r1 = x1 - __uint_as_float(a1 & 0xffff0000u);
  const __nv_bfloat162 p = __floats2bfloat162_rn(r0, r1);
  m = *reinterpret_cast<const uint32_t*>(&p);
}

// 16 values of a row as three terms at columns col + t * stride of A-operand tensor memory.
__device__ __forceinline__ void store_split3(uint32_t col, uint32_t stride, const float (&x)[16]) {
  uint32_t h[8], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) split3(x[2 * i], x[2 * i + 1], h[i], m[i], l[i]);
  tmem_st_x8(col, h);
  tmem_st_x8(col + stride, m);
  tmem_st_x8(col + 2 * stride, l);
}

__device__ __forceinline__ int sw128(int r, int j) { return r * 128 + ((j ^ (r & 7)) << 4); }

// Bit i set where x[i] is not finite.
template <int N>
__device__ __forceinline__ uint32_t not_finite(const float (&x)[N]) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) s = fmaf(x[i], 0.0f, s);
  if (s == 0.0f) return 0u;
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (!(fabsf(x[i]) <= 3.4028235e38f)) bits |= 1u << i;
  return bits;
}

constexpr int kPrepBar = 1;  // named barrier of the prep warps

template <int KA>
__global__ void __launch_bounds__(kChunkThreads, 1)
    delta_chunk_kernel(const __grid_constant__ ChunkMaps maps, const DeltaArgs a, int slices) {
  using M = ChunkSmem<KA>;
  constexpr int DK = 64 * KA;
  constexpr int HC = DK / 2;   // key channels of a state thread
  constexpr int BLK = HC / 2;  // of one half-step of the state's conversion
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int slice = static_cast<int>(blockIdx.x) % slices;
  const int unit = static_cast<int>(blockIdx.x) / slices;
  const int h = unit % static_cast<int>(a.H), s = unit / static_cast<int>(a.H);
  const int grp = h / static_cast<int>(a.H / a.G);

  int t0 = 0, len = static_cast<int>(a.L), seq = s;
  if (a.cu) {
    const int T = static_cast<int>(a.L);
    t0 = min(max(a.cu[s], 0), T);
    len = min(max(a.cu[s + 1], t0), T) - t0;
    seq = 0;
  }
  const int nc = (len + kC - 1) / kC;

  auto bar = [&](int b) { return sb + M::kBar + 8 * (kStages + b); };
  auto full = [&](int st) { return sb + M::kBar + 8 * st; };
  // 15 named barriers and one more: the output accumulator has been read.
  const uint32_t o_free = sb + M::kMisc + 8;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + M::kMisc + 4);
  const Waiter wait{abort, a.err};
  Coef* coefs = reinterpret_cast<Coef*>(smem + M::kCoef);
  int* bad = reinterpret_cast<int*>(smem + M::kBad);

  if (tid == 32 * kCtlWarp) {
    for (int i = 0; i < kStages; ++i) mbar_init(full(i), 1);
    const uint32_t counts[kNumNamed] = {1, 4, 4, 8, 8, 1, 1, 8, 1, 8, 1, 1, 8, 4, 1};
    for (int i = 0; i < kNumNamed; ++i) mbar_init(bar(i), counts[i]);
    mbar_init(o_free, 4);
    *abort = 0;
    mbar_fence_init();
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }
  if (warp == kCtlWarp) {
    __syncwarp();
    tmem_alloc(sb + M::kMisc, 512);
    tmem_relinquish();
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + M::kMisc);
  const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;  // this warp's lane quarter

  if (warp < kStateWarps) {
    // ------------------------------------------------------------- state ---
    setmaxnreg_inc<kStateRegs>();
    const int half = warp >> 2, row = 32 * (warp & 3) + lane;
    const int64_t r = static_cast<int64_t>(slice) * 128 + row;
    const bool row_in = r < a.dv;
    const int64_t sbase = ((static_cast<int64_t>(s) * a.H + h) * a.dv + (row_in ? r : 0)) * a.dk + half * HC;
    const int cols = static_cast<int>(min(static_cast<int64_t>(HC), max(a.dk - half * HC, static_cast<int64_t>(0))));
    float S[HC];
#pragma unroll
    for (int i = 0; i < HC; i += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.state_in && row_in && i < cols) v = *reinterpret_cast<const float4*>(a.state_in + sbase + i);
      S[i] = v.x, S[i + 1] = v.y, S[i + 2] = v.z, S[i + 3] = v.w;
    }
    const uint32_t tm = tmem + lanes;
    float decay = 0.0f;
    for (int c = 0; c < nc; ++c) {
      const uint32_t ph = c & 1;
      const Coef& cf = coefs[c & 3];
      const int n = min(kC, len - kC * c);
      // S, with the last chunk's contribution, as the A operand of Y and Q S^T
      wait(bar(kTPReady), ph, 31);
      if (c > 0) {
        wait(bar(kSDone0 + half), ph ^ 1u, 32);
        tcgen05_fence_after();
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int i0 = b * BLK; i0 < (b + 1) * BLK; i0 += 16) {
          float x[16];
          if (c > 0) {
            uint32_t d[16];
            tmem_ld_x16(tm + kTmDelta + half * HC + i0, d);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i0 + i] = fmaf(decay, S[i0 + i], __uint_as_float(d[i]));
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = S[i0 + i];
          store_split3(tm + kTmS + half * 96 + i0 / 2, HC / 2, x);
        }
        tmem_st_wait();
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSReady0 + b));
      }
      decay = cf.decay;
      // R = V - e^G Y
      const int st = c % kStages;
      const unsigned char* vt = smem + st * M::kStage + M::kKQ + row * 2;
      wait(full(st), (c / kStages) & 1, 33);
      wait(bar(kYDone), ph, 34);
      tcgen05_fence_after();
      uint32_t marks = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j0 = 32 * half + 16 * u;
        uint32_t d[16];
        float x[16];
        tmem_ld_x16(tm + kTmY + j0, d);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float v = __uint_as_float(static_cast<uint32_t>(
                              *reinterpret_cast<const uint16_t*>(vt + (j0 + i) * 256)) << 16);
          x[i] = j0 + i < n ? fmaf(-cf.eg[j0 + i], __uint_as_float(d[i]), v) : 0.0f;
        }
        const uint32_t nf = not_finite(x);
        if (nf) {
          marks |= nf << (16 * u);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (nf >> i & 1) x[i] = 0.0f;
        }
        __syncwarp();
        store_split3(tm + kTmDelta + j0 / 2, 32, x);
      }
      tmem_st_wait();
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kRReady));
      // U: scaled into the state's product, plain into the output's
      wait(bar(kUDone), ph, 35);
      tcgen05_fence_after();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j0 = 32 * half + 16 * u;
        uint32_t d[16];
        float x[16];
        tmem_ld_x16(tm + kTmY + j0, d);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(d[i]);
        marks |= not_finite(x) << (16 * u);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= cf.ec[j0 + i];
        const uint32_t mk = marks >> (16 * u) & 0xffffu;
        if (mk) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (mk >> i & 1) x[i] = __uint_as_float(0x7fffffffu);
        }
        __syncwarp();
        store_split3(tm + kTmS + 96 + j0 / 2, 32, x);
      }
      tmem_st_wait();
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kUsReady));
      const int first = marks ? __ffs(marks) - 1 : 32;
      bad[half * 128 + row] = marks ? 32 * half + first : kC;
      if (c + 1 < nc) wait(bar(kGFree), ph ^ 1u, 36);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t d[16], hi[8], mi[8];
        tmem_ld_x16(tm + kTmY + 32 * half + 16 * u, d);
        tmem_ld_wait();
        if (marks) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (16 * u + i >= first) d[i] = 0u;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          split2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1]), hi[i], mi[i]);
        tmem_st_x8(tm + kTmG + 16 * half + 8 * u, hi);
        tmem_st_x8(tm + kTmG + 32 + 16 * half + 8 * u, mi);
      }
      tmem_st_wait();
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kUoReady));
    }
    if (nc > 0) {
      wait(bar(kSDone0 + half), (nc - 1) & 1, 32);
      tcgen05_fence_after();
#pragma unroll
      for (int i0 = 0; i0 < HC; i0 += 16) {
        uint32_t d[16];
        tmem_ld_x16(tm + kTmDelta + half * HC + i0, d);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i0 + i] = fmaf(decay, S[i0 + i], __uint_as_float(d[i]));
      }
    }
    if (row_in) {
#pragma unroll
      for (int i = 0; i < HC; i += 4)
        if (i < cols)
          *reinterpret_cast<float4*>(a.state_out + sbase + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
    }
  } else if (warp < kOutWarp) {
    // -------------------------------------------------------------- prep ---
    const int pt = tid - 32 * kPrepWarp;  // row of [K; Q]
    const int i = pt & 63;                // its token
    const bool is_q = pt >= 64;
    float* As = reinterpret_cast<float*>(smem + M::kA);
    float* Ghi = reinterpret_cast<float*>(smem + M::kVec);
    float* Glo = Ghi + kC;
    float* rk = Glo + kC;
    float* betas = rk + kC;
    const int64_t gb0 = static_cast<int64_t>(seq) * a.gb_seq + static_cast<int64_t>(t0) * a.gb_tok + h;
    // g of tokens 2 l, 2 l + 1 in warp 0's lane l, beta of token pt - 64 in warps 2 and 3, one chunk ahead
    auto fetch = [&](int c, float& x, float& y) {
      x = y = 0.0f;
      if (pt < 32) {
        const int j = kC * c + 2 * pt;
        if (j < len) x = a.g[gb0 + j * a.gb_tok];
        if (j + 1 < len) y = a.g[gb0 + (j + 1) * a.gb_tok];
      } else if (is_q) {
        const int j = kC * c + i;
        if (j < len) x = a.beta[gb0 + j * a.gb_tok];
      }
    };
    float f0, f1;
    fetch(0, f0, f1);
    for (int c = 0; c < nc; ++c) {
      const uint32_t ph = c & 1;
      Coef& cf = coefs[c & 3];
      float* beta = betas + ph * kC;
      const int n = min(kC, len - kC * c);
      const int st = c % kStages;
      // Running sums of g in log2 units and fp64, kept as two floats: differences of far sums stay exact.
      if (pt < 32) {
        auto lg = [](float g) {
          const double v = static_cast<double>(g) * 1.4426950408889634;
          return v < -256.0 ? -256.0 : v;
        };
        const double g0 = lg(f0), g1 = lg(f1);
        double sum = g0 + g1;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const double o = __shfl_up_sync(0xffffffffu, sum, d);
          if (lane >= d) sum += o;
        }
        const double first = sum - g1;
        const float h0 = static_cast<float>(first), h1 = static_cast<float>(sum);
        Ghi[2 * lane] = h0, Ghi[2 * lane + 1] = h1;
        Glo[2 * lane] = static_cast<float>(first - h0), Glo[2 * lane + 1] = static_cast<float>(sum - h1);
      } else if (is_q) {
        beta[i] = f0;
      }
      if (c + 1 < nc) fetch(c + 1, f0, f1);
      wait(full(st), (c / kStages) & 1, 37);
      float rn = 1.0f;  // 1 / |row|
      if (a.l2norm) {
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < KA; ++t) {
          const unsigned char* base = smem + st * M::kStage + t * 2 * M::kAtom + (is_q ? M::kAtom : 0);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 w = *reinterpret_cast<const uint4*>(base + sw128(i, j));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float lo = __uint_as_float(u[e] << 16), hi = __uint_as_float(u[e] & 0xffff0000u);
              sum = fmaf(lo, lo, fmaf(hi, hi, sum));
            }
          }
        }
        rn = rsqrtf(sum + kL2Eps);
      }
      if (!is_q) rk[i] = rn;
      named_bar_sync(kPrepBar, 128);
      const float Gi = Ghi[i], Gl = Glo[i];
      if (is_q) {
        rn *= a.scale;
        cf.oq[i] = ex2_approx(Gi + Gl) * rn;
      } else {
        cf.eg[i] = ex2_approx(Gi + Gl) * rn;
        cf.ec[i] = i < n ? ex2_approx((Ghi[kC - 1] - Gi) + (Glo[kC - 1] - Gl)) * rn : 0.0f;
        if (i == 0) cf.decay = ex2_approx(Ghi[kC - 1] + Glo[kC - 1]);
      }
      // This row of [K; Q] K^T
      wait(bar(kGDone), ph, 38);
      tcgen05_fence_after();
      const int wi = 32 * ((warp >> 0) & 1);  // first token of this warp's rows
      const float lead = is_q ? rn : rn * beta[i];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t d[32];
        tmem_ld_x32(tmem + lanes + kTmG + 32 * b, d);
        tmem_ld_wait();
        if (b == 1) {
          tcgen05_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kGFree));
        }
        if (32 * b > wi) continue;  // columns behind every row of the warp: never read
#pragma unroll
        for (int j0 = 0; j0 < 32; j0 += 8) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const int j = 32 * b + j0 + e;
            const float4 gh = *reinterpret_cast<const float4*>(Ghi + j), gl = *reinterpret_cast<const float4*>(Glo + j);
            const float4 rj = *reinterpret_cast<const float4*>(rk + j);
            const float ghs[4] = {gh.x, gh.y, gh.z, gh.w}, gls[4] = {gl.x, gl.y, gl.z, gl.w};
            const float rjs[4] = {rj.x, rj.y, rj.z, rj.w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const float w = ex2_approx((Gi - ghs[z]) + (Gl - gls[z])) * rjs[z];
              const bool keep = is_q ? j + z <= i : (j + z < i && i < n);
              f[e + z] = keep ? lead * w * __uint_as_float(d[j0 + e + z]) : 0.0f;
            }
          }
          const int j = 32 * b + j0;
          if (is_q) {
            uint32_t hi[4], mi[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) split2(f[2 * z], f[2 * z + 1], hi[z], mi[z]);
            unsigned char* p = smem + M::kP + ph * 2 * M::kAtom + sw128(i, j >> 3);
            *reinterpret_cast<uint4*>(p) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(p + M::kAtom) = make_uint4(mi[0], mi[1], mi[2], mi[3]);
          } else {
            float4* p = reinterpret_cast<float4*>(As + i * kALd + j);
            p[0] = make_float4(f[0], f[1], f[2], f[3]);
            p[1] = make_float4(f[4], f[5], f[6], f[7]);
          }
        }
      }
      // Keys behind the sequence (the next packed sequence's) meet zeros of U: they must be finite.
      if (a.cu && n < kC && !is_q && i >= n) {
#pragma unroll
        for (int t = 0; t < KA; ++t)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(smem + st * M::kStage + t * 2 * M::kAtom + sw128(i, j)) = make_uint4(0, 0, 0, 0);
      }
      named_bar_sync(kPrepBar, 128);
      // (I + A)^-1: the two 32 x 32 diagonal blocks by substitution, a column per
      // thread; then the block below them, -T22 (A21 T11), eight rows of a column
      // per thread. The unused upper right block of As holds A21 T11.
      const int col = lane, rg = warp & 3;
      if (!is_q) {
        const float* Ab = As + wi * (kALd + 1);
        float x[32];
#pragma unroll
        for (int r = 0; r < 32; ++r) {
          float acc[4] = {r == col ? 1.0f : 0.0f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < r; k += 4) {
            const float4 w = *reinterpret_cast<const float4*>(Ab + r * kALd + k);
            acc[0] = fmaf(-w.x, x[k], acc[0]);
            if (k + 1 < r) acc[1] = fmaf(-w.y, x[k + 1], acc[1]);
            if (k + 2 < r) acc[2] = fmaf(-w.z, x[k + 2], acc[2]);
            if (k + 3 < r) acc[3] = fmaf(-w.w, x[k + 3], acc[3]);
          }
          x[r] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 32; ++r) As[(wi + r) * kALd + wi + col] = x[r];
      }
      named_bar_sync(kPrepBar, 128);
      {
        float acc[8] = {};
#pragma unroll 4
        for (int k = 0; k < 32; k += 4) {
          const float t0v = As[k * kALd + col], t1v = As[(k + 1) * kALd + col], t2v = As[(k + 2) * kALd + col],
                      t3v = As[(k + 3) * kALd + col];
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const float4 w = *reinterpret_cast<const float4*>(As + (32 + 8 * rg + r) * kALd + k);
            acc[r] = fmaf(w.x, t0v, fmaf(w.y, t1v, fmaf(w.z, t2v, fmaf(w.w, t3v, acc[r]))));
          }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) As[(8 * rg + r) * kALd + 32 + col] = acc[r];
        named_bar_sync(kPrepBar, 128);
#pragma unroll
        for (int r = 0; r < 8; ++r) acc[r] = 0.0f;
#pragma unroll 4
        for (int k = 0; k < 32; k += 4) {
          const float* w0 = As + k * kALd + 32 + col;
          const float t0v = w0[0], t1v = w0[kALd], t2v = w0[2 * kALd], t3v = w0[3 * kALd];
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const float4 w = *reinterpret_cast<const float4*>(As + (32 + 8 * rg + r) * kALd + 32 + k);
            acc[r] = fmaf(-w.x, t0v, fmaf(-w.y, t1v, fmaf(-w.z, t2v, fmaf(-w.w, t3v, acc[r]))));
          }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) As[(32 + 8 * rg + r) * kALd + col] = acc[r];
      }
      named_bar_sync(kPrepBar, 128);
      // T = the inverse times beta by column, three terms, once the last chunk's product has read the buffer
      if (c > 0) wait(bar(kUDone), ph ^ 1u, 39);
      {
        const int r = pt >> 1, j0 = 32 * (pt & 1);
#pragma unroll
        for (int jj = 0; jj < 32; jj += 8) {
          const int j = j0 + jj;
          if (j > (r | 15)) continue;  // columns that no product reads
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const float4 w = *reinterpret_cast<const float4*>(As + r * kALd + j + e);
            const float4 b4 = *reinterpret_cast<const float4*>(beta + j + e);
            f[e] = j + e <= r ? w.x * b4.x : 0.0f;
            f[e + 1] = j + e + 1 <= r ? w.y * b4.y : 0.0f;
            f[e + 2] = j + e + 2 <= r ? w.z * b4.z : 0.0f;
            f[e + 3] = j + e + 3 <= r ? w.w * b4.w : 0.0f;
          }
          uint32_t hi[4], mi[4], lo[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) split3(f[2 * z], f[2 * z + 1], hi[z], mi[z], lo[z]);
          unsigned char* p = smem + M::kT + sw128(r, j >> 3);
          *reinterpret_cast<uint4*>(p) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(p + M::kAtom) = make_uint4(mi[0], mi[1], mi[2], mi[3]);
          *reinterpret_cast<uint4*>(p + 2 * M::kAtom) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kTPReady));
    }
  } else if (warp < kCtlWarp) {
    // ------------------------------------------------------------ output ---
    setmaxnreg_dec<kOutRegs>();
    const int row = 32 * (warp & 3) + lane;
    const int64_t r = static_cast<int64_t>(slice) * 128 + row;
    const bool row_in = r < a.dv;
    __nv_bfloat16* op = a.out + static_cast<int64_t>(seq) * a.o_seq + static_cast<int64_t>(t0) * a.o_tok + h * a.dv +
                        (row_in ? r : 0);
    const uint32_t tm = tmem + lanes + kTmO;
    for (int c = 0; c < nc; ++c) {
      const uint32_t ph = c & 1;
      const Coef& cf = coefs[c & 3];
      const int n = min(kC, len - kC * c);
      uint32_t d0[32], d1[32];
      wait(bar(kOiDone), ph, 40);
      tcgen05_fence_after();
      tmem_ld_x32(tm, d0);
      tmem_ld_x32(tm + 32, d1);
      tmem_ld_wait();
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kOiRead));
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        d0[i] = __float_as_uint(cf.oq[i] * __uint_as_float(d0[i]));
        d1[i] = __float_as_uint(cf.oq[32 + i] * __uint_as_float(d1[i]));
      }
      wait(bar(kOaDone), ph, 41);
      tcgen05_fence_after();
      const int first = min(bad[row], bad[128 + row]);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t e[16];
        tmem_ld_x16(tm + 16 * b, e);
        tmem_ld_wait();
        if (b == 3) {
          tcgen05_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int t = 16 * b + i;
          const float inter = __uint_as_float(b < 2 ? d0[t & 31] : d1[t & 31]);
          const float o = t < first ? inter + __uint_as_float(e[i]) : __uint_as_float(0x7fffffffu);
          if (t < n && row_in) op[t * a.o_tok] = __float2bfloat16_rn(o);
        }
      }
      op += kC * a.o_tok;
    }
  } else {
    // ----------------------------------------------------------- control ---
    setmaxnreg_dec<kCtlRegs>();
    if (tid == 32 * kCtlWarp) {
    auto load = [&](int c) {
      if (*abort) return;
      const int st = c % kStages, tok = t0 + kC * c;
      const uint32_t base = sb + st * M::kStage;
      mbar_arrive_expect_tx(full(st), M::kTx);
#pragma unroll
      for (int t = 0; t < KA; ++t) {
        tma_load_4d(base + t * 2 * M::kAtom, &maps.k, 64 * t, grp, tok, seq, full(st));
        tma_load_4d(base + t * 2 * M::kAtom + M::kAtom, &maps.q, 64 * t, grp, tok, seq, full(st));
      }
      tma_load_4d(base + M::kKQ, &maps.v, 128 * slice, h, tok, seq, full(st));
    };
    int loaded = min(nc, kStages);
    for (int c = 0; c < loaded; ++c) load(c);
    auto katom = [&](int c, int t) { return sb + (c % kStages) * M::kStage + t * 2 * M::kAtom; };
    auto scores = [&](int c) {  // [K; Q] K^T
      wait(full(c % kStages), (c / kStages) & 1, 42);
      tcgen05_fence_after();
#pragma unroll
      for (int t = 0; t < KA; ++t)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t d = umma_desc_k_sw128(katom(c, t) + 32 * kk);
          umma_f16_ss(tmem + kTmG, d, d, chunk_idesc(64, false), t + kk > 0);
        }
      umma_commit(bar(kGDone));
    };
    if (nc > 0) scores(0);
    if (nc > 1) {
      wait(bar(kGFree), 0, 43);
      tcgen05_fence_after();
      scores(1);
    }
    for (int c = 0; c < nc; ++c) {
      const uint32_t ph = c & 1;
      wait(bar(kTPReady), ph, 44);
      // Y = S K^T, least terms first
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        wait(bar(kSReady0 + b), ph, 45);
        tcgen05_fence_after();
#pragma unroll
        for (int t = 2; t >= 0; --t)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int ks = 0; ks < BLK / 16; ++ks) {
              const int k = hf * HC + b * BLK + 16 * ks;
              umma_f16_ts(tmem + kTmY, tmem + kTmS + hf * 96 + t * (HC / 2) + (b * BLK + 16 * ks) / 2,
                          umma_desc_k_sw128(katom(c, k / 64) + (k % 64) * 2), chunk_idesc(64, false),
                          !(b == 0 && t == 2 && hf == 0 && ks == 0));
            }
      }
      umma_commit(bar(kYDone));
      // every use of chunk c - 1's stage is over: its product into S has been read
      if (c > 0 && c + kStages - 1 < nc) {
        load(c + kStages - 1);
        loaded = c + kStages;
      }
      // Q S^T
      if (c > 0) wait(o_free, ph ^ 1u, 46);
      tcgen05_fence_after();
#pragma unroll
      for (int t = 1; t >= 0; --t)
#pragma unroll
        for (int k = 0; k < DK; k += 16)
          umma_f16_ts(tmem + kTmO, tmem + kTmS + (k / HC) * 96 + t * (HC / 2) + (k % HC) / 2,
                      umma_desc_k_sw128(katom(c, k / 64) + M::kAtom + (k % 64) * 2), chunk_idesc(64, false),
                      !(t == 1 && k == 0));
      umma_commit(bar(kOiDone));
      // U = R T^T: 16 tokens j at a time meet the tokens i from theirs on
      wait(bar(kRReady), ph, 47);
      tcgen05_fence_after();
#pragma unroll
      for (int pr = 0; pr < 6; ++pr) {
        constexpr int kTt[6] = {2, 0, 1, 1, 0, 0}, kTr[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_ts(tmem + kTmY + 16 * kk, tmem + kTmDelta + 32 * kTr[pr] + 8 * kk,
                      umma_desc_k_sw128(sb + M::kT + kTt[pr] * M::kAtom + 2048 * kk + 32 * kk),
                      chunk_idesc(64 - 16 * kk, false), pr + kk > 0);
      }
      umma_commit(bar(kUDone));
      // the chunk's contribution to S
      wait(bar(kUsReady), ph, 48);
      tcgen05_fence_after();
#pragma unroll
      for (int at = 0; at < KA; ++at) {
#pragma unroll
        for (int t = 2; t >= 0; --t)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_f16_ts(tmem + kTmDelta + 64 * at, tmem + kTmS + 96 + 32 * t + 8 * kk,
                        umma_desc_k_sw128(katom(c, at) + 2048 * kk), chunk_idesc(64, true), !(t == 2 && kk == 0));
        umma_commit(bar(kSDone0 + at));
      }
      if (KA == 1) umma_commit(bar(kSDone1));
      // the scores times U
      wait(bar(kOiRead), ph, 49);
      wait(bar(kUoReady), ph, 50);
      tcgen05_fence_after();
#pragma unroll
      for (int pr = 0; pr < 3; ++pr) {
        constexpr int kTp[3] = {1, 0, 0}, kTu[3] = {0, 1, 0};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_ts(tmem + kTmO + 16 * kk, tmem + kTmG + 32 * kTu[pr] + 8 * kk,
                      umma_desc_k_sw128(sb + M::kP + (2 * ph + kTp[pr]) * M::kAtom + 2048 * kk + 32 * kk),
                      chunk_idesc(64 - 16 * kk, false), pr + kk > 0);
      }
      umma_commit(bar(kOaDone));
      if (c + 2 < nc) {
        wait(bar(kOaDone), ph, 51);
        scores(c + 2);
      }
    }
    // Nothing is in flight at the end of a run whose waits all came: each load and product has been waited for.
    // Otherwise wait for them here, with a limit.
    if (*abort) {
      for (int c = max(0, loaded - kStages); c < loaded; ++c)
        for (uint64_t w0 = globaltimer_ns(); !mbar_try_wait(full(c % kStages), (c / kStages) & 1);)
          if (globaltimer_ns() - w0 > 2000000000ull) break;
      spin_ns(1000000);  // products take microseconds
    } else if (nc > 0) {
      wait(bar(kOaDone), (nc - 1) & 1, 51);
    }
    }
    __syncwarp();
  }
  tcgen05_fence_before();
  __syncthreads();
  if (warp == kCtlWarp) {
    tcgen05_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int KA>
cudaError_t launch_chunk(const ChunkMaps& maps, const DeltaArgs& a, cudaStream_t st) {
  using M = ChunkSmem<KA>;
  const int smem = M::kTotal + 1024;
  auto kern = delta_chunk_kernel<KA>;
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  cudaFuncAttributes attr;
  const cudaError_t got = cudaFuncGetAttributes(&attr, kern);
  if (got != cudaSuccess) return got;
  if (attr.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;  // the register split would never complete
  const int slices = static_cast<int>((a.dv + 127) / 128);
  kern<<<static_cast<unsigned>(a.batch * a.H * slices), kChunkThreads, smem, st>>>(maps, a, slices);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chunk(const DeltaArgs& a, cudaStream_t st) {
  ChunkMaps m;
  const bool packed = a.cu != nullptr;
  auto map4 = [&](CUtensorMap* out, const void* base, int64_t n, int64_t heads, int64_t tok, int64_t seq,
                  uint32_t box, CUtensorMapSwizzle swz) {
    const uint64_t dims[4] = {uint64_t(n), uint64_t(heads), uint64_t(a.L), packed ? 1 : uint64_t(a.batch)};
    const uint64_t strides[3] = {uint64_t(n * 2), uint64_t(tok * 2), uint64_t(seq * 2)};
    const uint32_t b[4] = {box, 1, kC, 1};
    return encode_map(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, b, swz);
  };
  if (!map4(&m.q, a.q, a.dk, a.G, a.q_tok, a.q_seq, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !map4(&m.k, a.k, a.dk, a.G, a.k_tok, a.k_seq, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !map4(&m.v, a.v, a.dv, a.H, a.v_tok, a.v_seq, 128, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  return a.dk > 64 ? launch_chunk<2>(m, a, st) : launch_chunk<1>(m, a, st);
}

}  // namespace ssm
