// delta_chunk.cu -- the gated delta rule over whole sequences, 64 tokens at a
// time on the tensor cores (sm_100a).
//
// With G_i the running sum of g within a chunk, S the state before it and the
// keys k_i as rows of K, the chunk's updates u_i (rows of U) satisfy
//
//   (I + A) U = diag(beta) (V - diag(e^G) K S^T),
//   A_ij = beta_i e^{G_i - G_j} k_i.k_j   (j < i),
//
// so with T = (I + A)^-1 diag(beta), which does not depend on S, a chunk is
// four products around the state:
//
//   Y = K S^T,  R = V - diag(e^G) Y,  U = T R,
//   O = scale (diag(e^G) Q S^T + (Q K^T * e^{G_i - G_j}, j <= i) U),
//   S <- e^{G_C} S + sum_j e^{G_C - G_j} u_j k_j^T.
//
// Two kernels. What does not depend on S (T, the masked scores and the decay
// factors) is formed for all chunks at once by delta_prep_kernel and left in
// the workspace as the operand tiles that the second kernel's products read
// (26 KB per chunk and head). delta_chain_kernel then walks the chunks of a
// sequence. (One kernel with warps that prepare the next chunk beside those
// that walk took 10.9 us a chunk: the preparation alone is 2/3 of the
// instructions, and waits for nothing but the walk's place on the SM.)
//
// The walk. Transposed, with the 128 rows of S (a slice of d_value) as the 128
// lanes of tensor memory, every left operand (S, R, U) is an accumulator read
// back, scaled and split in registers, and stored to tensor memory as the next
// product's A operand: the state never leaves the SM, and shared memory holds
// only the right operands (K, Q, T and the scores, by TMA).
//
// Precision. q, k and v are bf16 and enter exactly; the key norms, decays and
// beta are fp32 factors of rows and columns, never folded into a bf16 operand.
// S, R, U and T are fp32 and go to the tensor cores as three bf16 terms (their
// sum is exact), as many products as pairs of terms above 2^-24. Before that,
// T's blocks beyond 8 x 8 are products of two tf32 terms an operand, which hold
// all but one bit of it. The tensor core adds into fp32 accumulators with
// truncation, so the state itself is added up in fp32 registers, and the
// accumulators hold one chunk's contribution at a time. (State against float64
// after 2048 tokens: 1.2e-7 of its norm; of one key throughout: 3.3e-6.)
// Only the output's own product takes fewer: two terms of the scores and of U,
// without the product of the two second ones, and two of S: 2^-17.3 of the
// output's RMS before its rounding to bf16 (2^-9), so that one output in 230
// rounds to the neighbour of what float64 rounds to (token by token one in
// 9000). Third terms would need 5 KB more an image, for which the stages of a
// pair leave no room, and columns of tensor memory, which is full.
//
// Values that are not finite: a product with a zero would spread them to tokens
// before theirs. Those of a token's k, g and beta (found by the prep) and of v
// (found while the walk waits for a product) are taken out of the operands; the
// state gets a NaN for them, and the outputs are NaN from the first such token
// on. A state that is not finite makes its row's outputs so by itself. Scores
// that are not finite touch their token alone, but where two heads share a walk
// they would meet the zeros in the other's rows, and are taken out too.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "delta_internal.h"
#include "delta_ptx.cuh"
#include "ssm.h"
#include "ssm_internal.h"
#include "ssm_math.cuh"
#include "tma_map.cuh"

namespace ssm {
namespace {

constexpr int kC = kDeltaChunk;   // tokens of a chunk
constexpr int kAtom = kC * 128;   // 64 rows of 64 bf16: one swizzled operand atom

// What the walk needs of a chunk and head, as the prep kernel leaves it: T in
// three terms and the scores in two, each as four panels of 16 columns j (the
// K of one MMA) and the rows i from 16 kk on, K-major without swizzle (8 rows
// x 16 bytes contiguous, the two halves of a panel's columns 128 bytes apart,
// 8-row groups 256 bytes apart); then the factors.
constexpr int kPanelTerm = (64 + 48 + 32 + 16) * 32;  // 5120 bytes of one term
__host__ __device__ constexpr int panel_off(int kk) { return 32 * (64 * kk - 8 * kk * (kk - 1)); }
struct Coef {
  float neg[kC]; // -e^{G_j} / |k_j|: scales Y
  float ec[kC];  // e^{G_C - G_j} / |k_j|, 0 behind the sequence: scales U into the state
  float oq[kC];  // scale e^{G_i} / |q_i|: scales Q S^T
  float decay;   // e^{G_C}
  uint32_t bad[2];  // bit j: token j's k, g or beta is not finite
  float pad;
};
constexpr int kImgP = 3 * kPanelTerm, kImgCoef = 5 * kPanelTerm;
constexpr int kImgBytes = kImgCoef + static_cast<int>(sizeof(Coef));
constexpr int kImgStride = (kImgBytes + 127) / 128 * 128;
static_assert(panel_off(1) == 2048 && panel_off(3) == 4608 && kImgBytes % 16 == 0 && kImgBytes + 8 <= kImgStride, "panel layout");

// 16-byte piece of row i, columns 8 j8 .. 8 j8 + 7 within a term's panels.
__device__ __forceinline__ int panel_piece(int i, int j8) {
  const int kk = j8 >> 1, r = i - 16 * kk;
  return panel_off(kk) + (r >> 3) * 256 + (j8 & 1) * 128 + (r & 7) * 16;
}

// Sequence s in rows: first row and length, in the packed buffer or on its own.
struct Span {
  int t0, len, seq;
};
__device__ __forceinline__ Span span_of(const DeltaArgs& a, int s) {
  if (!a.cu) return {0, static_cast<int>(a.L), s};
  const int T = static_cast<int>(a.L);
  const int t0 = min(max(a.cu[s], 0), T);
  return {t0, min(max(a.cu[s + 1], t0), T) - t0, 0};
}
// The first workspace slot of sequence s (a slot per chunk and head): chunks
// of sequences that follow one another in the buffer never share one.
__device__ __forceinline__ int64_t slot_of(const DeltaArgs& a, int s, int t0) {
  return a.cu ? t0 / kC + s : static_cast<int64_t>(s) * ((a.L + kC - 1) / kC);
}

__host__ __device__ constexpr uint32_t chunk_idesc(int n, bool b_mn_major) {  // bf16 x bf16 -> fp32, M = 128
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn_major ? (1u << 16) : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (8u << 24);
}
// Descriptor of a panel: K-major, no swizzle, 128 bytes between the halves of K, 256 between 8-row groups.
__device__ __forceinline__ uint64_t panel_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128u >> 4) << 16) |
         (static_cast<uint64_t>(256u >> 4) << 32) | (static_cast<uint64_t>(1u) << 46);
}
__device__ __forceinline__ uint64_t desc_add(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// A wait that all threads of a warp make together. Once any wait of the CTA
// has run out, the flag lets the others through: every loop ends, on memory
// of its own, and the error word tells the host.
struct Waiter {
  volatile int* abort;
  int* err;
  __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity, int code) const {
    if (mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
      if (*abort) return;
      if (globaltimer_ns() - t0 > 2000000000ull) {
        *abort = 1;
        if (err) atomicExch(err, code);
        return;
      }
    }
  }
};

// bf16 in the low half of w, as a float: times 65536 on the FMA pipe. The
// factor comes from memory (2^16, kept from the compiler), since a shift would
// go to the integer pipe, which the walk's conversions fill.
struct Shifter {
  uint32_t by;
  __device__ __forceinline__ float low(uint32_t w) const { return __uint_as_float(w * by); }
};
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// A pair of values as three packed bf16 pairs whose sum is exact: each rounding
// leaves at most 16, then 8 bits of the significand. Five integer-pipe
// instructions a pair; with masks and byte permutes instead of the conversions
// and the product, seven.
__device__ __forceinline__ void split3(const Shifter& sh, uint64_t x, uint32_t& h, uint32_t& m, uint32_t& l) {
  const uint64_t minus = pk2(-1.0f, -1.0f);
  float a, b;
  upk2(x, a, b);
  h = pack_bf16(a, b);
  const uint64_t r = ffma2(pk2(sh.low(h), high_bf16(h)), minus, x);
  upk2(r, a, b);
  m = pack_bf16(a, b);
  const uint64_t s = ffma2(pk2(sh.low(m), high_bf16(m)), minus, r);
  upk2(s, a, b);
  l = pack_bf16(a, b);
}
// As two: 2^-18 of the value is left out.
__device__ __forceinline__ void split2(const Shifter& sh, uint64_t x, uint32_t& h, uint32_t& m) {
  float a, b;
  upk2(x, a, b);
  h = pack_bf16(a, b);
  const uint64_t r = ffma2(pk2(sh.low(h), high_bf16(h)), pk2(-1.0f, -1.0f), x);
  upk2(r, a, b);
  m = pack_bf16(a, b);
}
__device__ __forceinline__ uint64_t pk2u(uint32_t a, uint32_t b) { return pk2(__uint_as_float(a), __uint_as_float(b)); }

// 16 values of a row as three terms at columns col + t * stride of A-operand tensor memory.
__device__ __forceinline__ void store_split3(const Shifter& sh, uint32_t col, uint32_t stride, const uint64_t (&x)[8]) {
  uint32_t h[8], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) split3(sh, x[i], h[i], m[i], l[i]);
  tmem_st_x8(col, h);
  tmem_st_x8(col + stride, m);
  tmem_st_x8(col + 2 * stride, l);
}

// a b + c of two bf16 each.
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

__device__ __forceinline__ int sw128(int r, int j) { return r * 128 + ((j ^ (r & 7)) << 4); }

// Bit i set where value i of the 16 is not finite. Nearly always none in the
// whole warp, which one vote tells without a divergent branch.
__device__ __forceinline__ uint32_t not_finite(const uint64_t (&x)[8]) {
  uint64_t s0 = 0, s1 = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) s0 = ffma2(x[i], 0ull, s0), s1 = ffma2(x[i + 1], 0ull, s1);
  float a, b;
  upk2(fadd2(s0, s1), a, b);
  uint32_t bits = 0;
  if (__any_sync(0xffffffffu, !(a + b == 0.0f))) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      upk2(x[i], a, b);
      bits |= (fabsf(a) <= 3.4028235e38f ? 0u : 1u << (2 * i)) | (fabsf(b) <= 3.4028235e38f ? 0u : 2u << (2 * i));
    }
  }
  return bits;
}
// Puts `to` in the place of the marked ones.
__device__ __forceinline__ void replace_marked(uint64_t (&x)[8], uint32_t marks, float to) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    upk2(x[i], a, b);
    x[i] = pk2(marks >> (2 * i) & 1 ? to : a, marks >> (2 * i + 1) & 1 ? to : b);
  }
}

struct ChunkMaps {
  CUtensorMap q, k, v, out;
};

// --------------------------------------------------------------- segments ---
// A long sequence with few heads leaves most SMs idle, so it may be walked in
// segments at once. The state is linear in the one before it: S_{p+1} = S_p M_p
// + H_p, H_p a segment's walk from zero and M_p its walk of the identity without
// values. Pass 1 (states only, OUT = false) forms both for every segment that
// needs them, segment 0 from the state given; delta_join_kernel folds them into
// the segments' first states; pass 2 walks all segments. More than twice the
// work of one walk, on more than twice the SMs.
//
// Sequences of one length are cut on the host (count segments of per chunks).
// The lengths of packed ones are known on the device alone: there a block of the
// prep works out the cut (delta_cut) and leaves it in the workspace. (With the
// code for it in the walk itself, the walk has to spill: 13% slower.)
struct Cut;
struct Segments {
  int count, per;   // 1: one walk
  Cut* cut;         // packed: cut on the device
  int items;        // walks of this launch, where the host knows them
  float* S;         // [segment][head][d_value][d_key]: the segments' first states
  float* M;         // [segment][head][d_key][d_key]
  uint32_t* next;   // walks (beyond one per block) or shares handed out: pass 1's, pass 2's
  uint32_t* flags;  // shares: [share] the last pass in which its first walk's state was left for the next share
  int job, share;   // shares: chunks of a walk, and a block's part of the line of all walks; job 0: whole walks
  int walkers;      // walks of one segment of a sequence: its heads times the slices of d_value, or pairs of heads
  int sms;
  int room;         // packed: segments that S and M hold
};

// What the choices between whole walks, segments and shares count with, in chunks of a walk (3.4 us), as measured.
constexpr double kWalkStart = 2.5;   // starting a walk
constexpr double kStatesOnly = 0.85; // a chunk of pass 1, which forms no outputs
constexpr double kMoreLaunches = 3.0;  // of pass 1 and the join

// Shares. Walks of one length, more than the SMs, are not handed out whole (320
// walks on 148 SMs would take three rounds, not 2.2) but laid end to end on a
// line that is cut into equal shares, one a block. A walk across a cut begins in
// the share before it and ends in the one behind: a block starts with the last
// walk of its share and ends with the first, so that its first item waits for
// nothing, and its last for the first item of the share before, begun long ago.
// Shares are handed out in order: what a block waits for is always running.
// (8 sequences of 64 chunks, 80 heads in pairs: 723 us whole, 588 so; 32 heads of
// 512 chunks in segments: both passes 937 and 827.) SHARE is a kernel of its own:
// one that did both ways would walk whole ones 8% slower.
constexpr int kStartChunks = 2;  // kWalkStart, in whole chunks: the line is counted in them
constexpr int kShareLeast = 16;  // chunks of a walk that may be cut
// The cut before share r: chunk `a` of walk `item`, on its first or last chunk where few would be left of one side.
__device__ __forceinline__ void share_cut(const Segments& sg, int r, int& item, int& a) {
  const int64_t x = static_cast<int64_t>(r) * sg.share;
  const int width = sg.job + kStartChunks;
  item = static_cast<int>(x / width);
  a = static_cast<int>(x - static_cast<int64_t>(item) * width) - kStartChunks;
  if (a < 4) a = 0;
  if (a > sg.job - 4) a = sg.job;
}
// One thread: the item of share r before `item` (-1: its first); its chunks are c0 .. c1 - 1. -1 where there is none.
__device__ __forceinline__ int3 share_item(const Segments& sg, int r, int items, int item) {
  int i0, a0, i1, a1;
  share_cut(sg, r, i0, a0);
  share_cut(sg, r + 1, i1, a1);
  int c0 = 0, c1 = sg.job;
  if (item < 0 && a1 > 0 && i1 < items) item = i1, c1 = a1;
  else item = min(item < 0 ? i1 : item, items) - 1;
  if (item == i0) c0 = a0;
  if (item < i0 || c0 >= sg.job) item = -1;
  return make_int3(item, c0, c1);
}

constexpr int kCutSeqs = 256;  // most packed sequences that are cut
constexpr int kCutLeast = 8;   // least chunks of a segment of theirs
// Sequences in the order of their lengths, the longest first, so that the last walks handed out are short. For each
// place: the sequence, and the segments before it (all; those pass 1 walks from a state; those it walks from the
// identity). `per`: chunks of a segment.
struct Cut {
  int all[kCutSeqs + 1], walk[kCutSeqs + 1], ident[kCutSeqs + 1];
  int chunks[kCutSeqs], seq[kCutSeqs];
  int per;
};

// Time of a packed batch in chunks, cut into segments of `per`: the longest walk or the work of all over the SMs,
// whichever is more, for both passes; launches as in choose_segments, and for each segment of the longest the join
// (`join`: its blocks for one sequence, over the SMs). 3e38 where the cut sequences have more segments than there is
// room for: offsets that do not ascend name rows twice.
__device__ __forceinline__ float cut_cost(const Cut& c, int n, int per, int longest, int heads, int walkers, int sms,
                                         int room, float join) {
  float w1 = 0.0f, w2 = 0.0f;
  int used = 0;
  for (int s = 0; s < n; ++s) {
    const int segs = (c.chunks[s] + per - 1) / per;
    w2 += static_cast<float>(c.chunks[s] * walkers);
    if (segs > 1) {
      w1 += static_cast<float>(((segs - 1) * walkers + (segs - 2) * heads) * per);
      used += segs;
    }
  }
  if (used > room) return 3.0e38f;
  const float scale = 1.0f / static_cast<float>(sms), len = static_cast<float>(per);
  constexpr float start = kWalkStart, more = kMoreLaunches, states = kStatesOnly;
  const float second = fmaxf(len, w2 * scale + 0.3f * len) + start;
  if (per >= longest) return second;
  return states * fmaxf(len, w1 * scale + 0.3f * len) + start + second + more +
         (0.4f + 0.7f * join) * static_cast<float>((longest + per - 1) / per - 2);
}

// All threads of a block, with `c` in shared memory; ends with a barrier.
__device__ __forceinline__ void delta_cut(const DeltaArgs& a, int walkers, int sms, int room, Cut& c) {
  const int n = static_cast<int>(a.batch), tid = threadIdx.x;
  for (int s = tid; s < n; s += blockDim.x) c.all[s] = (span_of(a, s).len + kC - 1) / kC;
  __syncthreads();
  for (int s = tid; s < n; s += blockDim.x) {
    int place = 0;
    for (int i = 0; i < n; ++i) place += c.all[i] > c.all[s] || (c.all[i] == c.all[s] && i < s);
    c.chunks[place] = c.all[s], c.seq[place] = s;
  }
  __syncthreads();
  if (tid < 32) {  // lane l: the longest in l + 1 segments
    const int longest = max(1, c.chunks[0]);
    const int per = (longest + tid) / (tid + 1);
    const float join = static_cast<float>(static_cast<int>(a.H) * ((static_cast<int>(a.dv) + 15) / 16)) / static_cast<float>(sms);
    float cost = cut_cost(c, n, per, longest, static_cast<int>(a.H), walkers, sms, room, join);
    if (tid > 0) cost = per < kCutLeast ? 3.0e38f : cost * 1.05f;
    int best = tid;
    for (int m = 16; m > 0; m >>= 1) {
      const float oc = __shfl_xor_sync(0xffffffffu, cost, m);
      const int ob = __shfl_xor_sync(0xffffffffu, best, m);
      if (oc < cost || (oc == cost && ob < best)) cost = oc, best = ob;
    }
    if (tid == 0) c.per = (longest + best) / (best + 1);
  }
  __syncthreads();
  if (tid < 3) {
    int* out = tid == 0 ? c.all : tid == 1 ? c.walk : c.ident;
    int sum = 0;
    for (int s = 0; s < n; ++s) {
      out[s] = sum;
      sum += max(max(1, (c.chunks[s] + c.per - 1) / c.per) - tid, 0);
    }
    out[n] = sum;
  }
  __syncthreads();
}
// `from` to `to`, by all threads of a block; no barrier.
__device__ __forceinline__ void copy_cut(const Cut* from, Cut* to) {
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(Cut) / 4); i += blockDim.x)
    reinterpret_cast<int*>(to)[i] = reinterpret_cast<const int*>(from)[i];
}
// The place that item i of a running sum belongs to.
__device__ __forceinline__ int cut_find(const int* sums, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (sums[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ------------------------------------------------------------------- prep ---
// One CTA of 4 warps per chunk and up to kPrepHeads heads of one key group:
// fewer where all of them still fit the SMs at once (64 tokens of 80 heads with
// one group: 20 us, with four heads a block 29).
// Thread pt owns row pt of the 128 x 64 product [K; Q] K^T (one
// set of MMAs per CTA; tensor memory keeps it for all its heads): rows 0-63
// give A, rows 64-127 the scores.
//
// Decays. Within a row's own 16 columns each e^{G_i - G_j} is an exponential;
// before them it is e^{G_i - G_m} e^{G_m - G_j}, m the token before the row's
// 16: two factors that the row and the column bring along, neither above 1
// where g <= 0, so that a product underflows only where the decay does.
//
// The inverse of I + A: 8 x 8 diagonal blocks by substitution (two a warp, a
// column per lane), then the block below a pair of inverted ones, T21 = -T22
// (A21 T11), for 8, 16 and 32 rows. (16 x 16 blocks by substitution, whose rows
// every lane reads: 18 us more for 8 sequences of 64 chunks and 80 heads.)
// Shared memory's bandwidth (0.67 of it used) and instruction issue (0.63) bound
// the kernel: 217 us for 8 sequences of 32 chunks and 80 heads, 500 MB; 420 for
// twice the chunks.
constexpr int kPrepHeads = 4;
constexpr int kALd = 68;  // floats between rows of A (16-byte rows, conflict-free columns)

template <int KA>  // 64-column atoms of d_key
struct PrepSmem {
  // from 0, per atom: K, then Q; A in their place once their product and norms are formed
  static constexpr int kA = 0;
  static constexpr int kAEnd = kC * kALd * 4;
  static constexpr int kVec = KA * 2 * kAtom > kAEnd ? KA * 2 * kAtom : kAEnd;  // per head: Ghi, Glo, beta [64]
  static constexpr int kRk = kVec + kPrepHeads * 3 * kC * 4;  // 1 / |k| [64]
  static constexpr int kCf = kRk + kC * 4;            // column factors [3][64]
  // full, done, TMEM address, abort flag, tokens not finite: behind block row 1's 16 factors, where a row has room,
  // so that six blocks fit an SM
  static constexpr int kBar = kCf + 64;
  static constexpr int kTotal = kCf + 3 * kC * 4;
};

// A fp32 value as two tf32 ones: 11 bits, rounded, and the rest (12 bits and a sign, of which the product reads 11).
// Where keys are alike the entries of A are too, and what a product leaves out adds up over all tokens of a chunk: with
// the first cut off, not rounded, and three products of terms, the state of 128 tokens of one key and beta = 1 was
// 2.2e-5 off, so 4.1e-6, at 8 x 4096 tokens of 80 heads for 2.7% of the time (in fp32 FMAs 0.6e-6).
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// One warp: the 16 x 8 NT block D = L R, L 16 x K and R K x 8 NT in As (row
// stride kALd), K a multiple of 8; two tf32 terms each, all four products.
// 16-row blocks are far below the 128 rows of a
// tcgen05 product, and in fp32 FMAs their operands' loads take the SM's whole
// shared-memory bandwidth (4096 chunks and heads: 69 us with them when these
// took 59).
template <int K, int NT>
__device__ __forceinline__ void block_product(const float* L, const float* R, int lane, float (&c)[NT][4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[j][e] = 0.0f;
#pragma unroll
  for (int k = 0; k < K; k += 8) {
    uint32_t ah[4], al[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split_tf32(L[(g + 8 * (e & 1)) * kALd + k + t + 4 * (e >> 1)], ah[e], al[e]);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      uint32_t bh[2], bl[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) split_tf32(R[(k + t + 4 * e) * kALd + 8 * j + g], bh[e], bl[e]);
      mma_tf32(c[j], al, bl);
      mma_tf32(c[j], al, bh);
      mma_tf32(c[j], ah, bl);
      mma_tf32(c[j], ah, bh);
    }
  }
}
// Stores it, times sign.
template <int NT>
__device__ __forceinline__ void block_store(float* D, int lane, const float (&c)[NT][4], float sign) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    *reinterpret_cast<float2*>(D + g * kALd + 8 * j + 2 * t) = make_float2(sign * c[j][0], sign * c[j][1]);
    *reinterpret_cast<float2*>(D + (g + 8) * kALd + 8 * j + 2 * t) = make_float2(sign * c[j][2], sign * c[j][3]);
  }
}

template <int KA, bool PAIR>
__global__ void __launch_bounds__(128, 6)
    delta_prep_kernel(const __grid_constant__ ChunkMaps maps, const DeltaArgs a, unsigned char* img0, int set_heads,
                      const Segments sg) {
  using M = PrepSmem<KA>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sb = smem_u32(smem);
  const int pt = threadIdx.x, lane = pt & 31;
  const Shifter sh{a.two16};
  const int warp = __shfl_sync(0xffffffffu, pt >> 5, 0);
  const int rep = static_cast<int>(a.H / a.G);
  if (blockIdx.x == 0) {
    if (pt < 2) sg.next[pt] = 0u;  // the walks handed out, pass 1 and 2
    if (sg.job)
      for (int i = pt; i < sg.sms; i += 128) sg.flags[i] = 0u;
  }
  int block = static_cast<int>(blockIdx.x);
  if (sg.cut && block-- == 0) {
    delta_cut(a, sg.walkers, sg.sms, sg.room, *reinterpret_cast<Cut*>(smem));
    copy_cut(reinterpret_cast<const Cut*>(smem), sg.cut);
    return;
  }
  const int head_sets = (rep + set_heads - 1) / set_heads, set = block % head_sets;
  const int64_t gslot = block / head_sets;
  const int grp = static_cast<int>(gslot % a.G);
  const int64_t slot = gslot / a.G;
  // the sequence and chunk of this slot
  int s, c;
  if (a.cu) {
    int lo = 0, hi = static_cast<int>(a.batch) - 1;  // the last sequence whose first slot is not behind this one
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (slot_of(a, mid, span_of(a, mid).t0) <= slot) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
    c = static_cast<int>(slot - slot_of(a, s, span_of(a, s).t0));
  } else {
    const int nc = static_cast<int>((a.L + kC - 1) / kC);
    s = static_cast<int>(slot / nc), c = static_cast<int>(slot % nc);
  }
  const Span sp = span_of(a, s);
  if (c < 0 || kC * c >= sp.len) return;
  const int n = min(kC, sp.len - kC * c), tok = sp.t0 + kC * c;

  const uint32_t full = sb + M::kBar, done = sb + M::kBar + 8;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + M::kBar + 20);
  const Waiter wait{abort, a.err};
  if (pt == 0) {
    mbar_init(full, 1);
    mbar_init(done, 1);
    *abort = 0;
    mbar_fence_init();
    mbar_arrive_expect_tx(full, KA * 2 * kAtom);
#pragma unroll
    for (int t = 0; t < KA; ++t) {
      tma_load_4d(sb + t * 2 * kAtom, &maps.k, 64 * t, grp, tok, sp.seq, full);
      tma_load_4d(sb + t * 2 * kAtom + kAtom, &maps.q, 64 * t, grp, tok, sp.seq, full);
    }
  }
  if (warp == 0) {
    __syncwarp();
    tmem_alloc(sb + M::kBar + 16, 64);
    tmem_relinquish();
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + M::kBar + 16);
  // The walk may set up; it waits for this grid before it reads the workspace. Not before this block has its tensor
  // memory: a walk's block takes all of an SM's and keeps it while it waits.
  griddep_launch_dependents();
  if (pt == 96) {
    wait(full, 0, 31);
#pragma unroll
    for (int t = 0; t < KA; ++t)
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const uint64_t d = umma_desc_k_sw128(sb + t * 2 * kAtom + 32 * kk);
        umma_f16_ss(tmem, d, d, chunk_idesc(64, false), t + kk > 0);
      }
    umma_commit(done);
  }
  __syncwarp();

  const int i = pt & 63;  // this row's token
  const bool is_q = pt >= 64;
  float* As = reinterpret_cast<float*>(smem + M::kA);
  float* rk = reinterpret_cast<float*>(smem + M::kRk);
  float* cfac = reinterpret_cast<float*>(smem + M::kCf);
  uint32_t* bad_tokens = reinterpret_cast<uint32_t*>(smem + M::kBar + 24);
  const int h0 = grp * rep + set * set_heads, nh = min(set_heads, rep - set * set_heads);
  // Warp w: head h0 + w. Running sums of g in log2 units and fp64, kept as two
  // floats, so that differences of far sums stay exact; a decay below 2^-256 is 0 anyway.
  if (warp < nh) {
    float* vec = reinterpret_cast<float*>(smem + M::kVec) + warp * 3 * kC;
    const int64_t gb = static_cast<int64_t>(sp.seq) * a.gb_seq + (static_cast<int64_t>(tok) + 2 * lane) * a.gb_tok + h0 + warp;
    const bool in0 = 2 * lane < n, in1 = 2 * lane + 1 < n;
    const float r0 = in0 ? a.g[gb] : 0.0f, r1 = in1 ? a.g[gb + a.gb_tok] : 0.0f;
    const float b0 = in0 ? a.beta[gb] : 0.0f, b1 = in1 ? a.beta[gb + a.gb_tok] : 0.0f;
    auto lg = [](float g) {
      const double v = static_cast<double>(g) * 1.4426950408889634;
      return v < -256.0 ? -256.0 : v;
    };
    const double g0 = lg(r0), g1 = lg(r1);
    double sum = g0 + g1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    const double before = __shfl_up_sync(0xffffffffu, sum, 1);
    const double first = (lane ? before : 0.0) + g0;  // not sum - g1: g1 may not be finite
    const float f0 = static_cast<float>(first), f1 = static_cast<float>(sum);
    *reinterpret_cast<float2*>(vec + 2 * lane) = make_float2(f0, f1);
    *reinterpret_cast<float2*>(vec + kC + 2 * lane) =
        make_float2(static_cast<float>(first - f0), static_cast<float>(sum - f1));
    *reinterpret_cast<float2*>(vec + 2 * kC + 2 * lane) = make_float2(b0, b1);
  }
  wait(full, 0, 31);
  float rn = 1.0f;  // 1 / |row|
  bool k_bad = false;
  if (a.l2norm || !is_q) {
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 1
    for (int t = 0; t < KA; ++t) {
      const unsigned char* base = smem + t * 2 * kAtom + (is_q ? kAtom : 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 w = *reinterpret_cast<const uint4*>(base + sw128(i, j));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = __uint_as_float(u[e] << 16), hi = __uint_as_float(u[e] & 0xffff0000u);
          s0 = fmaf(lo, lo, s0), s1 = fmaf(hi, hi, s1);
        }
      }
    }
    k_bad = !(s0 + s1 <= 3.4028235e38f);
    if (a.l2norm) rn = rsqrtf(s0 + s1 + kL2Eps);
    if (is_q) rn = fmaf(s0 + s1, 0.0f, rn);  // NaN where the squares overflow
  }
  if (!is_q) rk[i] = rn;
  wait(done, 0, 32);
  tcgen05_fence_after();
  __syncthreads();

  const uint32_t tmw = tmem + (static_cast<uint32_t>(32 * warp) << 16);
  const int b0 = 2 * (warp & 1), bi = i >> 4;  // 16-row blocks: this warp's first, this row's
  const bool upper = lane < 16;                // the row is in the warp's first block
#pragma unroll 1
  for (int hh = 0; hh < nh; ++hh) {
    const float* Ghi = reinterpret_cast<float*>(smem + M::kVec) + hh * 3 * kC;
    const float* Glo = Ghi + kC;
    const float* beta = Glo + kC;
    unsigned char* img = img0 + (slot * a.H + h0 + hh) * kImgStride;
    const float Gi = Ghi[i], Gl = Glo[i];
    Coef* cf = reinterpret_cast<Coef*>(img + kImgCoef);
    const float eg = ex2_approx(Gi + Gl);
    if (is_q) {
      cf->oq[i] = eg * (rn * a.scale);
    } else {
      cf->neg[i] = -eg * rn;
      cf->ec[i] = i < n ? ex2_approx((Ghi[kC - 1] - Gi) + (Glo[kC - 1] - Gl)) * rn : 0.0f;
      if (i == kC - 1) cf->decay = eg;
      const bool bad = i < n && (k_bad || !(fabsf(Gi) <= 3.4028235e38f) || !(fabsf(beta[i]) <= 3.4028235e38f));
      const uint32_t bits = __ballot_sync(0xffffffffu, bad);
      if (lane == 0) cf->bad[warp] = bits, bad_tokens[warp] = bits;
    }
    {  // column factors of block row b, columns j < 16 b
      const int b = pt < 48 ? 3 : pt < 96 ? 2 : 1, j = pt < 48 ? pt : pt < 96 ? pt - 64 : pt - 96;
      if (j >= 0 && j < 16 * b) {
        const int m = 16 * b - 1;
        cfac[(b - 1) * kC + j] = ex2_approx((Ghi[m] - Ghi[j]) + (Glo[m] - Glo[j])) * rk[j];
      }
    }
    __syncthreads();
    // Tokens that are not finite stay out of A: their rows and columns would spread to tokens before them.
    const uint64_t bad_mask = bad_tokens[0] | static_cast<uint64_t>(bad_tokens[1]) << 32;
    const float lead = is_q ? rn * a.scale : rn * beta[i];
    const float rfac = bi > 0 ? lead * ex2_approx((Gi - Ghi[16 * bi - 1]) + (Gl - Glo[16 * bi - 1])) : 0.0f;
    uint32_t marks = 0u;  // +-0 twice while this row's scores are finite
    // 8 values of this row from column j on: to A, or to the scores
    auto put = [&](int j, float (&f)[8], bool mine) {
      if (n < kC && !is_q && i >= n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.0f;
      }
      if (bad_mask && !is_q) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((bad_mask >> i | bad_mask >> (j + e)) & 1) f[e] = 0.0f;
      }
      if (mine) {
        if (is_q) {
          uint32_t hi[4], mi[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) split2(sh, pk2(f[2 * z], f[2 * z + 1]), hi[z], mi[z]);
          if constexpr (PAIR) {
#pragma unroll
            for (int z = 0; z < 4; ++z) marks = fma_bf16x2(hi[z], 0u, marks);
          }
          unsigned char* p = img + kImgP + panel_piece(i, j >> 3);
          *reinterpret_cast<uint4*>(p) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(p + kPanelTerm) = make_uint4(mi[0], mi[1], mi[2], mi[3]);
        } else {
          float4* p = reinterpret_cast<float4*>(As + i * kALd + j);
          p[0] = make_float4(f[0], f[1], f[2], f[3]);
          p[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
      __syncwarp();
    };
    auto before = [&](int j, const uint32_t (&d)[8], bool mine) {  // columns before the row's block
      const float4* cp = reinterpret_cast<const float4*>(cfac + (bi > 0 ? bi - 1 : 0) * kC + j);
      const float4 c0 = cp[0], c1 = cp[1];
      const float cv[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = rfac * cv[e] * __uint_as_float(d[e]);
      put(j, f, mine);
    };
#pragma unroll 1
    for (int j = 0; j < 16 * b0; j += 8) {
      uint32_t d[8];
      tmem_ld_x8(tmw + j, d);
      tmem_ld_wait();
      before(j, d, true);
    }
#pragma unroll 1
    for (int jj = 0; jj < 16; jj += 8) {
      uint32_t d[8], e2[8];
      tmem_ld_x8(tmw + 16 * b0 + jj, d);
      tmem_ld_x8(tmw + 16 * b0 + 16 + jj, e2);
      tmem_ld_wait();
      before(16 * b0 + jj, d, !upper);
      const int j = 16 * bi + jj, last = is_q ? i : i - 1;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 gh = *reinterpret_cast<const float4*>(Ghi + j + e), gl = *reinterpret_cast<const float4*>(Glo + j + e);
        const float4 rj = *reinterpret_cast<const float4*>(rk + j + e);
        const float ghs[4] = {gh.x, gh.y, gh.z, gh.w}, gls[4] = {gl.x, gl.y, gl.z, gl.w};
        const float rjs[4] = {rj.x, rj.y, rj.z, rj.w};
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const float w = ex2_approx((Gi - ghs[z]) + (Gl - gls[z])) * rjs[z];
          f[e + z] = j + e + z <= last ? lead * w * __uint_as_float(upper ? d[e + z] : e2[e + z]) : 0.0f;
        }
      }
      put(j, f, true);
    }
    if constexpr (PAIR) {
      // Scores that are not finite in bf16 (decays above 1 or NaN) would meet zeros in the other head's rows: zeros
      // take their place, and the row's output becomes NaN by its factor.
      if (is_q && (marks & 0x7fff7fffu)) {
        for (int j8 = 0; 8 * j8 <= (i | 15); ++j8) {
          unsigned char* p = img + kImgP + panel_piece(i, j8);
          *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(p + kPanelTerm) = make_uint4(0u, 0u, 0u, 0u);
        }
        cf->oq[i] = __uint_as_float(0x7fffffffu);
      }
    }
    __syncthreads();
    {  // rows 16 w .. of warp w: two 8 x 8 blocks, a column per lane (twice), then the block between them
      const int o = 16 * warp, blk = o + (lane & 8), col = lane & 7;
      const float* Ab = As + blk * (kALd + 1);
      float x[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        float acc[2] = {r == col ? 1.0f : 0.0f, 0.f};
#pragma unroll
        for (int k = 0; k < r; k += 4) {
          const float4 w = *reinterpret_cast<const float4*>(Ab + r * kALd + k);
          acc[0] = fmaf(-w.x, x[k], acc[0]);
          if (k + 1 < r) acc[1] = fmaf(-w.y, x[k + 1], acc[1]);
          if (k + 2 < r) acc[0] = fmaf(-w.z, x[k + 2], acc[0]);
          if (k + 3 < r) acc[1] = fmaf(-w.w, x[k + 3], acc[1]);
        }
        x[r] = acc[0] + acc[1];
      }
      __syncwarp();
      if (lane < 16) {
#pragma unroll
        for (int r = 0; r < 8; ++r) As[(blk + r) * kALd + blk + col] = x[r];
      }
      __syncwarp();
      const int g = lane >> 2, t = lane & 3;
      float* Ao = As + o * kALd + o;
      auto product8 = [&](const float* L, const float* R, float (&c)[4]) {  // 8 x 8 x 8 in the upper rows
        uint32_t ah[4] = {}, al[4] = {}, bh[2], bl[2];
        split_tf32(L[g * kALd + t], ah[0], al[0]);
        split_tf32(L[g * kALd + t + 4], ah[2], al[2]);
        split_tf32(R[t * kALd + g], bh[0], bl[0]);
        split_tf32(R[(t + 4) * kALd + g], bh[1], bl[1]);
        c[0] = c[1] = c[2] = c[3] = 0.0f;
        mma_tf32(c, al, bl);
        mma_tf32(c, al, bh);
        mma_tf32(c, ah, bl);
        mma_tf32(c, ah, bh);
      };
      float c[4];
      product8(Ao + 8 * kALd, Ao, c);
      *reinterpret_cast<float2*>(Ao + g * kALd + 8 + 2 * t) = make_float2(c[0], c[1]);
      __syncwarp();
      product8(Ao + 8 * kALd + 8, Ao + 8, c);
      __syncwarp();
      *reinterpret_cast<float2*>(Ao + (g + 8) * kALd + 2 * t) = make_float2(-c[0], -c[1]);
      *reinterpret_cast<float2*>(Ao + g * kALd + 8 + 2 * t) = make_float2(0.0f, 0.0f);
    }
    __syncthreads();
    auto pair_sync = [&]() {  // constant barrier ids: a variable one reserves all 16, and four blocks take an SM's 64
      if (warp < 2) named_bar_sync(1, 64);
      else named_bar_sync(2, 64);
    };
    {  // 16 -> 32: two pairs, two warps each; the unused block right of a pair's first holds A21 T11
      const int o = 32 * (warp >> 1), c0 = 8 * (warp & 1);
      float c[1][4];
      block_product<16, 1>(As + (o + 16) * kALd + o, As + o * kALd + o + c0, lane, c);
      block_store<1>(As + o * kALd + o + 16 + c0, lane, c, 1.0f);
      pair_sync();
      block_product<16, 1>(As + (o + 16) * kALd + o + 16, As + o * kALd + o + 16 + c0, lane, c);
      block_store<1>(As + (o + 16) * kALd + o + c0, lane, c, -1.0f);
      // that block is zero in T11 and T22, which the next products read
      pair_sync();
      const float zero[1][4] = {};
      block_store<1>(As + o * kALd + o + 16 + c0, lane, zero, 1.0f);
    }
    __syncthreads();
    {  // 32 -> 64: 16 x 16 of the block per warp
      const int r0 = 16 * (warp >> 1), c0 = 16 * (warp & 1);
      float c[2][4];
      block_product<32, 2>(As + (32 + r0) * kALd, As + c0, lane, c);
      block_store<2>(As + r0 * kALd + 32 + c0, lane, c, 1.0f);
      __syncthreads();
      block_product<32, 2>(As + (32 + r0) * kALd + 32, As + 32 + c0, lane, c);
      block_store<2>(As + (32 + r0) * kALd + c0, lane, c, -1.0f);
    }
    __syncthreads();
    // T = the inverse times beta by column, three terms; thread: a row, every other 8 columns
#pragma unroll 1
    for (int j8 = pt >> 6; 8 * j8 <= (i | 15); j8 += 2) {
      uint32_t hi[4], mi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const int j = 8 * j8 + e;
        const float4 w = *reinterpret_cast<const float4*>(As + i * kALd + j);
        const float4 b4 = *reinterpret_cast<const float4*>(beta + j);
        split3(sh, pk2(j <= i ? w.x * b4.x : 0.0f, j + 1 <= i ? w.y * b4.y : 0.0f), hi[e / 2], mi[e / 2], lo[e / 2]);
        split3(sh, pk2(j + 2 <= i ? w.z * b4.z : 0.0f, j + 3 <= i ? w.w * b4.w : 0.0f), hi[e / 2 + 1], mi[e / 2 + 1],
               lo[e / 2 + 1]);
      }
      unsigned char* p = img + panel_piece(i, j8);
      *reinterpret_cast<uint4*>(p) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(p + kPanelTerm) = make_uint4(mi[0], mi[1], mi[2], mi[3]);
      *reinterpret_cast<uint4*>(p + 2 * kPanelTerm) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    __syncthreads();
  }
  if (*abort && pt == 0) {  // a wait ran out: the loads and products end before the block does, with a limit
    const uint64_t w0 = globaltimer_ns();
    while (!mbar_try_wait(full, 0) && globaltimer_ns() - w0 < 2000000000ull) {
    }
    spin_ns(1000000);
  }
  __syncwarp();
  if (warp == 0) {
    tcgen05_fence_after();
    tmem_dealloc(tmem, 64);
  }
}

// ------------------------------------------------------------------- walk ---
// One CTA per (sequence, head, 128 rows of d_value), 17 warps:
//   warps 0-15  hold S (a thread: one row, a quarter of the key channels), form
//               the A operands between the products, and in their waits for
//               the products the outputs (a thread: one row, 16 tokens): Q S^T
//               is scaled where it lies, the scores' product adds to it there,
//               and the sum is rounded and stored a chunk later;
//   warp 16     one thread issues the loads (two chunks in flight) and every MMA.
// (Output warps of their own, 21 in all, leave 80 registers a thread: spills.)
//
// Bound by the chain through a chunk (state, Y, R, U, state), whose steps
// alternate between the tensor cores (0.46 of the time busy) and the warps'
// splits and scalings (issue 0.55): 3.4 us a chunk, 113 us for 2048 tokens.
constexpr int kStateWarps = 16, kCtlWarp = 16;
constexpr int kChainThreads = 32 * 17;
constexpr int kStages = 2;

// Tensor memory, 512 columns.
constexpr uint32_t kTmDelta = 0;  // the chunk's contribution to S; before it, R's three terms
constexpr uint32_t kTmS = 128;    // S's three terms: half h at 96 h; then U's scaled terms in the second half
constexpr uint32_t kTmY = 320;    // Y, then U
constexpr uint32_t kTmO = 384;    // Q S^T, then with the scores' product
constexpr uint32_t kTmU = 448;    // U's two output terms

template <int KA, bool PAIR>
struct ChainSmem {
  static constexpr int kImgs = PAIR ? 2 : 1;  // heads
  static constexpr int kOuts = PAIR ? 1 : 2;  // output tiles
  static constexpr int kKQ = KA * 2 * kAtom;  // per atom: K, then Q
  static constexpr int kV = kKQ;              // [token][128]
  static constexpr int kImg = kV + kC * 256;
  static constexpr int kStage = (kImg + kImgs * kImgStride + 1023) / 1024 * 1024;
  static constexpr int kOut = kStages * kStage;          // [token][128] bf16, kOuts chunks
  static constexpr int kBad = kOut + kOuts * kC * 256;   // int [4][128]
  static constexpr int kCut = kBad + 4 * 128 * 4;
  static constexpr int kBar = kCut + (static_cast<int>(sizeof(Cut)) + 15) / 16 * 16;
  static constexpr int kMisc = kBar + (kStages + 16) * 8;
  static constexpr int kTotal = kMisc + 64;  // TMEM address, abort flag, from 8 on the item (enum Plan)
  static_assert(kTotal + 1024 <= 232448, "227 KB of shared memory");
  static constexpr uint32_t kTx = static_cast<uint32_t>(kImg + kImgs * kImgBytes);
};

// A block's item, in shared memory: the walk (-1: none), its share, its chunks, and what it is a walk of. (In registers
// through the walk they spill.)
enum Plan { kItem, kShare, kFrom, kTo, kSeq, kHead, kSlice, kSeg, kCount, kFirstSeg, kIdent };
enum Bar {  // after the stages' full barriers; each completes once a chunk
  kSReady0, kSReady1, kSReady2, kSReady3, kYDone, kOiDone, kRReady, kUDone, kUsReady, kSDone0, kSDone1, kUoReady, kOiRead,
  kOaDone, kOFree, kNumNamed
};
static_assert(kNumNamed <= 15, "barrier count");

template <int KA, bool OUT, bool PAIR, bool SHARE>
__global__ void __launch_bounds__(kChainThreads, 1)
    delta_chain_kernel(const __grid_constant__ ChunkMaps maps, const DeltaArgs a, const unsigned char* img0,
                       int slices, const Segments sg) {
  using M = ChainSmem<KA, PAIR>;
  constexpr int DK = 64 * KA;
  constexpr int HC = DK / 2;  // key channels of a half: of two state warpgroups
  constexpr int QC = DK / 4;  // key channels of a state thread: KA steps of 16
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31;
  const Shifter sh{a.two16};
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  auto bar = [&](int b) { return sb + M::kBar + 8 * (kStages + b); };
  auto full = [&](int c) { return sb + M::kBar + 8 * (c & 1); };
  volatile int* abort = reinterpret_cast<volatile int*>(smem + M::kMisc + 4);
  const Waiter wait{abort, a.err};
  int* bad = reinterpret_cast<int*>(smem + M::kBad);

  if (tid == 32 * kCtlWarp) {
    for (int i = 0; i < kStages; ++i) mbar_init(sb + M::kBar + 8 * i, 1);
    const uint32_t counts[kNumNamed] = {8, 8, 8, 8, 1, 1, 16, 1, 16, 1, 1, 16, 16, 1, 16};
    for (int i = 0; i < kNumNamed; ++i) mbar_init(bar(i), counts[i]);
    *abort = 0;
    mbar_fence_init();
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
    prefetch_tensormap(&maps.out);
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
  const uint32_t tm = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);  // this warp's lane quarter
  const int row = 32 * (warp & 3) + lane;
  const int H = static_cast<int>(a.H), nseq = static_cast<int>(a.batch);
  Cut& cut = *reinterpret_cast<Cut*>(smem + M::kCut);
  griddep_wait();  // the prep's tiles, the counter of walks, the cut
  if (sg.cut) {
    copy_cut(sg.cut, &cut);
    __syncthreads();
  }
  const int walks = sg.cut ? cut.walk[nseq] * sg.walkers : nseq * sg.walkers * (sg.count - 1);
  const int items = !sg.cut ? sg.items : OUT ? cut.all[nseq] * sg.walkers : walks + cut.ident[nseq] * H;
  // Walks until none is left. `done`: chunks of the walks before this one, so that the barriers' phases run on.
  int done = 0;
  volatile int* plan = reinterpret_cast<volatile int*>(smem + M::kMisc + 8);
  if (tid == 0) plan[kItem] = -2;
  for (;;) {
  if (tid == 0) {  // the next item
    int item = plan[kItem];
    int3 p;
    if constexpr (SHARE) {
      if (item == -2) {
        plan[kShare] = static_cast<int>(atomicAdd(sg.next + (OUT ? 1 : 0), 1u));
        item = -1;
      } else if (plan[kTo] < sg.job) {  // the state of this walk is left for the next share; its writes are behind a barrier
        __threadfence();
        atomicExch(sg.flags + plan[kShare], OUT ? 2u : 1u);
      }
      p = share_item(sg, plan[kShare], items, item);
    } else {
      if (item == -2) item = static_cast<int>(blockIdx.x);
      else if (items > static_cast<int>(gridDim.x)) item = static_cast<int>(gridDim.x + atomicAdd(sg.next + (OUT ? 1 : 0), 1u));
      else item = items;
      p = make_int3(item < items ? item : -1, 0, 0x7fffffff);
    }
    plan[kItem] = p.x, plan[kFrom] = p.y, plan[kTo] = p.z;
    if (p.x >= 0) {
      const bool id = !OUT && p.x >= walks;
      int i = id ? p.x - walks : p.x;
      const int sl = id ? 1 : slices, heads = PAIR && !id ? H / 2 : H;
      plan[kIdent] = id;
      if (sg.cut) {
        plan[kSlice] = i % sl, i /= sl;
        plan[kHead] = i % heads, i /= heads;
        const int* sums = id ? cut.ident : OUT ? cut.all : cut.walk;
        const int place = cut_find(sums, nseq, i);
        plan[kSeq] = cut.seq[place];
        plan[kSeg] = i - sums[place] + (id ? 1 : 0);
        plan[kCount] = cut.all[place + 1] - cut.all[place];
        plan[kFirstSeg] = cut.all[place];
      } else {
        const int segs = OUT ? sg.count : id ? sg.count - 2 : sg.count - 1;
        plan[kSeg] = i % segs + (id ? 1 : 0), i /= segs;
        plan[kSlice] = i % sl, i /= sl;
        plan[kHead] = i % heads, i /= heads;
        plan[kSeq] = i;
        plan[kCount] = sg.count;
        plan[kFirstSeg] = i * sg.count;
      }
    }
  }
  __syncthreads();
  if (plan[kItem] < 0) break;
  // This walk's sequence, head, rows and segment; `ident`: of the identity; first_seg: the sequence's first segment.
  const bool ident = !OUT && plan[kIdent];
  const int slice = plan[kSlice], h = plan[kHead], s = plan[kSeq], seg = plan[kSeg], count = plan[kCount];
  const int first_seg = plan[kFirstSeg];
  const int per = sg.cut ? cut.per : sg.per;
  Span sp = span_of(a, s);
  const int64_t slot0 = slot_of(a, s, sp.t0) + static_cast<int64_t>(seg) * per + (SHARE ? plan[kFrom] : 0);
  if (count > 1) {
    sp.t0 += kC * per * seg;
    sp.len = max(0, min(sp.len - kC * per * seg, kC * per));
  }
  if constexpr (SHARE) {
    const int c0 = plan[kFrom];
    sp.t0 += kC * c0;
    sp.len = max(0, min(sp.len - kC * c0, kC * (plan[kTo] - c0)));
  }
  const int nc = (sp.len + kC - 1) / kC;
  // With PAIR, h is a pair of heads: rows 0-63 head 2 h, rows 64-127 head 2 h + 1. The identity is one head's.
  const int head0 = PAIR && !ident ? 2 * h : h, head1 = PAIR && !ident ? 2 * h + 1 : h;
  const int mine = PAIR ? (warp & 3) >> 1 : 0;  // which of the two this warp's rows are of
  const int r = slice * 128 + row, rows = static_cast<int>(ident ? a.dk : PAIR ? 128 : a.dv);
  const bool row_in = r < rows;
  auto arrive = [&](int b) {
    tcgen05_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };

  if (warp < kStateWarps) {
    // ------------------------------------------------------------- state ---
    const int quarter = warp >> 2, half = quarter >> 1;
    const int cols = static_cast<int>(min(static_cast<int64_t>(QC), max(a.dk - quarter * QC, static_cast<int64_t>(0))));
    const int64_t at = static_cast<int64_t>(row_in ? r : 0) * a.dk + quarter * QC;  // this thread's part of a state
    const int64_t shi = static_cast<int64_t>(s) * H + head0, one = a.dv * a.dk;  // a pair's states adjoin
    const float* from = a.state_in ? a.state_in + shi * one : nullptr;
    float* seg_state = sg.S + (static_cast<int64_t>(first_seg + seg) * H + head0) * one;
    if (count > 1) {
      if (OUT) {
        if (seg > 0 || a.state_in) from = seg_state;
      } else if (seg > 0) {
        from = nullptr;
      }
    }
    // Where this walk's state is left for the next share: where it goes in the end, or over the segment's first state.
    auto handed = [&]() -> float* {
      const int64_t at_seg = plan[kFirstSeg] + plan[kSeg];
      if (!OUT && plan[kIdent]) return sg.M + (at_seg * H + plan[kHead]) * a.dk * a.dk;
      const int64_t head = PAIR ? 2 * plan[kHead] : plan[kHead];
      if (OUT && plan[kCount] == 1) return a.state_out + (plan[kSeq] * a.H + head) * a.dv * a.dk;
      return sg.S + ((at_seg + (OUT ? 0 : 1)) * H + head) * a.dv * a.dk;
    };
    const bool begun = SHARE && plan[kFrom] > 0;
    if (begun) {
      from = handed();
      if (lane == 0) {
        const volatile uint32_t* flag = sg.flags + plan[kShare] - 1;
        const uint64_t w0 = globaltimer_ns();
        while (*flag < (OUT ? 2u : 1u) && !*abort) {
          if (globaltimer_ns() - w0 > 2000000000ull) {
            *abort = 1;
            if (a.err) atomicExch(a.err, 48);
          }
        }
      }
      __syncwarp();
      __threadfence();
    }
    uint64_t S[QC / 2];
#pragma unroll
    for (int i = 0; i < QC; i += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (from && row_in && i < cols) v = *reinterpret_cast<const float4*>(from + at + i);
      if (!OUT && !begun && from && row_in && i < cols)  // state_out may be state_in: pass 2 reads a copy
        *reinterpret_cast<float4*>(seg_state + at + i) = v;
      if (!OUT && ident && !begun) {
        const int d = r - quarter * QC - i;
        v = make_float4(d == 0, d == 1, d == 2, d == 3);
      }
      S[i / 2] = pk2(v.x, v.y), S[i / 2 + 1] = pk2(v.z, v.w);
    }
    float decay = 0.0f;
    // 16 columns of S: decayed, with the last chunk's contribution
    auto update = [&](int i0) {
      uint32_t d[16];
      tmem_ld_x16(tm + kTmDelta + quarter * QC + i0, d);
      tmem_ld_wait();
      const uint64_t dd = pk2(decay, decay);
#pragma unroll
      for (int i = 0; i < 8; ++i) S[i0 / 2 + i] = ffma2(dd, S[i0 / 2 + i], pk2u(d[2 * i], d[2 * i + 1]));
    };
    // Rounds and stores this thread's 16 tokens of chunk c, once the scores' product is in.
    auto store_chunk = [&](int c) {
      const int n = min(kC, sp.len - kC * c), t0 = 16 * quarter;
      __nv_bfloat16* tile = reinterpret_cast<__nv_bfloat16*>(smem + M::kOut + (c & 1) % M::kOuts * kC * 256) + t0 * 128 + row;
      wait(bar(kOaDone), (done + c) & 1, 39);
      tcgen05_fence_after();
      uint32_t d[16];
      tmem_ld_x16(tm + kTmO + t0, d);
      tmem_ld_wait();
      arrive(kOFree);
      const int first = min(min(bad[row], bad[128 + row]), min(bad[256 + row], bad[384 + row])) - t0;
      if (__any_sync(0xffffffffu, first < 16)) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i >= first) d[i] = 0x7fffffffu;
      }
      const bool issuer = (warp & 3) == 0 && lane == 0;
      if constexpr (M::kOuts == 1) {  // the last chunk's store has read the tile
        if (issuer) bulk_wait_read<0>();
        named_bar_sync(1 + quarter, 128);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) tile[i * 128] = __float2bfloat16_rn(__uint_as_float(d[i]));
      // A tile store per 16 tokens; it leaves out channels past d_value and tokens past L. The last tokens of a
      // packed sequence may end inside one: those rows are written one by one.
      if (!a.cu || n >= t0 + 16) {
        fence_proxy_async_smem();
        if (issuer) bulk_wait_read<0>();  // the last chunk's store has read its half of the tiles
        named_bar_sync(1 + quarter, 128);
        if (issuer) {
          tma_store_4d(&maps.out, sb + M::kOut + (c & 1) % M::kOuts * kC * 256 + t0 * 256, 128 * slice, h, sp.t0 + kC * c + t0,
                       sp.seq);
          bulk_commit();
        }
      } else if (row_in) {
        __nv_bfloat16* op = a.out + (static_cast<int64_t>(sp.t0) + kC * c + t0) * a.o_tok + head0 * a.dv + r;
        for (int t = 0; t0 + t < n; ++t) op[t * a.o_tok] = tile[t * 128];
      }
      __syncwarp();
    };
    const uint32_t tm_s = tm + kTmS + half * 96 + (quarter & 1) * (QC / 2);  // its columns of S's terms
    const uint32_t tm_y = tm + kTmY + 16 * quarter;                          // its 16 tokens
    const uint32_t tm_u = PAIR && mine ? tm + kTmS + 16 * quarter : tm_y;    // of U
#pragma unroll 1
    for (int c = 0; c < nc; ++c) {
      const int g = done + c;
      const uint32_t ph = g & 1;
      unsigned char* stage = smem + ph * M::kStage;
      const Coef& cf = *reinterpret_cast<const Coef*>(stage + M::kImg + mine * kImgStride + kImgCoef);
      const int n = min(kC, sp.len - kC * c);
      // S as the A operand of Y and Q S^T
      if (c > 0) {
        wait(bar(kSDone0 + half), ph ^ 1u, 33);
        tcgen05_fence_after();
      }
      if (a.cu && n < kC) {
        // Keys behind the sequence (the next packed one's) meet zeros of U: they must be finite.
        wait(full(g), (g >> 1) & 1, 34);
        for (int e = tid; e < KA * kC * 8; e += 32 * kStateWarps) {
          const int t = e / (kC * 8), i = e / 8 % kC;
          if (i >= n) *reinterpret_cast<uint4*>(stage + t * 2 * kAtom + i * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
#pragma unroll
      for (int b = 0; b < KA; ++b) {
        if (c > 0) update(16 * b);
        uint64_t x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = S[8 * b + i];
        store_split3(sh, tm_s + 8 * b, HC / 2, x);
        tmem_st_wait();
        arrive(kSReady0 + half * KA + b);
      }
      if (OUT && c > 0) store_chunk(c - 1);
      // R = V - e^G Y
      wait(full(g), (g >> 1) & 1, 34);
      decay = cf.decay;
      const unsigned char* vt = stage + M::kV + row * 2 + 16 * quarter * 256;
      // V, read while the product runs, and what must stay out of R: `marks`, tokens that are not finite, and `drop`,
      // those and the tokens behind the sequence.
      uint64_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = 0;
        if (OUT || !ident)
          v[i] = pk2(sh.low(*reinterpret_cast<const uint16_t*>(vt + 2 * i * 256)),
                     sh.low(*reinterpret_cast<const uint16_t*>(vt + (2 * i + 1) * 256)));
      }
      const int left = n - 16 * quarter;
      const uint32_t real = left >= 16 ? 0xffffu : left <= 0 ? 0u : 0xffffu >> (16 - left);
      const uint32_t marks = (not_finite(v) | cf.bad[half] >> (16 * (quarter & 1))) & real;
      const bool any_marks = __any_sync(0xffffffffu, marks != 0u);
      const uint32_t drop = marks | (~real & 0xffffu);
      const bool any_drop = any_marks || real != 0xffffu;
      wait(bar(kYDone), ph, 35);
      tcgen05_fence_after();
      {
        uint32_t d[16];
        uint64_t x[8];
        tmem_ld_x16(tm_y, d);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 e4 = *reinterpret_cast<const float4*>(cf.neg + 16 * quarter + i);
          x[i / 2] = ffma2(pk2(e4.x, e4.y), pk2u(d[i], d[i + 1]), v[i / 2]);
          x[i / 2 + 1] = ffma2(pk2(e4.z, e4.w), pk2u(d[i + 2], d[i + 3]), v[i / 2 + 1]);
        }
        if (any_drop) replace_marked(x, drop, 0.0f);
        store_split3(sh, tm + kTmDelta + 8 * quarter, 32, x);
      }
      tmem_st_wait();
      arrive(kRReady);
      if constexpr (OUT) {  // scale Q S^T
        wait(bar(kOiDone), ph, 38);
        tcgen05_fence_after();
        uint32_t d[16];
        tmem_ld_x16(tm + kTmO + 16 * quarter, d);
        float4 es[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) es[i] = *reinterpret_cast<const float4*>(cf.oq + 16 * quarter + 4 * i);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d[4 * i] = __float_as_uint(__uint_as_float(d[4 * i]) * es[i].x);
          d[4 * i + 1] = __float_as_uint(__uint_as_float(d[4 * i + 1]) * es[i].y);
          d[4 * i + 2] = __float_as_uint(__uint_as_float(d[4 * i + 2]) * es[i].z);
          d[4 * i + 3] = __float_as_uint(__uint_as_float(d[4 * i + 3]) * es[i].w);
        }
        tmem_st_x16(tm + kTmO + 16 * quarter, d);
        tmem_st_wait();
        arrive(kOiRead);
      }
      // U: scaled into the state's product, plain into the output's
      wait(bar(kUDone), ph, 36);
      tcgen05_fence_after();
      uint64_t x[8], y[8];
      {
        uint32_t d[16];
        tmem_ld_x16(tm_u, d);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = pk2u(d[2 * i], d[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 e4 = *reinterpret_cast<const float4*>(cf.ec + 16 * quarter + 4 * i);
          y[2 * i] = fmul2(x[2 * i], pk2(e4.x, e4.y));
          y[2 * i + 1] = fmul2(x[2 * i + 1], pk2(e4.z, e4.w));
        }
      }
      if (any_marks) replace_marked(y, marks, __uint_as_float(0x7fffffffu));
      store_split3(sh, tm + kTmS + 96 + 8 * quarter, 32, y);
      tmem_st_wait();
      arrive(kUsReady);
      if constexpr (OUT) {
        const int first = marks ? __ffs(marks) - 1 : 16;
        bad[quarter * 128 + row] = marks ? 16 * quarter + first : kC;
        if (any_marks) replace_marked(x, 0xffffu << first & 0xffffu, 0.0f);
        uint32_t hi[8], mi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) split2(sh, x[i], hi[i], mi[i]);
        // A thread's 16 columns: eight of each term. Of a pair, each head's rows are zero in the other's operand.
        const uint32_t other = tm + (mine ? kTmU : kTmY) + 16 * quarter;
        tmem_st_x8(tm + (PAIR && mine ? kTmY : kTmU) + 16 * quarter, hi);
        tmem_st_x8(tm + (PAIR && mine ? kTmY : kTmU) + 16 * quarter + 8, mi);
        if constexpr (PAIR) {
          const uint32_t zero[16] = {};
          tmem_st_x16(other, zero);
        }
        tmem_st_wait();
        arrive(kUoReady);
      }
    }
    if (nc > 0) {
      if constexpr (OUT) store_chunk(nc - 1);
      wait(bar(kSDone0 + half), (done + nc - 1) & 1, 33);
      tcgen05_fence_after();
#pragma unroll
      for (int i0 = 0; i0 < QC; i0 += 16) update(i0);
    }
    const bool ends = !SHARE || plan[kTo] >= sg.job;
    float* to = handed();
    if (OUT && ends)
      to = a.state_out + (static_cast<int64_t>(plan[kSeq]) * H + (PAIR ? 2 * plan[kHead] : plan[kHead])) * a.dv * a.dk;
    if (row_in && (!OUT || !ends || plan[kSeg] == plan[kCount] - 1)) {
#pragma unroll
      for (int i = 0; i < QC; i += 4)
        if (i < cols) {
          float4 v;
          upk2(S[i / 2], v.x, v.y);
          upk2(S[i / 2 + 1], v.z, v.w);
          *reinterpret_cast<float4*>(to + at + i) = v;
        }
    }
    if (OUT && (warp & 3) == 0 && lane == 0) bulk_wait_read<0>();  // the tiles stay until the last store has read them
    __syncwarp();
  } else {
    // ----------------------------------------------------------- control ---
    const int grp = head0 / static_cast<int>(a.H / a.G);
    const unsigned char* img = img0 + (slot0 * a.H + head0) * kImgStride;
    int loaded = 0;
    auto load = [&](int c) {
      if (*abort) return;
      loaded = c + 1;
      if (elect_one()) {
        const int tok = sp.t0 + kC * c;
        const int g = done + c;
        const uint32_t base = sb + (g & 1) * M::kStage;
        mbar_arrive_expect_tx(full(g), M::kTx);
#pragma unroll
        for (int t = 0; t < KA; ++t) {
          tma_load_4d(base + t * 2 * kAtom, &maps.k, 64 * t, grp, tok, sp.seq, full(g));
          tma_load_4d(base + t * 2 * kAtom + kAtom, &maps.q, 64 * t, grp, tok, sp.seq, full(g));
        }
        tma_load_4d(base + M::kV, &maps.v, 128 * slice, h, tok, sp.seq, full(g));
        bulk_load(base + M::kImg, img + static_cast<int64_t>(c) * a.H * kImgStride, kImgBytes, full(g));
        if constexpr (PAIR)
          bulk_load(base + M::kImg + kImgStride,
                    img + (static_cast<int64_t>(c) * a.H + head1 - head0) * kImgStride, kImgBytes, full(g));
      }
      __syncwarp();
    };
    for (int c = 0; c < min(nc, kStages); ++c) load(c);
#pragma unroll 1
    for (int c = 0; c < nc; ++c) {
      const int g = done + c;
      const uint32_t ph = g & 1;
      const uint32_t stage = sb + ph * M::kStage;
      const uint64_t kd = umma_desc_k_sw128(stage);
      const uint64_t td = panel_desc(stage + M::kImg);
      wait(full(g), (g >> 1) & 1, 40);
      // a pair's second scores' product reads an operand where Y goes
      if (PAIR && OUT && c > 0) wait(bar(kOaDone), ph ^ 1u, 47);
      // Y = S K^T, least terms first, a half's 32 key channels at a time: what is left after the last is short
#pragma unroll
      for (int st = 0; st < 2 * KA; ++st) {
        wait(bar(kSReady0 + st), ph, 41);
        tcgen05_fence_after();
        if (elect_one()) {
          const int hf = st / KA, b = st % KA;
#pragma unroll
          for (int t = 2; t >= 0; --t)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int k = hf * HC + w * QC + 16 * b;  // key channels k .. k + 15
              umma_f16_ts(tmem + kTmY, tmem + kTmS + hf * 96 + t * (HC / 2) + w * (QC / 2) + 8 * b,
                          desc_add(kd, (k / 64) * 2 * kAtom + (k % 64) * 2), chunk_idesc(64, false),
                          !(st == 0 && t == 2 && w == 0));
            }
          if (st == 2 * KA - 1) umma_commit(bar(kYDone));
        }
        __syncwarp();
      }
      // every use of the other stage is over: its chunk's last product is done
      if (c > 0 && c + 1 < nc) {
        if constexpr (OUT) wait(bar(kOaDone), ph ^ 1u, 47);
        load(c + 1);
      }
      // Q S^T
      if constexpr (OUT) {
        if (c > 0) wait(bar(kOFree), ph ^ 1u, 42);
        tcgen05_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int t = 1; t >= 0; --t)
#pragma unroll
            for (int k = 0; k < DK; k += 16)
              umma_f16_ts(tmem + kTmO, tmem + kTmS + (k / HC) * 96 + t * (HC / 2) + (k % HC) / 2,
                          desc_add(kd, (k / 64) * 2 * kAtom + kAtom + (k % 64) * 2), chunk_idesc(64, false),
                          !(t == 1 && k == 0));
          umma_commit(bar(kOiDone));
        }
        __syncwarp();
      }
      // U = R T^T: 16 tokens j at a time meet the tokens i from theirs on. Of a pair, each head's T meets all rows,
      // and its own rows are read of the result (the second where S's first terms were).
      wait(bar(kRReady), ph, 43);
      if (PAIR && OUT) wait(bar(kOiDone), ph, 38);
      tcgen05_fence_after();
      if (elect_one()) {
        constexpr int kTt[6] = {2, 0, 1, 1, 0, 0}, kTr[6] = {0, 2, 1, 0, 1, 0};  // terms of T and R, least first
#pragma unroll
        for (int hd = 0; hd < M::kImgs; ++hd)
#pragma unroll
          for (int pr = 0; pr < 6; ++pr)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f16_ts(tmem + (hd ? kTmS : kTmY) + 16 * kk, tmem + kTmDelta + 32 * kTr[pr] + 8 * kk,
                          desc_add(td, hd * kImgStride + kTt[pr] * kPanelTerm + panel_off(kk)),
                          chunk_idesc(64 - 16 * kk, false), pr + kk > 0);
        umma_commit(bar(kUDone));
      }
      __syncwarp();
      // the chunk's contribution to S
      wait(bar(kUsReady), ph, 44);
      tcgen05_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int at = 0; at < KA; ++at) {
#pragma unroll
          for (int t = 2; t >= 0; --t)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f16_ts(tmem + kTmDelta + 64 * at, tmem + kTmS + 96 + 32 * t + 8 * kk,
                          desc_add(kd, at * 2 * kAtom + 2048 * kk), chunk_idesc(64, true), !(t == 2 && kk == 0));
          umma_commit(bar(kSDone0 + at));
        }
        if (KA == 1) umma_commit(bar(kSDone1));
      }
      __syncwarp();
      // the scores times U
      if constexpr (OUT) {
        wait(bar(kOiRead), ph, 45);
        wait(bar(kUoReady), ph, 46);
        tcgen05_fence_after();
        if (elect_one()) {
          constexpr int kTp[3] = {1, 0, 0}, kTu[3] = {0, 1, 0};
#pragma unroll
          for (int hd = 0; hd < M::kImgs; ++hd)
#pragma unroll
            for (int pr = 0; pr < 3; ++pr)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_f16_ts(tmem + kTmO + 16 * kk, tmem + (hd ? kTmY : kTmU) + 16 * kk + 8 * kTu[pr],
                            desc_add(td, hd * kImgStride + kImgP + kTp[pr] * kPanelTerm + panel_off(kk)),
                            chunk_idesc(64 - 16 * kk, false), true);
          umma_commit(bar(kOaDone));
        }
        __syncwarp();
      }
    }
    // Nothing is in flight at the end of a run whose waits all came: each load and product has been waited for.
    // Otherwise wait for them here, with a limit.
    if (*abort) {
      for (int c = max(0, loaded - kStages); c < loaded; ++c) {
        const uint64_t w0 = globaltimer_ns();
        while (!mbar_try_wait(full(done + c), ((done + c) >> 1) & 1) && globaltimer_ns() - w0 < 2000000000ull) {
        }
      }
      spin_ns(1000000);  // products take microseconds
    } else if (nc > 0) {
      wait(bar(OUT ? kOaDone : kSDone1), (done + nc - 1) & 1, 39);
    }
  }
  __syncwarp();
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  done += nc;
  }
  if (warp == kCtlWarp) tmem_dealloc(tmem, 512);
}

// First states of segments 2 .. count - 1: S_{p+1} = S_p M_p + H_p, H_p lying
// where S_{p+1} goes. One block per R rows of a (sequence, head) through all
// segments, M_{p+1} on its way to shared memory while M_p is used. A warp takes
// every eighth four of the products' key channels for all R rows, so that M is
// read once, and the eight sums are added in a fixed order; fp32 throughout.
// (4 heads of 8192 tokens, 16 segments: 20.7 us; with 32 rows a block and a row
// a warp, M read by every warp, 58 us.)
constexpr int kJoinWarps = 8, kJoinLd = 132;
template <int R>
constexpr int kJoinSmem = (2 * 128 * 128 + R * kJoinLd + kJoinWarps * R * 128) * 4 + static_cast<int>(sizeof(Cut));
template <int R>
__global__ void __launch_bounds__(32 * kJoinWarps, 1)
    delta_join_kernel(const DeltaArgs a, const Segments sg, int row_blocks) {
  extern __shared__ __align__(16) float join_smem[];
  float* Ss = join_smem + 2 * 128 * 128;                    // S_p [row][key channel]
  float* parts = Ss + R * kJoinLd;                          // [warp][row][key channel]
  Cut& cut = *reinterpret_cast<Cut*>(parts + kJoinWarps * R * 128);
  const int H = static_cast<int>(a.H), dk = static_cast<int>(a.dk), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = 4 * lane;
  const bool in = col < dk;
  if (sg.cut) {
    copy_cut(sg.cut, &cut);
    __syncthreads();
  }
  for (int item = static_cast<int>(blockIdx.x); item < static_cast<int>(a.batch) * H * row_blocks; item += gridDim.x) {
    const int sh = item / row_blocks, s = sh / H;  // with a cut: the place in its order, the longest first
    int count = sg.count, first_seg = s * count;
    if (sg.cut) first_seg = cut.all[s], count = cut.all[s + 1] - first_seg;
    if (count < 3) break;
    const int r0 = item % row_blocks * R, nr = min(R, static_cast<int>(a.dv) - r0);
    const int64_t index = static_cast<int64_t>(first_seg) * H + sh % H, step = a.dv * a.dk * H;
    float* S = sg.S + index * a.dv * a.dk + static_cast<int64_t>(r0) * dk + col;
    const float* Mp = sg.M + index * dk * dk;
    auto fetch = [&](int p) {  // M_p, p >= 1
      if (p + 1 < count) {
        const uint32_t dst = smem_u32(join_smem + (p & 1) * 128 * 128);
        const float* src = Mp + static_cast<int64_t>(p) * H * dk * dk;
        for (int i = threadIdx.x; i < dk * dk / 4; i += 32 * kJoinWarps) cp_async_16(dst + 16 * i, src + 4 * i);
      }
      cp_async_commit();
    };
    auto load = [&](int p, float4 (&v)[R / kJoinWarps]) {  // S_p's or H_{p-1}'s part of this thread: rows warp, warp + 8 ..
#pragma unroll
      for (int i = 0; i < R / kJoinWarps; ++i) {
        const int r = warp + kJoinWarps * i;
        v[i] = r < nr && in ? *reinterpret_cast<const float4*>(S + p * step + r * dk) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    fetch(1);
    float4 mine[R / kJoinWarps];
    load(1, mine);
    for (int p = 1; p + 1 < count; ++p) {
      fetch(p + 1);
#pragma unroll
      for (int i = 0; i < R / kJoinWarps; ++i)
        *reinterpret_cast<float4*>(Ss + (warp + kJoinWarps * i) * kJoinLd + col) = mine[i];
      load(p + 1, mine);
      cp_async_wait<1>();
      __syncthreads();
      const float* Ms = join_smem + (p & 1) * 128 * 128 + (in ? col : 0);
      uint64_t acc[R][2] = {};
#pragma unroll 1
      for (int k = 4 * warp; k < dk; k += 4 * kJoinWarps) {
        ulonglong2 m[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) m[z] = *reinterpret_cast<const ulonglong2*>(Ms + (k + z) * dk);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 w = *reinterpret_cast<const float4*>(Ss + r * kJoinLd + k);
          const float wz[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            acc[r][0] = ffma2(pk2(wz[z], wz[z]), m[z].x, acc[r][0]);
            acc[r][1] = ffma2(pk2(wz[z], wz[z]), m[z].y, acc[r][1]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
        *reinterpret_cast<ulonglong2*>(parts + (warp * R + r) * 128 + col) = make_ulonglong2(acc[r][0], acc[r][1]);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < R / kJoinWarps; ++i) {
        const int r = warp + kJoinWarps * i;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
          const float4 v = *reinterpret_cast<const float4*>(parts + (w * R + r) * 128 + col);
          mine[i].x += v.x, mine[i].y += v.y, mine[i].z += v.z, mine[i].w += v.w;
        }
        if (r < nr && in) *reinterpret_cast<float4*>(S + (p + 1) * step + r * dk) = mine[i];
      }
    }
    __syncthreads();  // the next item's rows and M may overwrite these
  }
}

int64_t chunk_slots(int64_t batch, int64_t L, bool packed) {
  return packed ? L / kC + batch : batch * ((L + kC - 1) / kC);
}

// Rows of a join block: eight where such blocks fit the SMs at once.
int join_rows(int64_t seq_heads, int64_t dv, int sms) { return seq_heads * ((dv + 7) / 8) <= sms ? 8 : 16; }

// Time of `walks` walks of len chunks on `sms` SMs, in chunks: whole ones in rounds, or equal shares of them (8%
// slower, and 3 for the hand-over), whichever is less. scale: of a chunk, kStatesOnly in pass 1.
double walk_time(int64_t walks, int64_t len, int sms, double scale, bool* shares) {
  const double whole = static_cast<double>((walks + sms - 1) / sms) * (scale * static_cast<double>(len) + kWalkStart);
  const double shared = static_cast<double>(walks) / sms * (1.08 * scale * static_cast<double>(len) + kWalkStart) + 3.0;
  *shares = walks > sms && len >= kShareLeast && shared < whole;
  return *shares ? shared : whole;
}

// Segments of a walk of nc chunks with `units` (sequence, head, slice) on
// `sms` SMs: the time of both passes and the extra launches, and for each
// segment and wave of the join's blocks 0.4 (0.52 of 16 rows). (Times of 1 to
// 32 segments for 2 to 60 heads and 2048 to 32768 tokens: the choice is within
// 10% of the best.)
int choose_segments(int64_t nc, int64_t units, int64_t seq_heads, int64_t dv, int sms, int* per) {
  bool shares;
  const int rows = join_rows(seq_heads, dv, sms);
  const int64_t blocks = seq_heads * ((dv + rows - 1) / rows);
  const double join = (rows == 8 ? 0.4 : 0.52) * static_cast<double>((blocks + sms - 1) / sms);
  double best = 0.95 * walk_time(units, nc, sms, 1.0, &shares);
  int count = 1;
  *per = static_cast<int>(nc);
  for (int64_t p = 2; p <= 64 && 4 * p <= nc && units * p <= 64 * sms; ++p) {
    const int64_t len = (nc + p - 1) / p;
    if ((nc + len - 1) / len != p) continue;
    const double cost = walk_time(units * (p - 1) + seq_heads * (p - 2), len, sms, kStatesOnly, &shares) +
                        walk_time(units * p, len, sms, 1.0, &shares) + kMoreLaunches + join * static_cast<double>(p - 2);
    if (cost < best) best = cost, count = static_cast<int>(p), *per = static_cast<int>(len);
  }
  return count;
}

struct ChunkPlan {
  int64_t slots;
  int slices, walkers, count, per, sms, room;
  bool cut, pair;
  size_t next, flags, cuts, S, M, bytes;  // offsets of what is not operand tiles, and the end
};
ChunkPlan chunk_plan(int64_t batch, int64_t L, int64_t H, int64_t G, int64_t dk, int64_t dv, bool packed) {
  ChunkPlan p{};
  p.sms = device_sms();
  p.slots = chunk_slots(batch, L, packed);
  p.slices = static_cast<int>((dv + 127) / 128);
  p.pair = delta_pairs(H, G, dv);
  p.walkers = static_cast<int>(delta_walkers(H, G, dv));
  const int64_t nc = (L + kC - 1) / kC;
  p.count = 1, p.per = static_cast<int>(nc);
  if (packed)  // some sequence may be long enough to cut
    p.cut = batch <= kCutSeqs && nc >= 4 * kCutLeast && (nc + batch) * H * p.slices < (1 << 28);
  else
    p.count = choose_segments(nc, batch * p.walkers, batch * H, dv, p.sms, &p.per);
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  p.next = kImgBytes;  // behind the first slot's tiles, which leave room there
  p.flags = up(static_cast<size_t>(p.slots) * static_cast<size_t>(H) * kImgStride);
  // room for the shares' flags where one length and enough walks may have them
  const int64_t most = batch * p.count * (p.walkers + H);
  p.cuts = p.flags + (!packed && most > p.sms ? up(static_cast<size_t>(p.sms) * 4) : 0);
  p.S = p.M = p.bytes = p.cuts + (p.cut ? up(sizeof(Cut)) : 0);
  if (p.count > 1 || p.cut) {
    // Of packed sequences only those that are cut have states here, and as the longest they come first. Each has more
    // than kCutLeast chunks, only its last segment may be shorter than that, and it has 32 segments at most.
    const int64_t m = std::min(batch, L / (kC * kCutLeast + 1));
    const int64_t segs = !p.cut ? batch * p.count : std::min(32 * m, m + (L / kC + m) / kCutLeast);
    p.room = static_cast<int>(segs);
    p.M = up(p.S + static_cast<size_t>(segs * H * dv * dk) * 4);
    p.bytes = up(p.M + static_cast<size_t>(segs * H * dk * dk) * 4);
  }
  return p;
}

template <int KA, bool OUT, bool PAIR>
cudaError_t launch_chain(const ChunkMaps& maps, const DeltaArgs& a, const unsigned char* img, const ChunkPlan& p,
                         const Segments& sg, bool after_prep, cudaStream_t st) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(sg.cut || sg.items > p.sms ? p.sms : sg.items));
  cfg.blockDim = dim3(kChainThreads);
  cfg.dynamicSmemBytes = ChainSmem<KA, PAIR>::kTotal + 1024;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = after_prep ? 1 : 0;
  return sg.job ? cudaLaunchKernelEx(&cfg, delta_chain_kernel<KA, OUT, PAIR, true>, maps, a, img, p.slices, sg)
                : cudaLaunchKernelEx(&cfg, delta_chain_kernel<KA, OUT, PAIR, false>, maps, a, img, p.slices, sg);
}

template <int KA, bool PAIR>
cudaError_t launch_chunk(const ChunkMaps& maps, const DeltaArgs& a, const ChunkPlan& p, void* ws, cudaStream_t st) {
  unsigned char* img = static_cast<unsigned char*>(ws);
  const int prep_smem = PrepSmem<KA>::kTotal + 1024, smem = ChainSmem<KA, PAIR>::kTotal + 1024;
  auto prep = delta_prep_kernel<KA, PAIR>;
  // The kernels' shared-memory limits, once per device.
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    constexpr auto kAttr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    err = cudaFuncSetAttribute(prep, kAttr, prep_smem);
    if (err == cudaSuccess) err = cudaFuncSetAttribute(delta_chain_kernel<KA, true, PAIR, true>, kAttr, smem);
    if (err == cudaSuccess) err = cudaFuncSetAttribute(delta_chain_kernel<KA, true, PAIR, false>, kAttr, smem);
    if (err == cudaSuccess) err = cudaFuncSetAttribute(delta_chain_kernel<KA, false, PAIR, true>, kAttr, smem);
    if (err == cudaSuccess) err = cudaFuncSetAttribute(delta_chain_kernel<KA, false, PAIR, false>, kAttr, smem);
    if (err == cudaSuccess) err = cudaFuncSetAttribute(delta_join_kernel<8>, kAttr, kJoinSmem<8>);
    if (err == cudaSuccess) err = cudaFuncSetAttribute(delta_join_kernel<16>, kAttr, kJoinSmem<16>);
    if (err != cudaSuccess) return err;
    if (dev < 64) ready.fetch_or(uint64_t{1} << dev, std::memory_order_release);
  }
  const int64_t rep = a.H / a.G;
  auto prep_blocks = [&](int heads) { return p.slots * a.G * ((rep + heads - 1) / heads); };
  int set_heads = kPrepHeads;
  while (set_heads > 1 && prep_blocks(set_heads / 2) <= 5 * p.sms) set_heads /= 2;  // five blocks fit an SM
  const int64_t bh = a.batch * a.H, units = a.batch * p.walkers;
  Segments sg{p.count, p.per, p.cut ? reinterpret_cast<Cut*>(img + p.cuts) : nullptr, static_cast<int>(units * p.count), reinterpret_cast<float*>(img + p.S),
              reinterpret_cast<float*>(img + p.M), reinterpret_cast<uint32_t*>(img + p.next), reinterpret_cast<uint32_t*>(img + p.flags), 0, 0,
              p.walkers, p.sms, p.room};
  auto share = [&](Segments& g, double scale) {  // never for packed sequences
    bool shares = false;
    if (!a.cu) walk_time(g.items, p.per, p.sms, scale, &shares);
    if (!shares) return;
    g.job = p.per;
    g.share = static_cast<int>((static_cast<int64_t>(g.items) * (p.per + kStartChunks) + p.sms - 1) / p.sms);
  };
  Segments first = sg;
  first.items = static_cast<int>(units * (p.count - 1) + bh * (p.count - 2));
  if (p.count > 1) share(first, kStatesOnly);
  share(sg, 1.0);
  Segments both = sg;
  both.job = sg.job | first.job;
  prep<<<static_cast<unsigned>(prep_blocks(set_heads) + p.cut), 128, prep_smem, st>>>(maps, a, img, set_heads, both);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  if (p.count == 1 && !p.cut) return launch_chain<KA, true, PAIR>(maps, a, img, p, sg, true, st);
  err = launch_chain<KA, false, PAIR>(maps, a, img, p, first, true, st);
  if (err != cudaSuccess) return err;
  if (p.count > 2 || p.cut) {
    const int rows = join_rows(bh, a.dv, p.sms), rb = static_cast<int>((a.dv + rows - 1) / rows);
    const unsigned blocks = static_cast<unsigned>(bh * rb < p.sms ? bh * rb : p.sms);  // one an SM
    if (rows == 8) delta_join_kernel<8><<<blocks, 32 * kJoinWarps, kJoinSmem<8>, st>>>(a, sg, rb);
    else delta_join_kernel<16><<<blocks, 32 * kJoinWarps, kJoinSmem<16>, st>>>(a, sg, rb);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
  }
  return launch_chain<KA, true, PAIR>(maps, a, img, p, sg, false, st);
}

}  // namespace

int device_sms() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      sms <= 0) {
    cudaGetLastError();  // no device: a B200's
    sms = 148;
  }
  return sms;
}

size_t delta_chunk_workspace(int64_t batch, int64_t L, int64_t H, int64_t G, int64_t dk, int64_t dv, bool packed) {
  return chunk_plan(batch, L, H, G, dk, dv, packed).bytes;
}

cudaError_t launch_delta_chunk(const DeltaArgs& a, void* ws, cudaStream_t st) {
  ChunkMaps m;
  const bool packed = a.cu != nullptr;
  auto map4 = [&](CUtensorMap* out, const void* base, int64_t n, int64_t heads, int64_t tok, int64_t seq,
                  uint32_t box, uint32_t tokens, CUtensorMapSwizzle swz) {
    const uint64_t dims[4] = {uint64_t(n), uint64_t(heads), uint64_t(a.L), packed ? 1 : uint64_t(a.batch)};
    const uint64_t strides[3] = {uint64_t(n * 2), uint64_t(tok * 2), uint64_t(seq * 2)};
    const uint32_t b[4] = {box, 1, tokens, 1};
    return encode_map(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, b, swz);
  };
  const ChunkPlan p = chunk_plan(a.batch, a.L, a.H, a.G, a.dk, a.dv, packed);
  const int64_t rows = p.pair ? 128 : a.dv, heads = p.pair ? a.H / 2 : a.H;  // of v and out as the walk takes them
  if (!map4(&m.q, a.q, a.dk, a.G, a.q_tok, a.q_seq, 64, kC, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !map4(&m.k, a.k, a.dk, a.G, a.k_tok, a.k_seq, 64, kC, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !map4(&m.v, a.v, rows, heads, a.v_tok, a.v_seq, 128, kC, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !map4(&m.out, a.out, rows, heads, a.o_tok, a.o_seq, 128, 16, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  if (p.pair) return a.dk > 64 ? launch_chunk<2, true>(m, a, p, ws, st) : launch_chunk<1, true>(m, a, p, ws, st);
  return a.dk > 64 ? launch_chunk<2, false>(m, a, p, ws, st) : launch_chunk<1, false>(m, a, p, ws, st);
}

}  // namespace ssm
