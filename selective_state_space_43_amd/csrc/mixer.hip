// libselscan -- the Mamba-2 mixer between its two projections, for AMD
// Instinct MI355X (gfx950): the short causal convolution and the scan over
// packed prompts (ssm_conv_ssd_fwd), the same for one token a sequence
// (ssm_conv_ssd_update), and the gated group norm behind the scan with its
// gradient (ssm_group_norm_fwd, ssm_group_norm_bwd).
//
// Rows here are tokens: the tensors are slices of the input projection's
// rows, so every one of them has its own row stride.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "host.h"

namespace {

// ---------------------------------------------------------------- math and element access

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// log(1 + e^x): above 15 it is x to within 2e-8 of it; below, the rounding of
// u = 1 + e is taken back to first order, which keeps tiny steps exact.
__device__ __forceinline__ float softplus(float x) {
  const float e = ex2(x * kLog2e), u = 1.0f + e;
  const float l = __builtin_amdgcn_logf(u) * kLn2 - ((u - 1.0f) - e) * rcp(u);
  return x > 15.0f ? x : l;
}

__device__ __forceinline__ float sigmoid(float x) { return rcp(1.0f + ex2(-x * kLog2e)); }
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }

// float32 or bf16 (as its bits) elements, read and written as float32
template <typename IO>
__device__ __forceinline__ float ld(const void* p, int64_t i) {
  if constexpr (sizeof(IO) == 4) return static_cast<const float*>(p)[i];
  else return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}
template <typename IO>
__device__ __forceinline__ void st(void* p, int64_t i, float v) {
  if constexpr (sizeof(IO) == 4) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// ---------------------------------------------------------------- arguments

struct MixArgs {
  const void* xbc;
  const void* dt;
  const void* z;
  const float* cw;       // convolution taps [channels, W]
  const float* cb;       // convolution bias or NULL
  const float* A;
  const float* Dskip;
  const float* dt_bias;
  const int32_t* cu;     // starts of the packed sequences; not used by the one-token step
  const int32_t* slots;  // NULL: sequence s has slot s
  const uint8_t* has;    // NULL: no sequence continues; not used by the one-token step
  float* conv_state;     // [nslots, channels, W - 1]
  float* state;          // [nslots, H, P, N] or NULL
  void* y;
  int64_t xs, ds, zs, ys;  // row strides in elements
  int64_t tokens, nseq, nslots;
  int H, P, G, N, W, C;    // C: convolution channels, H P + 2 G N
  int softplus;
};

constexpr int kMaxN = 256;

// ---------------------------------------------------------------- packed prompts as block products
//
// The recurrence over a block of Q = 64 steps, with c_t the running sum of
// dt A inside the block and h the state entering it, is
//
//   y_t  = sum_{s<=t} M[t,s] x_s + exp(c_t) C_t . h
//   M    = (C_t . B_s) exp(c_t - c_s) dt_s,  D added on the diagonal
//   h'   = exp(c_Q) h + sum_s (exp(c_Q - c_s) dt_s x_s) B_s^T
//
// four products on the matrix cores.  B, C and C.B^T belong to a group of
// heads: mix_prep_kernel makes them once per block, in the order in which the
// matrix instructions take their operands.  mix_block_kernel then walks the
// blocks of a segment of a sequence, one wave per 16 PT channels of a head,
// the state in the wave's accumulators from block to block.  A sequence
// longer than a segment is cut: a first pass (SUM) gives each segment's state
// from zero, mix_join_kernel chains them, and the second pass starts every
// segment from the state entering it.
//
// Precision: the accumulators, the state, the running sums (float64) and all
// statistics are float32 or more.  The operands are fp16 in two pieces (hi + lo, 22
// bits, three products; lo x lo, 2^-24 of the product, is left out), scaled by a
// power of two from the largest value of the block: x and the state by channel, M by
// row, B, C and the state's weights as a whole.  fp16's exponents reach 2^40 below
// that: a value is held to 2^-22 of itself or 2^-40 of the largest one.  One scale for
// a wave's 32 channels would be 3 % faster (868 against 895 us for four prompts of
// 8192) and let a large channel take its neighbours' bits, another head's among
// them where a head ends inside a tile.  One piece for what enters y
// alone (11 bits beside the 8 of a stored bf16) would cost 1e-3 of y where two cost
// what the float32 sums do.

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

constexpr int kQ = 64;
constexpr int kTri = 6;  // 16 x 32 tiles of M on or below the diagonal

// 64 rows at most of one sequence
struct Chunk {
  int r0, r1;  // rows [r0, r1)
  int t0;      // the sequence's first row
  int from;    // the slot whose inputs come before it, or -1
};
// consecutive blocks of one sequence
struct Seg {
  int slot, t0, t1;  // the sequence's slot and rows
  int c0, nc;        // its blocks [c0, c0 + nc) of the sequence
  int gc;            // place of the first of them among all blocks
  int split;         // segments before this one among those of cut sequences; -1: not cut
  int cut;           // cut sequences before this one
  int resume;        // the sequence starts from its slot
};
// A cut sequence: its segments' places among those of cut sequences.
struct Cut {
  int slot, split, nseg, resume;
};

struct PlanHead {
  int nseg, nchunk, ncut, pad;
};

struct BlkArgs : MixArgs {
  PlanHead* head;
  Chunk* chunks;
  Seg* segs;
  Cut* cuts;
  char* ops;       // operands of (block, group)
  float* local;    // [split * sub][H, P, N] state of a piece from zero; of the first, then the state entering the segment
  float* decay;    // [split * sub][H] log2 of a piece's whole decay
  float* cs0;      // [cut][inner, 3] what the first rows of a cut sequence start from
  int seg_len;     // blocks of a segment at most
  int sub;         // pieces of a segment in the first pass
  int units;       // workgroups a segment needs
  int per_group;   // of them per group
  int fast;
};

// Offsets of the parts of one (block, group)'s operands.
template <int NT>
struct Ops {
  static constexpr int piece = kQ * NT * 16 * 2;  // one fp16 piece of B or C
  static constexpr int c = 0, b = 2 * piece, g = 4 * piece;
  static constexpr int gsize = kTri * 64 * 8 * 4;  // C.B^T in float32
  static constexpr int scale = g + gsize;          // B's and C's shifts
  static constexpr int bytes = scale + 64;
};

__device__ __forceinline__ float wave_max(float v) {  // v >= 0; uniform result
#define MIX_STEP(ctrl, rows)                                                                     \
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, rows, 0xf, \
                                                          rows == 0xf)));
  MIX_STEP(0x111, 0xf) MIX_STEP(0x112, 0xf) MIX_STEP(0x114, 0xf) MIX_STEP(0x118, 0xf)
  MIX_STEP(0x142, 0xa) MIX_STEP(0x143, 0xc)
#undef MIX_STEP
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// The largest of the four lanes i, i + 16, i + 32, i + 48.
__device__ __forceinline__ float row_max(float v) {
  u2 w = __builtin_bit_cast(u2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  v = fmaxf(__uint_as_float(w.x), __uint_as_float(w.y));
  w = __builtin_bit_cast(u2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return fmaxf(__uint_as_float(w.x), __uint_as_float(w.y));
}

// Inclusive sum over the wave's lanes in float64: steps of very different
// sizes follow each other in one block, and differences of the sums count.
__device__ __forceinline__ double wave_scan(double v) {
#define MIX_STEP(ctrl, rows)                                                                      \
  {                                                                                               \
    const u2 w = __builtin_bit_cast(u2, v);                                                       \
    u2 o;                                                                                         \
    o.x = __builtin_amdgcn_update_dpp(0, w.x, ctrl, rows, 0xf, rows == 0xf);                      \
    o.y = __builtin_amdgcn_update_dpp(0, w.y, ctrl, rows, 0xf, rows == 0xf);                      \
    v += __builtin_bit_cast(double, o);                                                           \
  }
  MIX_STEP(0x111, 0xf) MIX_STEP(0x112, 0xf) MIX_STEP(0x114, 0xf) MIX_STEP(0x118, 0xf)
  MIX_STEP(0x142, 0xa) MIX_STEP(0x143, 0xc)
#undef MIX_STEP
  return v;
}

__device__ __forceinline__ double lane63(double v) {
  const u2 w = __builtin_bit_cast(u2, v);
  u2 o;
  o.x = __builtin_amdgcn_readlane(w.x, 63);
  o.y = __builtin_amdgcn_readlane(w.y, 63);
  return __builtin_bit_cast(double, o);
}

// The power of two that brings the largest magnitude m of a tile to [2^14,
// 2^15), held where it is a float32 itself.
__device__ __forceinline__ int shift_for(float m) {
  const int e = 15 - __builtin_amdgcn_frexp_expf(m);
  return e < -113 ? -113 : (e > 111 ? 111 : e);
}
__device__ __forceinline__ float two(int e) { return __builtin_amdgcn_ldexpf(1.0f, e); }
// The larger of m and two magnitudes; a NaN among them is passed over.
__device__ __forceinline__ float max3(float m, float x, float y) {
  float o;
  asm("v_max3_f32 %0, %1, |%2|, |%3|" : "=v"(o) : "v"(m), "v"(x), "v"(y));
  return o;
}
// The same, and a NaN stays.
__device__ __forceinline__ float max3_nan(float m, float x, float y) {
  float o;
  asm("v_maximum3_f32 %0, %1, |%2|, |%3|" : "=v"(o) : "v"(m), "v"(x), "v"(y));
  return o;
}
// In a branch that is hardly ever taken: keeps the compiler from computing both sides.
__device__ __forceinline__ void rarely() { asm volatile(""); }
__device__ __forceinline__ bool finite(float v) { return fabsf(v) < __builtin_inff(); }

__device__ __forceinline__ f4 mfma(h8 a, h8 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// v w = hi + lo in fp16, to 22 bits; lo takes in what v w itself was rounded by
__device__ __forceinline__ void pieces(const float* v, const float* w, h8& hi, h8& lo) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const h2 a = __builtin_convertvector((f2){v[j] * w[j], v[j + 1] * w[j + 1]}, h2);
    hi[j] = a.x; hi[j + 1] = a.y;
    lo[j] = (_Float16)__builtin_fmaf(v[j], w[j], -(float)a.x);
    lo[j + 1] = (_Float16)__builtin_fmaf(v[j + 1], w[j + 1], -(float)a.y);
  }
}
// v = hi + lo in fp16, to 22 bits
__device__ __forceinline__ void pieces(const float* v, h8& hi, h8& lo) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const h2 a = __builtin_convertvector((f2){v[j], v[j + 1]}, h2);
    const h2 b = __builtin_convertvector(
        (f2){__builtin_fmaf((float)a.x, -1.0f, v[j]), __builtin_fmaf((float)a.y, -1.0f, v[j + 1])}, h2);
    hi[j] = a.x; hi[j + 1] = a.y; lo[j] = b.x; lo[j + 1] = b.y;
  }
}
// hi + lo
__device__ __forceinline__ void joined(const h8& hi, const h8& lo, float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __builtin_fmaf((float)hi[j], 1.0f, (float)lo[j]);
}

// ---- the plan: sequences -> blocks and segments (one workgroup)
//
// On the GPU, so that lengths that only it knows need no copy to the host.  6 us
// for one sequence, 8 for 512 blocks, most of it the latency of its loads and of
// five meetings a turn of 1024 sequences.

// Exclusive sums over the workgroup of four values at once, and their totals.
typedef int i4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i4 block_scan(i4 v, i4* red, i4& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  i4 x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    i4 o;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = __shfl_up(x[k], d, 64);
    if (lane >= d) x += o;
  }
  if (lane == 63) red[w] = x;
  __syncthreads();
  i4 before = {0, 0, 0, 0}, all = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const i4 r = red[i];
    if (i < w) before += r;
    all += r;
  }
  total = all;
  return before + x - v;
}
__device__ __forceinline__ int block_scan_max(int v, int* red) {  // inclusive, v >= 0
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d, 64);
    if (lane >= d) v = max(v, o);
  }
  if (lane == 63) red[w] = v;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < w) v = max(v, red[i]);
  return v;
}

// The last index whose prefix (of 1024) is at most i.
__device__ __forceinline__ int find(const int* prefix, int i) {
  int at = 0;
#pragma unroll
  for (int d = 512; d; d >>= 1)
    if (prefix[at + d] <= i) at += d;
  return at;
}

__global__ void __launch_bounds__(1024) mix_plan_kernel(const BlkArgs a) {
  __shared__ int red[16];
  __shared__ i4 red4[16];
  __shared__ int s_t0[1024], s_t1[1024], s_slot[1024], s_chunk[1024], s_seg[1024], s_split[1024], s_cut[1024];
  int nchunk = 0, nseg = 0, nsplit = 0, ncut = 0;
  const int i = threadIdx.x, tokens = (int)a.tokens;
  int reached = max(0, min(a.cu[0], tokens));  // the largest offset so far
  for (int64_t base = 0; base < a.nseq; base += 1024) {
    // the offsets' running maximum: whatever they hold, the sequences lie one
    // behind the other inside the rows, and the tables hold their blocks
    const int64_t s = base + i;
    const bool in = s < a.nseq;
    const int64_t slot = in && a.slots ? a.slots[s] : s;
    const bool resume = in && a.has && a.has[s];
    int end = in ? max(reached, min(a.cu[s + 1], tokens)) : reached;
    end = block_scan_max(end, red);
    s_t1[i] = end;
    __syncthreads();
    const int begin = i ? s_t1[i - 1] : reached;
    reached = s_t1[1023];
    s_t0[i] = begin;
    i4 n = {0, 0, 0, 0};  // blocks, segments, segments of cut sequences, cut sequences
    if (in && (!a.state || (slot >= 0 && slot < a.nslots))) {  // else padding
      n[0] = (end - begin + kQ - 1) / kQ;
      n[1] = n[0] ? (n[0] + a.seg_len - 1) / a.seg_len : 1;
      n[2] = n[1] > 1 ? n[1] : 0;
      n[3] = n[1] > 1;
    }
    i4 all;
    const i4 at = block_scan(n, red4, all);
    s_slot[i] = (int)slot | (resume ? (int)0x80000000 : 0);
    s_chunk[i] = at[0];
    s_seg[i] = at[1];
    s_split[i] = nsplit + at[2];
    s_cut[i] = ncut + at[3];
    if (n[3]) a.cuts[ncut + at[3]] = {(int)slot, nsplit + at[2], n[1], resume};
    __syncthreads();
    for (int c = i; c < all[0]; c += 1024) {
      const int k = find(s_chunk, c), r0 = s_t0[k] + (c - s_chunk[k]) * kQ, f = s_slot[k];
      a.chunks[nchunk + c] = {r0, min(s_t1[k], r0 + kQ), s_t0[k], f < 0 ? f & 0x7fffffff : -1};
    }
    for (int g = i; g < all[1]; g += 1024) {
      const int k = find(s_seg, g), nb = (s_t1[k] - s_t0[k] + kQ - 1) / kQ, of = nb ? (nb + a.seg_len - 1) / a.seg_len : 1;
      const int j = g - s_seg[k], lo = (int)((int64_t)nb * j / of), hi = (int)((int64_t)nb * (j + 1) / of);
      a.segs[nseg + g] = {s_slot[k] & 0x7fffffff, s_t0[k], s_t1[k], lo, hi - lo, nchunk + s_chunk[k] + lo,
                          of > 1 ? s_split[k] + j : -1, s_cut[k], s_slot[k] < 0};
    }
    nchunk += all[0];
    nseg += all[1];
    nsplit += all[2];
    ncut += all[3];
    __syncthreads();
  }
  if (i == 0) *a.head = {nseg, nchunk, ncut, 0};
}

// ---- the operands of one block and group
//
// One workgroup each: 9 us for one block of 128 states, which is latency, 21 for 512.
// Every wave of the group reads them: 160 of them at 80 heads of 64 channels.

constexpr int kPrep = 1024;  // threads: one round of loads up to 128 states

template <typename IO, int NT>
__global__ void __launch_bounds__(kPrep) mix_prep_kernel(const BlkArgs a) {
  constexpr int NP = NT * 16, LD = NP + 8;         // row pitch in LDS: 16 bytes more, banks apart
  constexpr int UN = (8 * NP + kPrep - 1) / kPrep;  // (channel, 16 rows) units of a thread
  using O = Ops<NT>;
  __shared__ __align__(16) _Float16 sm[2][2][kQ * LD];  // [B, C][hi, lo]
  __shared__ float red[2][16];
  const Chunk ck = a.chunks[blockIdx.x];  // garbage past the last one, which ends here
  if ((int)blockIdx.x >= a.head->nchunk) return;
  const int g = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int inner = a.H * a.P, W = a.W;
  const bool resume = ck.from >= 0;
  const int64_t slot = ck.from;
  float v[UN][16], mx[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < UN; ++i) {
    const int u = tid + kPrep * i, chn = u % (2 * NP), run = u / (2 * NP), which = chn / NP, n = chn % NP;
    const bool on = n < a.N && run < 4;
    const int c = inner + which * a.G * a.N + g * a.N + (on ? n : 0);
    // rows outside the block or the sequence are read from inside and replaced,
    // so that the loads of all rows are in flight together
    float in[19], w[4];
    const int lo = ck.r0 + 16 * run - 3, top = ck.r1 - 1;
    const float bias = a.cb ? a.cb[c] : 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = a.cw[(int64_t)c * W + max(W - 4 + k, 0)];
#pragma unroll
    for (int j = 0; j < 19; ++j)
      in[j] = ld<IO>(a.xbc, (int64_t)max(min(lo + j, top), ck.t0) * a.xs + c);
#pragma unroll
    for (int j = 0; j < 19; ++j) in[j] = on && lo + j >= ck.t0 && lo + j <= top ? in[j] : 0.0f;
    if (resume && lo < ck.t0 && on) {  // the sequence's first rows: the inputs before it
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (j - 3 + W - 1 >= 0) in[j] = a.conv_state[(slot * a.C + c) * (W - 1) + j - 3 + W - 1];
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) v[i][j] = bias;
#pragma unroll
    for (int k = 3; k >= 0; --k)  // the newest tap first
      if (3 - k < W)
#pragma unroll
        for (int j = 0; j < 16; ++j) v[i][j] = fmaf(w[k], in[j + k], v[i][j]);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float x = on && ck.r0 + 16 * run + j < ck.r1 ? silu(v[i][j]) : 0.0f;
      v[i][j] = x;
      if (finite(x)) mx[which] = fmaxf(mx[which], fabsf(x));
    }
  }
  mx[0] = wave_max(mx[0]);
  mx[1] = wave_max(mx[1]);
  if (lane == 0) red[0][wave] = mx[0], red[1][wave] = mx[1];
  __syncthreads();
  int sh[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
  {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kPrep / 64; ++i) m = fmaxf(m, red[k][i]);
    sh[k] = shift_for(m);
  }
#pragma unroll
  for (int i = 0; i < UN; ++i) {
    const int u = tid + kPrep * i, chn = u % (2 * NP), run = u / (2 * NP), which = chn / NP, n = chn % NP;
    if (run >= 4) continue;
    const float f = two(sh[which]);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float x = v[i][j] * f;
      const _Float16 hi = (_Float16)x;
      sm[which][0][(16 * run + j) * LD + n] = hi;
      sm[which][1][(16 * run + j) * LD + n] = (_Float16)(x - (float)hi);
    }
  }
  __syncthreads();
  char* out = a.ops + ((int64_t)blockIdx.x * a.G + g) * O::bytes;
  // C: lane (t, q) of tile (tt, m) holds n = 32 m + 4 q + {0..3} and 16 more,
  // the order in which the state's accumulators hold n
  for (int u = tid; u < 4 * (NT / 2) * 64; u += kPrep) {
    const int l = u & 63, m = (u >> 6) % (NT / 2), tt = (u >> 6) / (NT / 2);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const _Float16* s = sm[1][p] + (16 * tt + (l & 15)) * LD + 32 * m + 4 * (l >> 4);
      h8 o;
      const h4 x = *reinterpret_cast<const h4*>(s), y = *reinterpret_cast<const h4*>(s + 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = x[j], o[j + 4] = y[j];
      *reinterpret_cast<h8*>(out + O::c + p * O::piece + u * 16) = o;
    }
  }
  // B transposed: lane (n, q) of tile (nt, kb) holds t = 32 kb + 8 q + {0..7}
  for (int u = tid; u < NT * 2 * 64; u += kPrep) {
    const int l = u & 63, kb = (u >> 6) & 1, nt = u >> 7;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const _Float16* s = sm[0][p] + (32 * kb + 8 * (l >> 4)) * LD + 16 * nt + (l & 15);
      h8 o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = s[j * LD];
      *reinterpret_cast<h8*>(out + O::b + p * O::piece + u * 16) = o;
    }
  }
  if (wave >= 4) return;
  // C.B^T: wave w has the rows t of tile w; the rows s of B are taken in the order
  // that leaves lane (t, q) with s = 32 kb + 8 q + {0..7}
  f4 acc[2][2] = {};
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    if (kb > (wave >> 1)) break;
#pragma unroll
    for (int m = 0; m < NT / 2; ++m) {
      h8 cp[2], bp[2][2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        cp[p] = *reinterpret_cast<const h8*>(sm[1][p] + (16 * wave + (lane & 15)) * LD + 32 * m + 8 * (lane >> 4));
#pragma unroll
        for (int e = 0; e < 2; ++e)
          bp[e][p] = *reinterpret_cast<const h8*>(
              sm[0][p] + (32 * kb + 8 * ((lane & 15) >> 2) + 4 * e + (lane & 3)) * LD + 32 * m + 8 * (lane >> 4));
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        acc[kb][e] = mfma(bp[e][1], cp[0], acc[kb][e]);
        acc[kb][e] = mfma(bp[e][0], cp[1], acc[kb][e]);
        acc[kb][e] = mfma(bp[e][0], cp[0], acc[kb][e]);
      }
    }
  }
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    if (kb > (wave >> 1)) break;
    const int tile = wave < 2 ? wave : 2 * wave - 2 + kb;
    f4* o = reinterpret_cast<f4*>(out + O::g + (tile * 64 + lane) * 32);
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // its own size again: D joins it
      f4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = __builtin_amdgcn_ldexpf(acc[kb][e][r], -(sh[0] + sh[1]));
      o[e] = v;
    }
  }
  if (tid < 2) reinterpret_cast<int*>(out + O::scale)[tid] = sh[tid];
}

// ---- the walk over a segment

// Copies BYTES from global memory to LDS, 16 bytes a lane, on their way when it
// returns: arrived() waits for them, meet() for the other waves.
template <int WV, int BYTES>
__device__ __forceinline__ void stage(const char* from, char* to) {
  static_assert(BYTES % 1024 == 0, "whole waves");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < (BYTES / 1024 + WV - 1) / WV; ++i) {
    const int at = (i * WV + wave) * 1024;
    if (BYTES / 1024 % WV == 0 || at < BYTES)
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(from + at + lane * 16),
          (__attribute__((address_space(3))) void*)(to + at), 16, 0, 0);
  }
}
// The first LANES lanes' 16 bytes of a wave, by the first wave.
template <int LANES>
__device__ __forceinline__ void stage_few(const char* from, char* to) {
  if (threadIdx.x < LANES)
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(from + threadIdx.x * 16),
                                     (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}
// All of this wave's memory accesses but the last LEFT have ended.
template <int LEFT>
__device__ __forceinline__ void arrived() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
}
// The waves of the workgroup meet; what is on its way from memory stays so.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The last W - 1 inputs of channel c of a sequence into its slot.
template <typename IO>
__device__ __forceinline__ void keep_inputs(const MixArgs& a, const Seg& sg, int64_t slot, bool resume, int c) {
  const int W = a.W;
  float* own = a.conv_state + (slot * a.C + c) * (W - 1);
  float v[3];
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const int64_t r = (int64_t)sg.t1 - (W - 1) + j;
    v[j] = j >= W - 1 ? 0.0f : r >= sg.t0 ? ld<IO>(a.xbc, r * a.xs + c) : resume ? own[r - sg.t0 + W - 1] : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j < W - 1) own[j] = v[j];
}

// x of a wave's PB channels (bf16) at a block's 64 rows and the three before
// them, in LDS by direct loads of 16 bytes a lane: 1024 bytes at a time hold GP
// groups of eight rows, interleaved row by row so that the four rows that the
// lanes of a wave read together lie in different banks.
template <int PT>
struct XTile {
  static constexpr int RB = 32 * PT, RI = 1024 / RB, GP = RI / 8;  // bytes of a row, rows and groups a load
  static constexpr int step = PT == 2 ? 1152 : 1024, loads = (kQ + 3 + RI - 1) / RI;
  static constexpr int bytes = PT == 2 ? 4928 : loads * step;
  static_assert((loads - 1) * step + ((kQ + 2) % 8 * GP + 1) * RB <= bytes, "the last rows fit");
  // bytes of row 8 a + b
  __device__ static __forceinline__ int at(int a, int b) { return a / GP * step + (GP * b + a % GP) * RB; }
};

// What a wave reads of a block's rows ahead of time where they are not staged:
// x of its channels at rows 32 kb + 8 q - 3 .. + 7, as they lie in memory.
template <typename IO, int PT>
struct XRaw {
  uint32_t w[PT][2][11];
  __device__ __forceinline__ float get(int e, int kb, int j) const {
    if constexpr (sizeof(IO) == 2) return __uint_as_float(w[e][kb][j] << 16);
    else return __uint_as_float(w[e][kb][j]);
  }
};

// One wave per 16 PT channels of a head (PT = 2: channels 2 i and 2 i + 1 of
// its 32 are row i of the two tiles, so that a lane reads x two channels and
// z, y eight channels at a time).  The WV waves of a workgroup share a group
// of heads and its operands in LDS.  A block goes convolution, C.h, M x with y,
// state: C arrives while the waves convolve, B, in C's place, while they work on
// M x, and the next block's C.B^T while they update the state; the next block's x
// and dt come from the convolution's end on.  FAST: rows and channels allow whole
// vectors (headdim a multiple of 4 PT, dstate of 4, rows aligned to the accesses).
//
// Bound by vector instructions and their waits at two waves a SIMD, which the state (64
// registers) and the operands of x force: four prompts of 8192 with 80 heads of 64
// channels and 128 states take 686 us in the second pass and 176 in the first, of a call of
// 910 (on one card, traced; 895 to 910 on others).  A wave and block of the second is 2905
// vector instructions, 228 of them products: the vector units are busy 64 % of the
// time, the matrix cores 19 %, and a wave waits 29 % of its own (247 registers, 70 KB of
// LDS a workgroup).  B and C by turns in one place leave room for two workgroups of four
// waves a CU at 128 states; both at once, one workgroup of eight, took 2 % more there and
// 12 % more for 16 ragged prompts of 8111 tokens.  Past 128 states a wave has 16 channels
// instead of 32, so that its state stays at 64 registers.  Rows that are not on 16
// bytes go through the general kernel, which reads x element by element and spills at
// 128 states: 1621 us against 919.
template <typename IO, int NT, int PT, int WV, bool SUM, bool FAST>
__global__ void __launch_bounds__(64 * WV) __attribute__((amdgpu_waves_per_eu(2)))
mix_block_kernel(const BlkArgs a) {
  using O = Ops<NT>;
  constexpr int PB = 16 * PT;  // channels of a wave
  __shared__ __align__(16) char s_bc[2 * O::piece];  // C, then B
  __shared__ __align__(16) char s_g[SUM ? 16 : O::gsize];
  constexpr bool XLDS = FAST && sizeof(IO) == 2;
  using X = XTile<PT>;
  __shared__ __align__(16) char s_x[XLDS ? WV * X::bytes : 16];
  __shared__ __align__(16) int s_sc[2][4];
  __shared__ __align__(16) float s_w[WV][64];
  // for y alone
  __shared__ __align__(16) float s_cum[SUM ? 1 : WV][SUM ? 4 : 64], s_low[SUM ? 1 : WV][SUM ? 4 : 64];
  __shared__ __align__(16) float s_dt[SUM ? 1 : WV][SUM ? 4 : 64];
  __shared__ __align__(16) int s_ex[SUM ? 1 : WV][2][SUM ? 4 : PB];  // shifts of x and of the state, by channel
  __shared__ int s_bad[SUM ? 1 : WV][SUM ? 4 : PB];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int i16 = lane & 15, q4 = lane >> 4;
  const int sub = SUM ? a.sub : 1;
  const int si = blockIdx.x / (a.units * sub), unit = blockIdx.x % a.units;
  Seg sg = a.segs[si];  // garbage past the last one, which ends here
  if (si >= a.head->nseg) return;
  if (SUM && (sg.split < 0 || sg.c0 + sg.nc == (sg.t1 - sg.t0 + kQ - 1) / kQ)) return;  // no state asked
  const int piece_of = SUM ? (int)(blockIdx.x / a.units) % sub : 0;
  if constexpr (SUM) {  // a piece of the segment's blocks
    const int lo = sg.nc * piece_of / sub, hi = sg.nc * (piece_of + 1) / sub;
    sg.c0 += lo;
    sg.gc += lo;
    sg.nc = hi - lo;
  }
  const int g = unit / a.per_group, hpg = a.H / a.G, bph = (a.P + PB - 1) / PB;
  const int blk = (unit % a.per_group) * WV + wave;
  const bool on = blk < hpg * bph;  // else the wave only helps to stage
  const bool last = sg.t0 + (int64_t)(sg.c0 + sg.nc) * kQ >= sg.t1;
  const int inner = a.H * a.P, W = a.W, N = a.N;
  const bool resume = sg.resume;
  const int64_t slot = sg.slot;
  // the last inputs of B and C into the slot: nobody reads the old ones any more
  if (!SUM && last && a.state && W > 1 && unit % a.per_group == 0) {
    for (int u = threadIdx.x; u < 2 * N; u += 64 * WV)
      keep_inputs<IO>(a, sg, slot, resume, inner + (u / N) * a.G * N + g * N + u % N);
  }
  const int h = on ? g * hpg + blk / bph : 0, p0 = on ? (blk % bph) * PB : 0;
  // this lane's channels as rows of the tiles; past the head's last one a copy of a valid one
  int ch[PT];
#pragma unroll
  for (int e = 0; e < PT; ++e) {
    const int p = p0 + PT * i16 + e;
    ch[e] = h * a.P + (p < a.P ? p : FAST ? p0 + e : e && p - 1 < a.P ? p - 1 : p0);
  }
  float cw[PT][4], cb[PT];
#pragma unroll
  for (int e = 0; e < PT; ++e) {
    cb[e] = a.cb ? a.cb[ch[e]] : 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) cw[e][k] = k < W ? a.cw[(int64_t)ch[e] * W + (W - 1) - k] : 0.0f;  // k rows back
  }
  const float A2 = a.A[h] * kLog2e, db = a.dt_bias ? a.dt_bias[h] : 0.0f, D = a.Dskip ? a.Dskip[h] : 0.0f;

  // the state entering the segment: lane (i, q) holds n = 16 nt + 4 q + r of its channels
  f4 S[PT][NT];
  {
    const float* src = nullptr;
    // a cut sequence's first segment too has its start in `local`: the last one writes the slot in this same launch
    if (sg.split >= 0) src = SUM ? nullptr : a.local + (int64_t)sg.split * a.sub * inner * N;
    else if (!SUM && resume) src = a.state + slot * inner * N;
#pragma unroll
    for (int e = 0; e < PT; ++e)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        const int n = 16 * nt + 4 * q4;
        if (src) {
          const float* s = src + (int64_t)ch[e] * N + n;
          if constexpr (FAST) {
            if (n < N) v = *reinterpret_cast<const f4*>(s);
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (n + r < N) v[r] = s[r];
          }
        }
        S[e][nt] = v;
      }
  }
  double dsum = 0.0;  // log2 of the segment's decay

  // a block's x and dt, and its z, on their way
  XRaw<IO, PT> xr;
  float dt_raw = 0.0f;
  typedef uint32_t zv __attribute__((ext_vector_type(2 * PT)));
  constexpr bool ZAHEAD = FAST && !SUM && sizeof(IO) == 2;
  zv zr[4];
  auto fetch = [&](int c) {
    const int r0 = sg.t0 + (sg.c0 + c) * kQ, r1 = min(sg.t1, r0 + kQ);
    // rows outside the sequence are read from inside it and replaced later
    if constexpr (XLDS) {
#pragma unroll
      for (int i = 0; i < X::loads; ++i) {
        const int slot = lane / (X::RB / 16), row = X::RI * i + 8 * (slot % X::GP) + slot / X::GP;
        if (i + 1 < X::loads || row < kQ + 3) {
          const int64_t r = max(min(r0 + row - 3, r1 - 1), sg.t0);
          __builtin_amdgcn_global_load_lds(
              (const __attribute__((address_space(1))) void*)(static_cast<const IO*>(a.xbc) + r * a.xs + h * a.P +
                                                              p0 + lane % (X::RB / 16) * 8),
              (__attribute__((address_space(3))) void*)(s_x + wave * X::bytes + i * X::step), 16, 0, 0);
        }
      }
    } else {
      const int first = r0 + 8 * q4 - 3;
      const IO* base = static_cast<const IO*>(a.xbc) + ch[0];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int j = 0; j < 11; ++j) {
          const IO* x = base + (int64_t)max(min(first + 32 * kb + j, r1 - 1), sg.t0) * a.xs;
          if constexpr (FAST && PT == 2) {
            const u2 w = *reinterpret_cast<const u2*>(x);
            xr.w[0][kb][j] = w.x;
            xr.w[1][kb][j] = w.y;
          } else {
#pragma unroll
            for (int e = 0; e < PT; ++e) {
              if constexpr (sizeof(IO) == 2) xr.w[e][kb][j] = x[ch[e] - ch[0]];
              else xr.w[e][kb][j] = __float_as_uint(x[ch[e] - ch[0]]);
            }
          }
        }
    }
    dt_raw = ld<IO>(a.dt, (int64_t)min(r0 + lane, r1 - 1) * a.ds + h);
  };
  auto fetch_z = [&](int c) {
    if constexpr (ZAHEAD) {
      const int r0 = sg.t0 + (sg.c0 + c) * kQ, r1 = min(sg.t1, r0 + kQ), pw = p0 + 4 * PT * q4;
      const IO* base = static_cast<const IO*>(a.z) + h * a.P + (pw < a.P ? pw : p0);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
        zr[tt] = *reinterpret_cast<const zv*>(base + (int64_t)min(r0 + 16 * tt + i16, r1 - 1) * a.zs);
    }
  };
  const char* op = a.ops + ((int64_t)sg.gc * a.G + g) * O::bytes;
  const int64_t op_step = (int64_t)a.G * O::bytes;
  auto stage_b = [&] { stage<WV, 2 * O::piece>(op + O::b, s_bc); };
  auto stage_c = [&] { stage<WV, 2 * O::piece>(op + O::c, s_bc); };
  auto stage_scales = [&](const char* from, int at) {
    stage_few<1>(from + O::scale, reinterpret_cast<char*>(s_sc[at]));
  };
  auto stage_g = [&](const char* from, int at) {
    stage<WV, O::gsize>(from + O::g, s_g);
    stage_scales(from, at);
  };
  if (sg.nc > 0) {
    if (on) fetch(0);
    if constexpr (!SUM) stage_g(op, 0);
  }

  for (int c = 0; c < sg.nc; ++c) {
    const int r0 = sg.t0 + (sg.c0 + c) * kQ, r1 = min(sg.t1, r0 + kQ), cnt = r1 - r0;
    // places in LDS are computed from the lane in every turn: kept all through, they cost registers
    int here = threadIdx.x & 63;
    asm volatile("" : "+v"(here));
    const int lane = here, i16 = here & 15, q4 = here >> 4;
    arrived<0>();
    meet();  // x, dt and C.B^T are there; the waves are done with the last block's B
    if constexpr (SUM) {
      stage_b();
      stage_scales(op, 0);
    } else {
      stage_c();
    }
    h8 xh[PT][2], xl[PT][2];  // x as an operand; then, and at once in the first pass, weighted for the state
    float dec_all = 1.0f;
    int shx[PT] = {}, shw = 0;
    bool bad = false;
    if (on) {
      // ---- the convolution
      float v[PT][2][8];
      {
        float in[PT][2][11];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int j = 0; j < 11; ++j) {
            if constexpr (XLDS) {
              const char* x = s_x + wave * X::bytes + X::at(4 * kb + q4 + (j >> 3), j & 7) + i16 * 2 * PT;
              if constexpr (PT == 2) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(x);
                in[0][kb][j] = __uint_as_float(w << 16);
                in[1][kb][j] = __uint_as_float(w & 0xffff0000u);
              } else {
                in[0][kb][j] = __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t*>(x) << 16);
              }
            } else {
#pragma unroll
              for (int e = 0; e < PT; ++e) in[e][kb][j] = xr.get(e, kb, j);
            }
          }
        const bool first = sg.c0 + c == 0;
        if (first || cnt < kQ) {
          int first_row = r0;
          asm volatile("" : "+s"(first_row));  // keeps these comparisons in this branch
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int j = 0; j < 11; ++j) {
              const int r = first_row + 32 * kb + 8 * q4 + j - 3;
#pragma unroll
              for (int e = 0; e < PT; ++e) in[e][kb][j] = r >= sg.t0 && r < r1 ? in[e][kb][j] : 0.0f;
            }
          if (first && resume && W > 1 && q4 == 0) {  // the inputs before the sequence
            const bool saved = !SUM && sg.split >= 0;
#pragma unroll
            for (int e = 0; e < PT; ++e)
#pragma unroll
              for (int j = 0; j < 3; ++j) {
                const int at = j - 3 + W - 1;
                if (at >= 0)
                  in[e][0][j] = saved ? a.cs0[((int64_t)sg.cut * inner + ch[e]) * 3 + at]
                                      : a.conv_state[(slot * a.C + ch[e]) * (W - 1) + at];
              }
            if constexpr (SUM) {  // the second pass overwrites the slot: it reads these
#pragma unroll
              for (int e = 0; e < PT; ++e)
                if (p0 + PT * i16 + e < a.P)
#pragma unroll
                  for (int j = 0; j < 3; ++j)
                    if (j - 3 + W - 1 >= 0)
                      a.cs0[((int64_t)sg.cut * inner + ch[e]) * 3 + j - 3 + W - 1] = in[e][0][j];
            }
          }
        }
#pragma unroll
        for (int e = 0; e < PT; ++e)
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[e][kb][j] = fmaf(cw[e][0], in[e][kb][j + 3], cb[e]);
#pragma unroll
        for (int k = 1; k < 4; ++k)
          if (k < W)
#pragma unroll
            for (int e = 0; e < PT; ++e)
#pragma unroll
              for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[e][kb][j] = fmaf(cw[e][k], in[e][kb][j + 3 - k], v[e][kb][j]);
      }
      // ---- steps: lane t
      const bool live = lane < cnt;
      float dt = 0.0f, dA = 0.0f;
      if (live) {
        const float raw = dt_raw + db;
        dt = a.softplus ? softplus(raw) : raw;
        // below 2^-160 a decay is zero in float32; held there, no sum swallows the steps beside it
        dA = dt * A2;
        dA = dA < -160.0f ? -160.0f : dA;
        if (!finite(dt)) dA = __builtin_nanf("");  // and all after it
      }
      const double cum = wave_scan((double)dA), tot = lane63(cum);
      const float wt = dt * ex2((float)(tot - cum));
      dec_all = ex2((float)tot);
      dsum += tot;
      // what float32 leaves off a running sum goes with the step and with y's row, as a factor
      const float low = (float)(cum - (double)(float)cum);
      if constexpr (!SUM) s_cum[wave][lane] = (float)cum, s_low[wave][lane] = ex2(low);
      // the state's weights exp(c_Q - c_s) dt_s, by their own largest one
      shw = shift_for(wave_max(finite(wt) ? fabsf(wt) : 0.0f)) - 15;
      s_w[wave][lane] = wt * two(shw);
      if constexpr (!SUM) s_dt[wave][lane] = dt * ex2(-low);
      // ---- silu, every channel's scale
      float mx[PT] = {};
#pragma unroll
      for (int e = 0; e < PT; ++e)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = silu(v[e][kb][j]);
            v[e][kb][j] = x;
          }
#pragma unroll
      for (int e = 0; e < PT; ++e)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int j = 0; j < 8; j += 2) mx[e] = max3_nan(mx[e], v[e][kb][j], v[e][kb][j + 1]);
      // this block's x is used up: the next one's may come (the staged operand's loads have ended by now)
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      if (a.z) fetch_z(c);
      if (c + 1 < sg.nc) fetch(c + 1);
      if (cnt < kQ) {
        rarely();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < PT; ++e) v[e][kb][j] = 32 * kb + 8 * q4 + j < cnt ? v[e][kb][j] : 0.0f;
      }
      bad = __any(!(finite(mx[0]) && finite(mx[PT - 1])));
      if (bad) {
        rarely();
#pragma unroll
        for (int e = 0; e < PT; ++e) {
          int first = kQ;
          mx[e] = 0.0f;
#pragma unroll
          for (int kb = 1; kb >= 0; --kb)
#pragma unroll
            for (int j = 7; j >= 0; --j) {
              if (finite(v[e][kb][j])) mx[e] = fmaxf(mx[e], fabsf(v[e][kb][j]));
              else first = 32 * kb + 8 * q4 + j;
            }
          first = min(first, __shfl_xor(first, 16, 64));
          first = min(first, __shfl_xor(first, 32, 64));
          if constexpr (!SUM)
            if (q4 == 0) s_bad[wave][PT * i16 + e] = first;
        }
      }
      float fx[PT];
#pragma unroll
      for (int e = 0; e < PT; ++e) {
        shx[e] = shift_for(row_max(mx[e]));
        fx[e] = two(shx[e]);
        if constexpr (!SUM)
          if (q4 == 0) s_ex[wave][0][PT * i16 + e] = shx[e];
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int e = 0; e < PT; ++e) {
          if (!SUM && bad) {  // 0 x Inf is not 0: y's earlier rows must not meet them
            rarely();
#pragma unroll
            for (int j = 0; j < 8; ++j) v[e][kb][j] = finite(v[e][kb][j]) ? v[e][kb][j] : 0.0f;
          }
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = v[e][kb][j] * fx[e];
          if constexpr (SUM) {
            float w8[8];
            *reinterpret_cast<f4*>(w8) = *reinterpret_cast<const f4*>(&s_w[wave][32 * kb + 8 * q4]);
            *reinterpret_cast<f4*>(w8 + 4) = *reinterpret_cast<const f4*>(&s_w[wave][32 * kb + 8 * q4 + 4]);
            pieces(x, w8, xh[e][kb], xl[e][kb]);
          } else {
            pieces(x, xh[e][kb], xl[e][kb]);
          }
        }
    } else {
      arrived<0>();
    }
    if constexpr (!SUM) {
      meet();  // C is there
      f4 yc[4][PT] = {};
      if (on) {
        // ---- C.h for all rows: the state's pieces are made once and kept no longer than their products
        float fs[PT];
#pragma unroll
        for (int e = 0; e < PT; ++e) {
          float sm = 0.0f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; r += 2) sm = max3(sm, S[e][nt][r], S[e][nt][r + 1]);
          if (__any(!finite(sm))) {
            rarely();
            sm = 0.0f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (finite(S[e][nt][r])) sm = fmaxf(sm, fabsf(S[e][nt][r]));
          }
          const int shS = shift_for(row_max(sm));
          fs[e] = two(shS);
          if (q4 == 0) s_ex[wave][1][PT * i16 + e] = shS;
        }
#pragma unroll
        for (int m = 0; m < NT / 2; ++m) {
          h8 sh[PT], sl[PT];
#pragma unroll
          for (int e = 0; e < PT; ++e) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = S[e][2 * m + (j >> 2)][j & 3] * fs[e];
            pieces(x, sh[e], sl[e]);
          }
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) {
            const char* cq = s_bc + ((tt * (NT / 2) + m) * 64 + lane) * 16;
            const h8 ch = *reinterpret_cast<const h8*>(cq), cl = *reinterpret_cast<const h8*>(cq + O::piece);
#pragma unroll
            for (int e = 0; e < PT; ++e) {
              yc[tt][e] = mfma(sl[e], ch, yc[tt][e]);
              yc[tt][e] = mfma(sh[e], cl, yc[tt][e]);
              yc[tt][e] = mfma(sh[e], ch, yc[tt][e]);
            }
          }
        }
        // back from the channels' and C's scales; lane (t, q) has the channels 4 PT q + {0 .. 4 PT - 1}
        const int shC = __builtin_amdgcn_readfirstlane(s_sc[c & 1][1]);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int k = 0; k < 4 * PT; ++k) {
          const float f = two(min(127, -(shC + s_ex[wave][1][4 * PT * q4 + k])));
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) yc[tt][k % PT][k / PT] *= f;
        }
      }
      meet();  // the waves are done with C
      stage_b();
      asm volatile("" ::: "memory");  // the stores of y stay behind these loads: arrived<4>() counts on it
      if (on) {
        // ---- M x and y, 16 rows at a time
        float f_x[4 * PT];
#pragma unroll
        for (int k = 0; k < 4 * PT; ++k) f_x[k] = two(-s_ex[wave][0][4 * PT * q4 + k]);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          if (16 * tt >= cnt) break;
          const int t = 16 * tt + i16;
          const float cum_t = s_cum[wave][t], low_t = s_low[wave][t];
          const float Dm = D * rcp(low_t);
          f4 ym[PT] = {};
          int tq = t, s0 = 8 * q4;
          asm volatile("" : "+v"(tq), "+v"(s0));  // else the causal masks of all tiles are kept in registers
          float m[2][8], rm = 0.0f;
#pragma unroll
          for (int kb = 0; kb <= tt / 2; ++kb) {
            const int tile = tt < 2 ? tt : 2 * tt - 2 + kb;
            const f4* gp = reinterpret_cast<const f4*>(s_g + (tile * 64 + lane) * 32);
            float g[8], cs[8], ds[8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              *reinterpret_cast<f4*>(g + 4 * k) = gp[k];
              *reinterpret_cast<f4*>(cs + 4 * k) = *reinterpret_cast<const f4*>(&s_cum[wave][32 * kb + 8 * q4 + 4 * k]);
              *reinterpret_cast<f4*>(ds + 4 * k) = *reinterpret_cast<const f4*>(&s_dt[wave][32 * kb + 8 * q4 + 4 * k]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int s = 32 * kb + s0 + j;
              float x = g[j] * (ex2(cum_t - cs[j]) * ds[j]);
              if (kb == tt / 2) {
                x = s <= tq ? x : 0.0f;
                x = s == tq ? x + Dm : x;
              }
              m[kb][j] = x;
            }
#pragma unroll
            for (int j = 0; j < 8; j += 2) rm = max3(rm, m[kb][j], m[kb][j + 1]);
          }
          // every row by its own largest value: one token's outlier leaves the others their bits
          const int shM = shift_for(row_max(rm));
          const float fm = two(shM);
#pragma unroll
          for (int kb = 0; kb <= tt / 2; ++kb) {
#pragma unroll
            for (int j = 0; j < 8; ++j) m[kb][j] *= fm;
            h8 mh, ml;
            pieces(m[kb], mh, ml);
#pragma unroll
            for (int e = 0; e < PT; ++e) {
              ym[e] = mfma(xl[e][kb], mh, ym[e]);
              ym[e] = mfma(xh[e][kb], ml, ym[e]);
              ym[e] = mfma(xh[e][kb], mh, ym[e]);
            }
          }
          // lane (t, q): channels p0 + 4 PT q + {0 .. 4 PT - 1}
          const float f_cs = ex2(cum_t) * low_t, f_mx = __builtin_amdgcn_ldexpf(low_t, -shM);
          const int pw = p0 + 4 * PT * q4;
          const int64_t row = (int64_t)r0 + t, col = (int64_t)h * a.P + pw;
          float o[4 * PT];
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < PT; ++e)
              o[PT * r + e] = fmaf(ym[e][r] * f_x[PT * r + e], f_mx, yc[tt][e][r] * f_cs);
          if (bad) {
            rarely();
#pragma unroll
            for (int k = 0; k < 4 * PT; ++k) o[k] = t >= s_bad[wave][4 * PT * q4 + k] ? __builtin_nanf("") : o[k];
          }
          if (a.z) {
            if constexpr (ZAHEAD) {
#pragma unroll
              for (int k = 0; k < 2 * PT; ++k) {
                o[2 * k] *= silu(__uint_as_float(zr[tt][k] << 16));
                o[2 * k + 1] *= silu(__uint_as_float(zr[tt][k] & 0xffff0000u));
              }
            } else if constexpr (FAST) {
              if (t < cnt && pw < a.P) {
                float zz[4 * PT];
#pragma unroll
                for (int k = 0; k < PT; ++k)
                  *reinterpret_cast<f4*>(zz + 4 * k) = *reinterpret_cast<const f4*>(
                      static_cast<const float*>(a.z) + row * a.zs + col + 4 * k);
#pragma unroll
                for (int k = 0; k < 4 * PT; ++k) o[k] *= silu(zz[k]);
              }
            } else if (t < cnt) {
#pragma unroll
              for (int k = 0; k < 4 * PT; ++k)
                if (pw + k < a.P) o[k] *= silu(ld<IO>(a.z, row * a.zs + col + k));
            }
          }
          if (t < cnt) {
            if constexpr (FAST) {
              if (pw < a.P) {
                if constexpr (sizeof(IO) == 4) {
#pragma unroll
                  for (int k = 0; k < PT; ++k)
                    *reinterpret_cast<f4*>(static_cast<float*>(a.y) + row * a.ys + col + 4 * k) =
                        *reinterpret_cast<const f4*>(o + 4 * k);
                } else {
                  typedef __bf16 bf __attribute__((ext_vector_type(4 * PT)));
                  typedef float fv __attribute__((ext_vector_type(4 * PT)));
                  fv f;
#pragma unroll
                  for (int k = 0; k < 4 * PT; ++k) f[k] = o[k];
                  *reinterpret_cast<bf*>(static_cast<uint16_t*>(a.y) + row * a.ys + col) =
                      __builtin_convertvector(f, bf);
                }
              }
            } else {
#pragma unroll
              for (int k = 0; k < 4 * PT; ++k)
                if (pw + k < a.P) st<IO>(a.y, row * a.ys + col + k, o[k]);
            }
          }
        }
      }
      // B's loads have ended where at most the stores behind them are left: four at least
      // of a whole block's wave
      if (on && cnt == kQ) arrived<4>();
      else arrived<0>();
      meet();  // B is there; the waves are done with C.B^T
      if (c + 1 < sg.nc) stage_g(op + op_step, (c + 1) & 1);
    } else {
      meet();  // B is there
    }
    if (on) {  // ---- the state after the block
      if constexpr (!SUM) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          float w8[8];
          *reinterpret_cast<f4*>(w8) = *reinterpret_cast<const f4*>(&s_w[wave][32 * kb + 8 * q4]);
          *reinterpret_cast<f4*>(w8 + 4) = *reinterpret_cast<const f4*>(&s_w[wave][32 * kb + 8 * q4 + 4]);
#pragma unroll
          for (int e = 0; e < PT; ++e) {
            float x[8];
            joined(xh[e][kb], xl[e][kb], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= w8[j];
            if (bad) {  // a channel whose x was not finite has no state any more
              rarely();
              if (s_bad[wave][PT * i16 + e] < kQ)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = __builtin_nanf("");
            }
            pieces(x, xh[e][kb], xl[e][kb]);
          }
        }
      }
      const int shB = __builtin_amdgcn_readfirstlane(s_sc[SUM ? 0 : c & 1][0]);
      float f_su[PT];
#pragma unroll
      for (int e = 0; e < PT; ++e) f_su[e] = two(min(127, -(shB + shw + shx[e])));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        h8 bh[2], bl[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          bh[kb] = *reinterpret_cast<const h8*>(s_bc + ((nt * 2 + kb) * 64 + lane) * 16);
          bl[kb] = *reinterpret_cast<const h8*>(s_bc + O::piece + ((nt * 2 + kb) * 64 + lane) * 16);
        }
#pragma unroll
        for (int e = 0; e < PT; ++e) {
          f4 d = {};
#pragma unroll
          for (int kb = 0; kb < 2; ++kb) {
            d = mfma(bh[kb], xl[e][kb], d);
            d = mfma(bl[kb], xh[e][kb], d);
            d = mfma(bh[kb], xh[e][kb], d);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r)
            S[e][nt][r] = fmaf(d[r], f_su[e], S[e][nt][r] * dec_all);
        }
      }
    }
    op += op_step;
  }
  if (!on) return;

  // ---- what the segment leaves
  float* dst = nullptr;
  if constexpr (SUM) {
    const int64_t at = (int64_t)sg.split * sub + piece_of;
    dst = a.local + at * inner * N;
    if (lane == 0 && p0 == 0) a.decay[at * a.H + h] = (float)dsum;
  } else {
    if (last && a.state) dst = a.state + slot * inner * N;
  }
  if (dst) {
#pragma unroll
    for (int e = 0; e < PT; ++e)
      if (p0 + PT * i16 + e < a.P)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int n = 16 * nt + 4 * q4;
          float* s = dst + (int64_t)ch[e] * N + n;
          if constexpr (FAST) {
            if (n < N) *reinterpret_cast<f4*>(s) = S[e][nt];
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (n + r < N) s[r] = S[e][nt][r];
          }
        }
  }
  // the last inputs of the wave's own channels (read by nobody else, or saved by the first pass)
  if (!SUM && last && a.state && W > 1 && lane < PB && p0 + lane < a.P)
    keep_inputs<IO>(a, sg, slot, resume, h * a.P + p0 + lane);
}

// ---- the states entering the segments of a cut sequence, from their states from zero

// One pass over them, read and written once; four values a thread, four
// segments of each on their way together (four cut sequences, twelve segments of 2.6 MB
// in pieces: 21 us).  The parts of a state are neighbours in
// the grid: with the cut sequences innermost, one cut sequence of eight planned for
// ran on one of the eight dies (576 tokens, 80 heads: 40 us against 12).
__global__ void __launch_bounds__(256) mix_join_kernel(const BlkArgs a) {
  if ((int)blockIdx.y >= a.head->ncut) return;
  const Cut ct = a.cuts[blockIdx.y];
  const int64_t per = (int64_t)a.H * a.P * a.N;
  const int hs = a.P * a.N;  // values of a head
  const bool resume = ct.resume;
  const int64_t slot = ct.slot;
  const int sub = a.sub, last = (ct.nseg - 1) * sub;  // nothing enters a segment from the last one
  const float* d = a.decay + (int64_t)ct.split * sub * a.H;
  constexpr int V = 4, K = 4;
  int64_t at[V];
  int h[V];
  float s[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    at[v] = ((int64_t)blockIdx.x * V + v) * 256 + threadIdx.x;
    if (at[v] >= per) at[v] = per;
    h[v] = at[v] < per ? (int)(at[v] / hs) : 0;
    s[v] = resume && at[v] < per ? a.state[slot * per + at[v]] : 0.0f;
  }
  float* l = a.local + (int64_t)ct.split * sub * per;
  for (int k0 = 0; k0 < last; k0 += K) {
    float own[K][V], dec[K][V];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int k = min(k0 + j, last - 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        own[j][v] = l[k * per + (at[v] < per ? at[v] : 0)];
        dec[j][v] = d[(int64_t)k * a.H + h[v]];
      }
    }
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (k0 + j < last)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if ((k0 + j) % sub == 0 && at[v] < per) l[(k0 + j) * per + at[v]] = s[v];
          s[v] = fmaf(s[v], ex2(dec[j][v]), own[j][v]);
        }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (at[v] < per) l[last * per + at[v]] = s[v];
}

// ---------------------------------------------------------------- one token a sequence
//
// h' = exp(dt A) h + dt x B^T, y = h' C + D x: the state is read and written
// once, which is all the time there is.  A workgroup owns rows (channels) of one
// head of one entry, LN lanes a row with four states each, and RPL rows after
// one another whose loads go out first; meanwhile it makes B, C (again in every
// workgroup of a group: 4 KB from the cache beside 64 KB of state) and its x
// from the convolution's inputs.  253 tokens of 80 heads, 64 channels and 128 states take
// 274 us: 4.97 TB/s, what a large copy reaches.

// Sum over the LN lanes of a row.
template <int LN>
__device__ __forceinline__ float lane_sum(float v) {
  auto add = [&](int o) { v += __int_as_float(o); };
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xf, 0xf, true));
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xf, 0xf, true));
  if constexpr (LN >= 8) add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, true));
  if constexpr (LN >= 16) add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xf, 0xf, true));
  if constexpr (LN >= 32) {
    const u2 w = __builtin_bit_cast(u2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    v = __uint_as_float(w.x) + __uint_as_float(w.y);
  }
  if constexpr (LN >= 64) {
    const u2 w = __builtin_bit_cast(u2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    v = __uint_as_float(w.x) + __uint_as_float(w.y);
  }
  return v;
}

// VEC: a lane's states are neighbours (dstate a multiple of 4, the states on 16
// bytes); else they are 64 apart, any dstate.
template <typename IO, int LN, int RPL, bool VEC>
__global__ void __launch_bounds__(256) mix_step_kernel(const MixArgs a, int splits) {
  constexpr int RW = 256 / LN, ROWS = RW * RPL;
  static_assert(VEC || LN == 64, "four states a lane, 64 apart");
  __shared__ __align__(16) float s_bc[2][kMaxN];
  __shared__ float s_x[ROWS], s_y[ROWS];
  const int tid = threadIdx.x, ln = tid % LN, rg = tid / LN;
  const int64_t row = blockIdx.x / ((int64_t)a.H * splits);
  const int hs = (int)(blockIdx.x - row * a.H * splits), h = hs / splits, p0 = (hs - h * splits) * ROWS;
  const int64_t slot = a.slots ? (int64_t)a.slots[row] : row;
  if (slot < 0 || slot >= a.nslots) return;  // padding
  const int N = a.N, g = h / (a.H / a.G), inner = a.H * a.P, W = a.W;
  float* own = a.state + ((slot * a.H + h) * a.P + p0) * (int64_t)N;
  f4 hst[RPL];
#pragma unroll
  for (int i = 0; i < RPL; ++i) {
    const int p = rg + RW * i;
    hst[i] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (p0 + p < a.P) {
      if constexpr (VEC) {
        if (4 * ln < N) hst[i] = *reinterpret_cast<const f4*>(own + (int64_t)p * N + 4 * ln);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (ln + 64 * j < N) hst[i][j] = own[(int64_t)p * N + ln + 64 * j];
      }
    }
  }
  const float raw = ld<IO>(a.dt, row * a.ds + h) + (a.dt_bias ? a.dt_bias[h] : 0.0f);
  const float dt = a.softplus ? softplus(raw) : raw;
  const float e = ex2(dt * a.A[h] * kLog2e);
  for (int u = tid; u < 2 * N + ROWS; u += 256) {
    const int which = u < N ? 0 : u < 2 * N ? 1 : 2, n = u - (which < 2 ? which * N : 2 * N);
    if (which == 2 && p0 + n >= a.P) break;
    const int c = which == 2 ? h * a.P + p0 + n : inner + which * a.G * N + g * N + n;
    float in[4], w[4];
    float* st = a.conv_state + (slot * a.C + c) * (int64_t)(W - 1);
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // k: inputs before this one
      in[k] = k == 0 ? ld<IO>(a.xbc, row * a.xs + c) : k < W ? st[W - 1 - k] : 0.0f;
      w[k] = k < W ? a.cw[(int64_t)c * W + W - 1 - k] : 0.0f;
    }
    float v = a.cb ? a.cb[c] : 0.0f;
#pragma unroll
    for (int k = 3; k >= 0; --k)
      if (k < W) v = fmaf(w[k], in[k], v);
    v = silu(v);
    if (which < 2) {
      s_bc[which][n] = v;
    } else {
      s_x[n] = v;  // and this channel's inputs move on by one: nobody else reads them
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k < W - 1) st[W - 2 - k] = in[k];
    }
  }
  __syncthreads();
  float B[4], C[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = VEC ? 4 * ln + j : ln + 64 * j;
    B[j] = n < N ? s_bc[0][n] : 0.0f;
    C[j] = n < N ? s_bc[1][n] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < RPL; ++i) {
    const int p = rg + RW * i;
    const bool in = p0 + p < a.P;
    const float wx = in ? dt * s_x[p] : 0.0f;
    float acc = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hst[i][j] = fmaf(e, hst[i][j], wx * B[j]);
      acc = fmaf(C[j], hst[i][j], acc);
    }
    if (in) {
      if constexpr (VEC) {
        if (4 * ln < N) *reinterpret_cast<f4*>(own + (int64_t)p * N + 4 * ln) = hst[i];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (ln + 64 * j < N) own[(int64_t)p * N + ln + 64 * j] = hst[i][j];
      }
    }
    acc = lane_sum<LN>(acc);
    if (ln == 0) s_y[p] = acc;
  }
  __syncthreads();
  for (int p = tid; p < ROWS; p += 256) {
    if (p0 + p >= a.P) break;
    const int64_t j = (int64_t)h * a.P + p0 + p;
    float v = s_y[p];
    if (a.Dskip) v = fmaf(a.Dskip[h], s_x[p], v);
    if (a.z) v *= silu(ld<IO>(a.z, row * a.zs + j));
    st<IO>(a.y, row * a.ys + j, v);
  }
}

// The inputs of B and C move on by one, after every reader of the old ones.
template <typename IO>
__global__ void __launch_bounds__(256) mix_step_conv_kernel(const MixArgs a) {
  const int64_t row = blockIdx.x;
  const int c = a.H * a.P + blockIdx.y * 256 + threadIdx.x, W = a.W;
  const int64_t slot = a.slots ? (int64_t)a.slots[row] : row;
  if (c >= a.C || slot < 0 || slot >= a.nslots) return;
  float* st = a.conv_state + (slot * a.C + c) * (int64_t)(W - 1);
  float v[3];
#pragma unroll
  for (int j = 0; j < 3; ++j) v[j] = j + 1 < W - 1 ? st[j + 1] : j + 1 == W - 1 ? ld<IO>(a.xbc, row * a.xs + c) : 0.0f;
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j < W - 1) st[j] = v[j];
}

// ---------------------------------------------------------------- group norm

struct NormArgs {
  const void* x;
  const void* z;
  const void* dy;
  const float* w;
  const float* b;
  void* y;   // forward output, or dx
  void* dz;
  float* pw;  // the strips' sums of dweight, dbias [strips, C], or NULL
  float* pb;
  int strips;
  int64_t xs, zs, gs, ys, dzs;  // row strides; gs of dy
  int64_t rows;
  int C, G;
  float eps;
  int center, act, gate;
};

// A group is held in the registers of a team of TL threads, thread i with
// vectors i, i + TL, .. (K at most) of VE channels each: one pass over the
// rows, the statistics in two steps over registers (mean, then the squares
// around it), so nothing cancels.  Bound by memory (32768 rows of 5120 bf16 with a
// gate: 189 us, 5.3 TB/s).  VE is 16 bytes' worth where the rows and the
// groups allow it and one element elsewhere.

template <typename IO, int VE>
struct Vec {
  static constexpr int words = VE * (int)sizeof(IO) < 4 ? 1 : VE * (int)sizeof(IO) / 4;
  uint32_t w[words];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (VE > 1) {
      const u4 v = *reinterpret_cast<const u4*>(static_cast<const IO*>(p) + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = v[k];
    } else if constexpr (sizeof(IO) == 2) {
      w[0] = static_cast<const uint16_t*>(p)[i];
    } else {
      w[0] = static_cast<const uint32_t*>(p)[i];
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(IO) == 4) return __uint_as_float(w[j]);
    else return __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
  }
};
template <typename IO, int VE>
__device__ __forceinline__ void put(void* p, int64_t i, const float* v) {
  if constexpr (VE == 1) {
    st<IO>(p, i, v[0]);
  } else if constexpr (sizeof(IO) == 4) {
    *reinterpret_cast<f4*>(static_cast<float*>(p) + i) = *reinterpret_cast<const f4*>(v);
  } else {
    typedef __bf16 b8 __attribute__((ext_vector_type(8)));
    typedef float f8 __attribute__((ext_vector_type(8)));
    f8 f;
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = v[k];
    *reinterpret_cast<b8*>(static_cast<uint16_t*>(p) + i) = __builtin_convertvector(f, b8);
  }
}

// VE parameters from column c on, or the value that leaves things as they are.
template <int VE>
__device__ __forceinline__ void params(const float* p, int c, float none, float (&o)[VE]) {
  if (p) {
    if constexpr (VE == 1) {
      o[0] = p[c];
    } else {
#pragma unroll
      for (int j = 0; j < VE; j += 4) *reinterpret_cast<f4*>(o + j) = *reinterpret_cast<const f4*>(p + c + j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < VE; ++j) o[j] = none;
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// Sums of NV values over the team, the same bits in all of its threads.  Teams
// wider than a wave meet once a call, in two sets of places by turns.
template <int TL, int NV>
__device__ __forceinline__ void team_sum(float (&v)[NV], float (*red)[NV][TL < 64 ? 1 : TL / 64], int& turn) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = dpp_add<0xB1>(v[i]);   // lanes 1, 0, 3, 2
    v[i] = dpp_add<0x4E>(v[i]);   // lanes 2, 3, 0, 1
    v[i] = dpp_add<0x141>(v[i]);  // the half row mirrored: its other four
    if constexpr (TL >= 32) {
      v[i] = dpp_add<0x140>(v[i]);  // the row mirrored: its other eight
      const u2 w = __builtin_bit_cast(u2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[i]), false, false));
      v[i] = __uint_as_float(w.x) + __uint_as_float(w.y);
    }
    if constexpr (TL >= 64) {
      const u2 w = __builtin_bit_cast(u2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i]), false, false));
      v[i] = __uint_as_float(w.x) + __uint_as_float(w.y);
    }
  }
  if constexpr (TL > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) red[turn][i][wave] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = 0.0f;
#pragma unroll
      for (int k = 0; k < TL / 64; ++k) v[i] += red[turn][i][k];
    }
    turn ^= 1;
  }
}

constexpr int team_threads(int tl) { return tl < 256 ? 256 : tl; }

template <typename IO, int VE, int TL, int K>
__global__ void __launch_bounds__(team_threads(TL)) norm_fwd_kernel(const NormArgs a) {
  __shared__ float red[2][1][TL < 64 ? 1 : TL / 64];
  int turn = 0;
  const int gs = a.C / a.G, nv = gs / VE, i = threadIdx.x % TL;
  const int64_t item = (int64_t)blockIdx.x * (team_threads(TL) / TL) + threadIdx.x / TL;
  const bool on = item < a.rows * a.G;  // the others only keep the waves whole
  const int64_t r = on ? item / a.G : 0;
  const int c0 = on ? (int)(item - r * a.G) * gs : 0;
  Vec<IO, VE> xr[K], zr[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (k * TL >= nv) break;
    const int c = c0 + min(i + k * TL, nv - 1) * VE;
    xr[k].load(a.x, r * a.xs + c);
    if (a.gate) zr[k].load(a.z, r * a.zs + c);
  }
  const float inv = 1.0f / (float)gs;
  float v[K][VE];
  float sum[1] = {0.0f};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (k * TL >= nv) break;
    const bool in = i + k * TL < nv;
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      float x = xr[k].get(j);
      if (a.gate == SSM_GATE_BEFORE) x *= silu(zr[k].get(j));
      v[k][j] = in ? x : 0.0f;
      sum[0] += v[k][j];
    }
  }
  float mean = 0.0f;
  if (a.center) {
    team_sum<TL, 1>(sum, red, turn);
    mean = sum[0] * inv;
  }
  float sq[1] = {0.0f};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (k * TL >= nv) break;
    if (i + k * TL < nv)
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        v[k][j] -= mean;
        sq[0] = fmaf(v[k][j], v[k][j], sq[0]);
      }
  }
  team_sum<TL, 1>(sq, red, turn);
  const float rs = rsqrtf(fmaf(sq[0], inv, a.eps));
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (k * TL >= nv) break;
    if (on && i + k * TL < nv) {
      const int c = c0 + (i + k * TL) * VE;
      float o[VE], w[VE], b[VE];
      params<VE>(a.w, c, 1.0f, w);
      params<VE>(a.b, c, 0.0f, b);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        float y = fmaf(v[k][j] * rs, w[j], b[j]);
        if (a.act == SSM_ACT_SILU) y = silu(y);
        if (a.gate == SSM_GATE_AFTER) y *= silu(zr[k].get(j));
        o[j] = y;
      }
      put<IO, VE>(a.y, r * a.ys + c, o);
    }
  }
}

// The backward: with u = g w (g the gradient of the affine result) and n the
// normalised values, d = (u - mean(u) - n mean(u n)) / deviation, mean(u) only
// where the forward is centred.  A workgroup's teams keep their group and their columns'
// sums of g n and g in registers over a strip of rows; norm_bwd_sum_kernel adds
// the strips in order.
//
// PLAIN: no centring, no activation, no gate behind and no bias, as the Mamba-2
// block has it: then u does not wait for the statistics, and one meeting gives both
// sums.  Three waves a SIMD hide each other's loads better than two that fetch
// their next rows ahead (16384 x 5120 bf16, 8 groups: 204 against 254 us).
template <typename IO, int VE, int TL, int K, bool PLAIN>
__global__ void __launch_bounds__(team_threads(TL))
__attribute__((amdgpu_waves_per_eu(TL > 256 ? 4 : PLAIN || sizeof(IO) == 4 ? 3 : 2))) norm_bwd_kernel(const NormArgs a) {
  __shared__ float red1[2][1][TL < 64 ? 1 : TL / 64], red2[2][2][TL < 64 ? 1 : TL / 64];
  int turn1 = 0, turn2 = 0;
  constexpr int TW = team_threads(TL) / TL;  // teams of the workgroup: every TW-th row of the strip each
  const int gs = a.C / a.G, nv = gs / VE, i = threadIdx.x % TL, tw = threadIdx.x / TL;
  const int64_t strip = blockIdx.x / a.G;
  const int c0 = (int)(blockIdx.x - strip * a.G) * gs;
  const int64_t r0 = a.rows * strip / a.strips, r1 = a.rows * (strip + 1) / a.strips;
  const int64_t turns = (r1 - r0 + TW - 1) / TW;  // of every team: wide ones meet inside
  const float inv = 1.0f / (float)gs;
  const bool before = a.gate == SSM_GATE_BEFORE, after = !PLAIN && a.gate == SSM_GATE_AFTER;
  float dw[K][VE] = {}, db[PLAIN ? 1 : K][VE] = {};
  for (int64_t q = 0; q < turns; ++q) {
    const int64_t r = r0 + q * TW + tw;
    const bool live = r < r1;
    const int64_t rr = min(r, a.rows - 1);
    Vec<IO, VE> x[K], z[K], g[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k * TL >= nv) break;
      const int c = c0 + min(i + k * TL, nv - 1) * VE;
      x[k].load(a.x, rr * a.xs + c);
      g[k].load(a.dy, rr * a.gs + c);
      if (a.gate) z[k].load(a.z, rr * a.zs + c);
    }
    float v[K][VE];  // what is normalised; zero where there is nothing
    float both[2] = {0.0f, 0.0f}, rs;
    if constexpr (PLAIN) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (k * TL >= nv) break;
        const bool in = live && i + k * TL < nv;
        float w[VE];
        params<VE>(a.w, c0 + min(i + k * TL, nv - 1) * VE, 1.0f, w);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          float t = x[k].get(j);
          if (before) t *= silu(z[k].get(j));
          t = in ? t : 0.0f;
          v[k][j] = t;
          both[0] = fmaf(t, t, both[0]);
          both[1] = fmaf(g[k].get(j) * w[j], in ? t : 0.0f, both[1]);
        }
      }
      team_sum<TL, 2>(both, red2, turn2);
      rs = rsqrtf(fmaf(both[0], inv, a.eps));
      both[1] *= rs;
      both[0] = 0.0f;
    } else {
      float sum[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (k * TL >= nv) break;
        const bool in = live && i + k * TL < nv;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          float t = x[k].get(j);
          if (before) t *= silu(z[k].get(j));
          v[k][j] = in ? t : 0.0f;
          sum[0] += v[k][j];
        }
      }
      float mean = 0.0f;
      if (a.center) {
        team_sum<TL, 1>(sum, red1, turn1);
        mean = sum[0] * inv;
      }
      float sq[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (k * TL >= nv) break;
        if (live && i + k * TL < nv)
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            v[k][j] -= mean;
            sq[0] = fmaf(v[k][j], v[k][j], sq[0]);
          }
      }
      team_sum<TL, 1>(sq, red1, turn1);
      rs = rsqrtf(fmaf(sq[0], inv, a.eps));
    }
    // the gradient of the affine result n w + b; dz of a gate behind it
    auto grad = [&](int k, int j, float n, float w, float b, float& dz) {
      float t = g[k].get(j);
      if constexpr (!PLAIN) {
        if (a.act == SSM_ACT_SILU || after) {
          const float y = fmaf(n, w, b), sy = sigmoid(y);
          if (after) {
            const float zz = z[k].get(j), sz = sigmoid(zz);
            dz = t * (a.act == SSM_ACT_SILU ? y * sy : y) * sz * fmaf(zz, 1.0f - sz, 1.0f);
            t *= zz * sz;
          }
          if (a.act == SSM_ACT_SILU) t *= sy * fmaf(y, 1.0f - sy, 1.0f);
        }
      }
      return t;
    };
    if constexpr (!PLAIN) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (k * TL >= nv) break;
        if (live && i + k * TL < nv) {
          const int c = c0 + (i + k * TL) * VE;
          float w[VE], b[VE], dz[VE];
          params<VE>(a.w, c, 1.0f, w);
          params<VE>(a.b, c, 0.0f, b);
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const float n = v[k][j] * rs, t = grad(k, j, n, w[j], b[j], dz[j]), u = t * w[j];
            dw[k][j] = fmaf(t, n, dw[k][j]);
            db[k][j] += t;
            both[0] += u;
            both[1] = fmaf(u, n, both[1]);
          }
          if (after) put<IO, VE>(a.dz, r * a.dzs + c, dz);
        }
      }
      team_sum<TL, 2>(both, red2, turn2);
      if (!a.center) both[0] = 0.0f;
    }
    const float s1 = both[0] * inv, s2 = both[1] * inv;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k * TL >= nv) break;
      if (live && i + k * TL < nv) {
        const int c = c0 + (i + k * TL) * VE;
        float dx[VE], dz[VE], w[VE], b[VE], none;
        params<VE>(a.w, c, 1.0f, w);
        if constexpr (!PLAIN) params<VE>(a.b, c, 0.0f, b);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const float n = v[k][j] * rs, t = grad(k, j, n, w[j], PLAIN ? 0.0f : b[j], none);
          if constexpr (PLAIN) dw[k][j] = fmaf(t, n, dw[k][j]);
          float d = rs * (t * w[j] - fmaf(n, s2, s1));
          if (before) {
            const float zz = z[k].get(j), sz = sigmoid(zz);
            dz[j] = d * x[k].get(j) * sz * fmaf(zz, 1.0f - sz, 1.0f);
            d *= zz * sz;
          }
          dx[j] = d;
        }
        put<IO, VE>(a.y, r * a.ys + c, dx);
        if (before) put<IO, VE>(a.dz, r * a.dzs + c, dz);
      }
    }
  }
  // the teams' column sums, team by team in order
  auto keep = [&](float* p, const float (&v)[K][VE]) {
    constexpr int M = VE < 4 ? 1 : 4;
    float* out = p + strip * a.C + c0;
    if constexpr (TW > 1) {
      __shared__ __align__(16) float s_sum[TW][TL * K * VE];
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < VE; j += M) put<float, M>(s_sum[tw], (i + k * TL) * VE + j, v[k] + j);
      __syncthreads();
      for (int c = threadIdx.x; c < gs; c += TW * TL) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < TW; ++k) s += s_sum[k][c];
        out[c] = s;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (i + k * TL >= nv) break;
#pragma unroll
        for (int j = 0; j < VE; j += M) put<float, M>(out, (i + k * TL) * VE + j, v[k] + j);
      }
    }
  };
  if (a.pw) keep(a.pw, dw);
  if constexpr (!PLAIN)
    if (a.pb) keep(a.pb, db);
}

// Column sums of the strips' partial sums, in order: sixteen runs of strips a
// column, then the sixteen.  blockIdx.y: dweight or dbias.
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const NormArgs a, float* dw, float* db) {
  __shared__ float run[16][64];
  const float* part = blockIdx.y ? a.pb : a.pw;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), q = threadIdx.x >> 6;
  const int lo = a.strips * q / 16, hi = a.strips * (q + 1) / 16;
  float s = 0.0f;
  if (c < a.C) {
#pragma unroll 8
    for (int i = lo; i < hi; ++i) s += part[(int64_t)i * a.C + c];
  }
  run[q][threadIdx.x & 63] = s;
  __syncthreads();
  if (q == 0 && c < a.C) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += run[k][threadIdx.x];
    out[c] = s;
  }
}

// ---------------------------------------------------------------- host side

// Rows of a tensor that may be a slice of wider rows.
struct Rows {
  const void* p;
  int64_t rows, stride, width;  // bytes
  const char* name;
};

Rows flat(const void* p, int64_t bytes, const char* name) { return {p, 1, bytes, bytes, name}; }

// Whether two of them share a byte.  Slices of the same rows (equal strides,
// interleaved) share none where their columns are disjoint.
bool share(const Rows& x, const Rows& y) {
  const Span a = {x.p, (x.rows - 1) * x.stride + x.width, x.name};
  const Span b = {y.p, (y.rows - 1) * y.stride + y.width, y.name};
  if (!overlaps(a, b)) return false;
  const int64_t st = x.rows > 1 ? x.stride : y.stride;
  if ((x.rows > 1 && x.stride != st) || (y.rows > 1 && y.stride != st)) return true;
  if (x.width > st || y.width > st) return true;
  int64_t d = (int64_t)((intptr_t)x.p - (intptr_t)y.p) % st;
  if (d < 0) d += st;
  return d < y.width || d + x.width > st;
}

int check_rows(const char* name, const void* p, int64_t stride, int64_t width, int64_t rows, int esize) {
  if (stride < width || stride > kMaxExtent)
    return fail(SSM_E_SHAPE, "%s: row stride %lld is less than its %lld columns or too large", name,
                (long long)stride, (long long)width);
  if (!product_ok(rows, stride, esize)) return fail(SSM_E_SHAPE, "tensor sizes overflow");
  if ((uintptr_t)p % esize) return fail(SSM_E_ALIGN, "%s is not aligned to its elements", name);
  return SSM_OK;
}

int check_no_alias(const Rows* outs, int no, const Rows* ins, int ni) {
  for (int o = 0; o < no; ++o) {
    for (int i = 0; i < ni; ++i)
      if (share(outs[o], ins[i])) return fail(SSM_E_ALIAS, "%s overlaps %s", outs[o].name, ins[i].name);
    for (int i = 0; i < o; ++i)
      if (share(outs[o], outs[i])) return fail(SSM_E_ALIAS, "%s overlaps %s", outs[o].name, outs[i].name);
  }
  return SSM_OK;
}

int check_io(int io_dtype) {
  if (io_dtype != SSM_DTYPE_F32 && io_dtype != SSM_DTYPE_BF16)
    return fail(SSM_E_DTYPE, "io_dtype = %d is not SSM_DTYPE_F32 or SSM_DTYPE_BF16", io_dtype);
  return SSM_OK;
}

constexpr int64_t kMaxHeaddim = 256;

// A launch has less than 2^32 threads.
bool grid_ok(int64_t blocks, int threads) { return blocks <= 0xffffffffll / threads; }

int check_mix_extents(int64_t tokens, int64_t nseq, int64_t nheads, int64_t headdim,
                      int64_t ngroups, int64_t dstate) {
  int st;
  if ((st = check_extent("tokens", tokens)) || (st = check_extent("nseq", nseq)) ||
      (st = check_extent("nheads", nheads)) || (st = check_extent("headdim", headdim)) ||
      (st = check_extent("ngroups", ngroups)) || (st = check_extent("dstate", dstate)))
    return st;
  if (nheads % ngroups)
    return fail(SSM_E_SHAPE, "nheads = %lld is not a multiple of ngroups = %lld", (long long)nheads,
                (long long)ngroups);
  if (headdim > kMaxHeaddim || dstate > kMaxN)
    return fail(SSM_E_UNSUPPORTED, "headdim = %lld, dstate = %lld: each is at most 256",
                (long long)headdim, (long long)dstate);
  if (nheads > 16384)
    return fail(SSM_E_SHAPE, "nheads = %lld exceeds 16384", (long long)nheads);
  // one launch has a workgroup of 2^10 threads for each of tokens / 64 + nseq blocks
  if (nseq > 0xfffff || tokens / kQ + nseq >= ((int64_t)1 << 22))
    return fail(SSM_E_SHAPE, "tokens = %lld, nseq = %lld: nseq is at most 2^20 - 1, tokens / 64 + nseq 2^22 - 1",
                (long long)tokens, (long long)nseq);
  return SSM_OK;
}

// What the two entry points of the convolution and scan check alike; fills a.
int check_mix(MixArgs& a, bool step, int64_t rows, int64_t nseq, int64_t nslots, int64_t nheads,
              int64_t headdim, int64_t ngroups, int64_t dstate, int64_t width, int io_dtype,
              const Rows* extra, int nextra) {
  const struct { const void* p; const char* name; } req[] = {
      {a.xbc, "xbc"}, {a.dt, "dt"}, {a.cw, "conv_weight"}, {a.A, "A"}, {a.y, "y"}};
  for (const auto& r : req)
    if (!r.p) return fail(SSM_E_NULL, "%s is NULL", r.name);
  if (!step && !a.cu) return fail(SSM_E_NULL, "cu_seqlens is NULL");
  if (step && !a.state) return fail(SSM_E_NULL, "ssm_state is NULL");
  int st = check_mix_extents(rows, nseq, nheads, headdim, ngroups, dstate);
  if (st) return st;
  if (width < 1 || width > 4)
    return fail(SSM_E_UNSUPPORTED, "width = %lld: supported widths are 1..4", (long long)width);
  if ((st = check_io(io_dtype))) return st;
  const int es = io_dtype == SSM_DTYPE_BF16 ? 2 : 4;
  const int64_t inner = nheads * headdim, ch = inner + 2 * ngroups * dstate;
  if (a.state) {
    if (width > 1 && !a.conv_state)
      return fail(SSM_E_NULL, "conv_state is NULL beside an ssm_state");
    if ((st = check_extent("nslots", nslots))) return st;
    if (!a.slots && nslots < nseq)
      return fail(SSM_E_SHAPE, "nslots = %lld is less than the %lld sequences and slots is NULL",
                  (long long)nslots, (long long)nseq);
    if (!product_ok(nslots, inner, dstate, 4) || !product_ok(nslots, ch, 12))
      return fail(SSM_E_SHAPE, "tensor sizes overflow");
    if (((uintptr_t)a.state | (uintptr_t)a.conv_state) & 3)
      return fail(SSM_E_ALIGN, "a state is not aligned to its elements");
  } else if (a.conv_state || a.slots || a.has) {
    return fail(SSM_E_NULL, "ssm_state is NULL beside conv_state, slots or has_state");
  }
  if ((st = check_rows("xbc", a.xbc, a.xs, ch, rows, es)) ||
      (st = check_rows("dt", a.dt, a.ds, nheads, rows, es)) ||
      (a.z && (st = check_rows("z", a.z, a.zs, inner, rows, es))) ||
      (st = check_rows("y", a.y, a.ys, inner, rows, es)))
    return st;
  const Rows ins[] = {{a.xbc, rows, a.xs * es, ch * es, "xbc"},
                      {a.dt, rows, a.ds * es, nheads * es, "dt"},
                      {a.z, rows, a.zs * es, inner * es, "z"},
                      flat(a.cw, ch * width * 4, "conv_weight"),
                      flat(a.cb, ch * 4, "conv_bias"),
                      flat(a.A, nheads * 4, "A"),
                      flat(a.Dskip, nheads * 4, "D"),
                      flat(a.dt_bias, nheads * 4, "dt_bias"),
                      flat(a.cu, (nseq + 1) * 4, "cu_seqlens"),
                      flat(a.slots, nseq * 4, "slots"),
                      flat(a.has, nseq, "has_state")};
  Rows outs[4] = {{a.y, rows, a.ys * es, inner * es, "y"},
                  flat(a.conv_state, nslots * ch * (width - 1) * 4, "conv_state"),
                  flat(a.state, nslots * inner * dstate * 4, "ssm_state")};
  int no = 3;
  for (int i = 0; i < nextra; ++i) outs[no++] = extra[i];
  if ((st = check_no_alias(outs, no, ins, sizeof ins / sizeof *ins))) return st;
  a.tokens = rows; a.nseq = nseq; a.nslots = nslots;
  a.H = (int)nheads; a.P = (int)headdim; a.G = (int)ngroups; a.N = (int)dstate; a.W = (int)width;
  if (ch > 0x7fffffff) return fail(SSM_E_SHAPE, "too many convolution channels");
  a.C = (int)ch;
  return SSM_OK;
}

// Workspace of ssm_conv_ssd_fwd, and how its sequences are cut.
struct MixLayout {
  int nt, pt, wv;
  int64_t nchunk, nseg, nsplit, ncut;  // at most
  int seg_len, sub, per_group, units;
  int64_t chunks, segs, cuts, ops, local, decay, cs0, bytes;
};

// A segment is one workgroup's work, one after another, and the card holds 2048
// waves at two a SIMD.  Segments for 1024 waves leave it half empty where one
// long prompt has to fill it (four of 8192, 80 heads: 1151 against 919 us; one of 8000
// beside 15 of 10: 319 against 284) and win nothing where the prompts themselves do (16 of
// 8111 tokens in all: 265 against 262); for 4096 they come in two turns (1007, 316, 299).
// Up to three blocks one after another take less time than cut (128 tokens, 80
// heads: 43 against 52 us; four: 62 against 57).
constexpr int64_t kSegWaves = 2048;
constexpr int64_t kUncut = 3;

MixLayout mix_layout(int64_t tokens, int64_t nseq, int64_t H, int64_t P, int64_t G, int64_t N) {
  MixLayout l;
  l.nt = N <= 32 ? 2 : N <= 64 ? 4 : N <= 128 ? 8 : 16;
  l.pt = l.nt == 16 ? 1 : 2;
  const int64_t bph = (P + 16 * l.pt - 1) / (16 * l.pt);
  l.wv = l.nt == 16 ? 8 : 4;
  l.per_group = (int)((H / G * bph + l.wv - 1) / l.wv);
  l.units = (int)(l.per_group * G);
  l.nchunk = tokens / kQ + nseq;
  // as many segments as the card holds at once, not a few more
  const int64_t at_once = kSegWaves / l.wv / l.units, blocks = (tokens + kQ - 1) / kQ;
  int64_t len = at_once ? (blocks + at_once - 1) / at_once : blocks;
  if (len < kUncut && blocks <= kUncut) len = kUncut;
  l.seg_len = (int)len;
  // a sequence of t tokens has 1 + (t - 1) / (64 len) segments and is cut if that is more than one
  const int64_t more = (tokens - 1) / (kQ * len);
  l.nsplit = 2 * more;
  l.ncut = more;
  l.nseg = nseq + more;
  const bool cut = more > 0;
  // the first pass leaves out every sequence's last segment: its segments go in as many
  // pieces as fill the card's turns best
  const int64_t slots = kSegWaves / l.wv, first = (at_once - nseq) * l.units;
  l.sub = cut && at_once <= nseq ? 2 : 1;  // few of them are cut then
  if (cut && at_once > nseq)
    for (int n = 2; n <= 4; ++n)
      if ((first * n + slots - 1) / slots * l.sub < (first * l.sub + slots - 1) / slots * n) l.sub = n;
  if (l.sub > len) l.sub = (int)len;
  const int64_t piece = (int64_t)kQ * l.nt * 16 * 2;
  const int64_t op_bytes = 4 * piece + kTri * 64 * 32 + 64;
  int64_t at = 0;
  auto take = [&](int64_t n) {
    const int64_t o = at;
    at += (n + 255) / 256 * 256;
    return o;
  };
  take(sizeof(PlanHead));
  l.chunks = take(l.nchunk * sizeof(Chunk));
  l.segs = take(l.nseg * sizeof(Seg));
  l.cuts = take(l.ncut * sizeof(Cut));
  l.ops = take(l.nchunk * G * op_bytes);
  l.local = take(l.nsplit * l.sub * H * P * N * 4);
  l.decay = take(l.nsplit * l.sub * H * 4);
  l.cs0 = take(l.ncut * H * P * 3 * 4);
  l.bytes = at;
  return l;
}

template <typename IO, int NT, int PT, int WV>
void launch_mix_blocks(const BlkArgs& b, const MixLayout& l, hipStream_t s) {
  static_assert(Ops<NT>::bytes == 4 * kQ * NT * 32 + kTri * 64 * 32 + 64, "as in mix_layout");
  mix_plan_kernel<<<1, 1024, 0, s>>>(b);
  mix_prep_kernel<IO, NT><<<dim3((unsigned)l.nchunk, b.G), kPrep, 0, s>>>(b);
  const unsigned grid = (unsigned)(l.nseg * l.units);
  auto walk = [&](auto fast) {
    constexpr bool F = decltype(fast)::value;
    if (l.nsplit) {
      mix_block_kernel<IO, NT, PT, WV, true, F><<<grid * l.sub, 64 * WV, 0, s>>>(b);
      const int64_t per = (int64_t)b.H * b.P * b.N;
      mix_join_kernel<<<dim3((unsigned)((per + 1023) / 1024), (unsigned)l.ncut), 256, 0, s>>>(b);
    }
    mix_block_kernel<IO, NT, PT, WV, false, F><<<grid, 64 * WV, 0, s>>>(b);
  };
  if (b.fast) walk(std::integral_constant<bool, true>{});
  else walk(std::integral_constant<bool, false>{});
}

template <typename IO>
void launch_mix(const BlkArgs& b, const MixLayout& l, hipStream_t s) {
  switch (l.nt) {
    case 2: launch_mix_blocks<IO, 2, 2, 4>(b, l, s); break;
    case 4: launch_mix_blocks<IO, 4, 2, 4>(b, l, s); break;
    case 8: launch_mix_blocks<IO, 8, 2, 4>(b, l, s); break;
    default: launch_mix_blocks<IO, 16, 1, 8>(b, l, s); break;
  }
}

// Eight rows a lane where that leaves two workgroups for every CU (253 tokens, 80
// heads: 274 us against 291 with two rows), two where the card would stand half empty
// (one token: 11.3 against 12.4).
constexpr int64_t kStepWorkgroups = 512;

template <typename IO, int LN, bool VEC>
int launch_step(const MixArgs& a, hipStream_t s) {
  auto go = [&](auto rpl) {
    constexpr int R = decltype(rpl)::value, rows = 256 / LN * R;
    const int splits = (a.P + rows - 1) / rows;
    const int64_t grid = a.nseq * a.H * splits;
    if (!grid_ok(grid, 256)) return fail(SSM_E_SHAPE, "too many entries and heads for one call");
    mix_step_kernel<IO, LN, R, VEC><<<(unsigned)grid, 256, 0, s>>>(a, splits);
    return (int)SSM_OK;
  };
  const int64_t wide = a.nseq * a.H * ((a.P + 256 / LN * 8 - 1) / (256 / LN * 8));
  const int st = wide >= kStepWorkgroups ? go(std::integral_constant<int, 8>{}) : go(std::integral_constant<int, 2>{});
  if (st) return st;
  if (a.W > 1)
    mix_step_conv_kernel<IO><<<dim3((unsigned)a.nseq, (unsigned)((2 * a.G * a.N + 255) / 256)), 256, 0, s>>>(a);
  return launch_status("ssm_conv_ssd_update launch");
}

template <typename IO>
int launch_step_io(const MixArgs& a, hipStream_t s) {
  if (a.N % 4 || !aligned16(a.state)) return launch_step<IO, 64, false>(a, s);
  if (a.N <= 16) return launch_step<IO, 4, true>(a, s);
  if (a.N <= 32) return launch_step<IO, 8, true>(a, s);
  if (a.N <= 64) return launch_step<IO, 16, true>(a, s);
  if (a.N <= 128) return launch_step<IO, 32, true>(a, s);
  return launch_step<IO, 64, true>(a, s);
}

// Strips of rows whose column sums are kept apart, at most: three waves for every
// SIMD of the card where the partial sums stay under 16 MB a gradient.
int64_t norm_strips(int64_t rows, int64_t channels) {
  int64_t n = ((int64_t)1 << 22) / channels;
  n = n < 256 ? 256 : (n > 1024 ? 1024 : n);
  return n < rows ? n : rows;
}
constexpr int64_t kNormThreads = 256 * 4 * 3 * 64;

constexpr int64_t kMaxGroup = 32768;

int check_norm(const NormArgs& a, int64_t rows, int64_t channels, int64_t ngroups, int io_dtype) {
  int st;
  if ((st = check_extent("rows", rows)) || (st = check_extent("channels", channels)) ||
      (st = check_extent("ngroups", ngroups)))
    return st;
  if (channels % ngroups)
    return fail(SSM_E_SHAPE, "channels = %lld is not a multiple of ngroups = %lld",
                (long long)channels, (long long)ngroups);
  if (channels > 0x7fffffff || ngroups > 65535)
    return fail(SSM_E_SHAPE, "channels = %lld, ngroups = %lld: too many", (long long)channels,
                (long long)ngroups);
  if (channels / ngroups > kMaxGroup)
    return fail(SSM_E_UNSUPPORTED, "a group of %lld channels: at most %lld",
                (long long)(channels / ngroups), (long long)kMaxGroup);
  if (a.act != SSM_ACT_NONE && a.act != SSM_ACT_SILU)
    return fail(SSM_E_DTYPE, "activation = %d is not a known value", a.act);
  if (a.gate != SSM_GATE_NONE && a.gate != SSM_GATE_BEFORE && a.gate != SSM_GATE_AFTER)
    return fail(SSM_E_DTYPE, "gate = %d is not a known value", a.gate);
  if ((a.gate == SSM_GATE_NONE) != (a.z == nullptr))
    return fail(SSM_E_NULL, a.z ? "z without a gate" : "z is NULL beside a gate");
  if (!(a.eps >= 0.0f) || a.eps > 3e38f) return fail(SSM_E_SHAPE, "eps is negative or not finite");
  return check_io(io_dtype);
}

// Whole 16-byte vectors: the groups start and end on them in every tensor.
bool norm_vectors(const NormArgs& a, int es) {
  const uintptr_t at = (uintptr_t)a.x | (uintptr_t)a.z | (uintptr_t)a.dy | (uintptr_t)a.y | (uintptr_t)a.dz |
                       (uintptr_t)a.w | (uintptr_t)a.b;
  const int64_t all = (a.xs | a.zs | a.gs | a.ys | a.dzs | (int64_t)(a.C / a.G)) * es;
  return at % 16 == 0 && all % 16 == 0;
}

template <bool BWD, typename IO, int VE, int TL, int K>
int launch_norm_team(NormArgs& a, hipStream_t s) {
  if constexpr (BWD) {
    const int64_t fill = (kNormThreads + (int64_t)team_threads(TL) * a.G - 1) / ((int64_t)team_threads(TL) * a.G);
    if (fill < a.strips) a.strips = (int)fill;
  }
  const int64_t items = (BWD ? a.strips : a.rows) * (int64_t)a.G, per = BWD ? 1 : team_threads(TL) / TL;
  const int64_t blocks = (items + per - 1) / per;
  if (!grid_ok(blocks, team_threads(TL))) return fail(SSM_E_SHAPE, "rows and ngroups: too many for one call");
  if constexpr (BWD) {
    if (!a.center && a.act == SSM_ACT_NONE && a.gate != SSM_GATE_AFTER && !a.pb)
      norm_bwd_kernel<IO, VE, TL, K, true><<<(unsigned)blocks, team_threads(TL), 0, s>>>(a);
    else
      norm_bwd_kernel<IO, VE, TL, K, false><<<(unsigned)blocks, team_threads(TL), 0, s>>>(a);
  } else norm_fwd_kernel<IO, VE, TL, K><<<(unsigned)blocks, team_threads(TL), 0, s>>>(a);
  return launch_status(BWD ? "ssm_group_norm_bwd launch" : "ssm_group_norm_fwd launch");
}

// The smallest team whose registers hold the group, with as few of them unused as
// may be: a wave of up to ten vectors a lane took 203 us where 256 threads of four take
// 187 (32768 rows of 5120, bf16), and 318 where a wave of up to two takes 207 (eight
// groups of 640).  The backward holds more a vector: 1024 threads of four took 221 us where
// 512 of two take 171 (8000 rows of 8192), a wave of two 435 where 32 threads of three
// take 348 (32768 rows, eight groups of 640).
template <bool BWD, typename IO>
int launch_norm_io(NormArgs& a, bool vec, hipStream_t s) {
  constexpr int VE = 16 / sizeof(IO);
  const int gs = a.C / a.G, nv = vec ? gs / VE : gs;
  if (vec) {
    if constexpr (BWD) {
      if (nv <= 8 * 3) return launch_norm_team<true, IO, VE, 8, 3>(a, s);
      if (nv <= 32 * 3) return launch_norm_team<true, IO, VE, 32, 3>(a, s);
      if (nv <= 64 * 3) return launch_norm_team<true, IO, VE, 64, 3>(a, s);
      if (nv <= 256 * 3) return launch_norm_team<true, IO, VE, 256, 3>(a, s);
      if (nv <= 512 * 2) return launch_norm_team<true, IO, VE, 512, 2>(a, s);
    } else {
      if (nv <= 8) return launch_norm_team<false, IO, VE, 8, 1>(a, s);
      if (nv <= 8 * 4) return launch_norm_team<false, IO, VE, 8, 4>(a, s);
      if (nv <= 64 * 2) return launch_norm_team<false, IO, VE, 64, 2>(a, s);
      if (nv <= 64 * 4) return launch_norm_team<false, IO, VE, 64, 4>(a, s);
      if (nv <= 256 * 4) return launch_norm_team<false, IO, VE, 256, 4>(a, s);
    }
    if (nv <= 1024 * 4) return launch_norm_team<BWD, IO, VE, 1024, 4>(a, s);
    if constexpr (VE == 4) return launch_norm_team<BWD, IO, VE, 1024, 8>(a, s);
  }
  if (nv <= 8 * 8) return launch_norm_team<BWD, IO, 1, 8, 8>(a, s);
  // element by element: the forward is fastest with a wave a group (20000 rows of 1001: 30 us
  // against 37 with 256 threads), the backward, which holds four values where the forward
  // holds one, with more threads (94 against 144 us)
  if constexpr (BWD) {
    if (nv <= 64 * 4) return launch_norm_team<BWD, IO, 1, 64, 4>(a, s);
    if (nv <= 256 * 4) return launch_norm_team<BWD, IO, 1, 256, 4>(a, s);
  } else if (nv <= 64 * 16) {
    return launch_norm_team<BWD, IO, 1, 64, 16>(a, s);
  }
  if (nv <= 256 * 16) return launch_norm_team<BWD, IO, 1, 256, 16>(a, s);
  if (nv <= 1024 * 16) return launch_norm_team<BWD, IO, 1, 1024, 16>(a, s);
  return launch_norm_team<BWD, IO, 1, 1024, 32>(a, s);
}

template <bool BWD>
int launch_norm(NormArgs& a, bool vec, int io_dtype, hipStream_t s) {
  return io_dtype == SSM_DTYPE_BF16 ? launch_norm_io<BWD, uint16_t>(a, vec, s) : launch_norm_io<BWD, float>(a, vec, s);
}

}  // namespace

// ---------------------------------------------------------------- C ABI

extern "C" {

int64_t ssm_conv_ssd_workspace_size(int64_t tokens, int64_t nseq, int64_t nheads, int64_t headdim,
                                    int64_t ngroups, int64_t dstate, int io_dtype) {
  g_last_error[0] = 0;
  if (check_mix_extents(tokens, nseq, nheads, headdim, ngroups, dstate) || check_io(io_dtype)) return -1;
  return mix_layout(tokens, nseq, nheads, headdim, ngroups, dstate).bytes;
}

int ssm_conv_ssd_fwd(const void* xbc, int64_t xbc_stride, const void* dt, int64_t dt_stride,
                     const void* z, int64_t z_stride, const float* conv_weight,
                     const float* conv_bias, const float* A, const float* Dskip,
                     const float* dt_bias, int dt_softplus, const int32_t* cu_seqlens,
                     const int32_t* slots, const uint8_t* has_state, float* conv_state,
                     float* ssm_state, void* y, int64_t y_stride, void* workspace,
                     int64_t workspace_bytes, int64_t tokens, int64_t nseq, int64_t nslots,
                     int64_t nheads, int64_t headdim, int64_t ngroups, int64_t dstate,
                     int64_t width, int io_dtype, void* hip_stream) {
  g_last_error[0] = 0;
  BlkArgs a;
  memset(&a, 0, sizeof a);
  a.xbc = xbc; a.dt = dt; a.z = z; a.cw = conv_weight; a.cb = conv_bias; a.A = A; a.Dskip = Dskip;
  a.dt_bias = dt_bias; a.cu = cu_seqlens; a.slots = slots; a.has = has_state;
  a.conv_state = conv_state; a.state = ssm_state; a.y = y;
  a.xs = xbc_stride; a.ds = dt_stride; a.zs = z_stride; a.ys = y_stride;
  a.softplus = dt_softplus ? 1 : 0;
  if (!workspace) return fail(SSM_E_NULL, "workspace is NULL");
  const Rows ws = flat(workspace, workspace_bytes, "workspace");
  const int st = check_mix(a, false, tokens, nseq, nslots, nheads, headdim, ngroups, dstate, width,
                           io_dtype, &ws, 1);
  if (st) return st;
  const int64_t need = ssm_conv_ssd_workspace_size(tokens, nseq, nheads, headdim, ngroups, dstate, io_dtype);
  if (workspace_bytes < need)
    return fail(SSM_E_SHAPE, "workspace holds %lld bytes, needs %lld", (long long)workspace_bytes,
                (long long)need);
  if (!aligned16(workspace)) return fail(SSM_E_ALIGN, "workspace is not 16-byte aligned");
  const MixLayout l = mix_layout(tokens, nseq, nheads, headdim, ngroups, dstate);
  if (!grid_ok(l.nseg * l.units * l.sub, 64 * l.wv))
    return fail(SSM_E_SHAPE, "too many sequences and heads for one call");
  char* w = static_cast<char*>(workspace);
  a.head = reinterpret_cast<PlanHead*>(w);
  a.chunks = reinterpret_cast<Chunk*>(w + l.chunks);
  a.segs = reinterpret_cast<Seg*>(w + l.segs);
  a.cuts = reinterpret_cast<Cut*>(w + l.cuts);
  a.ops = w + l.ops;
  a.local = reinterpret_cast<float*>(w + l.local);
  a.decay = reinterpret_cast<float*>(w + l.decay);
  a.cs0 = reinterpret_cast<float*>(w + l.cs0);
  a.seg_len = l.seg_len; a.sub = l.sub; a.units = l.units; a.per_group = l.per_group;
  const int es = io_dtype == SSM_DTYPE_BF16 ? 2 : 4, wide = 4 * l.pt * es < 16 ? 4 * l.pt * es : 16;
  const int64_t inner = nheads * headdim, ch = inner + 2 * ngroups * dstate;
  auto lanes = [&](const void* p, int64_t stride, int bytes) {  // whole accesses of that many bytes
    return ((uintptr_t)p | (uintptr_t)(stride * es) | (uintptr_t)(headdim * es)) % bytes == 0;
  };
  a.fast = headdim % (4 * l.pt) == 0 && dstate % 4 == 0 && lanes(xbc, xbc_stride, es == 2 ? 16 : 4 * l.pt) && (es == 4 || ch >= inner + 32) &&
           lanes(y, y_stride, wide) && (!z || lanes(z, z_stride, wide)) && aligned16(ssm_state);
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (io_dtype == SSM_DTYPE_BF16) launch_mix<uint16_t>(a, l, s);
  else launch_mix<float>(a, l, s);
  return launch_status("ssm_conv_ssd_fwd launch");
}

int ssm_conv_ssd_update(const void* xbc, int64_t xbc_stride, const void* dt, int64_t dt_stride,
                        const void* z, int64_t z_stride, const float* conv_weight,
                        const float* conv_bias, const float* A, const float* Dskip,
                        const float* dt_bias, int dt_softplus, const int32_t* slots,
                        float* conv_state, float* ssm_state, void* y, int64_t y_stride,
                        int64_t batch, int64_t nslots, int64_t nheads, int64_t headdim,
                        int64_t ngroups, int64_t dstate, int64_t width, int io_dtype,
                        void* hip_stream) {
  g_last_error[0] = 0;
  MixArgs a;
  memset(&a, 0, sizeof a);
  a.xbc = xbc; a.dt = dt; a.z = z; a.cw = conv_weight; a.cb = conv_bias; a.A = A; a.Dskip = Dskip;
  a.dt_bias = dt_bias; a.slots = slots; a.conv_state = conv_state; a.state = ssm_state; a.y = y;
  a.xs = xbc_stride; a.ds = dt_stride; a.zs = z_stride; a.ys = y_stride;
  a.softplus = dt_softplus ? 1 : 0;
  const int st = check_mix(a, true, batch, batch, nslots, nheads, headdim, ngroups, dstate, width,
                           io_dtype, nullptr, 0);
  if (st) return st;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  return io_dtype == SSM_DTYPE_BF16 ? launch_step_io<uint16_t>(a, s) : launch_step_io<float>(a, s);
}

int ssm_group_norm_fwd(const void* x, int64_t x_stride, const void* z, int64_t z_stride,
                       const float* weight, const float* bias, float eps, int center,
                       int activation, int gate, void* y, int64_t y_stride, int64_t rows,
                       int64_t channels, int64_t ngroups, int io_dtype, void* hip_stream) {
  g_last_error[0] = 0;
  if (!x) return fail(SSM_E_NULL, "x is NULL");
  if (!y) return fail(SSM_E_NULL, "y is NULL");
  NormArgs a;
  memset(&a, 0, sizeof a);
  a.x = x; a.z = z; a.w = weight; a.b = bias; a.y = y; a.xs = x_stride; a.zs = z_stride;
  a.ys = y_stride; a.eps = eps; a.center = center ? 1 : 0; a.act = activation; a.gate = gate;
  int st = check_norm(a, rows, channels, ngroups, io_dtype);
  if (st) return st;
  const int es = io_dtype == SSM_DTYPE_BF16 ? 2 : 4;
  if ((st = check_rows("x", x, x_stride, channels, rows, es)) ||
      (z && (st = check_rows("z", z, z_stride, channels, rows, es))) ||
      (st = check_rows("y", y, y_stride, channels, rows, es)))
    return st;
  const Rows ins[] = {{x, rows, x_stride * es, channels * es, "x"},
                      {z, rows, z_stride * es, channels * es, "z"},
                      flat(weight, channels * 4, "weight"), flat(bias, channels * 4, "bias")};
  const Rows out = {y, rows, y_stride * es, channels * es, "y"};
  if ((st = check_no_alias(&out, 1, ins, 4))) return st;
  a.rows = rows; a.C = (int)channels; a.G = (int)ngroups;
  const bool vec = norm_vectors(a, es);
  return launch_norm<false>(a, vec, io_dtype, static_cast<hipStream_t>(hip_stream));
}

int64_t ssm_group_norm_bwd_workspace_size(int64_t rows, int64_t channels, int64_t ngroups) {
  g_last_error[0] = 0;
  if (check_extent("rows", rows) || check_extent("channels", channels) ||
      check_extent("ngroups", ngroups) || channels > 0x7fffffff)
    return -1;
  return (2 * norm_strips(rows, channels) * channels * 4 + 15) / 16 * 16;
}

int ssm_group_norm_bwd(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                       const void* z, int64_t z_stride, const float* weight, const float* bias,
                       float eps, int center, int activation, int gate, void* dx,
                       int64_t dx_stride, void* dz, int64_t dz_stride, float* dweight,
                       float* dbias, void* workspace, int64_t workspace_bytes, int64_t rows,
                       int64_t channels, int64_t ngroups, int io_dtype, void* hip_stream) {
  g_last_error[0] = 0;
  const struct { const void* p; const char* name; } req[] = {
      {dy, "dy"}, {x, "x"}, {dx, "dx"}, {workspace, "workspace"}};
  for (const auto& r : req)
    if (!r.p) return fail(SSM_E_NULL, "%s is NULL", r.name);
  NormArgs a;
  memset(&a, 0, sizeof a);
  a.x = x; a.z = z; a.dy = dy; a.w = weight; a.b = bias; a.y = dx; a.dz = dz; a.xs = x_stride;
  a.zs = z_stride; a.gs = dy_stride; a.ys = dx_stride; a.dzs = dz_stride; a.eps = eps;
  a.center = center ? 1 : 0; a.act = activation; a.gate = gate;
  int st = check_norm(a, rows, channels, ngroups, io_dtype);
  if (st) return st;
  if ((z == nullptr) != (dz == nullptr))
    return fail(SSM_E_NULL, z ? "dz is NULL beside z" : "dz without z");
  const int es = io_dtype == SSM_DTYPE_BF16 ? 2 : 4;
  if ((st = check_rows("dy", dy, dy_stride, channels, rows, es)) ||
      (st = check_rows("x", x, x_stride, channels, rows, es)) ||
      (z && (st = check_rows("z", z, z_stride, channels, rows, es))) ||
      (st = check_rows("dx", dx, dx_stride, channels, rows, es)) ||
      (dz && (st = check_rows("dz", dz, dz_stride, channels, rows, es))))
    return st;
  const int64_t need = ssm_group_norm_bwd_workspace_size(rows, channels, ngroups);
  if (workspace_bytes < need)
    return fail(SSM_E_SHAPE, "workspace holds %lld bytes, needs %lld", (long long)workspace_bytes,
                (long long)need);
  if (!aligned16(workspace)) return fail(SSM_E_ALIGN, "workspace is not 16-byte aligned");
  const int64_t wb = channels * es;
  const Rows ins[] = {{dy, rows, dy_stride * es, wb, "dy"}, {x, rows, x_stride * es, wb, "x"},
                      {z, rows, z_stride * es, wb, "z"}, flat(weight, channels * 4, "weight"),
                      flat(bias, channels * 4, "bias")};
  const Rows outs[] = {{dx, rows, dx_stride * es, wb, "dx"}, {dz, rows, dz_stride * es, wb, "dz"},
                       flat(dweight, channels * 4, "dweight"), flat(dbias, channels * 4, "dbias"),
                       flat(workspace, need, "workspace")};
  if ((st = check_no_alias(outs, 5, ins, 5))) return st;
  a.rows = rows; a.C = (int)channels; a.G = (int)ngroups;
  a.strips = (int)norm_strips(rows, channels);
  a.pw = dweight ? static_cast<float*>(workspace) : nullptr;
  a.pb = dbias ? static_cast<float*>(workspace) + a.strips * channels : nullptr;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if ((st = launch_norm<true>(a, norm_vectors(a, es), io_dtype, s))) return st;
  if (dweight || dbias)
    norm_bwd_sum_kernel<<<dim3((unsigned)((channels + 63) / 64), 2), 1024, 0, s>>>(a, dweight, dbias);
  return launch_status("ssm_group_norm_bwd launch");
}

}  // extern "C"
