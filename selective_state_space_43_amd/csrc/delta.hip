// libselscan -- the gated delta rule for AMD Instinct MI355X (gfx950): over packed
// prompts (ssm_gated_delta_fwd), its gradients (ssm_gated_delta_bwd) and one token a
// sequence (ssm_gated_delta_update).
//
// With k, q the normalised rows, b the write strengths, G the running sum of the log
// decays inside a block of 64 tokens and S [dstate, headdim] the state entering it,
// the recurrence over the block is
//
//   L_ij = b_i exp(G_i - G_j) k_i.k_j  (j < i),   T = (I + L)^-1
//   M_ij = exp(G_i - G_j) q_i.k_j      (j <= i)
//   U  = T R,   R_i = b_i (v_i - exp(G_i) k_i S)
//   Y_i = exp(G_i) q_i S + sum_j M_ij U_j
//   S' = exp(G_64) S + sum_j exp(G_64 - G_j) k_j U_j^T
//
// T, M and the rows belong to a block and are made for all blocks at once; what is left
// goes from block to block.  The columns of S (channels of v) do not meet: they are split
// over workgroups.  Backwards, with dS' the gradient of the state behind the block,
//
//   dU = M^T dY + (exp(G_64 - G) k) dS',   dR = T^T dU,   dv = b dR
//   dS = exp(G_64) dS' + (exp(G) q)^T dY - (b exp(G) k)^T dR
//
// and, again for all blocks at once, with dM = dY U^T, dL = -dR U^T (below the diagonal),
// D = exp(G_i - G_j):
//
//   dq = exp(G) dY S^T + (dM D) k
//   dk = (dM D)^T q + exp(G_64 - G) U dS'^T - b exp(G) dR S^T + (b dL D) k + (b dL D)^T k
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "rows.h"

namespace {

constexpr int kQ = 64;  // tokens of a block

// ---------------------------------------------------------------- arguments

// up to 64 rows of one sequence
struct DeltaChunk {
  int r0, r1;
};
struct DeltaSeq {
  int slot, t0, t1;  // slot -1: padding
  int c0;            // its first block
  int resume;
};
struct DeltaHead {
  int nchunk, first, last, pad;  // blocks in use; rows [first, last) belong to sequences
};

struct DeltaArgs {
  const void *q, *k, *v, *dt, *beta, *dy;
  const float *A, *dt_bias;
  const int32_t* cu;
  const int32_t* slots;
  const uint8_t* has;
  float* state;     // forward: read and written at the slot
  const float *h0, *dfinal;
  float* dh0;
  void* y;
  void *dq, *dk, *dv, *ddt, *dbeta;
  float *dA, *ddt_bias;
  int64_t qs, ks, vs, ds, bs, ys, gs;        // row strides
  int64_t dqs, dks, dvs, dds, dbs;
  int64_t tokens, nseq, nslots;
  int H, P, G, N, per;                       // per: heads of a group
  int softplus, sigmoid, norm;
  float eps, scale;
  // workspace
  DeltaHead* head;
  DeltaChunk* chunks;
  DeltaSeq* seqs;
  float *qh, *kh;        // [block, group][64][N] normalised rows
  float *T, *M;          // [block, head][64][64]
  double* cum;           // [block, head][64] G
  float* b;              // [block, head][64]
  char *gops, *hops;     // operands of a (block, group), of a (block, head)
  // backward
  float *S, *dS;         // [block, head][N][P] the state entering, its gradient behind
  float *U, *dR;         // [block, head][64][P]
  float *dqh, *dkh;      // [block, head][64][N]
  float *part;           // [block, head][2] sums of dA, ddt_bias
};

constexpr int64_t kMaxN = 256;

// ---------------------------------------------------------------- sequences -> blocks (one workgroup)

__global__ void __launch_bounds__(1024) delta_plan_kernel(const DeltaArgs a) {
  __shared__ int red[16];
  __shared__ i4 red4[16];
  __shared__ int s_t0[1024], s_t1[1024], s_chunk[1024];
  int nchunk = 0;
  const int i = threadIdx.x, tokens = (int)a.tokens;
  const int start = max(0, min(a.cu[0], tokens));
  int reached = start;  // the largest offset so far
  for (int64_t base = 0; base < a.nseq; base += 1024) {
    // the offsets' running maximum: whatever they hold, the sequences lie one
    // behind the other inside the rows, and the tables hold their blocks
    const int64_t s = base + i;
    const bool in = s < a.nseq;
    const int64_t slot = in && a.slots ? a.slots[s] : s;
    int end = in ? max(reached, min(a.cu[s + 1], tokens)) : reached;
    end = block_scan_max(end, red);
    s_t1[i] = end;
    __syncthreads();
    const int begin = i ? s_t1[i - 1] : reached;
    reached = s_t1[1023];
    s_t0[i] = begin;
    const bool use = in && (!a.state || (slot >= 0 && slot < a.nslots));
    i4 n = {use ? (end - begin + kQ - 1) / kQ : 0, 0, 0, 0}, all;
    const i4 at = block_scan(n, red4, all);
    s_chunk[i] = at[0];
    if (in) a.seqs[s] = {use ? (int)slot : -1, begin, end, nchunk + at[0], a.has ? a.has[s] != 0 : 0};
    __syncthreads();
    for (int c = i; c < all[0]; c += 1024) {
      const int k = find(s_chunk, c), r0 = s_t0[k] + (c - s_chunk[k]) * kQ;
      a.chunks[nchunk + c] = {r0, min(s_t1[k], r0 + kQ)};
    }
    nchunk += all[0];
    __syncthreads();
  }
  if (i == 0) *a.head = {nchunk, start, reached, 0};
}

// ---------------------------------------------------------------- a block's matrices

// the step of a head's row in units of log2 (at most 160 down: below that a decay is
// zero in float32, and no sum swallows the steps beside it), and the write strength
template <typename IO>
__device__ __forceinline__ void row_scalars(const DeltaArgs& a, int64_t r, int h, float& g, float& b) {
  const float raw = ld<IO>(a.dt, r * a.ds + h) + (a.dt_bias ? a.dt_bias[h] : 0.0f);
  const float dt = a.softplus ? softplus(raw) : raw;
  g = dt * (a.A[h] * kLog2e);
  g = g < -160.0f ? -160.0f : g;
  if (!finite(dt)) g = __builtin_nanf("");
  const float braw = ld<IO>(a.beta, r * a.bs + h);
  b = a.sigmoid ? sigmoid(braw) : braw;
}

// one workgroup per block and group: the normalised rows
template <typename IO>
__global__ void __launch_bounds__(256) delta_rows_kernel(const DeltaArgs a) {
  const int c = blockIdx.x, g = blockIdx.y, N = a.N;
  if (c >= a.head->nchunk) return;
  const DeltaChunk ck = a.chunks[c];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = wave; i < kQ; i += 4) {
    const bool in = ck.r0 + i < ck.r1;
    const int64_t r = in ? ck.r0 + i : ck.r0;
    for (int which = 0; which < 2; ++which) {
      const void* p = which ? a.k : a.q;
      const int64_t at = r * (which ? a.ks : a.qs) + (int64_t)g * N;
      float x[4], ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = in && lane + 64 * j < N ? ld<IO>(p, at + lane + 64 * j) : 0.0f;
        ss = fmaf(x[j], x[j], ss);
      }
      ss = lane_sum<64>(ss);
      const float f = (a.norm ? rsqrtf(ss + a.eps) : 1.0f) * (which ? 1.0f : a.scale);
      float* out = (which ? a.kh : a.qh) + (((int64_t)c * a.G + g) * kQ + i) * N;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (lane + 64 * j < N) out[lane + 64 * j] = x[j] * f;
    }
  }
}

// one workgroup per block and head: T, M, the running sum
template <typename IO>
__global__ void __launch_bounds__(256) delta_prep_kernel(const DeltaArgs a) {
  __shared__ float s_x[kQ][kQ + 1], s_l[kQ][kQ + 1], s_b[kQ];
  __shared__ double s_g[kQ];
  const int c = blockIdx.x, h = blockIdx.y, N = a.N, g = h / a.per;
  if (c >= a.head->nchunk) return;
  const DeltaChunk ck = a.chunks[c];
  const int tid = threadIdx.x;
  const int64_t at = (int64_t)c * a.H + h;
  if (tid < kQ) {
    float gr = 0.0f, b = 0.0f;
    if (ck.r0 + tid < ck.r1) row_scalars<IO>(a, ck.r0 + tid, h, gr, b);
    const double cum = wave_scan((double)gr);
    s_g[tid] = cum;
    s_b[tid] = b;
    a.cum[at * kQ + tid] = cum;
    a.b[at * kQ + tid] = b;
  }
  __syncthreads();
  const float* kh = a.kh + ((int64_t)c * a.G + g) * kQ * N;
  const float* qh = a.qh + ((int64_t)c * a.G + g) * kQ * N;
  for (int u = tid; u < kQ * kQ; u += 256) {
    const int i = u >> 6, j = u & 63;
    float kk = 0.0f, qk = 0.0f;
    if (j <= i)
      for (int n = 0; n < N; ++n) {
        kk = fmaf(kh[i * N + n], kh[j * N + n], kk);
        qk = fmaf(qh[i * N + n], kh[j * N + n], qk);
      }
    const float D = j <= i ? ex2((float)(s_g[i] - s_g[j])) : 0.0f;
    s_l[i][j] = j < i ? s_b[i] * D * kk : 0.0f;
    a.M[at * kQ * kQ + u] = j <= i ? D * qk : 0.0f;
  }
  __syncthreads();
  if (tid < kQ) {  // column tid of the inverse, row by row
    for (int i = 0; i < kQ; ++i) {
      float x = i == tid ? 1.0f : 0.0f;
      for (int m = tid; m < i; ++m) x = fmaf(-s_l[i][m], s_x[m][tid], x);
      s_x[i][tid] = i < tid ? 0.0f : x;
    }
  }
  __syncthreads();
  for (int u = tid; u < kQ * kQ; u += 256) a.T[at * kQ * kQ + u] = s_x[u >> 6][u & 63];
}

// ---------------------------------------------------------------- from block to block

// One workgroup per sequence, head and 32 channels.  KEEP: for the backward, which keeps
// S and U of every block and no y.
template <typename IO, bool KEEP>
__global__ void __launch_bounds__(256) delta_scan_kernel(const DeltaArgs a) {
  __shared__ float s_S[kMaxN][33], s_r[kQ][33];
  const DeltaSeq sq = a.seqs[blockIdx.x];
  if (sq.slot < 0) return;
  const int h = blockIdx.y, N = a.N, P = a.P, g = h / a.per;
  const int cl = threadIdx.x & 31, rg = threadIdx.x >> 5, p = blockIdx.z * 32 + cl;
  const bool on = p < P;
  const int64_t own = KEEP ? blockIdx.x : sq.slot;
  const float* src = KEEP ? a.h0 : sq.resume ? a.state : nullptr;
  for (int n = rg; n < N; n += 8)
    s_S[n][cl] = src && on ? src[((own * a.H + h) * P + p) * N + n] : 0.0f;
  __syncthreads();
  const int nc = (sq.t1 - sq.t0 + kQ - 1) / kQ;
  for (int b = 0; b < nc; ++b) {
    const int c = sq.c0 + b, r0 = sq.t0 + b * kQ, cnt = min(sq.t1 - r0, kQ);
    const int64_t at = (int64_t)c * a.H + h, ag = ((int64_t)c * a.G + g) * kQ;
    const double* cum = a.cum + at * kQ;
    const float *T = a.T + at * kQ * kQ, *M = a.M + at * kQ * kQ, *bb = a.b + at * kQ;
    if (KEEP && on)
      for (int n = rg; n < N; n += 8) a.S[(at * N + n) * P + p] = s_S[n][cl];
    float u[8];
    for (int ii = 0; ii < 8; ++ii) {
      const int i = rg + 8 * ii;
      float kS = 0.0f;
      for (int n = 0; n < N; ++n) kS = fmaf(a.kh[(ag + i) * N + n], s_S[n][cl], kS);
      const float v = on && i < cnt ? ld<IO>(a.v, (int64_t)(r0 + i) * a.vs + h * P + p) : 0.0f;
      s_r[i][cl] = bb[i] * (v - ex2((float)cum[i]) * kS);
    }
    __syncthreads();
    for (int ii = 0; ii < 8; ++ii) {
      const int i = rg + 8 * ii;
      u[ii] = 0.0f;
      for (int j = 0; j <= i; ++j) u[ii] = fmaf(T[i * kQ + j], s_r[j][cl], u[ii]);
    }
    __syncthreads();
    for (int ii = 0; ii < 8; ++ii) {
      s_r[rg + 8 * ii][cl] = u[ii];
      if (KEEP && on) a.U[(at * kQ + rg + 8 * ii) * P + p] = u[ii];
    }
    __syncthreads();
    if constexpr (!KEEP) {
      for (int ii = 0; ii < 8; ++ii) {
        const int i = rg + 8 * ii;
        float qS = 0.0f;
        for (int n = 0; n < N; ++n) qS = fmaf(a.qh[(ag + i) * N + n], s_S[n][cl], qS);
        float y = ex2((float)cum[i]) * qS;
        for (int j = 0; j <= i; ++j) y = fmaf(M[i * kQ + j], s_r[j][cl], y);
        if (on && i < cnt) st<IO>(a.y, (int64_t)(r0 + i) * a.ys + h * P + p, y);
      }
      __syncthreads();
    }
    const double last = cum[kQ - 1];
    for (int n = rg; n < N; n += 8) {
      float s = ex2((float)last) * s_S[n][cl];
      for (int j = 0; j < cnt; ++j)
        s = fmaf(a.kh[(ag + j) * N + n] * ex2((float)(last - cum[j])), s_r[j][cl], s);
      s_S[n][cl] = s;
    }
    __syncthreads();
  }
  if (!KEEP && a.state && on)
    for (int n = rg; n < N; n += 8) a.state[((own * a.H + h) * P + p) * N + n] = s_S[n][cl];
}

// against the blocks' order
template <typename IO>
__global__ void __launch_bounds__(256) delta_scan_bwd_kernel(const DeltaArgs a) {
  __shared__ float s_S[kMaxN][33], s_r[kQ][33], s_y[kQ][33];
  const DeltaSeq sq = a.seqs[blockIdx.x];
  const int h = blockIdx.y, N = a.N, P = a.P, g = h / a.per;
  const int cl = threadIdx.x & 31, rg = threadIdx.x >> 5, p = blockIdx.z * 32 + cl;
  const bool on = p < P;
  const int64_t own = ((int64_t)blockIdx.x * a.H + h) * P + p;
  for (int n = rg; n < N; n += 8) s_S[n][cl] = a.dfinal && on ? a.dfinal[own * N + n] : 0.0f;
  __syncthreads();
  const int nc = (sq.t1 - sq.t0 + kQ - 1) / kQ;
  for (int b = nc - 1; b >= 0; --b) {
    const int c = sq.c0 + b, r0 = sq.t0 + b * kQ, cnt = min(sq.t1 - r0, kQ);
    const int64_t at = (int64_t)c * a.H + h, ag = ((int64_t)c * a.G + g) * kQ;
    const double* cum = a.cum + at * kQ;
    const double last = cum[kQ - 1];
    const float *T = a.T + at * kQ * kQ, *M = a.M + at * kQ * kQ, *bb = a.b + at * kQ;
    if (on)
      for (int n = rg; n < N; n += 8) a.dS[(at * N + n) * P + p] = s_S[n][cl];
    for (int i = rg; i < kQ; i += 8)
      s_y[i][cl] = on && i < cnt ? ld<IO>(a.dy, (int64_t)(r0 + i) * a.gs + h * P + p) : 0.0f;
    __syncthreads();
    for (int j = rg; j < kQ; j += 8) {
      float u = 0.0f;
      for (int n = 0; n < N; ++n) u = fmaf(a.kh[(ag + j) * N + n], s_S[n][cl], u);
      u *= ex2((float)(last - cum[j]));
      for (int i = j; i < cnt; ++i) u = fmaf(M[i * kQ + j], s_y[i][cl], u);
      s_r[j][cl] = u;
    }
    __syncthreads();
    float dr[8];
    for (int ii = 0; ii < 8; ++ii) {
      const int j = rg + 8 * ii;
      dr[ii] = 0.0f;
      for (int i = j; i < cnt; ++i) dr[ii] = fmaf(T[i * kQ + j], s_r[i][cl], dr[ii]);
    }
    __syncthreads();
    for (int ii = 0; ii < 8; ++ii) {
      const int j = rg + 8 * ii;
      s_r[j][cl] = dr[ii];
      if (on) a.dR[(at * kQ + j) * P + p] = dr[ii];
      if (on && j < cnt) st<IO>(a.dv, (int64_t)(r0 + j) * a.dvs + h * P + p, bb[j] * dr[ii]);
    }
    __syncthreads();
    for (int n = rg; n < N; n += 8) {
      float s = ex2((float)last) * s_S[n][cl];
      for (int i = 0; i < cnt; ++i) {
        const float e = ex2((float)cum[i]);
        s = fmaf(e * a.qh[(ag + i) * N + n], s_y[i][cl], s);
        s = fmaf(-e * bb[i] * a.kh[(ag + i) * N + n], s_r[i][cl], s);
      }
      s_S[n][cl] = s;
    }
    __syncthreads();
  }
  if (a.dh0 && on)
    for (int n = rg; n < N; n += 8) a.dh0[own * N + n] = s_S[n][cl];
}

// ---------------------------------------------------------------- gradients of a block's rows and scalars

// one workgroup per block and head
template <typename IO>
__global__ void __launch_bounds__(256) delta_grad_kernel(const DeltaArgs a) {
  __shared__ float s_m[kQ][kQ + 1], s_l[kQ][kQ + 1], s_mm[kQ][kQ + 1], s_b[kQ], s_db[kQ], s_tail[kQ], s_red[256];
  __shared__ double s_g[kQ], s_dg[kQ];
  const int c = blockIdx.x, h = blockIdx.y, N = a.N, P = a.P, g = h / a.per;
  if (c >= a.head->nchunk) return;
  const DeltaChunk ck = a.chunks[c];
  const int tid = threadIdx.x, cnt = ck.r1 - ck.r0;
  const int64_t at = (int64_t)c * a.H + h, ag = ((int64_t)c * a.G + g) * kQ;
  const float *kh = a.kh + ag * N, *qh = a.qh + ag * N, *U = a.U + at * kQ * P, *dR = a.dR + at * kQ * P;
  const float *S = a.S + at * N * P, *dS = a.dS + at * N * P;
  if (tid < kQ) s_g[tid] = a.cum[at * kQ + tid], s_b[tid] = a.b[at * kQ + tid];
  __syncthreads();
  for (int u = tid; u < kQ * kQ; u += 256) {
    const int i = u >> 6, j = u & 63;
    float m = 0.0f, l = 0.0f, mm = 0.0f;
    if (j <= i && i < cnt) {
      float kk = 0.0f, qk = 0.0f;
      for (int p = 0; p < P; ++p) {
        m = fmaf(ld<IO>(a.dy, (int64_t)(ck.r0 + i) * a.gs + h * P + p), U[j * P + p], m);
        l = fmaf(-dR[i * P + p], U[j * P + p], l);
      }
      for (int n = 0; n < N; ++n) {
        kk = fmaf(kh[i * N + n], kh[j * N + n], kk);
        qk = fmaf(qh[i * N + n], kh[j * N + n], qk);
      }
      const float D = ex2((float)(s_g[i] - s_g[j]));
      m *= D;
      l = j < i ? l * D : 0.0f;
      // what the running sum's gradient takes from here; the diagonal's cancels
      mm = j < i ? fmaf(m, qk, l * kk * s_b[i]) : 0.0f;
      s_l[i][j] = l;
      s_mm[i][j] = mm;
      s_m[i][j] = m;
    } else {
      s_l[i][j] = s_m[i][j] = s_mm[i][j] = 0.0f;
    }
  }
  __syncthreads();
  const double last = s_g[kQ - 1];
  // row i, four lanes a row
  const int i = tid >> 2, ln = tid & 3;
  const float e = ex2((float)s_g[i]), et = ex2((float)(last - s_g[i])), bi = s_b[i];
  float qq = 0.0f, rk = 0.0f, tail = 0.0f, db = 0.0f, SdS = 0.0f;
  for (int n = ln; n < N; n += 4) {
    float yS = 0.0f, rS = 0.0f, uS = 0.0f;
    if (i < cnt)
      for (int p = 0; p < P; ++p) {
        const float s = S[(int64_t)n * P + p];
        yS = fmaf(ld<IO>(a.dy, (int64_t)(ck.r0 + i) * a.gs + h * P + p), s, yS);
        rS = fmaf(dR[i * P + p], s, rS);
        uS = fmaf(U[i * P + p], dS[(int64_t)n * P + p], uS);
      }
    yS *= e; rS *= e; uS *= et;
    const float kn = kh[i * N + n], qn = qh[i * N + n];
    qq = fmaf(yS, qn, qq);
    rk = fmaf(rS, kn, rk);
    tail = fmaf(uS, kn, tail);
    float dq = yS, dk = uS - bi * rS;
    for (int j = 0; j < kQ; ++j) {
      if (j <= i) dq = fmaf(s_m[i][j], kh[j * N + n], dq);
      if (j < i) dk = fmaf(s_l[i][j] * bi, kh[j * N + n], dk);
      if (j >= i) dk = fmaf(s_m[j][i], qh[j * N + n], dk);
      if (j > i) dk = fmaf(s_l[j][i] * s_b[j], kh[j * N + n], dk);
    }
    a.dqh[(at * kQ + i) * N + n] = dq;
    a.dkh[(at * kQ + i) * N + n] = dk;
  }
  // S . dS over the whole block
  for (int64_t u = tid; u < (int64_t)N * P; u += 256) SdS = fmaf(S[u], dS[u], SdS);
  if (i < cnt) {
    for (int p = ln; p < P; p += 4)
      db = fmaf(dR[i * P + p], ld<IO>(a.v, (int64_t)(ck.r0 + i) * a.vs + h * P + p), db);
    for (int j = ln; j < i; j += 4) {
      float kk = 0.0f;
      for (int n = 0; n < N; ++n) kk = fmaf(kh[i * N + n], kh[j * N + n], kk);
      db = fmaf(s_l[i][j], kk, db);
    }
  }
  qq = lane_sum<4>(qq); rk = lane_sum<4>(rk); tail = lane_sum<4>(tail); db = lane_sum<4>(db);
  if (ln == 0) {
    double d = (double)qq - (double)(bi * rk) - (double)tail;
    for (int j = 0; j < kQ; ++j) d += (double)s_mm[i][j] - (double)s_mm[j][i];
    s_dg[i] = d;
    s_db[i] = db - rk;
    s_tail[i] = tail;
  }
  s_red[tid] = SdS;
  __syncthreads();
  if (tid == 0) {
    double sum = 0.0;
    for (int t = 0; t < 256; ++t) sum += (double)s_red[t];
    sum *= (double)ex2((float)last);
    for (int j = 0; j < kQ; ++j) sum += (double)s_tail[j];
    double run = sum;
    float dA = 0.0f, dbias = 0.0f;
    for (int j = kQ - 1; j >= 0; --j) {
      run += s_dg[j];
      if (j >= cnt) continue;
      const int64_t r = ck.r0 + j;
      const float raw = ld<IO>(a.dt, r * a.ds + h) + (a.dt_bias ? a.dt_bias[h] : 0.0f);
      const float dg = (float)run, dt = a.softplus ? softplus(raw) : raw;
      const float ddt = dg * a.A[h] * (a.softplus ? sigmoid(raw) : 1.0f);
      dA = fmaf(dg, dt, dA);
      dbias += ddt;
      st<IO>(a.ddt, r * a.dds + h, ddt);
      const float b = s_b[j];
      st<IO>(a.dbeta, r * a.dbs + h, s_db[j] * (a.sigmoid ? b * (1.0f - b) : 1.0f));
    }
    a.part[at * 2] = dA;
    a.part[at * 2 + 1] = dbias;
  }
}

// the heads of a group together, and the normalisation: one wave a row
template <typename IO>
__global__ void __launch_bounds__(256) delta_qk_grad_kernel(const DeltaArgs a) {
  const int c = blockIdx.x, g = blockIdx.y, N = a.N;
  if (c >= a.head->nchunk) return;
  const DeltaChunk ck = a.chunks[c];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = wave; i < ck.r1 - ck.r0; i += 4) {
    const int64_t r = ck.r0 + i;
    for (int which = 0; which < 2; ++which) {
      const void* p = which ? a.k : a.q;
      const int64_t at = r * (which ? a.ks : a.qs) + (int64_t)g * N;
      float x[4], d[4], ss = 0.0f, xd = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = lane + 64 * j;
        x[j] = n < N ? ld<IO>(p, at + n) : 0.0f;
        d[j] = 0.0f;
        if (n < N)
          for (int m = 0; m < a.per; ++m)
            d[j] += (which ? a.dkh : a.dqh)[(((int64_t)c * a.H + g * a.per + m) * kQ + i) * N + n];
        ss = fmaf(x[j], x[j], ss);
      }
      const float f = a.norm ? rsqrtf(lane_sum<64>(ss) + a.eps) : 1.0f, sc = which ? 1.0f : a.scale;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] *= f, xd = fmaf(x[j], d[j], xd);
      xd = a.norm ? lane_sum<64>(xd) : 0.0f;
      const int64_t to = r * (which ? a.dks : a.dqs) + (int64_t)g * N;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (lane + 64 * j < N) st<IO>(which ? a.dk : a.dq, to + lane + 64 * j, (d[j] - x[j] * xd) * f * sc);
    }
  }
}

// dA and ddt_bias: one workgroup a head, blocks in runs of a fixed order
__global__ void __launch_bounds__(256) delta_sum_kernel(const DeltaArgs a) {
  __shared__ double red[2][256];
  const int h = blockIdx.x, t = threadIdx.x, nc = a.head->nchunk;
  double s0 = 0.0, s1 = 0.0;
  for (int c = t; c < nc; c += 256) {
    s0 += a.part[((int64_t)c * a.H + h) * 2];
    s1 += a.part[((int64_t)c * a.H + h) * 2 + 1];
  }
  red[0][t] = s0;
  red[1][t] = s1;
  __syncthreads();
  if (t < 2) {
    double s = 0.0;
    for (int k = 0; k < 256; ++k) s += red[t][k];
    float* out = t ? a.ddt_bias : a.dA;
    if (out) out[h] = (float)s;
  }
}

// rows of no sequence have no gradients
template <typename IO>
__global__ void __launch_bounds__(256) delta_zero_kernel(const DeltaArgs a) {
  const int first = a.head->first, last = a.head->last;
  const int64_t gn = (int64_t)a.G * a.N, hp = (int64_t)a.H * a.P, wide = 2 * gn + hp + 2 * a.H;
  const int64_t rows = a.tokens - (last - first);
  for (int64_t u = blockIdx.x * 256ll + threadIdx.x; u < rows * wide; u += gridDim.x * 256ll) {
    int64_t r = u / wide, c = u % wide;
    if (r >= first) r += last - first;
    if (c < gn) { st<IO>(a.dq, r * a.dqs + c, 0.0f); continue; }
    c -= gn;
    if (c < gn) { st<IO>(a.dk, r * a.dks + c, 0.0f); continue; }
    c -= gn;
    if (c < hp) { st<IO>(a.dv, r * a.dvs + c, 0.0f); continue; }
    c -= hp;
    if (c < a.H) st<IO>(a.ddt, r * a.dds + c, 0.0f);
    else st<IO>(a.dbeta, r * a.dbs + c - a.H, 0.0f);
  }
}

// ---------------------------------------------------------------- a block's operands
//
// The products run on the matrix cores in fp16 pieces.  A row of k or q is scaled by a
// power of two from its own largest value: bf16 values are then fp16 values (down to 2^-38
// of the row's largest), float32 ones two pieces (22 bits); its length goes with the row's
// scalars.  T, M, the state and what is made of them are float32, taken in two pieces each
// (22 bits; lo x lo, 2^-24 of a product, is left out), T and M scaled by row, the rest by
// column, which is a channel of v: a value is held to 2^-22 of itself or 2^-39 of the largest
// beside it.  Accumulators, the state, statistics and running sums (float64) are float32 or
// more.
//
// Order of rows and states: tile tt's row r of 16 is token 32 (tt / 2) + 8 (r / 4) +
// 4 (tt % 2) + r % 4, and the states' tiles alike, so that a lane of the matrix
// instructions, which has rows 4 q .. 4 q + 3 of a result's tile, has eight neighbours in a
// pair of tiles: what it needs of the next product's other operand, without any exchange.

__device__ __forceinline__ int place_of(int tile, int r) { return 32 * (tile >> 1) + 8 * (r >> 2) + 4 * (tile & 1) + (r & 3); }

constexpr int kTri = 6;  // 16 x 32 tiles of T and M on or below the diagonal
__device__ __forceinline__ int tri(int tt, int kb) { return tt < 2 ? tt : 2 * tt - 2 + kb; }

// Bytes of the operands of a (block, group): k and q, rows of 2 NP bytes a piece, a row's
// 16-byte parts in an order of its own (part()); and of a (block, head): T, M, scalars.
template <typename IO, int NT>
struct Ops {
  static constexpr int KP = sizeof(IO) == 4 ? 2 : 1, NP = 16 * NT, RB = 2 * NP;
  static constexpr int piece = kQ * RB, kq = KP * piece;  // one piece; all of k or q
  static constexpr int group = 2 * kq;
  static constexpr int tri_piece = kTri * 1024;
  static constexpr int t = 0, m = 2 * tri_piece, sc = 4 * tri_piece, head = sc + 2048;
  // where 16-byte part c of row r lies: rows that are read together are in different banks
  __device__ static __forceinline__ int part(int r, int c) {
    constexpr int rows = RB >= 256 ? 1 : 256 / RB;  // rows in one round of the banks
    const int f = rows == 1 ? (r & 3) | (r >> 3 & 3) << 2 : rows == 2 ? (r >> 1 & 1) | (r >> 3 & 3) << 1 : r >> 3 & 3;
    return r * RB + ((c ^ f) << 4);
  }
};
// a head's scalars: places of 64 floats each
enum { kS1, kBeta, kS2, kS3, kFT, kFM, kEC };

__device__ __forceinline__ float max_nan(float a, float b) { return max3_nan(0.0f, a, b); }
// 2^x of a running sum: what float32 leaves off it goes in to first order
__device__ __forceinline__ float ex2(double x) {
  const float hi = (float)x;
  return ex2(hi) * fmaf((float)(x - (double)hi), kLn2, 1.0f);
}
template <int LN>
__device__ __forceinline__ float lane_max(float v) {
#pragma unroll
  for (int d = 1; d < LN; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}
__device__ __forceinline__ f4 mfma32(float a, float b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// eight neighbours of a row as float32; zeros from n on
template <typename IO, bool VEC>
__device__ __forceinline__ void load8(const void* p, int64_t at, int n, float (&x)[8]) {
  if constexpr (VEC) {
    constexpr int E = 16 / sizeof(IO);
    if (n > 0) {
#pragma unroll
      for (int k = 0; k < 8 / E; ++k) {
        Vec<IO, E> v;
        if (E * k < n) v.load(p, at + E * k);
#pragma unroll
        for (int j = 0; j < E; ++j) x[E * k + j] = E * k < n ? v.get(j) : 0.0f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j < n ? ld<IO>(p, at + j) : 0.0f;
  }
}

// One workgroup per block and head; the first head of a group writes its k and q.
template <typename IO, int NT, bool VEC>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(3))) delta_ops_kernel(const DeltaArgs a) {
  using O = Ops<IO, NT>;
  constexpr int KP = O::KP, LN = 2 * NT, RW = 256 / LN, LD = kQ + 4;
  constexpr int lds = O::group > 2 * kQ * LD * 4 ? O::group : 2 * kQ * LD * 4;
  __shared__ __align__(16) char s_buf[lds];
  __shared__ float s_len[2][kQ];
  __shared__ __align__(16) double s_cum[kQ];
  __shared__ float s_b[kQ];
  __shared__ int s_bad;
  const int c = blockIdx.x, h = blockIdx.y, g = h / a.per, N = a.N;
  if (c >= a.head->nchunk) return;
  const DeltaChunk ck = a.chunks[c];
  const int tid = threadIdx.x, lane = tid & 63, i16 = lane & 15, q4 = lane >> 4, cnt = ck.r1 - ck.r0;
  const int tt = __builtin_amdgcn_readfirstlane(tid >> 6);
  float gr = 0.0f, b = 0.0f;
  if (tt == 0 && lane < cnt) row_scalars<IO>(a, ck.r0 + lane, h, gr, b);
  // ---- rows of k and q: scaled, their lengths
#pragma unroll
  for (int which = 0; which < 2; ++which) {
#pragma unroll 4
    for (int i0 = 0; i0 < kQ; i0 += RW) {
      const int i = i0 + tid / LN, p = tid % LN;
      float x[8], m = 0.0f, ss = 0.0f;
      load8<IO, VEC>(which ? a.q : a.k, (int64_t)(ck.r0 + min(i, cnt - 1)) * (which ? a.qs : a.ks) + (int64_t)g * N + 8 * p,
                     i < cnt ? N - 8 * p : 0, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, finite(x[j]) ? fabsf(x[j]) : 0.0f);
      const int e = shift_for(lane_max<LN>(m));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = __builtin_amdgcn_ldexpf(x[j], e);
        ss = fmaf(x[j], x[j], ss);
      }
      ss = lane_sum<LN>(ss);
      // x / sqrt(|x|^2 + eps) from the scaled row
      if (p == 0)
        s_len[which][i] = (a.norm ? rsqrtf(ss + __builtin_amdgcn_ldexpf(a.eps, 2 * e)) : two(-e)) * (which ? a.scale : 1.0f);
      h8 hi, lo;
      pieces(x, hi, lo);
      char* to = s_buf + which * O::kq + O::part(i, p);
      *reinterpret_cast<h8*>(to) = hi;
      if constexpr (KP == 2) *reinterpret_cast<h8*>(to + O::piece) = lo;
    }
  }
  __syncthreads();
  if (h == g * a.per) {
    char* out = a.gops + ((int64_t)c * a.G + g) * O::group;
#pragma unroll 4
    for (int u = tid * 16; u < O::group; u += 4096) *reinterpret_cast<u4*>(out + u) = *reinterpret_cast<const u4*>(s_buf + u);
  }
  // ---- their products: lane (i, q) has row i of tile tt at columns 32 kb + 8 q + {0 .. 7}
  f4 kk[2][2] = {}, qk[2][2] = {};
  const int row = place_of(tt, i16);
#pragma unroll
  for (int m = 0; m < NT / 2; ++m) {
    asm volatile("" ::: "memory");  // else all the operands are read ahead
    h8 kb_[KP], qb[KP];
#pragma unroll
    for (int p = 0; p < KP; ++p) {
      kb_[p] = *reinterpret_cast<const h8*>(s_buf + p * O::piece + O::part(row, 4 * m + q4));
      qb[p] = *reinterpret_cast<const h8*>(s_buf + O::kq + p * O::piece + O::part(row, 4 * m + q4));
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      if (kb > (tt >> 1)) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        h8 ka[KP];
#pragma unroll
        for (int p = 0; p < KP; ++p)
          ka[p] = *reinterpret_cast<const h8*>(s_buf + p * O::piece + O::part(place_of(2 * kb + e, i16), 4 * m + q4));
        if constexpr (KP == 2) {
          kk[kb][e] = mfma(ka[1], kb_[0], kk[kb][e]);
          kk[kb][e] = mfma(ka[0], kb_[1], kk[kb][e]);
          qk[kb][e] = mfma(ka[1], qb[0], qk[kb][e]);
          qk[kb][e] = mfma(ka[0], qb[1], qk[kb][e]);
        }
        kk[kb][e] = mfma(ka[0], kb_[0], kk[kb][e]);
        qk[kb][e] = mfma(ka[0], qb[0], qk[kb][e]);
      }
    }
  }
  float* s_l = reinterpret_cast<float*>(s_buf);  // L, then T beside it: k and q are used up
  float* s_t = s_l + kQ * LD;
  {
    char* out = a.hops + ((int64_t)c * a.H + h) * O::head;
    float* sc = reinterpret_cast<float*>(out + O::sc);
    if (tt == 0) {
      const double cum = wave_scan((double)gr), tot = lane63(cum);
      s_cum[lane] = cum;
      s_b[lane] = b;
      const float e = ex2(cum), lk = s_len[0][lane], lq = s_len[1][lane];
      sc[64 * kS1 + lane] = e * lk;
      sc[64 * kBeta + lane] = b;
      sc[64 * kS2 + lane] = e * lq;
      sc[64 * kS3 + lane] = ex2(tot - cum) * lk;
      sc[64 * kEC + lane] = ex2(tot);
      if (lane == 0) s_bad = kQ;
    }
    __syncthreads();  // k and q have been read, too
    // ---- L into LDS, M out
    const double ci = s_cum[row];
    const float bi = s_b[row], lki = s_len[0][row], lqi = s_len[1][row];
    float mv[2][8], mx = 0.0f;
    bool bad = false;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      if (kb > (tt >> 1)) break;
      float lv[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int col = 32 * kb + 8 * q4 + e;
        const float w = ex2((float)(ci - s_cum[col])) * s_len[0][col];
        const float l = bi * lki * (w * kk[kb][e >> 2][e & 3]);
        const float m = lqi * (w * qk[kb][e >> 2][e & 3]);
        lv[e] = col < row ? l : 0.0f;
        mv[kb][e] = col <= row ? m : 0.0f;
        if (!finite(lv[e])) bad = true, lv[e] = 0.0f;
        mx = finite(mv[kb][e]) ? fmaxf(mx, fabsf(mv[kb][e])) : mx;
      }
      f4* to = reinterpret_cast<f4*>(s_l + row * LD + 32 * kb + 8 * q4);
      to[0] = *reinterpret_cast<const f4*>(lv);
      to[1] = *reinterpret_cast<const f4*>(lv + 4);
    }
    if (bad) atomicMin(&s_bad, row);
    {
      const int sh = shift_for(row_max(mx));
      const float f = two(sh);
      if (q4 == 0) sc[64 * kFM + row] = two(-sh);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        if (kb > (tt >> 1)) break;
#pragma unroll
        for (int e = 0; e < 8; ++e) mv[kb][e] *= f;
        h8 hi, lo;
        pieces(mv[kb], hi, lo);
        char* to = out + O::m + (tri(tt, kb) * 64 + lane) * 16;
        *reinterpret_cast<h8*>(to) = hi;
        *reinterpret_cast<h8*>(to + O::tri_piece) = lo;
      }
    }
    __syncthreads();
    // ---- T: the inverses of the four diagonal tiles by substitution, a lane a column ...
    {
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float l[16];
#pragma unroll
        for (int m = 0; m < i; m += 4) *reinterpret_cast<f4*>(l + m) = *reinterpret_cast<const f4*>(s_l + (16 * tt + i) * LD + 16 * tt + m);
        x[i] = i == i16 ? 1.0f : 0.0f;
#pragma unroll
        for (int m = 0; m < i; ++m) x[i] = fmaf(-l[m], x[m], x[i]);
        if (i & 1) asm volatile("" ::: "memory");  // else all of L is held in registers
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if ((i >> 2) == q4) s_t[(16 * tt + i) * LD + 16 * tt + i16] = x[i];
    }
    __syncthreads();
    // ---- ... and the tiles below them, T_ij = -T_ii sum_{j <= m < i} L_im T_mj, in float32 products
    if (tt < 3) {
      f4 tc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < tt) continue;
        if (i == tt) {
#pragma unroll
          for (int r = 0; r < 4; ++r) tc[i][r] = s_t[(16 * i + 4 * q4 + r) * LD + 16 * i + i16];
          continue;
        }
        f4 y = {};
#pragma unroll
        for (int m = 0; m < i; ++m) {
          if (m < tt) continue;
          const f4 l = *reinterpret_cast<const f4*>(s_l + (16 * i + i16) * LD + 16 * m + 4 * q4);
#pragma unroll
          for (int r = 0; r < 4; ++r) y = mfma32(l[r], tc[m][r], y);
        }
        const f4 t = *reinterpret_cast<const f4*>(s_t + (16 * i + i16) * LD + 16 * i + 4 * q4);
        f4 z = {};
#pragma unroll
        for (int r = 0; r < 4; ++r) z = mfma32(-t[r], y[r], z);
        tc[i] = z;
#pragma unroll
        for (int r = 0; r < 4; ++r) s_t[(16 * i + 4 * q4 + r) * LD + 16 * tt + i16] = z[r];
      }
    }
    __syncthreads();
    {
      const bool lost = row >= s_bad;
      float t[2][8], m = 0.0f;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        if (kb > (tt >> 1)) break;
        const f4* s = reinterpret_cast<const f4*>(s_t + row * LD + 32 * kb + 8 * q4);
        *reinterpret_cast<f4*>(t[kb]) = s[0];
        *reinterpret_cast<f4*>(t[kb] + 4) = s[1];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          t[kb][e] = 32 * kb + 8 * q4 + e <= row ? t[kb][e] : 0.0f;
          m = finite(t[kb][e]) ? fmaxf(m, fabsf(t[kb][e])) : m;
        }
      }
      const int sh = shift_for(row_max(m));
      const float f = lost ? __builtin_nanf("") : two(sh);
      if (q4 == 0) sc[64 * kFT + row] = two(-sh);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        if (kb > (tt >> 1)) break;
#pragma unroll
        for (int e = 0; e < 8; ++e) t[kb][e] *= f;
        h8 hi, lo;
        pieces(t[kb], hi, lo);
        char* to = out + O::t + (tri(tt, kb) * 64 + lane) * 16;
        *reinterpret_cast<h8*>(to) = hi;
        *reinterpret_cast<h8*>(to + O::tri_piece) = lo;
      }
    }
  }
}

// ---------------------------------------------------------------- from block to block

// four rows of a column of 16-bit values, transposed on the way from LDS: lane i of
// sixteen points at four neighbours of row i / 4 and gets column i of all four rows
__device__ __forceinline__ u2 read_tr(const char* p) {
  typedef short s4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)p));
}
__device__ __forceinline__ h8 joined_tr(u2 a, u2 b) { return __builtin_bit_cast(h8, (u4){a.x, a.y, b.x, b.y}); }

// Copies BYTES from global memory to LDS, 16 bytes a lane, as stage() does, but out of the
// compiler's sight: it would wait for them before the next read of LDS, whatever that reads.
// landed() waits for them, meet() for the other waves.
template <int WV, int BYTES>
__device__ __forceinline__ void send(const char* from, char* to) {
  static_assert(BYTES % 1024 == 0, "whole waves");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)to + wave * 1024;
  const uint32_t off = wave * 1024 + lane * 16;
#pragma unroll
  for (int i = 0; i < (BYTES / 1024 + WV - 1) / WV; ++i)
    if (BYTES / 1024 % WV == 0 || (i * WV + wave) * 1024 < BYTES)
      asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at + i * WV * 1024), "v"(off),
                   "s"(from + i * WV * 1024)
                   : "memory", "m0");
}
// All of this wave's memory accesses have ended (a wait that the compiler sees).
__device__ __forceinline__ void landed() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70);
  asm volatile("" ::: "memory");
}

// The power of two for a column: its largest finite value over the four lanes that share it;
// bad: whether one of the wave's columns has a value that is not finite.
template <int PT, int NV>
__device__ __forceinline__ bool column_shifts(const f4 (&v)[NV][PT], int (&sh)[PT]) {
  float mx[PT];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < PT; ++e) {
    mx[e] = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int r = 0; r < 4; r += 2) mx[e] = max3_nan(mx[e], v[k][e][r], v[k][e][r + 1]);
    bad = bad || !finite(mx[e]);
  }
  bad = __any(bad);
  if (bad) {
    rarely();
#pragma unroll
    for (int e = 0; e < PT; ++e) {
      mx[e] = 0.0f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (finite(v[k][e][r])) mx[e] = fmaxf(mx[e], fabsf(v[k][e][r]));
    }
  }
#pragma unroll
  for (int e = 0; e < PT; ++e) sh[e] = shift_for(row_max(mx[e]));
  return bad;
}
// the pieces of a pair of tiles of a column, scaled
__device__ __forceinline__ void pair_pieces(const f4& x, const f4& y, float f, h8& hi, h8& lo) {
  float v[8];
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = x[r] * f, v[r + 4] = y[r] * f;
  pieces(v, hi, lo);
}

// A workgroup walks a sequence's blocks with WV waves of 16 PT channels of one head each, the
// states of a wave's channels in its accumulators.  DB: the next block's operands
// come while this block's are used.
template <typename IO, int NT, int PT, int WV, bool FAST>
__global__ void __launch_bounds__(64 * WV) delta_walk_kernel(const DeltaArgs a, int units) {
  using O = Ops<IO, NT>;
  constexpr int KP = O::KP, B = O::group + O::head, PB = 16 * PT;
  constexpr bool DB = 2 * B <= 160 * 1024;
  __shared__ __align__(16) char s_op[(DB ? 2 : 1) * B];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int i16 = lane & 15, q4 = lane >> 4;
  // eight dies take the workgroups by turns: the units of a head, and the heads of a
  // group where there are eight groups, share a die's cache
  const int item = blockIdx.x / (8 * units) * 8 + blockIdx.x % 8, unit = blockIdx.x / 8 % units;
  if (item >= a.nseq * a.H) return;
  const int s = item / a.H, g = item % a.G, h = g * a.per + item % a.H / a.G;
  const DeltaSeq sq = a.seqs[s];
  if (sq.slot < 0) return;
  const int N = a.N, P = a.P, p0 = (unit * WV + wave) * PB;
  const bool on = p0 < P;  // else the wave only helps to stage
  int col[PT];
#pragma unroll
  for (int e = 0; e < PT; ++e) {
    const int p = p0 + PT * i16 + e;
    col[e] = h * P + (p < P ? p : FAST ? (on ? p0 : 0) + e : 0);
  }
  const int nc = (sq.t1 - sq.t0 + kQ - 1) / kQ;
  auto stage_block = [&](int b) {
    const int64_t c = sq.c0 + b;
    char* to = s_op + (DB ? (b & 1) * B : 0);
    send<WV, O::group>(a.gops + (c * a.G + g) * O::group, to);
    send<WV, O::head>(a.hops + (c * a.H + h) * O::head, to + O::group);
  };
  if (nc > 0) stage_block(0);

  // lane (i, q) holds the states 32 m + 8 q + {0 .. 3} of its channels in tile 2 m, {4 .. 7} in 2 m + 1
  f4 S[NT][PT];
  const float* src = sq.resume ? a.state : nullptr;
#pragma unroll
  for (int e = 0; e < PT; ++e)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = 32 * (nt >> 1) + 8 * q4 + 4 * (nt & 1);
      f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
      if (src) {
        const float* at = src + ((int64_t)sq.slot * a.H * P + col[e]) * N + n;
        if constexpr (FAST) {
          if (n < N) v = *reinterpret_cast<const f4*>(at);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < N) v[r] = at[r];
        }
      }
      S[nt][e] = v;
    }
  // v of a block's rows 32 kb + 8 q + j.  Whole blocks go by an address of the row, the
  // same in all lanes, and the lane's own offset
  constexpr bool PAIR = FAST && PT == 2 && sizeof(IO) == 2;
  using Raw = typename std::conditional<PAIR, uint32_t, IO>::type;
  constexpr int RV = PAIR ? 1 : PT;
  Raw vr[2][8][RV];
  const uint32_t v_own = (uint32_t)((8 * q4 * a.vs + col[0]) * sizeof(IO)), y_own = (uint32_t)((8 * q4 * a.ys + col[0]) * sizeof(IO));
  auto fetch = [&](int b) {
    const int r0 = sq.t0 + b * kQ, cnt = min(sq.t1 - r0, kQ);
    if (FAST && cnt == kQ) {
      const char* row = static_cast<const char*>(a.v) + (int64_t)r0 * a.vs * sizeof(IO);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const char* at = row + (32 * kb + j) * a.vs * (int64_t)sizeof(IO);
#pragma unroll
          for (int e = 0; e < RV; ++e) vr[kb][j][e] = *reinterpret_cast<const Raw*>(at + (v_own + e * (uint32_t)sizeof(IO)));
        }
    } else {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const IO* at = static_cast<const IO*>(a.v) + (r0 + min(32 * kb + 8 * q4 + j, cnt - 1)) * a.vs;
#pragma unroll
          for (int e = 0; e < RV; ++e) vr[kb][j][e] = *reinterpret_cast<const Raw*>(at + col[e]);
        }
    }
  };
  auto value = [&](int kb, int j, int e) {
    if constexpr (PAIR) return __uint_as_float(e ? vr[kb][j][0] & 0xffff0000u : vr[kb][j][0] << 16);
    else if constexpr (sizeof(IO) == 2) return __uint_as_float((uint32_t)vr[kb][j][e] << 16);
    else return (float)vr[kb][j][e];
  };
  if (nc > 0 && on) fetch(0);

  // T or M times the pieces of a column's rows
  auto triangle = [&](const char* op, const h8 (&hi)[2][PT], const h8 (&lo)[2][PT], f4 (&out)[4][PT]) {
    h8 xh[kTri], xl[kTri];
#pragma unroll
    for (int i = 0; i < kTri; ++i) {
      xh[i] = *reinterpret_cast<const h8*>(op + (i * 64 + lane) * 16);
      xl[i] = *reinterpret_cast<const h8*>(op + O::tri_piece + (i * 64 + lane) * 16);
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int tt = 2 * kb; tt < 4; ++tt)
#pragma unroll
          for (int e = 0; e < PT; ++e)
            out[tt][e] = mfma(p == 0 ? xl[tri(tt, kb)] : xh[tri(tt, kb)], p == 1 ? lo[kb][e] : hi[kb][e], out[tt][e]);
  };

  for (int b = 0; b < nc; ++b) {
    const int r0 = sq.t0 + b * kQ, cnt = min(sq.t1 - r0, kQ);
    landed();
    meet();  // this block's operands are there; the waves are done with the last block's
    // v has come too: else the compiler would wait for it behind what is sent next
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < RV; ++e) asm volatile("" : "+v"(vr[kb][j][e]));
    if (DB && b + 1 < nc) stage_block(b + 1);
    const char* op = s_op + (DB ? (b & 1) * B : 0);
    const char* hop = op + O::group;
    const float* sc = reinterpret_cast<const float*>(hop + O::sc);
    if (on) {
      // ---- k S and q S
      f4 ks[4][PT] = {}, qs[4][PT] = {};
      int sh[PT];
      column_shifts<PT, NT>(S, sh);
      float f[PT], fi[PT];
#pragma unroll
      for (int e = 0; e < PT; ++e) f[e] = two(sh[e]), fi[e] = two(-sh[e]);
#pragma unroll
      for (int m = 0; m < NT / 2; ++m) {
        h8 hi[PT], lo[PT];
#pragma unroll
        for (int e = 0; e < PT; ++e) pair_pieces(S[2 * m][e], S[2 * m + 1][e], f[e], hi[e], lo[e]);
        h8 ka[4][KP], qa[4][KP];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const int at = O::part(place_of(tt, i16), 4 * m + q4);
#pragma unroll
          for (int p = 0; p < KP; ++p) {
            ka[tt][p] = *reinterpret_cast<const h8*>(op + p * O::piece + at);
            qa[tt][p] = *reinterpret_cast<const h8*>(op + O::kq + p * O::piece + at);
          }
        }
        // eight results by turns: a product does not wait for the one before it
        auto all = [&](int p, const h8 (&x)[PT]) {
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int e = 0; e < PT; ++e) {
              ks[tt][e] = mfma(ka[tt][p], x[e], ks[tt][e]);
              qs[tt][e] = mfma(qa[tt][p], x[e], qs[tt][e]);
            }
        };
        all(0, lo);
        if constexpr (KP == 2) all(1, hi);
        all(0, hi);
      }
      // ---- R = b (v - e^G k S); q S to its size
      if (cnt < kQ) {
        rarely();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < RV; ++e) vr[kb][j][e] = 32 * kb + 8 * q4 + j < cnt ? vr[kb][j][e] : 0;
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const int t = place_of(tt, 4 * q4);
        const f4 s1 = *reinterpret_cast<const f4*>(sc + 64 * kS1 + t), be = *reinterpret_cast<const f4*>(sc + 64 * kBeta + t);
        const f4 s2 = *reinterpret_cast<const f4*>(sc + 64 * kS2 + t);
#pragma unroll
        for (int e = 0; e < PT; ++e)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            ks[tt][e][r] = be[r] * fmaf(-(s1[r] * fi[e]), ks[tt][e][r], value(tt >> 1, 4 * (tt & 1) + r, e));
            qs[tt][e][r] *= s2[r] * fi[e];
          }
      }
      if (b + 1 < nc) fetch(b + 1);
      // ---- U = T R.  What is not finite stays behind the first such row of its column:
      // 0 x Inf is not 0, so the products leave those rows out
      int first[PT];
#pragma unroll
      for (int e = 0; e < PT; ++e) first[e] = kQ;
      auto clean = [&](f4 (&v)[4][PT]) {
#pragma unroll
        for (int e = 0; e < PT; ++e) {
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (!finite(v[tt][e][r])) first[e] = min(first[e], place_of(tt, 4 * q4 + r));
          first[e] = min(first[e], __shfl_xor(first[e], 16, 64));
          first[e] = min(first[e], __shfl_xor(first[e], 32, 64));
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (place_of(tt, 4 * q4 + r) >= first[e]) v[tt][e][r] = 0.0f;
        }
      };
      bool bad = column_shifts<PT, 4>(ks, sh);
      if (bad) {
        rarely();
        clean(ks);
      }
      f4 u[4][PT] = {};
      {
        h8 hi[2][PT], lo[2][PT];
#pragma unroll
        for (int e = 0; e < PT; ++e) {
          f[e] = two(sh[e]), fi[e] = two(-sh[e]);
#pragma unroll
          for (int kb = 0; kb < 2; ++kb) pair_pieces(ks[2 * kb][e], ks[2 * kb + 1][e], f[e], hi[kb][e], lo[kb][e]);
        }
        triangle(hop + O::t, hi, lo, u);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const f4 ft = *reinterpret_cast<const f4*>(sc + 64 * kFT + place_of(tt, 4 * q4));
#pragma unroll
          for (int e = 0; e < PT; ++e)
#pragma unroll
            for (int r = 0; r < 4; ++r) u[tt][e][r] *= ft[r] * fi[e];
        }
      }
      bad |= column_shifts<PT, 4>(u, sh);
      if (bad) {
        rarely();
        clean(u);
      }
      // ---- y = e^G q S + M U
      {
        h8 hi[2][PT], lo[2][PT];
#pragma unroll
        for (int e = 0; e < PT; ++e) {
          f[e] = two(sh[e]), fi[e] = two(-sh[e]);
#pragma unroll
          for (int kb = 0; kb < 2; ++kb) pair_pieces(u[2 * kb][e], u[2 * kb + 1][e], f[e], hi[kb][e], lo[kb][e]);
        }
        f4 y[4][PT] = {};
        triangle(hop + O::m, hi, lo, y);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const f4 fm = *reinterpret_cast<const f4*>(sc + 64 * kFM + place_of(tt, 4 * q4));
#pragma unroll
          for (int e = 0; e < PT; ++e)
#pragma unroll
            for (int r = 0; r < 4; ++r) y[tt][e][r] = fmaf(y[tt][e][r], fm[r] * fi[e], qs[tt][e][r]);
        }
        if (bad) {
          rarely();
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int e = 0; e < PT; ++e)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (place_of(tt, 4 * q4 + r) >= first[e]) y[tt][e][r] = __builtin_nanf("");
        }
        auto write = [&](char* at, int tt, int r) {
          if constexpr (PAIR) {
            typedef __bf16 b2 __attribute__((ext_vector_type(2)));
            *reinterpret_cast<b2*>(at) = __builtin_convertvector((f2){y[tt][0][r], y[tt][PT - 1][r]}, b2);
          } else {
#pragma unroll
            for (int e = 0; e < PT; ++e)
              if (FAST || p0 + PT * i16 + e < P) st<IO>(at, e, y[tt][e][r]);
          }
        };
        if (FAST && cnt == kQ) {
          if (p0 + PT * i16 < P) {
            char* row = static_cast<char*>(a.y) + (int64_t)r0 * a.ys * sizeof(IO);
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                write(row + (32 * (tt >> 1) + 4 * (tt & 1) + r) * a.ys * (int64_t)sizeof(IO) + y_own, tt, r);
          }
        } else if (p0 + PT * i16 < P) {
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int t = place_of(tt, 4 * q4 + r);
              if (t < cnt) write(static_cast<char*>(a.y) + ((r0 + t) * a.ys + col[0]) * (int64_t)sizeof(IO), tt, r);
            }
        }
      }
      // ---- S = e^G64 S + sum_j k_j (e^(G64 - G_j) U_j)
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const f4 s3 = *reinterpret_cast<const f4*>(sc + 64 * kS3 + place_of(tt, 4 * q4));
#pragma unroll
        for (int e = 0; e < PT; ++e)
#pragma unroll
          for (int r = 0; r < 4; ++r) u[tt][e][r] *= s3[r];
      }
      column_shifts<PT, 4>(u, sh);
      {
        h8 hi[2][PT], lo[2][PT];
#pragma unroll
        for (int e = 0; e < PT; ++e) {
          f[e] = two(sh[e]), fi[e] = two(-sh[e]);
          if (bad) fi[e] = first[e] < kQ ? __builtin_nanf("") : fi[e];  // such a column has no state any more
#pragma unroll
          for (int kb = 0; kb < 2; ++kb) pair_pieces(u[2 * kb][e], u[2 * kb + 1][e], f[e], hi[kb][e], lo[kb][e]);
        }
        const float ec = sc[64 * kEC];
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += 2) {
          f4 d[2][PT] = {};
          h8 kt[2][2][KP];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
              // rows 32 kb + 8 q + i16 / 4 (and four on), states 16 n0 + 8 (i16 % 4) + 4 i + {0 .. 3}
              const int r = 32 * kb + 8 * q4 + (i16 >> 2), pt = 2 * n0 + (i16 & 3);
#pragma unroll
              for (int p = 0; p < KP; ++p)
                kt[i][kb][p] = joined_tr(read_tr(op + p * O::piece + O::part(r, pt) + 8 * i),
                                         read_tr(op + p * O::piece + O::part(r + 4, pt) + 8 * i));
            }
          auto all = [&](int kb, int p, const h8 (&x)[PT]) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < PT; ++e) d[i][e] = mfma(kt[i][kb][p], x[e], d[i][e]);
          };
#pragma unroll
          for (int kb = 0; kb < 2; ++kb) {
            all(kb, 0, lo[kb]);
            if constexpr (KP == 2) all(kb, 1, hi[kb]);
            all(kb, 0, hi[kb]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < PT; ++e)
#pragma unroll
              for (int r = 0; r < 4; ++r) S[n0 + i][e][r] = fmaf(d[i][e][r], fi[e], S[n0 + i][e][r] * ec);
        }
      }
    }
    if (!DB && b + 1 < nc) {
      meet();  // the waves are done with this block's operands
      stage_block(b + 1);
    }
  }
  if (!a.state || !on) return;
#pragma unroll
  for (int e = 0; e < PT; ++e)
    if (p0 + PT * i16 + e < P)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int n = 32 * (nt >> 1) + 8 * q4 + 4 * (nt & 1);
        float* at = a.state + ((int64_t)sq.slot * a.H * P + col[e]) * N + n;
        if constexpr (FAST) {
          if (n < N) *reinterpret_cast<f4*>(at) = S[nt][e];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < N) at[r] = S[nt][e][r];
        }
      }
}

// ---------------------------------------------------------------- one token a sequence

// One workgroup per entry, head and 256 / LN rows (channels), LN lanes a row with four
// states each.  With s = a S: u = b (v - s.k), y = s.q + u k.q, S' = s + u k^T: one pass
// over the state, both products at once.  VEC: a lane's states are neighbours.
template <typename IO, int LN, bool VEC>
__global__ void __launch_bounds__(256) delta_step_kernel(const DeltaArgs a, int splits) {
  constexpr int ROWS = 256 / LN;
  __shared__ __align__(16) float s_qk[2][kMaxN];
  const int tid = threadIdx.x, ln = tid % LN;
  const int64_t row = blockIdx.x / ((int64_t)a.H * splits);
  const int hs = (int)(blockIdx.x - row * a.H * splits), h = hs / splits, p = (hs - h * splits) * ROWS + tid / LN;
  const int64_t slot = a.slots ? (int64_t)a.slots[row] : row;
  if (slot < 0 || slot >= a.nslots) return;  // padding
  const int N = a.N, P = a.P, g = h / a.per;
  const bool on = p < P;
  float* own = a.state + ((slot * a.H + h) * P + (on ? p : 0)) * (int64_t)N;
  float s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = VEC ? 4 * ln + j : ln + LN * j;
    s[j] = on && n < N ? own[n] : 0.0f;
  }
  float gr, b;
  row_scalars<IO>(a, row, h, gr, b);
  const float dec = ex2(gr);
  const int wave = tid >> 6, lane = tid & 63;
  if (wave < 2) {
    float x[4], ss = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = lane + 64 * j;
      x[j] = n < N ? ld<IO>(wave ? a.k : a.q, row * (wave ? a.ks : a.qs) + (int64_t)g * N + n) : 0.0f;
      ss = fmaf(x[j], x[j], ss);
    }
    const float f = (a.norm ? rsqrtf(lane_sum<64>(ss) + a.eps) : 1.0f) * (wave ? 1.0f : a.scale);
#pragma unroll
    for (int j = 0; j < 4; ++j) s_qk[wave][lane + 64 * j] = x[j] * f;
  }
  __syncthreads();
  float q[4], k[4], sk = 0.0f, sq = 0.0f, kq = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = VEC ? 4 * ln + j : ln + LN * j;
    q[j] = s_qk[0][n];
    k[j] = s_qk[1][n];
    s[j] *= dec;
    sk = fmaf(s[j], k[j], sk);
    sq = fmaf(s[j], q[j], sq);
    kq = fmaf(k[j], q[j], kq);
  }
  sk = lane_sum<LN>(sk);
  sq = lane_sum<LN>(sq);
  kq = lane_sum<LN>(kq);
  if (!on) return;
  const int64_t at = (int64_t)h * P + p;
  const float u = b * (ld<IO>(a.v, row * a.vs + at) - sk);
  if (ln == 0) st<IO>(a.y, row * a.ys + at, fmaf(u, kq, sq));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = VEC ? 4 * ln + j : ln + LN * j;
    if (n < N) own[n] = fmaf(u, k[j], s[j]);
  }
}

// ---------------------------------------------------------------- host side

constexpr int64_t kMaxHeaddim = 256;

int check_delta_extents(int64_t tokens, int64_t nseq, int64_t nheads, int64_t headdim, int64_t ngroups,
                        int64_t dstate) {
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
  if (nheads > 16384) return fail(SSM_E_SHAPE, "nheads = %lld exceeds 16384", (long long)nheads);
  if (nseq > 0xfffff || tokens / kQ + nseq >= ((int64_t)1 << 22))
    return fail(SSM_E_SHAPE, "tokens = %lld, nseq = %lld: nseq is at most 2^20 - 1, tokens / 64 + nseq 2^22 - 1",
                (long long)tokens, (long long)nseq);
  // a workgroup for every block or sequence and head
  if (!grid_ok((tokens / kQ + nseq) * nheads, 1024))
    return fail(SSM_E_SHAPE, "too many blocks and heads for one call");
  return SSM_OK;
}

struct DeltaCall {  // extents as the entry points take them
  int64_t rows, nseq, nslots, H, P, G, N;
  int io;
};

// What the entry points check alike; fills a.  outs: the outputs; the state is one of them.
int check_delta(DeltaArgs& a, const DeltaCall& c, const Rows* outs, int nouts, const Rows* more, int nmore) {
  const struct { const void* p; const char* name; } req[] = {
      {a.q, "q"}, {a.k, "k"}, {a.v, "v"}, {a.dt, "dt"}, {a.beta, "beta"}, {a.A, "A"}};
  for (const auto& r : req)
    if (!r.p) return fail(SSM_E_NULL, "%s is NULL", r.name);
  int st = check_delta_extents(c.rows, c.nseq, c.H, c.P, c.G, c.N);
  if (st || (st = check_io(c.io))) return st;
  if (!(a.eps >= 0.0f) || a.eps > 3e38f) return fail(SSM_E_SHAPE, "eps is negative or not finite");
  if (!(a.scale >= -3e38f && a.scale <= 3e38f)) return fail(SSM_E_SHAPE, "scale is not finite");
  const int es = c.io == SSM_DTYPE_BF16 ? 2 : 4;
  const int64_t gn = c.G * c.N, hp = c.H * c.P;
  if (!product_ok(c.nslots > c.nseq ? c.nslots : c.nseq, hp, c.N, 4)) return fail(SSM_E_SHAPE, "tensor sizes overflow");
  if ((st = check_rows("q", a.q, a.qs, gn, c.rows, es)) || (st = check_rows("k", a.k, a.ks, gn, c.rows, es)) ||
      (st = check_rows("v", a.v, a.vs, hp, c.rows, es)) || (st = check_rows("dt", a.dt, a.ds, c.H, c.rows, es)) ||
      (st = check_rows("beta", a.beta, a.bs, c.H, c.rows, es)))
    return st;
  for (int i = 0; i < nouts; ++i)
    if (outs[i].p && (uintptr_t)outs[i].p % es) return fail(SSM_E_ALIGN, "%s is not aligned to its elements", outs[i].name);
  Rows ins[16] = {{a.q, c.rows, a.qs * es, gn * es, "q"}, {a.k, c.rows, a.ks * es, gn * es, "k"},
                  {a.v, c.rows, a.vs * es, hp * es, "v"}, {a.dt, c.rows, a.ds * es, c.H * es, "dt"},
                  {a.beta, c.rows, a.bs * es, c.H * es, "beta"}, flat(a.A, c.H * 4, "A"),
                  flat(a.dt_bias, c.H * 4, "dt_bias"), flat(a.cu, (c.nseq + 1) * 4, "cu_seqlens"),
                  flat(a.slots, c.nseq * 4, "slots"), flat(a.has, c.nseq, "has_state")};
  for (int i = 0; i < nmore; ++i) ins[10 + i] = more[i];
  if ((st = check_no_alias(outs, nouts, ins, 10 + nmore))) return st;
  a.tokens = c.rows; a.nseq = c.nseq; a.nslots = c.nslots;
  a.H = (int)c.H; a.P = (int)c.P; a.G = (int)c.G; a.N = (int)c.N; a.per = (int)(c.H / c.G);
  return SSM_OK;
}

int check_state(const DeltaArgs& a, const DeltaCall& c) {
  int st;
  if (a.state) {
    if ((st = check_extent("nslots", c.nslots))) return st;
    if (!a.slots && c.nslots < c.nseq)
      return fail(SSM_E_SHAPE, "nslots = %lld is less than the %lld sequences and slots is NULL",
                  (long long)c.nslots, (long long)c.nseq);
    if (!product_ok(c.nslots, c.H * c.P, c.N, 4)) return fail(SSM_E_SHAPE, "tensor sizes overflow");
    if (c.nslots > 0x7fffffff) return fail(SSM_E_SHAPE, "nslots = %lld is out of range", (long long)c.nslots);
    if ((uintptr_t)a.state & 3) return fail(SSM_E_ALIGN, "ssm_state is not aligned to its elements");
  } else if (a.slots || a.has) {
    return fail(SSM_E_NULL, "ssm_state is NULL beside slots or has_state");
  }
  return SSM_OK;
}

struct DeltaLayout {
  int nt;  // tiles of 16 states
  int64_t nchunk;
  int64_t chunks, seqs, gops, hops, qh, kh, T, M, cum, b, S, dS, U, dR, dqh, dkh, part, bytes;
};

DeltaLayout delta_layout(int64_t tokens, int64_t nseq, int64_t H, int64_t P, int64_t G, int64_t N, int io_dtype, bool bwd) {
  DeltaLayout l;
  memset(&l, 0, sizeof l);
  l.nt = N <= 32 ? 2 : N <= 64 ? 4 : N <= 128 ? 8 : 16;
  l.nchunk = tokens / kQ + nseq;
  int64_t at = 0;
  auto take = [&](int64_t n) {
    const int64_t o = at;
    at += (n + 255) / 256 * 256;
    return o;
  };
  const int64_t ch = l.nchunk * H;
  take(sizeof(DeltaHead));
  l.chunks = take(l.nchunk * sizeof(DeltaChunk));
  l.seqs = take(nseq * sizeof(DeltaSeq));
  if (!bwd) {
    l.gops = take(l.nchunk * G * 2 * kQ * l.nt * 32 * (io_dtype == SSM_DTYPE_BF16 ? 1 : 2));
    l.hops = take(ch * (4 * kTri * 1024 + 2048));
  }
  if (bwd) {
    l.qh = take(l.nchunk * G * kQ * N * 4);
    l.kh = take(l.nchunk * G * kQ * N * 4);
    l.T = take(ch * kQ * kQ * 4);
    l.M = take(ch * kQ * kQ * 4);
    l.cum = take(ch * kQ * 8);
    l.b = take(ch * kQ * 4);
    l.S = take(ch * N * P * 4);
    l.dS = take(ch * N * P * 4);
    l.U = take(ch * kQ * P * 4);
    l.dR = take(ch * kQ * P * 4);
    l.dqh = take(ch * kQ * N * 4);
    l.dkh = take(ch * kQ * N * 4);
    l.part = take(ch * 8);
  }
  l.bytes = at;
  return l;
}

int check_workspace(const void* ws, int64_t have, int64_t need) {
  if (have < need)
    return fail(SSM_E_SHAPE, "workspace holds %lld bytes, needs %lld", (long long)have, (long long)need);
  if (!aligned16(ws)) return fail(SSM_E_ALIGN, "workspace is not 16-byte aligned");
  return SSM_OK;
}

void place(DeltaArgs& a, const DeltaLayout& l, void* workspace) {
  char* w = static_cast<char*>(workspace);
  a.head = reinterpret_cast<DeltaHead*>(w);
  a.chunks = reinterpret_cast<DeltaChunk*>(w + l.chunks);
  a.seqs = reinterpret_cast<DeltaSeq*>(w + l.seqs);
  auto f = [&](int64_t o) { return reinterpret_cast<float*>(w + o); };
  a.qh = f(l.qh); a.kh = f(l.kh); a.T = f(l.T); a.M = f(l.M); a.b = f(l.b);
  a.cum = reinterpret_cast<double*>(w + l.cum);
  a.S = f(l.S); a.dS = f(l.dS); a.U = f(l.U); a.dR = f(l.dR); a.dqh = f(l.dqh); a.dkh = f(l.dkh);
  a.part = f(l.part);
  a.gops = w + l.gops; a.hops = w + l.hops;
}

template <typename IO>
void launch_delta_prep(const DeltaArgs& a, const DeltaLayout& l, hipStream_t s) {
  delta_plan_kernel<<<1, 1024, 0, s>>>(a);
  delta_rows_kernel<IO><<<dim3((unsigned)l.nchunk, a.G), 256, 0, s>>>(a);
  delta_prep_kernel<IO><<<dim3((unsigned)l.nchunk, a.H), 256, 0, s>>>(a);
}

// 128 channels a workgroup where that gives every CU one, else 64.
constexpr int64_t kCUs = 256;

template <typename IO, int NT>
void launch_delta(const DeltaArgs& a, const DeltaLayout& l, bool vec, bool fast, hipStream_t s) {
  static_assert(Ops<IO, NT>::group == 2 * kQ * NT * 32 * Ops<IO, NT>::KP && Ops<IO, NT>::head == 4 * kTri * 1024 + 2048, "as in delta_layout");
  delta_plan_kernel<<<1, 1024, 0, s>>>(a);
  const dim3 grid((unsigned)l.nchunk, a.H);
  if (vec) delta_ops_kernel<IO, NT, true><<<grid, 256, 0, s>>>(a);
  else delta_ops_kernel<IO, NT, false><<<grid, 256, 0, s>>>(a);
  auto walk = [&](auto pt, auto fa) {
    constexpr int PT = decltype(pt)::value;
    const int units = (a.P + 64 * PT - 1) / (64 * PT);
    const int64_t items = (a.nseq * a.H + 7) / 8 * 8;
    delta_walk_kernel<IO, NT, PT, 4, decltype(fa)::value><<<(unsigned)(items * units), 256, 0, s>>>(a, units);
  };
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  bool wide = false;
  if constexpr (NT < 16) wide = a.nseq * a.H * ((a.P + 127) / 128) >= kCUs;
  if constexpr (NT < 16) {
    if (wide) {
      if (fast) walk(Two{}, std::true_type{});
      else walk(Two{}, std::false_type{});
      return;
    }
  }
  if (fast) walk(One{}, std::true_type{});
  else walk(One{}, std::false_type{});
}

template <typename IO>
void launch_delta_io(const DeltaArgs& a, const DeltaLayout& l, hipStream_t s) {
  constexpr int es = sizeof(IO);
  auto on = [&](const void* p, int64_t stride, int64_t width, int bytes) {
    return ((uintptr_t)p | (uintptr_t)(stride * es) | (uintptr_t)(width * es)) % bytes == 0;
  };
  const bool vec = on(a.q, a.qs, a.N, 16) && on(a.k, a.ks, a.N, 16);
  const bool fast = a.N % 4 == 0 && aligned16(a.state) && on(a.v, a.vs, a.P, 2 * es) && on(a.y, a.ys, a.P, 2 * es) &&
                    a.vs < (1 << 24) && a.ys < (1 << 24);  // a lane's offset to its rows in 32 bits
  switch (l.nt) {
    case 2: launch_delta<IO, 2>(a, l, vec, fast, s); break;
    case 4: launch_delta<IO, 4>(a, l, vec, fast, s); break;
    case 8: launch_delta<IO, 8>(a, l, vec, fast, s); break;
    default: launch_delta<IO, 16>(a, l, vec, fast, s); break;
  }
}

template <typename IO>
void launch_delta_bwd(const DeltaArgs& a, const DeltaLayout& l, hipStream_t s) {
  launch_delta_prep<IO>(a, l, s);
  const dim3 walk((unsigned)a.nseq, a.H, (a.P + 31) / 32);
  delta_scan_kernel<IO, true><<<walk, 256, 0, s>>>(a);
  delta_scan_bwd_kernel<IO><<<walk, 256, 0, s>>>(a);
  delta_grad_kernel<IO><<<dim3((unsigned)l.nchunk, a.H), 256, 0, s>>>(a);
  delta_qk_grad_kernel<IO><<<dim3((unsigned)l.nchunk, a.G), 256, 0, s>>>(a);
  delta_zero_kernel<IO><<<1024, 256, 0, s>>>(a);
  if (a.dA || a.ddt_bias) delta_sum_kernel<<<a.H, 256, 0, s>>>(a);
}

template <typename IO, int LN, bool VEC>
int launch_step(const DeltaArgs& a, hipStream_t s) {
  const int rows = 256 / LN, splits = (a.P + rows - 1) / rows;
  const int64_t grid = a.nseq * a.H * splits;
  if (!grid_ok(grid, 256)) return fail(SSM_E_SHAPE, "too many entries and heads for one call");
  delta_step_kernel<IO, LN, VEC><<<(unsigned)grid, 256, 0, s>>>(a, splits);
  return launch_status("ssm_gated_delta_update launch");
}

template <typename IO>
int launch_step_io(const DeltaArgs& a, hipStream_t s) {
  if (a.N % 4 || !aligned16(a.state)) return launch_step<IO, 64, false>(a, s);
  if (a.N <= 32) return launch_step<IO, 8, true>(a, s);
  if (a.N <= 64) return launch_step<IO, 16, true>(a, s);
  if (a.N <= 128) return launch_step<IO, 32, true>(a, s);
  return launch_step<IO, 64, true>(a, s);
}

int64_t delta_size(int64_t tokens, int64_t nseq, int64_t nheads, int64_t headdim, int64_t ngroups, int64_t dstate,
                   int io_dtype, bool bwd) {
  if (check_delta_extents(tokens, nseq, nheads, headdim, ngroups, dstate) || check_io(io_dtype)) return -1;
  return delta_layout(tokens, nseq, nheads, headdim, ngroups, dstate, io_dtype, bwd).bytes;
}

}  // namespace

// ---------------------------------------------------------------- C ABI

extern "C" {

int64_t ssm_gated_delta_workspace_size(int64_t tokens, int64_t nseq, int64_t nheads, int64_t headdim,
                                       int64_t ngroups, int64_t dstate, int io_dtype) {
  g_last_error[0] = 0;
  return delta_size(tokens, nseq, nheads, headdim, ngroups, dstate, io_dtype, false);
}

int64_t ssm_gated_delta_bwd_workspace_size(int64_t tokens, int64_t nseq, int64_t nheads, int64_t headdim,
                                           int64_t ngroups, int64_t dstate, int io_dtype) {
  g_last_error[0] = 0;
  return delta_size(tokens, nseq, nheads, headdim, ngroups, dstate, io_dtype, true);
}

int ssm_gated_delta_fwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                        int64_t v_stride, const void* dt, int64_t dt_stride, const void* beta,
                        int64_t beta_stride, const float* A, const float* dt_bias, int dt_softplus,
                        int beta_sigmoid, int qk_norm, float eps, float scale, const int32_t* cu_seqlens,
                        const int32_t* slots, const uint8_t* has_state, float* ssm_state, void* y,
                        int64_t y_stride, void* workspace, int64_t workspace_bytes, int64_t tokens,
                        int64_t nseq, int64_t nslots, int64_t nheads, int64_t headdim, int64_t ngroups,
                        int64_t dstate, int io_dtype, void* hip_stream) {
  g_last_error[0] = 0;
  DeltaArgs a;
  memset(&a, 0, sizeof a);
  a.q = q; a.k = k; a.v = v; a.dt = dt; a.beta = beta; a.A = A; a.dt_bias = dt_bias; a.cu = cu_seqlens;
  a.slots = slots; a.has = has_state; a.state = ssm_state; a.y = y;
  a.qs = q_stride; a.ks = k_stride; a.vs = v_stride; a.ds = dt_stride; a.bs = beta_stride; a.ys = y_stride;
  a.softplus = dt_softplus ? 1 : 0; a.sigmoid = beta_sigmoid ? 1 : 0; a.norm = qk_norm ? 1 : 0;
  a.eps = eps; a.scale = scale;
  const DeltaCall c = {tokens, nseq, ssm_state ? nslots : 0, nheads, headdim, ngroups, dstate, io_dtype};
  if (!cu_seqlens) return fail(SSM_E_NULL, "cu_seqlens is NULL");
  if (!y) return fail(SSM_E_NULL, "y is NULL");
  if (!workspace) return fail(SSM_E_NULL, "workspace is NULL");
  const int es = io_dtype == SSM_DTYPE_BF16 ? 2 : 4;
  int st = check_delta_extents(tokens, nseq, nheads, headdim, ngroups, dstate);
  if (st || (st = check_state(a, c))) return st;
  if ((st = check_rows("y", y, y_stride, nheads * headdim, tokens, es))) return st;
  const Rows outs[] = {{y, tokens, y_stride * es, nheads * headdim * es, "y"},
                       flat(ssm_state, c.nslots * nheads * headdim * dstate * 4, "ssm_state"),
                       flat(workspace, workspace_bytes, "workspace")};
  if ((st = check_delta(a, c, outs, 3, nullptr, 0))) return st;
  const DeltaLayout l = delta_layout(tokens, nseq, nheads, headdim, ngroups, dstate, io_dtype, false);
  if ((st = check_workspace(workspace, workspace_bytes, l.bytes))) return st;
  place(a, l, workspace);
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (io_dtype == SSM_DTYPE_BF16) launch_delta_io<uint16_t>(a, l, s);
  else launch_delta_io<float>(a, l, s);
  return launch_status("ssm_gated_delta_fwd launch");
}

int ssm_gated_delta_update(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, const void* dt, int64_t dt_stride, const void* beta,
                           int64_t beta_stride, const float* A, const float* dt_bias, int dt_softplus,
                           int beta_sigmoid, int qk_norm, float eps, float scale, const int32_t* slots,
                           float* ssm_state, void* y, int64_t y_stride, int64_t batch, int64_t nslots,
                           int64_t nheads, int64_t headdim, int64_t ngroups, int64_t dstate, int io_dtype,
                           void* hip_stream) {
  g_last_error[0] = 0;
  DeltaArgs a;
  memset(&a, 0, sizeof a);
  a.q = q; a.k = k; a.v = v; a.dt = dt; a.beta = beta; a.A = A; a.dt_bias = dt_bias;
  a.slots = slots; a.state = ssm_state; a.y = y;
  a.qs = q_stride; a.ks = k_stride; a.vs = v_stride; a.ds = dt_stride; a.bs = beta_stride; a.ys = y_stride;
  a.softplus = dt_softplus ? 1 : 0; a.sigmoid = beta_sigmoid ? 1 : 0; a.norm = qk_norm ? 1 : 0;
  a.eps = eps; a.scale = scale;
  if (!ssm_state) return fail(SSM_E_NULL, "ssm_state is NULL");
  if (!y) return fail(SSM_E_NULL, "y is NULL");
  const DeltaCall c = {batch, batch, nslots, nheads, headdim, ngroups, dstate, io_dtype};
  const int es = io_dtype == SSM_DTYPE_BF16 ? 2 : 4;
  int st = check_delta_extents(batch, batch, nheads, headdim, ngroups, dstate);
  if (st || (st = check_state(a, c))) return st;
  if ((st = check_rows("y", y, y_stride, nheads * headdim, batch, es))) return st;
  const Rows outs[] = {{y, batch, y_stride * es, nheads * headdim * es, "y"},
                       flat(ssm_state, nslots * nheads * headdim * dstate * 4, "ssm_state")};
  if ((st = check_delta(a, c, outs, 2, nullptr, 0))) return st;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  return io_dtype == SSM_DTYPE_BF16 ? launch_step_io<uint16_t>(a, s) : launch_step_io<float>(a, s);
}

int ssm_gated_delta_bwd(const void* dy, int64_t dy_stride, const void* q, int64_t q_stride, const void* k,
                        int64_t k_stride, const void* v, int64_t v_stride, const void* dt, int64_t dt_stride,
                        const void* beta, int64_t beta_stride, const float* A, const float* dt_bias,
                        int dt_softplus, int beta_sigmoid, int qk_norm, float eps, float scale,
                        const int32_t* cu_seqlens, const float* h0, const float* dfinal_state, void* dq,
                        int64_t dq_stride, void* dk, int64_t dk_stride, void* dv, int64_t dv_stride, void* ddt,
                        int64_t ddt_stride, void* dbeta, int64_t dbeta_stride, float* dA, float* ddt_bias,
                        float* dh0, void* workspace, int64_t workspace_bytes, int64_t tokens, int64_t nseq,
                        int64_t nheads, int64_t headdim, int64_t ngroups, int64_t dstate, int io_dtype,
                        void* hip_stream) {
  g_last_error[0] = 0;
  DeltaArgs a;
  memset(&a, 0, sizeof a);
  a.dy = dy; a.q = q; a.k = k; a.v = v; a.dt = dt; a.beta = beta; a.A = A; a.dt_bias = dt_bias;
  a.cu = cu_seqlens; a.h0 = h0; a.dfinal = dfinal_state;
  a.dq = dq; a.dk = dk; a.dv = dv; a.ddt = ddt; a.dbeta = dbeta; a.dA = dA; a.ddt_bias = ddt_bias; a.dh0 = dh0;
  a.gs = dy_stride; a.qs = q_stride; a.ks = k_stride; a.vs = v_stride; a.ds = dt_stride; a.bs = beta_stride;
  a.dqs = dq_stride; a.dks = dk_stride; a.dvs = dv_stride; a.dds = ddt_stride; a.dbs = dbeta_stride;
  a.softplus = dt_softplus ? 1 : 0; a.sigmoid = beta_sigmoid ? 1 : 0; a.norm = qk_norm ? 1 : 0;
  a.eps = eps; a.scale = scale;
  const struct { const void* p; const char* name; } req[] = {
      {dy, "dy"}, {cu_seqlens, "cu_seqlens"}, {dq, "dq"}, {dk, "dk"}, {dv, "dv"}, {ddt, "ddt"}, {dbeta, "dbeta"},
      {workspace, "workspace"}};
  for (const auto& r : req)
    if (!r.p) return fail(SSM_E_NULL, "%s is NULL", r.name);
  const DeltaCall c = {tokens, nseq, 0, nheads, headdim, ngroups, dstate, io_dtype};
  int st = check_delta_extents(tokens, nseq, nheads, headdim, ngroups, dstate);
  if (st || (st = check_io(io_dtype))) return st;
  const int es = io_dtype == SSM_DTYPE_BF16 ? 2 : 4;
  const int64_t gn = ngroups * dstate, hp = nheads * headdim, sb = nseq * hp * dstate * 4;
  if ((st = check_rows("dy", dy, dy_stride, hp, tokens, es)) || (st = check_rows("dq", dq, dq_stride, gn, tokens, es)) ||
      (st = check_rows("dk", dk, dk_stride, gn, tokens, es)) || (st = check_rows("dv", dv, dv_stride, hp, tokens, es)) ||
      (st = check_rows("ddt", ddt, ddt_stride, nheads, tokens, es)) ||
      (st = check_rows("dbeta", dbeta, dbeta_stride, nheads, tokens, es)))
    return st;
  for (const void* p : {(const void*)h0, (const void*)dfinal_state, (const void*)dh0, (const void*)dA, (const void*)ddt_bias})
    if ((uintptr_t)p & 3) return fail(SSM_E_ALIGN, "a float32 tensor is not aligned to its elements");
  const Rows outs[] = {{dq, tokens, dq_stride * es, gn * es, "dq"}, {dk, tokens, dk_stride * es, gn * es, "dk"},
                       {dv, tokens, dv_stride * es, hp * es, "dv"}, {ddt, tokens, ddt_stride * es, nheads * es, "ddt"},
                       {dbeta, tokens, dbeta_stride * es, nheads * es, "dbeta"}, flat(dA, nheads * 4, "dA"),
                       flat(ddt_bias, nheads * 4, "ddt_bias"), flat(dh0, sb, "dh0"),
                       flat(workspace, workspace_bytes, "workspace")};
  const Rows more[] = {{dy, tokens, dy_stride * es, hp * es, "dy"}, flat(h0, sb, "h0"),
                       flat(dfinal_state, sb, "dfinal_state")};
  if ((st = check_delta(a, c, outs, 9, more, 3))) return st;
  const DeltaLayout l = delta_layout(tokens, nseq, nheads, headdim, ngroups, dstate, io_dtype, true);
  if ((st = check_workspace(workspace, workspace_bytes, l.bytes))) return st;
  place(a, l, workspace);
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (io_dtype == SSM_DTYPE_BF16) launch_delta_bwd<uint16_t>(a, l, s);
  else launch_delta_bwd<float>(a, l, s);
  return launch_status("ssm_gated_delta_bwd launch");
}

}  // extern "C"
