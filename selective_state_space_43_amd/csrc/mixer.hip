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
  const int32_t* cu;     // NULL: sequence s is row s alone (the one-token step)
  const int32_t* slots;  // NULL: sequence s has slot s
  const uint8_t* has;    // NULL: cu given: none has a state; else all have
  float* conv_state;     // [nslots, channels, W - 1]
  float* state;          // [nslots, H, P, N] or NULL
  void* y;
  int64_t xs, ds, zs, ys;  // row strides in elements
  int64_t tokens, nseq, nslots;
  int H, P, G, N, W, C;    // C: convolution channels, H P + 2 G N
  int softplus;
};

// Sequence s: its rows [t0, t1), its slot and whether it starts from that
// slot's state.  Whatever the index tensors hold, the rows lie inside the
// tensors; false for a sequence whose slot is outside the cache (padding).
struct Seq {
  int64_t t0, t1, slot;
  bool resume;
};
__device__ __forceinline__ bool load_seq(const MixArgs& a, int64_t s, Seq& q) {
  if (a.cu) {
    const int64_t b = a.cu[s], e = a.cu[s + 1];
    q.t0 = b < 0 ? 0 : (b > a.tokens ? a.tokens : b);
    q.t1 = e < q.t0 ? q.t0 : (e > a.tokens ? a.tokens : e);
  } else {
    q.t0 = s;
    q.t1 = s + 1;
  }
  q.slot = a.slots ? (int64_t)a.slots[s] : s;
  if (a.state && (q.slot < 0 || q.slot >= a.nslots)) return false;
  q.resume = a.state && (a.cu ? (a.has && a.has[s]) : true);
  return true;
}

// One output of the convolution and its silu: channel c at row t of a
// sequence that starts at row t0.
template <typename IO>
__device__ __forceinline__ float conv_at(const MixArgs& a, const Seq& q, int64_t t, int c) {
  const int W = a.W;
  float acc = a.cb ? a.cb[c] : 0.0f;
  for (int k = 0; k < W; ++k) {
    const int64_t r = t - (W - 1) + k;
    float v = 0.0f;
    if (r >= q.t0)
      v = ld<IO>(a.xbc, r * a.xs + c);
    else if (q.resume)
      v = a.conv_state[(q.slot * a.C + c) * (W - 1) + (r - q.t0 + W - 1)];
    acc = fmaf(a.cw[(int64_t)c * W + k], v, acc);
  }
  return silu(acc);
}

// The recurrence in time order: a workgroup owns 16 channels of one head of
// one sequence, 16 lanes a channel, each with every sixteenth state.
constexpr int kMaxN = 256;

template <typename IO>
__global__ void __launch_bounds__(256) mix_scan_kernel(const MixArgs a) {
  __shared__ float sB[kMaxN], sC[kMaxN], sx[16];
  const int64_t s = blockIdx.x;
  const int h = blockIdx.y, p0 = blockIdx.z * 16;
  const int tid = threadIdx.x, pl = tid >> 4, nl = tid & 15, p = p0 + pl;
  const int N = a.N, g = h / (a.H / a.G), inner = a.H * a.P;
  Seq q;
  if (!load_seq(a, s, q)) return;
  float hst[kMaxN / 16];
  float* own = a.state ? a.state + ((q.slot * a.H + h) * a.P + p) * N : nullptr;
#pragma unroll
  for (int i = 0; i < kMaxN / 16; ++i) {
    const int n = nl + 16 * i;
    hst[i] = (q.resume && p < a.P && n < N) ? own[n] : 0.0f;
  }
  const float A = a.A[h], D = a.Dskip ? a.Dskip[h] : 0.0f, db = a.dt_bias ? a.dt_bias[h] : 0.0f;
  for (int64_t t = q.t0; t < q.t1; ++t) {
    __syncthreads();
    for (int i = tid; i < 2 * N; i += 256) {
      const int n = i < N ? i : i - N;
      const float v = conv_at<IO>(a, q, t, inner + (i < N ? 0 : a.G * N) + g * N + n);
      (i < N ? sB : sC)[n] = v;
    }
    if (tid < 16) sx[tid] = p0 + tid < a.P ? conv_at<IO>(a, q, t, h * a.P + p0 + tid) : 0.0f;
    __syncthreads();
    const float raw = ld<IO>(a.dt, t * a.ds + h) + db;
    const float dt = a.softplus ? softplus(raw) : raw;
    const float e = ex2(dt * A * kLog2e), x = sx[pl], w = dt * x;
    float acc = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxN / 16; ++i) {
      const int n = nl + 16 * i;
      if (n < N) {
        hst[i] = fmaf(e, hst[i], w * sB[n]);
        acc = fmaf(sC[n], hst[i], acc);
      }
    }
    for (int m = 8; m; m >>= 1) acc += __shfl_xor(acc, m, 16);
    if (nl == 0 && p < a.P) {
      float v = fmaf(D, x, acc);
      const int64_t j = (int64_t)h * a.P + p;
      if (a.z) v *= silu(ld<IO>(a.z, t * a.zs + j));
      st<IO>(a.y, t * a.ys + j, v);
    }
  }
  if (own && p < a.P) {
#pragma unroll
    for (int i = 0; i < kMaxN / 16; ++i) {
      const int n = nl + 16 * i;
      if (n < N) own[n] = hst[i];
    }
  }
}

// The last W - 1 inputs of every sequence into its slot, after every reader
// of the old ones.
template <typename IO>
__global__ void __launch_bounds__(256) mix_conv_state_kernel(const MixArgs a) {
  const int64_t s = blockIdx.x;
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c >= a.C) return;
  Seq q;
  if (!load_seq(a, s, q)) return;
  const int W = a.W;
  float* own = a.conv_state + (q.slot * a.C + c) * (W - 1);
  float v[3];
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    if (j >= W - 1) break;
    const int64_t r = q.t1 - (W - 1) + j;  // row of the input to keep
    if (r >= q.t0)
      v[j] = ld<IO>(a.xbc, r * a.xs + c);
    else
      v[j] = q.resume ? own[r - q.t0 + W - 1] : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j < W - 1) own[j] = v[j];
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
  float* pw;  // per-block sums of dweight, dbias [blocks, C]
  float* pb;
  int64_t xs, zs, gs, ys, dzs;  // row strides; gs of dy
  int64_t rows;
  int C, G;
  float eps;
  int center, act, gate;
};

__device__ __forceinline__ float block_sum(float v, float* red) {
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

template <typename IO>
__global__ void __launch_bounds__(256) norm_fwd_kernel(const NormArgs a) {
  __shared__ float red[4];
  const int gs = a.C / a.G, c0 = blockIdx.y * gs;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    auto val = [&](int c) {
      float v = ld<IO>(a.x, r * a.xs + c);
      if (a.gate == SSM_GATE_BEFORE) v *= silu(ld<IO>(a.z, r * a.zs + c));
      return v;
    };
    float mean = 0.0f;
    if (a.center) {
      float sum = 0.0f;
      for (int c = threadIdx.x; c < gs; c += 256) sum += val(c0 + c);
      mean = block_sum(sum, red) / gs;
    }
    float sq = 0.0f;
    for (int c = threadIdx.x; c < gs; c += 256) {
      const float v = val(c0 + c) - mean;
      sq = fmaf(v, v, sq);
    }
    const float rs = rsqrtf(block_sum(sq, red) / gs + a.eps);
    for (int c = c0 + threadIdx.x; c < c0 + gs; c += 256) {
      float v = (val(c) - mean) * rs;
      if (a.w) v *= a.w[c];
      if (a.b) v += a.b[c];
      if (a.act == SSM_ACT_SILU) v = silu(v);
      if (a.gate == SSM_GATE_AFTER) v *= silu(ld<IO>(a.z, r * a.zs + c));
      st<IO>(a.y, r * a.ys + c, v);
    }
  }
}

template <typename IO>
__global__ void __launch_bounds__(256) norm_bwd_kernel(const NormArgs a) {
  __shared__ float red[4];
  const int gs = a.C / a.G, c0 = blockIdx.y * gs;
  float* pw = a.pw + (int64_t)blockIdx.x * a.C;
  float* pb = a.pb + (int64_t)blockIdx.x * a.C;
  for (int c = c0 + threadIdx.x; c < c0 + gs; c += 256) pw[c] = pb[c] = 0.0f;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    auto val = [&](int c) {
      float v = ld<IO>(a.x, r * a.xs + c);
      if (a.gate == SSM_GATE_BEFORE) v *= silu(ld<IO>(a.z, r * a.zs + c));
      return v;
    };
    float mean = 0.0f;
    if (a.center) {
      float sum = 0.0f;
      for (int c = threadIdx.x; c < gs; c += 256) sum += val(c0 + c);
      mean = block_sum(sum, red) / gs;
    }
    float sq = 0.0f;
    for (int c = threadIdx.x; c < gs; c += 256) {
      const float v = val(c0 + c) - mean;
      sq = fmaf(v, v, sq);
    }
    const float rs = rsqrtf(block_sum(sq, red) / gs + a.eps);
    // gradient of the affine result, and what the gate behind it takes
    auto grad = [&](int c, float n, float* dz) {
      float g = ld<IO>(a.dy, r * a.gs + c);
      float v = n * (a.w ? a.w[c] : 1.0f) + (a.b ? a.b[c] : 0.0f);
      if (a.gate == SSM_GATE_AFTER) {
        const float z = ld<IO>(a.z, r * a.zs + c), sg = sigmoid(z);
        const float o = a.act == SSM_ACT_SILU ? silu(v) : v;
        if (dz) *dz = g * o * sg * fmaf(z, 1.0f - sg, 1.0f);
        g *= z * sg;
      }
      if (a.act == SSM_ACT_SILU) {
        const float sv = sigmoid(v);
        g *= sv * fmaf(v, 1.0f - sv, 1.0f);
      }
      return g;
    };
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = c0 + threadIdx.x; c < c0 + gs; c += 256) {
      const float n = (val(c) - mean) * rs, g = grad(c, n, nullptr);
      const float u = g * (a.w ? a.w[c] : 1.0f);
      s1 += u;
      s2 = fmaf(u, n, s2);
      pw[c] = fmaf(g, n, pw[c]);
      pb[c] += g;
    }
    s1 = block_sum(s1, red) / gs;
    s2 = block_sum(s2, red) / gs;
    if (!a.center) s1 = 0.0f;
    for (int c = c0 + threadIdx.x; c < c0 + gs; c += 256) {
      const float n = (val(c) - mean) * rs;
      float dz = 0.0f;
      const float u = grad(c, n, &dz) * (a.w ? a.w[c] : 1.0f);
      float d = rs * (u - n * s2 - s1);
      if (a.gate == SSM_GATE_BEFORE) {
        const float z = ld<IO>(a.z, r * a.zs + c), sg = sigmoid(z);
        dz = d * ld<IO>(a.x, r * a.xs + c) * sg * fmaf(z, 1.0f - sg, 1.0f);
        d *= z * sg;
      }
      st<IO>(a.y, r * a.ys + c, d);
      if (a.dz) st<IO>(a.dz, r * a.dzs + c, dz);
    }
  }
}

// column sums of the blocks' partial sums, in block order
__global__ void __launch_bounds__(256) norm_bwd_sum_kernel(const float* pw, const float* pb,
                                                           int blocks, int C, float* dw, float* db) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= C) return;
  float sw = 0.0f, sb = 0.0f;
  for (int i = 0; i < blocks; ++i) {
    sw += pw[(int64_t)i * C + c];
    sb += pb[(int64_t)i * C + c];
  }
  if (dw) dw[c] = sw;
  if (db) db[c] = sb;
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
  if (tokens > 0x7fffffff || nseq > 0xfffff)
    return fail(SSM_E_SHAPE, "tokens = %lld, nseq = %lld: at most 2^31 - 1 and 2^20 - 1",
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

template <typename IO>
void launch_mix_simple(const MixArgs& a, hipStream_t s) {
  mix_scan_kernel<IO><<<dim3((unsigned)a.nseq, a.H, (a.P + 15) / 16), 256, 0, s>>>(a);
  if (a.state && a.W > 1)
    mix_conv_state_kernel<IO><<<dim3((unsigned)a.nseq, (a.C + 255) / 256), 256, 0, s>>>(a);
}

constexpr int64_t kNormBlocks = 256;
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

}  // namespace

// ---------------------------------------------------------------- C ABI

extern "C" {

int64_t ssm_conv_ssd_workspace_size(int64_t tokens, int64_t nseq, int64_t nheads, int64_t headdim,
                                    int64_t ngroups, int64_t dstate, int io_dtype) {
  g_last_error[0] = 0;
  if (check_mix_extents(tokens, nseq, nheads, headdim, ngroups, dstate) || check_io(io_dtype)) return -1;
  return 256;
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
  MixArgs a;
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
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (io_dtype == SSM_DTYPE_BF16) launch_mix_simple<uint16_t>(a, s);
  else launch_mix_simple<float>(a, s);
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
  if (io_dtype == SSM_DTYPE_BF16) launch_mix_simple<uint16_t>(a, s);
  else launch_mix_simple<float>(a, s);
  return launch_status("ssm_conv_ssd_update launch");
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
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  const dim3 grid((unsigned)(rows < 65536 ? rows : 65536), a.G);
  if (io_dtype == SSM_DTYPE_BF16) norm_fwd_kernel<uint16_t><<<grid, 256, 0, s>>>(a);
  else norm_fwd_kernel<float><<<grid, 256, 0, s>>>(a);
  return launch_status("ssm_group_norm_fwd launch");
}

int64_t ssm_group_norm_bwd_workspace_size(int64_t rows, int64_t channels, int64_t ngroups) {
  g_last_error[0] = 0;
  if (check_extent("rows", rows) || check_extent("channels", channels) ||
      check_extent("ngroups", ngroups) || channels > 0x7fffffff)
    return -1;
  return 2 * kNormBlocks * channels * 4;
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
  a.pw = static_cast<float*>(workspace);
  a.pb = a.pw + kNormBlocks * channels;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  const int blocks = (int)(rows < kNormBlocks ? rows : kNormBlocks);
  if (io_dtype == SSM_DTYPE_BF16) norm_bwd_kernel<uint16_t><<<dim3(blocks, a.G), 256, 0, s>>>(a);
  else norm_bwd_kernel<float><<<dim3(blocks, a.G), 256, 0, s>>>(a);
  if (dweight || dbias)
    norm_bwd_sum_kernel<<<(a.C + 255) / 256, 256, 0, s>>>(a.pw, a.pb, blocks, a.C, dweight, dbias);
  return launch_status("ssm_group_norm_bwd launch");
}

}  // extern "C"
