// kl_layernorm.cu -- LayerNorm forward and backward over rows of any width,
// with an ordinary weight and bias, an adaLN scale and shift, or neither.
//
//   xhat = (x - mean) * rstd,  y = xhat * g + b,
//   g = gain (or 1 + gain with KL_LN_MODULATE; 1 without a gain)
//   h = dy * g
//   dx = rstd * (h - mean_c(h) - xhat * mean_c(h * xhat))
//   dgain[c] = sum_r dy * xhat,  dbias[c] = sum_r dy   (rows of the group)
//
// mean, rstd and every sum are fp32; the variance is taken about the mean in
// a second pass over the row in registers, so a large common offset costs
// nothing.  A row is held in registers by the threads of one thread row
// (blockDim.x; NV vectors of V elements each), so x (and dy) are read once:
// both directions are bound by HBM.  CTAs with narrow rows hold several rows
// (blockDim.y).
//
// Backward: a thread meets the same columns in every row of its CTA, so the
// sums for dgain and dbias stay in its registers; CTAs walk the rows of one
// group with a fixed stride and leave one partial row each, which a second
// kernel adds in index order -- no atomics, the same bits every run.
#include "../../include/klein.h"
#include "kl_common.cuh"
#include "kl_internal.h"

namespace kl {

struct LnParams {
  const void* x;
  int64_t rows, cols, ldx;
  const void* dy;
  int64_t ldy;  // of dy (backward) or y (forward)
  void* out;    // y (forward) or dx (backward)
  int64_t ldo;
  const void* gain;
  const void* bias;
  int ptype;    // KL_BF16 / KL_F32 / KL_F16 of gain and bias
  float plus;   // added to the gain: 1 with KL_LN_MODULATE
  int64_t group_rows;  // rows of one group; groups have consecutive rows
  float* mean;
  float* rstd;
  float eps;
  float* part;  // backward: [groups][splits][2][cols] partial sums (null: none wanted)
  int splits;   // CTAs of a group
};

// V parameter values from column c of a row of gains or biases
template <int V>
__device__ __forceinline__ void load_param(const void* base, int type, int64_t at, bool vec, float (&v)[V]) {
  if (type == KL_F32) {
    const float* p = reinterpret_cast<const float*>(base) + at;
    if (V % 4 == 0 && vec) {
#pragma unroll
      for (int i = 0; i + 3 < V; i += 4) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(p + i));
        v[i] = q.x;
        v[i + 1] = q.y;
        v[i + 2] = q.z;
        v[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __ldg(p + i);
    }
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + at;
    uint32_t w[(V + 1) / 2];
    if (V == 8 && vec) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = q.x;
      if constexpr (V == 8) {
        w[1] = q.y;
        w[2] = q.z;
        w[3] = q.w;
      }
    } else if (V == 4 && vec) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = q.x;
      if constexpr (V == 4) w[1] = q.y;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t u = __ldg(p + i);
        w[i / 2] = (i & 1) ? w[i / 2] | (u << 16) : u;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float lo, hi;
      if (type == KL_BF16)
        unpack2<__nv_bfloat16>(w[i / 2], lo, hi);
      else
        unpack2<__half>(w[i / 2], lo, hi);
      v[i] = (i & 1) ? hi : lo;
    }
  }
}

// parameter rows that suit vector loads from every multiple of V columns
template <int V>
__device__ __forceinline__ bool param_vec_ok(const void* base, int type, int64_t cols) {
  const int bytes = V * (type == KL_F32 ? 4 : 2);
  const int a = bytes > 16 ? 16 : bytes;
  return base && (reinterpret_cast<uintptr_t>(base) % a) == 0 && cols % V == 0;
}

// Sum of K values over the threads of one thread row.  red: [blockDim.y][32][K]
// floats, one buffer a call in flight.  A thread row is whole warps.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* red) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return;
  const int w = threadIdx.x >> 5;
  float* mine = red + threadIdx.y * 32 * K;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) mine[w * K + k] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float s = mine[k];
    for (int i = 1; i < nw; ++i) s += mine[i * K + k];
    v[k] = s;
  }
}

template <typename T, int V, int NV>
__global__ void __launch_bounds__(1024) ln_forward_kernel(const LnParams p) {
  extern __shared__ float ln_red[];  // [2][blockDim.y][32]
  pdl_wait();
  pdl_trigger();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < p.rows;
  const T* x = reinterpret_cast<const T*>(p.x) + (live ? row : 0) * p.ldx;
  uint4 q[NV];
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = (int64_t)(threadIdx.x + i * blockDim.x) * V;
    q[i] = live && c < p.cols ? load_vec<T, V>(x + c) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float v[V];
    unpack_vec<T, V>(q[i], v);
#pragma unroll
    for (int k = 0; k < V; ++k) s[0] += v[k];
  }
  row_sum<1>(s, ln_red);
  const float mean = s[0] / (float)p.cols;
  s[0] = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((int64_t)(threadIdx.x + i * blockDim.x) * V < p.cols) {
      float v[V];
      unpack_vec<T, V>(q[i], v);
#pragma unroll
      for (int k = 0; k < V; ++k) s[0] = fmaf(v[k] - mean, v[k] - mean, s[0]);
    }
  }
  row_sum<1>(s, ln_red + blockDim.y * 32);
  const float rstd = 1.0f / sqrtf(s[0] / (float)p.cols + p.eps);
  if (!live) return;
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  const int64_t pbase = row / p.group_rows * p.cols;
  const bool gvec = param_vec_ok<V>(p.gain, p.ptype, p.cols), bvec = param_vec_ok<V>(p.bias, p.ptype, p.cols);
  T* y = reinterpret_cast<T*>(p.out) + row * p.ldo;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = (int64_t)(threadIdx.x + i * blockDim.x) * V;
    if (c < p.cols) {
      float v[V], w[V];
      unpack_vec<T, V>(q[i], v);
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = (v[k] - mean) * rstd;
      if (p.gain) {
        load_param<V>(p.gain, p.ptype, pbase + c, gvec, w);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] *= w[k] + p.plus;
      }
      if (p.bias) {
        load_param<V>(p.bias, p.ptype, pbase + c, bvec, w);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] += w[k];
      }
      store_vec<T, V>(y + c, v);
    }
  }
}

// Rows wider than the register kernels hold: one CTA a row, re-reading it.
template <typename T>
__global__ void __launch_bounds__(1024) ln_forward_wide_kernel(const LnParams p) {
  extern __shared__ float ln_red[];
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx;
  float s[1] = {0.f};
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) s[0] += to_f32(x[c]);
  row_sum<1>(s, ln_red);
  const float mean = s[0] / (float)p.cols;
  s[0] = 0.f;
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float d = to_f32(x[c]) - mean;
    s[0] = fmaf(d, d, s[0]);
  }
  row_sum<1>(s, ln_red + 32);
  const float rstd = 1.0f / sqrtf(s[0] / (float)p.cols + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  const int64_t pbase = row / p.group_rows * p.cols;
  T* y = reinterpret_cast<T*>(p.out) + row * p.ldo;
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
    float v[1] = {(to_f32(x[c]) - mean) * rstd}, w[1];
    if (p.gain) {
      load_param<1>(p.gain, p.ptype, pbase + c, false, w);
      v[0] *= w[0] + p.plus;
    }
    if (p.bias) {
      load_param<1>(p.bias, p.ptype, pbase + c, false, w);
      v[0] += w[0];
    }
    y[c] = from_f32<T>(v[0]);
  }
}

// CTA (group, split): rows split * blockDim.y + threadIdx.y, then every
// splits * blockDim.y.  The next row's x and dy are loaded before this row's
// sums are waited for.
template <typename T, int V, int NV, bool PG>
__global__ void __launch_bounds__(512, NV == 1 || V == 1 ? 2 : 1)
    ln_backward_kernel(const LnParams p) {
  extern __shared__ float ln_red[];  // [2][blockDim.y][32][2]; then [blockDim.y][2][cols padded] if PG and blockDim.y > 1
  pdl_wait();
  pdl_trigger();
  const int64_t group = blockIdx.x / p.splits, split = blockIdx.x - group * p.splits;
  const int64_t r0 = group * p.group_rows;
  const int64_t step = (int64_t)p.splits * blockDim.y;
  const bool gvec = param_vec_ok<V>(p.gain, p.ptype, p.cols);
  const float inv_c = 1.0f / (float)p.cols;
  float sg[PG ? NV : 1][V], sb[PG ? NV : 1][V];
  if constexpr (PG) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) sg[i][k] = sb[i][k] = 0.f;
  }
  uint4 qx[NV], qd[NV];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](int64_t lr) {
    const bool live = lr < p.group_rows;
    const int64_t row = r0 + (live ? lr : 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(threadIdx.x + i * blockDim.x) * V;
      const bool in = live && c < p.cols;
      qx[i] = in ? load_vec<T, V>(reinterpret_cast<const T*>(p.x) + row * p.ldx + c) : make_uint4(0u, 0u, 0u, 0u);
      qd[i] = in ? load_vec<T, V>(reinterpret_cast<const T*>(p.dy) + row * p.ldy + c) : make_uint4(0u, 0u, 0u, 0u);
    }
    mean = live ? p.mean[row] : 0.f;
    rstd = live ? p.rstd[row] : 0.f;
  };
  // every thread row of the CTA makes the same number of turns (barriers inside)
  const int64_t first = split * blockDim.y;
  fetch(first + threadIdx.y);
  int buf = 0;
  for (int64_t base = first; base < p.group_rows; base += step, buf ^= 1) {
    const int64_t lr = base + threadIdx.y;
    const bool live = lr < p.group_rows;
    float xh[NV][V], h[NV][V];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(threadIdx.x + i * blockDim.x) * V;
      unpack_vec<T, V>(qx[i], xh[i]);
      unpack_vec<T, V>(qd[i], h[i]);
      if (live && c < p.cols) {
        float w[V];
        if (p.gain) load_param<V>(p.gain, p.ptype, group * p.cols + c, gvec, w);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          xh[i][k] = (xh[i][k] - mean) * rstd;
          if constexpr (PG) {
            sg[i][k] = fmaf(h[i][k], xh[i][k], sg[i][k]);
            sb[i][k] += h[i][k];
          }
          if (p.gain) h[i][k] *= w[k] + p.plus;
          s[0] += h[i][k];
          s[1] = fmaf(h[i][k], xh[i][k], s[1]);
        }
      }
    }
    const float rs = rstd;
    if (base + step < p.group_rows) fetch(lr + step);
    row_sum<2>(s, ln_red + buf * blockDim.y * 64);
    const float m0 = s[0] * inv_c, m1 = s[1] * inv_c;
    if (live) {
      T* dx = reinterpret_cast<T*>(p.out) + (r0 + lr) * p.ldo;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t)(threadIdx.x + i * blockDim.x) * V;
        if (c < p.cols) {
#pragma unroll
          for (int k = 0; k < V; ++k) h[i][k] = rs * (h[i][k] - m0 - xh[i][k] * m1);
          store_vec<T, V>(dx + c, h[i]);
        }
      }
    }
  }
  if constexpr (PG) {
    // the CTA's sums: thread rows added in order through shared memory
    float* out = p.part + (int64_t)blockIdx.x * 2 * p.cols;
    const int ny = blockDim.y;
    if (ny > 1) {
      const int width = NV * V * blockDim.x;
      float* mine = ln_red + ny * 128 + threadIdx.y * 2 * width;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int c = (threadIdx.x + i * blockDim.x) * V + k;
          mine[c] = sg[i][k];
          mine[width + c] = sb[i][k];
        }
      __syncthreads();
      for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < 2 * width; c += ny * blockDim.x) {
        float s = 0.f;
        for (int y = 0; y < ny; ++y) s += ln_red[ny * 128 + y * 2 * width + c];
        const int which = c >= width, col = c - which * width;
        if (col < p.cols) out[(int64_t)which * p.cols + col] = s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t)(threadIdx.x + i * blockDim.x) * V;
        if (c < p.cols) {
#pragma unroll
          for (int k = 0; k < V; ++k) {
            out[c + k] = sg[i][k];
            out[p.cols + c + k] = sb[i][k];
          }
        }
      }
    }
  }
}

// Wide rows: one CTA a row for dx, re-reading it ...
template <typename T>
__global__ void __launch_bounds__(1024) ln_backward_wide_kernel(const LnParams p) {
  extern __shared__ float ln_red[];
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x, pbase = row / p.group_rows * p.cols;
  const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx;
  const T* dy = reinterpret_cast<const T*>(p.dy) + row * p.ldy;
  T* dx = reinterpret_cast<T*>(p.out) + row * p.ldo;
  const float mean = p.mean[row], rstd = p.rstd[row];
  auto grad = [&](int64_t c) {
    float h = to_f32(dy[c]), w[1];
    if (p.gain) {
      load_param<1>(p.gain, p.ptype, pbase + c, false, w);
      h *= w[0] + p.plus;
    }
    return h;
  };
  float s[2] = {0.f, 0.f};
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float h = grad(c);
    s[0] += h;
    s[1] = fmaf(h, (to_f32(x[c]) - mean) * rstd, s[1]);
  }
  row_sum<2>(s, ln_red);
  const float inv_c = 1.0f / (float)p.cols, m0 = s[0] * inv_c, m1 = s[1] * inv_c;
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x)
    dx[c] = from_f32<T>(rstd * (grad(c) - m0 - (to_f32(x[c]) - mean) * rstd * m1));
}
// ... and a thread a column of one split of a group's rows for the parameters
template <typename T>
__global__ void __launch_bounds__(256) ln_param_wide_kernel(const LnParams p) {
  pdl_wait();
  pdl_trigger();
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t group = blockIdx.y / p.splits, split = blockIdx.y - group * p.splits;
  if (c >= p.cols) return;
  float g = 0.f, b = 0.f;
  for (int64_t lr = split; lr < p.group_rows; lr += p.splits) {
    const int64_t row = group * p.group_rows + lr;
    const float d = to_f32(reinterpret_cast<const T*>(p.dy)[row * p.ldy + c]);
    const float xh = (to_f32(reinterpret_cast<const T*>(p.x)[row * p.ldx + c]) - p.mean[row]) * p.rstd[row];
    g = fmaf(d, xh, g);
    b += d;
  }
  float* out = p.part + (int64_t)blockIdx.y * 2 * p.cols;
  out[c] = g;
  out[p.cols + c] = b;
}

// dgain / dbias [groups][cols] from the partial rows, in index order: 32
// columns a CTA, 8 thread rows taking every eighth partial.
__global__ void __launch_bounds__(256) ln_param_sum_kernel(const float* __restrict__ part, int splits, int64_t cols,
                                                           float* __restrict__ dgain, float* __restrict__ dbias) {
  __shared__ float red[8][33];
  pdl_wait();
  pdl_trigger();
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;  // of the 2 * cols sums
  const int64_t group = blockIdx.y;
  float s = 0.f;
  if (c < 2 * cols) {
    const float* src = part + group * splits * 2 * cols + c;
#pragma unroll 4
    for (int i = threadIdx.y; i < splits; i += 8) s += src[(int64_t)i * 2 * cols];
  }
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < 2 * cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][threadIdx.x];
    if (c < cols)
      dgain[group * cols + c] = s;
    else
      dbias[group * cols + c - cols] = s;
  }
}

// ---------------------------------------------------------------- launchers
// How a row is spread over threads: vectors of V elements where every row
// starts on 16 bytes, else single elements; nv vectors a thread (0: too wide
// for registers).
struct LnShape {
  bool vec;
  int nv, tx, ty;
};
static LnShape ln_shape(int64_t cols, int es, bool vec, bool backward) {
  LnShape s{vec, 0, 0, 1};
  const int64_t n = vec ? cols / (16 / es) : cols;  // vectors of a row
  if (vec)
    s.nv = n <= 512 ? 1 : n <= 1024 ? 2 : (n <= 4096 && !backward) ? 4 : 0;
  else
    s.nv = n <= 2048 ? 4 : (n <= 4096 || (n <= 8192 && !backward)) ? 8 : 0;
  if (s.nv == 0) {
    s.tx = 1024;
    return s;
  }
  const int64_t t = (n + s.nv - 1) / s.nv;
  s.tx = (int)((t + 31) / 32 * 32);
  s.ty = s.tx >= 256 ? 1 : 256 / s.tx;
  return s;
}

// CTAs of a group in the backward pass: enough to fill the GPU, no more than
// the group has rows for
static int ln_splits(int64_t groups, int64_t group_rows, const LnShape& sh) {
  const int64_t per_sm = sh.tx * sh.ty <= 512 ? 1024 / (sh.tx * sh.ty) : 1;
  int64_t s = (int64_t)kNumSMs * per_sm / groups;
  const int64_t most = (group_rows + sh.ty - 1) / sh.ty;
  s = s < 1 ? 1 : s;
  return (int)(s < most ? s : most);
}

template <typename T, int V, int NV>
static cudaError_t launch_ln_forward_nv(const LnParams& p, const LnShape& sh, cudaStream_t s) {
  return launch_pdl(ln_forward_kernel<T, V, NV>, dim3((unsigned)((p.rows + sh.ty - 1) / sh.ty)), dim3(sh.tx, sh.ty),
                    (size_t)sh.ty * 64 * sizeof(float), s, p);
}
template <typename T>
static cudaError_t launch_ln_forward(const LnParams& p, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const LnShape sh = ln_shape(p.cols, sizeof(T), vec, false);
  if (sh.nv == 0) return launch_pdl(ln_forward_wide_kernel<T>, dim3((unsigned)p.rows), dim3(1024), 256, s, p);
  if (vec) {
    if (sh.nv == 1) return launch_ln_forward_nv<T, V, 1>(p, sh, s);
    if (sh.nv == 2) return launch_ln_forward_nv<T, V, 2>(p, sh, s);
    return launch_ln_forward_nv<T, V, 4>(p, sh, s);
  }
  return sh.nv == 4 ? launch_ln_forward_nv<T, 1, 4>(p, sh, s) : launch_ln_forward_nv<T, 1, 8>(p, sh, s);
}

template <typename T, int V, int NV>
static cudaError_t launch_ln_backward_nv(const LnParams& p, const LnShape& sh, cudaStream_t s) {
  size_t smem = (size_t)sh.ty * 128 * sizeof(float);
  if (p.part && sh.ty > 1) smem += (size_t)sh.ty * 2 * NV * V * sh.tx * sizeof(float);
  const dim3 grid((unsigned)(p.rows / p.group_rows * p.splits)), block(sh.tx, sh.ty);
  return p.part ? launch_pdl(ln_backward_kernel<T, V, NV, true>, grid, block, smem, s, p)
                : launch_pdl(ln_backward_kernel<T, V, NV, false>, grid, block, smem, s, p);
}
template <typename T>
static cudaError_t launch_ln_backward(LnParams& p, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const LnShape sh = ln_shape(p.cols, sizeof(T), vec, true);
  if (sh.nv == 0) {
    cudaError_t e = launch_pdl(ln_backward_wide_kernel<T>, dim3((unsigned)p.rows), dim3(1024), 256, s, p);
    if (e != cudaSuccess || !p.part) return e;
    return launch_pdl(ln_param_wide_kernel<T>,
                      dim3((unsigned)((p.cols + 255) / 256), (unsigned)(p.rows / p.group_rows * p.splits)), dim3(256),
                      0, s, p);
  }
  if (vec) return sh.nv == 1 ? launch_ln_backward_nv<T, V, 1>(p, sh, s) : launch_ln_backward_nv<T, V, 2>(p, sh, s);
  return sh.nv == 4 ? launch_ln_backward_nv<T, 1, 4>(p, sh, s) : launch_ln_backward_nv<T, 1, 8>(p, sh, s);
}

static bool ln_dtype_ok(int t) { return t == KL_BF16 || t == KL_F32 || t == KL_F16; }
static int ln_es(int t) { return t == KL_F32 ? 4 : 2; }
// every row of a matrix starts on 16 bytes
static bool ln_rows_16(const void* p, int64_t ld, int es) { return aligned(p, 16) && (ld * es) % 16 == 0; }

static kl_status ln_check(int dtype, int64_t rows, int64_t cols, int64_t groups, int ptype, int flags) {
  if (!ln_dtype_ok(dtype) || !ln_dtype_ok(ptype) || (flags & ~KL_LN_MODULATE)) return KL_ERR_INVALID_ARG;
  if (rows < 1 || cols < 1 || rows > KL_LN_MAX_ROWS || cols > KL_LN_MAX_COLS || groups < 1 || rows % groups ||
      groups > KL_LN_MAX_GROUPS)
    return KL_ERR_UNSUPPORTED_SHAPE;
  return KL_OK;
}

}  // namespace kl

extern "C" {

kl_status kl_layer_norm_forward(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, const void* gain,
                                const void* bias, int param_dtype, int64_t groups, float eps, int flags, void* y,
                                int64_t ldy, float* mean, float* rstd, void* stream) {
  using namespace kl;
  if (!x || !y || !(eps >= 0.f)) return KL_ERR_INVALID_ARG;
  kl_status st = ln_check(dtype, rows, cols, groups, param_dtype, flags);
  if (st != KL_OK) return st;
  if (ldx < cols || ldy < cols) return KL_ERR_INVALID_ARG;
  const int es = ln_es(dtype), ps = ln_es(param_dtype);
  if (!aligned(x, es) || !aligned(y, es) || (gain && !aligned(gain, ps)) || (bias && !aligned(bias, ps)) ||
      (mean && !aligned(mean, 4)) || (rstd && !aligned(rstd, 4)))
    return KL_ERR_MISALIGNED;
  if ((st = check_arch()) != KL_OK) return st;
  LnParams p{};
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.ldx = ldx;
  p.out = y;
  p.ldo = ldy;
  p.gain = gain;
  p.bias = bias;
  p.ptype = param_dtype;
  p.plus = (flags & KL_LN_MODULATE) ? 1.f : 0.f;
  p.group_rows = rows / groups;
  p.mean = mean;
  p.rstd = rstd;
  p.eps = eps;
  const bool vec = cols % (16 / es) == 0 && ln_rows_16(x, ldx, es) && ln_rows_16(y, ldy, es);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == KL_BF16  ? launch_ln_forward<__nv_bfloat16>(p, vec, s)
                        : dtype == KL_F16 ? launch_ln_forward<__half>(p, vec, s)
                                          : launch_ln_forward<float>(p, vec, s);
  return e == cudaSuccess ? KL_OK : cuda_fail(e);
}

size_t kl_layer_norm_backward_workspace_size(int dtype, int64_t rows, int64_t cols, int64_t groups) {
  using namespace kl;
  if (ln_check(dtype, rows, cols, groups, KL_F32, 0) != KL_OK) return 0;
  // the layout with the most splits: the one a call may take depends on its
  // pointers and strides
  int most = 0;
  const int es = ln_es(dtype), layouts = cols % (16 / es) == 0 ? 2 : 1;
  for (int vec = 0; vec < layouts; ++vec) {
    const int s = ln_splits(groups, rows / groups, ln_shape(cols, es, vec != 0, true));
    most = s > most ? s : most;
  }
  return up256((size_t)groups * (size_t)most * 2 * (size_t)cols * sizeof(float));
}

kl_status kl_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, int dtype, int64_t rows,
                                 int64_t cols, const float* mean, const float* rstd, const void* gain, int param_dtype,
                                 int64_t groups, int flags, void* dx, int64_t lddx, float* dgain, float* dbias,
                                 void* workspace, size_t ws_bytes, void* stream) {
  using namespace kl;
  if (!dy || !x || !mean || !rstd || !dx || !dgain != !dbias) return KL_ERR_INVALID_ARG;
  kl_status st = ln_check(dtype, rows, cols, groups, param_dtype, flags);
  if (st != KL_OK) return st;
  if (ldx < cols || lddy < cols || lddx < cols || dx == x || dx == dy) return KL_ERR_INVALID_ARG;
  const int es = ln_es(dtype), ps = ln_es(param_dtype);
  if (!aligned(x, es) || !aligned(dy, es) || !aligned(dx, es) || (gain && !aligned(gain, ps)) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || (dgain && (!aligned(dgain, 4) || !aligned(dbias, 4))))
    return KL_ERR_MISALIGNED;
  if (dgain) {
    if (!workspace || ws_bytes < kl_layer_norm_backward_workspace_size(dtype, rows, cols, groups))
      return KL_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return KL_ERR_MISALIGNED;
  }
  if ((st = check_arch()) != KL_OK) return st;
  LnParams p{};
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.ldx = ldx;
  p.dy = dy;
  p.ldy = lddy;
  p.out = dx;
  p.ldo = lddx;
  p.gain = gain;
  p.ptype = param_dtype;
  p.plus = (flags & KL_LN_MODULATE) ? 1.f : 0.f;
  p.group_rows = rows / groups;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.part = dgain ? reinterpret_cast<float*>(workspace) : nullptr;
  const bool vec = cols % (16 / es) == 0 && ln_rows_16(x, ldx, es) && ln_rows_16(dy, lddy, es) && ln_rows_16(dx, lddx, es);
  p.splits = ln_splits(groups, p.group_rows, ln_shape(cols, es, vec, true));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = dtype == KL_BF16  ? launch_ln_backward<__nv_bfloat16>(p, vec, s)
                  : dtype == KL_F16 ? launch_ln_backward<__half>(p, vec, s)
                                    : launch_ln_backward<float>(p, vec, s);
  if (e == cudaSuccess && dgain)
    e = launch_pdl(ln_param_sum_kernel, dim3((unsigned)((2 * cols + 31) / 32), (unsigned)groups), dim3(32, 8), 0, s,
                   (const float*)p.part, p.splits, cols, dgain, dbias);
  return e == cudaSuccess ? KL_OK : cuda_fail(e);
}

}  // extern "C"
