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
// a second pass over the row, so a large common offset does not cancel in it.
// The mean's own rounding stays: its error times rstd shifts every y of the row.
// Many rows of up to 768 16-byte vectors (fp32: 1,024 forward, 1,152 backward)
// are bound by HBM in both directions, once their instructions are few enough
// (packed pairs, parameters staged or held in registers) and their loads far
// enough ahead.  x (and dy) are read once from memory up to 4,096 vectors forward
// and 1,024 backward, off 16 bytes 8,192 and 4,096 columns, the widest a CTA a row
// and bound by its instructions (72% of the issue slots at 4,096 x 16,384); wider
// rows are read again for every pass, an element at a time.
//
// Forward: a warp a row where there are rows enough, else a CTA a row.
// Backward: a thread meets the same columns in every row of its CTA, so the
// sums for dgain and dbias stay in its registers; CTAs walk the rows of one
// group with a fixed stride and leave one partial row each, which a second
// kernel adds in a fixed order -- no atomics, the same bits every run.  Few
// rows: one launch, whose other CTAs add the columns from x and dy themselves.
//
// B200, bf16, device time: forward 17,408 x 3,072 38.9 us (84% of the 32.6 us its bytes
// take at the copy's rate); backward 20,992 x 3,072 65.9 us (89% of 59), dx
// alone 61.7.  Rows that 16-byte vectors do not fit: 4,557 x 2,934 18.8 and 24.1
// us (two elements at a time; 25.6 and 33.3 with one), 5,000 x 2,047 18.1 and
// 23.0 (one); under the profiler 45 to 47% of the issue slots are busy at 11 to 28%
// of DRAM: latency and instructions both.  Wide rows, forward and backward: bf16
// 4,096 x 8,192 55.5 and 66.2, 4,096 x 16,384 81.3 and 435; fp32 4,096 x 5,120
// 36.0 and 193, 4,096 x 16,384 157 and 449.

#include <type_traits>

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
  float* dgain; // backward of few rows
  float* dbias;
};

// V parameter values of type KIND at an address aligned for a load of V (V = 1: any)
template <int KIND, int V>
__device__ __forceinline__ void load_param_as(const void* base, int64_t at, float (&v)[V]) {
  if constexpr (KIND == KL_F32) {
    const float* p = reinterpret_cast<const float*>(base) + at;
    if constexpr (V == 1) {
      v[0] = __ldg(p);
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(p + i));
        v[i] = q.x;
        v[i + 1] = q.y;
        v[i + 2] = q.z;
        v[i + 3] = q.w;
      }
    }
  } else {
    using P = std::conditional_t<KIND == KL_BF16, __nv_bfloat16, __half>;
    const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + at;
    uint32_t w[4] = {};
    if constexpr (V == 8) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = q.x;
      w[1] = q.y;
      w[2] = q.z;
      w[3] = q.w;
    } else if constexpr (V == 4) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = q.x;
      w[1] = q.y;
    } else {
      w[0] = __ldg(p);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float lo, hi;
      unpack2<P>(w[i / 2], lo, hi);
      v[i] = (i & 1) ? hi : lo;
    }
  }
}
template <int V>
__device__ __forceinline__ void load_param(const void* base, int type, int64_t at, float (&v)[V]) {
  if (type == KL_F32)
    load_param_as<KL_F32, V>(base, at, v);
  else if (type == KL_BF16)
    load_param_as<KL_BF16, V>(base, at, v);
  else
    load_param_as<KL_F16, V>(base, at, v);
}

// the factors on xhat of V columns (1 where there is no gain)
template <int V>
__device__ __forceinline__ void ln_factor(const LnParams& p, int64_t at, bool in, float (&g)[V]) {
  if (p.gain && in) {
    load_param<V>(p.gain, p.ptype, at, g);
#pragma unroll
    for (int k = 0; k < V; ++k) g[k] += p.plus;
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) g[k] = 1.f;
  }
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
        load_param<V>(p.gain, p.ptype, pbase + c, w);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] *= w[k] + p.plus;
      }
      if (p.bias) {
        load_param<V>(p.bias, p.ptype, pbase + c, w);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] += w[k];
      }
      store_vec<T, V>(y + c, v);
    }
  }
}

// Many rows: a warp a row, so no barrier; CTAs stay, for rows of one group,
// whose factors and shifts they hold in shared memory as fp32 (read per row
// they cost more instructions than the rest of the row's work).  Arithmetic is
// on packed pairs.  ln_smem: [gain + plus][bias], planes of four columns of
// every vector, so a warp's 16-byte reads are consecutive.
template <int V>
__device__ __forceinline__ void ln_stage_params(const LnParams& p, int64_t group, float* dst) {
  const int cols = (int)p.cols, nvec = cols / V;
#pragma unroll V == 1 ? 8 : 2
  for (int j = threadIdx.x; j < nvec; j += blockDim.x) {
    float g[V], b[V];
    ln_factor<V>(p, group * p.cols + j * V, true, g);
    if (p.bias) {
      load_param<V>(p.bias, p.ptype, group * p.cols + j * V, b);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) b[k] = 0.f;
    }
    if constexpr (V == 1) {
      dst[j] = g[0];
      dst[cols + j] = b[0];
    } else {
#pragma unroll
      for (int h = 0; h < V / 4; ++h) {
        *reinterpret_cast<float4*>(dst + (h * nvec + j) * 4) =
            make_float4(g[4 * h], g[4 * h + 1], g[4 * h + 2], g[4 * h + 3]);
        *reinterpret_cast<float4*>(dst + cols + (h * nvec + j) * 4) =
            make_float4(b[4 * h], b[4 * h + 1], b[4 * h + 2], b[4 * h + 3]);
      }
    }
  }
}

template <typename T, int V, int NV>
__global__ void __launch_bounds__(256, NV <= (V == 4 ? 24 : 16) ? 2 : 1) ln_forward_warp_kernel(const LnParams p) {
  extern __shared__ __align__(16) float ln_smem[];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, cols = (int)p.cols, nvec = cols / V;
  const int64_t group = blockIdx.x / p.splits, split = blockIdx.x - group * p.splits;
  const bool affine = p.gain || p.bias;
  if (affine) {
    ln_stage_params<V>(p, group, ln_smem);
    __syncthreads();
  }
  const float inv_c = 1.0f / (float)cols;
  for (int64_t lr = split * 8 + (threadIdx.x >> 5); lr < p.group_rows; lr += p.splits * 8) {
    const int64_t row = group * p.group_rows + lr;
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx;
    uint4 q[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = lane + i * 32;
      q[i] = j < nvec ? load_vec<T, V>(x + j * V) : make_uint4(0u, 0u, 0u, 0u);
    }
    // a vector is summed by itself first: short chains, small rounding errors
    uint64_t s2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint64_t v[V / 2];
      unpack_vec2<T, V>(q[i], v);
      uint64_t t = v[0];
#pragma unroll
      for (int k = 1; k < V / 2; ++k) t = add_f32x2(t, v[k]);
      s2 = add_f32x2(s2, t);
    }
    const float mean = warp_sum(sum_f32x2(s2)) * inv_c;
    const uint64_t nm2 = pack_f32x2(-mean, -mean);
    s2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (lane + i * 32 < nvec) {
        uint64_t v[V / 2];
        unpack_vec2<T, V>(q[i], v);
        uint64_t t = 0;
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
          const uint64_t d = add_f32x2(v[k], nm2);
          t = fma_f32x2(d, d, t);
        }
        s2 = add_f32x2(s2, t);
      }
    }
    const float rstd = 1.0f / sqrtf(warp_sum(sum_f32x2(s2)) * inv_c + p.eps);
    if (lane == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
    const uint64_t rs2 = pack_f32x2(rstd, rstd);
    T* y = reinterpret_cast<T*>(p.out) + row * p.ldo;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = lane + i * 32;
      if (j < nvec) {
        uint64_t v[V / 2];
        unpack_vec2<T, V>(q[i], v);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) v[k] = mul_f32x2(add_f32x2(v[k], nm2), rs2);
        if (affine) {
#pragma unroll
          for (int h = 0; h < V / 4; ++h) {
            const ulonglong2 g = *reinterpret_cast<const ulonglong2*>(ln_smem + (h * nvec + j) * 4);
            const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(ln_smem + cols + (h * nvec + j) * 4);
            v[2 * h] = fma_f32x2(v[2 * h], g.x, b.x);
            v[2 * h + 1] = fma_f32x2(v[2 * h + 1], g.y, b.y);
          }
        }
        store_vec2<T, V>(y + j * V, v);
      }
    }
  }
}

// The same for rows that 16-byte vectors do not fit: W = 2 or 1 elements at a
// time, the second and third reading of the row from the caches.
template <typename T, int W>
__global__ void __launch_bounds__(256, 5) ln_forward_warp1_kernel(const LnParams p) {
  extern __shared__ __align__(16) float ln_smem[];  // [gain + plus][bias]
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, cols = (int)p.cols;
  const int64_t group = blockIdx.x / p.splits, split = blockIdx.x - group * p.splits;
  ln_stage_params<1>(p, group, ln_smem);
  __syncthreads();
  const float* gp = ln_smem + lane * W;
  const float* bp = gp + cols;
  const float inv_c = 1.0f / (float)cols;
  // f(index, slot, values, exist) for the lane's columns, eight loads at a time
  auto each = [&](const T* x, auto f) {
    int c = 0;
#pragma unroll (W == 1 ? 4 : 2)
    for (; c + 256 * W <= cols; c += 256 * W) {
      uint4 q[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) q[k] = load_vec<T, W>(x + c + k * 32 * W);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float v[W];
        unpack_vec<T, W>(q[k], v);
        f(c + k * 32 * W, k, v, true);
      }
    }
    if (c < cols) {
      uint4 q[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        q[k] = c + (k * 32 + lane) * W < cols ? load_vec<T, W>(x + c + k * 32 * W) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float v[W];
        unpack_vec<T, W>(q[k], v);
        f(c + k * 32 * W, k, v, c + (k * 32 + lane) * W < cols);
      }
    }
  };
  for (int64_t lr = split * 8 + (threadIdx.x >> 5); lr < p.group_rows; lr += p.splits * 8) {
    const int64_t row = group * p.group_rows + lr;
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx + lane * W;
    T* y = reinterpret_cast<T*>(p.out) + row * p.ldo + lane * W;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    each(x, [&](int, int k, const float (&v)[W], bool) {
#pragma unroll
      for (int w = 0; w < W; ++w) s[(k * W + w) & 3] += v[w];
    });
    const float mean = warp_sum((s[0] + s[1]) + (s[2] + s[3])) * inv_c;
    s[0] = s[1] = s[2] = s[3] = 0.f;
    each(x, [&](int, int k, const float (&v)[W], bool in) {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float d = in ? v[w] - mean : 0.f;
        s[(k * W + w) & 3] = fmaf(d, d, s[(k * W + w) & 3]);
      }
    });
    const float rstd = 1.0f / sqrtf(warp_sum((s[0] + s[1]) + (s[2] + s[3])) * inv_c + p.eps);
    if (lane == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
    each(x, [&](int c, int, const float (&v)[W], bool in) {
      if (in) {
        float g[W], b[W], o[W];
        if constexpr (W == 2) {
          const float2 gq = *reinterpret_cast<const float2*>(gp + c), bq = *reinterpret_cast<const float2*>(bp + c);
          g[0] = gq.x;
          g[1] = gq.y;
          b[0] = bq.x;
          b[1] = bq.y;
        } else {
          g[0] = gp[c];
          b[0] = bp[c];
        }
#pragma unroll
        for (int w = 0; w < W; ++w) o[w] = fmaf((v[w] - mean) * rstd, g[w], b[w]);
        store_vec<T, W>(y + c, o);
      }
    });
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
      load_param<1>(p.gain, p.ptype, pbase + c, w);
      v[0] *= w[0] + p.plus;
    }
    if (p.bias) {
      load_param<1>(p.bias, p.ptype, pbase + c, w);
      v[0] += w[0];
    }
    y[c] = from_f32<T>(v[0]);
  }
}

// CTA (group, split): rows split * blockDim.y + threadIdx.y, then every
// splits * blockDim.y.  The next row's x and dy are loaded before this row's
// sums are waited for.
template <typename T, int V, int NV, bool PG>
__device__ __forceinline__ void ln_backward_rows(const LnParams& p) {
  extern __shared__ float ln_red[];  // [2][blockDim.y][32][2]; then [blockDim.y][2][cols padded] if PG and blockDim.y > 1
  const int64_t group = blockIdx.x / p.splits, split = blockIdx.x - group * p.splits;
  const int64_t r0 = group * p.group_rows;
  const int64_t step = (int64_t)p.splits * blockDim.y;
  const float inv_c = 1.0f / (float)p.cols;
  float sg[PG ? NV : 1][V], sb[PG ? NV : 1][V];
  if constexpr (PG) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) sg[i][k] = sb[i][k] = 0.f;
  }
  float g[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = (int64_t)(threadIdx.x + i * blockDim.x) * V;
    ln_factor<V>(p, group * p.cols + c, c < p.cols, g[i]);
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
#pragma unroll
        for (int k = 0; k < V; ++k) {
          xh[i][k] = (xh[i][k] - mean) * rstd;
          if constexpr (PG) {
            sg[i][k] = fmaf(h[i][k], xh[i][k], sg[i][k]);
            sb[i][k] += h[i][k];
          }
          h[i][k] *= g[i][k];
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
          if constexpr (V == 1) {
            out[c] = sg[i][0];
            out[p.cols + c] = sb[i][0];
          } else {
#pragma unroll
            for (int k = 0; k < V; k += 4) {
              *reinterpret_cast<float4*>(out + c + k) = make_float4(sg[i][k], sg[i][k + 1], sg[i][k + 2], sg[i][k + 3]);
              *reinterpret_cast<float4*>(out + p.cols + c + k) =
                  make_float4(sb[i][k], sb[i][k + 1], sb[i][k + 2], sb[i][k + 3]);
            }
          }
        }
      }
    }
  }
}
template <typename T, int V, int NV, bool PG>
__global__ void __launch_bounds__(512, NV == 1 || V == 1 ? 2 : 1) ln_backward_kernel(const LnParams p) {
  pdl_wait();
  pdl_trigger();
  ln_backward_rows<T, V, NV, PG>(p);
}

// Few rows: one launch.  The first row_ctas CTAs are the kernel above without
// the parameters' sums; the others take 32 columns of a group each and add
// those columns over the group's rows, warps taking rows in turn, from x and
// dy as the caches hold them.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(512, NV == 1 || V == 1 ? 2 : 1)
    ln_backward_few_kernel(const LnParams p, unsigned row_ctas) {
  __shared__ float red[2][16][33];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x < row_ctas) {
    ln_backward_rows<T, V, NV, false>(p);
    return;
  }
  const unsigned blocks = (unsigned)((p.cols + 31) / 32), at = blockIdx.x - row_ctas, group = at / blocks;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int nw = (blockDim.x * blockDim.y) >> 5, rows = (int)p.group_rows;
  const int64_t c = (int64_t)(at - group * blocks) * 32 + lane, r0 = group * p.group_rows;
  float g = 0.f, b = 0.f;
  if (c < p.cols) {
    const T* x = reinterpret_cast<const T*>(p.x) + r0 * p.ldx + c;
    const T* dy = reinterpret_cast<const T*>(p.dy) + r0 * p.ldy + c;
#pragma unroll 8
    for (int r = w; r < rows; r += nw) {
      const float d = to_f32(dy[r * p.ldy]);
      g = fmaf(d, (to_f32(x[r * p.ldx]) - p.mean[r0 + r]) * p.rstd[r0 + r], g);
      b += d;
    }
  }
  red[0][w][lane] = g;
  red[1][w][lane] = b;
  __syncthreads();
  if (w < 2 && c < p.cols) {
    float s = red[w][0][lane];
    for (int i = 1; i < nw; ++i) s += red[w][i][lane];
    (w == 0 ? p.dgain : p.dbias)[group * p.cols + c] = s;
  }
}

// Many rows: a CTA takes tiles of R rows of its group; a thread owns E columns
// in every row (their factors and sums stay in its registers), holds the tile's
// values of its columns, adds them to the parameters' sums and to the 2R row
// sums, which the CTA joins once per tile, and writes dx.  Arithmetic is on
// packed pairs: unpacked it would bound the kernel instead of HBM.
//
// warp_sums: v[i] summed over the warp, into v[0] of the lanes with lane % N == i
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = N / 2; h >= 1; h /= 2) {
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const bool up = lane & h;
      const float send = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, h);
    }
  }
#pragma unroll
  for (int o = N; o < 32; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
}

// Where rows are short a CTA, one a SM, is several teams of threads that take
// tiles independently (a barrier each) and add their parameter sums through
// shared memory at the end: one partial row a SM for the second kernel to read.
constexpr int kLnTileRows = 2;
constexpr int kLnTileWarps = 16;  // of a team, at most
constexpr int kLnTeams = 12;      // at most (a team is at least two warps)
__device__ __forceinline__ void team_sync(int team, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

// A team's sums of the columns at (c, c + step) join the others' and go out,
// in the order of the teams.  buf: [teams][2][width]
__device__ __forceinline__ void ln_join_teams(const float* buf, int teams, int width, int cols, float* out) {
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * width; c += blockDim.x) {
    float s = buf[c];
    for (int t = 1; t < teams; ++t) s += buf[t * 2 * width + c];
    const int which = c >= width, col = c - which * width;
    if (col < cols) out[(int64_t)which * cols + col] = s;
  }
}

// what a thread keeps over the tiles, and one tile's arithmetic
template <int E, bool PG>
struct LnColumns {
  static constexpr int R = kLnTileRows;
  uint64_t g[E / 2], sg[PG ? E / 2 : 1], sb[PG ? E / 2 : 1];
  __device__ __forceinline__ void clear() {
    if constexpr (PG) {
#pragma unroll
      for (int k = 0; k < E / 2; ++k) sg[k] = sb[k] = 0;
    }
  }
  // x, dy of the rows -> xhat and dy; the thread's part of the row sums of h
  // and h xhat.  (xhat first, as in the kernels above: dy (x - mean) leaves the
  // range of fp32 where dy xhat does not.)  A column that does not exist holds
  // dy = 0, and the mean or an existing column's x: the xhat of anything else
  // might not be finite.  A row that does not exist holds zeros.
  __device__ __forceinline__ void sums(uint64_t (&x)[R][E / 2], const uint64_t (&d)[R][E / 2], const float (&m)[R],
                                       const float (&rs)[R], float (&s)[2 * R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint64_t nm2 = pack_f32x2(-m[r], -m[r]), rs2 = pack_f32x2(rs[r], rs[r]);
      uint64_t s0 = 0, s1 = 0;
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        x[r][k] = mul_f32x2(add_f32x2(x[r][k], nm2), rs2);
        const uint64_t u = mul_f32x2(d[r][k], x[r][k]);  // dy * xhat
        if constexpr (PG) {
          sg[k] = add_f32x2(sg[k], u);
          sb[k] = add_f32x2(sb[k], d[r][k]);
        }
        s0 = fma_f32x2(d[r][k], g[k], s0);
        s1 = fma_f32x2(u, g[k], s1);
      }
      s[2 * r] = sum_f32x2(s0);
      s[2 * r + 1] = sum_f32x2(s1);
    }
    warp_sums<2 * R>(s);
  }
  // the tile's row sums over the CTA from the warps' ([warps][2R]); warps past
  // nw hold zeros.  tot[i]: i-th sum, in every lane
  static __device__ __forceinline__ void join(const float* red, int nw, float (&tot)[2 * R]) {
    static_assert(R == 2 && kLnTileWarps == 16, "two sums of 16 warps a register");
    const int lane = threadIdx.x & 31, w = lane & 15, hi = lane >> 4;
    float a = w < nw ? red[w * 4 + hi] : 0.f, b = w < nw ? red[w * 4 + 2 + hi] : 0.f;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    const float a2 = __shfl_xor_sync(0xffffffffu, a, 16), b2 = __shfl_xor_sync(0xffffffffu, b, 16);
    tot[0] = hi ? a2 : a;
    tot[1] = hi ? a : a2;
    tot[2] = hi ? b2 : b;
    tot[3] = hi ? b : b2;
  }
  // dx = rs * (h - mean(h) - xhat * mean(h xhat)) of row r
  __device__ __forceinline__ void dx(const uint64_t (&x)[E / 2], const uint64_t (&d)[E / 2], float rs, float mh,
                                     float mhx, uint64_t (&o)[E / 2]) const {
    const uint64_t a2 = pack_f32x2(-mhx, -mhx), b2 = pack_f32x2(-mh, -mh), rs2 = pack_f32x2(rs, rs);
#pragma unroll
    for (int k = 0; k < E / 2; ++k) o[k] = mul_f32x2(rs2, fma_f32x2(d[k], g[k], fma_f32x2(x[k], a2, b2)));
  }
};

// Rows of vectors: tiles are staged in shared memory by bulk copies a few
// tiles ahead.
template <typename T, int NV, bool PG, bool TEAMS>
__global__ void __launch_bounds__(TEAMS ? 512 : 384, !TEAMS && NV * 16 / sizeof(T) <= 8 ? 2 : 1)
    ln_backward_tile_kernel(const LnParams p, int team_threads, int stages) {
  constexpr int V = 16 / sizeof(T), E = NV * V, R = kLnTileRows;
  extern __shared__ __align__(16) uint8_t ln_tiles[];  // [team][stages][x, dy][R][cols]
  __shared__ float red[TEAMS ? kLnTeams : 1][2][kLnTileWarps][2 * R];
  __shared__ uint64_t full_all[TEAMS ? kLnTeams : 1][4];
  __shared__ int abort_smem;
  volatile int* abort_flag = &abort_smem;
  const int tx = TEAMS ? team_threads : blockDim.x;
  const int teams = TEAMS ? blockDim.x / tx : 1, team = TEAMS ? threadIdx.x / tx : 0;
  const int tid = threadIdx.x - team * tx;
  const int warp = tid >> 5, lane = tid & 31, nw = tx >> 5;
  if (threadIdx.x == 0) {
    for (int t = 0; t < teams; ++t)
      for (int i = 0; i < stages; ++i) mbar_init(&full_all[t][i], 1);
    abort_smem = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  uint64_t* full = full_all[team];
  const int cols = (int)p.cols;
  const int group = blockIdx.x / p.splits, split = (blockIdx.x - group * p.splits) * teams + team;
  const int step = p.splits * teams, rows = (int)p.group_rows, tiles = (rows - 1) / R + 1;
  const int64_t r0 = group * p.group_rows;
  const uint32_t row_bytes = (uint32_t)cols * sizeof(T), half = row_bytes * R;
  uint8_t* mine = ln_tiles + (size_t)team * stages * 2 * half;
  auto issue = [&](int tile, int st) {  // the team's thread 0
    const int n = min(R, rows - tile * R);
    mbar_arrive_expect_tx(&full[st], 2 * n * row_bytes);
    uint8_t* dst = mine + (size_t)st * 2 * half;
    for (int r = 0; r < n; ++r) {
      const int64_t row = r0 + tile * R + r;
      bulk_load(dst + r * row_bytes, reinterpret_cast<const T*>(p.x) + row * p.ldx, row_bytes, &full[st]);
      bulk_load(dst + half + r * row_bytes, reinterpret_cast<const T*>(p.dy) + row * p.ldy, row_bytes, &full[st]);
    }
  };
  if (tid == 0)
    for (int i = 0; i < stages - 1; ++i)
      if (split + i * step < tiles) issue(split + i * step, i);
  // lane r holds the next tile's row r's statistics
  float next_mean = 0.f, next_rstd = 0.f;
  auto stats = [&](int tile) {
    const int lr = tile * R + lane;
    const bool in = lane < R && lr < rows;
    next_mean = in ? __ldg(p.mean + r0 + lr) : 0.f;
    next_rstd = in ? __ldg(p.rstd + r0 + lr) : 0.f;
  };
  stats(split);
  const float inv_c = 1.0f / (float)cols;
  LnColumns<E, PG> col;
  col.clear();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (tid + i * tx) * V;
    float g[V];
    ln_factor<V>(p, (int64_t)group * cols + c, c < cols, g);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) col.g[i * V / 2 + k] = pack_f32x2(g[2 * k], g[2 * k + 1]);
  }
  int st = 0, buf = 0, done = 0;
  uint32_t phase = 0;
  for (int tile = split; tile < tiles; tile += step, buf ^= 1) {
    const int n = min(R, rows - tile * R);
    float m[R], rs[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = __shfl_sync(0xffffffffu, next_mean, r);
      rs[r] = __shfl_sync(0xffffffffu, next_rstd, r);
    }
    if (tile + step < tiles) stats(tile + step);
    // a wait that runs out is recorded and the turns go on: every thread takes
    // the same barriers, and the results are then void
    warp_wait(&full[st], phase, abort_flag);
    const uint8_t* xs = mine + (size_t)st * 2 * half;
    uint64_t x[R][E / 2], d[R][E / 2];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = tid + i * tx;
        const bool in = r < n && at * V < cols;
        const uint4 qx = r < n ? *reinterpret_cast<const uint4*>(xs + r * row_bytes + (at * V < cols ? at : 0) * 16)
                               : make_uint4(0, 0, 0, 0);
        const uint4 qd =
            in ? *reinterpret_cast<const uint4*>(xs + half + r * row_bytes + at * 16) : make_uint4(0, 0, 0, 0);
        unpack_vec2<T, V>(qx, *reinterpret_cast<uint64_t(*)[V / 2]>(&x[r][i * V / 2]));
        unpack_vec2<T, V>(qd, *reinterpret_cast<uint64_t(*)[V / 2]>(&d[r][i * V / 2]));
      }
    float s[2 * R], tot[2 * R];
    col.sums(x, d, m, rs, s);
    if (lane < 2 * R) red[team][buf][warp][lane] = s[0];
    if constexpr (TEAMS)
      team_sync(team, tx);
    else
      __syncthreads();
    // every thread holds this tile in registers: the stage before it has been
    // free for a turn, and is loaded again
    if (tid == 0) {
      const int next = tile + (stages - 1) * step;
      if (next < tiles) issue(next, st == 0 ? stages - 1 : st - 1);
    }
    col.join(&red[team][buf][0][0], nw, tot);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r < n) {
        uint64_t o[E / 2];
        col.dx(x[r], d[r], rs[r], tot[2 * r] * inv_c, tot[2 * r + 1] * inv_c, o);
        T* dx = reinterpret_cast<T*>(p.out) + (r0 + tile * R + r) * p.ldo;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (tid + i * tx) * V;
          if (c < cols) store_vec2<T, V>(dx + c, *reinterpret_cast<uint64_t(*)[V / 2]>(&o[i * V / 2]));
        }
      }
    }
    ++done;
    if (++st == stages) {
      st = 0;
      phase ^= 1u;
    }
  }
  if (tid == 0 && *abort_flag) {
    // the copies of the last tiles land before the CTA can leave
    volatile int no_abort = 0;
    for (int i = max(0, done - stages); i < done; ++i)
      mbar_wait(&full[i % stages], (uint32_t)((i / stages) & 1), &no_abort);
  }
  if constexpr (PG) {
    // the stages become the teams' sums (nothing is on its way to them)
    float* out = p.part + (int64_t)blockIdx.x * 2 * p.cols;
    float* sums = TEAMS ? reinterpret_cast<float*>(ln_tiles) + team * 2 * cols : out;
    if constexpr (TEAMS) __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (tid + i * tx) * V;
      if (c < cols) {
#pragma unroll
        for (int k = 0; k < V / 2; k += 2) {
          *reinterpret_cast<ulonglong2*>(sums + c + 2 * k) = make_ulonglong2(col.sg[i * V / 2 + k], col.sg[i * V / 2 + k + 1]);
          *reinterpret_cast<ulonglong2*>(sums + cols + c + 2 * k) =
              make_ulonglong2(col.sb[i * V / 2 + k], col.sb[i * V / 2 + k + 1]);
        }
      }
    }
    if constexpr (TEAMS) ln_join_teams(reinterpret_cast<const float*>(ln_tiles), teams, cols, cols, out);
  }
}

// Rows that 16-byte vectors do not fit: a thread owns every 32nd column (W = 1)
// or pair of columns (W = 2) of its warp's 32 E, two columns a packed pair, and
// loads the next tile's values before it works on this one's.
template <typename T, int E, int W, bool PG>
__global__ void __launch_bounds__(E == 4 ? 768 : 512) ln_backward_tile1_kernel(const LnParams p, int tx) {
  constexpr int R = kLnTileRows;
  extern __shared__ float ln_sums[];  // [team][2][32 E * warps]
  __shared__ float red[kLnTeams][2][kLnTileWarps][2 * R];
  pdl_wait();
  pdl_trigger();
  const int teams = blockDim.x / tx, team = threadIdx.x / tx, tid = threadIdx.x - team * tx;
  const int warp = tid >> 5, lane = tid & 31, nw = tx >> 5;
  constexpr int H = W == 2 ? 1 : 32;  // from a pair's first column to its second; pairs are 64 apart
  const int cols = (int)p.cols, c0 = warp * 32 * E + lane * W;
  const bool full = (warp + 1) * 32 * E <= cols;  // every column of the warp exists
  const int group = blockIdx.x / p.splits, split = (blockIdx.x - group * p.splits) * teams + team;
  const int step = p.splits * teams, rows = (int)p.group_rows, tiles = (rows - 1) / R + 1;
  const int64_t r0 = group * p.group_rows;
  const float inv_c = 1.0f / (float)cols;
  LnColumns<E, PG> col;
  col.clear();
#pragma unroll
  for (int k = 0; k < E / 2; ++k) {
    float ga[1], gb[1];
    const int a = c0 + 64 * k, b = a + H;
    ln_factor<1>(p, (int64_t)group * cols + a, a < cols, ga);
    ln_factor<1>(p, (int64_t)group * cols + b, b < cols, gb);
    col.g[k] = pack_f32x2(ga[0], gb[0]);
  }
  // as stored: an element, or the words of a pair
  using Raw = std::conditional_t<W == 1, T, std::conditional_t<sizeof(T) == 4, uint2, uint32_t>>;
  Raw rx[R][E / W], rd[R][E / W];
  auto values = [](const Raw* q, float (&v)[2]) {
    if constexpr (W == 1) {
      v[0] = to_f32(q[0]);
      v[1] = to_f32(q[1]);
    } else if constexpr (sizeof(T) == 4) {
      v[0] = __uint_as_float(q->x);
      v[1] = __uint_as_float(q->y);
    } else {
      unpack2<T>(*q, v[0], v[1]);
    }
  };
  // One copy of the loop for warps that have all their columns: with what the
  // others need in it, 4,557 x 2,934 bf16 took 30.9 us in place of 24.1.  In
  // place of the x of columns that do not exist (LnColumns::sums) pairs read the
  // row's first and single elements take the mean: 5,000 x 4,001 fp32 49.4 us,
  // 55.4 the other way; 4,557 x 2,934 bf16, dx alone, 20.9 and 25.5.
  auto walk = [&](auto whole) {
    constexpr bool FULL = decltype(whole)::value;
    float next_mean = 0.f, next_rstd = 0.f;  // lane r: row r's
    auto fetch = [&](int tile) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool live = tile * R + r < rows;
        const int64_t row = r0 + (live ? tile * R + r : 0);
        const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx + c0;
        const T* d = reinterpret_cast<const T*>(p.dy) + row * p.ldy + c0;
        if (live) {
#pragma unroll
          for (int k = 0; k < E / W; ++k) {
            const bool in = FULL || c0 + 32 * W * k < cols;
            if constexpr (W == 2)
              rx[r][k] = *reinterpret_cast<const Raw*>(x + (in ? 64 * k : -c0));
            else
              rx[r][k] = in ? *reinterpret_cast<const Raw*>(x + 32 * k) : Raw{};
            rd[r][k] = in ? *reinterpret_cast<const Raw*>(d + 32 * W * k) : Raw{};
          }
        } else {
#pragma unroll
          for (int k = 0; k < E / W; ++k) rx[r][k] = rd[r][k] = Raw{};
        }
      }
      const int lr = tile * R + lane;
      const bool in = lane < R && lr < rows;
      next_mean = in ? __ldg(p.mean + r0 + lr) : 0.f;
      next_rstd = in ? __ldg(p.rstd + r0 + lr) : 0.f;
    };
    if (split < tiles) fetch(split);
    int buf = 0;
    for (int tile = split; tile < tiles; tile += step, buf ^= 1) {
      const int n = min(R, rows - tile * R);
      float m[R], rs[R];
      uint64_t x[R][E / 2], d[R][E / 2];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        m[r] = __shfl_sync(0xffffffffu, next_mean, r);
        rs[r] = __shfl_sync(0xffffffffu, next_rstd, r);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          float xv[2], dv[2];
          values(&rx[r][k * (2 / W)], xv);
          values(&rd[r][k * (2 / W)], dv);
          if constexpr (!FULL && W == 1) {
            if (c0 + 64 * k >= cols) xv[0] = m[r];
            if (c0 + 64 * k + H >= cols) xv[1] = m[r];
          }
          x[r][k] = pack_f32x2(xv[0], xv[1]);
          d[r][k] = pack_f32x2(dv[0], dv[1]);
        }
      }
      if (tile + step < tiles) fetch(tile + step);
      float s[2 * R], tot[2 * R];
      col.sums(x, d, m, rs, s);
      if (lane < 2 * R) red[team][buf][warp][lane] = s[0];
      team_sync(team, tx);
      col.join(&red[team][buf][0][0], nw, tot);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r < n) {
          uint64_t o[E / 2];
          col.dx(x[r], d[r], rs[r], tot[2 * r] * inv_c, tot[2 * r + 1] * inv_c, o);
          T* dx = reinterpret_cast<T*>(p.out) + (r0 + tile * R + r) * p.ldo + c0;
#pragma unroll
          for (int k = 0; k < E / 2; ++k) {
            float v[2];
            unpack_f32x2(o[k], v[0], v[1]);
            if constexpr (W == 2) {
              if (FULL || c0 + 64 * k < cols) store_vec<T, 2>(dx + 64 * k, v);
            } else {
              if (FULL || c0 + 64 * k < cols) dx[64 * k] = from_f32<T>(v[0]);
              if (FULL || c0 + 64 * k + H < cols) dx[64 * k + H] = from_f32<T>(v[1]);
            }
          }
        }
      }
    }
  };
  if (full)
    walk(std::true_type{});
  else
    walk(std::false_type{});
  if constexpr (PG) {
    const int width = nw * 32 * E;
    float* sums = ln_sums + team * 2 * width + c0;
#pragma unroll
    for (int k = 0; k < E / 2; ++k) {
      unpack_f32x2(col.sg[k], sums[64 * k], sums[64 * k + H]);
      unpack_f32x2(col.sb[k], sums[width + 64 * k], sums[width + 64 * k + H]);
    }
    ln_join_teams(ln_sums, teams, width, cols, p.part + (int64_t)blockIdx.x * 2 * p.cols);
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
      load_param<1>(p.gain, p.ptype, pbase + c, w);
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

// dgain / dbias [groups][cols] from the partial rows, in a fixed order: 32
// columns a CTA, 32 thread rows taking every 32nd partial (296 partials: ten
// loads a thread, all in flight at once).
__global__ void __launch_bounds__(1024) ln_param_sum_kernel(const float* __restrict__ part, int splits, int64_t cols,
                                                           float* __restrict__ dgain, float* __restrict__ dbias) {
  __shared__ float red[32][33];
  pdl_wait();
  pdl_trigger();
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;  // of the 2 * cols sums
  const int64_t group = blockIdx.y;
  float s = 0.f;
  if (c < 2 * cols) {
    const float* src = part + group * splits * 2 * cols + c;
#pragma unroll 10
    for (int i = threadIdx.y; i < splits; i += 32) s += __ldg(src + (int64_t)i * 2 * cols);
  }
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < 2 * cols) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += red[i][threadIdx.x];
    if (c < cols)
      dgain[group * cols + c] = s;
    else
      dbias[group * cols + c - cols] = s;
  }
}

// ---------------------------------------------------------------- launchers
// From this many rows on a warp takes a row; fewer leave SMs idle that way,
// and a CTA takes one (as for groups of a few rows, whose parameters would be
// staged for nothing).
constexpr int64_t kLnWarpRows = 4 * kNumSMs;
// up to these rows of a group, and bytes of x, the backward is one launch
constexpr int64_t kLnFewRows = 400, kLnFewBytes = 8 << 20;

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
// the group has rows for.  Wide rows' parameter sums have CTAs of 256 columns
// beside: 64 of them a SM (all splits of 16,384 columns) are enough, and the
// workspace stays below 20 MB or one partial row a group.
constexpr int64_t kLnWideCtas = 64 * kNumSMs;
static int ln_splits(int64_t groups, int64_t group_rows, int64_t cols, const LnShape& sh) {
  const int64_t per_sm = sh.tx * sh.ty <= 512 ? 1024 / (sh.tx * sh.ty) : 1;
  int64_t s = (int64_t)kNumSMs * per_sm / groups;
  if (sh.nv == 0) {
    const int64_t enough = kLnWideCtas / (groups * ((cols + 255) / 256));
    if (s > enough) s = enough;
  }
  const int64_t most = (group_rows + sh.ty - 1) / sh.ty;
  s = s < 1 ? 1 : s;
  return (int)(s < most ? s : most);
}

// CTAs of a group of rows: `ctas` over all groups, at most one for `unit` rows
static int64_t ln_ctas(int64_t groups, int64_t group_rows, int64_t ctas, int64_t unit) {
  const int64_t s = ctas / groups, most = (group_rows + unit - 1) / unit;
  return s < 1 ? 1 : s < most ? s : most;
}

// The backward's tile kernels.  bf16 rows of 193 to 384 vectors give a thread
// two of them: 20,992 x 3,072 takes 65.6 us so and 72.8 with one, the work of
// joining the row sums being the same for a thread of 8 columns and one of 16.
// LnTile: threads of a team, teams, columns a thread,
// stages (0: single elements), CTAs of a group.  ok: 64 to 768 (fp32: 1152)
// vectors a row, or 256 to 4096 single elements, and rows enough for half the SMs.
struct LnTile {
  bool ok;
  int n, tx, teams, stages, splits;  // n: vectors, or single columns, of a thread
};
static LnTile ln_tile(int64_t groups, int64_t group_rows, int64_t cols, int es, bool vec) {
  LnTile t{};
  int threads, per_sm = 1;
  if (vec) {
    const int64_t n = cols / (16 / es);
    if (n < 64 || n > (es == 4 ? 1152 : 768)) return t;
    t.n = es == 2 && n > 192 && n <= 384 ? 2 : (int)((n + 383) / 384);
    t.tx = (int)(((n + t.n - 1) / t.n + 31) / 32 * 32);
    threads = t.tx <= 192 && t.n == 1 ? 512 : t.tx;
    per_sm = (t.tx > 192 && t.n * 16 / es <= 8) || (t.n == 2 && t.tx <= 192) ? 2 : 1;
  } else {
    if (cols < 256 || cols > 4096) return t;
    t.n = cols <= 1024 ? 4 : 8;
    t.tx = (int)((cols + 32 * t.n - 1) / (32 * t.n) * 32);
    threads = t.n == 4 ? 768 : 512;
  }
  const int64_t s = ln_ctas(groups, group_rows, kNumSMs * per_sm, 2 * kLnTileRows);
  t.splits = (int)s;
  // no team without two tiles
  int64_t teams = group_rows / (2 * kLnTileRows * s);
  teams = teams < 1 ? 1 : teams;
  t.teams = threads / t.tx;
  if (t.teams > teams) t.teams = (int)teams;
  if (vec) {
    const int64_t stage = 2 * kLnTileRows * cols * es, budget = (int64_t)216 * 1024 / (t.teams * per_sm);
    t.stages = (int)(budget / stage > 4 ? 4 : budget / stage);
    if (t.stages < 2) return t;
  }
  t.ok = group_rows >= 2 * kLnTileRows && s * groups >= kNumSMs / 2;
  return t;
}

// every row of x, dy and the output starts on two elements, and has an even number
static bool ln_pairs(const LnParams& p, size_t es) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.dy) | reinterpret_cast<uintptr_t>(p.out);
  return p.cols % 2 == 0 && at % (2 * es) == 0 && p.ldx % 2 == 0 && p.ldy % 2 == 0 && p.ldo % 2 == 0;
}

template <typename T, int V, int NV>
static cudaError_t launch_ln_forward_nv(const LnParams& p, const LnShape& sh, cudaStream_t s) {
  return launch_pdl(ln_forward_kernel<T, V, NV>, dim3((unsigned)((p.rows + sh.ty - 1) / sh.ty)), dim3(sh.tx, sh.ty),
                    (size_t)sh.ty * 64 * sizeof(float), s, p);
}
template <typename T, int V, int NV>
static cudaError_t launch_ln_forward_warp(LnParams& p, cudaStream_t s) {
  const size_t smem = p.gain || p.bias ? (size_t)p.cols * 8 : 0;
  const int per_sm = NV * V <= 16 ? 5 : NV * V <= 32 ? 3 : NV <= (V == 4 ? 24 : 16) ? 2 : 1;
  const int64_t groups = p.rows / p.group_rows;
  p.splits = (int)ln_ctas(groups, p.group_rows, (int64_t)kNumSMs * per_sm, 8);
  const cudaError_t e = cudaFuncSetAttribute(ln_forward_warp_kernel<T, V, NV>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, 32 * NV * V * 8);
  if (e != cudaSuccess) return e;
  return launch_pdl(ln_forward_warp_kernel<T, V, NV>, dim3((unsigned)(groups * p.splits)), dim3(256), smem, s, p);
}
template <typename T>
static cudaError_t launch_ln_forward(LnParams& p, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  if (p.rows >= kLnWarpRows && p.group_rows >= 16) {
    const int64_t groups = p.rows / p.group_rows, nv = (p.cols / V + 31) / 32;
    if (vec) {
      if (nv <= 1) return launch_ln_forward_warp<T, V, 1>(p, s);
      if (nv <= 2) return launch_ln_forward_warp<T, V, 2>(p, s);
      if (nv <= 4) return launch_ln_forward_warp<T, V, 4>(p, s);
      if (nv <= 8) return launch_ln_forward_warp<T, V, 8>(p, s);
      if (nv <= 12) return launch_ln_forward_warp<T, V, 12>(p, s);
      if (nv <= 16) return launch_ln_forward_warp<T, V, 16>(p, s);
      if (nv <= 24) return launch_ln_forward_warp<T, V, 24>(p, s);
      if constexpr (V == 4) {
        if (nv <= 32) return launch_ln_forward_warp<T, 4, 32>(p, s);
      }
    } else if (p.cols <= 6144) {
      const size_t smem = (size_t)p.cols * 8;
      p.splits = (int)ln_ctas(groups, p.group_rows, kNumSMs * 5, 8);
      auto kern = ln_pairs(p, sizeof(T)) ? ln_forward_warp1_kernel<T, 2> : ln_forward_warp1_kernel<T, 1>;
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 6144 * 8);
      if (e != cudaSuccess) return e;
      return launch_pdl(kern, dim3((unsigned)(groups * p.splits)), dim3(256), smem, s, p);
    }
  }
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
  if (p.dgain && !p.part) {
    const int64_t groups = p.rows / p.group_rows, row_ctas = groups * p.splits;
    return launch_pdl(ln_backward_few_kernel<T, V, NV>, dim3((unsigned)(row_ctas + groups * ((p.cols + 31) / 32))),
                      dim3(sh.tx, sh.ty), smem, s, p, (unsigned)row_ctas);
  }
  if (p.part && sh.ty > 1) smem += (size_t)sh.ty * 2 * NV * V * sh.tx * sizeof(float);
  const dim3 grid((unsigned)(p.rows / p.group_rows * p.splits)), block(sh.tx, sh.ty);
  return p.part ? launch_pdl(ln_backward_kernel<T, V, NV, true>, grid, block, smem, s, p)
                : launch_pdl(ln_backward_kernel<T, V, NV, false>, grid, block, smem, s, p);
}
// One launch for the rows and the parameters' sums where a second launch (3 us
// of the GPU, as much of the CPU) costs more than reading x and dy twice.
// One and two launches, us: 77 x 1155 fp32 2.9 and 5.2, 300 x 3072 bf16 5.1 and
// 7.9, 450 x 3072 8.7 and 8.8, 1000 x 1024 10.2 and 9.5.
static bool ln_few(int64_t groups, int64_t group_rows, int64_t cols, int es, bool vec) {
  return group_rows <= kLnFewRows && groups * group_rows * cols * es <= kLnFewBytes && ln_shape(cols, es, vec, true).nv > 0;
}

template <typename T, int NV, bool PG, bool TEAMS>
static cudaError_t launch_ln_tile(const LnParams& p, const LnTile& t, cudaStream_t s) {
  const size_t smem = (size_t)t.teams * t.stages * 2 * kLnTileRows * p.cols * sizeof(T);
  const cudaError_t e = cudaFuncSetAttribute(ln_backward_tile_kernel<T, NV, PG, TEAMS>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, 216 * 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(ln_backward_tile_kernel<T, NV, PG, TEAMS>, dim3((unsigned)(p.rows / p.group_rows * p.splits)),
                    dim3(t.tx * t.teams), smem, s, p, t.tx, t.stages);
}
template <typename T, bool PG>
static cudaError_t launch_ln_tiles(const LnParams& p, const LnTile& t, bool vec, cudaStream_t s) {
  if (!vec) {
    const dim3 grid((unsigned)(p.rows / p.group_rows * p.splits)), block(t.tx * t.teams);
    const size_t smem = PG ? (size_t)t.teams * t.tx * 2 * t.n * sizeof(float) : 0;  // at most 32 KB
    auto kern = ln_pairs(p, sizeof(T)) ? (t.n == 4 ? ln_backward_tile1_kernel<T, 4, 2, PG> : ln_backward_tile1_kernel<T, 8, 2, PG>)
                                       : (t.n == 4 ? ln_backward_tile1_kernel<T, 4, 1, PG> : ln_backward_tile1_kernel<T, 8, 1, PG>);
    return launch_pdl(kern, grid, block, smem, s, p, t.tx);
  }
  if (t.n == 1) return t.tx <= 192 ? launch_ln_tile<T, 1, PG, true>(p, t, s) : launch_ln_tile<T, 1, PG, false>(p, t, s);
  if constexpr (sizeof(T) == 4) {
    if (t.n == 3) return launch_ln_tile<T, 3, PG, false>(p, t, s);
  }
  return launch_ln_tile<T, 2, PG, false>(p, t, s);
}

template <typename T>
static cudaError_t launch_ln_backward(LnParams& p, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const LnTile t = ln_tile(p.rows / p.group_rows, p.group_rows, p.cols, sizeof(T), vec);
  if (t.ok && !ln_few(p.rows / p.group_rows, p.group_rows, p.cols, sizeof(T), vec))
    return p.part ? launch_ln_tiles<T, true>(p, t, vec, s) : launch_ln_tiles<T, false>(p, t, vec, s);
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

// parameters suit loads of as many elements as 16 bytes of a row hold
static bool ln_param_vec(const void* p, int es, int ps) {
  const int bytes = 16 / es * ps;
  return !p || aligned(p, bytes < 16 ? bytes : 16);
}

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
  const bool vec = cols % (16 / es) == 0 && ln_rows_16(x, ldx, es) && ln_rows_16(y, ldy, es) &&
                   ln_param_vec(gain, es, ps) && ln_param_vec(bias, es, ps);
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
    if (ln_few(groups, rows / groups, cols, es, vec != 0)) continue;
    const LnTile t = ln_tile(groups, rows / groups, cols, es, vec != 0);
    const int s = t.ok ? t.splits : ln_splits(groups, rows / groups, cols, ln_shape(cols, es, vec != 0, true));
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
    const size_t need = kl_layer_norm_backward_workspace_size(dtype, rows, cols, groups);
    if (need && (!workspace || ws_bytes < need)) return KL_ERR_WORKSPACE;
    if (need && !aligned(workspace, 16)) return KL_ERR_MISALIGNED;
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
  const bool vec = cols % (16 / es) == 0 && ln_rows_16(x, ldx, es) && ln_rows_16(dy, lddy, es) && ln_rows_16(dx, lddx, es) &&
                   ln_param_vec(gain, es, ps);
  const bool few = ln_few(groups, p.group_rows, cols, es, vec);
  p.part = dgain && !few ? reinterpret_cast<float*>(workspace) : nullptr;
  p.dgain = dgain;
  p.dbias = dbias;
  const LnTile tile = ln_tile(groups, p.group_rows, cols, es, vec);
  p.splits = tile.ok && !few ? tile.splits : ln_splits(groups, p.group_rows, cols, ln_shape(cols, es, vec, true));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = dtype == KL_BF16  ? launch_ln_backward<__nv_bfloat16>(p, vec, s)
                  : dtype == KL_F16 ? launch_ln_backward<__half>(p, vec, s)
                                    : launch_ln_backward<float>(p, vec, s);
  if (e == cudaSuccess && p.part)
    e = launch_pdl(ln_param_sum_kernel, dim3((unsigned)((2 * cols + 31) / 32), (unsigned)groups), dim3(32, 32), 0, s,
                   (const float*)p.part, p.splits, cols, dgain, dbias);
  return e == cudaSuccess ? KL_OK : cuda_fail(e);
}

}  // extern "C"
