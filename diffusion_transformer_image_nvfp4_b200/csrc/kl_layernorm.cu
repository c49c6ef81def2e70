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

// A warp a row: no barrier, and every load of the row is in flight before the
// first sum, so a few rows a scheduler already cover the memory latency.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(128) ln_forward_warp_kernel(const LnParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  const int cols = (int)p.cols;
  const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx;
  uint4 q[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * 32) * V;
    q[i] = c < cols ? load_vec<T, V>(x + c) : make_uint4(0u, 0u, 0u, 0u);
  }
  // a vector is summed by itself first: short chains, small rounding errors
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float v[V];
    unpack_vec<T, V>(q[i], v);
    float t = v[0];
#pragma unroll
    for (int k = 1; k < V; ++k) t += v[k];
    s += t;
  }
  const float mean = warp_sum(s) / (float)cols;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((lane + i * 32) * V < cols) {
      float v[V];
      unpack_vec<T, V>(q[i], v);
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < V; ++k) t = fmaf(v[k] - mean, v[k] - mean, t);
      s += t;
    }
  }
  const float rstd = 1.0f / sqrtf(warp_sum(s) / (float)cols + p.eps);
  if (lane == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  const int64_t pbase = row / p.group_rows * p.cols;
  T* y = reinterpret_cast<T*>(p.out) + row * p.ldo;
  // one loop per parameter type: a branch in it would scatter the unrolled
  // code over more than the instruction cache holds
  auto finish = [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * 32) * V;
      if (c < cols) {
        float v[V], w[V];
        unpack_vec<T, V>(q[i], v);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = (v[k] - mean) * rstd;
        if (p.gain) {
          load_param_as<KIND, V>(p.gain, pbase + c, w);
#pragma unroll
          for (int k = 0; k < V; ++k) v[k] *= w[k] + p.plus;
        }
        if (p.bias) {
          load_param_as<KIND, V>(p.bias, pbase + c, w);
#pragma unroll
          for (int k = 0; k < V; ++k) v[k] += w[k];
        }
        store_vec<T, V>(y + c, v);
      }
    }
  };
  if (p.ptype == KL_BF16)
    finish(std::integral_constant<int, KL_BF16>());
  else if (p.ptype == KL_F16)
    finish(std::integral_constant<int, KL_F16>());
  else
    finish(std::integral_constant<int, KL_F32>());
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
__global__ void __launch_bounds__(512, NV == 1 || V == 1 ? 2 : 1)
    ln_backward_kernel(const LnParams p) {
  extern __shared__ float ln_red[];  // [2][blockDim.y][32][2]; then [blockDim.y][2][cols padded] if PG and blockDim.y > 1
  pdl_wait();
  pdl_trigger();
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

// Many rows of at least 64 vectors: a CTA takes tiles of R rows of its group,
// staged in shared memory by bulk copies a few tiles ahead (the row-at-a-time
// kernel above has one row in flight and waits for it).  A thread owns NV
// vectors of the columns in every row: it adds to the parameters' sums and to
// the 2R row sums in one pass, the CTA joins the row sums once per tile, and a
// second pass over the staged rows writes dx.
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {  // v[i] summed over the warp into lanes with lane % N == i, all in v[0]
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

template <typename T, int NV, int R, bool PG>
__global__ void __launch_bounds__(NV == 1 ? 384 : 512, NV == 1 ? 2 : 1) ln_backward_tile_kernel(const LnParams p, int stages) {
  constexpr int V = 16 / sizeof(T);
  extern __shared__ __align__(16) uint8_t ln_tiles[];  // [stages][x, dy][R][cols]
  __shared__ float red[2][NV == 1 ? 12 : 16][2 * R];
  __shared__ uint64_t full[4];
  __shared__ int abort_smem;
  volatile int* abort_flag = &abort_smem;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = blockDim.x >> 5;
  if (tid == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
    abort_smem = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int cols = (int)p.cols;
  const int64_t group = blockIdx.x / p.splits, split = blockIdx.x - group * p.splits;
  const int64_t r0 = group * p.group_rows;
  const int64_t tiles = (p.group_rows + R - 1) / R;
  const uint32_t row_bytes = (uint32_t)cols * sizeof(T), half = row_bytes * R;
  auto issue = [&](int64_t tile, int st) {  // thread 0
    const int n = (int)min((int64_t)R, p.group_rows - tile * R);
    mbar_arrive_expect_tx(&full[st], 2 * n * row_bytes);
    uint8_t* dst = ln_tiles + (size_t)st * 2 * half;
    for (int r = 0; r < n; ++r) {
      const int64_t row = r0 + tile * R + r;
      bulk_load(dst + r * row_bytes, reinterpret_cast<const T*>(p.x) + row * p.ldx, row_bytes, &full[st]);
      bulk_load(dst + half + r * row_bytes, reinterpret_cast<const T*>(p.dy) + row * p.ldy, row_bytes, &full[st]);
    }
  };
  if (tid == 0)
    for (int i = 0; i < stages - 1; ++i)
      if (split + (int64_t)i * p.splits < tiles) issue(split + (int64_t)i * p.splits, i);
  // lane r holds row r's statistics of the next tile
  float nmean = 0.f, nrstd = 0.f;
  auto stats = [&](int64_t tile) {
    const int64_t lr = tile * R + lane;
    const bool in = lane < R && lr < p.group_rows;
    nmean = in ? p.mean[r0 + lr] : 0.f;
    nrstd = in ? p.rstd[r0 + lr] : 0.f;
  };
  stats(split);
  const float inv_c = 1.0f / (float)cols;
  float g[NV][V], sg[PG ? NV : 1][V], sb[PG ? NV : 1][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (tid + i * (int)blockDim.x) * V;
    ln_factor<V>(p, group * p.cols + c, c < cols, g[i]);
  }
  if constexpr (PG) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) sg[i][k] = sb[i][k] = 0.f;
  }
  int st = 0, buf = 0, issued = 0;
  uint32_t phase = 0;
  for (int64_t tile = split; tile < tiles; tile += p.splits, buf ^= 1) {
    const int n = (int)min((int64_t)R, p.group_rows - tile * R);
    const float mean_l = nmean, rstd_l = nrstd;
    if (tile + p.splits < tiles) stats(tile + p.splits);
    // a wait that runs out is recorded and the turns go on: every thread takes
    // the same barriers, and the results are then void
    warp_wait(&full[st], phase, abort_flag);
    const T* xs = reinterpret_cast<const T*>(ln_tiles + (size_t)st * 2 * half);
    const T* ds = reinterpret_cast<const T*>(ln_tiles + (size_t)st * 2 * half + half);
    float s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[2 * r] = s[2 * r + 1] = 0.f;
      const float m = __shfl_sync(0xffffffffu, mean_l, r), rs = __shfl_sync(0xffffffffu, rstd_l, r);
      if (r < n) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (tid + i * (int)blockDim.x) * V;
          if (c < cols) {
            float xv[V], dv[V];
            unpack_vec<T, V>(*reinterpret_cast<const uint4*>(xs + r * cols + c), xv);
            unpack_vec<T, V>(*reinterpret_cast<const uint4*>(ds + r * cols + c), dv);
#pragma unroll
            for (int k = 0; k < V; ++k) {
              const float u = dv[k] * (xv[k] - m);  // dy * xhat / rstd
              if constexpr (PG) {
                sg[i][k] = fmaf(u, rs, sg[i][k]);
                sb[i][k] += dv[k];
              }
              s[2 * r] = fmaf(dv[k], g[i][k], s[2 * r]);
              s[2 * r + 1] = fmaf(u, g[i][k], s[2 * r + 1]);
            }
          }
        }
      }
    }
    warp_sums<2 * R>(s);
    if (lane < 2 * R) red[buf][warp][lane] = s[0];
    __syncthreads();
    // every thread is past the tile before this one: its stage is free
    if (tid == 0) {
      const int64_t next = tile + (int64_t)(stages - 1) * p.splits;
      if (next < tiles) issue(next, st == 0 ? stages - 1 : st - 1);
    }
    float tot = 0.f;
    if (lane < 2 * R)
      for (int w = 0; w < nw; ++w) tot += red[buf][w][lane];
    tot *= inv_c;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float m = __shfl_sync(0xffffffffu, mean_l, r), rs = __shfl_sync(0xffffffffu, rstd_l, r);
      // dx = rs * (h - mean(h) - (x - m) * rs * (rs * mean(h (x - m))))
      const float b = -__shfl_sync(0xffffffffu, tot, 2 * r);
      const float a = -rs * (rs * __shfl_sync(0xffffffffu, tot, 2 * r + 1));
      if (r < n) {
        T* dx = reinterpret_cast<T*>(p.out) + (r0 + tile * R + r) * p.ldo;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (tid + i * (int)blockDim.x) * V;
          if (c < cols) {
            float xv[V], dv[V];
            unpack_vec<T, V>(*reinterpret_cast<const uint4*>(xs + r * cols + c), xv);
            unpack_vec<T, V>(*reinterpret_cast<const uint4*>(ds + r * cols + c), dv);
#pragma unroll
            for (int k = 0; k < V; ++k) dv[k] = rs * fmaf(dv[k], g[i][k], fmaf(xv[k] - m, a, b));
            store_vec<T, V>(dx + c, dv);
          }
        }
      }
    }
    ++issued;
    if (++st == stages) {
      st = 0;
      phase ^= 1u;
    }
  }
  if (tid == 0 && *abort_flag) {
    // the copies of the last tiles land before the CTA can leave
    volatile int no_abort = 0;
    for (int i = max(0, issued - stages); i < issued; ++i)
      mbar_wait(&full[i % stages], (uint32_t)((i / stages) & 1), &no_abort);
  }
  if constexpr (PG) {
    float* out = p.part + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (tid + i * (int)blockDim.x) * V;
      if (c < cols) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          out[c + k] = sg[i][k];
          out[p.cols + c + k] = sb[i][k];
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
// columns a CTA, 16 thread rows taking every 16th partial (148 partials: ten
// loads a thread, all in flight at once).
__global__ void __launch_bounds__(512) ln_param_sum_kernel(const float* __restrict__ part, int splits, int64_t cols,
                                                           float* __restrict__ dgain, float* __restrict__ dbias) {
  __shared__ float red[16][33];
  pdl_wait();
  pdl_trigger();
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;  // of the 2 * cols sums
  const int64_t group = blockIdx.y;
  float s = 0.f;
  if (c < 2 * cols) {
    const float* src = part + group * splits * 2 * cols + c;
#pragma unroll 10
    for (int i = threadIdx.y; i < splits; i += 16) s += __ldg(src + (int64_t)i * 2 * cols);
  }
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < 2 * cols) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += red[i][threadIdx.x];
    if (c < cols)
      dgain[group * cols + c] = s;
    else
      dbias[group * cols + c - cols] = s;
  }
}

// ---------------------------------------------------------------- launchers
// From this many rows on a warp takes a row; fewer rows leave SMs idle that
// way, and a CTA takes one (short rows: always a warp).
constexpr int64_t kLnWarpRows = 4 * kNumSMs;

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

// The backward's tile kernel: threads, CTAs of an SM and of a group, stages.
// ok: rows of 64 to 1024 vectors, and tiles enough to give every SM two.
struct LnTile {
  bool ok;
  int nv, tx, rows, stages, splits;
};
static LnTile ln_tile(int64_t groups, int64_t group_rows, int64_t cols, int es, bool vec) {
  LnTile t{};
  if (!vec) return t;
  const int64_t n = cols / (16 / es);
  if (n < 64 || n > 1024) return t;
  t.nv = n <= 384 ? 1 : 2;
  t.tx = (int)(((n + t.nv - 1) / t.nv + 31) / 32 * 32);
  const int per_sm = (t.nv == 1 ? 768 : 512) / t.tx;
  const int64_t row = 2 * cols * es, budget = (int64_t)216 * 1024 / per_sm;
  t.rows = budget / (4 * row) >= 3 ? 4 : 2;
  const int64_t st = budget / (t.rows * row);
  t.stages = (int)(st > 4 ? 4 : st);
  const int64_t tiles = (group_rows + t.rows - 1) / t.rows;
  int64_t s = (int64_t)kNumSMs * per_sm / groups;
  s = s < tiles / 2 ? s : tiles / 2;
  s = s < 1 ? 1 : s;
  t.splits = (int)s;
  t.ok = t.stages >= 2 && tiles >= 2 && s * groups >= kNumSMs;
  return t;
}

template <typename T, int V, int NV>
static cudaError_t launch_ln_forward_nv(const LnParams& p, const LnShape& sh, cudaStream_t s) {
  return launch_pdl(ln_forward_kernel<T, V, NV>, dim3((unsigned)((p.rows + sh.ty - 1) / sh.ty)), dim3(sh.tx, sh.ty),
                    (size_t)sh.ty * 64 * sizeof(float), s, p);
}
template <typename T, int V, int NV>
static cudaError_t launch_ln_forward_warp(const LnParams& p, cudaStream_t s) {
  return launch_pdl(ln_forward_warp_kernel<T, V, NV>, dim3((unsigned)((p.rows + 3) / 4)), dim3(128), 0, s, p);
}
template <typename T>
static cudaError_t launch_ln_forward(const LnParams& p, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int64_t lanes = (p.cols + 31) / 32;
  if (p.rows >= kLnWarpRows || lanes <= 4 * V) {
    if (vec) {
      const int64_t nv = (p.cols / V + 31) / 32;
      if (nv <= 1) return launch_ln_forward_warp<T, V, 1>(p, s);
      if (nv <= 2) return launch_ln_forward_warp<T, V, 2>(p, s);
      if (nv <= 4) return launch_ln_forward_warp<T, V, 4>(p, s);
      if (nv <= 8) return launch_ln_forward_warp<T, V, 8>(p, s);
      if (nv <= 12) return launch_ln_forward_warp<T, V, 12>(p, s);
      if (nv <= 16) return launch_ln_forward_warp<T, V, 16>(p, s);
    } else {
      if (lanes <= 4) return launch_ln_forward_warp<T, 1, 4>(p, s);
      if (lanes <= 16) return launch_ln_forward_warp<T, 1, 16>(p, s);
      if (lanes <= 32) return launch_ln_forward_warp<T, 1, 32>(p, s);
      if (lanes <= 48) return launch_ln_forward_warp<T, 1, 48>(p, s);
      if (lanes <= 64) return launch_ln_forward_warp<T, 1, 64>(p, s);
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
  if (p.part && sh.ty > 1) smem += (size_t)sh.ty * 2 * NV * V * sh.tx * sizeof(float);
  const dim3 grid((unsigned)(p.rows / p.group_rows * p.splits)), block(sh.tx, sh.ty);
  return p.part ? launch_pdl(ln_backward_kernel<T, V, NV, true>, grid, block, smem, s, p)
                : launch_pdl(ln_backward_kernel<T, V, NV, false>, grid, block, smem, s, p);
}
template <typename T, int NV, int R, bool PG>
static cudaError_t launch_ln_tile(const LnParams& p, const LnTile& t, cudaStream_t s) {
  const size_t smem = (size_t)t.stages * 2 * R * p.cols * sizeof(T);
  const cudaError_t e = cudaFuncSetAttribute(ln_backward_tile_kernel<T, NV, R, PG>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, 216 * 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(ln_backward_tile_kernel<T, NV, R, PG>, dim3((unsigned)(p.rows / p.group_rows * p.splits)),
                    dim3(t.tx), smem, s, p, t.stages);
}
template <typename T, int NV>
static cudaError_t launch_ln_tile_nv(const LnParams& p, const LnTile& t, cudaStream_t s) {
  if (t.rows == 4)
    return p.part ? launch_ln_tile<T, NV, 4, true>(p, t, s) : launch_ln_tile<T, NV, 4, false>(p, t, s);
  return p.part ? launch_ln_tile<T, NV, 2, true>(p, t, s) : launch_ln_tile<T, NV, 2, false>(p, t, s);
}

template <typename T>
static cudaError_t launch_ln_backward(LnParams& p, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const LnTile t = ln_tile(p.rows / p.group_rows, p.group_rows, p.cols, sizeof(T), vec);
  if (t.ok) return t.nv == 1 ? launch_ln_tile_nv<T, 1>(p, t, s) : launch_ln_tile_nv<T, 2>(p, t, s);
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
    const LnTile t = ln_tile(groups, rows / groups, cols, es, vec != 0);
    const int s = t.ok ? t.splits : ln_splits(groups, rows / groups, ln_shape(cols, es, vec != 0, true));
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
  const bool vec = cols % (16 / es) == 0 && ln_rows_16(x, ldx, es) && ln_rows_16(dy, lddy, es) && ln_rows_16(dx, lddx, es) &&
                   ln_param_vec(gain, es, ps);
  const LnTile tile = ln_tile(groups, p.group_rows, cols, es, vec);
  p.splits = tile.ok ? tile.splits : ln_splits(groups, p.group_rows, ln_shape(cols, es, vec, true));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = dtype == KL_BF16  ? launch_ln_backward<__nv_bfloat16>(p, vec, s)
                  : dtype == KL_F16 ? launch_ln_backward<__half>(p, vec, s)
                                    : launch_ln_backward<float>(p, vec, s);
  if (e == cudaSuccess && dgain)
    e = launch_pdl(ln_param_sum_kernel, dim3((unsigned)((2 * cols + 31) / 32), (unsigned)groups), dim3(32, 16), 0, s,
                   (const float*)p.part, p.splits, cols, dgain, dbias);
  return e == cudaSuccess ? KL_OK : cuda_fail(e);
}

}  // extern "C"
