// kl_rope.cu -- rotary positions with several axes (time, height, width, ...)
// applied to [batch, token, head, dim] tensors, and the inverse rotation,
// which is also the gradient (a rotation's transpose).
//
// Pair j of a head turns by pos[token, axis(j)] * f_j: the pairs are divided
// among the axes in order (`sections`), f_j = theta^(-u / n_a) with u the
// pair's index in its axis' section of n_a pairs (KL_ROPE_LADDER_AXIS), or
// theta^(-j / P) over all P pairs (KL_ROPE_LADDER_SHARED).  Dims past the
// pairs are copied.
//
// Angles: f_j / pi is made on the host in extended precision; position times
// it is one fp64 product, reduced by whole turns exactly (h - 2 rint(h / 2)),
// so positions far along an axis lose nothing; sincospif of the reduced angle
// is fp32.  Each angle is used by every head of its token, so a CTA makes its
// tokens' table in shared memory once and a thread keeps its pairs' cosines
// and sines in registers over the heads.
//
// Bound by HBM: one read and one write of the tensor; the fp64 work is one
// angle per (token, pair), a head's share of it 1 / H.
#include <cmath>

#include "../../include/klein.h"
#include "kl_common.cuh"
#include "kl_internal.h"

namespace kl {

constexpr int kRopeMaxPairs = 256;  // head dim 512
constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;  // heads a thread loads before it stores the first

struct RopeParams {
  const void* x;
  void* out;
  const void* pos;
  int64_t batch, tokens, heads;
  int64_t xs_b, xs_t, xs_h, os_b, os_t, os_h;  // strides in elements; dims are consecutive
  int64_t pos_b;                               // position rows between batches (0: shared)
  int dim, pairs, naxes, pos_type;
  int units;            // per head: vectors of dims (interleaved) or of pairs, then of copied dims (half)
  int tok_per_cta;
  float sign;           // -1: inverse
  int first[KL_ROPE_MAX_AXES + 1];  // first pair of each axis
  double freq[kRopeMaxPairs];       // f_j / pi
};

__device__ __forceinline__ double rope_pos(const RopeParams& p, int64_t i) {
  if (p.pos_type == KL_POS_I32) return (double)reinterpret_cast<const int32_t*>(p.pos)[i];
  if (p.pos_type == KL_POS_I64) return (double)reinterpret_cast<const int64_t*>(p.pos)[i];
  return (double)reinterpret_cast<const float*>(p.pos)[i];
}

// V elements a thread at a time (16 bytes, or V = 1 for what is not aligned;
// interleaved pairs then move two elements).  A thread keeps one unit u of the
// head and walks the heads: threads = units x slots.
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(512) rope_axes_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float2 rope_table_smem[];  // [tok_per_cta][pairs] (cos, sin)
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, nthreads = blockDim.x;
  const int64_t chunks = (p.tokens + p.tok_per_cta - 1) / p.tok_per_cta;
  const int64_t b = blockIdx.x / chunks, t0 = (blockIdx.x - b * chunks) * p.tok_per_cta;
  const int nt = (int)min((int64_t)p.tok_per_cta, p.tokens - t0);
  for (int i = tid; i < nt * p.pairs; i += nthreads) {
    const int t = i / p.pairs, j = i - t * p.pairs;
    int a = 0;
    while (j >= p.first[a + 1]) ++a;
    const double h = rope_pos(p, (b * p.pos_b + t0 + t) * p.naxes + a) * p.freq[j];
    float s, c;
    sincospif((float)(h - 2.0 * rint(0.5 * h)), &s, &c);
    rope_table_smem[i] = make_float2(c, p.sign * s);
  }
  __syncthreads();
  const int slots = nthreads / p.units;
  const int u = tid % p.units, slot = tid / p.units;
  if (slot >= slots) return;
  constexpr int NP = HALF ? V : (V == 1 ? 1 : V / 2);  // pairs of a unit
  const int pair_units = p.pairs / NP;
  // first pair of the unit; interleaved units may reach past the last pair
  const int j0 = u * NP;
  const int64_t hstep = (int64_t)gridDim.y * slots;
  for (int t = 0; t < nt; ++t) {
    const T* xt = reinterpret_cast<const T*>(p.x) + b * p.xs_b + (t0 + t) * p.xs_t;
    T* ot = reinterpret_cast<T*>(p.out) + b * p.os_b + (t0 + t) * p.os_t;
    float2 cs[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i)
      cs[i] = j0 + i < p.pairs ? rope_table_smem[t * p.pairs + j0 + i] : make_float2(1.f, 0.f);
    const int64_t h0 = (int64_t)blockIdx.y * slots + slot;
    if constexpr (HALF) {
      if (u < pair_units) {
        // (loads of several heads ahead of the first store: x and out may be
        // the same tensor, so the compiler cannot move them itself)
        for (int64_t h = h0; h < p.heads; h += kRopeBatch * hstep) {
          uint4 qa[kRopeBatch], qc[kRopeBatch];
#pragma unroll
          for (int k = 0; k < kRopeBatch; ++k) {
            if (h + k * hstep < p.heads) {
              const T* x = xt + (h + k * hstep) * p.xs_h + j0;
              qa[k] = load_vec<T, V>(x);
              qc[k] = load_vec<T, V>(x + p.pairs);
            }
          }
#pragma unroll
          for (int k = 0; k < kRopeBatch; ++k) {
            if (h + k * hstep < p.heads) {
              T* o = ot + (h + k * hstep) * p.os_h + j0;
              float a[V], c[V];
              unpack_vec<T, V>(qa[k], a);
              unpack_vec<T, V>(qc[k], c);
#pragma unroll
              for (int i = 0; i < V; ++i) {
                const float a0 = a[i], c0 = c[i];
                a[i] = a0 * cs[i].x - c0 * cs[i].y;
                c[i] = a0 * cs[i].y + c0 * cs[i].x;
              }
              store_vec<T, V>(o, a);
              store_vec<T, V>(o + p.pairs, c);
            }
          }
        }
      } else {
        const int d = 2 * p.pairs + (u - pair_units) * V;
        for (int64_t h = h0; h < p.heads; h += hstep) {
          if constexpr (V == 1)
            ot[h * p.os_h + d] = xt[h * p.xs_h + d];
          else
            *reinterpret_cast<uint4*>(ot + h * p.os_h + d) = load_vec<T, V>(xt + h * p.xs_h + d);
        }
      }
    } else if constexpr (V == 1) {
      const int d = 2 * u;
      const bool turn = u < p.pairs, two = d + 1 < p.dim;
      for (int64_t h = h0; h < p.heads; h += hstep) {
        const T* x = xt + h * p.xs_h + d;
        T* o = ot + h * p.os_h + d;
        if (turn) {
          const float a0 = to_f32(x[0]), c0 = to_f32(x[1]);
          o[0] = from_f32<T>(a0 * cs[0].x - c0 * cs[0].y);
          o[1] = from_f32<T>(a0 * cs[0].y + c0 * cs[0].x);
        } else {
          const T a0 = x[0];
          if (two) o[1] = x[1];
          o[0] = a0;
        }
      }
    } else {
      for (int64_t h = h0; h < p.heads; h += kRopeBatch * hstep) {
        uint4 q[kRopeBatch];
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k)
          if (h + k * hstep < p.heads) q[k] = load_vec<T, V>(xt + (h + k * hstep) * p.xs_h + u * V);
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k) {
          if (h + k * hstep < p.heads) {
            float v[V];
            unpack_vec<T, V>(q[k], v);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              if (j0 + i < p.pairs) {  // dims past the pairs stay as they are
                const float a0 = v[2 * i], c0 = v[2 * i + 1];
                v[2 * i] = a0 * cs[i].x - c0 * cs[i].y;
                v[2 * i + 1] = a0 * cs[i].y + c0 * cs[i].x;
              }
            }
            store_vec<T, V>(ot + (h + k * hstep) * p.os_h + u * V, v);
          }
        }
      }
    }
  }
}

template <typename T, int V>
static cudaError_t launch_rope_v(RopeParams& p, bool half, cudaStream_t s) {
  p.units = half ? p.pairs / V + (p.dim - 2 * p.pairs) / V : (V == 1 ? (p.dim + 1) / 2 : p.dim / V);
  const int slots = p.units >= kRopeThreads ? 1 : kRopeThreads / p.units;
  const int threads = (p.units * slots + 31) / 32 * 32;
  // a CTA takes several tokens once there are enough of them to fill the GPU
  // (the table is then made once, by all threads); with few tokens the heads
  // are split over CTAs instead
  const int64_t total = p.batch * p.tokens, want = (int64_t)device_sm_count() * 8;
  int tpc = (int)(total / want);
  tpc = tpc < 1 ? 1 : tpc > 8 ? 8 : tpc;
  p.tok_per_cta = tpc;
  const int64_t gx = p.batch * ((p.tokens + tpc - 1) / tpc);
  int64_t gy = total >= want ? 1 : (want + total - 1) / total;
  const int64_t hchunks = (p.heads + slots - 1) / slots;
  if (gy > hchunks) gy = hchunks;
  if (gx > 0x7FFFFFFF || gy > 65535) return cudaErrorInvalidValue;
  const size_t smem = (size_t)tpc * p.pairs * sizeof(float2);
  return half ? launch_pdl(rope_axes_kernel<T, V, true>, dim3((unsigned)gx, (unsigned)gy), dim3(threads), smem, s, p)
              : launch_pdl(rope_axes_kernel<T, V, false>, dim3((unsigned)gx, (unsigned)gy), dim3(threads), smem, s, p);
}

template <typename T>
static cudaError_t launch_rope(RopeParams& p, bool half, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int64_t str[6] = {p.xs_b, p.xs_t, p.xs_h, p.os_b, p.os_t, p.os_h};
  bool vec = ((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out)) & 15) == 0 && p.dim % V == 0;
  for (int64_t st : str) vec = vec && st % V == 0;
  if (half) vec = vec && p.pairs % V == 0;
  return vec ? launch_rope_v<T, V>(p, half, s) : launch_rope_v<T, 1>(p, half, s);
}

}  // namespace kl

extern "C" kl_status kl_rope_axes(const kl_rope_args* r, void* stream) {
  using namespace kl;
  if (!r || !r->x || !r->out || !r->pos) return KL_ERR_INVALID_ARG;
  if (r->dtype != KL_BF16 && r->dtype != KL_F32 && r->dtype != KL_F16) return KL_ERR_INVALID_ARG;
  if (r->pos_type < KL_POS_I32 || r->pos_type > KL_POS_F32) return KL_ERR_INVALID_ARG;
  if (r->flags & ~(KL_ROPE_HALF | KL_ROPE_LADDER_SHARED | KL_ROPE_INVERSE)) return KL_ERR_INVALID_ARG;
  if (!(r->theta > 1.0) || !(r->theta <= 1e30)) return KL_ERR_INVALID_ARG;
  if (r->naxes < 1 || r->naxes > KL_ROPE_MAX_AXES) return KL_ERR_UNSUPPORTED_SHAPE;
  RopeParams p{};
  int64_t pairs = 0;
  for (int a = 0; a < r->naxes; ++a) {
    if (r->sections[a] < 0 || r->sections[a] > kRopeMaxPairs) return KL_ERR_UNSUPPORTED_SHAPE;
    p.first[a] = (int)pairs;
    pairs += r->sections[a];
  }
  for (int a = r->naxes; a <= KL_ROPE_MAX_AXES; ++a) p.first[a] = (int)pairs;
  if (r->batch < 1 || r->tokens < 1 || r->heads < 1 || r->dim < 1 || r->dim > 2 * kRopeMaxPairs || pairs < 1 ||
      2 * pairs > r->dim)
    return KL_ERR_UNSUPPORTED_SHAPE;
  const int64_t lim = (int64_t)1 << 31;
  if (r->batch >= lim || r->tokens >= lim || r->heads >= lim || r->batch > lim / r->tokens)
    return KL_ERR_UNSUPPORTED_SHAPE;
  const int es = r->dtype == KL_F32 ? 4 : 2;
  if (!aligned(r->x, es) || !aligned(r->out, es) || !aligned(r->pos, r->pos_type == KL_POS_I64 ? 8 : 4))
    return KL_ERR_MISALIGNED;
  kl_status st = check_arch();
  if (st != KL_OK) return st;
  p.x = r->x;
  p.out = r->out;
  p.pos = r->pos;
  p.batch = r->batch;
  p.tokens = r->tokens;
  p.heads = r->heads;
  p.xs_b = r->x_stride[0];
  p.xs_t = r->x_stride[1];
  p.xs_h = r->x_stride[2];
  p.os_b = r->out_stride[0];
  p.os_t = r->out_stride[1];
  p.os_h = r->out_stride[2];
  p.pos_b = r->pos_shared ? 0 : r->tokens;
  p.dim = (int)r->dim;
  p.pairs = (int)pairs;
  p.naxes = r->naxes;
  p.pos_type = r->pos_type;
  p.sign = (r->flags & KL_ROPE_INVERSE) ? -1.f : 1.f;
  // ladders as running products in extended precision: their error stays far
  // below the one rounding to fp64
  const long double inv_pi = 0.318309886183790671537767526745028724L;
  for (int a = 0; a < r->naxes; ++a) {
    const int n = (int)r->sections[a];
    if (n == 0) continue;
    const bool shared = r->flags & KL_ROPE_LADDER_SHARED;
    const long double step = powl((long double)r->theta, -1.0L / (shared ? (long double)pairs : (long double)n));
    long double f = shared && a > 0 ? powl((long double)r->theta, -(long double)p.first[a] / (long double)pairs) : 1.0L;
    for (int u = 0; u < n; ++u, f *= step) p.freq[p.first[a] + u] = (double)(f * inv_pi);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool half = r->flags & KL_ROPE_HALF;
  const cudaError_t e = r->dtype == KL_BF16  ? launch_rope<__nv_bfloat16>(p, half, s)
                        : r->dtype == KL_F16 ? launch_rope<__half>(p, half, s)
                                             : launch_rope<float>(p, half, s);
  return e == cudaSuccess ? KL_OK : cuda_fail(e);
}
