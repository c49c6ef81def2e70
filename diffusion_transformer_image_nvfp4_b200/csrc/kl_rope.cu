// kl_rope.cu -- rotary positions with several axes (time, height, width, ...)
// applied to [batch, token, head, dim] tensors, and the inverse rotation,
// which is also the gradient (a rotation's transpose).
//
// Pair j of a head turns by pos[token, axis(j)] * f_j: the pairs are divided
// among the axes in order (`sections`), f_j = theta^(-u / n_a) with u the
// pair's index in its axis' section of n_a pairs, or theta^(-j / P) over all
// P pairs (KL_ROPE_LADDER_SHARED).  Dims past the pairs are copied.
//
// Angles: f_j / pi is made on the host in extended precision and rounded to
// fp64; position times it is one fp64 product, reduced by whole turns exactly
// (h - 2 rint(h / 2)).  An angle is off by at most 3 * 2^-53 of the position
// (3.5e-10 at 2^20, 3.7e-4 at 2^40), and int64 positions past 2^53 are rounded
// to fp64 first; sincospif of the reduced angle is fp32.  Each angle is used by every head of its token: a CTA makes the
// table of a few tokens in shared memory, then its threads walk the (token,
// head) rows, the next rows' loads ahead of this row's work.  CTAs stay for a
// few chunks of tokens; two table buffers leave one barrier a chunk.
//
// Bound by HBM: one read and one write of the tensor; the fp64 work is one
// angle per (token, pair), a head's share of it 1 / H.  B200, device time, bf16,
// 48 heads of 128: 4,608 tokens 22.2 us (78% of the copy's rate), 20,992 87.8
// (89%); fp32, 2 x 3,315 x 6 heads of 96 7.3.
#include <cmath>
#include <utility>

#include "../../include/klein.h"
#include "kl_common.cuh"
#include "kl_internal.h"

namespace kl {

constexpr int kRopeMaxPairs = 256;  // head dim 512
constexpr int kRopeThreads = 256;
// rows a thread loads, ahead of as many that it turns and stores
__host__ __device__ constexpr int rope_batch(int bytes, bool half) { return half && bytes >= 16 ? 2 : 4; }
// CTAs of a SM: with 16-byte vectors the fourth spills (4,608 x 48 heads, bf16,
// inputs from HBM: 20.9 us with three, 22.9 with four; 100 dims: 32.7 and 28.4)
__host__ __device__ constexpr int rope_ctas(int bytes) { return bytes >= 16 ? 3 : 4; }
constexpr int kRopeTable = 2560;    // (token, pair) entries of a table buffer: two are 40 KB

struct RopeParams {
  const void* x;
  void* out;
  const void* pos;
  int64_t batch, tokens;
  int64_t xs_b, xs_t, xs_h, os_b, os_t, os_h;  // strides in elements; dims are consecutive
  int64_t pos_b;                               // position rows between batches (0: shared)
  unsigned chunks;                             // token chunks of a batch
  unsigned items;                              // batch * chunks * head parts
  int heads, hparts, hper;                     // a chunk's heads are in hparts parts of hper
  int dim, pairs, naxes, pos_type;
  int units;            // per head: vectors of dims (interleaved) or of pairs, then of copied dims (half)
  int nt;               // tokens of a chunk
  float sign;           // -1: inverse
  int first[KL_ROPE_MAX_AXES + 1];  // first pair of each axis
  double freq[kRopeMaxPairs];       // f_j / pi
};

__device__ __forceinline__ double rope_pos(const RopeParams& p, int64_t i) {
  if (p.pos_type == KL_POS_I32) return (double)reinterpret_cast<const int32_t*>(p.pos)[i];
  if (p.pos_type == KL_POS_I64) return (double)reinterpret_cast<const int64_t*>(p.pos)[i];
  return (double)reinterpret_cast<const float*>(p.pos)[i];
}

// one unit of one row: loaded, turned by the row's table entries, stored
template <typename T, int V, bool HALF>
struct RopeUnit {
  static constexpr int NP = HALF ? V : (V == 1 ? 1 : V / 2);  // pairs
  uint4 a, c;  // c: the second halves, or the second element
  __device__ __forceinline__ void load(const T* x, const RopeParams& p, int u, int pair_units) {
    if constexpr (HALF) {
      if (u < pair_units) {
        a = load_vec<T, V>(x + u * V);
        c = load_vec<T, V>(x + p.pairs + u * V);
      } else {
        a = load_vec<T, V>(x + 2 * p.pairs + (u - pair_units) * V);
      }
    } else if constexpr (V == 1) {
      a = load_vec<T, 1>(x + 2 * u);
      if (2 * u + 1 < p.dim) c = load_vec<T, 1>(x + 2 * u + 1);
    } else {
      a = load_vec<T, V>(x + u * V);
    }
  }
  // whole: all its dims turn, by t; else cs is the table's row from the unit's first pair
  __device__ __forceinline__ void store(T* o, const RopeParams& p, int u, int pair_units, bool whole,
                                        const float2 (&t)[NP], const float2* cs) {
    if constexpr (HALF || V == 1) {
      if (whole) {
        float va[V], vc[V];
        unpack_vec<T, V>(a, va);
        unpack_vec<T, V>(c, vc);
#pragma unroll
        for (int i = 0; i < V; ++i) turn(va[i], vc[i], t[i]);
        if constexpr (HALF) {
          store_vec<T, V>(o + u * V, va);
          store_vec<T, V>(o + p.pairs + u * V, vc);
        } else {
          o[2 * u] = from_f32<T>(va[0]);
          o[2 * u + 1] = from_f32<T>(vc[0]);
        }
      } else if constexpr (HALF) {
        put(o + 2 * p.pairs + (u - pair_units) * V, a);
      } else {
        put(o + 2 * u, a);
        if (2 * u + 1 < p.dim) put(o + 2 * u + 1, c);
      }
    } else {
      float v[V];
      unpack_vec<T, V>(a, v);
      if (whole) {
#pragma unroll
        for (int i = 0; i < NP; ++i) turn(v[2 * i], v[2 * i + 1], t[i]);
      } else {
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (u * NP + i < p.pairs) turn(v[2 * i], v[2 * i + 1], cs[i]);  // dims past the pairs stay as they are
      }
      store_vec<T, V>(o + u * V, v);
    }
  }
  static __device__ __forceinline__ void turn(float& x0, float& x1, const float2& cs) {
    const float y = x0 * cs.x - x1 * cs.y;
    x1 = x0 * cs.y + x1 * cs.x;
    x0 = y;
  }
  static __device__ __forceinline__ void entries(const float2* cs, float2 (&t)[NP]) {
    if constexpr (NP == 1) {
      t[0] = cs[0];
    } else {  // table rows and units start on an even entry
#pragma unroll
      for (int i = 0; i < NP; i += 2) {
        const float4 f = *reinterpret_cast<const float4*>(cs + i);
        t[i] = make_float2(f.x, f.y);
        t[i + 1] = make_float2(f.z, f.w);
      }
    }
  }
  // the loaded bits themselves
  static __device__ __forceinline__ void put(T* o, const uint4& q) {
    if constexpr (V * sizeof(T) == 16)
      *reinterpret_cast<uint4*>(o) = q;
    else if constexpr (V * sizeof(T) == 8)
      *reinterpret_cast<uint2*>(o) = make_uint2(q.x, q.y);
    else if constexpr (V * sizeof(T) == 4)
      *reinterpret_cast<uint32_t*>(o) = q.x;
    else
      *reinterpret_cast<uint16_t*>(o) = (uint16_t)q.x;
  }
};

// V elements a thread at a time (16 bytes, two elements, or V = 1 for what is
// not aligned; interleaved pairs then move two elements).  A thread keeps one unit u of the
// head and walks the rows.
// HEADS: a token's heads are more than the slots, so a thread's rows of a token
// are `slots` heads apart and share its table entries; else several tokens'
// heads are spread over the slots, and a thread's rows are one head of tokens
// `tpar` apart.  Either way a batch of rows lies at one stride.
template <typename T, int V, bool HALF, bool HEADS>
__global__ void __launch_bounds__(kRopeThreads, rope_ctas(V * (int)sizeof(T))) rope_axes_kernel(const __grid_constant__ RopeParams p) {
  constexpr int B = rope_batch(V * (int)sizeof(T), HALF);
  using Unit = RopeUnit<T, V, HALF>;
  extern __shared__ __align__(16) float2 rope_tables[];  // [2][nt][pairs, even] (cos, sin)
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  // this thread's pair of the table, its frequency and axis
  const int tslots = kRopeThreads / p.pairs, tj = tid % p.pairs, ts = tid / p.pairs;
  const double freq = p.freq[tj];
  int axis = 0;
  while (tj >= p.first[axis + 1]) ++axis;
  const int ulim = min(p.units, kRopeThreads), slots = kRopeThreads / ulim;
  const int u0 = tid % ulim, slot = tid / ulim;
  const int pair_units = p.pairs / Unit::NP, pitch = (p.pairs + 1) & ~1;
  int buf = 0;
  for (unsigned item = blockIdx.x; item < p.items; item += gridDim.x, buf ^= 1) {
    const unsigned bc = p.hparts == 1 ? item : item / (unsigned)p.hparts, b = p.batch == 1 ? 0u : bc / p.chunks;
    const int64_t t0 = (int64_t)(bc - b * p.chunks) * p.nt;
    const int h0 = (int)(item - bc * p.hparts) * p.hper, nh = min(p.hper, p.heads - h0);
    const int nt = (int)min((int64_t)p.nt, p.tokens - t0);
    float2* table = rope_tables + buf * p.nt * pitch;
    const int tpar = HEADS ? 1 : slots / nh;  // tokens side by side
    const int h = HEADS ? slot : slot % nh, tp = HEADS ? 0 : slot / nh;
    const bool live = slot < slots && tp < tpar;
    // rows of a run (a token's heads, or all tokens), and what one is from the next
    const int run = !live ? 0 : HEADS ? (nh - h + slots - 1) / slots : (nt - tp + tpar - 1) / tpar;
    const int64_t xk = HEADS ? slots * p.xs_h : tpar * p.xs_t, ok = HEADS ? slots * p.os_h : tpar * p.os_t;
    const int ck = HEADS ? 0 : tpar * pitch;
    const T* x0 = reinterpret_cast<const T*>(p.x) + b * p.xs_b + (t0 + tp) * p.xs_t + (h0 + h) * p.xs_h;
    T* o0 = reinterpret_cast<T*>(p.out) + b * p.os_b + (t0 + tp) * p.os_t + (h0 + h) * p.os_h;
    struct Batch {
      const T* x;
      T* o;
      const float2* cs;
      int left, t;  // rows left in the run, the run
    } next;
    const int runs = HEADS ? nt : 1;
    Unit qn[B];
    int u = u0;
    auto start = [&] { next = Batch{x0, o0, table + tp * pitch + u * Unit::NP, run, run > 0 ? 0 : runs}; };
    auto fetch = [&] {
      const T* x = next.x;
#pragma unroll
      for (int k = 0; k < B; ++k, x += xk)
        if (k < next.left) qn[k].load(x, p, u, pair_units);
    };
    auto advance = [&] {
      next.left -= B;
      if (next.left > 0) {
        next.x += B * xk;
        next.o += B * ok;
        next.cs += B * ck;
      } else {
        ++next.t;
        if constexpr (HEADS) {
          next.left = run;
          next.x = x0 + next.t * p.xs_t;
          next.o = o0 + next.t * p.os_t;
          next.cs += pitch;
        }
      }
    };
    start();
    if (next.t < runs) fetch();  // under way while the table is made
    if (ts < tslots) {
      for (int t = ts; t < nt; t += tslots) {
        const double a = rope_pos(p, (b * p.pos_b + t0 + t) * p.naxes + axis) * freq;
        float sn, c;
        sincospif((float)(a - 2.0 * rint(0.5 * a)), &sn, &c);
        table[t * pitch + tj] = make_float2(c, p.sign * sn);
      }
    }
    __syncthreads();
    while (true) {
      const bool whole = u < pair_units;
#pragma unroll 2
      while (next.t < runs) {
        Unit q[B];
#pragma unroll
        for (int k = 0; k < B; ++k) q[k] = qn[k];
        const Batch cur = next;
        // x and out may be the same tensor: the compiler cannot move these
        // loads above the stores itself
        advance();
        if (next.t < runs) fetch();
        float2 e[Unit::NP];
        if (HEADS && whole) Unit::entries(cur.cs, e);
        T* o = cur.o;
        const float2* cs = cur.cs;
#pragma unroll
        for (int k = 0; k < B; ++k, o += ok, cs += ck) {
          if (k < cur.left) {
            if (!HEADS && whole) Unit::entries(cs, e);
            q[k].store(o, p, u, pair_units, whole, e, cs);
          }
        }
      }
      if ((u += kRopeThreads) >= p.units) break;
      // (heads of more than 256 units, which single elements can have: again from the first row)
      start();
      if (next.t < runs) fetch();
    }
  }
}

template <typename T, int V>
static cudaError_t launch_rope_v(RopeParams& p, bool half, cudaStream_t s) {
  p.units = half ? p.pairs / V + (p.dim - 2 * p.pairs) / V : (V == 1 ? (p.dim + 1) / 2 : p.dim / V);
  // Three or four CTAs a SM, each of one or a few chunks of tokens within the table:
  // the chunk that leaves the most loaded CTA the fewest tokens.  Fewer tokens
  // than CTAs: one each, and parts of the heads.
  const int64_t want = (int64_t)device_sm_count() * rope_ctas(V * (int)sizeof(T));
  const int64_t most = kRopeTable / (p.pairs + 1);
  const int64_t chunks_min = p.batch * ((p.tokens + most - 1) / most), rounds0 = (chunks_min + want - 1) / want;
  int64_t nt = 0, least = 0;
  for (int64_t rounds = rounds0; rounds < rounds0 + 8; ++rounds) {  // chunks of a CTA
    int64_t chunks = rounds * want / p.batch;                       // of a batch
    if (chunks < 1) chunks = 1;
    const int64_t c = (p.tokens + chunks - 1) / chunks;
    if (c <= most && (nt == 0 || rounds * c < least)) {
      nt = c;
      least = rounds * c;
    }
  }
  if (nt == 0) nt = most < p.tokens ? most : p.tokens;
  p.nt = (int)nt;
  p.chunks = (unsigned)((p.tokens + nt - 1) / nt);
  const int ulim = p.units < kRopeThreads ? p.units : kRopeThreads, slots = kRopeThreads / ulim;
  int64_t parts = want / (p.batch * p.chunks);
  const int64_t hchunks = (p.heads + slots - 1) / slots;  // no part without a row for every slot
  if (parts > hchunks) parts = hchunks;
  if (parts < 1) parts = 1;
  p.hper = (int)((p.heads + parts - 1) / parts);
  p.hparts = (p.heads + p.hper - 1) / p.hper;
  p.items = (unsigned)(p.batch * p.chunks * p.hparts);
  const unsigned grid = p.items < (unsigned)want ? p.items : (unsigned)want;
  const size_t smem = (size_t)2 * nt * ((p.pairs + 1) & ~1) * sizeof(float2);
  auto kern = p.hper >= slots ? (half ? rope_axes_kernel<T, V, true, true> : rope_axes_kernel<T, V, false, true>)
                              : (half ? rope_axes_kernel<T, V, true, false> : rope_axes_kernel<T, V, false, false>);
  return launch_pdl(kern, dim3(grid), dim3(kRopeThreads), smem, s, p);
}

template <typename T>
static cudaError_t launch_rope(RopeParams& p, bool half, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int64_t str[6] = {p.xs_b, p.xs_t, p.xs_h, p.os_b, p.os_t, p.os_h};
  auto fits = [&](int v) {  // every vector of v dims lies on its own size
    bool ok = ((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out)) % (v * sizeof(T))) == 0 &&
              p.dim % v == 0 && (!half || p.pairs % v == 0);
    for (int64_t st : str) ok = ok && st % v == 0;
    return ok;
  };
  // 3 x 4600 x 20 heads of 100 dims, bf16, in place of single elements: 28.4 us for
  // 47.7 interleaved, 34.4 for 57.4 half
  if (fits(V)) return launch_rope_v<T, V>(p, half, s);
  return fits(2) ? launch_rope_v<T, 2>(p, half, s) : launch_rope_v<T, 1>(p, half, s);
}

// Two of the size[0] x size[1] x size[2] heads of `dim` elements share one.
// Strides that nest (each at least what the smaller ones span) cannot; others
// are searched: over the differences of two of the indices, the third's is the
// quotient.  Past kSearch differences (a millisecond) the answer is yes.
static bool rope_heads_overlap(const int64_t (&size)[3], const int64_t (&stride)[3], int64_t dim) {
  using wide = __int128;
  constexpr wide kSearch = 1 << 16;
  int64_t n[3], st[3];
  int m = 0;
  for (int i = 0; i < 3; ++i) {
    if (size[i] == 1) continue;
    n[m] = size[i] - 1;  // the largest difference of two indices
    if (stride[i] == INT64_MIN) return true;
    st[m++] = stride[i] < 0 ? -stride[i] : stride[i];
  }
  for (int i = 1; i < m; ++i)  // by stride
    for (int j = i; j > 0 && st[j] < st[j - 1]; --j) {
      std::swap(st[j], st[j - 1]);
      std::swap(n[j], n[j - 1]);
    }
  wide span = dim;
  bool nested = true;
  for (int i = 0; i < m; ++i) {
    nested = nested && st[i] >= span;
    span += (wide)n[i] * st[i];
  }
  if (nested) return false;
  if (m == 1) return true;  // a stride below dim
  for (int i = 0; i < m; ++i)
    if (st[i] < dim) return true;
  int k = 0;  // the index solved for: the longest
  for (int i = 1; i < m; ++i)
    if (n[i] > n[k]) k = i;
  const int a = k == 0 ? 1 : 0, b = m == 3 ? 3 - k - a : -1;
  const int64_t nb = b >= 0 ? n[b] : 0, sb = b >= 0 ? st[b] : 0;
  if (((wide)n[a] + 1) * (2 * (wide)nb + 1) > kSearch) return true;
  for (int64_t i = 0; i <= n[a]; ++i)
    for (int64_t j = i == 0 ? 1 : -nb; j <= nb; ++j) {
      // a multiple q st[k], |q| <= n[k], within dim of this difference's opposite
      const wide at = (wide)i * st[a] + (wide)j * sb, mag = at < 0 ? -at : at;
      wide q = (mag + dim - 1) / st[k];  // the largest with q st[k] < mag + dim
      if (q > n[k]) q = n[k];
      if (q * st[k] > mag - dim) return true;
    }
  return false;
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
  if (r->batch >= lim || r->tokens >= lim || r->heads >= lim / 2 || r->batch > lim / r->tokens)
    return KL_ERR_UNSUPPORTED_SHAPE;
  // no output element twice; in place only element by element
  const int64_t size[3] = {r->batch, r->tokens, r->heads};
  if (rope_heads_overlap(size, r->out_stride, r->dim)) return KL_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (size[i] > 1 && r->x == r->out && r->x_stride[i] != r->out_stride[i]) return KL_ERR_INVALID_ARG;
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
  p.heads = (int)r->heads;
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
