// kl_fp8.cu -- FP8 (E4M3) encode with one power-of-two scale per block of 128.
//
// A block is 128 consecutive columns of one row or a 128 x 128
// tile (KL_FP8_TILE), of x or of its transpose.  Its scale is 2^e, e the
// least integer with amax <= 448 * 2^e, in [-127, 127] (0 if amax = 0), held
// as the E8M0 byte e + 127; a code is the E4M3 value nearest to x * 2^-e.
// Multiplying by a power of two is exact (a product below the fp32 normal
// range rounds, but E4M3's least step there is 2^-9 * 2^e, so its code is 0
// either way): the code has one rounding.  E4M3 floats, so against a scale
// amax / 448 the power of two costs at most one binade at the low end and no
// relative precision; in return the tensor cores apply it themselves.
//
// Bound by HBM (one read of x, one byte written per element).  Row blocks:
// a lane holds 16 columns, eight lanes a block, a warp four blocks -- the
// four scale bytes of one 32-bit word of the MMA scale layout -- so the amax
// is three shuffles and nothing goes through shared memory.  Tiles and
// transposes hold 128 rows of x in registers too: a thread of a transpose
// reads column pairs of 16 rows and writes 16 contiguous bytes of x^T.
// B200, device time: rows of bf16 4,608 x 9,216 21.2 us, 20,992 x 3,072 30.8 (91 and
// 96% of the copy's rate); tiles 20.4 and 29.7 (95 and 99%); transposed rows 30
// and 44 (64 and 67%; fp32 98%), where under the profiler neither DRAM (38%), L1
// (66%) nor issue (53% of the slots) is full: a CTA loads, waits for its columns'
// amax and converts in turn, and 43% of the warps are there to hide it; bf16 rows
// that no vector load suits, 20,000 x 2,001, 26.7 (52 with single-element loads).

#include <type_traits>

#include "../../include/klein.h"
#include "kl_common.cuh"
#include "kl_internal.h"

namespace kl {

constexpr uint32_t kF32Inf = 0x7F800000u;

// exponent byte and 2^-e of a block from the bits of its amax; a block with a
// NaN or an infinity (bits >= kF32Inf) gets the byte 255, E8M0's NaN
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= kF32Inf) return 255u;
  if (amax_bits == 0u) return 127u;
  // 448 = 1.75 * 2^8: e = exponent - 8, one more where the mantissa passes 1.75
  const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(max(e, -127) + 127);
}
// 2^(127 - byte); byte <= 247 for finite blocks, so the result is normal
__device__ __forceinline__ float fp8_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// what a block's values are multiplied by: 2^(127 - byte), or NaN
__device__ __forceinline__ uint64_t fp8_inv2(uint32_t byte) {
  const float inv = byte == 255u ? __uint_as_float(0x7FC00000u) : fp8_inv_scale(byte);
  return pack_f32x2(inv, inv);
}
// four values -> four E4M3 bytes
__device__ __forceinline__ uint32_t fp8_codes4(float a, float b, float c, float d, uint64_t inv2) {
  unpack_f32x2(mul_f32x2(pack_f32x2(a, b), inv2), a, b);
  unpack_f32x2(mul_f32x2(pack_f32x2(c, d), inv2), c, d);
  return f32x2_to_e4m3x2(a, b) | (f32x2_to_e4m3x2(c, d) << 16);
}
// 16 codes, of which n >= 16 or the first n exist (the others are 0)
__device__ __forceinline__ uint4 fp8_codes16(const float (&v)[16], uint64_t inv2, int n) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = fp8_codes4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], inv2);
  if (n < 16) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n < 4 * j + 4) w[j] = n <= 4 * j ? 0u : w[j] & ((1u << (8 * (n - 4 * j))) - 1u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// byte offset of (row, block) in the MMA scale layout
__device__ __forceinline__ int64_t fp8_mma_offset(int64_t row, int64_t blk, int64_t atoms_k) {
  return ((row >> 7) * atoms_k + (blk >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (blk & 3);
}

// 16 consecutive elements of a row as stored; those past n are 0
template <typename T>
struct Fp8Raw {
  uint4 q[sizeof(T)];
  // lo, hi: the matrix' first byte and the one after its last
  template <bool VEC>
  __device__ __forceinline__ void load(const T* p, int n, const uint8_t* lo, const uint8_t* hi) {
    constexpr int S = (int)sizeof(T);
    const uint8_t* base = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
    if (VEC && n >= 16) {
#pragma unroll
      for (int i = 0; i < S; ++i) q[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    } else if (!VEC && n >= 16 && base >= lo && base + 16 * (S + 1) <= hi) {
      // the aligned vectors around them, shifted into place word by word and,
      // for 16-bit elements, by half a word
      const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
      uint32_t w[4 * (S + 1)];
#pragma unroll
      for (int i = 0; i <= S; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(base) + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
      if (off & 8) {
#pragma unroll
        for (int i = 0; i < 4 * S + 2; ++i) w[i] = w[i + 2];
      }
      if (off & 4) {
#pragma unroll
        for (int i = 0; i < 4 * S + 1; ++i) w[i] = w[i + 1];
      }
      if constexpr (S == 2) {
#pragma unroll
        for (int i = 0; i < 4 * S; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (off & 2) * 8);
      }
#pragma unroll
      for (int i = 0; i < S; ++i) q[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
      uint32_t w[4 * sizeof(T)];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if constexpr (sizeof(T) == 4) {
          w[i] = i < n ? __ldg(reinterpret_cast<const uint32_t*>(p) + i) : 0u;
        } else {
          const uint32_t u = i < n ? __ldg(reinterpret_cast<const uint16_t*>(p) + i) : 0u;
          w[i / 2] = (i & 1) ? w[i / 2] | (u << 16) : u;
        }
      }
#pragma unroll
      for (int i = 0; i < (int)sizeof(T); ++i) q[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
  // bits of the largest magnitude as fp32 (magnitudes are in the order of their
  // bits, NaN above infinity; 16-bit ones two at a time)
  __device__ __forceinline__ uint32_t amax_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) {
      const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) m = sizeof(T) == 4 ? max(m, w[k] & 0x7FFFFFFFu) : __vmaxu2(m, w[k] & 0x7FFF7FFFu);
    }
    if constexpr (sizeof(T) == 2) {
      float lo, hi;
      m = max(m & 0xFFFFu, m >> 16);
      unpack2<T>(m, lo, hi);
      m = __float_as_uint(lo);
    }
    return m;
  }
  __device__ __forceinline__ void values(float (&v)[16]) const {
    constexpr int V = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) unpack_vec<T, V>(q[i], *reinterpret_cast<float(*)[V]>(&v[i * V]));
  }
};

struct Fp8EncodeParams {
  const void* x;
  int64_t rows, cols, ldx;  // of x as given
  uint8_t* codes;
  int64_t ldc;
  uint8_t* scales;
  int mma, tile, transpose;
};

// Row blocks.  A warp takes up to `seg` words (a word: the four blocks of 512
// columns) of one row; with the MMA layout also the padding rows up to a
// multiple of 128, whose words it zeroes.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) fp8_encode_rows_kernel(const Fp8EncodeParams p, int64_t tasks, uint64_t rcp_nseg,
                                                              int nseg, int seg, int words) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = (int64_t)gridDim.x * 8;
  const int cols = (int)p.cols, nblk = (cols - 1) / 128 + 1;
  const uint8_t* lo = reinterpret_cast<const uint8_t*>(p.x);
  const uint8_t* hi = lo + ((p.rows - 1) * p.ldx + p.cols) * sizeof(T);
  bool bad = false;
  for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < tasks; it += nwarps) {
    const int64_t row = div_rcp(it, rcp_nseg);
    const int k0 = (int)(it - row * nseg) * seg, k1 = min(k0 + seg, words);
    int c = k0 * 512 + lane * 16;
    // scale byte of this lane's block: MMA 512 bytes a word, linear 4
    uint8_t* sc = p.mma ? p.scales + fp8_mma_offset(row, (int64_t)k0 * 4 + (lane >> 3), words)
                        : p.scales + row * nblk + k0 * 4 + (lane >> 3);
    if (row >= p.rows) {
      for (int k = k0; k < k1; ++k, sc += 512)
        if ((lane & 7) == 0) *sc = 0;
      continue;
    }
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx + c;
    uint8_t* out = p.codes + row * p.ldc + c;
    const int sstep = p.mma ? 512 : 4;
    // scale byte of a lane's block from its part of the block's amax
    auto scale = [&](const Fp8Raw<T>& raw) {
      uint32_t m = raw.amax_bits();
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint32_t byte = fp8_scale_byte(m);
      bad |= byte == 255u;
      return byte;
    };
    int k = k0;
    if (VEC) {  // words without an end, two at a time
      const int kf = min(k1, cols >> 9);
      for (; k + 1 < kf; k += 2) {
        Fp8Raw<T> raw[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) raw[i].template load<true>(x + i * 512, 16, lo, hi);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t byte = scale(raw[i]);
          float v[16];
          raw[i].values(v);
          *reinterpret_cast<uint4*>(out + i * 512) = fp8_codes16(v, fp8_inv2(byte), 16);
          if ((lane & 7) == 0) sc[i * sstep] = (uint8_t)byte;
        }
        x += 1024;
        out += 1024;
        sc += 2 * sstep;
        c += 1024;
      }
    }
    for (; k < k1; ++k) {
      const int n = cols - c;
      Fp8Raw<T> raw;
      raw.template load<VEC>(x, n, lo, hi);
      const uint32_t byte = scale(raw);
      float v[16];
      raw.values(v);
      if (n > 0) *reinterpret_cast<uint4*>(out) = fp8_codes16(v, fp8_inv2(byte), n);
      if ((lane & 7) == 0) {
        if (k * 4 + (lane >> 3) < nblk)
          *sc = (uint8_t)byte;
        else if (p.mma)
          *sc = 0;
      }
      x += 512;
      out += 512;
      sc += sstep;
      c += 512;
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(KL_DEVERR_NONFINITE);
}

// x^T: 128 rows x 2 PAIRS columns of x a CTA.  A thread reads two columns of
// 16 rows and writes 16 bytes of both columns' rows of x^T; the amax of a
// column, or of the whole tile, goes through shared memory.
template <typename T, bool VEC, int PAIRS, bool TILE>
__global__ void __launch_bounds__(8 * PAIRS) fp8_encode_columns_kernel(const Fp8EncodeParams p, int tiles_c) {
  static_assert(!TILE || PAIRS == 64, "a tile is 128 columns");
  __shared__ uint32_t colmax[TILE ? 1 : 8][2 * PAIRS];
  pdl_wait();
  pdl_trigger();
  // a warp: LP pairs of 16 * 32 / LP rows, so both its reads and its writes are whole sectors
  constexpr int LP = sizeof(T) == 2 ? 16 : 8, WP = PAIRS / LP;
  const int tid = threadIdx.x, lane = tid & 31;
  const int pair = lane % LP + tid / 32 % WP * LP, q = lane / LP + tid / (32 * WP) * (32 / LP);
  const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int64_t r0 = tr * 128 + q * 16, c0 = tc * (2 * PAIRS) + 2 * pair;
  const int nr = (int)max((int64_t)0, min((int64_t)16, p.rows - r0));
  const bool ca = c0 < p.cols, cb = c0 + 1 < p.cols;
  const T* x = reinterpret_cast<const T*>(p.x) + r0 * p.ldx + c0;
  float a[16], b[16];
  uint32_t ma = 0, mb = 0;
  if (VEC && cb && nr == 16) {  // (every load before the first use)
    using W = std::conditional_t<sizeof(T) == 2, uint32_t, float2>;
    W w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __ldg(reinterpret_cast<const W*>(x + i * p.ldx));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (sizeof(T) == 2) {
        unpack2<T>(w[i], a[i], b[i]);
      } else {
        a[i] = w[i].x;
        b[i] = w[i].y;
      }
    }
  } else {
    T w[16], v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      w[i] = i < nr && ca ? x[i * p.ldx] : from_f32<T>(0.f);
      v[i] = i < nr && cb ? x[i * p.ldx + 1] : from_f32<T>(0.f);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      a[i] = to_f32(w[i]);
      b[i] = to_f32(v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    ma = max(ma, __float_as_uint(a[i]) & 0x7FFFFFFFu);
    mb = max(mb, __float_as_uint(b[i]) & 0x7FFFFFFFu);
  }
  if constexpr (TILE) {
    ma = __reduce_max_sync(0xffffffffu, max(ma, mb));
    if ((tid & 31) == 0) colmax[0][tid >> 5] = ma;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PAIRS / 4; ++i) ma = max(ma, colmax[0][i]);
    mb = ma;
  } else {
    *reinterpret_cast<uint2*>(&colmax[q][2 * pair]) = make_uint2(ma, mb);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint2 m = *reinterpret_cast<const uint2*>(&colmax[i][2 * pair]);
      ma = max(ma, m.x);
      mb = max(mb, m.y);
    }
  }
  const uint32_t sa = fp8_scale_byte(ma), sb = fp8_scale_byte(mb);
  if (nr > 0) {  // at most 15 columns past the last row
    uint8_t* out = p.codes + c0 * p.ldc + r0;
    if (ca) *reinterpret_cast<uint4*>(out) = fp8_codes16(a, fp8_inv2(sa), nr);
    if (cb) *reinterpret_cast<uint4*>(out + p.ldc) = fp8_codes16(b, fp8_inv2(sb), nr);
  }
  // scale bytes of this block of x^T's rows, by the first rows' threads; the last
  // block of a row zeroes the unused bytes of its word, the last columns' CTA
  // the rows up to a multiple of 128
  const int64_t nblk = (p.rows + 127) >> 7;
  if (p.mma) {
    const int64_t atoms_k = (nblk + 3) >> 2;
    auto put = [&](int64_t row, uint32_t byte) {
      uint8_t* dst = p.scales + fp8_mma_offset(row, tr, atoms_k);
      dst[0] = (uint8_t)byte;
      if (tr == nblk - 1)
        for (int64_t k = 1; ((tr + k) & 3) != 0; ++k) dst[k] = 0;
    };
    if (q == 0) {
      put(c0, ca ? sa : 0u);
      put(c0 + 1, cb ? sb : 0u);
    }
    if (PAIRS < 64 && tc == tiles_c - 1) {
      const int64_t row = tiles_c * (2 * PAIRS) + tid;
      if (row < (p.cols + 127) / 128 * 128) put(row, 0u);
    }
  } else if (TILE) {
    if (tid == 0) p.scales[tc * nblk + tr] = (uint8_t)sa;
  } else if (q == 0) {
    if (ca) p.scales[c0 * nblk + tr] = (uint8_t)sa;
    if (cb) p.scales[(c0 + 1) * nblk + tr] = (uint8_t)sb;
  }
  const bool bad = sa == 255u || sb == 255u;
  if (__any_sync(0xffffffffu, bad) && (tid & 31) == 0) record_error(KL_DEVERR_NONFINITE);
}

// Tile blocks: one 128 x 128 tile of x a CTA, in registers (16 columns of four
// rows a thread).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) fp8_encode_tile_kernel(const Fp8EncodeParams p, int tiles_c) {
  __shared__ uint32_t warpmax[8];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int64_t r0 = tr * 128 + (tid >> 3), c0 = tc * 128 + (tid & 7) * 16;
  const int n = (int)min((int64_t)128, p.cols - c0);  // may be negative
  const T* x = reinterpret_cast<const T*>(p.x) + r0 * p.ldx + c0;
  const uint8_t* lo = reinterpret_cast<const uint8_t*>(p.x);
  const uint8_t* hi = lo + ((p.rows - 1) * p.ldx + p.cols) * sizeof(T);
  Fp8Raw<T> raw[4];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) raw[i].template load<VEC>(x + i * 32 * p.ldx, r0 + i * 32 < p.rows ? n : 0, lo, hi);
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, raw[i].amax_bits());
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) warpmax[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, warpmax[i]);
  const uint32_t byte = fp8_scale_byte(m);
  const uint64_t inv2 = fp8_inv2(byte);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[16];
    raw[i].values(v);
    if (n > 0 && r0 + i * 32 < p.rows)
      *reinterpret_cast<uint4*>(p.codes + (r0 + i * 32) * p.ldc + c0) = fp8_codes16(v, inv2, n);
  }
  // scale bytes of this tile's rows; the last tile of a row block zeroes the
  // unused bytes of its words
  const int64_t nblk = (p.cols + 127) >> 7;
  if (p.mma) {
    if (tid < 128) {
      const int64_t row = tr * 128 + tid;
      uint8_t* dst = p.scales + fp8_mma_offset(row, tc, (nblk + 3) >> 2);
      dst[0] = (uint8_t)(row < p.rows ? byte : 0u);
      if (tc == nblk - 1)
        for (int64_t k = 1; ((tc + k) & 3) != 0; ++k) dst[k] = 0;
    }
  } else if (tid == 0) {
    p.scales[tr * nblk + tc] = (uint8_t)byte;
  }
  if (byte == 255u && tid == 0) record_error(KL_DEVERR_NONFINITE);
}

template <typename T, int PAIRS, bool TILE>
static cudaError_t launch_fp8_columns(const Fp8EncodeParams& p, cudaStream_t s) {
  const int64_t tiles_c = (p.cols + 2 * PAIRS - 1) / (2 * PAIRS), tiles = (p.rows + 127) / 128 * tiles_c;
  const bool pairs = (reinterpret_cast<uintptr_t>(p.x) % (2 * sizeof(T))) == 0 && p.ldx % 2 == 0;
  auto kern = pairs ? fp8_encode_columns_kernel<T, true, PAIRS, TILE> : fp8_encode_columns_kernel<T, false, PAIRS, TILE>;
  return launch_pdl(kern, dim3((unsigned)tiles), dim3(8 * PAIRS), 0, s, p, (int)tiles_c);
}

template <typename T>
static cudaError_t launch_fp8_encode(const Fp8EncodeParams& p, cudaStream_t s) {
  const bool vec = (reinterpret_cast<uintptr_t>(p.x) & 15) == 0 && (p.ldx * sizeof(T)) % 16 == 0;
  if (!p.tile && !p.transpose) {
    const int64_t words = (p.cols + 511) / 512, rows = p.mma ? (p.rows + 127) / 128 * 128 : p.rows;
    const int64_t cap = (int64_t)device_sm_count() * 8;
    // up to eight words a task, fewer where that leaves warps without one
    int64_t seg = rows * words / (cap * 8);
    seg = seg < 1 ? 1 : seg > 8 ? 8 : seg;
    const int64_t nseg = (words + seg - 1) / seg, tasks = rows * nseg, ctas = (tasks + 7) / 8;
    seg = (words + nseg - 1) / nseg;
    const dim3 grid((unsigned)(ctas < cap ? ctas : cap));
    auto kern = vec ? fp8_encode_rows_kernel<T, true> : fp8_encode_rows_kernel<T, false>;
    return launch_pdl(kern, grid, dim3(256), 0, s, p, tasks, rcp64((uint64_t)nseg), (int)nseg, (int)seg, (int)words);
  }
  if (p.transpose)  // rows of 128 bytes or more at a time
    return p.tile ? launch_fp8_columns<T, 64, true>(p, s) : launch_fp8_columns<T, 64 / sizeof(T), false>(p, s);
  const int64_t tiles_c = (p.cols + 127) / 128, tiles = (p.rows + 127) / 128 * tiles_c;
  auto kern = vec ? fp8_encode_tile_kernel<T, true> : fp8_encode_tile_kernel<T, false>;
  return launch_pdl(kern, dim3((unsigned)tiles), dim3(256), 0, s, p, (int)tiles_c);
}

}  // namespace kl

extern "C" {

size_t kl_fp8_scales_bytes(int64_t rows, int64_t cols, int flags) {
  if (rows < 0 || cols < 0 || rows > ((int64_t)1 << 40) || cols > ((int64_t)1 << 40)) return 0;
  const size_t blk = (size_t)((cols + 127) / 128), rb = (size_t)((rows + 127) / 128);
  if (flags & KL_SCALE_MMA) return rb * ((blk + 3) / 4) * 512;
  return ((flags & KL_FP8_TILE) ? rb : (size_t)rows) * blk;
}

kl_status kl_quantize_fp8_block(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, void* codes,
                                int64_t ldc, void* scales, int flags, void* stream) {
  using namespace kl;
  if (!x || !codes || !scales) return KL_ERR_INVALID_ARG;
  if (dtype != KL_BF16 && dtype != KL_F32 && dtype != KL_F16) return KL_ERR_INVALID_ARG;
  if (flags & ~(KL_SCALE_MMA | KL_FP8_TILE | KL_FP8_TRANSPOSE)) return KL_ERR_INVALID_ARG;
  if (rows < 1 || cols < 1 || rows > KL_FP8_MAX_DIM || cols > KL_FP8_MAX_DIM) return KL_ERR_UNSUPPORTED_SHAPE;
  const int64_t ocols = (flags & KL_FP8_TRANSPOSE) ? rows : cols;
  if (ldx < cols || ldc < (ocols + 15) / 16 * 16 || ldc % 16) return KL_ERR_INVALID_ARG;
  if ((rows + 127) / 128 * ((cols + 127) / 128) > KL_FP8_MAX_DIM / 4) return KL_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(x, dtype == KL_F32 ? 4 : 2) || !aligned(codes, 16) || !aligned(scales, 4)) return KL_ERR_MISALIGNED;
  kl_status st = check_arch();
  if (st != KL_OK) return st;
  Fp8EncodeParams p{};
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.ldx = ldx;
  p.codes = reinterpret_cast<uint8_t*>(codes);
  p.ldc = ldc;
  p.scales = reinterpret_cast<uint8_t*>(scales);
  p.mma = flags & KL_SCALE_MMA;
  p.tile = flags & KL_FP8_TILE;
  p.transpose = flags & KL_FP8_TRANSPOSE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == KL_BF16  ? launch_fp8_encode<__nv_bfloat16>(p, s)
                        : dtype == KL_F16 ? launch_fp8_encode<__half>(p, s)
                                          : launch_fp8_encode<float>(p, s);
  return e == cudaSuccess ? KL_OK : cuda_fail(e);
}

}  // extern "C"
