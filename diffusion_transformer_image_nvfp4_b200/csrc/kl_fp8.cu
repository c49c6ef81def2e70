// kl_fp8.cu -- FP8 (E4M3) encode with one power-of-two scale per block of 128.
//
// A block is 128 consecutive columns of one row (KL_FP8_ROW) or a 128 x 128
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
// transposes stage a 128 x 128 tile in shared memory (transposes read it by
// column pairs, 32 rows a thread, so a thread writes 32 contiguous bytes of
// x^T).
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

// four values -> four E4M3 bytes of a block (every code NaN if its byte is 255)
__device__ __forceinline__ uint32_t fp8_codes4(float a, float b, float c, float d, uint32_t byte) {
  if (byte == 255u) return 0x7F7F7F7Fu;
  const float inv = fp8_inv_scale(byte);
  return f32x2_to_e4m3x2(__fmul_rn(a, inv), __fmul_rn(b, inv)) |
         (f32x2_to_e4m3x2(__fmul_rn(c, inv), __fmul_rn(d, inv)) << 16);
}

// byte offset of (row, block) in the MMA scale layout
__device__ __forceinline__ int64_t fp8_mma_offset(int64_t row, int64_t blk, int64_t atoms_k) {
  return ((row >> 7) * atoms_k + (blk >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (blk & 3);
}

// 16 consecutive elements of a row, of which `n` exist, as fp32
template <typename T, bool VEC>
__device__ __forceinline__ void load16(const T* p, int n, float (&v)[16]) {
  if (VEC && n >= 16) {
    if constexpr (sizeof(T) == 2) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) unpack2<T>(w[i], v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p) + i);
        v[4 * i] = a.x;
        v[4 * i + 1] = a.y;
        v[4 * i + 2] = a.z;
        v[4 * i + 3] = a.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}

struct Fp8EncodeParams {
  const void* x;
  int64_t rows, cols, ldx;  // of x as given
  uint8_t* codes;
  int64_t ldc;
  uint8_t* scales;
  int mma, tile, transpose;
};

// Row blocks.  A warp takes the four blocks (512 columns) of word `ka` of one
// row; with the MMA layout also the padding rows up to a multiple of 128,
// whose words it zeroes.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) fp8_encode_rows_kernel(const Fp8EncodeParams p, int64_t words, uint64_t rcp_ka,
                                                              int atoms_k) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = (int64_t)gridDim.x * 8;
  const int nblk = (int)((p.cols + 127) >> 7);
  const int64_t cols16 = (p.cols + 15) & ~int64_t(15);
  bool bad = false;
  for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < words; it += nwarps) {
    const int64_t row = div_rcp(it, rcp_ka);
    const int ka = (int)(it - row * atoms_k);
    const int64_t c0 = (int64_t)ka * 512 + lane * 16;
    const bool live = row < p.rows;
    float v[16];
    const int n = live ? (int)max((int64_t)0, min((int64_t)16, p.cols - c0)) : 0;
    if (n > 0) {
      load16<T, VEC>(reinterpret_cast<const T*>(p.x) + row * p.ldx + c0, n, v);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.f;
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t byte = fp8_scale_byte(m);
    bad |= byte == 255u;
    if (live && c0 < cols16) {
      uint4 q;
      q.x = fp8_codes4(v[0], v[1], v[2], v[3], byte);
      q.y = fp8_codes4(v[4], v[5], v[6], v[7], byte);
      q.z = fp8_codes4(v[8], v[9], v[10], v[11], byte);
      q.w = fp8_codes4(v[12], v[13], v[14], v[15], byte);
      *reinterpret_cast<uint4*>(p.codes + row * p.ldc + c0) = q;
    }
    const int blk = ka * 4 + (lane >> 3);
    if (p.mma) {
      const uint32_t mine = live && blk < nblk ? byte : 0u;
      uint32_t w = __shfl_sync(0xffffffffu, mine, 0);
      w |= __shfl_sync(0xffffffffu, mine, 8) << 8;
      w |= __shfl_sync(0xffffffffu, mine, 16) << 16;
      w |= __shfl_sync(0xffffffffu, mine, 24) << 24;
      if (lane == 0) *reinterpret_cast<uint32_t*>(p.scales + fp8_mma_offset(row, (int64_t)ka * 4, atoms_k)) = w;
    } else if ((lane & 7) == 0 && blk < nblk) {
      p.scales[row * nblk + blk] = (uint8_t)byte;
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(KL_DEVERR_NONFINITE);
}

// One 128 x 128 tile of x a CTA, staged in shared memory as it is stored.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) fp8_encode_tile_kernel(const Fp8EncodeParams p, int tiles_c) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  T* tile = reinterpret_cast<T*>(smem_raw);  // [128][128]
  __shared__ uint32_t colmax[4][128];
  __shared__ uint32_t warpmax[8];
  __shared__ uint8_t row_byte[128];  // scale byte of each encoded row
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x % tiles_c;
  const int64_t r0 = tr * 128, c0 = tc * 128;
  const T* x = reinterpret_cast<const T*>(p.x);
  constexpr int E = 16 / sizeof(T);      // elements of a 16-byte vector
  constexpr int VPR = 128 / E;           // vectors of a tile row
  uint32_t m = 0;
#pragma unroll 4
  for (int i = tid; i < 128 * VPR; i += 256) {
    const int r = i / VPR, c = (i % VPR) * E;
    alignas(16) T v[E];
    const int64_t left = r0 + r < p.rows ? p.cols - c0 - c : 0;
    if (VEC && left >= E) {
      *reinterpret_cast<uint4*>(v) = __ldg(reinterpret_cast<const uint4*>(x + (r0 + r) * p.ldx + c0 + c));
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = j < left ? x[(r0 + r) * p.ldx + c0 + c + j] : from_f32<T>(0.f);
    }
    if (p.tile) {
#pragma unroll
      for (int j = 0; j < E; ++j) m = max(m, __float_as_uint(to_f32(v[j])) & 0x7FFFFFFFu);
    }
    *reinterpret_cast<uint4*>(tile + r * 128 + c) = *reinterpret_cast<const uint4*>(v);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) warpmax[warp] = m;
  __syncthreads();
  if (p.tile) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, warpmax[i]);
  }
  // rows and columns of the encoded matrix (x or its transpose), this tile's origin in it
  const int64_t orows = p.transpose ? p.cols : p.rows, ocols = p.transpose ? p.rows : p.cols;
  const int64_t or0 = p.transpose ? c0 : r0, oc0 = p.transpose ? r0 : c0;
  const int64_t ocols16 = (ocols + 15) & ~int64_t(15);
  bool bad = false;
  if (p.transpose) {
    // column pair (of 64) and row quarter of this thread
    const int pair = (warp & 1) * 32 + lane, q = warp >> 1;
    float a[32], b[32];
    uint32_t ma = 0, mb = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if constexpr (sizeof(T) == 2) {
        unpack2<T>(*reinterpret_cast<const uint32_t*>(tile + (q * 32 + i) * 128 + 2 * pair), a[i], b[i]);
      } else {
        const float2 w = *reinterpret_cast<const float2*>(tile + (q * 32 + i) * 128 + 2 * pair);
        a[i] = w.x;
        b[i] = w.y;
      }
      ma = max(ma, __float_as_uint(a[i]) & 0x7FFFFFFFu);
      mb = max(mb, __float_as_uint(b[i]) & 0x7FFFFFFFu);
    }
    if (!p.tile) {
      colmax[q][2 * pair] = ma;
      colmax[q][2 * pair + 1] = mb;
      __syncthreads();
      ma = max(max(colmax[0][2 * pair], colmax[1][2 * pair]), max(colmax[2][2 * pair], colmax[3][2 * pair]));
      mb = max(max(colmax[0][2 * pair + 1], colmax[1][2 * pair + 1]),
               max(colmax[2][2 * pair + 1], colmax[3][2 * pair + 1]));
    } else {
      ma = mb = m;
    }
    const uint32_t sa = fp8_scale_byte(ma), sb = fp8_scale_byte(mb);
    bad = sa == 255u || sb == 255u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t oc = oc0 + q * 32 + h * 16;
      if (oc >= ocols16) continue;
      uint32_t wa[4], wb[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = h * 16 + j * 4;
        wa[j] = fp8_codes4(a[i], a[i + 1], a[i + 2], a[i + 3], sa);
        wb[j] = fp8_codes4(b[i], b[i + 1], b[i + 2], b[i + 3], sb);
      }
      const int64_t orow = or0 + 2 * pair;
      if (orow < orows)
        *reinterpret_cast<uint4*>(p.codes + orow * p.ldc + oc) = make_uint4(wa[0], wa[1], wa[2], wa[3]);
      if (orow + 1 < orows)
        *reinterpret_cast<uint4*>(p.codes + (orow + 1) * p.ldc + oc) = make_uint4(wb[0], wb[1], wb[2], wb[3]);
    }
    if (q == 0) {
      row_byte[2 * pair] = (uint8_t)sa;
      row_byte[2 * pair + 1] = (uint8_t)sb;
    }
  } else {
    const uint32_t s = fp8_scale_byte(m);
    bad = s == 255u;
#pragma unroll 2
    for (int i = tid; i < 128 * 8; i += 256) {
      const int r = i >> 3, c = (i & 7) * 16;
      if (r0 + r >= p.rows || c0 + c >= ocols16) continue;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const T* t = tile + r * 128 + c + 4 * j;
        w[j] = fp8_codes4(to_f32(t[0]), to_f32(t[1]), to_f32(t[2]), to_f32(t[3]), s);
      }
      *reinterpret_cast<uint4*>(p.codes + (r0 + r) * p.ldc + c0 + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (tid < 128) row_byte[tid] = (uint8_t)s;
  }
  __syncthreads();
  // scale bytes of this tile's rows; the last tile of a row block zeroes the
  // unused bytes of its words
  const int64_t oblk = oc0 >> 7, nblk = (ocols + 127) >> 7;
  if (tid < 128) {
    const int64_t row = or0 + tid;
    const uint32_t byte = row < orows ? row_byte[tid] : 0u;
    if (p.mma) {
      const int64_t atoms_k = (nblk + 3) >> 2;
      uint8_t* dst = p.scales + fp8_mma_offset(row, oblk, atoms_k);
      dst[0] = (uint8_t)byte;
      if (oblk == nblk - 1)
        for (int64_t k = 1; ((oblk + k) & 3) != 0; ++k) dst[k] = 0;
    } else if (!p.tile) {
      if (row < orows) p.scales[row * nblk + oblk] = (uint8_t)byte;
    } else if (tid == 0) {
      p.scales[(or0 >> 7) * nblk + oblk] = (uint8_t)byte;
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(KL_DEVERR_NONFINITE);
}

template <typename T>
static cudaError_t launch_fp8_encode(const Fp8EncodeParams& p, cudaStream_t s) {
  const bool vec = (reinterpret_cast<uintptr_t>(p.x) & 15) == 0 && (p.ldx * sizeof(T)) % 16 == 0;
  if (!p.tile && !p.transpose) {
    const int64_t atoms_k = (p.cols + 511) / 512;
    const int64_t words = (p.mma ? (p.rows + 127) / 128 * 128 : p.rows) * atoms_k;
    const int64_t ctas = (words + 7) / 8, cap = (int64_t)device_sm_count() * 8;
    const dim3 grid((unsigned)(ctas < cap ? ctas : cap));
    const uint64_t r = rcp64((uint64_t)atoms_k);
    return vec ? launch_pdl(fp8_encode_rows_kernel<T, true>, grid, dim3(256), 0, s, p, words, r, (int)atoms_k)
               : launch_pdl(fp8_encode_rows_kernel<T, false>, grid, dim3(256), 0, s, p, words, r, (int)atoms_k);
  }
  const int64_t tiles_c = (p.cols + 127) / 128, tiles = (p.rows + 127) / 128 * tiles_c;
  const size_t smem = 128 * 128 * sizeof(T);
  auto kern = vec ? fp8_encode_tile_kernel<T, true> : fp8_encode_tile_kernel<T, false>;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3((unsigned)tiles), dim3(256), smem, s, p, (int)tiles_c);
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
  if ((rows + 127) / 128 * ((cols + 127) / 128) > KL_FP8_MAX_DIM) return KL_ERR_UNSUPPORTED_SHAPE;
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
