// kl_fp8_gemm.cu -- C[M,N] = sum_k dec(A)[m,k] dec(W)[n,k] over E4M3 operands
// with one power-of-two scale per block of 128 (kl_fp8.cu), on tcgen05
// kind::mxf8f6f4: the tensor core multiplies every group of 32 products by
// both operands' scale bytes, so scaling and the whole K sum stay in the fp32
// TMEM accumulator.  A block of 128 is four such groups with the same byte: a
// K stage is one block (128 bytes of each row, four MMAs), and one 512-byte
// scale atom serves four stages, the stage's byte chosen in the instruction.
//
// Two kernels, chosen by how much work there is (launch_gemm_fp8):
//
//  * gemm_fp8_pair_kernel: CTA pairs (cluster of 2, cta_group::2) on 256 x BN
//    output tiles, persistent, six warp roles as in the NVFP4 pair kernel:
//    TMA producer (both CTAs), scale copies + MMAs (leader), eight epilogue
//    warps per CTA that drain the accumulator to registers, release it and
//    store while the next tile's MMAs run.  Bound by the tensor cores and, in
//    long runs, by power: 4,608 x 9,216 x 3,072 in 97 us (2.7 PFLOP/s), 20,992 x
//    3,072 x 9,216 in 404 (2.9) in short runs, 114 and 468 in long ones.
//  * gemm_fp8_split_kernel: few rows, or few tiles.  The weights take the
//    128-row side of the MMA and the tokens the N side (16 to 128), so one
//    token wastes 15 of 16 columns instead of 127 of 128 rows; where tiles are
//    few and K is long, K is split over a cluster of up to eight CTAs so that
//    about every SM streams a part of the weights, and the parts' fp32 sums are
//    added in rank order through distributed shared memory: one launch, no
//    workspace, the same bits every run.  At one token bound by latency and the launch
//    (1 x 9,216 x 3,072 in 6.8 us, 8.5 with the weights in HBM: 3.3 TB/s over the
//    launch, half the copy's rate): a CTA asks for the first 10 of its 12 K
//    blocks at once and for the last two as the first are consumed.
//
// Either kernel can take the roles of A and W exchanged (each thread then
// owns an output column and a warp stores 32 consecutive ones): the split
// kernel always does, the pair kernel when the output rows are not 16-byte
// aligned, where a thread that owns a row would have to store single elements.
#include "../../include/klein.h"
#include "kl_common.cuh"
#include "kl_internal.h"

namespace kl {

struct GemmFp8Params {
  int64_t rows_a, rows_b, K;  // MMA's M side and N side
  void* out;
  int64_t ldo;
  int out_f32;
  int vec4;  // four consecutive outputs of any row from a multiple of 4 can be stored as one vector
  int num_kb, atoms_k, num_a, num_b, num_tiles;
};

// -------------------------------------------------------------- pair kernel
template <int BN>
struct GemmFp8Cfg {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = (BN / 2) * 128;
  static constexpr int SF_BYTES = 2048;  // A atom, BN / 128 W atoms, padding to the 1 KB operand alignment
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SF_BYTES;
  static constexpr int TX_BYTES = A_BYTES + B_BYTES + 512 * (1 + BN / 128);
  static constexpr int STAGES = BN == 256 ? 6 : 8;
  static constexpr int ACC = BN == 256 ? 1 : 2;
  static constexpr uint32_t SF_COLS = 16;  // A 4, W 4 * BN / 128
  static constexpr uint32_t SF_BASE = ACC * BN;
  static constexpr int EPI_BYTES = 8 * 2048;  // a warp: 64 bytes of 32 output rows
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_BYTES + 1024 + 512;
  static_assert(SF_BASE + STAGES * SF_COLS <= 512, "TMEM budget");
  static_assert(SMEM_BYTES <= 232448, "smem budget");
  static_assert(STAGE_BYTES % 1024 == 0, "stage alignment");
};

// Tile order: groups of 8 tiles along the M side, across the whole N side
// before the next group, so the tiles in flight (74 pairs: about 8 x 9) share
// both operands' rows in L2 and each group's A rows come from HBM once.
__device__ __forceinline__ void fp8_tile_at(const GemmFp8Params& p, int tile, int& ab, int& bb) {
  const int g = tile / (8 * p.num_b), r = tile - g * 8 * p.num_b;
  const int ga = min(8, p.num_a - g * 8);
  bb = r / ga;
  ab = g * 8 + r - bb * ga;
}

// 64 bytes of 32 output rows from (row0, n0), a row a lane: through shared
// memory, so that a store writes 8 rows' whole sectors instead of 16 bytes of
// 32 rows.  16-byte unit u of row r stands at r * 64 + (u ^ (r / 2 % 4)) * 16:
// neither side meets a bank twice.  Output rows start on 16 bytes.
__device__ __forceinline__ void fp8_store_rows(const GemmFp8Params& p, uint8_t* buf, int lane, int64_t row0, int64_t n0,
                                               int64_t M, int64_t N, const uint4 (&w)[4]) {
  const int es = p.out_f32 ? 4 : 2;
#pragma unroll
  for (int u = 0; u < 4; ++u) *reinterpret_cast<uint4*>(buf + lane * 64 + ((u ^ (lane >> 1 & 3)) << 4)) = w[u];
  __syncwarp();
  const int unit = lane & 3;
  const int64_t n = n0 + unit * 16 / es;
  const int left = (int)min((int64_t)(16 / es), N - n);  // elements of the unit that exist
  uint8_t* out = reinterpret_cast<uint8_t*>(p.out) + n * es;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    const uint4 q = *reinterpret_cast<const uint4*>(buf + r * 64 + ((unit ^ (r >> 1 & 3)) << 4));
    if (row0 + r < M) {
      uint8_t* o = out + (row0 + r) * p.ldo * es;
      if (left * es == 16) {
        *reinterpret_cast<uint4*>(o) = q;
      } else if (left > 0) {
        const uint32_t e[4] = {q.x, q.y, q.z, q.w};
        if (p.out_f32) {
#pragma unroll
          for (int k = 0; k < 3; ++k)
            if (k < left) reinterpret_cast<uint32_t*>(o)[k] = e[k];
        } else {
#pragma unroll
          for (int k = 0; k < 7; ++k)
            if (k < left) reinterpret_cast<uint16_t*>(o)[k] = (uint16_t)(e[k / 2] >> (k & 1) * 16);
        }
      }
    }
  }
  __syncwarp();
}

__device__ __forceinline__ void fp8_store_one(const GemmFp8Params& p, int64_t m, int64_t n, float v) {
  if (p.out_f32)
    reinterpret_cast<float*>(p.out)[m * p.ldo + n] = v;
  else
    reinterpret_cast<uint16_t*>(p.out)[m * p.ldo + n] = (uint16_t)f32_to_bf16_bits(v);
}

// SWAP: the MMA's M side is the product's W (output columns), its N side A.
template <int BN, bool SWAP>
__global__ void __launch_bounds__(320, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                         const __grid_constant__ CUtensorMap tmap_sfa, const __grid_constant__ CUtensorMap tmap_sfb,
                         const GemmFp8Params p) {
  using C = GemmFp8Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* epi = smem + C::STAGES * C::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + C::EPI_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;  // ACC
  uint64_t* tempty = tfull + C::ACC;    // ACC (leader: 16 arrivals each)
  uint64_t* drain = tempty + C::ACC;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < C::ACC; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 16);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmap_a);
    prefetch_tmap(&tmap_b);
    prefetch_tmap(&tmap_sfa);
    prefetch_tmap(&tmap_sfb);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait();  // no global memory before the previous kernel of the stream is done
  pdl_trigger();
  const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
  const uint32_t tempty_leader = mapa_shared(smem_u32(tempty), 0);
  const uint64_t desc_a0 = smem_desc(smem_u32(smem), 16, 1024, kLayoutSw128);
  const uint64_t desc_b0 = smem_desc(smem_u32(smem + C::A_BYTES), 16, 1024, kLayoutSw128);
  const uint64_t desc_sf0 = smem_desc(smem_u32(smem + C::A_BYTES + C::B_BYTES), 0, 128, kLayoutNone);

  if (warp == 0) {
    // ------------------------------------------------- producer (both CTAs)
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = pair; tile < p.num_tiles && ok; tile += npairs) {
      int ab, bb;
      fp8_tile_at(p, tile, ab, bb);
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (!warp_wait(&empty[stage], phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* sa = smem + stage * C::STAGE_BYTES;
          uint8_t* sb = sa + C::A_BYTES;
          uint8_t* ssf = sb + C::B_BYTES;
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * C::TX_BYTES);
          const uint32_t fb = full_leader + (uint32_t)stage * 8u;
          tma_load_2d_pair(sa, &tmap_a, kb * 128, ab * 256 + (int)rank * 128, fb);
          tma_load_2d_pair(sb, &tmap_b, kb * 128, bb * BN + (int)rank * (BN / 2), fb);
          tma_load_2d_pair(ssf, &tmap_sfa, 0, (ab * 2 + (int)rank) * p.atoms_k + (kb >> 2), fb);
          tma_load_3d_pair(ssf + 512, &tmap_sfb, 0, kb >> 2, bb * (BN / 128), fb);
        }
        __syncwarp();
        ++issued;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && leader) {
      // every load already issued by the pair lands before a CTA can leave
      volatile int no_abort = 0;
      for (int i = max(0, issued - C::STAGES); i < issued; ++i)
        warp_wait(&full[i % C::STAGES], (uint32_t)((i / C::STAGES) & 1), &no_abort);
    }
  } else if (warp == 1) {
    // ------------------------------- scale copies and MMAs (leader's warp)
    if (leader) {
      constexpr uint32_t idesc = idesc_mxf8(256, BN);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int tile = pair; tile < p.num_tiles && ok; tile += npairs) {
        if (!warp_wait(&tempty[acc], acc_phase ^ 1u, abort_flag)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + (uint32_t)(acc * BN);
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!warp_wait(&full[stage], phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t soff = (uint64_t)((stage * C::STAGE_BYTES) >> 4);
            const uint32_t sfa_t = tmem + C::SF_BASE + (uint32_t)stage * C::SF_COLS;
            const uint32_t sfb_t = sfa_t + 4;
            // tcgen05.cp then tcgen05.mma from one thread run in issue order
            tmem_cp_32x128b_x4_pair(sfa_t, desc_sf0 + soff);
#pragma unroll
            for (int j = 0; j < BN / 128; ++j)
              tmem_cp_32x128b_x4_pair(sfb_t + 4 * j, desc_sf0 + soff + (uint64_t)(32 * (j + 1)));
            const uint32_t id = idesc | idesc_scale_byte((uint32_t)kb & 3u);
            // groups of 32 past K hold zeros: left out
            const int nk = (int)min((int64_t)4, (p.K - (int64_t)kb * 128 + 31) >> 5);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk < nk)
                mma_mxf8_pair(d_tmem, desc_a0 + soff + (uint64_t)(kk * 2), desc_b0 + soff + (uint64_t)(kk * 2), id,
                              sfa_t, sfb_t, (kb | kk) != 0 ? 1u : 0u);
            }
            tc_commit_pair_mc(&empty[stage], 3);
          }
          __syncwarp();
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one()) tc_commit_pair_mc(&tfull[acc], 3);
        __syncwarp();
        if (++acc == C::ACC) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (elect_one()) tc_commit_pair(drain);
      __syncwarp();
      volatile int no_abort = 0;
      warp_wait(drain, 0, &no_abort);
    }
  } else {
    // ---------------------------------------------- epilogue (both CTAs)
    const int quad = warp & 3;
    const int half = (warp - 2) >> 2;
    int acc = 0;
    uint32_t acc_phase = 0;
    float v[BN / 2];
    for (int tile = pair; tile < p.num_tiles; tile += npairs) {
      int ab, bb;
      fp8_tile_at(p, tile, ab, bb);
      if (!warp_wait(&tfull[acc], acc_phase, abort_flag)) break;
      tc_fence_after();
      const uint32_t tb = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(acc * BN + half * (BN / 2));
      if constexpr (BN == 256)
        tmem_ld128(tb, v);
      else
        tmem_ld64(tb, v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty_leader + (uint32_t)acc * 8u);
      if (++acc == C::ACC) {
        acc = 0;
        acc_phase ^= 1u;
      }
      const int64_t ra0 = (int64_t)ab * 256 + rank * 128 + quad * 32, ra = ra0 + lane;
      const int64_t rb0 = (int64_t)bb * BN + half * (BN / 2);
      if constexpr (SWAP) {
        if (ra < p.rows_a) {
          const int rows = (int)min((int64_t)(BN / 2), p.rows_b - rb0);  // of the output; may be negative
          if (p.out_f32) {
            float* o = reinterpret_cast<float*>(p.out) + rb0 * p.ldo + ra;
#pragma unroll
            for (int i = 0; i < BN / 2; ++i, o += p.ldo)
              if (i < rows) *o = v[i];
          } else {
            uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + rb0 * p.ldo + ra;
#pragma unroll
            for (int i = 0; i < BN / 2; ++i, o += p.ldo)
              if (i < rows) *o = (uint16_t)f32_to_bf16_bits(v[i]);
          }
        }
      } else if (ra0 < p.rows_a) {
        uint8_t* buf = epi + (warp - 2) * 2048;
        uint4 w[4];
        if (p.out_f32) {
#pragma unroll
          for (int c = 0; c < BN / 2; c += 16) {
            if (rb0 + c >= p.rows_b) break;
#pragma unroll
            for (int u = 0; u < 4; ++u)
              w[u] = make_uint4(__float_as_uint(v[c + 4 * u]), __float_as_uint(v[c + 4 * u + 1]),
                                __float_as_uint(v[c + 4 * u + 2]), __float_as_uint(v[c + 4 * u + 3]));
            fp8_store_rows(p, buf, lane, ra0, rb0 + c, p.rows_a, p.rows_b, w);
          }
        } else {
#pragma unroll
          for (int c = 0; c < BN / 2; c += 32) {
            if (rb0 + c >= p.rows_b) break;
#pragma unroll
            for (int u = 0; u < 4; ++u)
              w[u] = make_uint4(pack_bf16x2(v[c + 8 * u], v[c + 8 * u + 1]), pack_bf16x2(v[c + 8 * u + 2], v[c + 8 * u + 3]),
                                pack_bf16x2(v[c + 8 * u + 4], v[c + 8 * u + 5]),
                                pack_bf16x2(v[c + 8 * u + 6], v[c + 8 * u + 7]));
            fp8_store_rows(p, buf, lane, ra0, rb0 + c, p.rows_a, p.rows_b, w);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncwarp();
  cluster_sync_all();  // no CTA leaves while its pair may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------- split kernel
// BT: the tokens of a tile.
template <int BT>
struct GemmFp8SplitCfg {
  static constexpr int W_BYTES = 128 * 128;
  static constexpr int X_BYTES = BT * 128;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES + 1024;  // + one scale atom each
  static constexpr int STAGES = (200 * 1024) / STAGE_BYTES;
  static constexpr uint32_t SF_COLS = 8;
  static constexpr uint32_t SF_BASE = 128;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + 512;
  static_assert(SF_BASE + STAGES * SF_COLS <= 256, "TMEM budget");
  static_assert(BT * 128 * 4 <= STAGES * STAGE_BYTES, "partial sums reuse the stages");
};

template <int BT>
__global__ void __launch_bounds__(192, 1)
    gemm_fp8_split_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                          const uint8_t* __restrict__ sfw, const uint8_t* __restrict__ sfx, const GemmFp8Params p) {
  using C = GemmFp8SplitCfg<BT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* done = empty + C::STAGES;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int tile = blockIdx.y;
  const int wb = tile % p.num_a, xb = tile / p.num_a;
  // this CTA's K blocks: [kb0, kb1), as even as they come
  const int kb0 = (int)((int64_t)p.num_kb * rank / S), kb1 = (int)((int64_t)p.num_kb * (rank + 1) / S);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmap_w);
    prefetch_tmap(&tmap_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait();  // no global memory before the previous kernel of the stream is done
  pdl_trigger();
  const int64_t tok0 = (int64_t)xb * BT;
  const int live = (int)min((int64_t)BT, p.rows_b - tok0);  // tokens of this tile that exist

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    const uint8_t* sw = sfw + (int64_t)wb * p.atoms_k * 512;
    const uint8_t* sx = sfx + (tok0 >> 7) * p.atoms_k * 512;
    int issued = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!warp_wait(&empty[stage], phase ^ 1u, abort_flag)) {
        ok = false;
        break;
      }
      if (elect_one()) {
        uint8_t* s = smem + stage * C::STAGE_BYTES;
        mbar_arrive_expect_tx(&full[stage], C::STAGE_BYTES);
        tma_load_2d(s, &tmap_w, kb * 128, wb * 128, &full[stage]);
        tma_load_2d(s + C::W_BYTES, &tmap_x, kb * 128, (int)tok0, &full[stage]);
        bulk_load(s + C::W_BYTES + C::X_BYTES, sw + (int64_t)(kb >> 2) * 512, 512, &full[stage]);
        bulk_load(s + C::W_BYTES + C::X_BYTES + 512, sx + (int64_t)(kb >> 2) * 512, 512, &full[stage]);
      }
      __syncwarp();
      ++issued;
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) {
      // every load already issued lands before the CTA can leave
      volatile int no_abort = 0;
      for (int i = max(0, issued - C::STAGES); i < issued; ++i)
        warp_wait(&full[i % C::STAGES], (uint32_t)((i / C::STAGES) & 1), &no_abort);
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_mxf8(128, BT);
    const uint64_t desc_w0 = smem_desc(smem_u32(smem), 16, 1024, kLayoutSw128);
    const uint64_t desc_x0 = smem_desc(smem_u32(smem + C::W_BYTES), 16, 1024, kLayoutSw128);
    const uint64_t desc_sf0 = smem_desc(smem_u32(smem + C::W_BYTES + C::X_BYTES), 0, 128, kLayoutNone);
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!warp_wait(&full[stage], phase, abort_flag)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t soff = (uint64_t)((stage * C::STAGE_BYTES) >> 4);
        const uint32_t sfw_t = tmem + C::SF_BASE + (uint32_t)stage * C::SF_COLS;
        tmem_cp_32x128b_x4(sfw_t, desc_sf0 + soff);
        tmem_cp_32x128b_x4(sfw_t + 4, desc_sf0 + soff + 32);
        // a column of the copied atom holds 32 of its 128 tokens: a tile of 64
        // starts at its first or third (smaller tiles are the only one, launch_gemm_fp8)
        const uint32_t sfx_t = sfw_t + 4 + (BT == 64 ? (uint32_t)(xb & 1) * 2u : 0u);
        const uint32_t id = idesc | idesc_scale_byte((uint32_t)kb & 3u);
        const int nk = (int)min((int64_t)4, (p.K - (int64_t)kb * 128 + 31) >> 5);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk < nk)
            mma_mxf8(tmem, desc_w0 + soff + (uint64_t)(kk * 2), desc_x0 + soff + (uint64_t)(kk * 2), id, sfw_t, sfx_t,
                     (kb > kb0 || kk > 0) ? 1u : 0u);
        }
        tc_commit(&empty[stage]);
      }
      __syncwarp();
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // every MMA issued by this warp has completed before anyone reads the
    // accumulator, reuses the stages or frees TMEM
    if (elect_one()) tc_commit(done);
    __syncwarp();
    volatile int no_abort = 0;
    warp_wait(done, 0, &no_abort);
  } else {
    volatile int no_abort = 0;
    if (warp_wait(done, 0, &no_abort)) {
      tc_fence_after();
      const int quad = warp & 3;  // warps 2..5 read TMEM lanes 64.., 96.., 0.., 32..
      const uint32_t tb = tmem + ((uint32_t)(quad * 32) << 16);
      const int r = quad * 32 + lane;
      const int64_t n = (int64_t)wb * 128 + r;
      constexpr int CH = BT < 32 ? BT : 32;
      float* part = reinterpret_cast<float*>(smem) + r;
      // (rolled: a launch this short is bound by fetching its instructions)
#pragma unroll 1
      for (int c = 0; c < BT; c += CH) {
        float v[CH];
        if constexpr (CH == 32)
          tmem_ld32(tb + (uint32_t)c, v);
        else
          tmem_ld16(tb, v);
        if (S > 1) {
          // partial sums [token][128] over the stages, which nothing reads any more
#pragma unroll
          for (int t = 0; t < CH; ++t) part[(c + t) * 128] = v[t];
        } else if (n < p.rows_a) {
          if (p.out_f32) {
            float* o = reinterpret_cast<float*>(p.out) + (tok0 + c) * p.ldo + n;
#pragma unroll
            for (int t = 0; t < CH; ++t, o += p.ldo)
              if (c + t < live) *o = v[t];
          } else {
            uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + (tok0 + c) * p.ldo + n;
#pragma unroll
            for (int t = 0; t < CH; ++t, o += p.ldo)
              if (c + t < live) *o = (uint16_t)f32_to_bf16_bits(v[t]);
          }
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
  if (S > 1) {
    cluster_sync_all();  // every CTA's partial sums are written
    // token t of the tile belongs to rank t mod S; a warp sums one token, four
    // columns a lane, the ranks' parts in rank order
    const int64_t n = (int64_t)wb * 128 + lane * 4;
    const bool vec = p.rows_a - n >= 4 && p.vec4;
    for (int t = rank + S * warp; t < live; t += S * 6) {
      const uint32_t at = smem_u32(smem) + (uint32_t)(t * 128 + lane * 4) * 4u;
      float4 q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < S) q[i] = ld_shared_cluster_f32x4(mapa_shared(at, (uint32_t)i));
      float4 s = q[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        if (i < S) {
          s.x += q[i].x;
          s.y += q[i].y;
          s.z += q[i].z;
          s.w += q[i].w;
        }
      }
      if (vec) {
        if (p.out_f32)
          *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + (tok0 + t) * p.ldo + n) = s;
        else
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + (tok0 + t) * p.ldo + n) =
              make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
      } else {
        const float e[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < p.rows_a) fp8_store_one(p, tok0 + t, n + i, e[i]);
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while another may read its sums
  }
}

// ---------------------------------------------------------------- launchers
// operand rows [row, K] of E4M3 codes, boxes of 128 bytes x `box` rows
static bool fp8_operand_map(CUtensorMap* m, const void* codes, int64_t rows, int64_t K, int64_t ld, int box) {
  return make_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, (uint64_t)K, (uint64_t)rows, (uint64_t)ld, 128,
                      (uint32_t)box, 128);
}

template <int BN, bool SWAP>
static cudaError_t launch_fp8_pair(const GemmFp8Args& a, cudaStream_t s) {
  using C = GemmFp8Cfg<BN>;
  CUtensorMap ta, tb, tsa, tsb;
  const uint64_t atoms_k = (uint64_t)((a.K + 511) / 512);
  const uint64_t sfb_dims[3] = {128, atoms_k, (uint64_t)((a.rows_b + 127) / 128)};
  const uint64_t sfb_strides[2] = {512, atoms_k * 512};
  const uint32_t sfb_box[3] = {128, 1, (uint32_t)(BN / 128)};
  if (!fp8_operand_map(&ta, a.a_codes, a.rows_a, a.K, a.lda, 128) ||
      !fp8_operand_map(&tb, a.b_codes, a.rows_b, a.K, a.ldb, BN / 2) ||
      !make_tmap_2d(&tsa, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.a_scales, 128,
                    (uint64_t)((a.rows_a + 127) / 128) * atoms_k, 512, 128, 1, 0) ||
      !make_tmap_3d(&tsb, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.b_scales, sfb_dims, sfb_strides, sfb_box))
    return cudaErrorInvalidValue;
  GemmFp8Params p;
  p.rows_a = a.rows_a;
  p.rows_b = a.rows_b;
  p.K = a.K;
  p.out = a.out;
  p.ldo = a.ldo;
  p.out_f32 = a.out_f32;
  p.vec4 = (reinterpret_cast<uintptr_t>(a.out) & (a.out_f32 ? 15 : 7)) == 0 && a.ldo % 4 == 0;
  p.num_kb = (int)((a.K + 127) / 128);
  p.atoms_k = (int)atoms_k;
  p.num_a = (int)((a.rows_a + 255) / 256);
  p.num_b = (int)((a.rows_b + BN - 1) / BN);
  p.num_tiles = p.num_a * p.num_b;
  cudaError_t e = cudaFuncSetAttribute(gemm_fp8_pair_kernel<BN, SWAP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int pairs_max = device_sm_count() / 2;
  const int pairs = p.num_tiles < pairs_max ? p.num_tiles : pairs_max;
  return launch_pdl_cluster(gemm_fp8_pair_kernel<BN, SWAP>, dim3((unsigned)(2 * pairs)), dim3(320), 2, C::SMEM_BYTES,
                            s, ta, tb, tsa, tsb, p);
}

// a: the product's W takes the A side
template <int BT>
static cudaError_t launch_fp8_split(const GemmFp8Args& a, int split, cudaStream_t s) {
  using C = GemmFp8SplitCfg<BT>;
  CUtensorMap tw, tx;
  if (!fp8_operand_map(&tw, a.a_codes, a.rows_a, a.K, a.lda, 128) ||
      !fp8_operand_map(&tx, a.b_codes, a.rows_b, a.K, a.ldb, BT))
    return cudaErrorInvalidValue;
  GemmFp8Params p;
  p.rows_a = a.rows_a;
  p.rows_b = a.rows_b;
  p.K = a.K;
  p.out = a.out;
  p.ldo = a.ldo;
  p.out_f32 = a.out_f32;
  p.vec4 = (reinterpret_cast<uintptr_t>(a.out) & (a.out_f32 ? 15 : 7)) == 0 && a.ldo % 4 == 0;
  p.num_kb = (int)((a.K + 127) / 128);
  p.atoms_k = (int)((a.K + 511) / 512);
  p.num_a = (int)((a.rows_a + 127) / 128);
  p.num_b = (int)((a.rows_b + BT - 1) / BT);
  p.num_tiles = p.num_a * p.num_b;
  cudaError_t e = cudaFuncSetAttribute(gemm_fp8_split_kernel<BT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(gemm_fp8_split_kernel<BT>, dim3((unsigned)split, (unsigned)p.num_tiles), dim3(192),
                            (unsigned)split, C::SMEM_BYTES, s, tw, tx, reinterpret_cast<const uint8_t*>(a.a_scales),
                            reinterpret_cast<const uint8_t*>(a.b_scales), p);
}

// Which kernel: by estimated times in us, fitted to measurements on a B200 (148
// SMs, weights from HBM, bf16 results).  The first of the terms is what a
// launch, or a wave of CTAs, costs without any K block; the other is the time of
// a K block.
//   M x N x K              measured (us)                            taken
//   10 x 1000 x 1000       split, 16 tokens, S = 4 3.9; pair 128 5.2    split
//   333 x 1000 x 1328      64 tokens, S = 1 5.9, 2 7.0; 128 tokens, S = 4 7.3; pair 128 9.2, 256 13.5   64, S = 1
//   64 x 3072 x 9216       64 tokens, S = 1 21.1, 4 10.5; pair 128 20.6   64, S = 4
//   128 x 9216 x 3072      64 tokens, S = 1 10.0; 128 tokens 10.7; pair 128 11.3   64, S = 1
//   256 x 9216 x 3072      pair 128 11.2, 256 13.0; 128 tokens 17.0    pair 128
//   512 x 9216 x 3072      pair 256 14.1, 128 16.8                     pair 256
static double fp8_pair_time(const GemmFp8Args& g, int bn) {
  const double kb = (double)((g.K + 127) / 128);
  const int64_t tiles = (g.rows_a + 255) / 256 * ((g.rows_b + bn - 1) / bn), pairs = device_sm_count() / 2;
  const double rounds = (double)((tiles + pairs - 1) / pairs);
  return bn == 256 ? 6.0 + rounds * (0.30 * kb + 0.8) : 5.0 + rounds * (0.20 * kb + 0.8);
}

// CTAs that clusters of `split` fill at once (a GPC's SMs hold whole clusters only)
template <int BT>
static int64_t fp8_split_slots(int split) {
  static DeviceValue slots[9];
  int dev = 0;
  if (split == 1 || cudaGetDevice(&dev) != cudaSuccess) return device_sm_count() / split * split;
  return slots[split].get(dev, [split] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split, 64);
    cfg.blockDim = dim3(192);
    cfg.dynamicSmemBytes = GemmFp8SplitCfg<BT>::SMEM_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(gemm_fp8_split_kernel<BT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             GemmFp8SplitCfg<BT>::SMEM_BYTES) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, gemm_fp8_split_kernel<BT>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = device_sm_count() / (2 * split);  // an estimate that always fits
    }
    return n * split;
  });
}

// Best tokens a tile and CTAs a cluster of the split kernel, and its time.
static double fp8_split_plan(const GemmFp8Args& g, int64_t* bt_out, int64_t* split_out) {
  const int64_t kb = (g.K + 127) / 128, wt = (g.rows_b + 127) / 128;
  double best = 1e30;
  for (int64_t bt = 16; bt <= 128; bt *= 2) {
    const int64_t tiles = wt * ((g.rows_a + bt - 1) / bt);
    // the scales of 16 or 32 tokens are read from the first of their 128
    if (tiles > 65535 || (bt < 64 && g.rows_a > bt)) continue;
    // the operands of all tiles, through L2
    const double traffic = 2.0 + (double)tiles * (128 + bt) * g.K / 11e6;
    for (int64_t split = 1; split <= 8 && split <= kb; ++split) {
      if (split > 1 && tiles * split > device_sm_count()) break;
      const int64_t slots = bt == 16   ? fp8_split_slots<16>((int)split)
                            : bt == 32 ? fp8_split_slots<32>((int)split)
                            : bt == 64 ? fp8_split_slots<64>((int)split)
                                       : fp8_split_slots<128>((int)split);
      const double waves = (double)((tiles * split + slots - 1) / slots);
      const double blocks = (double)((kb + split - 1) / split);
      double wave = 1.8 + 0.013 * bt + (bt == 128 ? 0.30 : 0.25) * blocks;
      if (split > 1) wave += 1.1 + 0.03 * bt / split;
      double t = 0.6 + waves * wave;
      if (t < traffic) t = traffic;
      if (t < best) {
        best = t;
        *bt_out = bt;
        *split_out = split;
      }
    }
    if (g.rows_a <= bt) break;
  }
  return best;
}

cudaError_t launch_gemm_fp8(const GemmFp8Args& g, cudaStream_t s) {
  // g: A = the product's A (M rows), B = its W (N rows)
  GemmFp8Args x = g;  // roles exchanged
  x.a_codes = g.b_codes;
  x.a_scales = g.b_scales;
  x.lda = g.ldb;
  x.rows_a = g.rows_b;
  x.b_codes = g.a_codes;
  x.b_scales = g.a_scales;
  x.ldb = g.lda;
  x.rows_b = g.rows_a;
  const int es = g.out_f32 ? 4 : 2;
  const bool rows_ok = (reinterpret_cast<uintptr_t>(g.out) & 15) == 0 && (g.ldo * es) % 16 == 0;
  int kind = g.force;
  int64_t bt = 0, split = 0;
  if (kind == KL_FP8_GEMM_AUTO || kind == KL_FP8_GEMM_SPLIT) {
    const double t = fp8_split_plan(g, &bt, &split);
    if (kind == KL_FP8_GEMM_AUTO) {
      const double t256 = fp8_pair_time(g, 256), t128 = fp8_pair_time(g, 128);
      kind = t <= t256 && t <= t128 ? KL_FP8_GEMM_SPLIT
             : t128 < t256          ? KL_FP8_GEMM_PAIR_256x128
                                    : KL_FP8_GEMM_PAIR_256x256;
    }
  }
  if (kind == KL_FP8_GEMM_SPLIT) {
    switch (bt) {
      case 0: return cudaErrorInvalidValue;  // more tiles than a grid's second dimension takes
      case 16: return launch_fp8_split<16>(x, (int)split, s);
      case 32: return launch_fp8_split<32>(x, (int)split, s);
      case 64: return launch_fp8_split<64>(x, (int)split, s);
      default: return launch_fp8_split<128>(x, (int)split, s);
    }
  }
  if (kind == KL_FP8_GEMM_PAIR_256x256)
    return rows_ok ? launch_fp8_pair<256, false>(g, s) : launch_fp8_pair<256, true>(x, s);
  return rows_ok ? launch_fp8_pair<128, false>(g, s) : launch_fp8_pair<128, true>(x, s);
}

}  // namespace kl

extern "C" kl_status kl_gemm_fp8_block(const kl_fp8_tensor* A, const kl_fp8_tensor* W, int64_t M, int64_t N,
                                       int64_t K, void* out, int out_dtype, int64_t ldo, int kernel, void* stream) {
  using namespace kl;
  if (!A || !W || !out || !A->codes || !A->scales || !W->codes || !W->scales) return KL_ERR_INVALID_ARG;
  if (out_dtype != KL_OUT_BF16 && out_dtype != KL_OUT_F32) return KL_ERR_INVALID_ARG;
  if (kernel < KL_FP8_GEMM_AUTO || kernel > KL_FP8_GEMM_SPLIT) return KL_ERR_INVALID_ARG;
  if (M < 1 || N < 1 || K < 1 || M > KL_FP8_GEMM_MAX || N > KL_FP8_GEMM_MAX || K > KL_FP8_GEMM_MAX)
    return KL_ERR_UNSUPPORTED_SHAPE;
  // tile counts and scale atoms are counted in 32 bits
  const int64_t lim = (int64_t)1 << 30, mt = (M + 127) / 128, nt = (N + 127) / 128, ka = (K + 511) / 512;
  if (mt * nt > lim || (mt + 2) * ka > lim || (nt + 2) * ka > lim) return KL_ERR_UNSUPPORTED_SHAPE;
  if (A->ld < K || A->ld % 16 || W->ld < K || W->ld % 16 || ldo < N) return KL_ERR_INVALID_ARG;
  if (!aligned(A->codes, 16) || !aligned(W->codes, 16) || !aligned(A->scales, 16) || !aligned(W->scales, 16) ||
      !aligned(out, out_dtype == KL_OUT_F32 ? 4 : 2))
    return KL_ERR_MISALIGNED;
  kl_status st = check_arch();
  if (st != KL_OK) return st;
  GemmFp8Args g{};
  g.a_codes = A->codes;
  g.a_scales = A->scales;
  g.lda = A->ld;
  g.rows_a = M;
  g.b_codes = W->codes;
  g.b_scales = W->scales;
  g.ldb = W->ld;
  g.rows_b = N;
  g.K = K;
  g.out = out;
  g.ldo = ldo;
  g.out_f32 = out_dtype == KL_OUT_F32;
  g.force = kernel;
  const cudaError_t e = launch_gemm_fp8(g, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KL_OK : cuda_fail(e);
}
