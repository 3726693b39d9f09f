// Grouped output projection in MXFP4 (see mxfp4.cuh for the format): weights
// held in 4 bits, activations quantised per token in blocks of 32 along the
// inner dimension, products on the 5th-generation tensor cores with their
// block scales (tcgen05.mma kind::mxf4), fp32 accumulation.
//
//   y[t, j*d_g + r] = bf16( sum_c W_g[j, r, c] * q(o)[t, j*H/g*D + c] )
//   z[t, n]         = bf16( sum_i W_o[n, i]    * q(y)[t, i] )
//
// with q() the quantisation to MXFP4.  (The passages and the bf16 form: see
// proj.cu.)
//
// One operand layout serves weights and activations: codes [rows, K/2]
// row-major, loaded by TMA (128 bytes = 256 values a row and chunk, 128-byte
// swizzle), and scale bytes in tiles of 128 rows x 4 blocks (512 bytes: byte
// (r % 32) * 16 + (r % 128) / 32 * 4 + block % 4), the form in which
// tcgen05.cp brings them to tensor memory (32 lanes x 16 bytes, replicated to
// the four lane quarters): row r's four bytes sit in lane r % 32, column
// r / 32.
//
// A chunk of 256 K values is 4 MMAs of K = 64.  Each ring stage has its own
// scale columns in tensor memory, so a stage's copies are issued only after
// the MMAs that read its former scales have completed (its `full` barrier
// follows its `empty` barrier).
//
// Up to 256 tokens, and for feature counts that are no multiple of 256, two forms
// of one kernel (mx_gemm_kernel):
//   - few tokens (T <= 128): weights are the MMA's M = 128 rows, tokens its N.
//     The weights' bytes bound it.
//   - more tokens: tokens are the M = 128 rows, weights N = 128, so that a
//     thread of the epilogue holds one token's neighbouring features and
//     quantises y in registers.
// Either way K is split over the CTAs of a cluster where the tiles alone do
// not fill the SMs (two CTAs each); the CTAs add their sums up over shared
// memory, in the order of the splits, and finish the tile's tokens.
// More tokens go to a second kernel, on CTA pairs (mx_pair_kernel).
#include <algorithm>
#include <atomic>

#include "kernels.h"
#include "mxfp4.cuh"
#include "tma.h"

namespace csa {
namespace {

constexpr int kThreads = 192;
constexpr int BM = 128;         // rows of the MMA's A operand
constexpr int KB = 128;         // bytes of a row and chunk (256 values)
constexpr int kScaleTile = 512; // scale bytes of 128 rows x 128 values

CSA_DEV uint64_t desc_kmaj(uint32_t saddr) { return sdesc_sw128(saddr, 16, 1024); }

// Scale tile in shared memory: 32 rows of 16 bytes, no swizzle (8-row groups
// 128 bytes apart).
CSA_DEV uint64_t desc_scale(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}

// kind::mxf4 (E2M1 operands, E8M0 scales per 32 values, K = 64, K-major,
// fp32 accumulator); `id` selects the half (0 or 2) of the 4 scale bytes.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, int id) {
  return ((uint32_t)id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 4) << 24) | ((uint32_t)id << 29);
}

CSA_DEV void mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                      uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;"
      "\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sa_tmem), "r"(sb_tmem)
      : "memory");
}

// 512 bytes of shared memory -> 4 columns of 32 lanes, in every lane quarter.
CSA_DEV void copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// `bytes` (a multiple of 16) of global memory into shared memory, on bar.
CSA_DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

struct GemmArgs {
  const uint8_t* tok_scale;  // token scale tiles [ceil(T/128), tok_k/128, 512]
  const uint8_t* w_scale;    // weight scale tiles [w_rows/128, K/128, 512]
  int T, chunks;             // tokens; K chunks per group
  int64_t tok_tiles, w_tiles;  // scale tiles per 128 rows (of all groups; of one)
  int groups_k;              // token chunks between groups (= chunks)
  int N, splits, ldc;        // output features per group; K splits; features in all
  __nv_bfloat16* c;          // [T, ldc] bf16 or null, and with yq != null
  uint8_t* yq;               // codes [T, ldc/2] and
  uint8_t* ys;               // scale tiles [ceil(T/128), ldc/128, 512] of the bf16 values
  int32_t* status;
};

// One 32-value block of a token's row (fp32 in v): bf16 into c, and quantised
// into the next product's operand (yq, and its scale byte returned).
CSA_DEV uint32_t store_block(const GemmArgs& p, int t, int k, const uint32_t* v, bool live) {
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j)
    w[j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
  if (live && p.c) {
    uint4* dst = reinterpret_cast<uint4*>(p.c + (int64_t)t * p.ldc + k);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      dst[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  }
  if (!p.yq) return 0;
  uint32_t am = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    am = max(am, mx_amax8(*reinterpret_cast<const uint32_t(*)[4]>(&w[4 * j])));
  const uint32_t sb = mx_scale_byte(am);
  uint32_t cd[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    cd[j] = mx_quantise8(*reinterpret_cast<const uint32_t(*)[4]>(&w[4 * j]), sb);
  if (live)
    *reinterpret_cast<uint4*>(p.yq + (int64_t)t * (p.ldc / 2) + k / 2) =
        make_uint4(cd[0], cd[1], cd[2], cd[3]);
  return sb;
}
// Where the four scale bytes of token t, columns k/128*128 .. + 127 are.
CSA_DEV uint8_t* scale_word_at(const GemmArgs& p, int t, int k) {
  return p.ys + ((int64_t)(t / 128) * (p.ldc / 128) + k / 128) * kScaleTile + (t % 32) * 16 +
         (t % 128) / 32 * 4;
}
CSA_DEV void store_scales(const GemmArgs& p, int t, int k, uint32_t word) {
  *reinterpret_cast<uint32_t*>(scale_word_at(p, t, k)) = word;
}

// Four values per lane, the 128 features of a tile row (k = its feature
// 4 * lane): bf16 into c, and quantised into the next product's operand.
CSA_DEV void store_quad(const GemmArgs& p, int t, int k, const float4& x, int lane) {
  const uint32_t w[4] = {pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), 0u, 0u};
  if (p.c) *reinterpret_cast<uint2*>(p.c + (int64_t)t * p.ldc + k) = make_uint2(w[0], w[1]);
  if (!p.yq) return;
  uint32_t am = mx_amax8(w);
  am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
  am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
  am = max(am, __shfl_xor_sync(0xffffffffu, am, 4));
  const uint32_t sb = mx_scale_byte(am);
  *reinterpret_cast<uint16_t*>(p.yq + (int64_t)t * (p.ldc / 2) + k / 2) =
      (uint16_t)mx_quantise8(w, sb);
  uint32_t word = sb << (8 * (lane >> 3));
  word |= __shfl_xor_sync(0xffffffffu, word, 8);
  word |= __shfl_xor_sync(0xffffffffu, word, 16);
  if (lane == 0) store_scales(p, t, k, word);
}

CSA_DEV float4 ld_cluster_v4(uint32_t caddr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(caddr)
               : "memory");
  return v;
}

constexpr int kSumRow = 132;  // floats per token of the sums (padded: spreads the banks)

template <int BN, bool kTokM>
struct Cfg {
  static constexpr int kABytes = BM * KB;
  static constexpr int kBBytes = BN * KB;
  static constexpr int kScaleBytes = 4 * kScaleTile;       // two tiles of A, two of B
  static constexpr int kStageBytes = kABytes + kBBytes + kScaleBytes;
  static constexpr int kStages = 103 * 1024 / kStageBytes; // two CTAs per SM
  static constexpr int kScaleCols = 16;                    // columns of a stage's scales
  static constexpr int kCols0 = (BN < 32 ? 32 : BN) + kStages * kScaleCols;
  static constexpr uint32_t kCols = kCols0 <= 128 ? 128 : 256;
  static_assert(BN <= 128 && kStages >= 2 && kCols0 <= 256, "tensor memory of two CTAs");
  static_assert(kStages * (kABytes + kBBytes) >= (kTokM ? BM : BN) * kSumRow * 4, "the sums");
};

template <int BN, bool kTokM>
__global__ void __launch_bounds__(kThreads)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap map_tok,
                   const __grid_constant__ CUtensorMap map_w, const GemmArgs p) {
  using C = Cfg<BN, kTokM>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  // Codes first (1024-byte aligned), then every stage's scale tiles.
  uint8_t* scales = smem + C::kStages * (C::kABytes + C::kBBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + C::kStages * C::kScaleBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* accf = empty + C::kStages;  // the accumulator is complete
  uint64_t* drain = accf + 1;           // issued MMAs finished (abort path)
  uint64_t* done = drain + 1;           // one arrival per warp when its role is over
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* sums = reinterpret_cast<float*>(smem);  // [tokens][kSumRow], over the ring

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int group = blockIdx.z, split = blockIdx.x % p.splits;
  // The chunks [k0, k1) of the group's inner dimension.
  const int k0 = (int)((int64_t)p.chunks * split / p.splits);
  const int nk = (int)((int64_t)p.chunks * (split + 1) / p.splits) - k0;
  const int w_tile = kTokM ? BN : BM, t_tile = kTokM ? BM : BN;
  const int n0 = blockIdx.x / p.splits * w_tile;  // first feature within the group
  const int t0 = blockIdx.y * t_tile;   // first token
  const int w_row = group * p.N + n0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(accf, 1);
    mbar_init(drain, 1);
    mbar_init(done, kThreads / 32);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_scale = tmem + (BN < 32 ? 32 : BN);
  pdl_trigger();  // the next kernel may set itself up while this one runs

  if (warp == 0) {
    // ---------------------------------------------------------- producer --
    // Weights are caller inputs: the first ring's worth is requested before
    // the wait on the previous kernel, which writes the tokens' operand.
    if (elect_one()) {
      tma_prefetch_desc(&map_tok);
      tma_prefetch_desc(&map_w);
      constexpr int kS = C::kStages;
      auto weights = [&](int it) {
        const int s = it % kS;
        uint8_t* st = smem + s * (C::kABytes + C::kBBytes);
        uint8_t* sc = scales + s * C::kScaleBytes;
        mbar_expect_tx(&full[s], C::kStageBytes);
        tma_load_2d(st + (kTokM ? C::kABytes : 0), &map_w, &full[s], (k0 + it) * KB, w_row);
        bulk_load(sc + (kTokM ? 2 * kScaleTile : 0),
                  p.w_scale + (w_row / 128 * p.w_tiles + 2 * (k0 + it)) * kScaleTile,
                  2 * kScaleTile, &full[s]);
      };
      auto tokens = [&](int it) {
        const int s = it % kS;
        uint8_t* st = smem + s * (C::kABytes + C::kBBytes);
        uint8_t* sc = scales + s * C::kScaleBytes;
        const int kc = group * p.groups_k + k0 + it;
        tma_load_2d(st + (kTokM ? 0 : C::kABytes), &map_tok, &full[s], kc * KB, t0);
        bulk_load(sc + (kTokM ? 0 : 2 * kScaleTile),
                  p.tok_scale + (t0 / 128 * p.tok_tiles + 2 * kc) * kScaleTile, 2 * kScaleTile,
                  &full[s]);
      };
      const int pre = nk < kS ? nk : kS;
      for (int it = 0; it < pre; ++it) weights(it);
      pdl_wait();
      for (int it = 0; it < pre; ++it) tokens(it);
      int it = pre;
      for (; it < nk; ++it) {
        if (!mbar_wait(&empty[it % kS], ((it / kS) & 1) ^ 1, p.status, abort_flag)) break;
        weights(it);
        tokens(it);
      }
      if (*abort_flag) {  // copies still in flight land before the CTA exits
        for (int j = it - kS > 0 ? it - kS : 0; j < it; ++j)
          mbar_wait(&full[j % kS], (j / kS) & 1, p.status);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------- MMA issuer --
    bool issued = false;
    for (int it = 0; it < nk; ++it) {
      const int s = it % C::kStages;
      const bool ok = mbar_wait(&full[s], (it / C::kStages) & 1, p.status, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t ab = smem_u32(smem + s * (C::kABytes + C::kBBytes)), bb = ab + C::kABytes;
        const uint32_t sc = smem_u32(scales + s * C::kScaleBytes);
        // Scale columns of the stage: A's two tiles, then B's (4 columns each).
        const uint32_t ta = t_scale + s * C::kScaleCols, tb = ta + 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          copy_scales(ta + 4 * h, desc_scale(sc + h * kScaleTile));
          copy_scales(tb + 4 * h, desc_scale(sc + (2 + h) * kScaleTile));
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_mxf4(tmem, desc_kmaj(ab + kk * 32), desc_kmaj(bb + kk * 32),
                   idesc_mxf4(BM, BN, 2 * (kk & 1)), ta + 4 * (kk >> 1),
                   tb + 4 * (kk >> 1), (it > 0 || kk > 0) ? 1u : 0u);
        mma_commit(&empty[s]);
        if (it == nk - 1) mma_commit(accf);
      }
      __syncwarp();
      issued = true;
    }
    if (*abort_flag && issued) {  // let issued MMAs finish before TMEM is freed
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      mbar_wait(drain, 0, p.status);
    }
  } else {
    // ---------------------------------------------------------- epilogue --
    const int q = warp & 3;
    const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16);
    const bool ok = mbar_wait(accf, 0, p.status, abort_flag);
    if (__all_sync(0xffffffffu, ok) && !*abort_flag) {
      tc_fence_after();
      if constexpr (!kTokM) {
        // Lane = feature, columns = tokens.  (Every chunk has been consumed:
        // the ring holds the sums.)
        float* dst = sums + 32 * q + lane;
#pragma unroll 1
        for (int c = 0; c < BN && t0 + c < p.T; c += 16) {
          uint32_t v[16];
          tmem_ld16(acc + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) dst[(c + j) * kSumRow] = __uint_as_float(v[j]);
        }
      } else {
        // Lane = token, columns = features.
        const int t = t0 + 32 * q + lane;
        const bool live = t < p.T;
        if (p.splits > 1) {
          float* dst = sums + (32 * q + lane) * kSumRow;
#pragma unroll 1
          for (int c = 0; c < BN; c += 32) {
            uint32_t v[32];
            tmem_ld32(acc + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint4*>(dst + c + j) =
                  make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
          }
        } else {
          uint32_t sw = 0;
#pragma unroll 1
          for (int c = 0; c < BN; c += 32) {
            uint32_t v[32];
            tmem_ld32(acc + c, v);
            tmem_wait_ld();
            sw |= store_block(p, t, w_row + c, v, live) << (c & 96) / 4;
            if ((c & 96) == 96) {
              if (live && p.yq) store_scales(p, t, w_row + c - 96, sw);
              sw = 0;
            }
          }
        }
      }
    }
  }
  // Teardown: every warp reports (converged) that it is done with tensor
  // memory; warp 0 frees it after all of them (bounded wait).
  __syncwarp();
  tc_fence_before();
  if (lane == 0) mbar_arrive(done);
  if (warp == 0) {
    mbar_wait(done, 0, p.status);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  if (kTokM && p.splits == 1) return;
  // The splits of a tile are one cluster: every CTA adds up some of the
  // tile's tokens (in the order of the splits) over the cluster's shared
  // memory and finishes them.  Every wait above is bounded, so every thread
  // of every CTA arrives here.
  __syncwarp();
  const bool cluster = p.splits > 1;
  if (cluster)
    cluster_sync();
  else
    __syncthreads();
  const int nt = min(t_tile, p.T - t0);
  for (int i = split + p.splits * warp; i < nt; i += p.splits * (kThreads / 32)) {
    // Lane: features 4 * lane .. + 3 of token i.
    const uint32_t at = smem_u32(sums + i * kSumRow + 4 * lane);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (cluster) {
#pragma unroll 4
      for (int s = 0; s < p.splits; ++s) {
        const float4 v = ld_cluster_v4(mapa(at, s));
        x.x += v.x;
        x.y += v.y;
        x.z += v.z;
        x.w += v.w;
      }
    } else {
      x = *reinterpret_cast<const float4*>(sums + i * kSumRow + 4 * lane);
    }
    store_quad(p, t0 + i, w_row + 4 * lane, x, lane);
  }
  if (cluster) cluster_sync();  // no CTA leaves while another reads its sums
}

// ------------------------------------------------------------- CTA pairs --
// Many tokens: tiles of 256 tokens x 256 features on pairs of CTAs
// (cta_group::2).  Each CTA loads its 128 tokens and half of the weight rows,
// so a chunk costs an SM 35 KB from L2 for 128 x 256 x 256 products (48 KB
// where each CTA loads a whole 256-row weight tile: that form was bound by L2
// at 12 TB/s).  The grid is persistent (one CTA per SM); the epilogue's eight
// warps take the accumulator into registers at once, so the next tile's MMAs
// start while they convert and store it.  Where the last round of tiles would
// leave half of the pairs or more idle, its tiles are cut into two of 128
// features.
constexpr int kPairThreads = 320;  // producer, MMA, eight epilogue warps
struct Pair {
  static constexpr int kStages = 6;
  static constexpr int kOperand = BM * KB;            // 128 token rows, or 128 weight rows
  static constexpr int kScaleBytes = 6 * kScaleTile;  // the tokens' tiles, all weight rows'
  static constexpr int kStageBytes = 2 * kOperand + kScaleBytes;
  static constexpr int kScaleCols = 24;               // A 2 x 4, B 2 x 8 columns
  static constexpr int kAccCols = 256;
  static constexpr uint32_t kCols = 512;
  static_assert(kAccCols + kStages * kScaleCols <= 512, "tensor memory");
};

// Work item i of the launch: a whole tile, or (the last round) half of one.
struct PairItem {
  int m, n, half;  // half: 0 / 1, or -1 for a whole tile
  CSA_DEV PairItem(int i, int m_tiles, int whole) {
    half = i < whole ? -1 : (i - whole) & 1;
    const int tile = i < whole ? i : whole + ((i - whole) >> 1);
    m = tile % m_tiles;
    n = tile / m_tiles;
  }
};

CSA_DEV void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x,
                              int32_t y) {
  // The bytes count on the even CTA's barrier (bit 24 of the cluster shared
  // address tells the CTAs of a pair apart).
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar) & 0xFEFFFFFFu), "r"(x), "r"(y)
      : "memory");
}
CSA_DEV void mma_mxf4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                           uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;"
      "\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sa_tmem), "r"(sb_tmem)
      : "memory");
}
CSA_DEV void copy_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
// Arrive on `bar` of both CTAs when the pair's earlier MMAs have completed.
CSA_DEV void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

__global__ void __launch_bounds__(kPairThreads, 1)
    mx_pair_kernel(const __grid_constant__ CUtensorMap map_tok,
                   const __grid_constant__ CUtensorMap map_w,
                   const __grid_constant__ CUtensorMap map_ts,
                   const __grid_constant__ CUtensorMap map_ws, const GemmArgs p) {
  using C = Pair;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* scales = smem + C::kStages * 2 * C::kOperand;
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + C::kStages * C::kScaleBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* accf = empty + C::kStages;  // a tile's accumulator is complete
  uint64_t* acce = accf + 1;            // (even CTA) both CTAs have read it
  uint64_t* drain = acce + 1;           // issued MMAs finished (abort path)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)cluster_ctarank();
  const int m_tiles = (p.T + 255) / 256, n_group = p.N / 256;
  const int tiles = m_tiles * (p.ldc / 256);
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  // Items [0, whole) are tiles, the others halves of the remaining ones.
  const int rest = tiles % step;
  const int whole = 2 * rest <= step ? tiles - rest : tiles;
  const int items = whole + 2 * (tiles - whole);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(accf, 1);
    mbar_init(acce, 16);  // eight epilogue warps of either CTA
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers and tensor memory are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();

  if (warp == 0) {
    // ---------------------------------------------------------- producer --
    if (elect_one()) {
      tma_prefetch_desc(&map_tok);
      tma_prefetch_desc(&map_w);
      tma_prefetch_desc(&map_ts);
      tma_prefetch_desc(&map_ws);
      pdl_wait();
      int it = 0;
      bool ok = true;
      for (int i = first; ok && i < items; i += step) {
        const PairItem w(i, m_tiles, whole);
        const int kg = w.n / n_group * p.chunks;  // the group's first token chunk
        // Half a tile: 64 weight rows each (the box loads 64 more, unused).
        const int w_row = w.n * 256 + (w.half < 0 ? rank * 128 : w.half * 128 + rank * 64);
        const int ts_row = (int32_t)((2 * w.m + rank) * p.tok_tiles) + 2 * kg;
        const int ws_row0 = (int32_t)((2 * w.n + max(w.half, 0)) * p.w_tiles);
        const int ws_row1 = (int32_t)((2 * w.n + 1) * p.w_tiles);
        for (int c = 0; c < p.chunks; ++c, ++it) {
          const int s = it % C::kStages;
          if (!mbar_wait(&empty[s], ((it / C::kStages) & 1) ^ 1, p.status, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + s * 2 * C::kOperand;
          uint8_t* sc = scales + s * C::kScaleBytes;
          if (rank == 0) mbar_expect_tx(&full[s], 2 * C::kStageBytes);
          tma_load_2d_pair(st, &map_tok, &full[s], (kg + c) * KB, w.m * 256 + rank * 128);
          tma_load_2d_pair(st + C::kOperand, &map_w, &full[s], c * KB, w_row);
          // (Scale tiles past the last token lie past the map: zeros.)
          tma_load_2d_pair(sc, &map_ts, &full[s], 0, ts_row + 2 * c);
          tma_load_2d_pair(sc + 2 * kScaleTile, &map_ws, &full[s], 0, ws_row0 + 2 * c);
          tma_load_2d_pair(sc + 4 * kScaleTile, &map_ws, &full[s], 0, ws_row1 + 2 * c);
        }
      }
      // The MMAs' last arrivals on `empty` come from the even CTA: they land
      // before this CTA leaves.
      for (int j = it - C::kStages > 0 ? it - C::kStages : 0; ok && j < it; ++j)
        ok = mbar_wait(&empty[j % C::kStages], (j / C::kStages) & 1, p.status, abort_flag);
      if (*abort_flag) {  // copies still in flight land before the CTA exits
        if (rank == 0)
          for (int j = it - C::kStages > 0 ? it - C::kStages : 0; j < it; ++j)
            mbar_wait(&full[j % C::kStages], (j / C::kStages) & 1, p.status);
        // (The odd CTA's copies count on the even CTA's barriers: wait out
        // their latency.)
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------- MMA issuer --
    if (rank == 0) {
      const uint32_t t_scale = tmem + C::kAccCols;
      bool issued = false, ok = true;
      int it = 0, j = 0;
      for (int i = first; ok && i < items; i += step, ++j) {
        const bool half = i >= whole;
        if (j > 0) {
          ok = mbar_wait<true>(acce, (j - 1) & 1, p.status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
        }
        for (int c = 0; ok && c < p.chunks; ++c, ++it) {
          const int s = it % C::kStages;
          ok = mbar_wait<true>(&full[s], (it / C::kStages) & 1, p.status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t ab = smem_u32(smem + s * 2 * C::kOperand), bb = ab + C::kOperand;
            const uint32_t sc = smem_u32(scales + s * C::kScaleBytes);
            const uint32_t ta = t_scale + s * C::kScaleCols, tb = ta + 8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              copy_scales_pair(ta + 4 * h, desc_scale(sc + h * kScaleTile));
#pragma unroll
              for (int b = 0; b < 2; ++b)
                copy_scales_pair(tb + 8 * h + 4 * b,
                                 desc_scale(sc + ((1 + b) * 2 + h) * kScaleTile));
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_mxf4_pair(tmem, desc_kmaj(ab + kk * 32), desc_kmaj(bb + kk * 32),
                            idesc_mxf4(256, half ? 128 : 256, 2 * (kk & 1)), ta + 4 * (kk >> 1),
                            tb + 8 * (kk >> 1), (c > 0 || kk > 0) ? 1u : 0u);
            mma_commit_pair(&empty[s]);
            if (c == p.chunks - 1) mma_commit_pair(accf);
          }
          __syncwarp();
          issued = true;
        }
      }
      if (*abort_flag && issued) {  // let issued MMAs finish before TMEM is freed
        if (elect_one())
          asm volatile(
              "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                  smem_u32(drain))
              : "memory");
        __syncwarp();
        mbar_wait(drain, 0, p.status);
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue --
    // Two warps per lane quarter, 128 columns each (64 of a half tile); lane =
    // token.
    const int q = warp & 3, side = (warp - 2) >> 2;
    const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16);
    const uint32_t acce0 = mapa(smem_u32(acce), 0);
    int j = 0;
    for (int i = first; i < items; i += step, ++j) {
      const PairItem w(i, m_tiles, whole);
      const bool ok = mbar_wait<true>(accf, j & 1, p.status, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const int cols = w.half < 0 ? 128 : 64;
      uint32_t v[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (32 * c < cols) tmem_ld32(acc + side * cols + 32 * c, v[c]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(acce0);
      const int t = w.m * 256 + rank * 128 + 32 * q + lane;
      const int k = w.n * 256 + max(w.half, 0) * 128 + side * cols;
      const bool live = t < p.T;
      uint32_t sw = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (32 * c < cols) sw |= store_block(p, t, k + 32 * c, v[c], live) << (8 * c);
      if (live && p.yq) {
        if (w.half < 0)
          store_scales(p, t, k, sw);
        else
          *reinterpret_cast<uint16_t*>(scale_word_at(p, t, k) + 2 * side) = (uint16_t)sw;
      }
    }
  }
  // Every wait above is bounded, so every thread of both CTAs arrives here;
  // after it nothing of the pair reads the other's memory.
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols)
                 : "memory");
}

// Rows of bf16 -> operand (codes and scale tiles).  blockIdx.x: 256 columns,
// blockIdx.y: 128 rows, a warp per row: 512 bytes read and one full line of
// codes written at a time.  The scale bytes of rows past the last one are
// written as zeros.
__global__ void __launch_bounds__(256) mx_quantise_kernel(const uint8_t* x, int64_t ld_bytes,
                                                          int64_t rows, int64_t cols,
                                                          uint8_t* codes, uint8_t* scales,
                                                          int head) {
  constexpr int kU = 8;  // rows in flight per warp
  if (head)
    pdl_head();
  else
    pdl_trigger();
  __shared__ __align__(16) uint8_t sc[2][kScaleTile];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r0 = (int64_t)blockIdx.y * 128, k0 = (int64_t)blockIdx.x * 256;
  const bool in = k0 + 8 * lane < cols;
  const uint8_t* src = x + (r0 + warp) * ld_bytes + (k0 + 8 * lane) * 2;
  uint8_t* dst = codes + (r0 + warp) * (cols / 2) + (k0 + 8 * lane) / 2;
  const int live = (int)min((int64_t)128, rows - r0);
  if (threadIdx.x < 2 * kScaleTile / 16)  // rows past the last one: zeros
    reinterpret_cast<uint4*>(&sc[0][0])[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
#pragma unroll 1
  for (int g = 0; g < live; g += 8 * kU) {
    uint4 v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      v[u] = in && warp + g + 8 * u < live
                 ? __ldcg(reinterpret_cast<const uint4*>(src + (int64_t)(g + 8 * u) * ld_bytes))
                 : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int r = warp + g + 8 * u;
      if (r >= live) break;  // the same for the whole warp
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      uint32_t am = mx_amax8(w);
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      const uint32_t s = mx_scale_byte(am), cd = mx_quantise8(w, s);
      uint32_t b = s << (8 * ((lane >> 2) & 3));
      b |= __shfl_xor_sync(0xffffffffu, b, 4);
      b |= __shfl_xor_sync(0xffffffffu, b, 8);
      if (in)
        *reinterpret_cast<uint32_t*>(dst + (int64_t)(g + 8 * u) * (cols / 2)) = cd;
      if ((lane & 15) == 0)
        *reinterpret_cast<uint32_t*>(&sc[lane >> 4][(r % 32) * 16 + r / 32 * 4]) = b;
    }
  }
  __syncthreads();
  const int64_t tile = (int64_t)blockIdx.y * (cols / 128) + 2 * blockIdx.x;
  const int i = threadIdx.x;  // 16 bytes of the two tiles each
  if (i < 2 * kScaleTile / 16 && k0 + 128 * (i / (kScaleTile / 16)) < cols)
    reinterpret_cast<uint4*>(scales + tile * kScaleTile)[i] =
        reinterpret_cast<const uint4*>(&sc[0][0])[i];
}

template <int BN, bool kTokM>
cudaError_t launch_gemm(const MxGemm& g, cudaStream_t stream) {
  using C = Cfg<BN, kTokM>;
  CUtensorMap map_tok, map_w;
  cudaError_t e = make_tmap_2d(&map_tok, g.tok, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)g.T,
                               (uint64_t)g.tok_k / 2, kTokM ? BM : BN, KB,
                               CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  e = make_tmap_2d(&map_w, g.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)g.groups * g.N,
                   (uint64_t)g.K / 2, kTokM ? BN : BM, KB, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  GemmArgs p{};
  p.tok_scale = static_cast<const uint8_t*>(g.tok_scale);
  p.w_scale = static_cast<const uint8_t*>(g.w_scale);
  p.T = g.T;
  p.chunks = g.K / 256;
  p.tok_tiles = g.tok_k / 128;
  p.w_tiles = g.K / 128;
  p.groups_k = p.chunks;
  p.N = g.N;
  p.ldc = g.groups * g.N;
  p.c = static_cast<__nv_bfloat16*>(g.c);
  p.yq = static_cast<uint8_t*>(g.yq);
  p.ys = static_cast<uint8_t*>(g.ys);
  p.status = g.status;
  const size_t smem = 1024 + (size_t)C::kStages * C::kStageBytes + (2 * C::kStages + 3) * 8 + 16;
  auto kern = mx_gemm_kernel<BN, kTokM>;
  int slot = kTokM ? 30 : 26;
  if (!kTokM)
    for (int b = 16; b < BN; b <<= 1) ++slot;
  e = ensure_smem_attr(reinterpret_cast<const void*>(kern), slot, smem);
  if (e != cudaSuccess) return e;
  const int x = g.N / (kTokM ? BN : BM), y = (g.T + (kTokM ? BM : BN) - 1) / (kTokM ? BM : BN);
  // K splits (one cluster per tile): a power of two of CTAs, as many as fit
  // beside each other (two on an SM; clusters leave some SMs of a GPC over),
  // at least four chunks each.  8 tokens, 16 groups to 1024 and 7168 features
  // (128 and 56 tiles, so 2 and 4 splits): 25.5 us; 28.9 with 1 and 2, 30.9
  // with 4 and 2.
  const int64_t slots = 2 * (int64_t)device_sm_count();
  p.splits = 1;
  while (p.splits < 8 && 8 * (int64_t)x * y * g.groups * p.splits * 2 <= 7 * slots &&
         p.chunks >= 4 * p.splits * 2)
    p.splits *= 2;
  return launch_pdl(kern, dim3(x * p.splits, y, g.groups), dim3(kThreads), smem, stream,
                    p.splits > 1 ? p.splits : 0, g.chained, map_tok, map_w, p);
}

// Pairs of CTAs that can be resident at once on the current device (one
// persistent pair each); cached per device.
int pairs_resident(size_t smem) {
  static std::atomic<int> cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return std::max(1, device_sm_count() / 2);
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n) return n;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kPairThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, mx_pair_kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();  // a refused query is not the caller's error
    n = std::max(1, device_sm_count() / 2);
  }
  cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

cudaError_t launch_pair(const MxGemm& g, cudaStream_t stream) {
  using C = Pair;
  CUtensorMap map_tok, map_w, map_ts, map_ws;
  cudaError_t e = make_tmap_2d(&map_tok, g.tok, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)g.T,
                               (uint64_t)g.tok_k / 2, BM, KB, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  e = make_tmap_2d(&map_w, g.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)g.groups * g.N,
                   (uint64_t)g.K / 2, BM, KB, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  // Scale tiles as rows of 128 words, two neighbouring tiles a load.
  const uint64_t t_rows = (uint64_t)(g.T + 127) / 128 * (g.tok_k / 128);
  const uint64_t w_rows = (uint64_t)g.groups * g.N / 128 * (g.K / 128);
  e = make_tmap_2d(&map_ts, g.tok_scale, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, t_rows,
                   kScaleTile / 4, 2, kScaleTile / 4, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (e != cudaSuccess) return e;
  e = make_tmap_2d(&map_ws, g.w_scale, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, w_rows, kScaleTile / 4,
                   2, kScaleTile / 4, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (e != cudaSuccess) return e;
  GemmArgs p{};
  p.T = g.T;
  p.chunks = g.K / 256;
  p.tok_tiles = g.tok_k / 128;
  p.w_tiles = g.K / 128;
  p.N = g.N;
  p.ldc = g.groups * g.N;
  p.c = static_cast<__nv_bfloat16*>(g.c);
  p.yq = static_cast<uint8_t*>(g.yq);
  p.ys = static_cast<uint8_t*>(g.ys);
  p.status = g.status;
  const size_t smem = 1024 + (size_t)C::kStages * C::kStageBytes + (2 * C::kStages + 3) * 8 + 16;
  e = ensure_smem_attr(reinterpret_cast<const void*>(mx_pair_kernel), 31, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)((g.T + 255) / 256) * (p.ldc / 256);
  // Up to twice as many pairs as tiles: those of a last round may be halved.
  const int pairs = (int)std::min<int64_t>(2 * tiles, pairs_resident(smem));
  return launch_pdl(mx_pair_kernel, dim3(2 * pairs), dim3(kPairThreads), smem, stream, 2, g.chained,
                    map_tok, map_w, map_ts, map_ws, p);
}

}  // namespace

cudaError_t launch_mx_quantise(const void* x, int64_t ld, int64_t rows, int64_t cols, void* codes,
                               void* scales, cudaStream_t stream) {
  const dim3 grid((unsigned)((cols + 255) / 256), (unsigned)((rows + 127) / 128));
  // Head mode where one wave of CTAs takes the rows (8 tokens: the whole
  // projection 25.8 us a call among others, 28.6 without; in a graph 24.5 and 25.4);
  // with many CTAs, each of which would start with the wait, it costs more than it
  // saves (4096 tokens: 473 us with, 452 without; in a short graph 406 and 379).
  const int head = rows <= 128;
  return launch_pdl(mx_quantise_kernel, grid, dim3(256), 0, stream, 0, head,
                    static_cast<const uint8_t*>(x), ld * 2, rows, cols,
                    static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), head);
}

cudaError_t launch_mx_gemm(const MxGemm& g, cudaStream_t stream) {
  if (g.T < 1 || g.N % 128 || g.K % 256) return cudaErrorInvalidValue;
  if ((g.T + 127) / 128 > 65535 || g.groups > 65535) return cudaErrorInvalidConfiguration;
  if (g.T <= 16) return launch_gemm<16, false>(g, stream);
  if (g.T <= 32) return launch_gemm<32, false>(g, stream);
  if (g.T <= 64) return launch_gemm<64, false>(g, stream);
  if (g.T <= 128) return launch_gemm<128, false>(g, stream);
  // CTA pairs from the second tile of 256 tokens on (300 tokens, the sizes
  // above: 57 us, 65 with single CTAs; 200 tokens: 49 us, 45).  (Tile rows of
  // their scale maps are 32-bit coordinates.)
  const bool fits = ((int64_t)(g.T + 255) / 256 * 2 + 1) * (g.tok_k / 128) <= 0x7FFFFFFF;
  if (g.T > 256 && g.N % 256 == 0 && fits) return launch_pair(g, stream);
  return launch_gemm<128, true>(g, stream);
}

}  // namespace csa
