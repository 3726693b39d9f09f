// The 4-bit (MXFP4, see mxfp4.cuh) cache: rows written into it and read back,
// and the operands of the 4-bit product.
//
// All three are one pass over memory on CUDA cores: a thread holds eight
// neighbouring values (16 bytes of bf16, one 32-bit word of codes), so every
// access of a warp is contiguous, four lanes hold one block of 32 (its
// largest magnitude takes two shuffles), and each thread has kUnroll
// independent loads in flight.
#include <algorithm>

#include "kernels.h"
#include "mxfp4.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// Largest magnitude over the four lanes that share a block.
CSA_DEV uint32_t block_amax(uint32_t a) {
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  return max(a, __shfl_xor_sync(0xffffffffu, a, 2));
}

// The scale bytes of the four blocks of 16 lanes as one word (every lane).
CSA_DEV uint32_t scale_word(uint32_t s, int lane) {
  uint32_t v = s << (8 * ((lane >> 2) & 3));
  v |= __shfl_xor_sync(0xffffffffu, v, 4);
  return v | __shfl_xor_sync(0xffffffffu, v, 8);
}

// The rows of one sequence: row i of the call is cache entry first + i.
struct Range {
  int64_t first, count;
  CSA_DEV Range(const int64_t* f, const int64_t* c, int b, int64_t n)
      : first(f ? f[b] : 0), count(c ? c[b] : n) {
    if (count > n) count = n;
  }
  // first + i lies in [0, n_cap) (no sum that could overflow).
  CSA_DEV bool inside(int64_t i, int64_t n_cap) const {
    return first >= 0 ? first < n_cap - i : first >= -i && first + i < n_cap;
  }
  // So do all of rows i .. i + k - 1, none past the count.
  CSA_DEV bool whole(int64_t i, int k, int64_t n_cap) const {
    return i + k <= count && first >= 0 && first <= n_cap - (i + k);
  }
};

struct WriteArgs {
  const uint8_t* rows;  // [B] sequences of n rows of d bf16, seq_bytes apart
  int64_t seq_bytes, n, n_cap;
  const int64_t* first;
  const int64_t* count;
  uint8_t* cache;       // [B, n_cap, row bytes]
  int32_t* status;
};

// blockIdx.y = sequence, kRows of its n rows per CTA.  A thread keeps its chunk
// (8 values) of the row and steps over rows, so its addresses are one sum.
// kWhole: every row of the CTA is written and lies in the cache (most CTAs),
// so no row is checked: the checks cost as much as the conversion.
template <int D>
struct Rows {
  static constexpr int kC = D / 8;              // chunks per row
  static constexpr int kStep = kThreads / kC;   // rows a step
  static constexpr int kRows = kStep * kUnroll;
};

template <int D, bool kWhole>
CSA_DEV void write_rows(const WriteArgs& a, const Range& rg) {
  using C = Rows<D>;
  constexpr int kRow = mx_row_bytes(D);
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int j = threadIdx.x % C::kC;  // chunk within the row
  const int64_t i0 = (int64_t)blockIdx.x * C::kRows + threadIdx.x / C::kC;
  const uint8_t* src = a.rows + (int64_t)b * a.seq_bytes + i0 * (2 * D) + 16 * j;
  uint4 v[kUnroll];
  bool live[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    live[u] = true;
    if (!kWhole) {
      const int64_t i = i0 + u * C::kStep;
      live[u] = i < rg.count;
      if (live[u] && !rg.inside(i, a.n_cap)) {
        report(a.status, CSA_ERR_DEVICE_INDEX);
        live[u] = false;
      }
    }
    v[u] = live[u] ? __ldcg(reinterpret_cast<const uint4*>(src + u * C::kStep * (2 * D)))
                   : make_uint4(0, 0, 0, 0);
  }
  uint8_t* row = a.cache + ((int64_t)b * a.n_cap + rg.first + i0) * kRow;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    const uint32_t s = mx_scale_byte(block_amax(mx_amax8(w)));
    const uint32_t codes = mx_quantise8(w, s), sw = scale_word(s, lane);
    if (live[u]) {
      uint8_t* at = row + u * C::kStep * kRow;
      *reinterpret_cast<uint32_t*>(at + 4 * j) = codes;
      if ((j & 15) == 0) *reinterpret_cast<uint32_t*>(at + D / 2 + j / 4) = sw;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const WriteArgs a) {
  pdl_head();
  const Range rg(a.first, a.count, blockIdx.y, a.n);
  if (rg.whole((int64_t)blockIdx.x * Rows<D>::kRows, Rows<D>::kRows, a.n_cap))
    write_rows<D, true>(a, rg);
  else
    write_rows<D, false>(a, rg);
}

struct ReadArgs {
  const uint8_t* cache;
  int64_t n, n_cap;
  const int32_t* idx;  // [B, n] or null
  const int64_t* first;
  const int64_t* count;
  uint8_t* rows;       // [B, n, d] bf16
  int32_t* status;
};

// kWhole: as in write_rows, and no index list.
template <int D, bool kWhole>
CSA_DEV void read_rows(const ReadArgs& a, const Range& rg) {
  using C = Rows<D>;
  constexpr int kRow = mx_row_bytes(D);
  const int b = blockIdx.y;
  const int j = threadIdx.x % C::kC;
  const int64_t i0 = (int64_t)blockIdx.x * C::kRows + threadIdx.x / C::kC;
  const uint8_t* src = a.cache + (int64_t)b * a.n_cap * kRow;
  uint32_t codes[kUnroll], s[kUnroll];
  bool live[kUnroll];
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = i0 + u * C::kStep;
    live[u] = true;
    int64_t e = (int64_t)((uint64_t)rg.first + (uint64_t)i);
    if (!kWhole) {
      live[u] = i < rg.count;
      if (live[u]) {
        bool ok;
        if (a.idx) {
          e = a.idx[(int64_t)b * a.n + i];
          ok = e >= 0 && e < a.n_cap;
          if (e == -1) live[u] = false;  // padding of a selection: nothing to read
        } else {
          ok = rg.inside(i, a.n_cap);
        }
        if (live[u] && !ok) {
          report(a.status, CSA_ERR_DEVICE_INDEX);
          live[u] = false;
        }
      }
    }
    codes[u] = s[u] = 0;
    if (live[u]) {
      const uint8_t* row = src + e * kRow;
      codes[u] = __ldcg(reinterpret_cast<const uint32_t*>(row + 4 * j));
      s[u] = __ldcg(row + D / 2 + j / 4);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) top = max(top, s[u]);
  const bool wide = __any_sync(0xffffffffu, top > 128u);  // a second factor is needed
  uint8_t* dst = a.rows + ((int64_t)b * a.n + i0) * (2 * D) + 16 * j;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    uint32_t o[4];
    mx_values8(codes[u], mx_bf16_lo(s[u]), o);
    if (wide) {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = mul_bf16x2(o[i], mx_bf16_hi(s[u]));
    }
    if (live[u])
      *reinterpret_cast<uint4*>(dst + u * C::kStep * (2 * D)) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const ReadArgs a) {
  pdl_head();
  const Range rg(a.first, a.count, blockIdx.y, a.n);
  if (!a.idx && rg.whole((int64_t)blockIdx.x * Rows<D>::kRows, Rows<D>::kRows, a.n_cap))
    read_rows<D, true>(a, rg);
  else
    read_rows<D, false>(a, rg);
}

}  // namespace

cudaError_t launch_mx_cache_write(const MxCacheLaunch& c, cudaStream_t stream) {
  WriteArgs a{static_cast<const uint8_t*>(c.rows_in), c.seq_bytes, c.n, c.n_cap, c.first, c.count,
              static_cast<uint8_t*>(c.cache), c.status};
  const int rows = c.d == 512 ? Rows<512>::kRows : Rows<128>::kRows;
  const int64_t gx = (c.n + rows - 1) / rows;
  if (gx == 0) return cudaSuccess;
  if (gx > 0x7FFFFFFF || c.B > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)gx, (unsigned)c.B);
  if (c.d == 512) return launch_pdl(cache_write_kernel<512>, grid, dim3(kThreads), 0, stream, 0, 1, a);
  if (c.d == 128) return launch_pdl(cache_write_kernel<128>, grid, dim3(kThreads), 0, stream, 0, 1, a);
  return cudaErrorInvalidValue;
}

cudaError_t launch_mx_cache_read(const MxCacheLaunch& c, cudaStream_t stream) {
  ReadArgs a{static_cast<const uint8_t*>(c.cache), c.n, c.n_cap, c.idx, c.first, c.count,
             static_cast<uint8_t*>(c.rows_out), c.status};
  const int rows = c.d == 512 ? Rows<512>::kRows : Rows<128>::kRows;
  const int64_t gx = (c.n + rows - 1) / rows;
  if (gx == 0) return cudaSuccess;
  if (gx > 0x7FFFFFFF || c.B > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)gx, (unsigned)c.B);
  if (c.d == 512) return launch_pdl(cache_read_kernel<512>, grid, dim3(kThreads), 0, stream, 0, 1, a);
  if (c.d == 128) return launch_pdl(cache_read_kernel<128>, grid, dim3(kThreads), 0, stream, 0, 1, a);
  return cudaErrorInvalidValue;
}

}  // namespace csa
