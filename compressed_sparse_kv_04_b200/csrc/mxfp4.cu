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
};

struct WriteArgs {
  const uint8_t* rows;  // [B] sequences of n rows of d bf16, seq_bytes apart
  int64_t seq_bytes, n, n_cap;
  const int64_t* first;
  const int64_t* count;
  uint8_t* cache;       // [B, n_cap, row bytes]
  int32_t* status;
};

// blockIdx.y = sequence; the chunks (8 values) of its n rows over blockIdx.x.
template <int D>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const WriteArgs a) {
  constexpr int kC = D / 8;  // chunks per row
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const Range rg(a.first, a.count, b, a.n);
  const int64_t c0 = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  const uint8_t* src = a.rows + (int64_t)b * a.seq_bytes;
  uint8_t* dst = a.cache + (int64_t)b * a.n_cap * mx_row_bytes(D);
  uint4 v[kUnroll];
  bool live[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t c = c0 + u * kThreads, i = c / kC;
    live[u] = i < rg.count;
    if (live[u] && !rg.inside(i, a.n_cap)) {
      report(a.status, CSA_ERR_DEVICE_INDEX);
      live[u] = false;
    }
    v[u] = live[u] ? __ldg(reinterpret_cast<const uint4*>(src + c * 16)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t c = c0 + u * kThreads, i = c / kC;
    const int j = (int)(c % kC);  // chunk within the row
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    const uint32_t s = mx_scale_byte(block_amax(mx_amax8(w)));
    const uint32_t codes = mx_quantise8(w, s), sw = scale_word(s, lane);
    if (live[u]) {
      uint8_t* row = dst + (rg.first + i) * mx_row_bytes(D);
      *reinterpret_cast<uint32_t*>(row + 4 * j) = codes;
      if ((j & 15) == 0) *reinterpret_cast<uint32_t*>(row + D / 2 + j / 4) = sw;
    }
  }
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

template <int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const ReadArgs a) {
  constexpr int kC = D / 8;
  const int b = blockIdx.y;
  const Range rg(a.first, a.count, b, a.n);
  const int64_t c0 = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  const uint8_t* src = a.cache + (int64_t)b * a.n_cap * mx_row_bytes(D);
  uint8_t* dst = a.rows + (int64_t)b * a.n * (2 * D);
  uint32_t codes[kUnroll], s[kUnroll];
  bool live[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t c = c0 + u * kThreads, i = c / kC;
    const int j = (int)(c % kC);
    live[u] = i < rg.count;
    int64_t e = (int64_t)((uint64_t)rg.first + (uint64_t)i);
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
    codes[u] = s[u] = 0;
    if (live[u]) {
      const uint8_t* row = src + e * mx_row_bytes(D);
      codes[u] = __ldg(reinterpret_cast<const uint32_t*>(row + 4 * j));
      s[u] = __ldg(row + D / 2 + j / 4);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (!live[u]) continue;
    uint32_t o[4];
    const MxScale scale(s[u]);
    mx_values8(codes[u], scale.lo, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = mul_bf16x2(o[i], scale.hi);
    *reinterpret_cast<uint4*>(dst + (c0 + u * kThreads) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

}  // namespace

cudaError_t launch_mx_cache_write(const MxCacheLaunch& c, cudaStream_t stream) {
  WriteArgs a{static_cast<const uint8_t*>(c.rows_in), c.seq_bytes, c.n, c.n_cap, c.first, c.count,
              static_cast<uint8_t*>(c.cache), c.status};
  const int64_t chunks = c.n * (c.d / 8);
  const int64_t gx = (chunks + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  if (gx == 0) return cudaSuccess;
  if (gx > 0x7FFFFFFF || c.B > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)gx, (unsigned)c.B);
  if (c.d == 512) return launch_pdl(cache_write_kernel<512>, grid, dim3(kThreads), 0, stream, 0, 0, a);
  if (c.d == 128) return launch_pdl(cache_write_kernel<128>, grid, dim3(kThreads), 0, stream, 0, 0, a);
  return cudaErrorInvalidValue;
}

cudaError_t launch_mx_cache_read(const MxCacheLaunch& c, cudaStream_t stream) {
  ReadArgs a{static_cast<const uint8_t*>(c.cache), c.n, c.n_cap, c.idx, c.first, c.count,
             static_cast<uint8_t*>(c.rows_out), c.status};
  const int64_t chunks = c.n * (c.d / 8);
  const int64_t gx = (chunks + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  if (gx == 0) return cudaSuccess;
  if (gx > 0x7FFFFFFF || c.B > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)gx, (unsigned)c.B);
  if (c.d == 512) return launch_pdl(cache_read_kernel<512>, grid, dim3(kThreads), 0, stream, 0, 0, a);
  if (c.d == 128) return launch_pdl(cache_read_kernel<128>, grid, dim3(kThreads), 0, stream, 0, 0, a);
  return cudaErrorInvalidValue;
}

}  // namespace csa
