// The paged key-value cache of the target's attention layers on gfx950: rows written (bf16, or
// quantised to e4m3), rows read back, and the accepted path's rows moved together.
//
// Quantisation of one row x of d channels (one token, one head): with amax the largest finite
// |x|, e the least integer with amax <= 448 2^e (448 = 1.75 2^8 is the largest e4m3 number),
// code = RNE(x 2^-e).  A power of two instead of amax / 448: x 2^-e is exact in fp32, so the one
// rounding is the conversion's (half a step, 2^-4 of the value), the same on any machine, and a
// code times its scale is a bf16 number, which the attention puts into its products as it is.
// The format is a floating-point one, so the up to one bit of range the power of two leaves
// unused costs nothing until values fall 2^-14 below the largest.
//
// All three are bound by HBM (a few integer operations per 16 bytes): a row is one 16-byte load
// per lane, d / 8 lanes per row, so a wave moves 4 (d = 128) or 8 rows of keys and as many of
// values at a time, in whole 128-byte lines.

#include "target_internal.h"

namespace gdntree {
namespace {

// Eight fp32 values of a row from 16 bytes of bf16 or 32 bytes of fp32.
template <bool BF16>
__device__ __forceinline__ void load8(const void *base, size_t elem, float x[8]) {
  if constexpr (BF16) {
    const u16x8 h = *reinterpret_cast<const u16x8 *>(static_cast<const uint16_t *>(base) + elem);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = bf16_bits_to_f32(h[i]);
  } else {
    const f32x4 a = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(base) + elem);
    const f32x4 b = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(base) + elem + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[i] = a[i]; x[4 + i] = b[i]; }
  }
}

// The biased exponent byte of a row's scale from its largest finite |x|.
__device__ __forceinline__ unsigned scale_byte(float amax) {
  const unsigned u = __float_as_uint(amax);
  // amax = m 2^k with m in [1, 2): e = k - 8 while m <= 1.75, else k - 7 (a subnormal amax has
  // exponent bits 0 and meets the lower bound)
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (unsigned)((e < -117 ? -117 : e) + 127);
}

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// Eight e4m3 codes of x * inv (a power of two, so the products are exact); not finite: NaN.
__device__ __forceinline__ u32x2 codes8(const float x[8], float inv) {
  u32x2 c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h] * inv, x[4 * h + 1] * inv, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h + 2] * inv, x[4 * h + 3] * inv, w, true);
    unsigned u = (unsigned)w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!finite(x[4 * h + i])) u |= 0x7fu << (8 * i);
    c[h] = u;
  }
  return c;
}

template <int D, bool FP8, bool BF16ROWS>
__global__ __launch_bounds__(256) void cache_write_kernel(RowsParams p) {
  constexpr int LPR = D / 8;  // lanes per row
  const long long rows = (long long)p.B * p.R * p.c.H;
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) / LPR;
  const int c = threadIdx.x % LPR;
  if (i >= rows) return;  // whole rows: LPR divides 64
  const int h = (int)(i % p.c.H);
  const long long bt = i / p.c.H;
  const int b = (int)(bt / p.R), t = (int)(bt - (long long)b * p.R);
  const int n = p.count ? p.count[b] : p.R;
  const long long pos = (long long)p.start[b] + t;
  if (t >= n || pos < 0 || pos >= (long long)p.c.max_pages << p.c.shift) return;
  const int page = p.c.table[(size_t)b * p.c.max_pages + (size_t)(pos >> p.c.shift)];
  if (page < 0 || page >= p.c.pages) return;
  const size_t row = p.c.row(page, h, (int)pos);
  float x[2][8];
  load8<BF16ROWS>(p.k, (size_t)i * D + 8 * c, x[0]);
  load8<BF16ROWS>(p.v, (size_t)i * D + 8 * c, x[1]);
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    unsigned char *out = kv ? p.c.v : p.c.k;
    if constexpr (FP8) {
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, finite(x[kv][j]) ? fabsf(x[kv][j]) : 0.f);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
      const unsigned byte = scale_byte(amax);
      *reinterpret_cast<u32x2 *>(out + row * D + 8 * c) = codes8(x[kv], scale_of(254u - byte));
      if (c == 0) (kv ? p.c.vs : p.c.ks)[row] = (uint8_t)byte;
    } else {
      u16x8 y;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = f32_to_bf16_bits(x[kv][j]);
      *reinterpret_cast<u16x8 *>(reinterpret_cast<uint16_t *>(out) + row * D + 8 * c) = y;
    }
  }
}

template <int D, bool FP8, bool BF16ROWS>
__global__ __launch_bounds__(256) void cache_read_kernel(RowsParams p) {
  constexpr int LPR = D / 8;
  const long long rows = (long long)p.B * p.R * p.c.H;
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) / LPR;
  const int c = threadIdx.x % LPR;
  if (i >= rows) return;
  const int h = (int)(i % p.c.H);
  const long long bt = i / p.c.H;
  const int b = (int)(bt / p.R), t = (int)(bt - (long long)b * p.R);
  if (t >= (p.count ? p.count[b] : p.R)) return;
  const long long pos = (long long)p.start[b] + t;
  int page = -1;
  if (pos >= 0 && pos < (long long)p.c.max_pages << p.c.shift)
    page = p.c.table[(size_t)b * p.c.max_pages + (size_t)(pos >> p.c.shift)];
  const bool ok = page >= 0 && page < p.c.pages;
  const size_t row = ok ? p.c.row(page, h, (int)pos) : 0;  // row 0 is read and dropped
  u16x8 y[2];  // the row's values as bf16 bits
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const unsigned char *in = kv ? p.c.v : p.c.k;
    if constexpr (FP8) {
      const float s = scale_of((kv ? p.c.vs : p.c.ks)[row]);
      const u32x2 w = *reinterpret_cast<const u32x2 *>(in + row * D + 8 * c);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bf16x2 r = q & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[q >> 1], s, true)
                               : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[q >> 1], s, false);
        const unsigned u = __builtin_bit_cast(unsigned, r);
        y[kv][2 * q] = (uint16_t)u;
        y[kv][2 * q + 1] = (uint16_t)(u >> 16);
      }
    } else {
      y[kv] = *reinterpret_cast<const u16x8 *>(reinterpret_cast<const uint16_t *>(in) + row * D + 8 * c);
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    if (!ok)
#pragma unroll
      for (int j = 0; j < 8; ++j) y[kv][j] = 0x7fc0u;
    void *out = kv ? p.v : p.k;
    if constexpr (BF16ROWS) {
      *reinterpret_cast<u16x8 *>(static_cast<uint16_t *>(out) + (size_t)i * D + 8 * c) = y[kv];
    } else {
      f32x4 a, b4;
#pragma unroll
      for (int j = 0; j < 4; ++j) { a[j] = bf16_bits_to_f32(y[kv][j]); b4[j] = bf16_bits_to_f32(y[kv][4 + j]); }
      *reinterpret_cast<f32x4 *>(static_cast<float *>(out) + (size_t)i * D + 8 * c) = a;
      *reinterpret_cast<f32x4 *>(static_cast<float *>(out) + (size_t)i * D + 8 * c + 4) = b4;
    }
  }
}

// The accepted path of one (layer, request, head): one workgroup reads every moved row of the
// keys and the values into registers, waits for all of them, and stores them at their new places
// (sources and destinations overlap, so nothing may be stored before everything is read).
// Latency-bound: at most 17 rows of 256 bytes.
template <int D, bool FP8>
__global__ __launch_bounds__(256) void cache_commit_kernel(CacheCommitParams p) {
  constexpr int ROWB = FP8 ? D : 2 * D;
  constexpr int CPR = ROWB / 16;                       // 16-byte chunks per row
  constexpr int PER = (2 * kMaxAnc * CPR + 255) / 256;  // chunks per thread, keys and values
  __shared__ long long s_src[kMaxAnc], s_dst[kMaxAnc];
  __shared__ int s_ok;
  const int tid = threadIdx.x;
  const int h = blockIdx.x % p.c.H, lb = blockIdx.x / p.c.H;
  const int b = lb % p.B, l = lb / p.B;
  const int tau = p.acc_len[b];
  const long long ctx = p.ctx[b];
  if (tau < 1 || tau > p.P + 1 || ctx < 0) return;
  if (tid == 0) s_ok = 1;
  __syncthreads();
  if (tid < tau) {
    const int32_t *path = p.acc_node + (size_t)b * (p.P + 1);
    const int node = path[tid], before = tid ? path[tid - 1] : -1;
    bool ok = node > before && node <= p.N && (tid || node == 0);
    const long long src = ctx + node, dst = ctx + tid, cap = (long long)p.c.max_pages << p.c.shift;
    ok = ok && node >= 0 && src < cap && dst < cap;
    if (ok) {
      const int32_t *tb = p.c.table + (size_t)b * p.c.max_pages;
      const int ps = tb[src >> p.c.shift], pd = tb[dst >> p.c.shift];
      ok = ps >= 0 && ps < p.c.pages && pd >= 0 && pd < p.c.pages;
      s_src[tid] = (long long)p.c.row(ps, h, (int)src) + l * p.c.layer_rows;
      s_dst[tid] = (long long)p.c.row(pd, h, (int)dst) + l * p.c.layer_rows;
    }
    if (!ok) s_ok = 0;
  }
  __syncthreads();
  if (!s_ok) return;
  u32x4 r[PER];
  uint8_t sc = 0;
  const int chunks = 2 * tau * CPR;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = tid + 256 * j, rr = e / CPR, kv = rr >= tau;
    if (e < chunks)
      r[j] = *reinterpret_cast<const u32x4 *>((kv ? p.c.v : p.c.k) + s_src[rr - (kv ? tau : 0)] * ROWB + 16 * (e % CPR));
  }
  const bool scale_lane = FP8 && tid < 2 * tau;
  if (scale_lane) sc = (tid >= tau ? p.c.vs : p.c.ks)[s_src[tid >= tau ? tid - tau : tid]];
  __builtin_amdgcn_s_waitcnt(0);  // this wave's reads have returned
  __syncthreads();                // and every wave's
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = tid + 256 * j, rr = e / CPR, kv = rr >= tau;
    if (e < chunks)
      *reinterpret_cast<u32x4 *>((kv ? p.c.v : p.c.k) + s_dst[rr - (kv ? tau : 0)] * ROWB + 16 * (e % CPR)) = r[j];
  }
  if (scale_lane) (tid >= tau ? p.c.vs : p.c.ks)[s_dst[tid >= tau ? tid - tau : tid]] = sc;
}

template <int D, bool FP8, bool BF16ROWS>
hipError_t launch_rows(const RowsParams &p, bool write, hipStream_t stream) {
  const long long threads = (long long)p.B * p.R * p.c.H * (D / 8);
  const dim3 grid((unsigned)((threads + 255) / 256));
  if (write)
    hipLaunchKernelGGL((cache_write_kernel<D, FP8, BF16ROWS>), grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((cache_read_kernel<D, FP8, BF16ROWS>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <int D>
hipError_t launch_rows_d(const RowsParams &p, bool write, hipStream_t stream) {
  if (p.fp8) return p.rows_bf16 ? launch_rows<D, true, true>(p, write, stream) : launch_rows<D, true, false>(p, write, stream);
  return p.rows_bf16 ? launch_rows<D, false, true>(p, write, stream) : launch_rows<D, false, false>(p, write, stream);
}

template <int D, bool FP8>
hipError_t launch_commit_rows(const CacheCommitParams &p, hipStream_t stream) {
  hipLaunchKernelGGL((cache_commit_kernel<D, FP8>), dim3((unsigned)((long long)p.L * p.B * p.c.H)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_write(const RowsParams &p, hipStream_t stream) {
  return p.D == 64 ? launch_rows_d<64>(p, true, stream) : launch_rows_d<128>(p, true, stream);
}
hipError_t launch_cache_read(const RowsParams &p, hipStream_t stream) {
  return p.D == 64 ? launch_rows_d<64>(p, false, stream) : launch_rows_d<128>(p, false, stream);
}
hipError_t launch_cache_commit(const CacheCommitParams &p, hipStream_t stream) {
  if (p.D == 64) return p.fp8 ? launch_commit_rows<64, true>(p, stream) : launch_commit_rows<64, false>(p, stream);
  return p.fp8 ? launch_commit_rows<128, true>(p, stream) : launch_commit_rows<128, false>(p, stream);
}

}  // namespace gdntree
