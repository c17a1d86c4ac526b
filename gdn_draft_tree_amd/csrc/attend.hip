// Attention of each request's new rows (one token, a chain, or a draft tree) over its paged cache
// on gfx950.
//
// For a request with ctx committed positions and n new rows at positions ctx + t, query row
// (t, head) attends to every position p < ctx and to the new positions its mask leaves:
//     o = sum_p w_p v_p / sum_p w_p,   w_p = exp2(c q.k_p - m),   c = scale log2(e),
// with a running maximum m: one pass over the keys.  Splitting the positions gives partial
// (m, sum w, sum w v) triples that join by rescaling with exp2(m_i - max m).
//
// All G query heads of a key-value head and all rows share its keys, so their R G query rows are
// the columns of 16-wide MFMA tiles.  Both products take their operands as the cache holds them,
// straight from global memory to registers, with no LDS between:
//  * scores, transposed: S^T (keys x queries) = K Q^T on 16x16x32 products.  Lane (g, c) of an
//    operand holds 8 consecutive channels of one key: a 16-byte load.  The keys of a 32-key tile
//    go to its two 16-row products in such an order (row r of product h holds key
//    8 (r / 4) + 4 h + r % 4) that a lane ends up with the scores of the 8 consecutive keys
//    8 g .. 8 g + 7 of query c;
//  * which is the operand layout the second product needs: O^T (channels x queries) = V^T P^T over
//    the 32 keys.  Lane (g, c) loads, for each of its keys 8 g + e, the d / 16 consecutive channels
//    that start at c d / 16 (whole rows, coalesced), and interleaves the keys' 16-bit halves in
//    registers (v_perm), so that product j has channel c d / 16 + j.
// The softmax is thus per lane except for the maximum, and that is only joined across lanes when a
// score exceeds the running one by 2^8: until then the old maximum serves (weights up to 2^8 in
// fp32 and bf16 lose nothing).
//
// Arithmetic.  bf16 rows: the products of bf16 numbers are exact, accumulated in fp32; the weights
// are rounded to bf16 for the second product (half a step, 2^-9 of a weight, against an output
// that is rounded to bf16 itself), their sum is of the fp32 weights.  fp32 rows: q and the weights
// are split into three bf16 parts that hold their 24 bits, so every product is exact to fp32.
// e4m3 cache rows become bf16 with their power-of-two scale in the conversion, exactly.

#include "target_internal.h"

namespace gdntree {
namespace {

constexpr int kTile = 32;         // keys per step of a wave
constexpr int kWaves = 4;
constexpr int kItems = 1024;      // workgroups to fill the chip with: 256 CUs, four each
constexpr float kLazy = 8.f;      // how far (log2) a score may exceed the running maximum

typedef unsigned long long u64;

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 x) { return __builtin_bit_cast(bf16x8, x); }

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  const bf16x2 r = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(unsigned, r);
}

// Three bf16 parts of eight fp32 numbers, each hi + mid + lo exactly (24 bits); a number that is
// not finite stays in the high part alone.
__device__ __forceinline__ void split3(const float x[8], bf16x8 part[3]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __bf16 hi = (__bf16)x[i];
    float r = x[i] - (float)hi;
    if (!((__float_as_uint((float)hi) & 0x7f800000u) != 0x7f800000u)) r = 0.f;
    const __bf16 mid = (__bf16)r;
    part[0][i] = hi;
    part[1][i] = mid;
    part[2][i] = (__bf16)(r - (float)mid);
  }
}

// How the positions of all requests are cut into work items.  Request b has tiles(b) 32-key tiles;
// an item is at most `span` of them, and the span is the least multiple of the workgroup's waves
// with which the whole batch makes about kItems workgroups.  It follows from the lengths on the
// device, so that a captured launch serves any lengths, and is computed by every wave for itself:
// lane l reads requests l, l + 64, ...
struct Item {
  int b;             // request; -1: no item
  int split, count;  // this item among the request's
  int slot;          // the request's first partial-result slot (requests of one item have none)
  int span;          // tiles per item
};

struct Lens {
  int ctx, n;  // committed positions, new rows in use (0: no output)
  bool bad;    // positions out of the table's range: the rows in use get NaN
  int tiles;
};

__device__ __forceinline__ Lens lens_of(const AttendParams &p, int b) {
  Lens r;
  r.ctx = p.ctx[b];
  r.n = p.n_rows ? p.n_rows[b] : p.R;
  if (r.n < 1 || r.n > p.R) r.n = 0;
  r.bad = r.ctx < 0 || r.ctx > 0x7fffff00 || (long long)r.ctx + r.n > (long long)p.c.max_pages << p.c.shift;
  r.tiles = r.n == 0 ? 0 : r.bad ? 1 : (int)(((long long)r.ctx + r.n + kTile - 1) / kTile);
  return r;
}

__device__ __forceinline__ int wave_scan(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  return x;
}

__device__ __forceinline__ int span_of(long long tiles, int units) {
  const long long least = (tiles * units + kItems - 1) / kItems;
  return (int)((least + kWaves - 1) / kWaves * kWaves);
}

// Item j of the batch (the same for every unit of `units` key-value heads and row blocks).
__device__ __forceinline__ Item find_item(const AttendParams &p, int j, int units, int lane) {
  long long total = 0;
  for (int b0 = 0; b0 < p.B; b0 += 64) {
    long long t = b0 + lane < p.B ? lens_of(p, b0 + lane).tiles : 0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) t += __shfl_xor(t, o);
    total += t;
  }
  Item it{-1, 0, 0, 0, span_of(total, units)};
  if (it.span == 0) return it;  // no request has rows
  int items = 0, slots = 0;     // of the requests before b0
  for (int b0 = 0; b0 < p.B; b0 += 64) {
    const int tiles = b0 + lane < p.B ? lens_of(p, b0 + lane).tiles : 0;
    const int cnt = (tiles + it.span - 1) / it.span, multi = cnt > 1 ? cnt : 0;
    const int end = wave_scan(cnt, lane), send = wave_scan(multi, lane);
    const u64 mine = __ballot(j >= items + end - cnt && j < items + end);
    if (mine) {
      const int l = __ffsll((long long)mine) - 1;
      it.b = b0 + l;
      it.count = __shfl(cnt, l);
      it.split = j - (items + __shfl(end - cnt, l));
      it.slot = slots + __shfl(send - multi, l);
      return it;
    }
    items += __shfl(end, 63);
    slots += __shfl(send, 63);
  }
  return it;
}

// Request b's items (for the join).
__device__ __forceinline__ Item find_request(const AttendParams &p, int b, int units, int lane) {
  long long total = 0;
  for (int b0 = 0; b0 < p.B; b0 += 64) {
    long long t = b0 + lane < p.B ? lens_of(p, b0 + lane).tiles : 0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) t += __shfl_xor(t, o);
    total += t;
  }
  Item it{b, 0, 0, 0, span_of(total, units)};
  if (it.span == 0) return it;
  for (int b0 = 0; b0 <= b; b0 += 64) {
    const int tiles = b0 + lane < p.B ? lens_of(p, b0 + lane).tiles : 0;
    const int cnt = (tiles + it.span - 1) / it.span, multi = cnt > 1 ? cnt : 0;
    const int send = wave_scan(multi, lane);
    if (b < b0 + 64) {
      it.count = __shfl(cnt, b - b0);
      it.slot += __shfl(send - multi, b - b0);
    } else {
      it.slot += __shfl(send, 63);
    }
  }
  return it;
}

// Upper bounds that hold for any lengths: sum ceil(tiles / span) <= sum tiles / span + B, and a
// request of two items or more has fewer than twice its tiles / span.
__host__ __device__ constexpr int items_most(int B, int units) { return (kItems + units - 1) / units + B; }
__host__ __device__ constexpr int slots_most(int units) { return 2 * ((kItems + units - 1) / units); }

// Partial results: [row block][key-value head][slot][BM][D + 2], the last two (m, sum of weights).
struct Part {
  int BM, stride;
  __device__ __forceinline__ size_t at(int rb, int h, int H, int units, int slot) const {
    return (((size_t)rb * H + h) * slots_most(units) + slot) * (size_t)BM * stride;
  }
};

template <bool BF16>
__device__ __forceinline__ void store_o(void *o, size_t e, float x) {
  if constexpr (BF16) static_cast<uint16_t *>(o)[e] = f32_to_bf16_bits(x);
  else static_cast<float *>(o)[e] = x;
}

// One item: keys [32 t0, 32 t1) of request b for one key-value head and 16 MT query rows.  The
// waves take every kWaves-th tile each, with statistics and sums of their own, and join in LDS.
template <int D, bool FP8, bool BF16ROWS, int MT>
__global__ __launch_bounds__(64 * kWaves, MT == 1 ? 2 : 1) void attend_kernel(AttendParams p) {
  constexpr int KS = D / 32;               // 32-channel steps of the scores' product
  constexpr int DV = D / 16;               // channels per lane of the values' product
  constexpr int NQ = BF16ROWS ? 1 : 3;     // bf16 parts of q and of the weights
  constexpr int BM = 16 * MT;
  constexpr int OST = D + 4;               // padded row of the joined sums
  __shared__ float s_o[BM * OST];
  __shared__ float s_m[kWaves][BM], s_l[kWaves][BM];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int rows = p.R * p.G;              // query rows of a key-value head
  const int nrb = (rows + BM - 1) / BM, units = nrb * p.c.H;
  const int rb = blockIdx.x % nrb, h = blockIdx.x / nrb % p.c.H, j = blockIdx.x / units;
  const Item it = find_item(p, j, units, lane);
  if (it.b < 0) return;
  const int b = it.b;
  const Lens len = lens_of(p, b);
  if (rb * BM >= len.n * p.G) return;      // no row of this block is in use
  const int Hq = p.c.H * p.G;
  const int total = len.ctx + len.n;

  // the query rows of this lane's columns, as operands; rows not in use are zero
  bf16x8 qf[MT][KS][NQ];
  u64 see[MT];                             // bit s - 1: new row s is visible to the column
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int m = rb * BM + 16 * mt + c, t = m / p.G;
    const bool used = t < len.n;
    const size_t qrow = ((size_t)b * p.R + (used ? t : 0)) * Hq + (size_t)h * p.G + (used ? m % p.G : 0);
    see[mt] = !used ? 0 : p.anc ? p.anc[(size_t)b * p.R + t] : t >= 64 ? ~0ull : (1ull << t) - 1;
    if (len.n < 65) see[mt] &= (1ull << (len.n - 1)) - 1;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      // channels of this lane in step ks: as the cache rows' loads give them
      const int d0 = FP8 ? 64 * (ks >> 1) + 16 * g + 8 * (ks & 1) : 32 * ks + 8 * g;
      if constexpr (BF16ROWS) {
        u32x4 x = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p.q) + qrow * D + d0);
        if (!used) x = u32x4{0, 0, 0, 0};
        qf[mt][ks][0] = as_bf16x8(x);
      } else {
        const float *src = static_cast<const float *>(p.q) + qrow * D + d0;
        const f32x4 x0 = *reinterpret_cast<const f32x4 *>(src), x1 = *reinterpret_cast<const f32x4 *>(src + 4);
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) { x[i] = used ? x0[i] : 0.f; x[4 + i] = used ? x1[i] : 0.f; }
        split3(x, qf[mt][ks]);
      }
    }
  }

  f32x4 acc[MT][DV];
  float m_run[MT], l_run[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    m_run[mt] = -__builtin_inff();
    l_run[mt] = 0.f;
#pragma unroll
    for (int d = 0; d < DV; ++d) acc[mt][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int tiles = len.bad ? 0 : len.tiles;
  const int t0 = it.split * it.span, t1 = min(tiles, t0 + it.span);
  const int32_t *tab = p.c.table + (size_t)b * p.c.max_pages;
  bool bad = false;                        // a page id out of range

  for (int tile = t0 + wave; tile < t1; tile += kWaves) {
    const int pos0 = tile * kTile;
    // Positions past the last row are loaded as the last row (and masked), pages out of range as
    // page 0 (and the result becomes NaN): every load is in bounds.
    const int pk = min(pos0 + 8 * (c >> 2), total - 1), pv = min(pos0 + 8 * g, total - 1);
    int pgk = tab[pk >> p.c.shift], pgv = tab[pv >> p.c.shift];
    if ((unsigned)pgk >= (unsigned)p.c.pages) { bad = true; pgk = 0; }
    if ((unsigned)pgv >= (unsigned)p.c.pages) { bad = true; pgv = 0; }

    u32x4 kr[2][KS];                       // bf16 operands of the two 16-key products
    u32x4 vr[8];                           // DV bf16 channels of keys 8 g + e
    if constexpr (FP8) {
      const u64 ksc = *reinterpret_cast<const u64 *>(p.c.ks + p.c.row(pgk, h, pk & ~7));
      const u64 vsc = *reinterpret_cast<const u64 *>(p.c.vs + p.c.row(pgv, h, pv & ~7));
      u32x4 raw[2][KS / 2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int pos = min(pos0 + 8 * (c >> 2) + 4 * hh + (c & 3), total - 1);
        const unsigned char *src = p.c.k + p.c.row(pgk, h, pos) * D + 16 * g;
#pragma unroll
        for (int s2 = 0; s2 < KS / 2; ++s2) raw[hh][s2] = *reinterpret_cast<const u32x4 *>(src + 64 * s2);
      }
      u32x2 vraw[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int pos = min(pos0 + 8 * g + e, total - 1);
        const unsigned char *src = p.c.v + p.c.row(pgv, h, pos) * D + DV * c;
        if constexpr (DV == 8) vraw[e] = *reinterpret_cast<const u32x2 *>(src);
        else vraw[e] = u32x2{*reinterpret_cast<const unsigned *>(src), 0u};
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int pos = min(pos0 + 8 * (c >> 2) + 4 * hh + (c & 3), total - 1);
        const float s = scale_of((unsigned)(ksc >> (8 * (pos & 7))) & 255u);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const unsigned src = raw[hh][ks >> 1][2 * (ks & 1) + (w >> 1)];
            kr[hh][ks][w] = __builtin_bit_cast(unsigned, w & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(src, s, true)
                                                               : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(src, s, false));
          }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int pos = min(pos0 + 8 * g + e, total - 1);
        const float s = scale_of((unsigned)(vsc >> (8 * (pos & 7))) & 255u);
#pragma unroll
        for (int w = 0; w < DV / 2; ++w)
          vr[e][w] = __builtin_bit_cast(unsigned, w & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(vraw[e][w >> 1], s, true)
                                                        : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(vraw[e][w >> 1], s, false));
      }
    } else {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int pos = min(pos0 + 8 * (c >> 2) + 4 * hh + (c & 3), total - 1);
        const unsigned char *src = p.c.k + p.c.row(pgk, h, pos) * (2 * D) + 16 * g;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) kr[hh][ks] = *reinterpret_cast<const u32x4 *>(src + 64 * ks);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int pos = min(pos0 + 8 * g + e, total - 1);
        const unsigned char *src = p.c.v + p.c.row(pgv, h, pos) * (2 * D) + 2 * DV * c;
        if constexpr (DV == 8) {
          vr[e] = *reinterpret_cast<const u32x4 *>(src);
        } else {
          const u32x2 x = *reinterpret_cast<const u32x2 *>(src);
          vr[e] = u32x4{x[0], x[1], 0u, 0u};
        }
      }
    }

    const bool masked = pos0 + kTile > len.ctx;  // the tile holds new rows, or ends past the last one
    // A masked value that is not finite would enter the sums as 0 * inf: such tiles (new rows only)
    // are summed term by term over what each column sees.
    bool odd = false;
    if (masked) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int w = 0; w < DV / 2; ++w)
          odd = odd || (vr[e][w] & 0x7f80u) == 0x7f80u || (vr[e][w] & 0x7f800000u) == 0x7f800000u;
      odd = __any(odd);
    }
    bf16x8 vt[DV];  // operand j: channel DV c + j of the 8 keys
#pragma unroll
    for (int d = 0; d < DV; ++d) {
      u32x4 x;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        x[w] = __builtin_amdgcn_perm(vr[2 * w + 1][d >> 1], vr[2 * w][d >> 1], d & 1 ? 0x07060302u : 0x05040100u);
      vt[d] = as_bf16x8(x);
    }

#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      f32x4 s[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        s[hh] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int q = NQ - 1; q >= 0; --q) s[hh] = mfma(as_bf16x8(kr[hh][ks]), qf[mt][ks][q], s[hh]);
      }
      unsigned vis = 0xffu;  // which of the 8 keys the column sees
      if (masked) {
        vis = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int sl = pos0 + 8 * g + e - len.ctx;
          const bool on = sl <= 0 || (sl < len.n && ((see[mt] >> (sl - 1)) & 1));
          vis |= (unsigned)on << e;
          if (!on) s[e >> 2][e & 3] = -__builtin_inff();
        }
      }
      float top = s[0][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e >> 2][e & 3]);
      top *= p.scale_log2;
      if (__any(top > m_run[mt] + kLazy)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m_new = fmaxf(m_run[mt], top);
        const float f = m_run[mt] == m_new ? 1.f : __builtin_amdgcn_exp2f(m_run[mt] - m_new);
        m_run[mt] = m_new;
        l_run[mt] *= f;
#pragma unroll
        for (int d = 0; d < DV; ++d) acc[mt][d] *= f;
      }
      const float ms = m_run[mt] == -__builtin_inff() ? 0.f : m_run[mt];  // a column that sees nothing yet
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e >> 2][e & 3], p.scale_log2, -ms));
        l_run[mt] += w[e];
      }
      if (!odd) {
        bf16x8 pf[NQ];
        if constexpr (BF16ROWS)
          pf[0] = as_bf16x8(u32x4{pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]), pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7])});
        else
          split3(w, pf);
#pragma unroll
        for (int d = 0; d < DV; ++d)
#pragma unroll
          for (int q = NQ - 1; q >= 0; --q) acc[mt][d] = mfma(vt[d], pf[q], acc[mt][d]);
      } else {
        for (int gk = 0; gk < 4; ++gk) {
          const unsigned seen = (unsigned)__shfl((int)vis, 16 * gk + c);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float we = __shfl(w[e], 16 * gk + c);
            const bool on = (seen >> e) & 1;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int d2 = 0; d2 < DV / 2; ++d2) {
                const unsigned v2 = (unsigned)__shfl((int)vr[e][d2], 16 * gk + 4 * g + i);
                if (on) {
                  acc[mt][2 * d2][i] += we * __uint_as_float(v2 << 16);
                  acc[mt][2 * d2 + 1][i] += we * __uint_as_float(v2 & 0xffff0000u);
                }
              }
          }
        }
      }
    }
  }

  // the column's sum of weights over the lane groups, then the waves joined
  bad = __any(bad) || len.bad;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    float l = l_run[mt];
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (bad) l = __builtin_nanf("");
    if (g == 0) {
      s_m[wave][16 * mt + c] = m_run[mt];
      s_l[wave][16 * mt + c] = l;
    }
  }
  __syncthreads();
  float fac[MT], m_all[MT], l_all[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int col = 16 * mt + c;
    float m = s_m[0][col];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, s_m[w][col]);
    m_all[mt] = m;
    l_all[mt] = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = s_m[w][col] == m ? 1.f : __builtin_amdgcn_exp2f(s_m[w][col] - m);
      l_all[mt] += s_l[w][col] * f;
      if (w == wave) fac[mt] = f;
    }
  }
  for (int w = 0; w < kWaves; ++w) {  // in order: the sums do not depend on which wave is first
    if (w == wave) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int d = 0; d < DV; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float *dst = &s_o[(16 * mt + c) * OST + DV * (4 * g + i) + d];
            const float x = acc[mt][d][i] * fac[mt];
            *dst = w == 0 ? x : *dst + x;
          }
    }
    __syncthreads();
  }
  const bool whole = it.count == 1;
  if (wave == 0 && g == 0) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      s_m[0][16 * mt + c] = m_all[mt];
      s_l[0][16 * mt + c] = l_all[mt];
    }
  }
  __syncthreads();
  const Part part{BM, D + 2};
  float *mine = p.part + part.at(rb, h, p.c.H, units, it.slot + it.split);
  for (int e = tid; e < BM * D; e += 64 * kWaves) {
    const int r = e / D, d = e % D, m = rb * BM + r, t = m / p.G;
    if (t >= len.n) break;
    const float x = s_o[r * OST + d];
    if (whole)
      store_o<BF16ROWS>(p.o, (((size_t)b * p.R + t) * Hq + (size_t)h * p.G + m % p.G) * D + d, x / s_l[0][r]);
    else
      mine[r * (D + 2) + d] = x;
  }
  if (!whole && tid < BM) {
    mine[tid * (D + 2) + D] = s_m[0][tid];
    mine[tid * (D + 2) + D + 1] = s_l[0][tid];
  }
}

// Joins the items of every request that was cut into more than one: one wave per query row.
template <int D, bool BF16ROWS, int MT>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendParams p) {
  constexpr int BM = 16 * MT, PL = D / 64;
  const int lane = threadIdx.x & 63;
  const int Hq = p.c.H * p.G;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= (long long)p.B * p.R * Hq) return;
  const int b = (int)(row / (p.R * Hq)), rem = (int)(row - (long long)b * p.R * Hq);
  const int t = rem / Hq, hq = rem % Hq, h = hq / p.G, m = t * p.G + hq % p.G;
  const int nrb = (p.R * p.G + BM - 1) / BM, units = nrb * p.c.H;
  if (t >= lens_of(p, b).n) return;
  const Item it = find_request(p, b, units, lane);
  if (it.count < 2) return;  // written by its one item
  const Part part{BM, D + 2};
  const float *base = p.part + part.at(m / BM, h, p.c.H, units, it.slot) + (size_t)(m % BM) * (D + 2);
  const size_t step = (size_t)BM * (D + 2);
  float top = -__builtin_inff();
  for (int s = lane; s < it.count; s += 64) top = fmaxf(top, base[s * step + D]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  float x[PL], l = 0.f;
#pragma unroll
  for (int i = 0; i < PL; ++i) x[i] = 0.f;
  for (int s = 0; s < it.count; ++s) {
    const float *src = base + s * step;
    const float ms = src[D], f = ms == top ? 1.f : __builtin_amdgcn_exp2f(ms - top);
    l += f * src[D + 1];
#pragma unroll
    for (int i = 0; i < PL; ++i) x[i] += f * src[lane + 64 * i];
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) store_o<BF16ROWS>(p.o, (size_t)row * D + lane + 64 * i, x[i] / l);
}

// 16-row tiles per workgroup: the least that holds the query rows of a key-value head.
int tiles_of(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

template <int D, bool FP8, bool BF16ROWS, int MT>
hipError_t launch_mt(const AttendParams &p, hipStream_t stream) {
  const int nrb = (p.R * p.G + 16 * MT - 1) / (16 * MT), units = nrb * p.c.H;
  hipLaunchKernelGGL((attend_kernel<D, FP8, BF16ROWS, MT>), dim3((unsigned)(units * items_most(p.B, units))),
                     dim3(64 * kWaves), 0, stream, p);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  const long long rows = (long long)p.B * p.R * p.c.H * p.G;
  hipLaunchKernelGGL((attend_join_kernel<D, BF16ROWS, MT>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <int D, bool FP8, bool BF16ROWS>
hipError_t launch_rows(const AttendParams &p, hipStream_t stream) {
  switch (tiles_of(p.R * p.G)) {
    case 1: return launch_mt<D, FP8, BF16ROWS, 1>(p, stream);
    case 2: return launch_mt<D, FP8, BF16ROWS, 2>(p, stream);
    default: return launch_mt<D, FP8, BF16ROWS, 4>(p, stream);
  }
}

template <int D>
hipError_t launch_d(const AttendParams &p, hipStream_t stream) {
  if (p.fp8) return p.rows_bf16 ? launch_rows<D, true, true>(p, stream) : launch_rows<D, true, false>(p, stream);
  return p.rows_bf16 ? launch_rows<D, false, true>(p, stream) : launch_rows<D, false, false>(p, stream);
}

}  // namespace

size_t attend_workspace(int B, int R, int G, int H, int D) {
  (void)B;  // the items of a batch are bounded by the chip, not by the batch
  const int BM = 16 * tiles_of(R * G), units = (R * G + BM - 1) / BM * H;
  return (size_t)units * slots_most(units) * BM * (D + 2) * sizeof(float);
}

bool attend_fits(int B, int R, int G, int H) {
  const int BM = 16 * tiles_of(R * G);
  const long long units = (long long)((R * G + BM - 1) / BM) * H;
  const long long rows = (long long)B * R * G;  // < 2^42: no overflow in the product below
  return units < (1LL << 24) && units * (kItems + 1LL + B) < 0x7fffffffLL && rows * H / 4 < 0x7ffffffeLL;
}

hipError_t launch_attend(const AttendParams &p, hipStream_t stream) {
  return p.D == 64 ? launch_d<64>(p, stream) : launch_d<128>(p, stream);
}

}  // namespace gdntree
