// Acceptance of a draft tree at a temperature on gfx950: the walk down the tree by
// inverse-transform sampling from the target's distribution at each accepted node, and the bonus
// token from what the last node's children leave.
//
// With w(x) = exp((l_x - max l) / T) and Z = sum w over the vocabulary, p(x) = w(x) / Z.  At node
// u, with children c_1, c_2, ... and the random number U: child i is taken when U falls into its
// interval of the running sum of the p(c_i); else the bonus is the token at which the running sum
// of w over the vocabulary without the children first exceeds U Z - sum w(c_i).
//
// Which rows the walk visits is known only once their parents' are read, so every used row is
// read once, at full bandwidth, by a first kernel (it is bound by HBM: one fp32 exponential per
// logit); the rest is latency.  Three kernels on the stream:
//  1. sample_stats_kernel: workgroup (chunk, row) reduces up to kChunkGroups pieces of 8192 logits
//     to their maximum and the sum of fp32 exponentials (a greedy request: the maximum and its
//     lowest index).  At most kMaxChunks chunks a row, however long the vocabulary is.
//  2. sample_walk_kernel: every workgroup of a request does the walk (one wave, the statistics and
//     the children's logits staged in LDS by one round of loads), then sums its part of the last
//     node's row without the children, in fp64.
//  3. sample_pick_kernel: finds the part, then the token, by fp64 prefix sums.
// The bonus token's place among 10^5 tokens is what needs fp64: the borders between tokens lie
// 10^-6 and less apart, and an fp32 sum would put a random number on the wrong side of one about
// once in a hundred draws.  A child's interval is held to the fp32 statistics (1e-7).

#include "target_internal.h"

namespace gdntree {
namespace {

typedef unsigned long long u64;

constexpr int kPiece = 8192;       // logits one workgroup of 256 lanes holds in registers
constexpr int kMaxChunks = 32;     // statistics per row
constexpr int kPart = 4096;        // logits per fp64 partial sum: 16 per lane
constexpr float kNegInf = -__builtin_inff();

__host__ __device__ inline int stat_pieces(int V) { return (V + 7 + kPiece * kMaxChunks - 1) / (kPiece * kMaxChunks); }
__host__ __device__ inline int stat_chunks(int V) {
  const int per = kPiece * stat_pieces(V);
  return (V + 7 + per - 1) / per;
}
__host__ __device__ inline int sum_parts(int V) { return (V + kPart - 1) / kPart; }

struct Stat {
  float m;      // maximum
  unsigned s;   // fp32 bits of the sum of exp2((l - m) log2(e) / T); greedy: lowest index of the maximum
};

// What kernel 2 leaves for kernel 3.
struct Pending {
  double u, children;  // the node's random number; sum of w over its children's tokens
  float top;           // the node's largest logit
  int node;            // -1: nothing left to draw
  int len;             // tau
  int kids;            // whether the children were candidates
};

struct Workspace {
  Stat *stat;       // [B][R][stat_chunks]
  double *part;     // [B][sum_parts]
  Pending *pend;    // [B]
};

__host__ __device__ inline size_t round16(size_t x) { return (x + 15) & ~(size_t)15; }

__host__ __device__ inline Workspace carve(void *ws, int B, int R, int V) {
  unsigned char *at = static_cast<unsigned char *>(ws);
  Workspace w;
  w.stat = reinterpret_cast<Stat *>(at);
  at += round16((size_t)B * R * stat_chunks(V) * sizeof(Stat));
  w.part = reinterpret_cast<double *>(at);
  at += round16((size_t)B * sum_parts(V) * sizeof(double));
  w.pend = reinterpret_cast<Pending *>(at);
  return w;
}

template <bool BF16>
__device__ __forceinline__ float logit(const void *logits, size_t e) {
  if constexpr (BF16) return bf16_bits_to_f32(static_cast<const uint16_t *>(logits)[e]);
  else return static_cast<const float *>(logits)[e];
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor(x, o));
  return x;
}
__device__ __forceinline__ float wave_add(float x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}
__device__ __forceinline__ double wave_add(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}
__device__ __forceinline__ unsigned wave_min(unsigned x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = min(x, (unsigned)__shfl_xor((int)x, o));
  return x;
}

__device__ __forceinline__ bool temperature_ok(float t) { return t >= 0.f && t < __builtin_inff(); }
// log2(e) / T, kept finite (a product with 0 is then 0)
__device__ __forceinline__ float inverse_log2(float t) { return fminf(1.4426950408889634f / t, 3.0e38f); }

template <bool BF16>
__global__ __launch_bounds__(256) void sample_stats_kernel(SampleParams p, Workspace ws) {
  __shared__ float s_m[4], s_s[4];
  __shared__ unsigned s_i[4];
  const int nc = stat_chunks(p.V), pieces = stat_pieces(p.V);
  const int chunk = blockIdx.x % nc, row = blockIdx.x / nc;
  const int b = row / p.R, t = row - b * p.R;
  const int n = p.n_nodes[b];
  if (n < 1 || n > p.R || t >= n) return;
  const float temp = p.temperature[b];
  if (!temperature_ok(temp)) return;
  const bool greedy = temp == 0.f;
  const float c = inverse_log2(temp);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;

  // element 0 of the row sits `pad` elements behind a 16-byte boundary: pieces are cut at boundaries
  constexpr int ES = BF16 ? 2 : 4;
  const unsigned char *base = static_cast<const unsigned char *>(p.logits) + (size_t)row * p.V * ES;
  const int pad = (int)((reinterpret_cast<uintptr_t>(base) & 15) / ES);
  base -= (size_t)pad * ES;

  float m_run = kNegInf, s_run = 0.f;
  unsigned i_run = 0xffffffffu;
  for (int piece = 0; piece < pieces; ++piece) {
    const int first = (chunk * pieces + piece) * kPiece;  // in padded elements
    if (first >= p.V + pad) break;
    float x[32];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e = first + 8 * (tid + 256 * q);
      if (e >= pad && e + 8 <= p.V + pad) {
        if constexpr (BF16) {
          const u16x8 h = *reinterpret_cast<const u16x8 *>(base + (size_t)e * 2);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[8 * q + i] = bf16_bits_to_f32(h[i]);
        } else {
          const f32x4 a = *reinterpret_cast<const f32x4 *>(base + (size_t)e * 4);
          const f32x4 d = *reinterpret_cast<const f32x4 *>(base + (size_t)e * 4 + 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) { x[8 * q + i] = a[i]; x[8 * q + 4 + i] = d[i]; }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[8 * q + i] = e + i >= pad && e + i < p.V + pad ? logit<BF16>(base, (size_t)(e + i)) : kNegInf;
      }
    }
    float m = x[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) m = fmaxf(m, x[i]);
    m = wave_max(m);
    if (greedy) {
      unsigned idx = 0xffffffffu;
      bool nan = false;
#pragma unroll
      for (int i = 31; i >= 0; --i) {
        if (x[i] == m) idx = (unsigned)(first + 8 * (tid + 256 * (i >> 3)) + (i & 7) - pad);
        nan = nan || x[i] != x[i];
      }
      idx = wave_min(m == kNegInf ? 0xffffffffu : idx);
      if (m > m_run) { m_run = m; i_run = idx; }  // pieces come in order: the first stays on a tie
      if (__any(nan)) s_run = __builtin_nanf("");
    } else {
      const float m_new = fmaxf(m_run, m);
      if (m_new > kNegInf) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += __builtin_amdgcn_exp2f((x[i] - m_new) * c);
        s = wave_add(s);
        s_run = (m_run == kNegInf ? 0.f : s_run * __builtin_amdgcn_exp2f((m_run - m_new) * c)) + s;
        m_run = m_new;
      } else {
        bool nan = false;  // nothing but -inf and NaN so far
#pragma unroll
        for (int i = 0; i < 32; ++i) nan = nan || x[i] != x[i];
        if (__any(nan)) s_run = __builtin_nanf("");
      }
    }
  }
  if (lane == 0) { s_m[wave] = m_run; s_s[wave] = s_run; s_i[wave] = i_run; }
  __syncthreads();
  if (tid == 0) {
    float m = kNegInf, s = 0.f;
    unsigned idx = 0xffffffffu;
    for (int w = 0; w < 4; ++w) m = fmaxf(m, s_m[w]);
    for (int w = 0; w < 4; ++w) {
      if (s_m[w] == m) idx = min(idx, s_i[w]);
      // a NaN sum stays one; a wave of -inf alone adds nothing
      s += s_m[w] == kNegInf || greedy ? s_s[w] : s_s[w] * __builtin_amdgcn_exp2f((s_m[w] - m) * c);
    }
    Stat st;
    st.m = s != s ? __builtin_nanf("") : m;  // the row holds a NaN
    st.s = greedy ? idx : __float_as_uint(s);
    ws.stat[(size_t)row * nc + chunk] = st;
  }
}

// The tokens of the children of `node` in slots < n, as bits of one part of the vocabulary.
__device__ __forceinline__ void mark_children(const SampleParams &p, int b, int n, int node, int first, u64 *bits,
                                              int tid, int threads) {
  for (int i = tid; i < kPart / 64; i += threads) bits[i] = 0;
  __syncthreads();
  for (int t = 1 + tid; t < n; t += threads) {
    const unsigned at = (unsigned)p.token[(size_t)b * p.R + t] - (unsigned)first;
    if (p.parent[(size_t)b * p.R + t] == node && at < (unsigned)kPart) atomicOr(&bits[at >> 6], 1ull << (at & 63));
  }
  __syncthreads();
}

// The fp64 weights of this lane's 16 tokens of a part; children and tokens past V weigh nothing.
template <bool BF16>
__device__ __forceinline__ void weights16(const SampleParams &p, size_t row, int first, const u64 *bits, float top,
                                          double temp, int tid, double w[16]) {
  const unsigned out = (unsigned)(bits[tid >> 2] >> (16 * (tid & 3))) & 0xffffu;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int x = first + 16 * tid + i;
    w[i] = 0.0;
    if (x < p.V && !((out >> i) & 1)) {
      const float l = logit<BF16>(p.logits, row * p.V + x);
      w[i] = exp(((double)l - (double)top) / temp);
    }
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void sample_walk_kernel(SampleParams p, Workspace ws) {
  __shared__ Stat s_stat[kMaxSlots * kMaxChunks];
  __shared__ float s_logit[kMaxSlots];
  __shared__ int s_par[kMaxSlots], s_tok[kMaxSlots], s_path[kMaxAnc];
  __shared__ Pending s_pend;
  __shared__ int s_bonus;
  __shared__ u64 s_bits[kPart / 64];
  __shared__ double s_sum[4];
  const int parts = sum_parts(p.V);
  const int b = blockIdx.x / parts, part = blockIdx.x - b * parts;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = p.n_nodes[b];
  if (n < 1 || n > p.R) return;
  const int nc = stat_chunks(p.V);
  const float temp = p.temperature[b];
  const bool t_ok = temperature_ok(temp), greedy = temp == 0.f;
  if (t_ok)
    for (int i = tid; i < n * nc; i += 256) s_stat[i] = ws.stat[(size_t)b * p.R * nc + i];
  if (tid < n) {
    const int par = tid ? p.parent[(size_t)b * p.R + tid] : -1, tok = p.token[(size_t)b * p.R + tid];
    s_par[tid] = par;
    s_tok[tid] = tok;
    // a child's logit under its parent; outside the vocabulary or without a parent: no mass
    s_logit[tid] = par >= 0 && par < n && tok >= 0 && tok < p.V
                       ? logit<BF16>(p.logits, ((size_t)b * p.R + par) * p.V + tok) : kNegInf;
  }
  __syncthreads();

  if (wave == 0) {
    const double *uni = p.uniform + (size_t)b * p.R;
    int u = 0, len = 1, bonus = -1;
    Pending pend{0.0, 0.0, 0.f, -1, 0, 0};
    if (lane == 0) s_path[0] = 0;
    while (t_ok) {
      // the row's maximum and normaliser
      const Stat st = lane < nc ? s_stat[u * nc + lane] : Stat{kNegInf, greedy ? 0xffffffffu : 0u};
      const float top = wave_max(st.m);
      if (__any(st.m != st.m) || top == kNegInf || top == __builtin_inff()) break;  // no distribution
      const bool more = len <= p.P;
      // lane l has slot l, and lane 0 slot 64 as well (the last one)
      const bool kid0 = more && lane >= 1 && lane < n && s_par[lane] == u;
      const bool kid1 = more && lane == 0 && n > 64 && s_par[64] == u;
      const int tok0 = lane < n ? s_tok[lane] : -1, tok1 = n > 64 ? s_tok[64] : -1;
      int next = -1;
      if (greedy) {
        const unsigned best = wave_min(st.m == top ? st.s : 0xffffffffu);
        const u64 hit = __ballot(kid0 && tok0 == (int)best);
        if (hit) next = __ffsll((long long)hit) - 1;
        else if (__any(kid1 && tok1 == (int)best)) next = 64;
        if (next < 0) { bonus = (int)best; break; }
      } else {
        const double z = wave_add(st.m == kNegInf ? 0.0 : (double)__uint_as_float(st.s) *
                                                              exp(((double)st.m - (double)top) / (double)temp));
        // weights of the children, nothing for one that repeats an earlier sibling's token
        bool dup0 = false, dup1 = false;
        for (u64 rest = __ballot(kid0); rest; rest &= rest - 1) {
          const int s = __ffsll((long long)rest) - 1, ts = __builtin_amdgcn_readlane(tok0, s);
          dup0 = dup0 || (s < lane && ts == tok0);
          dup1 = dup1 || ts == tok1;
        }
        const double w0 = kid0 && !dup0 ? exp(((double)s_logit[lane] - (double)top) / (double)temp) : 0.0;
        const double w1 = kid1 && !dup1 ? exp(((double)s_logit[64] - (double)top) / (double)temp) : 0.0;
        double end = w0;  // running sum in slot order
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const double y = __shfl_up(end, o);
          if (lane >= o) end += y;
        }
        const double all0 = __shfl(end, 63), last1 = __shfl(w1, 0);
        const double at = uni[u] * z;
        const u64 hit = __ballot(kid0 && at >= end - w0 && at < end);
        if (hit) next = __ffsll((long long)hit) - 1;
        else if (__any(kid1 && at >= all0 && at < all0 + w1)) next = 64;
        if (next < 0) {
          pend = Pending{uni[u], all0 + last1, top, u, len, more ? 1 : 0};
          break;
        }
      }
      u = next;
      if (lane == 0) s_path[len] = u;
      ++len;
    }
    if (lane == 0) {
      pend.len = len;
      s_pend = pend;
      s_bonus = bonus;
    }
  }
  __syncthreads();
  const Pending pend = s_pend;
  if (part == 0) {
    if (tid <= p.P) {
      const size_t ab = (size_t)b * (p.P + 1);
      const int len = pend.len;
      if (tid == 0) p.acc_len[b] = len;
      p.acc_node[ab + tid] = tid < len ? s_path[tid] : -1;
      // a pending bonus is written by the pick
      p.acc_tok[ab + tid] = tid < len - 1 ? s_tok[s_path[tid + 1]] : tid == len - 1 ? s_bonus : -1;
    }
    if (tid == 0) ws.pend[b] = pend;
  }
  if (pend.node < 0) return;
  const int first = part * kPart;
  mark_children(p, b, pend.kids ? n : 0, pend.node, first, s_bits, tid, 256);
  double w[16], sum = 0.0;
  weights16<BF16>(p, (size_t)b * p.R + pend.node, first, s_bits, pend.top, (double)temp, tid, w);
#pragma unroll
  for (int i = 0; i < 16; ++i) sum += w[i];
  sum = wave_add(sum);
  if (lane == 0) s_sum[wave] = sum;
  __syncthreads();
  if (tid == 0) ws.part[(size_t)b * parts + part] = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
}

template <bool BF16>
__global__ __launch_bounds__(256) void sample_pick_kernel(SampleParams p, Workspace ws) {
  __shared__ u64 s_bits[kPart / 64];
  __shared__ double s_end[256];
  __shared__ double s_before;
  __shared__ int s_part, s_found, s_last;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  const int n = p.n_nodes[b];
  if (n < 1 || n > p.R) return;
  const Pending pend = ws.pend[b];
  if (pend.node < 0) return;
  const int parts = sum_parts(p.V);
  const double *sums = ws.part + (size_t)b * parts;
  // where the random number falls among the parts: the first whose running sum exceeds it, else
  // the last with any weight
  if (tid < 64) {
    double total = 0.0;
    for (int i = lane; i < parts; i += 64) total += sums[i];
    total = wave_add(total);
    const double at = fmax(0.0, pend.u * (total + pend.children) - pend.children);
    double run = 0.0, before = 0.0;
    int found = -1, last = -1;
    for (int i0 = 0; i0 < parts && found < 0; i0 += 64) {
      const double x = i0 + lane < parts ? sums[i0 + lane] : 0.0;
      double end = x;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double y = __shfl_up(end, o);
        if (lane >= o) end += y;
      }
      end += run;
      const u64 hit = __ballot(x > 0.0 && end > at), any = __ballot(x > 0.0);
      if (hit) {
        const int l = __ffsll((long long)hit) - 1;
        found = i0 + l;
        before = __shfl(end - x, l);
      } else if (any) {
        last = i0 + 63 - __clzll((long long)any);
      }
      run = __shfl(end, 63);
    }
    if (lane == 0) {
      s_part = found >= 0 ? found : last;
      s_before = found >= 0 ? at - before : __builtin_inf();  // what is left within the part
      s_found = 0x7fffffff;
      s_last = -1;
    }
  }
  __syncthreads();
  const size_t out = (size_t)b * (p.P + 1) + pend.len - 1;
  if (s_part < 0) {
    // The children hold all the mass (the walk left them by the rounding of its normaliser): the
    // last of them that has any is the token the random number stands for.
    if (tid == 0)
      for (int t = n - 1; t >= 1; --t) {
        const int x = p.token[(size_t)b * p.R + t];
        if (p.parent[(size_t)b * p.R + t] == pend.node && x >= 0 && x < p.V &&
            logit<BF16>(p.logits, ((size_t)b * p.R + pend.node) * p.V + x) > kNegInf) {
          p.acc_tok[out] = x;
          break;
        }
      }
    return;
  }
  const int first = s_part * kPart;
  mark_children(p, b, pend.kids ? n : 0, pend.node, first, s_bits, tid, 256);
  double w[16], sum = 0.0;
  weights16<BF16>(p, (size_t)b * p.R + pend.node, first, s_bits, pend.top, (double)p.temperature[b], tid, w);
#pragma unroll
  for (int i = 0; i < 16; ++i) sum += w[i];
  s_end[tid] = sum;
  __syncthreads();
#pragma unroll
  for (int o = 1; o < 256; o <<= 1) {
    const double y = tid >= o ? s_end[tid - o] : 0.0;
    __syncthreads();
    s_end[tid] += y;
    __syncthreads();
  }
  double run = s_end[tid] - sum;
  const double at = s_before;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    run += w[i];
    if (w[i] > 0.0) {
      const int x = first + 16 * tid + i;
      if (run > at) atomicMin(&s_found, x);
      atomicMax(&s_last, x);
    }
  }
  __syncthreads();
  if (tid == 0) p.acc_tok[out] = s_found != 0x7fffffff ? s_found : s_last;
}

template <bool BF16>
hipError_t launch(const SampleParams &p, hipStream_t stream) {
  const Workspace ws = carve(p.ws, p.B, p.R, p.V);
  hipLaunchKernelGGL((sample_stats_kernel<BF16>), dim3((unsigned)(p.B * p.R * stat_chunks(p.V))), dim3(256), 0, stream, p, ws);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  hipLaunchKernelGGL((sample_walk_kernel<BF16>), dim3((unsigned)(p.B * sum_parts(p.V))), dim3(256), 0, stream, p, ws);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  hipLaunchKernelGGL((sample_pick_kernel<BF16>), dim3((unsigned)p.B), dim3(256), 0, stream, p, ws);
  return hipGetLastError();
}

}  // namespace

size_t accept_sample_workspace(int B, int R, int V) {
  return round16((size_t)B * R * stat_chunks(V) * sizeof(Stat)) + round16((size_t)B * sum_parts(V) * sizeof(double)) +
         round16((size_t)B * sizeof(Pending));
}

bool sample_fits(int B, int R, int V) {
  return (long long)B * R * stat_chunks(V) < 0x7fffffffLL && (long long)B * sum_parts(V) < 0x7fffffffLL;
}

hipError_t launch_accept_sample(const SampleParams &p, hipStream_t stream) {
  return p.bf16 ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace gdntree
