// Internal declarations shared by the kernels of the target's attention layers, sampled
// acceptance and their C-ABI layer.
#pragma once

#include "../../include/gdntree_target.h"
#include "gdntree_internal.h"

namespace gdntree {

constexpr int kMinPage = 16;   // positions of 8 consecutive keys share a page
constexpr int kMaxPage = 256;
constexpr int kMaxGroup = 16;  // query heads per key-value head
constexpr int kMaxVocab = 1 << 24;
constexpr long long kMaxGroups = 0xffffffffLL / 256;  // workgroups a launch: its work items are counted in 32 bits

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// One layer's view of the cache.
struct CacheView {
  unsigned char *k, *v;
  uint8_t *ks, *vs;
  const int32_t *table;  // [B][max_pages]
  int pages, H, shift, max_pages;
  long long layer_rows;  // pages * H * page_size: rows of one layer

  // the cache row of position pos (its page id given) for head h
  __device__ __forceinline__ size_t row(int page, int h, int pos) const {
    return ((((size_t)page * H + h) << shift) | (size_t)(pos & ((1 << shift) - 1)));
  }
};

struct RowsParams {  // gdntree_cache_write and gdntree_cache_read
  CacheView c;
  const int32_t *start, *count;
  void *k, *v;
  int B, R, D;
  int fp8, rows_bf16;
};
hipError_t launch_cache_write(const RowsParams &p, hipStream_t stream);
hipError_t launch_cache_read(const RowsParams &p, hipStream_t stream);

struct CacheCommitParams {
  CacheView c;
  const int32_t *ctx, *acc_len, *acc_node;
  int B, N, P, L, D;
  int fp8;
};
hipError_t launch_cache_commit(const CacheCommitParams &p, hipStream_t stream);

struct AttendParams {
  CacheView c;
  const int32_t *ctx, *n_rows;       // n_rows null: R
  const unsigned long long *anc;     // null: chain
  const void *q;
  void *o;
  float *part;                       // workspace: partial outputs and softmax statistics
  float scale_log2;                  // scale * log2(e)
  int B, R, G, D;                    // G: query heads per key-value head
  int fp8, rows_bf16;
  bool whole = false;                // one workgroup per (request, head, row block): nothing to join
};
hipError_t launch_attend(const AttendParams &p, hipStream_t stream);
size_t attend_workspace(int R, int G, int D, long long positions);  // positions: most a table holds
bool attend_fits(int B, int R, int G, int H);  // the launches' grids

struct SampleParams {
  const int32_t *parent, *token, *n_nodes;
  const void *logits;
  const float *temperature;
  const double *uniform;
  int32_t *acc_len, *acc_tok, *acc_node;
  void *ws;
  int B, R, P, V;
  int bf16;
};
hipError_t launch_accept_sample(const SampleParams &p, hipStream_t stream);
size_t accept_sample_workspace(int B, int R, int V);
bool sample_fits(int B, int R, int V);  // the launches' grids

// x / 2^e as an fp32 factor: 2^(byte - 127), byte in [1, 254].
__device__ __forceinline__ float scale_of(unsigned byte) { return __uint_as_float(byte << 23); }

}  // namespace gdntree
