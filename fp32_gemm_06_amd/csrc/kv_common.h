// Declarations of the paged key-value cache's operators: head norms with the
// position rotation, the cache's writing and reading, and attention over it.
#pragma once

#include "s8_common.h"

namespace fp32gemm {

constexpr int kTypeS8 = 3;  // of a cache: codes with a scale for each row

// The cache: K and V, pages x heads x page_size x dim, packed; scales pages x
// heads x page_size.  Row (page, head, offset) has 32-bit numbers only: pages
// heads page_size < 2^31.
struct KvCache {
  int type, pages, page_size, heads, dim;
  void *K, *V;
  float *scaleK, *scaleV;
};

// One row operator's call, already validated: T tokens with Hq query, Hk key
// and Hv value heads of D values, each set at its own address and leading
// dimension.
struct KvRowArgs {
  int T, D, Hq, Hk, Hv;
  const void *Q, *K, *V;
  int ldq, ldk, ldv;
  void *Yq, *Yk;          // NULL Yk: keys go to the cache
  int ldyq, ldyk;
  const void *Wq, *Wk;    // NULL: no norm
  float eps;
  double inv_dim;         // 1 / D
  int R, style;           // R values of a head turn; 0: none
  const double *freq;
  const int *pos;
  const int *slots;       // with a cache
  KvCache cache;          // type < 0: none
  bool past_caches;       // floats are stored past the caches
};
hipError_t launch_kv_rows(const KvRowArgs &a, int type, hipStream_t s);

// The cache's rows of T slots, as floats.
struct KvReadArgs {
  int T;
  const int *slots;
  KvCache cache;
  void *K, *V;
  int ldk, ldv;
  bool past_caches;
};
hipError_t launch_kv_read(const KvReadArgs &a, int type, hipStream_t s);

// Attention of one token for each of B sequences, already validated.
struct AttendArgs {
  int B, Hq, Hk, G, RG;   // G query heads for each key head, in RG groups of 16 at most
  const void *Q;
  int ldq;
  KvCache cache;
  const int *table;
  int ldt;
  const int *lengths;
  int most;               // tokens that a table's row has pages for
  int window;
  float scale2;           // the scale times log2(e)
  void *O;
  int ldo;
  float *lse;             // NULL: not wanted
  unsigned *cnt;          // for each workgroup three arrival counters of 5 bits, zero between calls
  float *part;            // two partial results for each workgroup
  int groups;             // workgroups of the launch
  uint32_t magic, shift;  // t / page_size = (t magic) >> shift for t < 2^31
};
constexpr int kAttendGroups = 512;  // most workgroups of a launch
hipError_t launch_attend_s8(const AttendArgs &a, int type, hipStream_t s);
hipError_t launch_attend_float(const AttendArgs &a, int type, hipStream_t s);
// Floats of a partial result: rows query heads with dim values, maximum and
// sum, from a multiple of 16 bytes.
__host__ __device__ inline size_t attend_record(int rows, int dim) { return ((size_t)rows * (dim + 2) + 3) / 4 * 4; }
// Tokens of a workgroup's step.
inline int attend_step(int cache_type) { return cache_type == kTypeS8 ? 256 : cache_type == kTypeF32 ? 64 : 128; }

}  // namespace fp32gemm
