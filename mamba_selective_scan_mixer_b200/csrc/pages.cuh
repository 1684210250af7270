// The paged key-value cache on the device: its geometry as kernels take it,
// and the reads of table entries, lengths and token starts that every kernel
// makes the same way (clamped, so that no device value becomes a bad address).
#pragma once
#include "common.cuh"

namespace jb {

constexpr int PG_D = 128;        // head width (the only one supported)

struct PageGeom {
  int num_pages, G, shift;       // page_size = 1 << shift tokens
  int planes, S, max_pages, ld_table;
  __host__ __device__ int page() const { return 1 << shift; }
  // elements of one page in one plane, and of one plane
  __host__ __device__ long long page_elems() const { return (long long)G * (PG_D << shift); }
  __host__ __device__ long long plane_elems() const { return page_elems() * num_pages; }
};

__device__ __forceinline__ int held_pages(const PageGeom& g, int len) { return (len + g.page() - 1) >> g.shift; }
__device__ __forceinline__ int clamp_len(const PageGeom& g, int len, int* err) {
  const long long most = (long long)g.max_pages << g.shift;
  checked(len >= 0 && len <= most, err);
  return len < 0 ? 0 : (len > most ? (int)most : len);
}
// a page number from the table, or -1 when it is none
__device__ __forceinline__ int good_page(const PageGeom& g, int e, int* err) {
  const bool ok = e >= 0 && e < g.num_pages;
  checked(ok, err);
  return ok ? e : -1;
}
// tokens [a, b) of sequence s among the `tokens` rows of a ragged batch
__device__ __forceinline__ void token_range(const int* q_start, int s, int tokens, int& a, int& b) {
  a = max(0, min(q_start[s], tokens));
  b = max(a, min(q_start[s + 1], tokens));
}
// the sequence of token t: the last s with q_start[s] <= t (q_start ascending); -1 if none counts t
__device__ __forceinline__ int token_seq(const int* q_start, int S, int t) {
  int lo = 0, hi = S;            // q_start[lo] <= t < q_start[hi], as far as q_start ascends
  if (q_start[0] > t || q_start[S] <= t) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (q_start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace jb
