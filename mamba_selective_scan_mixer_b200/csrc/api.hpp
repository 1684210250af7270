// What the C entry points share: workspace carving, argument checks and the
// dense GEMM description.
#pragma once
#include <string>

#include "host.hpp"

namespace jb {

constexpr size_t kAlign = 256;
inline size_t al(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }

// Sequential carve-out of a workspace; with a null base it only measures.
struct Carver {
  uint8_t* base;
  size_t off = 0;
  explicit Carver(void* b) : base(reinterpret_cast<uint8_t*>(b)) {}
  template <typename T = void>
  T* take(size_t bytes) {
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off += al(bytes);
    return p;
  }
};

inline cudaStream_t cs(jamba_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

inline GemmDesc gdesc(const void* a, long long lda, const void* b, long long ldb, int M, int N, int K, int epi,
                      void* out, long long ldo) {
  GemmDesc g = {};
  g.a = a; g.lda = lda; g.b = b; g.ldb = ldb; g.M = M; g.N = N; g.K = K; g.epi = epi; g.out = out; g.ldo = ldo;
  g.splits = 1;
  return g;
}

inline jamba_status check_ptr(const void* p, const char* name, bool required = true) {
  if (!p) return required ? fail(JAMBA_ERR_INVALID_ARG, std::string(name) + " is null") : JAMBA_OK;
  if (!aligned16(p)) return fail(JAMBA_ERR_INVALID_ARG, std::string(name) + " is not 16-byte aligned");
  return JAMBA_OK;
}

jamba_status check_attn_cfg(const jamba_attn_config* c);

}  // namespace jb
