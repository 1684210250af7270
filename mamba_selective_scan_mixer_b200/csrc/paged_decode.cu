// Attention of one new token per sequence over the paged key-value cache, grouped
// query heads:
//   o = sum_j softmax_j(q . k_j / sqrt(d)) v_j over the sequence's positions,
//   lse = log sum_j exp(q . k_j / sqrt(d)),
// in one pass over the keys with a running maximum and sum.
//
// A CTA takes one sequence, up to eight query heads of one KV head and a part of
// the positions; the partial softmaxes of the parts are joined by a second kernel.
#include "host.hpp"
#include "pages.cuh"

namespace jb {

constexpr int ROW_REP = 8;                   // query heads per CTA (the padded N of its tiles)
constexpr int ROW_PITCH = 272;               // bytes per staged row (256 + 16)
constexpr int ROW_TILE = 16 * ROW_PITCH;     // 16 rows
constexpr uint32_t ROW_SMEM = 4 * 2 * 2 * ROW_TILE;   // warps x buffers x (K, V)

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
// 16 bytes global -> shared; src_bytes 0 writes zeros (the source is not read)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

struct PagedAttnParams {
  PageGeom g;
  int H, rep;
  const bf16* q; long long ld_q;
  const bf16 *k, *v;
  const int *table, *lengths;
  bf16* o; long long ld_o;
  float* lse;
  float sl2;                       // log2(e) / sqrt(head_dim)
  float* part;                     // [tokens * H][splits][D + 2]
  int splits;
  int* err;
};

__global__ void __launch_bounds__(128)
paged_decode_kernel(const PagedAttnParams p) {
  extern __shared__ uint8_t dsm[];
  __shared__ float w_m[4][ROW_REP], w_l[4][ROW_REP];
  __shared__ float w_o[4][ROW_REP][PG_D];
  griddep_wait();
  griddep_launch();
  const int hgs = (p.rep + ROW_REP - 1) / ROW_REP;
  const int hg = blockIdx.x % hgs, g = blockIdx.x / hgs % p.g.G, t = blockIdx.x / hgs / p.g.G, split = blockIdx.y;
  const int rep = min(ROW_REP, p.rep - hg * ROW_REP);
  const int head0 = g * p.rep + hg * ROW_REP;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, tq = lane & 3;   // mma fragment coordinates
  const int n = clamp_len(p.g, p.lengths[t], p.err);
  const int per = (n + p.splits - 1) / p.splits;
  const int p0 = min(n, split * per), p1 = min(n, p0 + per);
  uint32_t qb[8][2];                          // B fragments of Q^T
  {
    const bf16* qrow = p.q + t * p.ld_q + (long long)(head0 + (gq < rep ? gq : 0)) * PG_D;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      uint32_t lo = 0, hi = 0;
      if (gq < rep) {
        lo = *reinterpret_cast<const uint32_t*>(qrow + 16 * kk + 2 * tq);
        hi = *reinterpret_cast<const uint32_t*>(qrow + 16 * kk + 2 * tq + 8);
      }
      qb[kk][0] = lo;
      qb[kk][1] = hi;
    }
  }
  const int* trow = p.table + (long long)t * p.g.ld_table;
  const uint32_t wbase = smem_u32(dsm) + warp * 2 * 2 * ROW_TILE;
  // stage 16 rows of K and V at positions c0.. (within one page) into buffer `buf`, zeros past p1
  auto stage = [&](int c0, int buf) {
    const uint32_t kd = wbase + buf * 2 * ROW_TILE, vd = kd + ROW_TILE;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int idx = lane + 32 * i;
      const int row = idx >> 4, piece = idx & 15;
      const int pos = c0 + row;
      const bool in = pos < p1;
      const int e = in ? max(0, good_page(p.g, trow[pos >> p.g.shift], p.err)) : 0;
      const long long off = e * p.g.page_elems() + ((long long)g << p.g.shift) * PG_D +
                            (long long)(pos & (p.g.page() - 1)) * PG_D + piece * 8;
      cp_async16(kd + row * ROW_PITCH + piece * 16, p.k + off, in ? 16 : 0);
      cp_async16(vd + row * ROW_PITCH + piece * 16, p.v + off, in ? 16 : 0);
    }
    cp_async_commit();
  };
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // heads 2tq, 2tq + 1
  float acc[8][4];
#pragma unroll
  for (int mm = 0; mm < 8; ++mm) acc[mm][0] = acc[mm][1] = acc[mm][2] = acc[mm][3] = 0.f;
  const int mi = lane >> 3, rr = lane & 7;
  int c0 = p0 + warp * 16, buf = 0;
  if (c0 < p1) stage(c0, 0);
  for (; c0 < p1; c0 += 64, buf ^= 1) {
    if (c0 + 64 < p1) {
      stage(c0 + 64, buf ^ 1);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncwarp();
    const uint32_t kt = wbase + buf * 2 * ROW_TILE, vt = kt + ROW_TILE;
    float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      uint32_t a[4];
      ldsm_x4(a, kt + (rr + 8 * (mi & 1)) * ROW_PITCH + (16 * kk + 8 * (mi >> 1)) * 2);
      mma_bf16_16816(sc, a, qb[kk][0], qb[kk][1]);
    }
    const bool in0 = c0 + gq < p1, in8 = c0 + gq + 8 < p1;
    float pr[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float s0 = in0 ? sc[e] * p.sl2 : -INFINITY, s8 = in8 ? sc[2 + e] * p.sl2 : -INFINITY;
      float mx = fmaxf(s0, s8);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m[e], mx);                  // position c0 is in
      const float corr = ex2(m[e] - mn);
      pr[e] = ex2(s0 - mn);
      pr[2 + e] = ex2(s8 - mn);
      float sum = pr[e] + pr[2 + e];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l[e] = l[e] * corr + sum;
      m[e] = mn;
#pragma unroll
      for (int mm = 0; mm < 8; ++mm) {
        acc[mm][e] *= corr;
        acc[mm][2 + e] *= corr;
      }
    }
    uint32_t pb0, pb1;
    {
      const int srcA = (2 * tq) * 4 + (gq >> 1), srcB = (2 * tq + 1) * 4 + (gq >> 1);
      const bool odd = gq & 1;
      const float a0 = __shfl_sync(0xffffffffu, pr[0], srcA), a1 = __shfl_sync(0xffffffffu, pr[1], srcA);
      const float b0 = __shfl_sync(0xffffffffu, pr[0], srcB), b1 = __shfl_sync(0xffffffffu, pr[1], srcB);
      const float a2 = __shfl_sync(0xffffffffu, pr[2], srcA), a3 = __shfl_sync(0xffffffffu, pr[3], srcA);
      const float b2 = __shfl_sync(0xffffffffu, pr[2], srcB), b3 = __shfl_sync(0xffffffffu, pr[3], srcB);
      __nv_bfloat162 h01 = __floats2bfloat162_rn(odd ? a1 : a0, odd ? b1 : b0);
      __nv_bfloat162 h23 = __floats2bfloat162_rn(odd ? a3 : a2, odd ? b3 : b2);
      pb0 = *reinterpret_cast<uint32_t*>(&h01);
      pb1 = *reinterpret_cast<uint32_t*>(&h23);
    }
#pragma unroll
    for (int mm = 0; mm < 8; ++mm) {
      uint32_t a[4];
      ldsm_x4_t(a, vt + (rr + 8 * (mi >> 1)) * ROW_PITCH + (16 * mm + 8 * (mi & 1)) * 2);
      mma_bf16_16816(acc[mm], a, pb0, pb1);
    }
    __syncwarp();
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int hq = 2 * tq + e;
    if (hq < rep) {
      if (gq == 0) {
        w_m[warp][hq] = m[e];
        w_l[warp][hq] = l[e];
      }
#pragma unroll
      for (int mm = 0; mm < 8; ++mm) {
        w_o[warp][hq][16 * mm + gq] = acc[mm][e];
        w_o[warp][hq][16 * mm + gq + 8] = acc[mm][2 + e];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rep * PG_D; i += 128) {
    const int h = i / PG_D, d = i % PG_D;
    float mm = -INFINITY;
    for (int w = 0; w < 4; ++w) mm = fmaxf(mm, w_m[w][h]);
    float ls = 0.f, os = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float f = w_m[w][h] == -INFINITY ? 0.f : ex2(w_m[w][h] - mm);
      ls += w_l[w][h] * f;
      os += w_o[w][h][d] * f;
    }
    float* dst = p.part + (((long long)t * p.H + head0 + h) * p.splits + split) * (PG_D + 2);
    dst[d] = os;
    if (d == 0) {
      dst[PG_D] = mm;
      dst[PG_D + 1] = ls;
    }
  }
}

// joins the parts of (token, head): o = sum of o_i 2^(m_i - m) / sum of l_i 2^(m_i - m)
__global__ void __launch_bounds__(128)
paged_decode_join_kernel(const PagedAttnParams p) {
  griddep_wait();
  griddep_launch();
  const int t = blockIdx.x / p.H, h = blockIdx.x % p.H, d = threadIdx.x;
  const float* src = p.part + (long long)blockIdx.x * p.splits * (PG_D + 2);
  float mm = -INFINITY;
  for (int s = 0; s < p.splits; ++s) mm = fmaxf(mm, src[s * (PG_D + 2) + PG_D]);
  float ls = 0.f, os = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float ms = src[s * (PG_D + 2) + PG_D];
    const float f = ms == -INFINITY ? 0.f : ex2(ms - mm);
    ls += src[s * (PG_D + 2) + PG_D + 1] * f;
    os += src[s * (PG_D + 2) + d] * f;
  }
  p.o[t * p.ld_o + h * PG_D + d] = __float2bfloat16_rn(ls > 0.f ? os / ls : 0.f);
  if (p.lse && d == 0)
    p.lse[(long long)t * p.H + h] = ls > 0.f ? (mm + log2f(ls)) * 0.6931471805599453f : -INFINITY;
}

static int row_splits(const PageGeom& g, int H, int tokens) {
  const int rep = H / g.G, hgs = (rep + ROW_REP - 1) / ROW_REP;
  const long long ctas = (long long)tokens * g.G * hgs;
  long long s = (16LL * num_sms() + ctas - 1) / ctas;
  const long long cap = (((long long)g.max_pages << g.shift) + 255) / 256;   // at least 256 positions per split
  if (s > cap) s = cap;
  return s < 1 ? 1 : (int)s;
}

size_t paged_decode_workspace_bytes(const PageGeom& g, int H) {
  return (size_t)g.S * H * row_splits(g, H, g.S) * (PG_D + 2) * 4;
}

jamba_status paged_decode(const PageGeom& g, int H, const void* q, long long ld_q, const void* k_pages,
                          const void* v_pages, const int* table, const int* lengths, void* o, long long ld_o,
                          float* lse, void* ws, cudaStream_t s) {
  const int tokens = g.S;
  PagedAttnParams p;
  p.g = g;
  p.H = H;
  p.rep = H / g.G;
  p.q = reinterpret_cast<const bf16*>(q);
  p.ld_q = ld_q;
  p.k = reinterpret_cast<const bf16*>(k_pages);
  p.v = reinterpret_cast<const bf16*>(v_pages);
  p.table = table;
  p.lengths = lengths;
  p.o = reinterpret_cast<bf16*>(o);
  p.ld_o = ld_o;
  p.lse = lse;
  p.sl2 = 1.4426950408889634f / sqrtf((float)PG_D);
  p.part = reinterpret_cast<float*>(ws);
  p.splits = row_splits(g, H, tokens);
  p.err = device_error_word();
  const int hgs = (p.rep + ROW_REP - 1) / ROW_REP;
  static std::atomic<bool> configured[64];
  int dev = 0;
  JB_CUDA(cudaGetDevice(&dev));
  if (dev < 64 && !configured[dev]) {
    JB_CUDA(cudaFuncSetAttribute(paged_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ROW_SMEM));
    configured[dev] = true;
  }
  JB_CUDA(launch_pdl(paged_decode_kernel, dim3((unsigned)(tokens * g.G * hgs), p.splits), dim3(128), ROW_SMEM, s, p));
  JB_CUDA(launch_pdl(paged_decode_join_kernel, dim3((unsigned)(tokens * H)), dim3(PG_D), 0, s, p));
  return JAMBA_OK;
}

}  // namespace jb
