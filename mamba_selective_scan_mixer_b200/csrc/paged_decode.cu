// Attention of one new token per sequence over the paged key-value cache, grouped
// query heads:
//   o = sum_j softmax_j(q . k_j / sqrt(d)) v_j over the sequence's positions,
//   lse = log sum_j exp(q . k_j / sqrt(d)),
// in one pass over the keys with a running maximum and sum.  Bound by reading the cache:
// 512 bytes per position and KV head, for 4 d operations per query head.
//
// Work split: a unit is a sequence and a KV head, its work the blocks of 64 positions
// it holds (an empty sequence counts one, which writes its zeros).  The blocks of all units, one
// after another, are cut into equal ranges, two CTAs per SM, so one long sequence among short
// ones costs no more than the same bytes spread evenly.  A unit inside one range is written out at
// once; of one that crosses ranges each CTA writes its part (unnormalised o, maximum,
// sum) and paged_decode_join_kernel adds the parts in order.
//
// A CTA is a producer warp, which copies pages by TMA into a ring of blocks (128-byte swizzle, so
// that ldmatrix reads hit 32 distinct banks), and four warps that take 16 positions of a block
// each, with two tensor-core products (mma.sync m16n8k16, bf16 in, fp32 out; the work per
// byte is far below what tcgen05 is needed for, and its 128-row tiles would be padding):
//   S^T = K Q^T      positions on M, query heads (padded to 8 or 16) on N, head width as K;
//   O^T += V^T P^T   head width on M, heads on N, positions as K (V^T through ldmatrix .trans).
// A lane of S^T holds two heads for two positions, which is where O^T keeps those heads, so maximum, sum
// and rescaling stay in its lanes; P^T's fragment is S^T's transposed by movmatrix.  P enters its
// product as a bf16 and the bf16 of what that left out: the tensor cores have time to spare, and the
// output is then rounded once instead of twice.
//
// Measured: 64 sequences of 2048 tokens, 32 heads on 8, 89.8 us with the join, 6.0 TB/s, 0.91 of the
// copy rate (one CTA per part with plain loads before it: 108.5 us); 24 sequences of 1 to 131072
// tokens, 64 heads, pages of 16: 235 us, 0.91; one sequence of 200 tokens 7.6 us, two launches and
// the latency of four blocks.  Parts joined inside this kernel by the CTA that ends last took 91 to
// 93 us at the first size (fences under full memory traffic).
#include "host.hpp"
#include "pages.cuh"

namespace jb {

constexpr int DP_BK = 64;                        // positions per block
constexpr int DP_THREADS = 160;                  // 4 consumer warps, 1 producer
constexpr int DP_CTAS = 2;                       // per SM
constexpr int DP_WHOLE = 4;                      // blocks of a unit that is not worth cutting

template <int NT> struct DpSmem {                // NT: tiles of eight query heads
  static constexpr int STAGES = NT == 1 ? 3 : 2;
  static constexpr uint32_t HALF = DP_BK * 128;  // 64 rows x 64 bf16, swizzled
  static constexpr uint32_t STAGE = 4 * HALF;    // K dims 0-63 | 64-127, V the same
  static constexpr uint32_t Q_OFF = STAGES * STAGE;
  static constexpr uint32_t Q_SLOT = NT * 8 * 256;
  static constexpr uint32_t M_OFF = Q_OFF + 2 * Q_SLOT;                      // two warps' o, m, l
  static constexpr uint32_t M_WARP = NT * 8 * (PG_D + 2) * 4;
  static constexpr uint32_t BAR_OFF = M_OFF + 2 * M_WARP;
  static constexpr uint32_t BYTES = BAR_OFF + 128 + 1024;
};

struct DpMeta {                                  // of a CTA's first and last item
  int tail, s, g;                                // tail: the last item begins a unit that ends in another CTA
  int ends;                                      // the first item ends its unit
};

struct DpParams {
  PageGeom g;
  int H, rep;
  const bf16* q; long long ld_q;
  const int *table, *lengths;
  bf16* o; long long ld_o;
  float* lse;
  float sl2;                                     // log2(e) / sqrt(head_dim)
  float* part;                                   // [2 grid][rep][D + 2]: o, m, l
  DpMeta* meta;                                  // [grid]
  int* err;
};

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// slot 0 of the join has been read by warp 0 (which only arrives) before warps 2 and 3 write the next item's
__device__ __forceinline__ void join_read_arrive() { asm volatile("bar.arrive 2, 96;" ::: "memory"); }
__device__ __forceinline__ void join_read_wait() { asm volatile("bar.sync 2, 96;" ::: "memory"); }

// One stretch of blocks [kb0, kb1) of unit (s, g); every warp walks the same items.
struct DpWalk {
  int s, g, kb0, kb1, nb, len;
  long long left;                                // blocks of the CTA's range from kb0 on
  __device__ void load(const DpParams& p) {
    len = clamp_len(p.g, p.lengths[s], p.err);
    nb = max(1, (len + DP_BK - 1) / DP_BK);
  }
  __device__ bool open() {
    if (left <= 0) return false;
    kb1 = (int)min((long long)nb, kb0 + left);
    return true;
  }
  __device__ bool next(const DpParams& p) {
    left -= kb1 - kb0;
    if (left <= 0) return false;
    kb0 = 0;
    if (++g == p.g.G) {
      g = 0;
      if (++s >= p.g.S) return false;
      load(p);
    }
    return open();
  }
};

template <int NT>
__global__ void __launch_bounds__(DP_THREADS, DP_CTAS)
paged_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const DpParams p) {
  using S = DpSmem<NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long sh_warp[DP_THREADS / 32], sh_left;
  __shared__ int sh_pos[3];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR_OFF);
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + S::STAGES);
  const uint32_t qfull0 = smem_u32(bars + 2 * S::STAGES), qempty0 = smem_u32(bars + 2 * S::STAGES + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(qfull0 + 8 * i, 1);
      mbar_init(qempty0 + 8 * i, 4);
    }
    mbar_fence_init();
    tma_prefetch(&tmK);
    tma_prefetch(&tmV);
  }
  griddep_wait();
  griddep_launch();

  // the range of this CTA: where it starts (sequence, head, block) and its length
  {
    const int per_t = (p.g.S + DP_THREADS - 1) / DP_THREADS;
    const int s0 = threadIdx.x * per_t, s1 = min(p.g.S, s0 + per_t);
    DpWalk w;
    long long sum = 0;
    for (w.s = s0; w.s < s1; ++w.s) {
      w.load(p);
      sum += (long long)w.nb * p.g.G;
    }
    long long x = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh_warp[warp] = x;
    __syncthreads();
    long long N = 0, before = x - sum;
    for (int i = 0; i < DP_THREADS / 32; ++i) {
      if (i < warp) before += sh_warp[i];
      N += sh_warp[i];
    }
    // With few blocks, ranges of a unit up to DP_WHOLE blocks, of two blocks beyond: a block more costs
    // a CTA 0.5 us, joining parts 1 to 2 us (one sequence of 64 tokens whole 5.9 us, two of its heads in
    // one range 7.4 us; of 500 tokens whole 9.5 us, in four parts 8.1 us; of 1000 tokens whole 13.3 us,
    // in eight parts 9.5 us)
    const long long units = (long long)p.g.S * p.g.G, mean = (N + units - 1) / units;
    const long long per = max((N + gridDim.x - 1) / gridDim.x, mean <= DP_WHOLE ? mean : 2);
    const long long a = min(N, blockIdx.x * per), b = min(N, a + per);
    if (b > a && a >= before && a < before + sum) {
      long long rem = a - before;
      for (w.s = s0;; ++w.s) {
        w.load(p);
        const long long t = (long long)w.nb * p.g.G;
        if (rem < t) break;
        rem -= t;
      }
      sh_pos[0] = w.s;
      sh_pos[1] = (int)(rem / w.nb);
      sh_pos[2] = (int)(rem % w.nb);
    }
    if (threadIdx.x == 0) sh_left = b - a;
  }
  __syncthreads();
  DpWalk w;
  w.left = sh_left;
  if (w.left > 0) {
    w.s = sh_pos[0];
    w.g = sh_pos[1];
    w.kb0 = sh_pos[2];
    w.load(p);
  }

  if (warp == 4) {
    // ---- producer: lane i loads the i-th box of a block
    const int br = min(p.g.page(), DP_BK);       // rows of a box
    int fill = 0, items = 0, e = 0;
    long long ebase = -32;                       // table entries ebase .. ebase + 31 of the row are in e, a lane each
    bool ok = true;
    for (bool more = w.open(); more && ok; more = w.next(p), ++items) {
      const int qs = items & 1;
      ok = mbar_wait_warp(qempty0 + 8 * qs, ((items >> 1) & 1) ^ 1, p.err);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_tx(qfull0 + 8 * qs, p.rep * 256);
        bulk_load(smem_u32(smem + S::Q_OFF + qs * S::Q_SLOT), p.q + w.s * p.ld_q + (long long)w.g * p.rep * PG_D,
                  p.rep * 256, qfull0 + 8 * qs);
      }
      ebase = -32;
      const int* row = p.table + (long long)w.s * p.g.ld_table;
      const int held = held_pages(p.g, w.len);
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++fill) {
        const int slot = fill % S::STAGES;
        const int i0 = (kb * DP_BK) >> p.g.shift;           // first table entry of the block
        const int valid = max(0, min(DP_BK, w.len - kb * DP_BK)), nbox = (valid + br - 1) / br;
        if (i0 + 4 > ebase + 32) {               // a block has at most four entries
          ebase = i0;
          e = ebase + lane < held ? max(0, good_page(p.g, row[ebase + lane], p.err)) : 0;
        }
        const int pos = kb * DP_BK + lane * br;
        const int page = __shfl_sync(0xffffffffu, e, (int)((pos >> p.g.shift) - ebase) & 31);
        ok = mbar_wait_warp(empty0 + 8 * slot, ((fill / S::STAGES) & 1) ^ 1, p.err);
        if (!ok) break;
        const uint32_t bar = full0 + 8 * slot;
        if (lane == 0) mbar_arrive_tx(bar, nbox * br * 512);
        __syncwarp();
        if (lane < nbox) {
          const int r = ((page * p.g.G + w.g) << p.g.shift) + (pos & (p.g.page() - 1));
          const uint32_t dst = smem_u32(smem) + slot * S::STAGE + lane * br * 128;
          tma_load_2d(dst, &tmK, bar, 0, r);
          tma_load_2d(dst + S::HALF, &tmK, bar, 64, r);
          tma_load_2d(dst + 2 * S::HALF, &tmV, bar, 0, r);
          tma_load_2d(dst + 3 * S::HALF, &tmV, bar, 64, r);
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {                      // gave up: let the copies in flight land before the CTA ends
      const uint64_t t0 = globaltimer();
      for (int i = max(0, fill - S::STAGES); i < fill; ++i)
        while (!mbar_try(full0 + 8 * (i % S::STAGES), (i / S::STAGES) & 1) && globaltimer() - t0 < 10000000ull) {
        }
      for (int i = max(0, items - 1); i <= items; ++i)
        while (!mbar_try(qfull0 + 8 * (i & 1), (i >> 1) & 1) && globaltimer() - t0 < 20000000ull) {
        }
    }
  } else {
    // ---- consumers: warp w takes positions 16 w .. 16 w + 15 of each block
    const int gq = lane >> 2, tq = lane & 3;     // mma fragment coordinates
    const int mi = lane >> 3, rr = lane & 7;     // ldmatrix: matrix and row this lane addresses
    const uint32_t k_row = (16 * warp + rr + 8 * (mi & 1)) * 128, v_row = (16 * warp + rr + 8 * (mi >> 1)) * 128;
    int fill = 0, items = 0;
    bool first_item = true;
    if (threadIdx.x == 0) p.meta[blockIdx.x].tail = 0;
    // After a failed wait the loops still run to their end (on whatever the buffers hold), so that
    // every warp reaches every consumer_sync; the error is latched and later waits end at once.
    for (bool more = w.open(); more; more = w.next(p), ++items, first_item = false) {
      const bool whole = w.kb0 == 0 && w.kb1 == w.nb;
      if (threadIdx.x == 0) {
        DpMeta* m = p.meta + blockIdx.x;
        if (first_item) m->ends = w.kb1 == w.nb;
        m->tail = w.kb0 == 0 && w.kb1 < w.nb;    // only the last item can be one
        m->s = w.s;
        m->g = w.g;
      }
      const int qs = items & 1;
      mbar_wait_warp(qfull0 + 8 * qs, (items >> 1) & 1, p.err);
      __syncwarp();
      if (warp == 0 && !first_item) join_read_arrive();
      // B fragments of Q^T (k = head dims, n = head gq of each tile; heads past rep are zero)
      uint32_t qb[NT][8][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint8_t* qrow = smem + S::Q_OFF + qs * S::Q_SLOT + (n * 8 + gq) * 256;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const bool in = n * 8 + gq < p.rep;
          qb[n][kk][0] = in ? *reinterpret_cast<const uint32_t*>(qrow + 32 * kk + 4 * tq) : 0u;
          qb[n][kk][1] = in ? *reinterpret_cast<const uint32_t*>(qrow + 32 * kk + 4 * tq + 16) : 0u;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(qempty0 + 8 * qs);
      float m[NT][2], l[NT][2], acc[NT][8][4];   // heads 2 tq, 2 tq + 1 of each tile; l: this lane's positions only
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int mm = 0; mm < 8; ++mm) acc[n][mm][0] = acc[n][mm][1] = acc[n][mm][2] = acc[n][mm][3] = 0.f;
      }
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++fill) {
        const int slot = fill % S::STAGES;
        mbar_wait_warp(full0 + 8 * slot, (fill / S::STAGES) & 1, p.err);
        const int valid = w.len - kb * DP_BK - 16 * warp;   // of this warp's positions
        if (valid > 0) {
          const uint32_t kt = smem_u32(smem) + slot * S::STAGE, vt = kt + 2 * S::HALF;
          if (valid < 16) {                      // rows behind the last token may hold anything: V's become zero
            for (int i = lane; i < (16 - valid) * 16; i += 32) {
              const int r = 16 * warp + valid + (i >> 4), c = i & 15;
              *reinterpret_cast<uint4*>(smem + slot * S::STAGE + (2 + (c >> 3)) * S::HALF + r * 128 + (c & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
          }
          // S^T = K Q^T, two chains a tile
          float sc[NT][2][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) sc[n][c][0] = sc[n][c][1] = sc[n][c][2] = sc[n][c][3] = 0.f;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            uint32_t a[4];
            ldsm_x4(a, kt + (kk >> 2) * S::HALF + k_row + (((2 * (kk & 3) + (mi >> 1)) ^ rr) << 4));
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_bf16_16816(sc[n][kk & 1], a, qb[n][kk][0], qb[n][kk][1]);
          }
          const bool in0 = gq < valid, in8 = gq + 8 < valid;
          uint32_t ph[NT][2], pl[NT][2];         // P^T's fragments: bf16, and what it left out
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float pr[4], corr[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float s0 = in0 ? (sc[n][0][e] + sc[n][1][e]) * p.sl2 : -INFINITY;
              const float s8 = in8 ? (sc[n][0][2 + e] + sc[n][1][2 + e]) * p.sl2 : -INFINITY;
              float mx = fmaxf(s0, s8);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              const float mn = fmaxf(m[n][e], mx);
              const float ref = mn == -INFINITY ? 0.f : mn;  // so far every score is -inf: their terms are 0
              corr[e] = ex2(m[n][e] - ref);
              pr[e] = ex2(s0 - ref);
              pr[2 + e] = ex2(s8 - ref);
              l[n][e] = l[n][e] * corr[e] + pr[e] + pr[2 + e];
              m[n][e] = mn;
            }
            if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
              for (int mm = 0; mm < 8; ++mm) {
                acc[n][mm][0] *= corr[0];
                acc[n][mm][1] *= corr[1];
                acc[n][mm][2] *= corr[0];
                acc[n][mm][3] *= corr[1];
              }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {        // positions gq, gq + 8: transposed to positions 2 tq, 2 tq + 1 (+ 8)
              const __nv_bfloat162 hi = __floats2bfloat162_rn(pr[2 * h], pr[2 * h + 1]);
              const __nv_bfloat162 lo =
                  __floats2bfloat162_rn(pr[2 * h] - __low2float(hi), pr[2 * h + 1] - __high2float(hi));
              ph[n][h] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&hi));
              pl[n][h] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&lo));
            }
          }
          // O^T += V^T P^T: 8 tiles of 16 head dims
#pragma unroll
          for (int mm = 0; mm < 8; ++mm) {
            uint32_t a[4];
            ldsm_x4_t(a, vt + (mm >> 2) * S::HALF + v_row + (((2 * (mm & 3) + (mi & 1)) ^ rr) << 4));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_bf16_16816(acc[n][mm], a, ph[n][0], ph[n][1]);
              mma_bf16_16816(acc[n][mm], a, pl[n][0], pl[n][1]);
            }
          }
          if (valid < 16) fence_async_shared();  // the zeroed rows are TMA's again
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty0 + 8 * slot);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
      // join the warps, 2 and 3 into 0 and 1, then 1 into 0: through a slot of [head][o, m, l]
      auto put = [&](int slot) {
        float* dst = reinterpret_cast<float*>(smem + S::M_OFF + slot * S::M_WARP);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* h = dst + (n * 8 + 2 * tq + e) * (PG_D + 2);
#pragma unroll
            for (int mm = 0; mm < 8; ++mm) {
              h[16 * mm + gq] = acc[n][mm][e];
              h[16 * mm + gq + 8] = acc[n][mm][2 + e];
            }
            if (gq == 0) {
              h[PG_D] = m[n][e];
              h[PG_D + 1] = l[n][e];
            }
          }
      };
      auto add = [&](int slot) {
        const float* src = reinterpret_cast<const float*>(smem + S::M_OFF + slot * S::M_WARP);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float* h = src + (n * 8 + 2 * tq + e) * (PG_D + 2);
            const float mo = h[PG_D], mn = fmaxf(m[n][e], mo);
            const float fa = m[n][e] == -INFINITY ? 0.f : ex2(m[n][e] - mn), fb = mo == -INFINITY ? 0.f : ex2(mo - mn);
            l[n][e] = l[n][e] * fa + h[PG_D + 1] * fb;
            m[n][e] = mn;
#pragma unroll
            for (int mm = 0; mm < 8; ++mm) {
              acc[n][mm][e] = acc[n][mm][e] * fa + h[16 * mm + gq] * fb;
              acc[n][mm][2 + e] = acc[n][mm][2 + e] * fa + h[16 * mm + gq + 8] * fb;
            }
          }
      };
      if (warp >= 2) {
        if (!first_item) join_read_wait();
        put(warp - 2);
      }
      consumer_sync();
      if (warp < 2) add(warp);
      consumer_sync();
      if (warp == 1) put(0);
      consumer_sync();
      if (warp == 0) {
        add(0);
        const long long row = w.s;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = n * 8 + 2 * tq + e;
            if (h >= p.rep) continue;
            const int head = w.g * p.rep + h;
            if (whole) {
              const float inv = l[n][e] != 0.f ? 1.f / l[n][e] : 0.f;   // a NaN stays one
              bf16* dst = p.o + row * p.ld_o + (long long)head * PG_D;
#pragma unroll
              for (int mm = 0; mm < 8; ++mm) {
                dst[16 * mm + gq] = __float2bfloat16_rn(acc[n][mm][e] * inv);
                dst[16 * mm + gq + 8] = __float2bfloat16_rn(acc[n][mm][2 + e] * inv);
              }
              if (p.lse && gq == 0)
                p.lse[row * p.H + head] =
                    l[n][e] != 0.f ? (m[n][e] + log2f(l[n][e])) * 0.6931471805599453f : -INFINITY;
            } else {
              float* dst = p.part + ((long long)(2 * blockIdx.x + (w.kb0 == 0)) * p.rep + h) * (PG_D + 2);
#pragma unroll
              for (int mm = 0; mm < 8; ++mm) {
                dst[16 * mm + gq] = acc[n][mm][e];
                dst[16 * mm + gq + 8] = acc[n][mm][2 + e];
              }
              if (gq == 0) {
                dst[PG_D] = m[n][e];
                dst[PG_D + 1] = l[n][e];
              }
            }
          }
      }
    }
  }
}

// CTA (c, h): head h of the unit whose parts begin in CTA c of the kernel above, a thread per element:
// o = sum of o_i 2^(m_i - m) / sum of l_i 2^(m_i - m), in the order of the parts.
__global__ void __launch_bounds__(PG_D)
paged_decode_join_kernel(const DpParams p, int ctas) {
  griddep_wait();
  griddep_launch();
  const int c = blockIdx.x, h = blockIdx.y, d = threadIdx.x;
  const DpMeta me = p.meta[c];
  if (!me.tail) return;
  int parts = 2;
  while (c + parts < ctas && !p.meta[c + parts - 1].ends) ++parts;   // CTA c + i continues the unit, the last ends it
  auto src = [&](int k) { return p.part + ((long long)(k == 0 ? 2 * c + 1 : 2 * (c + k)) * p.rep + h) * (PG_D + 2); };
  float m = -INFINITY;
  for (int k = 0; k < parts; ++k) m = fmaxf(m, src(k)[PG_D]);
  float l = 0.f, o = 0.f;
#pragma unroll 4
  for (int k = 0; k < parts; ++k) {
    const float* x = src(k);
    const float f = x[PG_D] == -INFINITY ? 0.f : ex2(x[PG_D] - m);
    l += x[PG_D + 1] * f;
    o += x[d] * f;
  }
  const int head = me.g * p.rep + h;
  p.o[me.s * p.ld_o + (long long)head * PG_D + d] = __float2bfloat16_rn(l != 0.f ? o / l : 0.f);
  if (p.lse && d == 0)
    p.lse[(long long)me.s * p.H + head] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// CTAs: no more than the blocks that the table can hold
static int decode_grid(const PageGeom& g) {
  const long long most = (long long)g.S * g.G * ((((long long)g.max_pages << g.shift) + DP_BK - 1) / DP_BK);
  const long long full = (long long)DP_CTAS * num_sms();
  return (int)(most < full ? most : full);
}
static size_t decode_meta_bytes(int grid) { return ((size_t)grid * sizeof(DpMeta) + 255) & ~size_t(255); }

size_t paged_decode_workspace_bytes(const PageGeom& g, int H) {
  const int grid = decode_grid(g);
  return decode_meta_bytes(grid) + (size_t)2 * grid * (H / g.G) * (PG_D + 2) * 4;
}

template <int NT>
static jamba_status launch_decode(const CUtensorMap& mk, const CUtensorMap& mv, const DpParams& p, int grid,
                                  cudaStream_t s) {
  static std::atomic<bool> configured[64];
  int dev = 0;
  JB_CUDA(cudaGetDevice(&dev));
  if (dev >= 64 || !configured[dev]) {
    JB_CUDA(cudaFuncSetAttribute(paged_decode_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)DpSmem<NT>::BYTES));
    if (dev < 64) configured[dev] = true;
  }
  JB_CUDA(launch_pdl(paged_decode_kernel<NT>, dim3(grid), dim3(DP_THREADS), DpSmem<NT>::BYTES, s, mk, mv, p));
  return JAMBA_OK;
}

jamba_status paged_decode(const PageGeom& g, int H, const void* q, long long ld_q, const void* k_pages,
                          const void* v_pages, const int* table, const int* lengths, void* o, long long ld_o,
                          float* lse, void* ws, cudaStream_t s) {
  const int grid = decode_grid(g);
  DpParams p;
  p.g = g;
  p.H = H;
  p.rep = H / g.G;
  p.q = reinterpret_cast<const bf16*>(q);
  p.ld_q = ld_q;
  p.table = table;
  p.lengths = lengths;
  p.o = reinterpret_cast<bf16*>(o);
  p.ld_o = ld_o;
  p.lse = lse;
  p.sl2 = 1.4426950408889634f / sqrtf((float)PG_D);
  p.meta = reinterpret_cast<DpMeta*>(ws);
  p.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + decode_meta_bytes(grid));
  p.err = device_error_word();
  CUtensorMap mk, mv;
  const uint64_t rows = (uint64_t)g.num_pages * g.G << g.shift;
  const uint32_t br = g.page() < DP_BK ? g.page() : DP_BK;
  JB_TRY(make_map_2d(&mk, k_pages, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, PG_D, rows, PG_D * 2, 64, br,
                     CU_TENSOR_MAP_SWIZZLE_128B));
  JB_TRY(make_map_2d(&mv, v_pages, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, PG_D, rows, PG_D * 2, 64, br,
                     CU_TENSOR_MAP_SWIZZLE_128B));
  if (p.rep <= 8)
    JB_TRY(launch_decode<1>(mk, mv, p, grid, s));
  else
    JB_TRY(launch_decode<2>(mk, mv, p, grid, s));
  JB_CUDA(launch_pdl(paged_decode_join_kernel, dim3(grid, p.rep), dim3(PG_D), 0, s, p, grid));
  return JAMBA_OK;
}

}  // namespace jb
