// Causal attention of a ragged batch of new tokens over the paged cache.
//
//   o_t = sum_j softmax_j(q_t . k_j / sqrt(d)) v_j over the positions j <= pos(t),
//   lse_t = log sum_j exp(q_t . k_j / sqrt(d)),
// in one pass over the keys with a running maximum and sum.
//
// Rows: the query heads of a KV head's group stand next to one another, row r of
// a tile is token r / rep, head r % rep, so that one token with a wide group, a few
// drafted tokens and a long chunk all fill the 128 rows of a tile from the same keys.  A
// unit is one sequence, one KV head and two such tiles (A and B); its work is the
// blocks of 128 keys that its last token sees.
//
// Work split: the blocks of all units, one after another, are cut into as many equal
// ranges as there are SMs, and a CTA walks its range.  A unit that ends inside the range
// it began in is written out at once; of one that crosses into other ranges each CTA
// writes its part (unnormalised o, maximum, sum) and paged_extend_join_kernel adds the
// parts in order.  So one long sequence, many short ones and mixtures of them all keep
// every SM equally long, and at most two parts per CTA go through memory.
//
// Per block: S = Q K^T (tcgen05, fp32 in tensor memory), softmax by four warps per tile, a
// thread per row; P goes back over S in tensor memory in bf16 and is the A operand of
// O += P V there.  Keys come K-major and values MN-major as the pages hold them: V needs
// no transposed copy.  The tensor core alternates between the tiles (O_A += P_A V_j,
// S_A(j+1), O_B += P_B V_j, S_B(j+1)), one tile's softmax runs under the other's products.
// The reference of the softmax is raised only when a row's maximum grows by more than 8
// (log2 units), then O is rescaled in tensor memory; terms stay below 2^8.  Rows of V behind
// the sequence's last token are zeroed in shared memory, their memory may hold anything.
// Every wait is bounded (see common.cuh).
#include "host.hpp"
#include "pages.cuh"

namespace jb {

constexpr int EX_BK = 128;                       // keys per block
constexpr int EX_SLOTS = 5;                      // ring of K and V blocks
constexpr int EX_THREADS = 384;                  // producer, MMA, two idle warps, 4 + 4 softmax warps
constexpr int EX_MIN_BLOCKS = 2;                 // of a CTA's range

struct ExSmem {
  static constexpr uint32_t SUB = 128 * 128;     // 128 rows x 64 bf16, swizzled
  static constexpr uint32_t Q_OFF = 0;           // Q_A, Q_B: dims 0-63 | 64-127 each
  static constexpr uint32_t KV_OFF = 4 * SUB;
  static constexpr uint32_t BAR_OFF = KV_OFF + EX_SLOTS * 2 * SUB;
  static constexpr uint32_t BYTES = BAR_OFF + 256 + 1024;
};

struct ExMeta {                                  // of a CTA's first and last item
  int tail, s, g, u;                             // tail: the last item begins a unit that ends in another CTA
  int head, ends;                                // head: the first item continues a unit; ends: and ends it
};

struct ExParams {
  PageGeom g;
  int H, rep, tokens;
  int tpt;                                       // tokens per tile: 128 / rep
  const int *q_start, *table, *lengths;
  bf16* o; long long ld_o;
  float* lse;
  float sl2;                                     // log2(e) / sqrt(head_dim)
  float *part_o, *part_ml;                       // [2 grid][256][128], [2 grid][256][2]
  ExMeta* meta;                                  // [grid]
  int fill;
  int* err;
};

// sum over i < n of floor((a i + b) / m), a, b >= 0 (Euclid-like reduction)
__device__ long long floor_sum(long long n, long long m, long long a, long long b) {
  long long r = 0;
  while (n > 0) {
    r += (a / m) * (n * (n - 1) / 2) + (b / m) * n;
    a %= m;
    b %= m;
    const long long y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const long long t = a;
    a = m;
    m = t;
  }
  return r;
}

// A sequence as the kernel sees it: n new tokens, rows q0 .. of the batch, the last of `len`.
struct ExSeq {
  int n, q0, len, units;
  __device__ void load(const ExParams& p, int s) {
    int a, b;
    token_range(p.q_start, s, p.tokens, a, b);
    n = b - a;
    q0 = a;
    len = clamp_len(p.g, p.lengths[s], p.err);
    const int tc = 2 * p.tpt;
    units = (n + tc - 1) / tc;
  }
  // blocks of unit u: at least one, so that tokens that see nothing get their zeros
  __device__ int blocks(const ExParams& p, int u) const {
    const int seen = len - n + min(n, (u + 1) * 2 * p.tpt);
    return seen <= EX_BK ? 1 : (seen + EX_BK - 1) / EX_BK;
  }
  // blocks of the units before u (of one KV head)
  __device__ long long before(const ExParams& p, int u) const {
    const long long tc = 2 * p.tpt, base = len - n;
    if (u <= 0) return 0;
    long long last = 0;
    if (u == units) {                            // the last unit may be short
      last = blocks(p, units - 1);
      --u;
    }
    // units 0 .. u-1 end at base + (i + 1) tc: ceil(x / 128) = floor((x + 127) / 128), 1 where x <= 0
    long long ones = 0;
    if (base < 0) {
      ones = -base / tc;                         // units that end at or before position 0
      if (ones > u) ones = u;
    }
    return last + ones + floor_sum(u - ones, EX_BK, tc, base + (ones + 1) * tc + EX_BK - 1);
  }
  __device__ long long total(const ExParams& p) const { return units ? before(p, units) * p.g.G : 0; }
};

// One stretch of blocks [kb0, kb1) of unit (s, g, u); every role walks the same items.
struct ExWalk {
  ExSeq q;
  int s, g, u, kb0, kb1, nb;                     // nb: blocks of the unit
  long long left;                                // blocks of the CTA's range from kb0 on
  __device__ bool open(const ExParams& p) {      // the item at (s, g, u, kb0)
    if (left <= 0) return false;
    nb = q.blocks(p, u);
    kb1 = (int)min((long long)nb, kb0 + left);
    return true;
  }
  __device__ bool next(const ExParams& p) {
    left -= kb1 - kb0;
    if (left <= 0) return false;
    kb0 = 0;
    if (++u == q.units) {
      u = 0;
      if (++g == p.g.G) {
        g = 0;
        do {
          if (++s >= p.g.S) return false;
          q.load(p, s);
        } while (q.units == 0);
      }
    }
    return open(p);
  }
  __device__ int tokens_of(const ExParams& p, int t) const {   // of tile t
    return max(0, min(p.tpt, q.n - (2 * u + t) * p.tpt));
  }
};

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// Instruction descriptor: as idesc_bf16 with B in MN-major order (bit 16)
constexpr uint32_t EX_IDESC_S = idesc_bf16(128, 128);
constexpr uint32_t EX_IDESC_PV = idesc_bf16(128, 128) | (1u << 16);

// Descriptor of V, MN-major, written by TMA with 128-byte swizzle: 64 head dims (128 bytes)
// per row, eight rows (keys) 1024 bytes on (stride offset), the next 64 dims one
// sub-tile on (leading offset).
__device__ __forceinline__ uint64_t v_desc(uint32_t smem_addr) {
  return (uint64_t)((smem_addr >> 4) & 0x3FFF) | ((uint64_t)(ExSmem::SUB >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// waits a short time for a phase, whatever the error word says
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try(bar, parity) && globaltimer() - t0 < 10000000ull) {
  }
}

__global__ void __launch_bounds__(EX_THREADS, 1)
paged_extend_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const ExParams p) {
  using S = ExSmem;
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long sh_left;
  __shared__ int sh_pos[4];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR_OFF);
  long long* sh_sum = reinterpret_cast<long long*>(smem + S::KV_OFF);   // until the first copies
  const uint32_t q_full = smem_u32(bars), q_empty = smem_u32(bars + 1);
  const uint32_t kv_full0 = smem_u32(bars + 2), kv_empty0 = smem_u32(bars + 2 + EX_SLOTS);
  const uint32_t land = smem_u32(bars + 2 + 2 * EX_SLOTS), drain = smem_u32(bars + 3 + 2 * EX_SLOTS);
  const uint32_t tb0 = smem_u32(bars + 4 + 2 * EX_SLOTS);   // per tile: S full, P full, O full
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 10 + 2 * EX_SLOTS);
#define S_FULL(t) (tb0 + 24 * (t))
#define P_FULL(t) (tb0 + 24 * (t) + 8)
#define O_FULL(t) (tb0 + 24 * (t) + 16)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0 && lane == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < EX_SLOTS; ++i) {
      mbar_init(kv_full0 + 8 * i, 1);
      mbar_init(kv_empty0 + 8 * i, 1);
    }
    mbar_init(land, 1);
    mbar_init(drain, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(S_FULL(t), 1);
      mbar_init(P_FULL(t), 4);
      mbar_init(O_FULL(t), 1);
    }
    mbar_fence_init();
    tma_prefetch(&tmQ);
    tma_prefetch(&tmK);
    tma_prefetch(&tmV);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_holder), 512);
  griddep_wait();
  griddep_launch();

  // the range of this CTA: its first block's sequence, head, unit and block
  {
    const int per_t = (p.g.S + EX_THREADS - 1) / EX_THREADS;
    const int s0 = threadIdx.x * per_t, s1 = min(p.g.S, s0 + per_t);
    long long sum = 0;
    for (int s = s0; s < s1; ++s) {
      ExSeq q;
      q.load(p, s);
      sum += q.total(p);
    }
    sh_sum[threadIdx.x] = sum;
    __syncthreads();
    if (warp == 0) {                             // inclusive scan, twelve sums a lane
      long long mine = 0;
      for (int i = 0; i < EX_THREADS / 32; ++i) mine += sh_sum[lane * (EX_THREADS / 32) + i];
      long long x = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      long long at = x - mine;
      for (int i = 0; i < EX_THREADS / 32; ++i) {
        at += sh_sum[lane * (EX_THREADS / 32) + i];
        sh_sum[lane * (EX_THREADS / 32) + i] = at;
      }
    }
    __syncthreads();
    const long long N = sh_sum[EX_THREADS - 1];
    long long per = (N + gridDim.x - 1) / gridDim.x;
    if (per < EX_MIN_BLOCKS) per = EX_MIN_BLOCKS;
    const long long a = min(N, blockIdx.x * per), b = min(N, a + per);
    const long long mine0 = sh_sum[threadIdx.x] - sum;
    if (b > a && a >= mine0 && a < mine0 + sum) {
      long long rem = a - mine0;
      ExSeq q;
      for (int s = s0; s < s1; ++s) {
        q.load(p, s);
        const long long t = q.total(p);
        if (rem < t) {
          const long long head = t / p.g.G;
          const int g = (int)(rem / head);
          rem -= g * head;
          int lo = 0, hi = q.units;              // before(lo) <= rem < before(hi)
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (q.before(p, mid) <= rem) lo = mid; else hi = mid;
          }
          sh_pos[0] = s;
          sh_pos[1] = g;
          sh_pos[2] = lo;
          sh_pos[3] = (int)(rem - q.before(p, lo));
          break;
        }
        rem -= t;
      }
    }
    if (threadIdx.x == 0) sh_left = b - a;
  }
  fence_async_shared();                          // the sums' memory goes to the copies
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;           // tile t: S and P at 256 t, O at 256 t + 128
  ExWalk w;
  w.left = sh_left;
  const bool any = w.left > 0;
  if (any) {
    w.s = sh_pos[0];
    w.g = sh_pos[1];
    w.u = sh_pos[2];
    w.kb0 = sh_pos[3];
    w.q.load(p, w.s);
  }
  const bool mid_start = any && w.kb0 > 0;       // the first item continues a unit

  // registers go from the first four warps to the softmax warps: 128 * (88 + 208 + 208) = 384 * 168
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == 0) {
    // ---- producer: lane i loads page i of a block
    const int br = min(p.g.page(), EX_BK);       // rows of a box
    int kv = 0, items = 0, landed = 0;
    bool ok = true;
    auto load_block = [&](const CUtensorMap* m, int kb, bool is_v) {
      const int slot = kv % EX_SLOTS;
      if (!mbar_wait_warp(kv_empty0 + 8 * slot, ((kv / EX_SLOTS) & 1) ^ 1, p.err)) return false;
      const uint32_t dst = smem_u32(smem + S::KV_OFF + slot * 2 * S::SUB);
      const int valid = max(0, min(EX_BK, w.q.len - kb * EX_BK));
      const int nbox = (valid + br - 1) / br;
      const bool part = is_v && valid < EX_BK;   // rows behind the last token
      const uint32_t bar = part ? land : kv_full0 + 8 * slot;
      if (lane == 0) mbar_arrive_tx(bar, nbox * br * 256);
      __syncwarp();
      if (lane < nbox) {
        const int pos = kb * EX_BK + lane * br;
        const int e = max(0, good_page(p.g, p.table[(long long)w.s * p.g.ld_table + (pos >> p.g.shift)], p.err));
        const int row = ((e * p.g.G + w.g) << p.g.shift) + (pos & (p.g.page() - 1));
        tma_load_2d(dst + lane * br * 128, m, bar, 0, row);
        tma_load_2d(dst + S::SUB + lane * br * 128, m, bar, 64, row);
      }
      if (part) {
        if (!mbar_wait_warp(land, landed & 1, p.err)) return false;
        ++landed;
        uint8_t* base = smem + S::KV_OFF + slot * 2 * S::SUB;
        for (int i = lane; i < (EX_BK - valid) * 16; i += 32) {
          const int row = valid + (i >> 4), c = i & 15;
          *reinterpret_cast<uint4*>(base + (c >> 3) * S::SUB + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(kv_full0 + 8 * slot);
      }
      ++kv;
      return true;
    };
    for (bool more = w.open(p); more && ok; more = w.next(p), ++items) {
      ok = mbar_wait_warp(q_empty, (items & 1) ^ 1, p.err);
      if (!ok) break;
      const int nt = w.tokens_of(p, 1) > 0 ? 2 : 1;
      if (lane == 0) {
        mbar_arrive_tx(q_full, nt * p.tpt * p.rep * 256);
        for (int t = 0; t < nt; ++t)
          for (int h = 0; h < 2; ++h)
            tma_load_3d(smem_u32(smem + S::Q_OFF + (2 * t + h) * S::SUB), &tmQ, q_full, 64 * h, w.g * p.rep,
                        w.q.q0 + (2 * w.u + t) * p.tpt);
      }
      __syncwarp();
      for (int kb = w.kb0; kb < w.kb1 && ok; ++kb) ok = load_block(&tmK, kb, false) && load_block(&tmV, kb, true);
    }
    if (!ok) {   // gave up: let the copies in flight land before the CTA ends
      for (int i = max(0, kv - EX_SLOTS); i < kv; ++i) drain_wait(kv_full0 + 8 * (i % EX_SLOTS), (i / EX_SLOTS) & 1);
      drain_wait(q_full, items & 1);
      drain_wait(land, landed & 1);
    }
  } else if (warp == 1) {
    // ---- MMA issuer
    if (lane == 0) {
      int kv = 0, items = 0, np[2] = {0, 0};
      bool ok = true;
      auto kv_base = [&](int i) { return smem_u32(smem + S::KV_OFF + (i % EX_SLOTS) * 2 * S::SUB); };
      auto wait_kv = [&](int i) { return mbar_wait(kv_full0 + 8 * (i % EX_SLOTS), (i / EX_SLOTS) & 1, p.err); };
      auto issue_s = [&](int t, int i) {
        const uint32_t kb = kv_base(i), qb = smem_u32(smem + S::Q_OFF + 2 * t * S::SUB);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_bf16(tbase + 256 * t, sw128_desc(qb + (kk >> 2) * S::SUB) + 2 * (kk & 3),
                    sw128_desc(kb + (kk >> 2) * S::SUB) + 2 * (kk & 3), EX_IDESC_S, kk > 0 ? 1u : 0u);
        umma_commit(S_FULL(t));
      };
      auto issue_pv = [&](int t, int i, bool first) {
        const uint64_t vd = v_desc(kv_base(i));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)   // 16 keys a step: 2048 bytes of V, 8 columns of P
          umma_bf16_ta(tbase + 256 * t + 128, tbase + 256 * t + 8 * kk, vd + 128 * kk, EX_IDESC_PV,
                       (!first || kk > 0) ? 1u : 0u);
      };
      for (bool more = w.open(p); more && ok; more = w.next(p), ++items) {
        const int nt = w.tokens_of(p, 1) > 0 ? 2 : 1, nbk = w.kb1 - w.kb0;
        ok = mbar_wait(q_full, items & 1, p.err) && wait_kv(kv);
        if (!ok) break;
        tc_fence_after();
        for (int t = 0; t < nt; ++t) issue_s(t, kv);
        umma_commit(kv_empty0 + 8 * (kv % EX_SLOTS));
        if (nbk == 1) umma_commit(q_empty);
        for (int j = 0; j < nbk && ok; ++j) {
          const int vi = kv + 2 * j + 1, ki = kv + 2 * j + 2;
          const bool last = j + 1 == nbk;
          ok = wait_kv(vi);
          for (int t = 0; t < nt && ok; ++t) {
            ok = mbar_wait(P_FULL(t), np[t] & 1, p.err);
            if (!ok) break;
            ++np[t];
            tc_fence_after();
            issue_pv(t, vi, j == 0);
            if (t == nt - 1) umma_commit(kv_empty0 + 8 * (vi % EX_SLOTS));
            if (last) {
              umma_commit(O_FULL(t));
            } else {
              if (t == 0) {
                ok = wait_kv(ki);
                if (!ok) break;
                tc_fence_after();
              }
              issue_s(t, ki);
              if (t == nt - 1) {
                umma_commit(kv_empty0 + 8 * (ki % EX_SLOTS));
                if (j + 2 == nbk) umma_commit(q_empty);
              }
            }
          }
        }
        kv += 2 * nbk;
      }
      umma_commit(drain);
      drain_wait(drain, 0);
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---- softmax of tile t: thread = row
    const int t = (warp - 4) >> 2, q4 = warp & 3, r = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tbase + 256 * t + lane_off, tO = tS + 128;
    const int tok_r = r / p.rep, head_r = r % p.rep;
    int ns = 0, no = 0;
    bool ok = true, first_item = true;
    for (bool more = w.open(p); more && ok; more = w.next(p), first_item = false) {
      const int nt = w.tokens_of(p, t);
      const bool whole = w.kb0 == 0 && w.kb1 == w.nb;
      if (r == 0 && t == 0) {
        ExMeta* m = p.meta + blockIdx.x;
        if (first_item) {
          m->head = mid_start;
          m->ends = w.kb1 == w.nb;
        }
        const bool tail = w.kb0 == 0 && w.kb1 < w.nb;   // only the last item can be one
        m->tail = tail;
        m->s = w.s;
        m->g = w.g;
        m->u = w.u;
      }
      if (nt == 0) continue;                     // the unit has no tile B
      const int tok = (2 * w.u + t) * p.tpt + tok_r;   // of the sequence's new tokens
      const bool row_in = tok_r < nt;
      const int pos = row_in ? w.q.len - w.q.n + tok : -1;
      float m = -INFINITY, l = 0.f;
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++ns) {
        ok = mbar_wait_warp(S_FULL(t), ns & 1, p.err);
        if (!ok) break;
        tc_fence_after();
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, s + 32 * c);
        tmem_wait_ld();
        const int lim = pos - kb * EX_BK;        // keys c <= lim are seen
        if (!__all_sync(0xffffffffu, lim >= EX_BK - 1)) {
#pragma unroll
          for (int c = 0; c < EX_BK; ++c)
            if (c > lim) s[c] = -INFINITY;
        }
        float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < 124; c += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) mx4[i] = max3(mx4[i], s[c + i], s[c + 4 + i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) mx4[i] = fmaxf(mx4[i], s[124 + i]);
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.sl2;
        float corr = 1.f;
        if (mx > m + 8.f) {                      // also the first finite maximum (m = -inf)
          corr = ex2(m - mx);
          m = mx;
        }
        // the products that read O's last value are done: S_j was issued after them
        if (kb > w.kb0 && __any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k2 = 0; k2 < 32; ++k2) o[k2] *= corr;
            tmem_st32(tO + 32 * c, o);
          }
          tmem_wait_st();
        }
        const float ref = m == -INFINITY ? 0.f : -m;
        const float2 sl = make_float2(p.sl2, p.sl2), rf = make_float2(ref, ref);
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 x = ffma2(make_float2(s[64 * hf + 2 * i], s[64 * hf + 2 * i + 1]), sl, rf);
            const float ea = ex2(x.x), eb = ex2(x.y);
            sum[i & 3] += ea + eb;
            __nv_bfloat162 hh = __floats2bfloat162_rn(ea, eb);
            pk[i] = *reinterpret_cast<uint32_t*>(&hh);
          }
          tmem_st32u(tS + 32 * hf, pk);
        }
        l = l * corr + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(P_FULL(t));
      }
      if (!ok) break;
      ok = mbar_wait_warp(O_FULL(t), no & 1, p.err);
      ++no;
      if (!ok) break;
      tc_fence_after();
      if (whole) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const long long row = w.q.q0 + tok;
        const int head = w.g * p.rep + head_r;
        bf16* dst = p.o + row * p.ld_o + (long long)head * PG_D;
        if (row_in && p.lse)
          p.lse[row * p.H + head] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float o[32];
          tmem_ld32(tO + 32 * c, o);
          tmem_wait_ld();
          if (row_in) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint4 u;
              __nv_bfloat162* hh = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
              for (int i = 0; i < 4; ++i) hh[i] = __floats2bfloat162_rn(o[8 * k + 2 * i] * inv, o[8 * k + 2 * i + 1] * inv);
              *reinterpret_cast<uint4*>(dst + 32 * c + 8 * k) = u;
            }
          }
        }
      } else {
        const int slot = 2 * blockIdx.x + (w.kb0 == 0);   // continued: 0, begun here: 1
        float* dst = p.part_o + ((long long)slot * 256 + t * 128 + r) * PG_D;
        if (row_in) *reinterpret_cast<float2*>(p.part_ml + ((long long)slot * 256 + t * 128 + r) * 2) = make_float2(m, l);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float o[32];
          tmem_ld32(tO + 32 * c, o);
          tmem_wait_ld();
          if (row_in) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<float4*>(dst + 32 * c + 4 * k) = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
      }
      tc_fence_before();   // O is read before the next item's first product is issued (after its P)
    }
    if (!any && r == 0 && t == 0) {
      p.meta[blockIdx.x].tail = 0;
      p.meta[blockIdx.x].head = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}
#undef S_FULL
#undef P_FULL
#undef O_FULL

// CTA (c, y): rows 32 y .. of the unit whose parts begin in CTA c of the kernel above, a warp per
// row: o = sum of o_i 2^(m_i - m) / sum of l_i 2^(m_i - m), in the order of the parts.
// With fill, rows that no sequence counts are zeroed too.
__global__ void __launch_bounds__(256)
paged_extend_join_kernel(const ExParams p) {
  griddep_wait();
  griddep_launch();
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (p.fill) {
    const int a = max(0, min(p.q_start[0], p.tokens)), b = max(0, min(p.q_start[p.g.S], p.tokens));
    const int cta = blockIdx.y * gridDim.x + c, ctas = gridDim.x * gridDim.y;
    for (int r = cta; r < a + p.tokens - b; r += ctas) {
      bf16* dst = p.o + (long long)(r < a ? r : r - a + b) * p.ld_o;
      for (int i = threadIdx.x; i < p.H * (PG_D / 8); i += 256)
        *reinterpret_cast<uint4*>(dst + i * 8) = make_uint4(0, 0, 0, 0);
    }
  }
  const ExMeta me = p.meta[c];
  if (!me.tail) return;
  int parts = 2;
  while (c + parts < (int)gridDim.x && !p.meta[c + parts - 1].ends) ++parts;   // CTA c + i continues the unit; the last one ends it
  ExSeq q;
  q.load(p, me.s);
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int rr = blockIdx.y * 32 + warp * 4 + i, t = rr >> 7, r = rr & 127;
    const int tok_r = r / p.rep, tok = (2 * me.u + t) * p.tpt + tok_r;
    if (tok_r >= p.tpt || tok >= q.n) continue;
    auto slot = [&](int k) { return (long long)(k == 0 ? 2 * c + 1 : 2 * (c + k)) * 256 + rr; };
    float mm = -INFINITY;
    for (int k = 0; k < parts; ++k) mm = fmaxf(mm, p.part_ml[slot(k) * 2]);
    float ls = 0.f;
    float4 os = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < parts; ++k) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + slot(k) * 2);
      const float4 x = *reinterpret_cast<const float4*>(p.part_o + slot(k) * PG_D + lane * 4);
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mm);
      ls += ml.y * f;
      os.x += x.x * f;
      os.y += x.y * f;
      os.z += x.z * f;
      os.w += x.w * f;
    }
    const float inv = ls > 0.f ? 1.f / ls : 0.f;
    const long long row = q.q0 + tok;
    const int head = me.g * p.rep + r % p.rep;
    __nv_bfloat162 h01 = __floats2bfloat162_rn(os.x * inv, os.y * inv), h23 = __floats2bfloat162_rn(os.z * inv, os.w * inv);
    uint2 u;
    u.x = *reinterpret_cast<uint32_t*>(&h01);
    u.y = *reinterpret_cast<uint32_t*>(&h23);
    *reinterpret_cast<uint2*>(p.o + row * p.ld_o + (long long)head * PG_D + lane * 4) = u;
    if (p.lse && lane == 0)
      p.lse[row * p.H + head] = ls > 0.f ? (mm + log2f(ls)) * 0.6931471805599453f : -INFINITY;
  }
}

static size_t al256(size_t v) { return (v + 255) & ~size_t(255); }

size_t paged_extend_workspace_bytes() {
  const size_t slots = 2 * (size_t)num_sms() * 256;
  return al256(slots * PG_D * 4) + al256(slots * 8) + al256(num_sms() * sizeof(ExMeta));
}

jamba_status paged_extend(const PageGeom& g, int H, const void* q, long long ld_q, int tokens, const int* q_start,
                          const void* k_pages, const void* v_pages, const int* table, const int* lengths, void* o,
                          long long ld_o, float* lse, bool fill, void* ws, cudaStream_t s) {
  ExParams p;
  const int grid = num_sms();
  const size_t slots = 2 * (size_t)grid * 256;
  uint8_t* b = reinterpret_cast<uint8_t*>(ws);
  p.g = g;
  p.H = H;
  p.rep = H / g.G;
  p.tokens = tokens;
  p.tpt = 128 / p.rep;
  p.q_start = q_start;
  p.table = table;
  p.lengths = lengths;
  p.o = reinterpret_cast<bf16*>(o);
  p.ld_o = ld_o;
  p.lse = lse;
  p.sl2 = 1.4426950408889634f / sqrtf((float)PG_D);
  p.part_o = reinterpret_cast<float*>(b);
  p.part_ml = reinterpret_cast<float*>(b + al256(slots * PG_D * 4));
  p.meta = reinterpret_cast<ExMeta*>(b + al256(slots * PG_D * 4) + al256(slots * 8));
  p.fill = fill;
  p.err = device_error_word();
  CUtensorMap mq, mk, mv;
  const uint64_t rows = (uint64_t)g.num_pages * g.G << g.shift;
  const uint32_t br = g.page() < EX_BK ? g.page() : EX_BK;
  JB_TRY(make_map_3d(&mq, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, PG_D, H, tokens, PG_D * 2, (uint64_t)ld_q * 2, 64,
                     p.rep, CU_TENSOR_MAP_SWIZZLE_128B, p.tpt));
  JB_TRY(make_map_2d(&mk, k_pages, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, PG_D, rows, PG_D * 2, 64, br,
                     CU_TENSOR_MAP_SWIZZLE_128B));
  JB_TRY(make_map_2d(&mv, v_pages, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, PG_D, rows, PG_D * 2, 64, br,
                     CU_TENSOR_MAP_SWIZZLE_128B));
  static std::atomic<bool> configured[64];
  int dev = 0;
  JB_CUDA(cudaGetDevice(&dev));
  if (dev < 64 && !configured[dev]) {
    JB_CUDA(cudaFuncSetAttribute(paged_extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ExSmem::BYTES));
    configured[dev] = true;
  }
  JB_CUDA(launch_pdl(paged_extend_kernel, dim3(grid), dim3(EX_THREADS), ExSmem::BYTES, s, mq, mk, mv, p));
  JB_CUDA(launch_pdl(paged_extend_join_kernel, dim3(grid, 8), dim3(256), 0, s, p));
  return JAMBA_OK;
}

}  // namespace jb
