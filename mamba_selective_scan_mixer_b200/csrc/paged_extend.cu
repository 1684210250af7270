// Causal attention of a ragged batch of new tokens over the paged cache.
//
//   o_t = sum_j softmax_j(q_t . k_j / sqrt(d)) v_j over the positions j <= pos(t),
//   lse_t = log sum_j exp(q_t . k_j / sqrt(d)),
// in one pass over the keys with a running reference and sum of the exponentials.
//
// Rows: the query heads of a KV head's group stand next to one another, row r of a tile is token
// r / rep, head r % rep, so that one token with a wide group, a few drafted tokens and a long chunk
// all fill the 128 rows of a tile from the same keys.  A unit is one sequence, one KV head and two
// such tiles (A and B); its work is the blocks of 128 keys that its last token sees.
//
// Work split: the blocks of all units, one after another, are cut by cost into as many equal ranges
// as there are SMs, and a CTA walks its range.  A unit that ends inside the range it began in is
// written out at once; of one that crosses into other ranges each CTA writes its part (unnormalised
// o, reference, sum) and paged_extend_join_kernel adds the parts in order.  So one long sequence,
// many short ones and mixtures of them keep every SM equally long, and at most two parts per CTA go
// through memory.
//
// Per block and tile: S = Q K^T (tcgen05, fp32 in tensor memory), softmax by eight warps, two rows to
// four lanes; P goes back over S in tensor memory in bf16 and is the A operand of O += P V there.
// Keys come K-major and values MN-major as the pages hold them: V needs no transposed copy.  The
// tiles take turns at the tensor core (O_A += P_A V_j and S_A(j+1), then the same of B), each issued
// by a warp of its own, and one tile's softmax runs under the other's products.  One softmax
// reference per row: terms are formed against the one from the blocks before (0 for a first block
// without a mask), so scores are read once and no maximum is looked for; when a row's terms add up to
// more than 2^16 it is raised for the next block, by a power of two, and O is then rescaled in tensor
// memory.  Rows of V behind the sequence's last token are zeroed in shared memory, their memory may
// hold anything.
//
// Rounding: P is bf16 (the tensor core's type; the sum is taken before), o is rounded once from fp32.
//
// Bounds: chunks by the tensor core and the softmax it waits for.  4096 tokens behind 12288, 32 heads
// on 8: 0.885 ms, 1.09 PFLOP/s, 0.66 of the burst rate and 0.80 of the sustained one (the card holds
// 1.55 to 1.65 GHz under it): a pair of blocks takes about 3600 cycles, its four products 2500 with
// the shared memory's other traffic, the rest is the chain softmax (1600) -> products (1270) -> the
// next wait.  Measured there, when this form took 0.87 ms: a maximum taken of every block and the reference
// raised from 2^8 on 0.95 ms; before that without turns 1.07 ms; P handed over in halves 1.03 ms; 64-key
// blocks with two score buffers a tile 1.18 ms; all 16 warps on one tile's softmax 1.20 ms.  24 sequences
// of 1 to 1500 tokens behind up to 6000: 0.146 ms (one warp issuing for both tiles 0.245 ms).  A few
// drafted tokens (32 sequences of 5 behind 300 to 4096): 58 us, by the latency of a block, at half the
// rate that reading their pages allows.  Every wait is bounded (see common.cuh).
#include <climits>

#include "host.hpp"
#include "pages.cuh"

namespace jb {

constexpr int EX_BK = 128;                       // keys per block
constexpr int EX_SLOTS = 5;                      // ring of K and V blocks
constexpr int EX_THREADS = 640;                  // producer, an MMA warp per tile, V tails, 8 + 8 softmax warps
constexpr int EX_MIN_COST = 4;                   // of a CTA's range
constexpr int EX_UNIT_COST = 2;                  // what a unit costs beyond its blocks (Q, output), in blocks

struct ExSmem {
  static constexpr uint32_t SUB = 128 * 128;     // 128 rows x 64 bf16, swizzled
  static constexpr uint32_t Q_OFF = 0;           // Q_A, Q_B: dims 0-63 | 64-127 each
  static constexpr uint32_t KV_OFF = 4 * SUB;
  static constexpr uint32_t BAR_OFF = KV_OFF + EX_SLOTS * 2 * SUB;
  static constexpr uint32_t BYTES = BAR_OFF + 256 + 1024;
};

struct ExMeta {                                  // of a CTA's first and last item
  int tail, s, g, u;                             // tail: the last item begins a unit that ends in another CTA
  int ends;                                      // the first item ends its unit
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

// sum over i < n of floor((a i + b) / m) (Euclid-like reduction); a n + b below 2^32
__device__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  long long r = 0;
  while (n > 0) {
    r += (long long)(a / m) * ((long long)n * (n - 1) / 2) + (long long)(b / m) * n;
    a %= m;
    b %= m;
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const uint32_t t = a;
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
  // cost of the units before u (of one KV head)
  __device__ long long before(const ExParams& p, int u) const {
    const int tc = 2 * p.tpt, base = len - n;
    if (u <= 0) return 0;
    long long last = (long long)EX_UNIT_COST * u;
    if (u == units) {                            // the last unit may be short
      last += blocks(p, units - 1);
      --u;
    }
    // units 0 .. u-1 end at base + (i + 1) tc: ceil(x / 128) = floor((x + 127) / 128), 1 where x <= 0
    int ones = 0;
    if (base < 0) ones = min(-base / tc, u);     // units that end at or before position 0
    return last + ones + floor_sum(u - ones, EX_BK, tc, base + (ones + 1) * tc + EX_BK - 1);
  }
  __device__ long long total(const ExParams& p) const { return units ? before(p, units) * p.g.G : 0; }
};

// One stretch of blocks [kb0, kb1) of unit (s, g, u); every role walks the same items.  Ranges are
// cut by cost: a unit is EX_UNIT_COST steps without a block, then a step per block.
struct ExWalk {
  ExSeq q;
  int s, g, u, kb0, kb1, nb;                     // nb: blocks of the unit
  long long at, left;                            // step of the unit at the item's start, steps of the range from there
  __device__ bool open(const ExParams& p) {      // the item at (s, g, u, at); false: no block is left
    if (left <= 0) return false;
    nb = q.blocks(p, u);
    kb0 = max(0, (int)at - EX_UNIT_COST);
    kb1 = max(0, (int)min((long long)nb, at + left - EX_UNIT_COST));
    return kb1 > kb0;
  }
  __device__ bool next(const ExParams& p) {
    left -= EX_UNIT_COST + nb - at;
    if (left <= 0) return false;
    at = 0;
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

// a row's terms in one block add up to more than this: the reference is raised, to even the exponents
constexpr float EX_MAX_SUM = 0x1p16f;
// ... to more than this, or to less than EX_MIN_SUM in a first block: the block is formed again.  So |O| stays below
// 2^40 max |v| (2^23 blocks of up to EX_MAX_SUM, one of up to EX_FAR), and of a row's terms the largest above 2^-40:
// values from 2^-80 to 2^80 in size keep fp32's precision in the products.
constexpr float EX_FAR = 0x1p32f, EX_MIN_SUM = 0x1p-32f;

// Softmax warps hold 16 rows of a tile each: in tcgen05.ld / st .16x256b and .16x128b a row's columns
// lie over the four lanes of a quad (lane i: rows i / 4 and i / 4 + 8; of each 8 columns of 32
// bits numbers 2 (i % 4) and the next; of each 4 columns of packed bf16 number i % 4), so a thread
// has 32 scores of two rows, and a row's maximum and sum are two shuffles away.
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, float (&v)[16]) {   // 32 columns
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_16x256b(uint32_t taddr, const float (&v)[16]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_16x128b(uint32_t taddr, const uint32_t (&r)[32]) {   // 64 columns
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// waits for the loads so far, tied to the registers of one (see tmem_wait_ld32)
__device__ __forceinline__ void tmem_wait_ld16(float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ float nan_max(float a, float b) {   // NaN where either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
// column of register k of 32-column chunk c in a .16x256b load; its row is k & 2 (0: lane / 4, 2: + 8)
__device__ __forceinline__ int chunk_col(int c, int k, int quad) { return 32 * c + 8 * (k >> 2) + 2 * quad + (k & 1); }

// the largest score of the thread's two rows in one block (raw, before the scale), keys past lim left out when masked
__device__ __forceinline__ void ex_row_max(uint32_t tS, bool masked, const int (&lim)[2], int quad, float (&mx)[2]) {
  mx[0] = mx[1] = -INFINITY;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float v[16];
    tmem_ld_16x256b(tS + 32 * c, v);
    tmem_wait_ld16(v);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int e = (k >> 1) & 1;
      mx[e] = fmaxf(mx[e], masked && chunk_col(c, k, quad) > lim[e] ? -INFINITY : v[k]);
    }
  }
  mx[0] = quad_max(mx[0]);
  mx[1] = quad_max(mx[1]);
}

constexpr int EX_FMA_EVERY = 4;    // of the pairs of terms, one in so many goes to ex2_fma
constexpr float EXC0 = 0.99999926144f, EXC1 = 0.69312181475f, EXC2 = 0.24024744849f, EXC3 = 0.05591786025f,
                EXC4 = 0.00957010107f;

// 2^x for both halves on the FMA pipe, x taken into [-126, 127]: the nearest integer n through the
// mantissa of x + 1.5 2^23, a degree-4 polynomial for 2^f with f = x - n in [-1/2, 1/2] (fitted for
// the least largest relative error, 2.6e-6; P keeps 2^-9), and n added to its exponent.  Below the range the
// result, some 2^-126, is as good as none; above it and for a NaN it is at least 2^126, which the row's sum
// shows.  Without the upper limit the exponent would run into the sign and a far key vanish.  Takes some of the
// terms because ex2 alone runs at 16 a cycle and SM: 128 x 256 terms take the 2048 cycles that their
// four products take.  The upper limit costs 1.3 % of a chunk (873 to 884 us).
__device__ __forceinline__ float2 ex2_fma(float2 x) {
  const float big = 12582912.f;
  x.x = fminf(nan_max(x.x, -126.f), 127.f);      // a NaN becomes 127
  x.y = fminf(nan_max(x.y, -126.f), 127.f);
  const float2 one = make_float2(1.f, 1.f);
  const float2 t = ffma2(x, one, make_float2(big, big));
  const float2 n = ffma2(t, one, make_float2(-big, -big));
  const float2 f = ffma2(n, make_float2(-1.f, -1.f), x);
  float2 y = make_float2(EXC4, EXC4);
  y = ffma2(y, f, make_float2(EXC3, EXC3));
  y = ffma2(y, f, make_float2(EXC2, EXC2));
  y = ffma2(y, f, make_float2(EXC1, EXC1));
  y = ffma2(y, f, make_float2(EXC0, EXC0));
  return make_float2(__int_as_float(__float_as_int(y.x) + (__float_as_int(t.x) << 23)),
                     __int_as_float(__float_as_int(y.y) + (__float_as_int(t.y) << 23)));
}

// The terms 2^(s sl2 + ref) of the thread's two rows in bf16 pairs, and their sums (before rounding) over the
// thread's own columns.
template <bool MASKED>
__device__ __forceinline__ void ex_terms_t(uint32_t tS, const int (&lim)[2], int quad, const float (&ref)[2], float sl2,
                                           uint32_t (&pk)[32], float (&sum)[2]) {
  const float2 sl = make_float2(sl2, sl2);
  float2 sm[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  float s[2][16];
  tmem_ld_16x256b(tS, s[0]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float(&v)[16] = s[c & 1];
    tmem_wait_ld16(v);
    if (c < 3) tmem_ld_16x256b(tS + 32 * (c + 1), s[(c + 1) & 1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {                // pairs of columns: group i / 2, row i % 2
      const int e = i & 1;
      float a = v[2 * i], b = v[2 * i + 1];
      if (MASKED) {
        if (chunk_col(c, 2 * i, quad) > lim[e]) a = -INFINITY;
        if (chunk_col(c, 2 * i + 1, quad) > lim[e]) b = -INFINITY;
      }
      const float2 x = ffma2(make_float2(a, b), sl, make_float2(ref[e], ref[e]));
      float2 t;
      if (!MASKED && i % EX_FMA_EVERY == EX_FMA_EVERY - 1 - (c & 1))   // masked scores: their terms are exactly 0
        t = ex2_fma(x);
      else
        t = make_float2(ex2(x.x), ex2(x.y));
      sm[e] = ffma2(t, make_float2(1.f, 1.f), sm[e]);
      __nv_bfloat162 hh = __floats2bfloat162_rn(t.x, t.y);
      pk[8 * c + i] = *reinterpret_cast<uint32_t*>(&hh);
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) sum[e] = sm[e].x + sm[e].y;
}
__device__ __forceinline__ void ex_terms(uint32_t tS, bool masked, const int (&lim)[2], int quad, const float (&m)[2],
                                         float sl2, uint32_t (&pk)[32], float (&sum)[2]) {
  const float ref[2] = {m[0] == -INFINITY ? 0.f : -m[0], m[1] == -INFINITY ? 0.f : -m[1]};
  if (masked)
    ex_terms_t<true>(tS, lim, quad, ref, sl2, pk, sum);
  else
    ex_terms_t<false>(tS, lim, quad, ref, sl2, pk, sum);
}
// w[g] of lane l of a quad becomes w[l] of lane g
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int quad) {
#pragma unroll
  for (int b = 1; b < 4; b <<= 1) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (g & b) continue;
      const bool up = quad & b;
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[g] : w[g | b], b);
      if (up) w[g] = got; else w[g | b] = got;
    }
  }
}

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

// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(ok));
  return ok != 0;
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
  __shared__ long long sh_left, sh_rem, sh_warp[EX_THREADS / 32];
  __shared__ ExSeq sh_seq;
  __shared__ int sh_pos[4];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR_OFF);
  const uint32_t q_full = smem_u32(bars), q_empty = smem_u32(bars + 1);
  const uint32_t kv_full0 = smem_u32(bars + 2), kv_empty0 = smem_u32(bars + 2 + EX_SLOTS);
  const uint32_t land0 = smem_u32(bars + 2 + 2 * EX_SLOTS);   // a V block with rows to be zeroed has landed
  const uint32_t tb0 = smem_u32(bars + 2 + 3 * EX_SLOTS);     // per tile: S full, P full, O full, drained
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 10 + 3 * EX_SLOTS);
#define S_FULL(t) (tb0 + 32 * (t))
#define P_FULL(t) (tb0 + 32 * (t) + 8)
#define O_FULL(t) (tb0 + 32 * (t) + 16)
#define DRAINED(t) (tb0 + 32 * (t) + 24)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0 && lane == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);                       // both MMA warps
    for (int i = 0; i < EX_SLOTS; ++i) {
      mbar_init(kv_full0 + 8 * i, 1);
      mbar_init(kv_empty0 + 8 * i, 2);
      mbar_init(land0 + 8 * i, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(S_FULL(t), 1);
      mbar_init(P_FULL(t), 9);                   // the softmax warps, and whoever passes the turn on
      mbar_init(O_FULL(t), 1);
      mbar_init(DRAINED(t), 1);
    }
    mbar_fence_init();
    tma_prefetch(&tmQ);
    tma_prefetch(&tmK);
    tma_prefetch(&tmV);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_holder), 512);
  griddep_wait();
  griddep_launch();

  // the range of this CTA: where it starts (sequence, head, unit, step) and its length
  {
    const int per_t = (p.g.S + EX_THREADS - 1) / EX_THREADS;
    const int s0 = threadIdx.x * per_t, s1 = min(p.g.S, s0 + per_t);
    long long sum = 0;
    ExSeq q;
    for (int s = s0; s < s1; ++s) {
      q.load(p, s);
      sum += q.total(p);
    }
    long long x = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh_warp[warp] = x;
    __syncthreads();
    long long N = 0, mine0 = x - sum;
    for (int i = 0; i < EX_THREADS / 32; ++i) {
      if (i < warp) mine0 += sh_warp[i];
      N += sh_warp[i];
    }
    long long per = (N + gridDim.x - 1) / gridDim.x;
    if (per < EX_MIN_COST) per = EX_MIN_COST;
    const long long a = min(N, blockIdx.x * per), b = min(N, a + per);
    if (b > a && a >= mine0 && a < mine0 + sum) {
      long long rem = a - mine0;
      for (int s = s0; s < s1; ++s) {
        if (s1 - s0 > 1) q.load(p, s);
        const long long head = q.units ? q.before(p, q.units) : 0, all = head * p.g.G;
        if (rem < all) {
          const int g = (int)(rem / head);
          sh_pos[0] = s;
          sh_pos[1] = g;
          sh_rem = rem - g * head;
          sh_seq = q;
          break;
        }
        rem -= all;
      }
    }
    if (threadIdx.x == 0) sh_left = b - a;
  }
  __syncthreads();
  if (warp == 0 && sh_left > 0) {                // the unit: before(lo) <= sh_rem < before(hi), 32 places at a time
    const ExSeq q = sh_seq;
    int lo = 0, hi = q.units;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const uint32_t below = __ballot_sync(0xffffffffu, at < hi && q.before(p, at) <= sh_rem);
      lo += (31 - __clz(below)) * step;          // lane 0's place is always below
      hi = min(hi, lo + step);
    }
    if (lane == 0) {
      sh_pos[2] = lo;
      sh_pos[3] = (int)(sh_rem - q.before(p, lo));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;           // tile t: S and P at 256 t, O at 256 t + 128
  ExWalk w;
  w.left = sh_left;
  if (w.left > 0) {
    w.s = sh_pos[0];
    w.g = sh_pos[1];
    w.u = sh_pos[2];
    w.at = sh_pos[3];
    w.q = sh_seq;
  }

  // registers go from the first four warps to the softmax warps: 128 * 64 + 512 * 104 = 640 * 96
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  if (warp == 0) {
    // ---- producer: lane i loads page i of a block
    const int br = min(p.g.page(), EX_BK);       // rows of a box
    int kv = 0, items = 0;
    bool ok = true;
    auto load_block = [&](const CUtensorMap* m, int kb, bool is_v) {
      const int slot = kv % EX_SLOTS;
      if (!mbar_wait_warp(kv_empty0 + 8 * slot, ((kv / EX_SLOTS) & 1) ^ 1, p.err)) return false;
      const uint32_t dst = smem_u32(smem + S::KV_OFF + slot * 2 * S::SUB);
      const int valid = max(0, min(EX_BK, w.q.len - kb * EX_BK));
      const int nbox = (valid + br - 1) / br;
      // rows behind the last token: the block lands for the V-tail warp first
      const uint32_t bar = (is_v && valid < EX_BK ? land0 : kv_full0) + 8 * slot;
      if (lane == 0) mbar_arrive_tx(bar, nbox * br * 256);
      __syncwarp();
      if (lane < nbox) {
        const int pos = kb * EX_BK + lane * br;
        const int e = max(0, good_page(p.g, p.table[(long long)w.s * p.g.ld_table + (pos >> p.g.shift)], p.err));
        const int row = ((e * p.g.G + w.g) << p.g.shift) + (pos & (p.g.page() - 1));
        tma_load_2d(dst + lane * br * 128, m, bar, 0, row);
        tma_load_2d(dst + S::SUB + lane * br * 128, m, bar, 64, row);
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
      for (int i = max(0, kv - EX_SLOTS); i < kv; ++i) {
        drain_wait(kv_full0 + 8 * (i % EX_SLOTS), (i / EX_SLOTS) & 1);
        drain_wait(land0 + 8 * (i % EX_SLOTS), 0);
      }
      drain_wait(q_full, items & 1);
    }
  } else if (warp == 3) {
    // ---- V tails: zero the rows behind a sequence's last token before the products read them
    int kv = 0;
    uint32_t par = 0;                            // bit i: parity of the next landing in slot i
    bool ok = true;
    for (bool more = w.open(p); more && ok; more = w.next(p)) {
      const int nbk = w.kb1 - w.kb0, slot = (kv + 2 * nbk - 1) % EX_SLOTS;
      const int valid = max(0, w.q.len - (w.kb1 - 1) * EX_BK);   // of the last block; the others are whole
      kv += 2 * nbk;
      if (valid >= EX_BK) continue;
      ok = mbar_wait_warp(land0 + 8 * slot, (par >> slot) & 1, p.err);
      if (!ok) break;
      par ^= 1u << slot;
      uint8_t* base = smem + S::KV_OFF + slot * 2 * S::SUB;
      for (int i = lane; i < (EX_BK - valid) * 16; i += 32) {
        const int row = valid + (i >> 4), c = i & 15;
        *reinterpret_cast<uint4*>(base + (c >> 3) * S::SUB + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(kv_full0 + 8 * slot);
    }
  } else {
    // ---- MMA warp of tile t: the whole warp walks in step, one elected lane issues.  A product is
    // accepted only as the last one runs (64 cycles each), so whatever a warp does between its
    // products would leave the tensor core idle; with a warp per tile the other one's products run then.
    const int t = warp - 1;
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0) + 256 * t;
    const uint64_t qd = sw128_desc(smem_u32(smem + S::Q_OFF) + t * (2 * S::SUB));
    int kv = 0, items = 0, np = 0;
    bool ok = true;
    if (t == 0 && lane == 0) mbar_arrive(P_FULL(0));   // tile A has the first turn
    auto kv_base = [&](int i) { return smem_u32(smem + S::KV_OFF) + (uint32_t)(i % EX_SLOTS) * (2 * S::SUB); };
    auto wait_kv = [&](int i) { return mbar_wait_warp(kv_full0 + 8 * (i % EX_SLOTS), (i / EX_SLOTS) & 1, p.err); };
    // S = Q K^T of fill i, and what else is done once the products issued so far are
    auto issue_s = [&](int i, uint64_t kd, bool last) {
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {         // 16 head dims a step
          const uint64_t off = (kk >> 2) * (S::SUB >> 4) + 2 * (kk & 3);
          umma_bf16(tb, qd + off, kd + off, EX_IDESC_S, kk > 0 ? 1u : 0u);
        }
        umma_commit(S_FULL(t));
        umma_commit(kv_empty0 + 8 * (i % EX_SLOTS));
        if (last) umma_commit(q_empty);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int i, uint64_t vd, bool first, bool last) {
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)           // 16 keys a step: 2048 bytes of V, 8 columns of P
          umma_bf16_ta(tb + 128, tb + 8 * kk, vd + 128 * kk, EX_IDESC_PV, (!first || kk > 0) ? 1u : 0u);
        umma_commit(kv_empty0 + 8 * (i % EX_SLOTS));
        if (last) umma_commit(O_FULL(t));
      }
      __syncwarp();
    };
    for (bool more = w.open(p); __any_sync(0xffffffffu, more) && ok; more = w.next(p), ++items) {
      const bool both = __any_sync(0xffffffffu, w.tokens_of(p, 1) > 0), has = both || t == 0;
      const int nbk = __shfl_sync(0xffffffffu, w.kb1 - w.kb0, 0);
      ok = mbar_wait_warp(q_full, items & 1, p.err);
      if (!ok) break;
      if (!has) {                                // no tile B: its share of the releases
        if (lane == 0) mbar_arrive(q_empty);
        for (int j = 0; j < 2 * nbk && ok; ++j) {
          ok = wait_kv(kv + j);                  // this fill's, not an earlier one's
          if (ok && lane == 0) mbar_arrive(kv_empty0 + 8 * ((kv + j) % EX_SLOTS));
        }
      } else {
        ok = wait_kv(kv);
        if (!ok) break;
        tc_fence_after();
        issue_s(kv, sw128_desc(kv_base(kv)), nbk == 1);
        for (int j = 0; j < nbk; ++j) {
          const int vi = kv + 2 * j + 1;
          const bool last = j + 1 == nbk;
          const uint64_t vd = v_desc(kv_base(vi)), kd = sw128_desc(kv_base(vi + 1));
          ok = wait_kv(vi) && (last || wait_kv(vi + 1)) && mbar_wait_warp(P_FULL(t), np & 1, p.err);
          if (!ok) break;
          ++np;
          tc_fence_after();
          issue_pv(vi, vd, j == 0, last);
          if (!last) issue_s(vi + 1, kd, j + 2 == nbk);
          // the tiles take turns, PV and the next S together: mixed, both would end late and both softmaxes run at
          // once.  After an item the turn is tile A's again; where there is no tile B it stays there.
          if (lane == 0) mbar_arrive(P_FULL(both ? t ^ 1 : 0));
        }
      }
      kv += 2 * nbk;
    }
    if (elect_one()) umma_commit(DRAINED(t));
    __syncwarp();
    drain_wait(DRAINED(t), 0);
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ---- softmax of tile t: 16 rows a warp, two rows a quad of lanes
    const int t = (warp - 4) >> 3, quad = lane & 3;
    const int row0 = (warp & 3) * 32 + ((warp >> 2) & 1) * 16;   // of the warp; warps reach the lanes of their quarter
    const uint32_t tS = tbase + 256 * t + ((uint32_t)row0 << 16), tO = tS + 128;
    const int r[2] = {row0 + (lane >> 2), row0 + (lane >> 2) + 8};
    const int tok_r[2] = {r[0] / p.rep, r[1] / p.rep};
    int ns = 0, no = 0;
    bool ok = true, first_item = true;
    const bool scribe = t == 0 && row0 == 0 && lane == 0;
    if (scribe) p.meta[blockIdx.x].tail = 0;
    for (bool more = w.open(p); more && ok; more = w.next(p), first_item = false) {
      const int nt = w.tokens_of(p, t);
      const bool whole = w.kb0 == 0 && w.kb1 == w.nb;
      if (scribe) {
        ExMeta* m = p.meta + blockIdx.x;
        if (first_item) m->ends = w.kb1 == w.nb;
        m->tail = w.kb0 == 0 && w.kb1 < w.nb;    // only the last item can be one
        m->s = w.s;
        m->g = w.g;
        m->u = w.u;
      }
      if (nt == 0) continue;                     // the unit has no tile B
      const int tok0 = (2 * w.u + t) * p.tpt;    // of the sequence's new tokens
      const bool row_in[2] = {tok_r[0] < nt, tok_r[1] < nt};
      // rows without a token hold anything and are never written: let them see everything, masks cost time
      const int pos[2] = {row_in[0] ? w.q.len - w.q.n + tok0 + tok_r[0] : INT_MAX,
                          row_in[1] ? w.q.len - w.q.n + tok0 + tok_r[1] : INT_MAX};
      // pend: factor that O still has to be scaled by
      float m[2] = {0.f, 0.f}, l[2] = {0.f, 0.f}, pend[2] = {1.f, 1.f};
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++ns) {
        const int lim[2] = {pos[0] - kb * EX_BK, pos[1] - kb * EX_BK};   // keys c <= lim are seen
        const bool masked = !__all_sync(0xffffffffu, lim[0] >= EX_BK - 1 && lim[1] >= EX_BK - 1);
        ok = mbar_wait_warp(S_FULL(t), ns & 1, p.err);
        if (!ok) break;
        tc_fence_after();
        // The terms are formed against the reference from the blocks before; P replaces S only afterwards.  A
        // reference that is off by up to 2^32 does no harm (see EX_FAR); the rows' sums tell how far it is: beyond EX_MAX_SUM it is raised for the next block, beyond EX_FAR the warp forms the
        // block again.  A unit's first block takes 0, where no key is masked, and its maximum beforehand where
        // some are (it may be that of none: -inf).
        uint32_t pk[32];
        float sum[2];
        const bool first = kb == w.kb0;
        if (first && masked) {
          float mx[2];
          ex_row_max(tS, masked, lim, quad, mx);
          m[0] = mx[0] * p.sl2;
          m[1] = mx[1] * p.sl2;
        }
        ex_terms(tS, masked, lim, quad, m, p.sl2, pk, sum);
        const float low = first && !masked ? EX_MIN_SUM : 0.f;
        auto odd = [&](int e) {
          return row_in[e] && (!(sum[e] <= EX_MAX_SUM) || sum[e] < low || m[e] == -INFINITY || pend[e] != 1.f);
        };
        // what is rare takes one vote, by the thread's own columns: a row's sum is at most four times as much
        const bool rare = __any_sync(0xffffffffu, odd(0) || odd(1));
        if (rare) {
          float mx[2], all[2] = {quad_sum(sum[0]), quad_sum(sum[1])};
          auto far = [&](int e) {
            return row_in[e] && lim[e] >= 0 &&
                   (!(all[e] < EX_FAR) || (((first && !masked) || m[e] == -INFINITY) && all[e] < EX_MIN_SUM));
          };
          const bool again[2] = {far(0), far(1)};
          if (__any_sync(0xffffffffu, again[0] || again[1])) {
            ex_row_max(tS, masked, lim, quad, mx);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (!again[e]) continue;
              mx[e] *= p.sl2;
              const float corr = first || m[e] == -INFINITY ? 1.f : ex2(m[e] - mx[e]);   // nothing before it otherwise
              l[e] *= corr;
              pend[e] *= corr;
              m[e] = mx[e];
            }
            __syncwarp();                        // the loads are the whole warp's
            ex_terms(tS, masked, lim, quad, m, p.sl2, pk, sum);
            // ex2_fma takes -inf for a small term: where every score is -inf there is nothing
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (again[e] && m[e] == -INFINITY && sum[e] < 1.f) sum[e] = 0.f;
          }
          // the product that wrote O last is done: S_j was issued after it
          if (!first && __any_sync(0xffffffffu, pend[0] != 1.f || pend[1] != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              float o[16];
              tmem_ld_16x256b(tO + 32 * c, o);
              tmem_wait_ld16(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= pend[(k >> 1) & 1];
              tmem_st_16x256b(tO + 32 * c, o);
            }
          }
        }
        tmem_st_16x128b(tS, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(P_FULL(t));
#pragma unroll
        for (int e = 0; e < 2; ++e)
          l[e] += sum[e] < 0x1p100f ? sum[e] : NAN;   // a NaN that went through ex2_fma is one again
        if (rare) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float all = quad_sum(sum[e]);
            pend[e] = 1.f;
            if (m[e] == -INFINITY && all > 0.f) m[e] = 0.f;   // the terms were formed against 0
            if (all > EX_MAX_SUM && all < 0x1p100f) {         // by a power of two: exact
              const int up = (__float_as_int(all) >> 23) - 127;
              pend[e] = __int_as_float((127 - up) << 23);
              l[e] *= pend[e];
              m[e] += (float)up;
            }
          }
        }
      }
      if (!ok) break;
      l[0] = quad_sum(l[0]);
      l[1] = quad_sum(l[1]);
      ok = mbar_wait_warp(O_FULL(t), no & 1, p.err);
      ++no;
      if (!ok) break;
      tc_fence_after();
      // a CTA's parts: 0 continues a unit, 1 begins one
      const long long part = ((long long)(2 * blockIdx.x + (w.kb0 == 0)) * 2 + t) * 128;
      float f[2];
      bf16* dst[2];
      float* pdst[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const long long row = w.q.q0 + tok0 + tok_r[e];
        const int head = w.g * p.rep + r[e] - tok_r[e] * p.rep;
        f[e] = whole ? (l[e] != 0.f ? pend[e] / l[e] : 0.f) : pend[e];
        dst[e] = p.o + row * p.ld_o + (long long)head * PG_D;
        pdst[e] = p.part_o + (part + r[e]) * PG_D;
        if (row_in[e] && quad == 0) {
          if (!whole)
            *reinterpret_cast<float2*>(p.part_ml + (part + r[e]) * 2) = make_float2(m[e], l[e]);
          else if (p.lse)
            p.lse[row * p.H + head] = l[e] != 0.f ? (m[e] + log2f(l[e])) * 0.6931471805599453f : -INFINITY;
        }
      }
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float o[16];
        tmem_ld_16x256b(tO + 32 * c, o);
        tmem_wait_ld16(o);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (whole) {                           // eight columns a lane after the transpose
            uint32_t x[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              __nv_bfloat162 hh = __floats2bfloat162_rn(o[4 * g + 2 * e] * f[e], o[4 * g + 2 * e + 1] * f[e]);
              x[g] = *reinterpret_cast<uint32_t*>(&hh);
            }
            quad_transpose(x, quad);
            if (row_in[e]) *reinterpret_cast<uint4*>(dst[e] + 32 * c + 8 * quad) = make_uint4(x[0], x[1], x[2], x[3]);
          } else if (row_in[e]) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
              *reinterpret_cast<float2*>(pdst[e] + 32 * c + 8 * g + 2 * quad) =
                  make_float2(o[4 * g + 2 * e] * f[e], o[4 * g + 2 * e + 1] * f[e]);
          }
        }
      }
      tc_fence_before();   // O is read before the next item's first product is issued (after its P)
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
#undef DRAINED

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
  // CTA c + i continues the unit, the last one ends it
  while (c + parts < (int)gridDim.x && !p.meta[c + parts - 1].ends) ++parts;
  ExSeq q;
  q.load(p, me.s);
  // four rows at once, so that their loads are in flight together
  const int rr = blockIdx.y * 32 + warp * 4, t = rr >> 7;
  int tok[4];
  bool in[4], any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tok_r = ((rr & 127) + i) / p.rep;
    tok[i] = (2 * me.u + t) * p.tpt + tok_r;
    in[i] = tok_r < p.tpt && tok[i] < q.n;
    any = any || in[i];
  }
  if (!any) return;
  float m[4], l[4];
  float4 o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll 2
  for (int k = 0; k < parts; ++k) {
    const long long row0 = (long long)(k == 0 ? 2 * c + 1 : 2 * (c + k)) * 256 + rr;
    float2 ml[4];
    float4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!in[i]) continue;
      ml[i] = *reinterpret_cast<const float2*>(p.part_ml + (row0 + i) * 2);
      x[i] = *reinterpret_cast<const float4*>(p.part_o + (row0 + i) * PG_D + lane * 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!in[i] || ml[i].y == 0.f) continue;   // a part whose keys the row does not see
      const float mn = fmaxf(m[i], ml[i].x), fa = ex2(m[i] - mn), fb = ex2(ml[i].x - mn);
      m[i] = mn;
      l[i] = l[i] * fa + ml[i].y * fb;
      o[i].x = o[i].x * fa + x[i].x * fb;
      o[i].y = o[i].y * fa + x[i].y * fb;
      o[i].z = o[i].z * fa + x[i].z * fb;
      o[i].w = o[i].w * fa + x[i].w * fb;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!in[i]) continue;
    const float inv = l[i] != 0.f ? 1.f / l[i] : 0.f;
    const long long row = q.q0 + tok[i];
    const int head = me.g * p.rep + ((rr & 127) + i) % p.rep;
    const __nv_bfloat162 h01 = __floats2bfloat162_rn(o[i].x * inv, o[i].y * inv);
    const __nv_bfloat162 h23 = __floats2bfloat162_rn(o[i].z * inv, o[i].w * inv);
    uint2 u;
    u.x = *reinterpret_cast<const uint32_t*>(&h01);
    u.y = *reinterpret_cast<const uint32_t*>(&h23);
    *reinterpret_cast<uint2*>(p.o + row * p.ld_o + (long long)head * PG_D + lane * 4) = u;
    if (p.lse && lane == 0)
      p.lse[row * p.H + head] = l[i] != 0.f ? (m[i] + log2f(l[i])) * 0.6931471805599453f : -INFINITY;
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
  if (dev >= 64 || !configured[dev]) {
    JB_CUDA(cudaFuncSetAttribute(paged_extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ExSmem::BYTES));
    if (dev < 64) configured[dev] = true;
  }
  JB_CUDA(launch_pdl(paged_extend_kernel, dim3(grid), dim3(EX_THREADS), ExSmem::BYTES, s, mq, mk, mv, p));
  JB_CUDA(launch_pdl(paged_extend_join_kernel, dim3(grid, 8), dim3(256), 0, s, p));
  return JAMBA_OK;
}

}  // namespace jb
