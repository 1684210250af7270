// Upkeep of the paged key-value cache: forking and freeing sequences, taking
// pages for new tokens (with copies of shared last pages), compaction, and
// writing new keys and values into their pages.
//
// Everything the calls decide is decided on the device from refs, table and
// lengths, in an order that does not depend on timing: holders are counted with
// integer atomics (whose order changes nothing), and free pages are handed out by
// rank, from prefix sums.  fork is two launches (read the old rows, write the new
// ones); grow and compact are a plan made by one CTA and a grid that carries it
// out.  The plans are bound by the latency of a few dependent reads, the copies
// by HBM.  Rows move as they are: nothing is rounded.
//
// Measured, on the GPU alone: fork and grow of 8 slots of up to 900 tokens, one layer, 8 us
// (24 us with the host's part, which bounds it); of 256 slots of up to 1500 tokens, four layers,
// a quarter of them copying a shared last page, 21 us; compaction that moves 0.51 GB 166 us, 0.94 of the
// copy rate with its plan, in a pool of 160 pages 8 us; append of 33 prompts of 17 to 4001 tokens
// 36 us, 0.89 of the copy rate, of one token for each of 64 sequences 4 us.
#include <climits>

#include "host.hpp"
#include "pages.cuh"

namespace jb {

constexpr int PLAN_THREADS = 1024;

// Exclusive prefix sum over the CTA's PLAN_THREADS threads; `total` gets the sum.
template <typename T>
__device__ __forceinline__ T block_exclusive(T v, T* warp_sums, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();               // the last call's sums have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[PLAN_THREADS / 32 - 1];
  return x - v + (warp ? warp_sums[warp - 1] : 0);
}

// ------------------------------------------------------------------- fork

// CTA per slot: of a slot that changes, the parent's row and length into the
// workspace; the pages of its old row lose a holder, those of its new row gain one.
__global__ void __launch_bounds__(256)
pages_fork_read_kernel(PageGeom g, const int* __restrict__ parent, int* refs, const int* __restrict__ table,
                       const int* __restrict__ lengths, int* __restrict__ rows, int* __restrict__ lens, int* err) {
  griddep_wait();
  const int s = blockIdx.x, p = parent[s];
  if (p != s && checked(p >= -1 && p < g.S, err) && p >= -1 && p < g.S) {
    const int n_old = held_pages(g, clamp_len(g, lengths[s], err));
    for (int j = threadIdx.x; j < n_old; j += 256) {
      const int e = good_page(g, table[(long long)s * g.ld_table + j], err);
      if (e >= 0) atomicSub(refs + e, 1);
    }
    int len = 0;
    if (p >= 0) {
      len = clamp_len(g, lengths[p], err);
      const int n = held_pages(g, len);
      for (int j = threadIdx.x; j < n; j += 256) {
        const int e = good_page(g, table[(long long)p * g.ld_table + j], err);
        rows[(long long)s * g.max_pages + j] = e;
        if (e >= 0) atomicAdd(refs + e, 1);
      }
    }
    if (threadIdx.x == 0) lens[s] = len;
  }
  griddep_launch();
}

// CTA per slot: the new row and length of a slot that changes.
__global__ void __launch_bounds__(256)
pages_fork_write_kernel(PageGeom g, const int* __restrict__ parent, int* __restrict__ table, int* __restrict__ lengths,
                        const int* __restrict__ rows, const int* __restrict__ lens) {
  griddep_wait();
  const int s = blockIdx.x, p = parent[s];
  if (p != s && p >= -1 && p < g.S) {
    const int n_old = held_pages(g, clamp_len(g, lengths[s], nullptr)), n = held_pages(g, lens[s]);
    for (int j = threadIdx.x; j < max(n, n_old); j += 256)
      table[(long long)s * g.ld_table + j] = j < n ? rows[(long long)s * g.max_pages + j] : -1;
    __syncthreads();             // every thread has read the old length
    if (threadIdx.x == 0) lengths[s] = lens[s];
  }
  griddep_launch();
}

// The two launches as one CTA, for tables of up to FORK_SMALL entries and as many slots: a thread per entry keeps
// what it read of the old rows, and all have read before any writes.  One launch instead of two saves the host 2 us of
// 11.5; on the GPU both take 3 us at 8 slots of 17 pages, and at 256 slots of 26 pages one CTA would take 7.1 us
// against 3.9 us.
constexpr int FORK_SMALL = PLAN_THREADS;
__global__ void __launch_bounds__(PLAN_THREADS)
pages_fork_small_kernel(PageGeom g, const int* __restrict__ parent, int* refs, int* table, int* lengths, int* err) {
  griddep_wait();
  griddep_launch();
  const int i = threadIdx.x, s = i / g.max_pages, j = i - s * g.max_pages;
  int entry = -2, len = -2;      // -2: nothing to write
  if (i < g.S) {
    const int p = parent[i];
    if (p != i && checked(p >= -1 && p < g.S, err) && p >= -1 && p < g.S)
      len = p >= 0 ? clamp_len(g, lengths[p], err) : 0;
  }
  if (s < g.S) {
    const int p = parent[s];
    if (p != s && p >= -1 && p < g.S) {
      if (j < held_pages(g, clamp_len(g, lengths[s], err))) {
        const int e = good_page(g, table[(long long)s * g.ld_table + j], err);
        if (e >= 0) atomicSub(refs + e, 1);
        entry = -1;
      }
      if (p >= 0 && j < held_pages(g, clamp_len(g, lengths[p], err))) {
        entry = good_page(g, table[(long long)p * g.ld_table + j], err);
        if (entry >= 0) atomicAdd(refs + entry, 1);
      }
    }
  }
  __syncthreads();
  if (len >= 0) lengths[i] = len;
  if (entry >= -1) table[(long long)s * g.ld_table + j] = entry;
}

// ------------------------------------------------------------------- grow

struct GrowRecord {
  int len, add;      // tokens before, tokens to add
  int first, end;    // ranks of the free pages wanted: first .. end - 1 (INT_MAX: further than any pool)
  int src;           // page to copy the rows of (-1: none); its copy takes rank `first`
  int fits;          // 0: would pass max_pages
};

// One CTA.  ws: counts[0] = free pages found (all of them, or as many as are
// wanted), counts[1] = slots that copy a page.
__global__ void __launch_bounds__(PLAN_THREADS)
pages_grow_plan_kernel(PageGeom g, const int* __restrict__ add, const int* __restrict__ refs,
                       const int* __restrict__ table, const int* __restrict__ lengths, GrowRecord* __restrict__ rec,
                       int* __restrict__ free_list, int* __restrict__ copiers, int* __restrict__ counts, int* err) {
  __shared__ int sums[32];
  __shared__ long long wide_sums[32];
  griddep_wait();
  griddep_launch();
  long long wanted = 0, wide_total;              // refused slots' pages count too: more than 2^31 in a large table
  int copying = 0, total;
  for (int s0 = 0; s0 < g.S; s0 += PLAN_THREADS) {
    const int s = s0 + threadIdx.x;
    GrowRecord r = {};
    r.src = -1;
    int want = 0;
    if (s < g.S) {
      r.len = clamp_len(g, lengths[s], err);
      r.add = max(0, add[s]);
      const long long to = (long long)r.len + r.add;
      r.fits = to <= ((long long)g.max_pages << g.shift);
      if (r.fits && r.add > 0) {
        want = held_pages(g, (int)to) - held_pages(g, r.len);
        if (r.len & (g.page() - 1)) {
          const int e = good_page(g, table[(long long)s * g.ld_table + (r.len >> g.shift)], err);
          if (e >= 0 && refs[e] > 1) {
            r.src = e;
            ++want;
          }
        }
      }
    }
    const long long at = wanted + block_exclusive((long long)want, wide_sums, wide_total);
    r.first = (int)min(at, (long long)INT_MAX);
    r.end = (int)min(at + want, (long long)INT_MAX);
    wanted += wide_total;
    const int c = block_exclusive((int)(r.src >= 0), sums, total);
    if (r.src >= 0) copiers[copying + c] = s;
    copying += total;
    if (s < g.S) rec[s] = r;
  }
  int found = 0;
  for (int p0 = 0; p0 < g.num_pages && found < wanted; p0 += 4 * PLAN_THREADS) {
    const int p = p0 + 4 * threadIdx.x;
    int4 v = make_int4(1, 1, 1, 1);
    if (p + 3 < g.num_pages) {
      v = *reinterpret_cast<const int4*>(refs + p);
    } else {
      if (p < g.num_pages) v.x = refs[p];
      if (p + 1 < g.num_pages) v.y = refs[p + 1];
      if (p + 2 < g.num_pages) v.z = refs[p + 2];
    }
    const int f0 = v.x == 0, f1 = v.y == 0, f2 = v.z == 0, f3 = v.w == 0;
    int at = found + block_exclusive(f0 + f1 + f2 + f3, sums, total);
    if (f0) free_list[at++] = p;
    if (f1) free_list[at++] = p + 1;
    if (f2) free_list[at++] = p + 2;
    if (f3) free_list[at] = p + 3;
    found += total;
  }
  if (threadIdx.x == 0) {
    counts[0] = found;
    counts[1] = copying;
  }
}

// Copies n 16-byte units within the pool; 256 threads, eight loads in flight each.
__device__ __forceinline__ void copy_units(uint4* __restrict__ dst, const uint4* __restrict__ src, int n) {
  int i = threadIdx.x;
  for (; i + 7 * 256 < n; i += 8 * 256) {
    uint4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = src[i + k * 256];
#pragma unroll
    for (int k = 0; k < 8; ++k) dst[i + k * 256] = v[k];
  }
  for (; i < n; i += 256) dst[i] = src[i];
}

// Items: first one per slot (its table entries, counts, length), then one per
// copied (slot, plane, head): the rows in use of the shared page.
__global__ void __launch_bounds__(256)
pages_grow_apply_kernel(PageGeom g, bf16* __restrict__ data, int* refs, int* __restrict__ table,
                        int* __restrict__ lengths, int* __restrict__ granted, const GrowRecord* __restrict__ rec,
                        const int* __restrict__ free_list, const int* __restrict__ copiers,
                        const int* __restrict__ counts) {
  griddep_wait();
  griddep_launch();
  const int found = counts[0];
  const int pieces = g.planes * g.G;
  const long long items = g.S + (long long)counts[1] * pieces;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    if (it < g.S) {
      const int s = (int)it;
      const GrowRecord r = rec[s];
      const bool ok = r.fits && (r.end == r.first || r.end <= found);
      if (ok && r.add > 0) {
        int j = held_pages(g, r.len);
        if (r.src >= 0) {
          --j;
          if (threadIdx.x == 0) atomicSub(refs + r.src, 1);
        }
        for (int i = threadIdx.x; i < r.end - r.first; i += 256) {
          const int e = free_list[r.first + i];
          table[(long long)s * g.ld_table + j + i] = e;
          refs[e] = 1;
        }
        if (threadIdx.x == 0) lengths[s] = r.len + r.add;
      }
      if (threadIdx.x == 0) granted[s] = ok;
    } else {
      const int c = (int)((it - g.S) / pieces), piece = (int)((it - g.S) % pieces);
      const GrowRecord r = rec[copiers[c]];
      if (r.end > found) continue;   // refused
      const int plane = piece / g.G, head = piece % g.G;
      const long long base = plane * g.plane_elems() + (long long)head * (PG_D << g.shift);
      const bf16* src = data + base + r.src * g.page_elems();
      bf16* dst = data + base + free_list[r.first] * g.page_elems();
      copy_units(reinterpret_cast<uint4*>(dst), reinterpret_cast<const uint4*>(src),
                 (r.len & (g.page() - 1)) * (PG_D / 8));
    }
  }
}

// out[s] = lengths[s] of the slots that take part, 0 of the others; a thread per slot, bound by the launch.
__global__ void __launch_bounds__(256)
pages_active_kernel(int S, const int* active, const int* lengths, int* out) {
  griddep_wait();
  griddep_launch();
  const int s = blockIdx.x * 256 + threadIdx.x;
  if (s < S) out[s] = active[s] > 0 ? lengths[s] : 0;
}

// ---------------------------------------------------------------- compact

// One CTA: remap, and the pairs (mover -> hole).  counts[0] = pages that move.
__global__ void __launch_bounds__(PLAN_THREADS)
pages_compact_plan_kernel(PageGeom g, const int* __restrict__ refs, int* __restrict__ remap, int* __restrict__ holes,
                          int* __restrict__ movers, int* __restrict__ counts) {
  __shared__ int sums[32];
  griddep_wait();
  griddep_launch();
  int total, live = 0;
  for (int p = threadIdx.x; p < g.num_pages; p += PLAN_THREADS) live += refs[p] > 0;
  block_exclusive(live, sums, total);
  const int n = total;
  int nh = 0, nm = 0;
  for (int p0 = 0; p0 < g.num_pages; p0 += PLAN_THREADS) {
    const int p = p0 + threadIdx.x;
    const bool in = p < g.num_pages, used = in && refs[p] > 0;
    const bool hole = in && !used && p < n, mover = used && p >= n;
    // holes and movers of one stretch in one sum: holes in the low half (a stretch has at most 1024 of either)
    const int at = block_exclusive((hole ? 1 : 0) + (mover ? 1 << 16 : 0), sums, total);
    if (hole) holes[nh + (at & 0xffff)] = p;
    if (mover) movers[nm + (at >> 16)] = p;
    if (in && !mover) remap[p] = used ? p : -1;
    nh += total & 0xffff;
    nm += total >> 16;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nm; i += PLAN_THREADS) remap[movers[i]] = holes[i];   // as many holes as movers
  if (threadIdx.x == 0) counts[0] = nm;
}

constexpr int MOVE_BYTES = 32768;   // of a page in one plane, per CTA and step

// Items: first one per slot (its table entries), then (page, plane, part).
__global__ void __launch_bounds__(256)
pages_compact_apply_kernel(PageGeom g, bf16* __restrict__ data, int* __restrict__ refs, int* __restrict__ table,
                           const int* __restrict__ lengths, const int* __restrict__ remap,
                           const int* __restrict__ holes, const int* __restrict__ movers,
                           const int* __restrict__ counts, int* err) {
  griddep_wait();
  griddep_launch();
  const int page_units = (int)(g.page_elems() / 8);               // 16-byte units
  const int parts = (page_units * 16 + MOVE_BYTES - 1) / MOVE_BYTES;
  const int per = MOVE_BYTES / 16;
  const long long items = g.S + (long long)counts[0] * g.planes * parts;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    if (it < g.S) {
      const int s = (int)it, n = held_pages(g, clamp_len(g, lengths[s], err));
      for (int j = threadIdx.x; j < n; j += 256) {
        int* e = table + (long long)s * g.ld_table + j;
        const int p = good_page(g, *e, err);
        if (p >= 0) *e = remap[p];
      }
    } else {
      const long long k = it - g.S;
      const int part = (int)(k % parts), plane = (int)(k / parts % g.planes), m = (int)(k / parts / g.planes);
      const int from = movers[m], to = holes[m];
      uint4* base = reinterpret_cast<uint4*>(data + plane * g.plane_elems());
      const int u0 = part * per;
      copy_units(base + (long long)to * page_units + u0, base + (long long)from * page_units + u0,
                 min(per, page_units - u0));
      if (part == 0 && plane == 0 && threadIdx.x == 0) {
        refs[to] = refs[from];
        refs[from] = 0;
      }
    }
  }
}

// ----------------------------------------------------------------- append

// Bound by HBM (a prompt's rows) or the launch (one token each): each row is read and written once.
// A CTA writes 1024 16-byte pieces (four per thread, loads before stores):
// 1024 / (32 G) tokens, or one token in steps when it has more pieces.
__global__ void __launch_bounds__(256)
paged_append_kernel(PageGeom g, const bf16* __restrict__ k, const bf16* __restrict__ v, long long ld, int tokens,
                    const int* __restrict__ q_start, bf16* __restrict__ kp, bf16* __restrict__ vp,
                    const int* __restrict__ table, const int* __restrict__ lengths, int per_cta, int* err) {
  __shared__ long long where[32];   // element offset of a token's row of head 0 in the planes; -1: not written
  griddep_wait();
  griddep_launch();
  const int t0 = blockIdx.x * per_cta, nt = min(per_cta, tokens - t0);
  if ((int)threadIdx.x < nt) {
    const int t = t0 + threadIdx.x;
    const int s = q_start ? token_seq(q_start, g.S, t) : t;
    long long off = -1;
    if (s >= 0) {
      const int len = clamp_len(g, lengths[s], err);
      const int pos = q_start ? len - q_start[s + 1] + t : len - 1;
      if (pos >= 0 && pos < len) {
        const int e = good_page(g, table[(long long)s * g.ld_table + (pos >> g.shift)], err);
        if (e >= 0) off = e * g.page_elems() + (long long)(pos & (g.page() - 1)) * PG_D;
      }
    }
    where[threadIdx.x] = off;
  }
  __syncthreads();
  const int pieces = 32 * g.G, n = nt * pieces;   // per token: K heads, then V heads, 16 pieces each
  for (int i0 = threadIdx.x; i0 < n; i0 += 1024) {
    uint4 x[4];
    bf16* dst[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + 256 * u;
      dst[u] = nullptr;
      if (i < n) {
        const int t = i / pieces, c = i % pieces, kv = c >= 16 * g.G, hd = (c >> 4) - kv * g.G, col = (c & 15) * 8;
        if (where[t] >= 0) {
          x[u] = *reinterpret_cast<const uint4*>((kv ? v : k) + (t0 + t) * ld + hd * PG_D + col);
          dst[u] = (kv ? vp : kp) + where[t] + (long long)hd * (PG_D << g.shift) + col;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (dst[u]) *reinterpret_cast<uint4*>(dst[u]) = x[u];
  }
}

// ------------------------------------------------------------------- host

struct PagesWs {
  int *rows, *lens;                              // fork
  GrowRecord* rec; int *free_list, *copiers;     // grow
  int *holes, *movers;                           // compact
  int* counts;
  size_t total;
};

static PagesWs carve_pages(const PageGeom& g, void* ws) {
  // the three calls use the same bytes, each laid out its own way
  uint8_t* b = reinterpret_cast<uint8_t*>(ws);
  auto al = [](size_t v) { return (v + 255) & ~size_t(255); };
  PagesWs w = {};
  const size_t ints = al((size_t)g.num_pages * 4), slots = al((size_t)g.S * 4);
  const size_t counts = 256;
  w.counts = reinterpret_cast<int*>(b);
  size_t fork = counts, grow = counts, comp = counts;
  w.rows = reinterpret_cast<int*>(b + fork); fork += al((size_t)g.S * g.max_pages * 4);
  w.lens = reinterpret_cast<int*>(b + fork); fork += slots;
  w.rec = reinterpret_cast<GrowRecord*>(b + grow); grow += al((size_t)g.S * sizeof(GrowRecord));
  w.free_list = reinterpret_cast<int*>(b + grow); grow += ints;
  w.copiers = reinterpret_cast<int*>(b + grow); grow += slots;
  w.holes = reinterpret_cast<int*>(b + comp); comp += ints;
  w.movers = reinterpret_cast<int*>(b + comp); comp += ints;
  w.total = fork > grow ? fork : grow;
  if (comp > w.total) w.total = comp;
  return w;
}

size_t pages_workspace_bytes(const PageGeom& g) { return carve_pages(g, nullptr).total; }

jamba_status pages_fork(const PageGeom& g, const int* parent, int* refs, int* table, int* lengths, void* ws,
                        cudaStream_t s) {
  const PagesWs w = carve_pages(g, ws);
  if ((long long)g.S * g.max_pages <= FORK_SMALL) {   // and S <= FORK_SMALL
    JB_CUDA(launch_pdl(pages_fork_small_kernel, dim3(1), dim3(PLAN_THREADS), 0, s, g, parent, refs, table, lengths,
                       device_error_word()));
    return JAMBA_OK;
  }
  JB_CUDA(launch_pdl(pages_fork_read_kernel, dim3(g.S), dim3(256), 0, s, g, parent, refs, (const int*)table,
                     (const int*)lengths, w.rows, w.lens, device_error_word()));
  JB_CUDA(launch_pdl(pages_fork_write_kernel, dim3(g.S), dim3(256), 0, s, g, parent, table, lengths,
                     (const int*)w.rows, (const int*)w.lens));
  return JAMBA_OK;
}

jamba_status pages_grow(const PageGeom& g, const int* add, void* data, int* refs, int* table, int* lengths,
                        int* granted, void* ws, cudaStream_t s) {
  const PagesWs w = carve_pages(g, ws);
  JB_CUDA(launch_pdl(pages_grow_plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, s, g, add, (const int*)refs,
                     (const int*)table, (const int*)lengths, w.rec, w.free_list, w.copiers, w.counts,
                     device_error_word()));
  const long long most = g.S + (long long)g.S * g.planes * g.G;
  const int grid = (int)(most < 8LL * num_sms() ? most : 8LL * num_sms());
  JB_CUDA(launch_pdl(pages_grow_apply_kernel, dim3(grid), dim3(256), 0, s, g, reinterpret_cast<bf16*>(data), refs,
                     table, lengths, granted, (const GrowRecord*)w.rec, (const int*)w.free_list,
                     (const int*)w.copiers, (const int*)w.counts));
  return JAMBA_OK;
}

jamba_status pages_active(int S, const int* active, const int* lengths, int* out, cudaStream_t s) {
  JB_CUDA(launch_pdl(pages_active_kernel, dim3((S + 255) / 256), dim3(256), 0, s, S, active, lengths, out));
  return JAMBA_OK;
}

jamba_status pages_compact(const PageGeom& g, void* data, int* refs, int* table, const int* lengths, int* remap,
                           void* ws, cudaStream_t s) {
  const PagesWs w = carve_pages(g, ws);
  JB_CUDA(launch_pdl(pages_compact_plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, s, g, (const int*)refs, remap,
                     w.holes, w.movers, w.counts));
  // at most half the pages move; a CTA per item up to 64 per SM evens out the ends (1 GB: 166 us, with 8 per SM 182 us;
  // a pool of 160 pages would lose 6 us to CTAs without an item)
  const long long parts = (g.page_elems() * 2 + MOVE_BYTES - 1) / MOVE_BYTES;
  const long long most = g.S + (long long)(g.num_pages / 2) * g.planes * parts;
  const int grid = (int)(most < 64LL * num_sms() ? most : 64LL * num_sms());
  JB_CUDA(launch_pdl(pages_compact_apply_kernel, dim3(grid), dim3(256), 0, s, g,
                     reinterpret_cast<bf16*>(data), refs, table, lengths, (const int*)remap, (const int*)w.holes,
                     (const int*)w.movers, (const int*)w.counts, device_error_word()));
  return JAMBA_OK;
}

jamba_status paged_append(const PageGeom& g, const void* k, const void* v, int ld, int tokens, const int* q_start,
                          void* k_pages, void* v_pages, const int* table, const int* lengths, cudaStream_t s) {
  int per = 1024 / (32 * g.G);
  if (per < 1) per = 1;
  JB_CUDA(launch_pdl(paged_append_kernel, dim3((tokens + per - 1) / per), dim3(256), 0, s, g,
                     reinterpret_cast<const bf16*>(k), reinterpret_cast<const bf16*>(v), (long long)ld, tokens,
                     q_start, reinterpret_cast<bf16*>(k_pages), reinterpret_cast<bf16*>(v_pages), table, lengths, per,
                     device_error_word()));
  return JAMBA_OK;
}

}  // namespace jb
