// The pages of a cache: sequences forked, trimmed, freed and given room (update),
// the pages in use moved to the low end (compact), and pages copied.
//
// The page counts and tables are small (a pool of 64k pages has 256 KB of counts), and what
// happens to them is a chain of steps that each need all of the one before: counts
// given up and gained, then the pages that are free, then who gets which. So one
// cluster of blocks works through them, with a cluster barrier between steps; the
// steps' sums (pages wanted before a sequence, free pages before an index) are block
// scans and one exchange through distributed shared memory. Counts change by integer
// atomics, whose order does not matter. What has to be copied goes onto a list that a
// second kernel, over all SMs, works off: it is launched whatever the list holds,
// because the host does not know it.
//
// The first is bound by the latency of its steps (about a microsecond each): 128 sequences of
// up to 2000 tokens, pages of 16, take 10 to 11 us with the launch of the second, and 16
// prompts forked into 128 sequences, with 128 copies on write (16 MB read and written), 15. Blocks
// with half or twice the work (below) took as long or longer; a pool of 524288 pages
// takes 26. The second is bound by
// memory, 16-byte loads, eight in flight a thread: 495 MB read and written by a
// compaction take 72 us, a copy's rate, of the call's 87.
#include "serve_ptx.cuh"
#include "serve_util.cuh"

namespace moe {
namespace {

constexpr int kThreads = 1024;  // of a planning block
constexpr int kWarps = kThreads / 32;
constexpr int kMaxParts = 16;
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 8;  // 16-byte vectors a thread has in flight

// A page to copy: its first tokens, from page src to page dst.
struct PageCopy {
  int src, dst, tokens, pad;
};
struct PlanHead {
  int n_copies;
  int pad[63];
};
// What the update keeps of a sequence between its steps: in shared memory for the
// first kRowsHeld of a block's, in the workspace for others.
struct RowPlan {
  int kept, need;   // tokens
  int last;         // the page of token kept - 1, if the sequence writes behind it, else -1
  int want;         // pages it wants, times 2, and 1 with a copy on write
  long long before; // pages that the block's earlier sequences want
};
// What lies in the workspace behind the status word's 256 bytes.
struct Scratch {
  PlanHead* head;
  PageCopy* copies;  // at most a page a sequence, or half of the pool
  RowPlan* rows;     // [n_seqs]
  int* free;         // [n_pages] free pages, or those below the number in use
  int* high;         // [n_pages] by rank, pages in use at that number or above
  size_t bytes;
};
template <typename T>
T* carve(char*& at, size_t n) {
  T* p = reinterpret_cast<T*>(at);
  at += align_up(n * sizeof(T), 256);
  return p;
}
Scratch scratch_of(const moe_attn_config& c, void* base) {
  char* at = static_cast<char*>(base);
  const size_t pages = (size_t)c.n_pages, seqs = (size_t)c.n_seqs;
  Scratch s;
  s.head = carve<PlanHead>(at, 1);
  s.copies = carve<PageCopy>(at, seqs > pages / 2 + 1 ? seqs : pages / 2 + 1);
  s.rows = carve<RowPlan>(at, seqs);
  s.free = carve<int>(at, pages);
  s.high = carve<int>(at, pages);
  s.bytes = (size_t)(at - static_cast<char*>(base));
  return s;
}

static_assert(kWarps == 32, "a block's warps are a warp's lanes");
// ---- sums over a block and over the cluster ------------------------------------
struct Shared {
  long long warp[kWarps], also[kWarps];
  long long inbox[2][kMaxParts];
};
// The sum of v over the block's threads before this one; total, also_total: of v and of
// `also` over all of them.
__device__ __forceinline__ long long block_scan(Shared& sh, long long v, long long& total, long long also,
                                                long long& also_total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  long long upto = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long w = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += w;
    also += __shfl_xor_sync(0xffffffffu, also, o);
  }
  if (lane == 31) sh.warp[warp] = upto, sh.also[warp] = also;
  __syncthreads();
  long long s = sh.warp[lane], t = sh.also[lane];  // as many warps as lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long w = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += w;
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  also_total = t;
  const long long before = warp > 0 ? __shfl_sync(0xffffffffu, s, warp - 1) : 0;
  __syncthreads();
  return before + upto - v;
}
// Sends the block's sums a and b to all blocks; they are there after the barrier.
__device__ __forceinline__ void exchange(Shared& sh, int part, int parts, long long a, long long b) {
  if ((int)threadIdx.x < parts) {
    ptx::st_cluster_u64(ptx::mapa_shared(ptx::smem_addr(&sh.inbox[0][part]), threadIdx.x), (uint64_t)a);
    ptx::st_cluster_u64(ptx::mapa_shared(ptx::smem_addr(&sh.inbox[1][part]), threadIdx.x), (uint64_t)b);
  }
  __syncwarp();
  ptx::cluster_sync();
}
__device__ __forceinline__ long long sum_before(const Shared& sh, int which, int part) {
  long long s = 0;
  for (int i = 0; i < part; ++i) s += sh.inbox[which][i];
  return s;
}

// Four counts from page i on (i a multiple of 4); 1 past the end: not free.
__device__ __forceinline__ int4 counts_at(const int32_t* refs, int i, int n) {
  if (i + 4 <= n) return __ldcg(reinterpret_cast<const int4*>(refs + i));
  int4 r = make_int4(1, 1, 1, 1);
  if (i < n) r.x = __ldcg(refs + i);
  if (i + 1 < n) r.y = __ldcg(refs + i + 1);
  if (i + 2 < n) r.z = __ldcg(refs + i + 2);
  return r;
}
__device__ __forceinline__ int get(const int4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// A sequence as the update's lists give it, clamped to the arrays.
struct Wish {
  int parent, len, kept, need;
  bool ok;
};
__device__ __forceinline__ Wish wish_of(const PagesArgs& a, int b) {
  const int most = a.c.max_pages * a.c.page_size;
  Wish w;
  const int p = a.parent ? a.parent[b] : b, len = a.len[b], kept = a.kept[b], need = a.need[b];
  w.parent = p >= 0 && p < a.c.n_seqs ? p : -1;
  w.len = clamp_int(len, 0, most);
  const int has = w.parent < 0 ? 0 : clamp_int(a.len[w.parent], 0, most);
  w.kept = clamp_int(kept, 0, has);
  w.need = clamp_int(need, w.kept, most);
  w.ok = p >= -1 && p < a.c.n_seqs && w.len == len && w.kept == kept && w.need == need;
  return w;
}
__device__ __forceinline__ int pages_of(const PagesArgs& a, int tokens) {
  return (tokens + a.c.page_size - 1) / a.c.page_size;
}

constexpr int kRowsHeld = 1024;
// Entries of a table that a lane has in flight: 100 tables of 5000 pages 27 us (one: 47).
constexpr int kEntries = 4;

__global__ void __launch_bounds__(kThreads, 1)
    pages_update_kernel(const __grid_constant__ PagesArgs a, const Scratch ws, int parts) {
  __shared__ Shared sh;
  __shared__ RowPlan held[kRowsHeld];
  const moe_attn_config& c = a.c;
  const int part = blockIdx.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int thread = part * kThreads + threadIdx.x, threads = parts * kThreads;
  auto valid = [&](int page) { return page >= 0 && page < c.n_pages; };
  // This block's sequences, and its share of the pool.
  const int rows = (c.n_seqs + parts - 1) / parts, row0 = min(part * rows, c.n_seqs);
  const int row1 = min(row0 + rows, c.n_seqs);
  const int share = ((c.n_pages + parts - 1) / parts + 3) / 4 * 4;
  const int page0 = (int)min((long long)part * share, (long long)c.n_pages);
  const int page1 = min(page0 + share, c.n_pages);
  auto plan = [&](int b) { return b - row0 < kRowsHeld ? held + (b - row0) : ws.rows + b; };
  pdl_wait();
  pdl_trigger();

  // Counts as they are; meanwhile what the first sequence of each warp becomes, and its pages.
  if (thread == 0) {
    *a.status = MOE_OK;
    ws.head->n_copies = 0;
  }
  Wish w = {-1, 0, 0, 0, true};
  int page_kept = -1, page_held = -1;
  auto look = [&](int b) {
    w = wish_of(a, b);
    const int kept = pages_of(a, w.kept), from = w.parent == b ? kept : 0;
    if (lane < kept) page_kept = a.table[(int64_t)w.parent * c.max_pages + lane];
    if (from + lane < pages_of(a, w.len)) page_held = a.table[(int64_t)b * c.max_pages + from + lane];
  };
  if (row0 + warp < row1) look(row0 + warp);
  if (a.refs_out != a.refs) {
    const int vecs = c.n_pages / 4;
#pragma unroll 4
    for (int i = thread; i < vecs; i += threads)
      reinterpret_cast<int4*>(a.refs_out)[i] = reinterpret_cast<const int4*>(a.refs)[i];
    for (int i = 4 * vecs + thread; i < c.n_pages; i += threads) a.refs_out[i] = a.refs[i];
  }
  ptx::cluster_sync();

  // Pages given up and gained.
  bool bad = false;
  for (int b = row0 + warp; b < row1; b += kWarps) {
    if (b != row0 + warp) look(b);
    bad |= !w.ok;
    const int kept = pages_of(a, w.kept), len = pages_of(a, w.len);
    const int32_t* old = a.table + (int64_t)b * c.max_pages;
    const int32_t* from = a.table + (int64_t)max(w.parent, 0) * c.max_pages;
    int32_t* to = a.table_out + (int64_t)b * c.max_pages;
    const bool same = w.parent == b, writes = w.need > w.kept && w.kept % c.page_size != 0;
    for (int i0 = lane; i0 < kept; i0 += 32 * kEntries) {
      int page[kEntries];
#pragma unroll
      for (int k = 0; k < kEntries; ++k) {
        const int i = i0 + 32 * k;
        page[k] = i == lane ? page_kept : i < kept ? from[i] : -1;
      }
#pragma unroll
      for (int k = 0; k < kEntries; ++k) {
        const int i = i0 + 32 * k;
        if (i >= kept) break;
        if (!valid(page[k]))
          bad = true;
        else if (!same)
          atomicAdd(a.refs_out + page[k], 1);
        if (to != from) to[i] = page[k];
        if (i == kept - 1) plan(b)->last = writes && valid(page[k]) ? page[k] : -1;
      }
    }
    if (lane == 0) {
      if (kept == 0) plan(b)->last = -1;
      plan(b)->kept = w.kept;
      plan(b)->need = w.need;
    }
    const int first = same ? kept : 0;
    for (int i0 = first + lane; i0 < len; i0 += 32 * kEntries) {
      int page[kEntries];
#pragma unroll
      for (int k = 0; k < kEntries; ++k) {
        const int i = i0 + 32 * k;
        page[k] = i == first + lane ? page_held : i < len ? old[i] : -1;
      }
#pragma unroll
      for (int k = 0; k < kEntries; ++k) {
        if (i0 + 32 * k >= len) break;
        if (valid(page[k]))
          atomicSub(a.refs_out + page[k], 1);
        else
          bad = true;
      }
    }
  }
  ptx::cluster_sync();

  // Free pages of this block's share (the first four of each thread stay in registers), and
  // pages that each of its sequences wants.
  const int mine = page0 + 4 * (int)threadIdx.x;
  const int4 none = make_int4(1, 1, 1, 1), n0 = mine < page1 ? counts_at(a.refs_out, mine, page1) : none;
  auto free_of = [](const int4& n) { return (n.x == 0) + (n.y == 0) + (n.z == 0) + (n.w == 0); };
  auto below = [](const int4& n) { return n.x < 0 || n.y < 0 || n.z < 0 || n.w < 0; };
  long long count = 0, wanted = 0, free_here = 0;
  for (int b0 = row0; b0 < row1 || b0 == row0; b0 += kThreads) {
    const int b = b0 + (int)threadIdx.x;
    int want = 0;
    bool copied = false;
    if (b < row1) {
      const RowPlan* p = plan(b);
      copied = p->last >= 0 && __ldcg(a.refs_out + p->last) > 1;
      want = pages_of(a, p->need) - pages_of(a, p->kept) + copied;
    }
    if (b0 == row0) {
      count = free_of(n0);
      bad |= below(n0);
      for (int i = mine + 4 * kThreads; i < page1; i += 4 * kThreads) {
        const int4 n = counts_at(a.refs_out, i, page1);
        count += free_of(n);
        bad |= below(n);
      }
    }
    long long total, counted;
    const long long before = block_scan(sh, want, total, b0 == row0 ? count : 0, counted);
    if (b < row1) {
      plan(b)->before = wanted + before;
      plan(b)->want = 2 * want + copied;
    }
    wanted += total;
    free_here += counted;
  }
  exchange(sh, part, parts, wanted, free_here);
  const long long free_all = sum_before(sh, 1, parts);
  const long long listed = min(sum_before(sh, 0, parts), free_all);

  // The list of free pages, as far as it will be used.
  long long rank = sum_before(sh, 1, part);
  for (int i0 = page0; i0 < page1 && rank < listed; i0 += 4 * kThreads) {
    const int i = i0 + 4 * (int)threadIdx.x;
    const int4 n = i0 == page0 ? n0 : i < page1 ? counts_at(a.refs_out, i, page1) : none;
    long long total, unused;
    long long at = rank + block_scan(sh, free_of(n), total, 0, unused);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (get(n, k) == 0) {
        if (at < listed) ws.free[at] = i + k;
        ++at;
      }
    rank += total;
  }
  ptx::cluster_sync();

  // Who gets which.
  const long long base = sum_before(sh, 0, part);
  for (int b = row0 + warp; b < row1; b += kWarps) {
    const RowPlan p = *plan(b);
    const int want = p.want / 2, copied = p.want & 1;
    const long long at = base + p.before;
    const bool served = at + want <= free_all;
    if (lane == 0) a.granted[b] = served ? p.need : p.kept;
    if (!served) continue;
    int32_t* to = a.table_out + (int64_t)b * c.max_pages + pages_of(a, p.kept) - copied;
    if (copied && lane == 0) {
      atomicSub(a.refs_out + p.last, 1);
      ws.copies[atomicAdd(&ws.head->n_copies, 1)] = {p.last, __ldcg(ws.free + at), p.kept % c.page_size, 0};
    }
    for (int i0 = lane; i0 < want; i0 += 32 * kEntries) {
      int page[kEntries];
#pragma unroll
      for (int k = 0; k < kEntries; ++k) page[k] = i0 + 32 * k < want ? __ldcg(ws.free + at + i0 + 32 * k) : 0;
#pragma unroll
      for (int k = 0; k < kEntries; ++k) {
        if (i0 + 32 * k >= want) break;
        to[i0 + 32 * k] = page[k];
        a.refs_out[page[k]] = 1;
      }
    }
  }
  if (__syncthreads_or(bad) && threadIdx.x == 0) set_status(a.status, status_check());
}

__global__ void __launch_bounds__(kThreads, 1)
    pages_compact_kernel(const __grid_constant__ PagesArgs a, const Scratch ws, int parts) {
  __shared__ Shared sh;
  const moe_attn_config& c = a.c;
  const int part = blockIdx.x, lane = threadIdx.x % 32;
  const int thread = part * kThreads + threadIdx.x, threads = parts * kThreads;
  pdl_wait();
  pdl_trigger();
  if (thread == 0) {
    *a.status = MOE_OK;
    ws.head->n_copies = 0;
  }
  ptx::cluster_sync();  // the cluster's blocks have started

  // Pages in use, of this block's share of the pool and of all of it.
  const int share = ((c.n_pages + parts - 1) / parts + 3) / 4 * 4;
  const int page0 = (int)min((long long)part * share, (long long)c.n_pages);
  const int page1 = min(page0 + share, c.n_pages);
  bool bad = false;
  int count = 0;
#pragma unroll 4
  for (int i = page0 + threadIdx.x; i < page1; i += kThreads) {
    const int n = a.refs[i];
    count += n > 0;
    bad |= n < 0;
  }
  long long live_here, unused;
  block_scan(sh, count, live_here, 0, unused);
  exchange(sh, part, parts, live_here, 0);
  const int live = (int)sum_before(sh, 0, parts);

  // Holes below that number and pages in use above it, by rank.
  int rank = (int)sum_before(sh, 0, part);  // pages in use before
  for (int i0 = page0; i0 < page1; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const int n = i < page1 ? max(a.refs[i], 0) : 0;
    long long total;
    const int before = rank + (int)block_scan(sh, n > 0, total, 0, unused);
    if (i < page1) {
      if (i == live) ws.head->n_copies = live - before;  // the holes below
      const bool stays = n > 0 && i < live;
      if (n > 0 && !stays) {
        ws.high[before] = i;
      } else {
        a.page_map[i] = stays ? i : -1;
        a.refs_out[i] = n;
        if (i < live && !stays) ws.free[i - before] = i;
      }
    }
    rank += (int)total;
  }
  ptx::cluster_sync();
  const int moves = __ldcg(&ws.head->n_copies);
  for (int k = thread; k < moves; k += threads) {
    const int src = __ldcg(ws.high + live - moves + k), dst = __ldcg(ws.free + k);
    const int n = a.refs[src];
    a.page_map[src] = dst;
    a.refs_out[dst] = n;
    a.refs_out[src] = 0;
    ws.copies[k] = {src, dst, c.page_size, 0};
  }
  ptx::cluster_sync();
  for (int b = thread / 32; b < c.n_seqs; b += threads / 32) {
    const int most = c.max_pages * c.page_size, len = a.len[b];
    bad |= len < 0 || len > most;
    const int held = pages_of(a, clamp_int(len, 0, most));
    const int64_t row = (int64_t)b * c.max_pages;
    for (int i0 = lane; i0 < held; i0 += 32 * kEntries) {
      int page[kEntries], now[kEntries];
#pragma unroll
      for (int k = 0; k < kEntries; ++k) page[k] = i0 + 32 * k < held ? a.table[row + i0 + 32 * k] : -1;
#pragma unroll
      for (int k = 0; k < kEntries; ++k)
        now[k] = page[k] >= 0 && page[k] < c.n_pages ? __ldcg(a.page_map + page[k]) : -1;
#pragma unroll
      for (int k = 0; k < kEntries; ++k) {
        if (i0 + 32 * k >= held) break;
        bad |= now[k] < 0;
        a.table_out[row + i0 + 32 * k] = now[k] < 0 ? page[k] : now[k];
      }
    }
  }
  if (thread == 0) *a.n_live = live;
  if (__syncthreads_or(bad) && threadIdx.x == 0) set_status(a.status, status_check());
}

// ---- copies --------------------------------------------------------------------
struct CopyArgs {
  PagesArgs a;
  const PlanHead* head;  // the list of a plan, or null: a's
  const PageCopy* copies;
  int elem;              // bytes of a cached element
  int row_vecs;          // 16-byte vectors of a token's head
  int chunks;            // of a page, a warp each
  int units;             // of a copy: the chunks of keys and of values, and one of scales
  int scale_tokens;      // scales of a head: a token's each, one (a page's), or none (0)
  int packed;            // a page's tokens are one run of bytes, in order
};

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ CopyArgs p) {
  const PagesArgs& a = p.a;
  const moe_attn_config& c = a.c;
  const int lane = threadIdx.x % 32;
  const bool list = p.head == nullptr;
  pdl_wait();
  pdl_trigger();
  int block = blockIdx.x, blocks = gridDim.x;
  if (list) {
    if (block == 0) {
      bool bad = false;
#pragma unroll 8
      for (int i = threadIdx.x; i < a.n_copies; i += kCopyThreads) {
        const int src = __ldg(a.src + i), dst = __ldg(a.dst + i);
        bad |= src < 0 || src >= a.n_src_pages || dst < 0 || dst >= c.n_pages;
      }
      bad = __syncthreads_or(bad);
      if (threadIdx.x == 0) *a.status = bad ? status_check() : MOE_OK;
      return;
    }
    --block, --blocks;
  }
  const long long n = list ? a.n_copies : p.head->n_copies, units = n * p.units;
  constexpr int kBlockWarps = kCopyThreads / 32;
  for (long long u = (long long)block * kBlockWarps + threadIdx.x / 32; u < units;
       u += (long long)blocks * kBlockWarps) {
    const long long i = u / p.units;
    const int unit = (int)(u - i * p.units);
    PageCopy cp;
    if (list) {
      cp = {a.src[i], a.dst[i], c.page_size, 0};
      if (cp.src < 0 || cp.src >= a.n_src_pages || cp.dst < 0 || cp.dst >= c.n_pages) continue;
    } else {
      cp = p.copies[i];
    }
    if (unit == 2 * p.chunks) {  // scales: of every head, those of the tokens
      const int words = p.scale_tokens == 1 ? 1 : cp.tokens;
      const int64_t from = (int64_t)cp.src * c.n_kv_heads * p.scale_tokens;
      const int64_t to = (int64_t)cp.dst * c.n_kv_heads * p.scale_tokens;
      for (int h = 0; h < c.n_kv_heads; ++h)
        for (int w = lane; w < words; w += 32) {
          const int64_t at = (int64_t)h * p.scale_tokens + w;
          a.k_scale[to + at] = a.k_from_scale[from + at];
          a.v_scale[to + at] = a.v_from_scale[from + at];
        }
      continue;
    }
    const bool key = unit < p.chunks;
    const char* from = static_cast<const char*>(key ? a.k_from : a.v_from) +
                       (int64_t)cp.src * c.page_stride * p.elem;
    char* to = static_cast<char*>(key ? a.k_cache : a.v_cache) + (int64_t)cp.dst * c.page_stride * p.elem;
    const int v0 = (key ? unit : unit - p.chunks) * 32 * kCopyVecs + lane;
    const int v1 = cp.tokens * c.n_kv_heads * p.row_vecs;
    uint4 x[kCopyVecs];
    int64_t at[kCopyVecs];
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k) {
      const int v = v0 + 32 * k;
      at[k] = (int64_t)v * 16;
      if (!p.packed) {
        const int row = v / p.row_vecs, token = row / c.n_kv_heads;
        at[k] = ((int64_t)token * c.token_stride + (int64_t)(row - token * c.n_kv_heads) * c.head_stride) *
                    p.elem +
                (int64_t)(v - row * p.row_vecs) * 16;
      }
      if (v < v1) x[k] = *reinterpret_cast<const uint4*>(from + at[k]);
    }
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k)
      if (v0 + 32 * k < v1) *reinterpret_cast<uint4*>(to + at[k]) = x[k];
  }
}

cudaError_t launch_copies(const PagesArgs& a, const Scratch* ws, long long most, cudaStream_t s) {
  const moe_attn_config& c = a.c;
  CopyArgs p = {};
  p.a = a;
  p.head = ws ? ws->head : nullptr;
  p.copies = ws ? ws->copies : nullptr;
  p.elem = is_e4m3(c.cache_dtype) ? 1 : c.cache_dtype == MOE_F32 ? 4 : 2;
  p.row_vecs = c.head_dim * p.elem / 16;
  const int page_vecs = c.page_size * c.n_kv_heads * p.row_vecs;  // of a page
  p.chunks = ceil_div(page_vecs, 32 * kCopyVecs);
  p.scale_tokens = c.cache_dtype == MOE_E4M3 ? c.page_size : c.cache_dtype == MOE_E4M3_PAGE ? 1 : 0;
  p.units = 2 * p.chunks + (p.scale_tokens > 0);
  p.packed = c.head_stride == c.head_dim && c.token_stride == (int64_t)c.n_kv_heads * c.head_dim;
  const long long fill = 8LL * num_sms(), need = (most * p.units + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  const unsigned blocks = (unsigned)(need < fill ? need : fill) + (ws ? 0 : 1);
  if (blocks == 0) return cudaSuccess;
  ProfScope prof(K_PAGES_COPY, s);
  return launch_pdl(pages_copy_kernel, dim3(blocks), dim3(kCopyThreads), 0, s, 1, p);
}

// Blocks of a plan's cluster: one for each 8192 counts and entries (4096 and 16384: as long
// or longer). us of an update in up to eight blocks and in up to 16: 65536 pages and 256
// sequences 15 and 13, 524288 and 1000 44 and 30, 4 million and 2000 204 and 115.
int plan_parts(const moe_attn_config& c) {
  const long long work = c.n_pages + (long long)c.n_seqs * c.max_pages;
  int parts = 1;
  while (parts < kMaxParts && work > 8192LL * parts) parts *= 2;
  return parts;
}
// Clusters of more than eight blocks, once per device.
cudaError_t allow_parts(const void* kernel, int parts, int* configured) {
  int dev = 0;
  cudaError_t e = parts > 8 ? cudaGetDevice(&dev) : cudaSuccess;
  if (e != cudaSuccess || parts <= 8 || *configured == dev) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) *configured = dev;
  return e;
}

}  // namespace

size_t pages_scratch_bytes(const moe_attn_config& c) {
  return scratch_of(c, reinterpret_cast<void*>(256)).bytes;
}

cudaError_t launch_pages_update(const PagesArgs& a, void* scratch, cudaStream_t s) {
  static thread_local int configured = -1;
  const Scratch ws = scratch_of(a.c, scratch);
  const int parts = plan_parts(a.c);
  cudaError_t e = allow_parts(reinterpret_cast<const void*>(pages_update_kernel), parts, &configured);
  if (e == cudaSuccess) {
    ProfScope p(K_PAGES, s);
    e = launch_pdl(pages_update_kernel, dim3((unsigned)parts), dim3(kThreads), 0, s, parts, a, ws, parts);
  }
  return e == cudaSuccess ? launch_copies(a, &ws, a.c.n_seqs, s) : e;
}
cudaError_t launch_pages_compact(const PagesArgs& a, void* scratch, cudaStream_t s) {
  static thread_local int configured = -1;
  const Scratch ws = scratch_of(a.c, scratch);
  const int parts = plan_parts(a.c);
  cudaError_t e = allow_parts(reinterpret_cast<const void*>(pages_compact_kernel), parts, &configured);
  if (e == cudaSuccess) {
    ProfScope p(K_PAGES, s);
    e = launch_pdl(pages_compact_kernel, dim3((unsigned)parts), dim3(kThreads), 0, s, parts, a, ws, parts);
  }
  return e == cudaSuccess ? launch_copies(a, &ws, a.c.n_pages / 2, s) : e;
}
cudaError_t launch_pages_copy(const PagesArgs& a, cudaStream_t s) {
  return launch_copies(a, nullptr, a.n_copies, s);
}

}  // namespace moe
