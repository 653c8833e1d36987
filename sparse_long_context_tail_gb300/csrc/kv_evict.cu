// Eviction of cache entries by accumulated attention weight.
//
// Two launches.  The first finds each request's kept entries: the first `sinks`, the last
// `recent`, and of those between the heaviest, as many as the budget leaves; weights are not
// negative, so their bit patterns are ordered as they are, and the least kept weight is
// found digit by digit (11, 10 and 10 bits) from histograms, one cluster of CTAs a request.
// Of entries as heavy as it the first ones are kept.  Each CTA then lists the kept ones of its
// run of entries, in order.
//
// Bound by latency: about ten steps over the whole cluster, a load, a barrier or a scan each (131072 entries 15 us, 1088 8 us).
//
// The second moves them together.  Entry j of the result was entry s_j >= j, so chunks of
// places written in ascending order never overwrite what a later chunk has yet to read.  To run
// them at the same time, a CTA reads its whole chunk (64 entries of one kv head) into shared memory, says so, and
// writes once the chunks have been read whose entries lie in its places: the entries in 64 places go to
// 64 places in a row at most, which two chunks hold.  Chunks are taken by ticket, so those that
// a CTA waits for have been taken before by CTAs that wait for nothing to read them.
//
// Bound by HBM and by the records' layout: a row's values are 4 to 8 bytes side by side, so that of a scattered
// entry whole 32-byte sectors are read.  32768 of 131072 entries of 8 heads of d = 128: 106 MB read for 38 MB of entries, 26 us.
#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include "kv_layout.cuh"
#include "sm100_ptx.cuh"
#include "upf_internal.cuh"

namespace upf {

struct KvEvictPlan {
  int32_t n, left;    // entries before and after
  int32_t move;       // 1: some are to be moved or copied
  int32_t pad;
};

namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 16, kManyCluster = 8;    // of few requests, of many
constexpr int kUnroll = 2;
constexpr int kPasses = 3, kBins = 2048, kOwnBins = 4;   // digits; bins of a digit; of a thread
constexpr int kMaxHeld = 9;           // fours of weights of a thread that stay in shared memory (144 KB a CTA)
constexpr int kChunk = 64;            // places of a moving CTA (16 ragged requests of d = 128: 59 us, with 32 places 62)
// Threads of a moving CTA (evicting of 64 requests of d = 256: 55.6 us with 128, 51.5 with 256; 16 of d = 128: 58.9 and 60.8).
constexpr int move_threads(int d) { return d == 256 ? 256 : 128; }
static_assert(move_threads(64) >= kChunk, "a thread for each entry of a chunk");

__host__ __device__ constexpr int64_t chunks_of(int64_t places) { return (places + kChunk - 1) / kChunk; }

// The slot of entry e of a table row, or -1 if its page is bad.
__device__ __forceinline__ int64_t slot_of(const int32_t* row, int e, int shift, int64_t num_slots) {
  const int page = row[e >> shift];
  const int64_t slot = ((int64_t)page << shift) + (e & ((1 << shift) - 1));
  return page >= 0 && slot < num_slots ? slot : -1;
}

// In the shared memory of the cluster's CTA `rank`, at the place that `mine` has in this one's.
__device__ __forceinline__ int4 ld_cluster4(const int32_t* mine, uint32_t rank) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(ptx::mapa_shared(ptx::smem_u32(mine), rank))
               : "memory");
  return v;
}
__device__ __forceinline__ void add_cluster(int32_t* mine, uint32_t rank, int32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(ptx::mapa_shared(ptx::smem_u32(mine), rank)), "r"(v)
               : "memory");
}
__device__ __forceinline__ void or_cluster(int32_t* mine, uint32_t rank, int32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(ptx::mapa_shared(ptx::smem_u32(mine), rank)), "r"(v)
               : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

__device__ __forceinline__ void copy_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}

// Sum over the threads before this one.
__device__ __forceinline__ int block_scan(int v, int* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  return __reduce_add_sync(0xFFFFFFFFu, lane < warp ? scratch[lane] : 0) + x - v;
}
static_assert(kSelWarps <= 32, "a warp adds up the warps' sums");

// A cluster of `ctas` CTAs a request.  A warp has a run of entries of its own, `held` times 128 of them
// in shared memory through all passes (294912 entries with eight CTAs, 589824 with 16; of more, the rest is read again).
// What bounds it is the instructions of few SMs: four entries a lane at a time.  Loops stay rolled: the instructions of a launch run
// a few times only, so that fetching long unrolled ones costs more than it saves (weights in registers,
// 16 times unrolled: 22 us for 1088 entries, 10 rolled).
__global__ void __launch_bounds__(kSelThreads) kv_evict_select_kernel(const KvEvictArgs a, const uint32_t ctas,
                                                                    const int held) {
  extern __shared__ int4 held_bits[];    // [warp][held at most][lane], and before it, in a cluster, [kPasses][kBins] sums
  __shared__ __align__(16) int32_t hist[kPasses][kBins];     // entries of this CTA by digit
  __shared__ int32_t scratch[kPasses][32], found[kPasses][2], warp_counts[kSelWarps][2];
  __shared__ int32_t bad_any, counts[2];                     // of all CTAs; of those before this one
  // of all CTAs, each CTA a run of the bins
  int32_t* const sums = ctas > 1 ? reinterpret_cast<int32_t*>(held_bits) : &hist[0][0];
  const uint32_t rank = blockIdx.x % ctas;   // in the request's cluster
  const int r = blockIdx.x / ctas, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int first = rank * kSelThreads + tid, stride = ctas * kSelThreads;   // of the cluster's threads
  auto sync = [&] {
    if (ctas > 1) ptx::cluster_sync();
    else __syncthreads();
  };
  const float* const w = a.w + r * a.w_stride;
  const int32_t* const row = a.table + r * a.table_stride;
  for (int i = tid; i < kPasses * kBins / 4; i += kSelThreads) {
    reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
    if (ctas > 1) reinterpret_cast<int4*>(sums)[i] = make_int4(0, 0, 0, 0);
  }
  if (tid == 0) bad_any = counts[0] = counts[1] = 0;
  if (ctas > 1) cluster_arrive();        // the others may add to these
  pdl_wait();
  pdl_trigger();         // only now: the second launch writes what launches before this one may read
  const int n = a.kv_len[r];
  // the second launch's ticket and marks
  if (r == 0 && first == 0) *a.ticket = 0;
  const int64_t marks = a.H * chunks_of(a.cap);
  for (int64_t i = first; i < marks; i += stride) a.read[r * marks + i] = 0;

  // ---- is there anything to do, and can it be done?
  bool fine = n >= 0 && n <= ((int64_t)a.max_pages << a.page_shift) && n <= a.w_cols;
  const bool cut = fine && n > a.trigger;
  const int left = cut ? a.budget : n;
  const bool move = cut || a.table_out || a.w_out != a.w;
  if (move) fine = fine && left <= a.w_out_cols && (!a.table_out || left <= ((int64_t)a.max_pages_out << a.page_shift));

  // ---- the weights between the ends: a warp has 128 `its` of them, a lane four side by side at a time
  const int middle = n - a.sinks - a.recent, want = a.budget - a.sinks - a.recent;
  const float* const m = w + a.sinks;
  const int its = fine && cut ? (middle + 128 * kSelWarps * int(ctas) - 1) / (128 * kSelWarps * int(ctas)) : 0;
  const int from = (rank * kSelWarps + warp) * its * 128;           // under 2^30 + 2^18
  const int in_smem = min(its, held);
  // what is looked at once is on its way first: a load takes longer than counting does
  const int page = 1 << a.page_shift, ends = fine && cut ? a.sinks + a.recent : 0;
  const int pages = fine && (cut || a.table_out) ? (n + page - 1) / page : 0;
  const int pages_out = fine && a.table_out ? (left + page - 1) / page : 0;
  const int32_t* const row_out = a.table_out + r * a.table_out_stride;
  auto end_weight = [&](int e) { return __float_as_int(w[e < a.sinks ? e : e + middle]); };
  const int32_t page0 = first < pages ? row[first] : 0, page_out0 = first < pages_out ? row_out[first] : 0;
  const int end0 = first < ends ? end_weight(first) : 0;
  int4* const mine = held_bits + (ctas > 1 ? kPasses * kBins / 4 : 0) + warp * in_smem * 32;
  for (int k = lane; k < 128 * in_smem && from + k < middle; k += 32) copy_async4(reinterpret_cast<int32_t*>(mine) + k, m + from + k);
  asm volatile("cp.async.commit_group;" ::: "memory");
  // Bits of a weight as a signed number: their order is that of the weights; -0 is 0, and an entry that
  // is not there -1, which no kept weight is or is below.
  auto key_of = [&](int bits) { return bits == INT_MIN ? 0 : bits; };
  auto fetch = [&](int it) {
    int v[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int i = from + it * 128 + lane * 4 + y;
      v[y] = i >= middle ? -1 : key_of(it < in_smem ? reinterpret_cast<const int32_t*>(mine)[it * 128 + lane * 4 + y] : __float_as_int(m[i]));
    }
    return make_int4(v[0], v[1], v[2], v[3]);
  };
  // f(iteration, the lane's four): entries from + 128 iteration + 4 lane ..
  auto each = [&](auto&& f) {
#pragma unroll kUnroll
    for (int it = 0; it < its; ++it) f(it, it < in_smem ? mine[it * 32 + lane] : fetch(it));
  };
  // One to the bin of each entry whose upper bits are those of `least`.
  auto count = [&](int pass, int least) {
    const int shift = 20 - 10 * pass, bits = pass == 0 ? 11 : 10, mask = (1 << bits) - 1;
    int zeros = 0;     // they may be many, and equal bins wait for one another
    each([&](int, int4 v) {
      const int x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const bool on = pass == 0 ? x[y] >= 0 : x[y] >> (shift + bits) == least >> (shift + bits);
        if (on && x[y] != 0) atomicAdd(&hist[pass][x[y] >> shift & mask], 1);
        zeros += on && x[y] == 0;
      }
    });
    zeros = __reduce_add_sync(0xFFFFFFFFu, zeros);
    if (lane == 0 && zeros) atomicAdd(&hist[pass][0], zeros);
    if (ctas == 1) return;
    // what this CTA has found goes to the sums (all of them in every CTA, as 16 additions a bin: 3 us more at 131072 entries)
    __syncthreads();
    if (pass == 0) cluster_wait();
#pragma unroll 1
    for (int i = tid; i <= mask; i += kSelThreads)
      if (const int x = hist[pass][i]) add_cluster(sums + pass * kBins + i, uint32_t(i) * ctas >> bits, x);
  };
  __syncthreads();   // the bins are empty
  int bad = 0;
  if (fine) {
    // is the p-th page, of `all` entries, outside the cache?  (The cache may end inside a page, behind the entries.)
    auto bad_page = [&](int32_t id, int p, int all) {
      return id < 0 || ((int64_t)id << a.page_shift) + min(page, all - (p << a.page_shift)) > a.num_slots;
    };
    for (int p = first; p < pages; p += stride) bad |= bad_page(p == first ? page0 : row[p], p, n);
    for (int p = first; p < pages_out; p += stride) bad |= bad_page(p == first ? page_out0 : row_out[p], p, left);
    auto is_bad = [&](int bits) { return key_of(bits) < 0 || bits >= 0x7F800000; };
    if (cut) {
      for (int e = first; e < ends; e += stride)
        if (is_bad(e == first ? end0 : end_weight(e))) bad |= 2;
      // the lanes' own copies, and the others': as keys from here on
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
#pragma unroll kUnroll
      for (int it = 0; it < its; ++it) {
        const int4 v = fetch(it);
        const int last = middle - (from + it * 128 + lane * 4);   // of the four, those that are there
        if ((last > 0 && is_bad(v.x)) || (last > 1 && is_bad(v.y)) || (last > 2 && is_bad(v.z)) || (last > 3 && is_bad(v.w))) bad |= 2;
        if (it < in_smem) mine[it * 32 + lane] = v;
      }
      if (want > 0) count(0, 0);
    }
  }
  if (ctas > 1 && !(fine && cut && want > 0)) cluster_wait();   // as in the first count
  if (bad) {
    if (ctas == 1) atomicOr(&bad_any, bad);
    for (uint32_t k = 0; ctas > 1 && k < ctas; ++k) or_cluster(&bad_any, k, bad);
  }
  sync();
  bad = bad_any;
  if (!fine || bad) {
    if (first == 0) set_status(a.status, !fine || (bad & 1) ? UPF_ERR_INVALID_ARG : UPF_ERR_NONFINITE);
    fine = false;
  }
  int32_t* const list = a.list + (int64_t)r * a.cap;
  float* const list_w = a.list_w + (int64_t)r * a.cap;
  int32_t* const kept = a.kept ? a.kept + r * a.kept_stride : nullptr;
  int32_t* const bounds = a.bounds + r * (chunks_of(a.cap) + 1);
  if (!fine || !cut) {
    // a request that is skipped: its length, which of other pages' entries is 0, and where that would be the last
    // to be known of it, its length marked as a bad one
    const int gone = a.len_out != a.kv_len ? 0 : n < 0 ? n : -1 - n;
    const int now = fine ? left : a.table_out ? gone : n;
    if (first == 0) {
      a.plan[r] = KvEvictPlan{n, now, fine && move ? 1 : 0, 0};
      a.len_out[r] = now;
    }
    for (int j = first; kept && j < a.budget; j += stride) kept[j] = fine && j < left ? j : -1;
    for (int j = first; fine && move && j < left; j += stride) {
      list[j] = j;
      list_w[j] = w[j];
      if (j % kChunk == 0) bounds[j / kChunk] = j;
    }
    return;
  }
  // ---- the least kept weight
  int least = INT_MAX;     // its bits, as far as they are known; none to be kept: above every weight
  int need = 0;            // how many of the entries as heavy as it are kept
  if (want > 0) {
    least = 0;
    need = want;
#pragma unroll 1
    for (int pass = 0; pass < kPasses; ++pass) {
      const int shift = 20 - 10 * pass, bins = pass == 0 ? 2048 : 1024;
      if (pass > 0) {
        count(pass, least);
        sync();
      }
      // thread t: kOwnBins bins below bins - kOwnBins t, from the heaviest on
      const int first_bin = bins - kOwnBins * (tid + 1);
      int c[kOwnBins] = {}, mine_all = 0;
      if (first_bin >= 0)
#pragma unroll
        for (int y = 0; y < kOwnBins; y += 4) {
          const int32_t* const at = sums + pass * kBins + first_bin + y;
          const int4 v = ctas > 1 ? ld_cluster4(at, uint32_t(first_bin) * ctas / bins) : *reinterpret_cast<const int4*>(at);
          c[y] = v.x, c[y + 1] = v.y, c[y + 2] = v.z, c[y + 3] = v.w;
          mine_all += v.x + v.y + v.z + v.w;
        }
      int before = block_scan(mine_all, scratch[pass]);
      if (before < need && before + mine_all >= need) {
#pragma unroll
        for (int y = kOwnBins - 1; y >= 0; --y) {
          if (before < need && before + c[y] >= need) {
            found[pass][0] = first_bin + y;
            found[pass][1] = need - before;
          }
          before += c[y];
        }
      }
      __syncthreads();
      least |= found[pass][0] << shift;
      need = found[pass][1];
    }
  }
  // ---- entries above it and as heavy: before this warp, before this CTA
  int above = 0, equal = 0;
  each([&](int, int4 v) {
    above += (v.x > least) + (v.y > least) + (v.z > least) + (v.w > least);
    equal += (v.x == least) + (v.y == least) + (v.z == least) + (v.w == least);
  });
  above = __reduce_add_sync(0xFFFFFFFFu, above);
  equal = __reduce_add_sync(0xFFFFFFFFu, equal);
  if (lane == 0) {
    warp_counts[warp][0] = above;
    warp_counts[warp][1] = equal;
  }
  __syncthreads();
  {
    const int x = lane < kSelWarps ? warp_counts[lane][0] : 0, y = lane < kSelWarps ? warp_counts[lane][1] : 0;
    above = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? x : 0);
    equal = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? y : 0);
    if (warp == 0) {
      const int all_x = __reduce_add_sync(0xFFFFFFFFu, x), all_y = __reduce_add_sync(0xFFFFFFFFu, y);
      if (lane > rank && lane < ctas) {
        add_cluster(&counts[0], lane, all_x);
        add_cluster(&counts[1], lane, all_y);
      }
    }
  }
  if (ctas > 1) {
    ptx::cluster_sync();      // the last: no CTA reads or writes another's words from here on
    above += counts[0];
    equal += counts[1];
  }
  // ---- the list
  auto put = [&](int j, int e, float x) {
    list[j] = e;
    list_w[j] = x;
    if (kept) kept[j] = e;
  };
  // of the places' chunks: how many kept entries lie before them now
  auto bound = [&](int j, int e) {
    if (e % kChunk == 0 && e < left + kChunk) bounds[e / kChunk] = j;
  };
  const uint32_t before_lane = (1u << lane) - 1;
  each([&](int it, int4 v) {
    const int x[4] = {v.x, v.y, v.z, v.w};
    int over = above, same = equal;        // before the lane
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, x[y] > least), s = __ballot_sync(0xFFFFFFFFu, x[y] == least);
      over += __popc(m & before_lane);
      same += __popc(s & before_lane);
      above += __popc(m);
      equal += __popc(s);
    }
    const int e0 = a.sinks + from + it * 128 + lane * 4;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int j = a.sinks + over + min(same, need);   // kept entries before this one
      if (x[y] > least || (x[y] == least && same < need)) put(j, e0 + y, __int_as_float(x[y]));
      if (x[y] >= 0) bound(j, e0 + y);
      over += x[y] > least;
      same += x[y] == least;
    }
  });
  for (int j = first; j < a.sinks + a.recent; j += stride) {
    const int e = j < a.sinks ? j : j + middle;
    put(j < a.sinks ? j : j + want, e, w[e]);
    bound(j < a.sinks ? j : j + want, e);
  }
  if (first == 0) {
    a.plan[r] = KvEvictPlan{n, left, 1, 0};
    a.len_out[r] = left;
  }
}

__device__ __forceinline__ int32_t load_acquire(const int32_t* p) {
  int32_t v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(int32_t* p, int32_t v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// A CTA per chunk.  Of a record a row's keys are one run of bytes, its values eight (64 bytes apart at d = 128) and its
// scales one and many: lanes side by side take the pieces of one entry, which lie in a few lines, while
// the kept entries may lie anywhere.
template <int kDim>
__global__ void __launch_bounds__(move_threads(kDim)) kv_evict_move_kernel(const KvEvictArgs a) {
  constexpr int kRecord = kv::record_bytes(kDim), kD = kv::part_dims(kDim), kParts = kDim / kD, kC = kD / 16;
  constexpr int kRecords = kChunk / 16, kGroups = kDim / 16, kThreads = move_threads(kDim);
  __shared__ __align__(128) uint8_t rec[kRecords * kRecord];
  __shared__ const uint8_t* base[kChunk];   // records of the entries
  __shared__ uint8_t old_row[kChunk];       // and their rows in them
  __shared__ uint8_t* place[kRecords];      // records of the places
  __shared__ uint32_t said;
  const int tid = threadIdx.x;
  const uint32_t per = a.R * a.H;
  const int64_t per_head = chunks_of(a.cap);
  pdl_wait();
  if (tid == 0) said = atomicAdd(a.ticket, 1);
  __syncthreads();
  // chunk first, so that tickets of one request and head ascend with the chunk
  const uint32_t u = said;
  const int c = int(u / per), rh = int(u - c * per), r = rh / a.H, h = rh - r * a.H;
  const int j0 = c * kChunk;
  const int64_t at = (int64_t)r * a.cap + j0;
  const KvEvictPlan plan = a.plan[r];
  const int mine = tid < kChunk && j0 + tid < a.cap ? a.list[at + tid] : 0;
  const int64_t bound = r * (per_head + 1) + c;
  const int lo = a.bounds[bound], next = a.bounds[bound + 1];
  if (!plan.move) return;
  const int places = min(kChunk, plan.left - j0);
  // ---- weights: this chunk's, and this chunk's share of the places that fall free
  if (h == 0) {
    float* const w = a.w_out + r * a.w_out_stride;
    if (tid < places) w[j0 + tid] = a.list_w[at + tid];
    const int end = min(plan.n, a.w_out_cols), chunks = max(1, int(chunks_of(plan.left)));
    if (c < chunks)
      for (int64_t e = plan.left + (int64_t)c * kThreads + tid; e < end; e += (int64_t)chunks * kThreads) w[e] = 0.f;
  }
  if (places <= 0) return;
  int32_t* const mark = a.read + rh * per_head;
  auto record_of = [&](int64_t slot) { return a.data + ((slot >> 4) * a.H + h) * (int64_t)kRecord; };
  const int whole = (places + 15) / 16;
  if (tid < places) {
    const int64_t slot = slot_of(a.table + r * a.table_stride, mine, a.page_shift, a.num_slots);
    base[tid] = record_of(slot);
    old_row[tid] = uint8_t(slot & 15);
  }
  if (const int k = kThreads - 1 - tid; k < whole)
    place[k] = record_of(slot_of(a.table_out ? a.table_out + r * a.table_out_stride : a.table + r * a.table_stride, j0 + k * 16,
                                 a.page_shift, a.num_slots));
  // ---- nothing to move where all entries stay where they are: list[j] >= j, so that the last one tells
  const bool in_place = !a.table_out || (a.table_out == a.table && (r == 0 || a.table_out_stride == a.table_stride));
  if (__syncthreads_or(in_place && tid == places - 1 && mine == j0 + tid)) {
    if (tid == 0) store_release(mark + c, 1);
    return;
  }
  // ---- read.  V scales are bytes, through registers; the rest goes to shared memory by itself
  constexpr int kBytes = kChunk * kGroups / kThreads;
  uint8_t scale[kBytes];
#pragma unroll
  for (int i = 0; i < kBytes; ++i) {
    const int k = (i * kThreads + tid) / kGroups;
    scale[i] = k < places ? base[k][kv::v_scale(kDim, old_row[k], tid % kGroups)] : 0;
  }
  // the record that the request ends in keeps its other rows
  if (places & 15) {
    for (int i = tid; i < kRecord / 16; i += kThreads)
      reinterpret_cast<uint4*>(rec + (whole - 1) * kRecord)[i] = reinterpret_cast<const uint4*>(place[whole - 1])[i];
    __syncthreads();
  }
  constexpr int kKeyVecs = kD / 32;    // 16-byte vectors of a row's keys in a part
#pragma unroll
  for (int i0 = 0; i0 < kChunk * kParts * kKeyVecs; i0 += kThreads) {
    const int i = i0 + tid, k = i / (kParts * kKeyVecs), v = i % (kParts * kKeyVecs), p = v / kKeyVecs, y = v % kKeyVecs;
    const int off = p * 8 * kD + y * 16;
    if (k < places) copy_async16(rec + (k >> 4) * kRecord + off + (k & 15) * (kD / 2), base[k] + off + old_row[k] * (kD / 2));
  }
#pragma unroll
  for (int i0 = 0; i0 < kChunk * kParts * 8; i0 += kThreads) {
    const int i = i0 + tid, k = i / (kParts * 8), z = i % (kParts * 8), p = z / 8, y = z % 8;
    auto off = [&](int s) { return 8 * kDim + p * 8 * kD + (s >> 3) * 4 * kD + y * 8 * kC + (s & 7) * kC; };
    if (k >= places) continue;
    uint8_t* const dst = rec + (k >> 4) * kRecord + off(k & 15);
    if constexpr (kC == 8) copy_async8(dst, base[k] + off(old_row[k]));
    else copy_async4(dst, base[k] + off(old_row[k]));
  }
#pragma unroll
  for (int i0 = 0; i0 < kChunk * kGroups / 4; i0 += kThreads) {
    const int i = i0 + tid, k = i / (kGroups / 4), y = i % (kGroups / 4) * 4;
    if (i < kChunk * kGroups / 4 && k < places)
      copy_async4(rec + (k >> 4) * kRecord + kv::k_scale(kDim, k & 15, y), base[k] + kv::k_scale(kDim, old_row[k], y));
  }
#pragma unroll
  for (int i = 0; i < kBytes; ++i) {
    const int k = (i * kThreads + tid) / kGroups;
    if (k < places) rec[(k >> 4) * kRecord + kv::v_scale(kDim, k & 15, tid % kGroups)] = scale[i];
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  // ---- say that it has been read, and wait until the entries in these places have been
  __syncthreads();
  if (tid == 0) {
    store_release(mark + c, 1);
    const int hi = j0 + kChunk >= plan.n ? plan.left : next;   // entries lo .. hi - 1 of the list lie in the places
    bool ok = true;
    const long long t0 = clock64();
    for (int k = lo / kChunk; lo < hi && k <= (hi - 1) / kChunk && k < c && ok; ++k)
      while (ok && load_acquire(mark + k) == 0) ok = clock64() - t0 < a.wait_limit;
    if (!ok) set_status(a.status, UPF_ERR_TIMEOUT);
    said = ok;
  }
  __syncthreads();
  if (!said) return;
  for (int i = tid; i < whole * (kRecord / 16); i += kThreads)
    reinterpret_cast<uint4*>(place[i / (kRecord / 16)])[i % (kRecord / 16)] = reinterpret_cast<const uint4*>(rec)[i];
}

template <int kDim>
cudaError_t launch_move(const KvEvictArgs& a, cudaStream_t s) {
  const int64_t units = (int64_t)a.R * a.H * chunks_of(a.cap);   // under 2^31 (checked by the caller)
  return launch_kernel(kv_evict_move_kernel<kDim>, dim3(unsigned(units)), move_threads(kDim), 0, s, true, a);
}

// CTAs of a request's cluster: one per 8192 entries that there may be, up to kMaxCluster for at most four
// requests.  A GPC holds one cluster of 16, and seven are there at once: 7 requests of 131072 entries take 34.5 us with
// 16 CTAs and 35.5 with 8, 8 requests 54.8 and 37.2.  One request: 262144 entries 37 and 43 us, 10^6 82 and 126.  One per 4096 or per
// 16384 entries: 64 requests of up to 9000 60.2 and 50.6 us (51.4 with 8192), one of 131072 43.5 and 48.9 (43.4).
int cluster_of(const KvEvictArgs& a) {
  const int64_t most = std::min<int64_t>((int64_t)a.max_pages << a.page_shift, a.w_cols);
  const int limit = a.R <= 4 ? kMaxCluster : kManyCluster;
  int c = 1;
  while (c < limit && most > (int64_t)c * 8192) c *= 2;
  return c;
}

}  // namespace

size_t kv_evict_workspace(KvEvictArgs& a, void* ws) {
  const int64_t places = std::min<int64_t>((int64_t)a.max_pages << a.page_shift, a.trigger);
  a.cap = int(places);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    void* const p = static_cast<char*>(ws) + (ws ? off : 0);
    off = (off + bytes + 255) & ~size_t(255);
    return p;
  };
  a.plan = static_cast<KvEvictPlan*>(take(sizeof(KvEvictPlan) * a.R));
  a.ticket = static_cast<int32_t*>(take(sizeof(int32_t)));
  a.list = static_cast<int32_t*>(take(sizeof(int32_t) * a.R * a.cap));
  a.list_w = static_cast<float*>(take(sizeof(float) * a.R * a.cap));
  a.read = static_cast<int32_t*>(take(sizeof(int32_t) * a.R * a.H * chunks_of(a.cap)));
  a.bounds = static_cast<int32_t*>(take(sizeof(int32_t) * a.R * (chunks_of(a.cap) + 1)));
  return off;
}

cudaError_t launch_kv_evict(const KvEvictArgs& a, cudaStream_t s) {
  const int ctas = cluster_of(a);
  const int64_t most = std::min<int64_t>((int64_t)a.max_pages << a.page_shift, a.w_cols);
  const int held = int(std::min<int64_t>(kMaxHeld, (most + 4LL * ctas * kSelThreads - 1) / (4LL * ctas * kSelThreads)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas) * unsigned(a.R));
  cfg.blockDim = kSelThreads;
  cfg.dynamicSmemBytes = size_t(held) * kSelThreads * 16 + (ctas > 1 ? kPasses * kBins * 4 : 0);
  // once per device and process (and before the first capture, or in it: this launches nothing)
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << (a.device & 63);
  if (a.device > 63 || !(ready.load(std::memory_order_relaxed) & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kv_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kMaxHeld * kSelThreads * 16 + kPasses * kBins * 4);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kv_evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_evict_select_kernel, a, uint32_t(ctas), held);
  if (e != cudaSuccess) return e;
  return a.d == 64 ? launch_move<64>(a, s) : a.d == 128 ? launch_move<128>(a, s) : launch_move<256>(a, s);
}

}  // namespace upf
