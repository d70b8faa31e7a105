// kda_pages.cu -- pages of the attention cache taken and given back on the device
// (kda_cache_reserve, kda_cache_release).
//
// Both are prefix sums over the sequences and a scatter: sequence n's pages lie in the
// free list behind those of the sequences before it.  Every CTA takes the
// sums over all sequences into its own shared memory (a few thousand lengths, from L2),
// then the CTAs share the rows (reserve) or the pages (release) and find the sequence of
// each by a binary search in shared memory.  Where lengths or the count of free pages are
// updated in place, which others still read, the CTAs are one cluster and write them after
// its barrier.  No sum depends on the order in which anything runs.  Launch latency bounds
// both; 256 rows take less than the 9 us in which the host makes the call and its results.
#include "kda_layers.cuh"

namespace kda {

namespace {

constexpr int PG_THREADS = 1024;
constexpr int PG_CTAS = 8;               // of a cluster
constexpr int PG_ROWS = 4 * PG_THREADS;  // rows of a CTA at a time

struct Sums {
  long long x, y;
};

// Inclusive sums over the CTA's threads, and the totals.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* warp_sums, Sums& total) {
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (l >= o) {
      v.x += x;
      v.y += y;
    }
  }
  if (l == 31) warp_sums[w] = v;
  __syncthreads();
  if (w == 0) {
    Sums s = warp_sums[l];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, s.x, o), y = __shfl_up_sync(0xffffffffu, s.y, o);
      if (l >= o) {
        s.x += x;
        s.y += y;
      }
    }
    warp_sums[l] = s;
  }
  __syncthreads();
  if (w > 0) {
    v.x += warp_sums[w - 1].x;
    v.y += warp_sums[w - 1].y;
  }
  total = warp_sums[31];
  __syncthreads();
  return v;
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ int clamp32(long long x, long long most) {
  return static_cast<int>(x < 0 ? 0 : (x > most ? most : x));
}

// The last n in [0, N) with first[n] <= s, for a first that does not decrease.
__device__ __forceinline__ int last_at(const int* first, int N, int s) {
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= s) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ void bad(int* err) { atomicCAS(err, 0, static_cast<int>(KDA_ERR_INVALID_ARG)); }

// Free pages: the count, or what the list has room for.
__device__ __forceinline__ int free_count_of(const PagesArgs& a, int* err) {
  const int c = *a.free_count;  // may be written at the end: not the read-only path
  if (c < 0 || c > a.pages) bad(err);
  return clamp32(c, a.pages);
}

// A sequence's rows in the table: [first, upto) are its new slots.
struct Span {
  long long first, upto;
  bool fits;  // false: refused, whatever is free
};
__device__ __forceinline__ Span span_of(const PagesArgs& a, int n, int* err) {
  const long long most = static_cast<long long>(a.width) << a.lg;
  const long long len = a.lens[n], add = a.other[n];
  if (len < 0 || len > most || add < 0) bad(err);
  const long long rows = add < 0 ? 0 : add;
  return {len, len + rows, len >= 0 && len + rows <= most};
}
__device__ __forceinline__ long long pages_of(const PagesArgs& a, long long slots) {
  return (slots + (1LL << a.lg) - 1) >> a.lg;
}

// Pages for the new rows of every sequence, in the order of the sequences: off[n] is the
// number of pages taken before sequence n, or -1 if its rows get none.
__global__ void __launch_bounds__(PG_THREADS)
reserve_kernel(PagesArgs a, bool in_place, int* err) {
  extern __shared__ int pages_smem[];
  __shared__ Sums warp_sums[32];
  __shared__ int taken;
  int* cu = pages_smem;                  // [N + 1]
  int* off = pages_smem + a.N + 1;       // [N]
  int* lens = pages_smem + 2 * a.N + 1;  // [N]
  grid_dep_wait();
  grid_dep_launch();
  const unsigned rank = blockIdx.x, ctas = gridDim.x;
  const int free_pages = free_count_of(a, err);
  if (threadIdx.x == 0) taken = 0;
  __syncthreads();
  Sums before{0, 0};  // rows and pages of the tiles before
  for (int n0 = 0; n0 < a.N; n0 += PG_THREADS) {
    const int n = n0 + threadIdx.x;
    Sums mine{0, 0};
    bool fits = true;
    int len = 0;
    if (n < a.N) {
      const Span s = span_of(a, n, err);
      fits = s.fits;
      len = static_cast<int>(s.first);
      mine.x = s.upto - s.first;
      mine.y = s.fits ? pages_of(a, s.upto) - pages_of(a, s.first) : 0;
    }
    Sums total;
    const Sums upto = block_scan(mine, warp_sums, total);
    if (n < a.N) {
      const long long rows = before.x + upto.x, pages = before.y + upto.y;
      if (rows > a.T) {  // more new rows than the call has
        bad(err);
        fits = false;
      }
      const bool granted = fits && (mine.y == 0 || pages <= free_pages);
      cu[n + 1] = clamp32(rows, a.T);
      lens[n] = len;
      off[n] = granted ? static_cast<int>(mine.y == 0 ? 0 : pages - mine.y) : -1;
      if (granted && mine.y > 0) atomicMax(&taken, static_cast<int>(pages));
    }
    before.x += total.x;
    before.y += total.y;
  }
  if (threadIdx.x == 0) cu[0] = 0;
  __syncthreads();
  // Rows: four at a time to a thread.  The row at a fresh page's first slot enters the page
  // in the table.
  const int total = cu[a.N];
  const long long page = 1LL << a.lg;
  const long long rows = a.slots ? a.T : total;
  for (long long t0 = (static_cast<long long>(rank) * PG_THREADS + threadIdx.x) * 4; t0 < rows;
       t0 += static_cast<long long>(ctas) * PG_THREADS * 4) {
    int n = t0 < total ? last_at(cu, a.N, static_cast<int>(t0)) : 0;
    long long slot[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const long long t = t0 + e;
      slot[e] = -1;
      if (t >= total) continue;
      if (t >= cu[n + 1] && t >= cu[++n + 1]) n = last_at(cu, a.N, static_cast<int>(t));  // (t < cu[N]; empty ones between)
      if (off[n] < 0) continue;
      const long long len = lens[n], p = len + (t - cu[n]);
      const long long j = p >> a.lg, had = pages_of(a, len);
      int id;
      if (j >= had) {
        id = a.free_pages[free_pages - 1 - (off[n] + (j - had))];
        if (id < 0 || id >= a.pages) id = -1;
        if ((p & (page - 1)) == 0) a.table[static_cast<long long>(n) * a.width + j] = id;
      } else {
        id = a.table[static_cast<long long>(n) * a.width + j];
      }
      if (id >= 0 && id < a.pages) slot[e] = static_cast<long long>(id) * page + (p & (page - 1));
      else bad(err);
    }
    if (a.slots) {
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        if (t0 + e + 1 < rows) *reinterpret_cast<longlong2*>(a.slots + t0 + e) = make_longlong2(slot[e], slot[e + 1]);
        else if (t0 + e < rows) a.slots[t0 + e] = slot[e];
      }
    }
  }
  if (in_place) cluster_barrier();  // every CTA has read the lengths and the count
  for (int n = rank * PG_THREADS + threadIdx.x; n < a.N; n += ctas * PG_THREADS) {
    const int len = lens[n];
    a.new_lens[n] = off[n] < 0 ? len : len + (cu[n + 1] - cu[n]);
    a.cu[n + 1] = cu[n + 1];
  }
  if (rank == 0 && threadIdx.x == 0) {
    a.cu[0] = 0;
    *a.new_free_count = free_pages - taken;
  }
}

// Pages behind the slots that sequences keep, to the end of the free list.
__global__ void __launch_bounds__(PG_THREADS)
release_kernel(PagesArgs a, bool in_place, int* err) {
  extern __shared__ int pages_smem[];
  __shared__ Sums warp_sums[32];
  int* from = pages_smem;             // [N + 1]: pages before sequence n's
  int* first = pages_smem + a.N + 1;  // [N]: its first page that goes
  grid_dep_wait();
  grid_dep_launch();
  const unsigned rank = blockIdx.x, ctas = gridDim.x;
  const int count = free_count_of(a, err);
  const int room = a.pages - count;
  long long before = 0;
  for (int n0 = 0; n0 < a.N; n0 += PG_THREADS) {
    const int n = n0 + threadIdx.x;
    Sums mine{0, 0};
    if (n < a.N) {
      const long long most = static_cast<long long>(a.width) << a.lg;
      const long long len = a.lens[n], keep = a.other ? a.other[n] : 0;
      if (len < 0 || len > most) bad(err);
      const long long had = pages_of(a, len < 0 ? 0 : (len > most ? most : len));
      const long long kept = pages_of(a, keep < 0 ? 0 : keep);
      mine.x = had > kept ? had - kept : 0;
      first[n] = static_cast<int>(had > kept ? kept : had);
    }
    Sums total;
    const Sums upto = block_scan(mine, warp_sums, total);
    if (n < a.N) from[n + 1] = clamp32(before + upto.x, room);
    before += total.x;
  }
  if (threadIdx.x == 0) from[0] = 0;
  __syncthreads();
  if (before > room) bad(err);  // more than the pool has
  const int pages = from[a.N];
  // (64 bits: the step behind the last page of the largest pool passes 32)
  for (long long i = rank * PG_THREADS + threadIdx.x; i < pages; i += ctas * PG_THREADS) {
    const int n = last_at(from, a.N, static_cast<int>(i));
    const int id = a.table[static_cast<long long>(n) * a.width + first[n] + (i - from[n])];
    const bool there = id >= 0 && id < a.pages;
    if (!there) bad(err);
    a.free_pages[count + i] = there ? id : -1;
  }
  if (in_place) cluster_barrier();
  if (rank == 0 && threadIdx.x == 0) *a.new_free_count = count + pages;
}

std::atomic<uint64_t> g_reserve_set{0}, g_release_set{0};

// Over `work` rows or pages at most, with `arrays` arrays of N in shared memory.
cudaError_t launch(void (*kernel)(PagesArgs, bool, int*), const PagesArgs& a, int64_t work, int arrays, bool in_place,
                   int* err, cudaStream_t stream, std::atomic<uint64_t>& set) {
  const cudaError_t e =
      ensure_smem_limit(reinterpret_cast<const void*>(kernel), (arrays * kPagesMaxN + 1) * 4, set);
  if (e != cudaSuccess) return e;
  const int64_t most = in_place ? PG_CTAS : 128, want = (work + PG_ROWS - 1) / PG_ROWS;
  const int ctas = want <= 1 ? 1 : in_place ? PG_CTAS : static_cast<int>(want < most ? want : most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(PG_THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(arrays * a.N + 1) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = in_place ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, in_place, err);
}

}  // namespace

cudaError_t launch_reserve(const PagesArgs& a, int* err, cudaStream_t stream) {
  const bool in_place = a.new_lens == a.lens || a.new_free_count == a.free_count;
  // without slots the rows may not be known: no more than the tables hold
  const int64_t most = (static_cast<int64_t>(a.N) * a.width) << a.lg;
  return launch(reserve_kernel, a, a.slots || a.T < most ? a.T : most, 3, in_place, err, stream, g_reserve_set);
}

cudaError_t launch_release(const PagesArgs& a, int* err, cudaStream_t stream) {
  return launch(release_kernel, a, static_cast<int64_t>(a.N) * a.width, 2, a.new_free_count == a.free_count, err,
                stream, g_release_set);
}

}  // namespace kda
