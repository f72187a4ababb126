// specv_sample.cu -- one token per row of logits under a temperature, top-k, top-p
// and min-p, drawn by inverse CDF from a given uniform; and the filtered logits.
//
// For a row z of V logits, its largest entry m and r = fl(1 / T):
//   w_v = exp(fl(fl(z_v - m) r))                     (fp32, at most 1)
//   order: z falling, index rising; entries of -inf are in no set
//   top-k  the first k entries of that order
//   top-p  the fewest first entries whose weights sum to p times the sum over top-k
//   min-p  the entries of those with w_v >= a
//   token  the first index whose running sum of kept weights, in index order, exceeds
//          u times their sum W;  ln p = fl(fl(z - m) r) - ln W
// T = 0 keeps the first entry of the order alone.
//
// Weights are added as whole numbers of 2^-44 (less for V above 2^18), so a border (a prefix
// against u W, a mass against p W) is decided on the sum of the fp32 weights and not on an
// order of addition, and sums of different passes agree.  Nothing here is fp64: its
// instructions run at 1/64 of the fp32 rate, and a dozen of them in every thread of a row
// took 6 us.
//
// One CTA per row (a warp for short rows: specv_sample_short.cu) of 256 to 1024 threads
// (row_threads).  The first pass takes the maximum, the maxima of 4096 strips
// of the row (32 vectors apart, a lane's share of some batches) and, where the row's whole
// mass is needed, its sum in fp32 about a reference that moves.  Then, by what the row asks:
//   * top-k, or top-p where few entries hold that share: the strips' maxima alone reach the
//     target at some value, so the row does; the strips above it, few, are read again, their
//     entries above it listed in shared memory, sorted, and everything is read off the list.
//     top-p takes the fp32 sum if its error bound leaves one answer.  min-p's threshold
//     follows from the maximum.  The filtered row is then -inf and the list, written without
//     reading the row again.
//   * no filter: the fp32 sums of the warps' runs tell the run that holds u W, exact sums
//     within it the token, and whether it lies closer to a border than those sums are off.
//   * anything else (a flat row under top-p, thousands of entries under top-k): a sample of
//     the row brackets the threshold; one pass sums what lies before the bracket and lists
//     what lies within (search_bracket); a bracket that misses moves, a crowded one is
//     narrowed by a histogram; rows of few levels go through histograms alone (cut_order).
//     The draw continues from the pass's sums over the warps' runs.
//
// Measured, with the filtered row written in brackets.  2048 rows of 128256 fp32 entries
// (1.05 GB, 157 us at the copy rate; 313): top-k 50 192 us (368), min-p 0.05 170 (350),
// nothing 316 to filter; bound by HBM.  Nothing 235 to 289 to sample: the second read of an
// eighth of the row, and of all of it where u W lies too close to a border to tell.  top-p
// 0.95: 300 us where every row has some likely entries, 691 where all are flat: bound by
// instructions, some forty for each entry of the pass over the whole row; one flat row of
// bf16 66.  One with top-k 50 and top-p 0.9 16 us, bound by a dozen barriers and loads that
// wait for one another.
#include "specv_internal.h"
#include "specv_rowstat.cuh"
#include "specv_sample.cuh"

namespace specv {

namespace {

constexpr int kList = 2048;   // entries of the sorted list
constexpr int kBins = 1024;
constexpr int kUnroll = 4;    // vectors in flight per thread
constexpr int kSample = 32768;  // entries of a row's sample
constexpr int kStrips = 4096;  // strips of a row, whatever the threads
constexpr float kBinsPerUnit = 32.0f;  // bins of the first histogram: m - z in steps of 1/32

// Where a running sum exceeds a value: the index, the sum before it and its own part.
struct Place {
  int index;
  uint64_t below, own;
};

// A cut of the order that is looked for in a bracket of m - z, [d_lo, d_hi).
//   top_k   the target count, or
//   share   of the sum over the entries that p keeps, the target mass: `all` is that sum,
//           `exact` or nearly
struct Search {
  bool by_mass, exact;
  uint64_t top_k;
  float share;
  uint64_t all;             // in units
  float d_lo, d_hi;
  // what a pass has found: before the bracket, within it (about, where the target lies
  // nearer), and the target
  uint64_t before, within, target;
};
enum Found { kFound, kNearer, kFarther, kCrowded };

template <int NT>
struct SampleShared {
  uint64_t part[NT / 32];
  uint64_t part2[NT / 32];
  float fpart[NT / 32], fsum[NT / 32];
  float2 scan[NT / 32];
  uint64_t key[kList];      // the list: order_key of its entries
  union {
    uint64_t upto[kList];   // running sums of their weights
    float strip[kStrips];   // before that: the strips' maxima
  };
  uint32_t count[kBins];
  uint32_t mass_lo[kBins], mass_hi[kBins];
  // for_vectors' places, four for each thread: those of 256 threads are upto's, which no
  // pass uses while it runs
  uint4 more_places[NT > 256 ? kUnroll * NT : 1];
  __device__ __forceinline__ uint4 *places() {
    static_assert(NT > 256 || sizeof(upto) >= sizeof(uint4) * kUnroll * NT);
    return NT > 256 ? more_places : reinterpret_cast<uint4 *>(upto);
  }
  int n;                    // entries in the list
  int found, last;
  uint64_t before;
  Place place;
  // What further passes share (as arguments they would lie in every thread's local memory).
  RowParams params;
  Search search;
  alignas(16) unsigned char row_bytes[64];
  template <typename T>
  __device__ __forceinline__ RowVectors<T> &row() {
    static_assert(sizeof(RowVectors<T>) <= sizeof(row_bytes));
    return *reinterpret_cast<RowVectors<T> *>(row_bytes);
  }
};
template <int NT>
__device__ __forceinline__ SampleShared<NT> &shared_of() {
  extern __shared__ __align__(16) unsigned char raw[];
  return *reinterpret_cast<SampleShared<NT> *>(raw);
}
// The row's threshold, from all threads.
template <int NT>
__device__ __forceinline__ void set_cut(SampleShared<NT> &sh, float tau, int tie) {
  __syncthreads();
  if (threadIdx.x == 0) {
    sh.params.tau = tau;
    sh.params.tie = tie;
  }
  __syncthreads();
}


// f(vector, k) for this thread's share of the vectors [lo, hi), me of STEP: four are on their
// way into the thread's own places in shared memory while one is looked at (registers for
// them would spill).  The row's edge vectors, which may have to be put together from single
// entries, come last.  LAST_FIRST: from the end.
template <typename T, int NT, int STEP, bool LAST_FIRST = false, typename F>
__device__ __forceinline__ void for_vectors(SampleShared<NT> &sh, const RowVectors<T> &row, int lo,
                                            int hi, int me, F f) {
  const int a = max(lo, row.full_lo), b = min(hi, row.full_hi);
  const int count = b - a > me ? (b - a - me + STEP - 1) / STEP : 0;
  uint4 *const place = sh.places() + threadIdx.x;
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(place);
  const int first = LAST_FIRST ? a + me + (count - 1) * STEP : a + me;
  constexpr int kStep = LAST_FIRST ? -STEP : STEP;
  const char *from = row.base + (int64_t)first * 16;
  auto fetch = [&](int i) {  // vectors i and i + 1
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (i + u < count)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                     :
                     : "r"(at + (uint32_t)((i + u) % kUnroll) * (NT * 16)),
                       "l"(from + (int64_t)(i + u) * (kStep * 16))
                     : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  static_assert(kUnroll == 4);
  fetch(0);
  fetch(2);
#pragma unroll 1
  for (int i = 0; i < count; i += 2) {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const uint4 v0 = place[(i % kUnroll) * NT], v1 = place[((i + 1) % kUnroll) * NT];
    fetch(i + 4);
    f(v0, first + i * kStep);
    if (i + 1 < count) f(v1, first + (i + 1) * kStep);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll 1
  for (int j = 0; j < 2; ++j) {
    const int k = j == 0 ? 0 : row.full_hi;
    const bool edge = j == 0 ? row.full_lo > 0 : k < row.count && k >= row.full_lo;
    if (edge && k >= lo && k < hi && me == 0) f(load_vec<T>(row, k), k);
  }
}

// What run_sums and locate add up: one(z, index) for an entry, and of a vector whose largest
// entry is below `floor` nothing.
struct EveryWeight {
  RowParams p;
  static constexpr bool kFloor = false;
  __device__ __forceinline__ uint64_t one(float z, int) const { return p.units(p.weight(z)); }
};
struct KeptWeight {
  RowParams p;
  float floor;
  static constexpr bool kFloor = true;
  __device__ __forceinline__ explicit KeptWeight(const RowParams &p_) : p(p_), floor(p_.tau) {}
  __device__ __forceinline__ uint64_t one(float z, int i) const {
    if (!p.in_order(z, i)) return 0;
    const float w = p.weight(z);
    return w >= p.min_p ? p.units(w) : 0;
  }
};
struct OrderWeight {  // whatever min-p is
  RowParams p;
  float floor;
  static constexpr bool kFloor = true;
  __device__ __forceinline__ explicit OrderWeight(const RowParams &p_) : p(p_), floor(p_.tau) {}
  __device__ __forceinline__ uint64_t one(float z, int i) const {
    return p.in_order(z, i) ? p.units(p.weight(z)) : 0;
  }
};
struct EqualEntries {
  RowParams p;
  float floor;  // the value
  static constexpr bool kFloor = true;
  __device__ __forceinline__ uint64_t one(float z, int i) const {
    return z == floor && p.in_order(z, i) ? 1 : 0;
  }
};
template <typename T, typename F>
__device__ __forceinline__ uint64_t sum_of(const F &f, const uint4 &v, int at) {
  if constexpr (F::kFloor)
    if (vector_max<T>(v) < f.floor) return 0;
  uint64_t s = 0;
#pragma unroll
  for (int e = 0; e < Elem<T>::kPerVec; ++e) s += f.one(Elem<T>::get(v, e), at + e);
  return s;
}

// Sums of f over NT / 32 equal runs of vectors [lo, hi), one per warp, in sh.part.  Every
// thread calls it; the sums are visible afterwards.
template <typename T, int NT, typename F>
__device__ __forceinline__ void run_sums(SampleShared<NT> &sh, const RowVectors<T> &row, int lo,
                                         int hi, const F &f) {
  constexpr int NW = NT / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (hi - lo + NW - 1) / NW;
  const int first = (int)min((int64_t)hi, lo + (int64_t)warp * per);
  const int end = (int)min((int64_t)hi, (int64_t)first + per);
  uint64_t s = 0;
  if constexpr (!F::kFloor) {  // every weight
    const Units units(f.p.scale);
    for_vectors<T, NT, 32>(sh, row, first, end, lane, [&](const uint4 &v, int) {
      UnitSum sum = units.begin(Elem<T>::kPerVec), a, b;
#pragma unroll
      for (int e = 0; e < Elem<T>::kPerVec; e += 2) {
        units.split(f.p.weight(Elem<T>::get(v, e)), f.p.weight(Elem<T>::get(v, e + 1)), a, b);
        Units::add(sum, a, b);
      }
      s += units.total(sum);
    });
  } else {
    for_vectors<T, NT, 32>(sh, row, first, end, lane, [&](const uint4 &v, int k) {
      s += sum_of<T>(f, v, (int)row.index(k, 0));
    });
  }
  s = warp_sum_u64(s);
  if (lane == 0) sh.part[warp] = s;
  __syncthreads();
}

template <int NT>
__device__ __forceinline__ uint64_t total_of(const SampleShared<NT> &sh) {
  uint64_t s = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) s += sh.part[w];
  return s;
}

// The first index of vectors [lo, hi) at which the running sum of f exceeds t (t below the
// sum over them).  `summed`: sh.part holds run_sums of this range.  Every thread gets it.
template <typename T, int NT, typename F>
__device__ __forceinline__ Place locate(SampleShared<NT> &sh, const RowVectors<T> &row, int lo,
                                       int hi, uint64_t t, bool summed, const F &f) {
  constexpr int VW = Elem<T>::kPerVec, NW = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t outside = 0;  // the sum before lo
  while (hi - lo > 2 * NT) {
    if (!summed) run_sums<T, NT>(sh, row, lo, hi, f);
    summed = false;
    const int per = (hi - lo + NW - 1) / NW;
    int w = 0;
    uint64_t before = 0;
    for (; w < NW - 1; ++w) {
      if (before + sh.part[w] > t) break;
      before += sh.part[w];
    }
    t -= before;
    outside += before;
    const int64_t first = lo + (int64_t)w * per;
    lo = (int)min((int64_t)hi, first);
    hi = (int)min((int64_t)hi, first + per);
    __syncthreads();
  }
  // two vectors per thread, in order
  uint4 v[2];
  uint64_t own[2] = {0, 0};
  const int k0 = lo + 2 * tid;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (k0 + j < hi) {
      v[j] = load_vec<T>(row, k0 + j);
      own[j] = sum_of<T>(f, v[j], (int)row.index(k0 + j, 0));
    }
  uint64_t upto = own[0] + own[1];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint64_t x = __shfl_up_sync(~0u, (unsigned long long)upto, off);
    if (lane >= off) upto += x;
  }
  if (lane == 31) sh.part2[warp] = upto;
  if (tid == 0) sh.place = Place{-1, 0, 0};
  __syncthreads();
  uint64_t sum = upto - own[0] - own[1];
  for (int w = 0; w < warp; ++w) sum += sh.part2[w];
  if (sum <= t && sum + own[0] + own[1] > t) {  // one thread
    const int j = sum + own[0] > t ? 0 : 1;
    if (j == 1) sum += own[0];
    const int at = (int)row.index(k0 + j, 0);
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const float z = Elem<T>::get(j == 0 ? v[0] : v[1], e);
      const uint64_t x = f.one(z, at + e);
      if (sum <= t && sum + x > t) sh.place = Place{at + e, outside + sum, x};
      sum += x;
    }
  }
  __syncthreads();
  return sh.place;
}

// Sorts key[0, n) in falling order: n <= kList different keys, room for the next power of
// two; every thread calls it.  Short lists by counting the larger keys of each, in two
// barriers; longer ones by a bitonic network.
template <int NT>
__device__ __forceinline__ void sort_keys(uint64_t *key, int n) {
  const int tid = threadIdx.x;
  if (n <= (NT < 256 ? NT : 256)) {
    const uint64_t own = tid < n ? key[tid] : 0;
    int rank = 0;
    if (tid < n)
#pragma unroll 4
      for (int i = 0; i < n; ++i) rank += key[i] > own ? 1 : 0;
    __syncthreads();
    if (tid < n) key[rank] = own;
    __syncthreads();
    return;
  }
  int size = 512;
  while (size < n) size <<= 1;
  for (int i = n + tid; i < size; i += NT) key[i] = 0;
  __syncthreads();
  for (int run = 2; run <= size; run <<= 1)
    for (int off = run >> 1; off > 0; off >>= 1) {
      for (int p = tid; p < size / 2; p += NT) {
        const int i = 2 * p - (p & (off - 1)), j = i + off;  // the lower of the p-th pair
        const uint64_t a = key[i], b = key[j];
        const bool falling = run == size || (i & run) == 0;
        if ((a < b) == falling) {
          key[i] = b;
          key[j] = a;
        }
      }
      __syncthreads();
    }
}

// Running sums of value(i), i in [0, n), in sh.upto.
template <int NT, typename F>
__device__ __forceinline__ void scan_list(SampleShared<NT> &sh, int n, F value) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t base = 0;
  for (int at = 0; at < n; at += NT) {
    const int i = at + tid;
    uint64_t x = i < n ? value(i) : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint64_t y = __shfl_up_sync(~0u, (unsigned long long)x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) sh.part2[warp] = x;
    __syncthreads();
    uint64_t all = 0;
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) x += sh.part2[w];
      all += sh.part2[w];
    }
    if (i < n) sh.upto[i] = base + x;
    base += all;
    __syncthreads();
  }
}

// The first i in [0, n) with sh.upto[i] >= target, n if there is none.
template <int NT>
__device__ __forceinline__ int first_reaching(const SampleShared<NT> &sh, int n, uint64_t target) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sh.upto[mid] >= target) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// The first bin of sh's histogram at which `base` plus the running sum of the counts (or
// of the masses) reaches `target`: sh.found (kBins: none) and in sh.before what lies
// before it, base included.
template <int NT>
__device__ __forceinline__ void find_bin(SampleShared<NT> &sh, uint64_t base, uint64_t target,
                                         bool by_mass) {
  constexpr int kEach = kBins / NT > 0 ? kBins / NT : 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto value = [&](int b) -> uint64_t {
    return by_mass ? ((uint64_t)sh.mass_hi[b] << 32) + sh.mass_lo[b] : sh.count[b];
  };
  if (tid == 0) sh.found = kBins;
  uint64_t own = 0;
  for (int j = 0; j < kEach; ++j) own += value(tid * kEach + j);
  uint64_t upto = own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint64_t y = __shfl_up_sync(~0u, (unsigned long long)upto, off);
    if (lane >= off) upto += y;
  }
  if (lane == 31) sh.part2[warp] = upto;
  __syncthreads();
  uint64_t at = base + upto - own;
  for (int w = 0; w < warp; ++w) at += sh.part2[w];
  if (at < target && at + own >= target) {  // one thread at most
    int b = tid * kEach;
    // (not past the thread's own bins, whatever the sums are)
    while ((b + 1) % kEach != 0 && at + value(b) < target) at += value(b++);
    sh.found = b;
    sh.before = at;
  }
  __syncthreads();
}

template <int NT>
__device__ __forceinline__ void add_mass(SampleShared<NT> &sh, int b, uint64_t x) {
  const uint32_t lo = (uint32_t)x, old = atomicAdd(&sh.mass_lo[b], lo);
  const uint32_t hi = (uint32_t)(x >> 32) + (old + lo < old ? 1u : 0u);
  if (hi != 0) atomicAdd(&sh.mass_hi[b], hi);
}

// Histogram of the entries in order (those that p keeps) with bin(z) in [0, kBins).
template <typename T, int NT, typename F>
__device__ __forceinline__ void histogram(SampleShared<NT> &sh, const RowVectors<T> &row,
                                          const RowParams &p, bool by_mass, F bin) {
  constexpr int VW = Elem<T>::kPerVec;
  for (int b = threadIdx.x; b < kBins; b += NT) sh.count[b] = sh.mass_lo[b] = sh.mass_hi[b] = 0;
  __syncthreads();
  for_vectors<T, NT, NT>(sh, row, 0, row.count, threadIdx.x, [&](const uint4 &v, int k) {
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const float z = Elem<T>::get(v, e);
      const int b = bin(z);
      if (b < 0 || b >= kBins || !p.in_order(z, (int)row.index(k, e))) continue;
      atomicAdd(&sh.count[b], 1u);
      if (by_mass) add_mass(sh, b, p.units(p.weight(z)));
    }
  });
  __syncthreads();
}

// Puts the entries in order whose value key lies in [lo, hi] into the list (in any order;
// there are at most kList).  Returns how many.
template <typename T, int NT>
__device__ __forceinline__ int gather(SampleShared<NT> &sh, const RowVectors<T> &row,
                                      const RowParams &p, uint32_t lo, uint32_t hi) {
  constexpr int VW = Elem<T>::kPerVec;
  if (threadIdx.x == 0) sh.n = 0;
  __syncthreads();
  for_vectors<T, NT, NT>(sh, row, 0, row.count, threadIdx.x, [&](const uint4 &v, int k) {
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const float z = Elem<T>::get(v, e);
      const int i = (int)row.index(k, e);
      const uint32_t key = value_key(z);
      if (z > -INFINITY && key >= lo && key <= hi && p.in_order(z, i)) {
        const int at = atomicAdd(&sh.n, 1);
        if (at < kList) sh.key[at] = order_key(z, (uint32_t)i);
      }
    }
  });
  __syncthreads();
  return min(sh.n, kList);
}

// The keys [lo, hi] of the values that the first histogram puts into bin b: m - z is
// monotone in z, and so is the bin.
__device__ __forceinline__ int linear_bin(float m, float z) {
  return (int)fminf(__fmul_rn(__fsub_rn(m, z), kBinsPerUnit), (float)(kBins - 1));
}
__device__ __forceinline__ uint32_t lowest_key_of_bin(float m, int b) {
  if (b >= kBins - 1) return value_key(-3.402823466e38f);
  uint32_t lo = value_key(-3.402823466e38f), hi = value_key(m);  // bin(hi) = 0 <= b
  while (lo < hi) {  // the lowest key whose bin is b or a nearer one
    const uint32_t mid = lo + (hi - lo) / 2;
    if (linear_bin(m, value_of(mid)) <= b) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// ------------------------------------------------------------------ the first pass
// How the row's vectors are dealt: warp w takes run w of `per` vectors, in batches of
// 32 kUnroll; a lane's vectors of `seg_batches` batches are a strip.
template <int NT>
struct Deal {
  static constexpr int kBatch = 32 * kUnroll;
  int per, seg_batches, segs;
  __device__ __forceinline__ explicit Deal(int count) {
    per = (count + NT / 32 - 1) / (NT / 32);
    const int batches = (per + kBatch - 1) / kBatch;
    seg_batches = (batches + kStrips / NT - 1) / (kStrips / NT);
    segs = (batches + seg_batches - 1) / seg_batches;
  }
  __device__ __forceinline__ int lo(int warp, int count) const {
    return (int)min((int64_t)count, (int64_t)warp * per);
  }
};

// One pass over the thread's vectors: the strips' maxima in sh.strip, the thread's
// maximum (NaN if it met one) in m, and with SUMS the sum of e^{(z - ref) r} in s about a
// reference that moves when the maximum has risen by more than 8 T.  What a strip adds is
// summed by itself first: a sum is off by the strip's terms and the strips, not by all
// terms.
template <typename T, int NT, bool SUMS>
__device__ __forceinline__ void first_pass(SampleShared<NT> &sh, const RowVectors<T> &row,
                                           const Deal<NT> &deal, float r, float &m, float &ref,
                                           float &s) {
  constexpr int kBatch = Deal<NT>::kBatch;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lo = deal.lo(warp, row.count), hi = deal.lo(warp + 1, row.count);
  constexpr uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
  const int plain_hi = min(hi, row.full_hi);
  auto load_batch = [&](int base, uint4 (&v)[kUnroll]) {
    if (base >= row.full_lo && base <= plain_hi - kBatch) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        v[u] = load16(row.base + (int64_t)(base + u * 32 + lane) * 16);
    } else {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int k = base + u * 32 + lane;
        v[u] = make_uint4(none, none, none, none);
        if (k >= row.full_lo && k < plain_hi) v[u] = load16(row.base + (int64_t)k * 16);
      }
    }
  };
  m = -INFINITY;
  ref = -3.402823466e38f;
  s = 0.0f;
  const float rl2 = __fmul_rn(r, kLog2e);
  const uint64_t scale = pack2(rl2, rl2);
  // The reference moves so that the exponents of entries up to `top` stay small.
  auto move_to = [&](float top, uint64_t &part) {
    if (__fmul_rn(__fsub_rn(top, ref), r) > 8.0f) {
      const float f = ex2(fmaxf(__fmul_rn(__fsub_rn(ref, top), rl2), kFarBelow));
      part = mul2(part, pack2(f, f));
      s = __fmul_rn(s, f);
      ref = top;
    }
  };
  auto add_vector = [&](const uint4 &v, uint64_t neg, uint64_t &part) {
#pragma unroll
    for (int i = 0; i < Elem<T>::kPerVec / 2; ++i) {
      float x0, x1;
      unpack2(mul2(add2(pair_of<T>(v, i), neg), scale), x0, x1);
      part = add2(part, pack2(ex2(x0), ex2(x1)));
    }
  };
  auto add_part = [&](uint64_t part) {
    float a, b;
    unpack2(part, a, b);
    s = __fadd_rn(s, __fadd_rn(a, b));
  };
  uint4 cur[kUnroll], next[kUnroll];
  load_batch(lo, cur);
  int base = lo;
  for (int g = 0; g < deal.segs; ++g) {
    float top = -INFINITY;
    uint64_t part = 0;
    for (int b = 0; b < deal.seg_batches && base < hi; ++b, base += kBatch) {
      if (base < hi - kBatch) load_batch(base + kBatch, next);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) top = max_nan(top, vector_max_nan<T>(cur[u]));
      if (SUMS) {
        move_to(top, part);
        const uint64_t neg = pack2(-ref, -ref);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) add_vector(cur[u], neg, part);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) cur[u] = next[u];
    }
    sh.strip[g * NT + tid] = top;
    m = max_nan(m, top);
    if (SUMS) add_part(part);
  }
  // The row's edge vectors, entry by entry, by the lanes that they are dealt to: after the
  // others, when no loads are in flight that a call would have to save (amid them, one
  // request's row 18.7 us against 16.6, 2304 rows under top-k and top-p 398 against 390).
#pragma unroll 1
  for (int j = 0; j < 2; ++j) {
    const int k = j == 0 ? 0 : row.full_hi;
    const bool edge = j == 0 ? row.full_lo > 0 : k < row.count && k >= row.full_lo;
    if (!edge || k < lo || k >= hi || ((k - lo) & 31) != lane) continue;
    const uint4 v = load_entries<T>(row.row, row.index(k, 0), row.V);
    const float top = vector_max_nan<T>(v);
    float &strip = sh.strip[(k - lo) / (kBatch * deal.seg_batches) * NT + tid];
    strip = max_nan(strip, top);
    m = max_nan(m, top);
    if (SUMS) {
      uint64_t part = 0;
      move_to(top, part);
      add_vector(v, pack2(-ref, -ref), part);
      add_part(part);
    }
  }
}

// The list of all entries z with fl(m - z) < limit, by the strips whose maximum is one of
// them.  Returns how many there are, more than kList if they do not fit.
template <typename T, int NT>
__device__ __forceinline__ int gather_strips(SampleShared<NT> &sh, const RowVectors<T> &row,
                                             const Deal<NT> &deal, float m, float limit) {
  constexpr int VW = Elem<T>::kPerVec;
  const int tid = threadIdx.x;
  uint32_t *ids = sh.mass_lo;  // (the masses have been read)
  if (tid == 0) sh.n = sh.found = 0;
  __syncthreads();
  for (int g = 0; g < deal.segs; ++g)
    if (__fsub_rn(m, sh.strip[g * NT + tid]) < limit) {
      const int at = atomicAdd(&sh.found, 1);
      if (at < kBins) ids[at] = g * NT + tid;
    }
  __syncthreads();
  const int strips = sh.found;
  if (strips > kBins) return kList + 1;
  const int each = deal.seg_batches * kUnroll;  // vectors of a strip
  for (int64_t i = tid; i < (int64_t)strips * each; i += NT) {
    const int at = (int)(i / each), of = (int)(i - (int64_t)at * each);
    const int id = ids[at], g = id / NT, t = id % NT, w = t >> 5;
    const int64_t k = (int64_t)deal.lo(w, row.count) +
                      ((int64_t)g * deal.seg_batches * kUnroll + of) * 32 + (t & 31);
    if (k >= deal.lo(w + 1, row.count)) continue;
    const uint4 v = load_vec<T>(row, (int)k);
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const float z = Elem<T>::get(v, e);
      if (__fsub_rn(m, z) < limit) {
        const int slot = atomicAdd(&sh.n, 1);
        if (slot < kList) sh.key[slot] = order_key(z, (uint32_t)row.index((int)k, e));
      }
    }
  }
  __syncthreads();
  return sh.n;
}

// Cuts the order where the count (by_mass: the mass) of the entries that p keeps reaches
// `target`: sets the params' tau and tie to the last entry within.
template <typename T, int NT>
__device__ __noinline__ void cut_order(uint64_t target, bool by_mass) {
  SampleShared<NT> &sh = shared_of<NT>();
  const RowVectors<T> row = sh.template row<T>();
  const RowParams p = sh.params;
  const float m = p.m;
  histogram<T, NT>(sh, row, p, by_mass, [&](float z) {
    return z > -INFINITY ? linear_bin(m, z) : -1;
  });
  find_bin(sh, 0, target, by_mass);
  const int b = sh.found;
  if (b >= kBins) return;  // never: nothing is cut off
  uint64_t before = sh.before;
  uint32_t in_bin = sh.count[b], hi = value_key(m), lo = lowest_key_of_bin(m, b);
  if (b > 0) hi = lowest_key_of_bin(m, b - 1) - 1;
  __syncthreads();
  while (in_bin > kList && lo < hi) {
    int shift = 0;
    while ((hi - lo) >> shift >= (uint32_t)kBins) ++shift;
    histogram<T, NT>(sh, row, p, by_mass, [&](float z) {
      const uint32_t key = value_key(z);
      return z > -INFINITY && key >= lo && key <= hi ? (int)((hi - key) >> shift) : -1;
    });
    find_bin(sh, before, target, by_mass);
    const uint32_t c = min(sh.found, kBins - 1);
    before = sh.before;
    in_bin = sh.count[c];
    const uint32_t top = hi - (c << shift), width = (1u << shift) - 1;
    lo = top - lo > width ? top - width : lo;
    hi = top;
    __syncthreads();
  }
  if (in_bin > kList) {
    // one value that fills more than the list: the n-th of its entries in index order
    const float tau = value_of(lo);
    uint64_t each = 1;
    if (by_mass) each = p.units(p.weight(tau));
    // (a mass of 0 each reaches nothing: the bin would not have been found)
    const uint64_t n = each != 0 ? (target - before + each - 1) / each : 1;
    set_cut(sh, tau,
            locate<T, NT>(sh, row, 0, row.count, n - 1, false, EqualEntries{p, tau}).index);
    return;
  }
  const int n = gather<T, NT>(sh, row, p, lo, hi);
  sort_keys<NT>(sh.key, n);
  int64_t at;
  if (by_mass) {
    scan_list<NT>(sh, n, [&](int i) { return p.units(p.weight(key_value(sh.key[i]))); });
    at = first_reaching(sh, n, target - before);
  } else {
    at = (int64_t)(target - before) - 1;
  }
  // (within the list whatever happens: a caller may write the row meanwhile)
  at = max((int64_t)0, min(at, (int64_t)n - 1));
  const uint64_t edge = sh.key[at];
  set_cut(sh, key_value(edge), (int)key_index(edge));
}

// One pass over the row sums exactly what lies before the bracket, run by run, and lists what
// lies within.  kFound: p is cut, and the runs' sums over the entries in order are in
// sh.part.  Else the target lies nearer to the maximum than the bracket or farther from it,
// or more entries than the list holds lie within.
template <typename T, int NT>
__device__ __noinline__ Found search_bracket() {
  SampleShared<NT> &sh = shared_of<NT>();
  const RowVectors<T> row = sh.template row<T>();
  const RowParams p = sh.params;
  const Search q = sh.search;
  constexpr int VW = Elem<T>::kPerVec, NW = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float m = p.m, d_lo = q.d_lo, d_hi = q.d_hi;
  const bool cut = p.cut(), by_mass = q.by_mass;
  const int per = (row.count + NW - 1) / NW;
  const int begin = (int)min((int64_t)row.count, (int64_t)warp * per);
  const int end = (int)min((int64_t)row.count, (int64_t)begin + per);
  if (tid == 0) sh.n = sh.last = 0;
  for (int b = tid; b < kBins; b += NT) sh.count[b] = sh.mass_lo[b] = sh.mass_hi[b] = 0;
  __syncthreads();
  auto list = [&](float z, int i) {
    const int slot = atomicAdd(&sh.n, 1);
    if (slot < kList) sh.key[slot] = order_key(z, (uint32_t)i);
  };
  uint64_t above = 0, mass = 0, whole = 0;  // before the bracket: entries, weights; all weights
  if (by_mass && !q.exact) {
    const Units units(p.scale);  // (nothing is cut yet)
    for_vectors<T, NT, 32>(sh, row, begin, end, lane, [&](const uint4 &v, int k) {
      bool some = false;
      UnitSum all = units.begin(VW), near = units.begin(VW), a, b;
#pragma unroll
      for (int e = 0; e < VW; e += 2) {
        const float z0 = Elem<T>::get(v, e), z1 = Elem<T>::get(v, e + 1);
        const float d0 = __fsub_rn(m, z0), d1 = __fsub_rn(m, z1);
        units.split(p.weight(z0), p.weight(z1), a, b);
        Units::add(all, a, b);
        Units::add(near, d0 < d_lo ? a : units.none(), d1 < d_lo ? b : units.none());
        some |= (d0 >= d_lo && d0 < d_hi) || (d1 >= d_lo && d1 < d_hi);
      }
      if (some) {
        const int at = (int)row.index(k, 0);
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          const float z = Elem<T>::get(v, e), d = __fsub_rn(m, z);
          if (d >= d_lo && d < d_hi) list(z, at + e);
        }
      }
      whole += units.total(all);
      mass += units.total(near);
    });
  } else {
    for_vectors<T, NT, 32>(sh, row, begin, end, lane, [&](const uint4 &v, int k) {
      if (!(__fsub_rn(m, vector_max<T>(v)) < d_hi)) return;
      const int at = (int)row.index(k, 0);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        const float z = Elem<T>::get(v, e), d = __fsub_rn(m, z);
        if (!(d < d_hi) || (cut && !p.in_order(z, at + e))) continue;
        if (d < d_lo) {
          ++above;
          mass += p.units(p.weight(z));
        } else {
          list(z, at + e);
        }
      }
    });
    above = warp_sum_u64(above);
  }
  mass = warp_sum_u64(mass);
  whole = warp_sum_u64(whole);
  if (lane == 0) {
    sh.part[warp] = mass;
    sh.part2[warp] = by_mass ? whole : above;
  }
  __syncthreads();
  const int n = sh.n;
  uint64_t before = 0;  // the bracket, in what is counted
#pragma unroll 8
  for (int w = 0; w < NW; ++w) before += sh.part2[w];
  uint64_t target = q.top_k;
  if (by_mass) {
    target = share_of(q.share, q.exact ? q.all : before);
    before = total_of(sh);
  }
  if (tid == 0) {
    sh.search.before = before;
    sh.search.target = target;
    const float each =  // of the bracket's middle
        by_mass ? ex2(__fmul_rn(-0.5f * (d_lo + d_hi), __fmul_rn(p.r, kLog2e))) * p.scale : 1.0f;
    sh.search.within = __float2ull_rn(fminf((float)n * each, 4e18f));
  }
  if (before >= target) return kNearer;
  if (n > kList) return kCrowded;
  // the bracket in finer bins; the entries of the bin that holds the target are sorted
  const float fine = __fdiv_rn((float)kBins, __fsub_rn(d_hi, d_lo));
  auto fine_bin = [&](uint64_t key) {
    return (int)fminf(__fmul_rn(__fsub_rn(__fsub_rn(m, key_value(key)), d_lo), fine),
                      (float)(kBins - 1));
  };
  for (int i = tid; i < n; i += NT) {
    const uint64_t key = sh.key[i];
    const int b = fine_bin(key);
    atomicAdd(&sh.count[b], 1u);
    if (by_mass) add_mass(sh, b, p.units(p.weight(key_value(key))));
  }
  __syncthreads();
  find_bin(sh, before, target, by_mass);
  const int b = sh.found;
  if (b >= kBins) {
    uint64_t within = 0;  // (find_bin's sums)
#pragma unroll 8
    for (int w = 0; w < NW; ++w) within += sh.part2[w];
    if (tid == 0) sh.search.within = within;
    return kFarther;
  }
  const uint64_t start = sh.before;
  const int few = sh.count[b];
  for (int i = tid; i < n; i += NT)
    if (fine_bin(sh.key[i]) == b) sh.upto[min(atomicAdd(&sh.last, 1), kList - 1)] = sh.key[i];
  __syncthreads();
  uint64_t edge = 0;  // the key of the last entry kept
  if (few <= 32) {
    const uint64_t key = warp_sort(lane < few ? sh.upto[lane] : 0);  // (every warp the same)
    uint64_t x = lane >= few ? 0 : by_mass ? p.units(p.weight(key_value(key))) : 1;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint64_t y = __shfl_up_sync(~0u, (unsigned long long)x, off);
      if (lane >= off) x += y;
    }
    const uint32_t there = __ballot_sync(~0u, lane < few && start + x >= target);
    edge = __shfl_sync(~0u, (unsigned long long)key, there != 0 ? __ffs(there) - 1 : 0);
  } else {
    sort_keys<NT>(sh.upto, few);
    uint64_t base = start;
    for (int at = 0; at < few; at += NT) {
      const int i = at + tid;
      const uint64_t own = i >= few ? 0 : by_mass ? p.units(p.weight(key_value(sh.upto[i]))) : 1;
      uint64_t x = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint64_t y = __shfl_up_sync(~0u, (unsigned long long)x, off);
        if (lane >= off) x += y;
      }
      __syncthreads();
      if (lane == 31) sh.part2[warp] = x;
      __syncthreads();
      x += base;
      for (int w = 0; w < NW; ++w) {
        if (w < warp) x += sh.part2[w];
        base += sh.part2[w];
      }
      if (x - own < target && x >= target) sh.before = sh.upto[i];
    }
    __syncthreads();
    edge = sh.before;
  }
  set_cut(sh, key_value(edge), (int)key_index(edge));
  // the entries of the list that are in order join their runs
  if (tid < NW) sh.mass_lo[tid] = sh.mass_hi[tid] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += NT) {
    const uint64_t key = sh.key[i];
    if (key < edge) continue;
    const int k = (int)(((int64_t)key_index(key) + row.mis) / VW);
    add_mass(sh, min(k / per, NW - 1), p.units(p.weight(key_value(key))));
  }
  __syncthreads();
  if (tid < NW) sh.part[tid] += ((uint64_t)sh.mass_hi[tid] << 32) + sh.mass_lo[tid];
  __syncthreads();
  return kFound;
}

// A crowded bracket: a histogram of it narrows it to about a three hundredth.  Returns whether
// that holds the target and got narrower.
template <typename T, int NT>
__device__ __noinline__ bool narrow_bracket() {
  SampleShared<NT> &sh = shared_of<NT>();
  const RowVectors<T> row = sh.template row<T>();
  const RowParams p = sh.params;
  const Search q = sh.search;
  const float m = p.m, d_lo = q.d_lo, d_hi = q.d_hi;
  if (!(d_hi < INFINITY)) return false;
  const float fine = __fdiv_rn((float)kBins, __fsub_rn(d_hi, d_lo));
  histogram<T, NT>(sh, row, p, q.by_mass, [&](float z) {
    const float d = __fsub_rn(m, z);
    return d >= d_lo && d < d_hi
               ? (int)fminf(__fmul_rn(__fsub_rn(d, d_lo), fine), (float)(kBins - 1))
               : -1;
  });
  find_bin(sh, q.before, q.target, q.by_mass);
  const int b = sh.found;
  __syncthreads();
  if (b >= kBins || sh.count[b] > kList / 4) return false;
  // a bin more on either side, for the edges' roundings
  const float step = __fdiv_rn(__fsub_rn(d_hi, d_lo), (float)kBins);
  const float lo = fmaxf(d_lo, __fmaf_rn((float)(b - 1), step, d_lo));
  const float hi = fminf(d_hi, __fmaf_rn((float)(b + 2), step, d_lo));
  if (threadIdx.x == 0) {
    sh.search.d_lo = lo;
    sh.search.d_hi = hi;
  }
  return lo < hi;
}

// A cut that a sample points to.  A line of 32 vectors in every `every` is counted into the
// bins of m - z, and the bins are bracketed in which the target can lie: for a count by the
// sample's own counts, two standard deviations either way; for a mass by what lies beyond a
// bin, estimated from the sample as well, against the part of the whole that may (the
// sample's many light entries say that well, its few heavy ones would not say the rest),
// 2.4 deviations either way, to a part of a bin.  Half the entries sampled and
// 1.7 deviations: 64 flat rows of 128256 under top-p 0.95 66 us against 68 in fp32, 82 against 68
// in bf16 (a miss costs a pass, and the slowest row decides); 2048 such rows 646 against 692.
// Where a pass does not find the target in the bracket it says where to go on.  Returns
// whether it was found (else nothing is set).  `limit`: the first top_k entries have m - z
// below it.
template <typename T, int NT>
__device__ __noinline__ bool cut_sampled(float limit) {
  SampleShared<NT> &sh = shared_of<NT>();
  const RowVectors<T> row = sh.template row<T>();
  const RowParams p = sh.params;
  const Search q = sh.search;
  constexpr int VW = Elem<T>::kPerVec, NW = NT / 32;
  constexpr int kEach = kBins / NT > 0 ? kBins / NT : 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float m = p.m, rl2 = __fmul_rn(p.r, kLog2e);
  const bool cut = p.cut(), by_mass = q.by_mass;
  const int lines = (row.count + 31) / 32;
  const int every = max(1, (int)((int64_t)lines * (32 * VW) / kSample));
  const float rest = by_mass ? (1.0f - q.share) * ((float)q.all / p.scale) : 0.0f;
  // Beyond this an entry is not counted: of a count it cannot be; of a mass the sample's
  // weights are added up, together a quarter of the rest at most.
  const float far =
      by_mass ? __fdiv_rn(-logf(fmaxf(rest / (4.0f * row.V), 1e-30f)), p.r) : limit;
  for (int b = tid; b < kBins; b += NT) sh.count[b] = 0;
  if (tid == 0) {
    sh.found = by_mass ? -1 : kBins;
    sh.last = by_mass ? -1 : 0;
    sh.n = 0;
  }
  __syncthreads();
  float tail = 0.0f;
  for (int64_t line = (int64_t)warp * every; line < lines; line += (int64_t)NW * every * kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t k = (line + (int64_t)u * NW * every) * 32 + lane;
      constexpr uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
      v[u] = make_uint4(none, none, none, none);
      if (k < row.count) v[u] = load_vec<T>(row, (int)k);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int at = (int)row.index((int)((line + (int64_t)u * NW * every) * 32 + lane), 0);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        const float z = Elem<T>::get(v[u], e), d = __fsub_rn(m, z);
        if (!(z > -INFINITY) || (cut && !p.in_order(z, at + e))) continue;
        // (above m only where a caller writes the row meanwhile: it may come out wrong, but
        // nothing is counted outside the histogram)
        if (d >= 0.0f && d < far)
          atomicAdd(&sh.count[linear_bin(m, z)], 1u);
        else if (by_mass)
          tail += ex2(__fmul_rn(-d, rl2));
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) tail += __shfl_xor_sync(~0u, tail, off);
  if (lane == 0) sh.fpart[warp] = tail;
  __syncthreads();
  // the bracket: bins [sh.found, sh.last]
  const float factor = (float)every;
  if (by_mass) {
    // from the last bin: every thread takes some bins, the lower ones those farther out
    float mass = 0.0f, square = 0.0f;
    auto weight = [&](int b) {  // in the middle of the bin
      return ex2(__fmul_rn(-((float)b + 0.5f) * (1.0f / kBinsPerUnit), rl2));
    };
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int b = kBins - 1 - (tid * kEach + j);
      const float w = weight(b), x = w * (float)sh.count[b];
      mass += x;
      square += x * w;
    }
    float upto = mass, upto2 = square;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const float x = __shfl_up_sync(~0u, upto, off), y = __shfl_up_sync(~0u, upto2, off);
      if (lane >= off) upto += x, upto2 += y;
    }
    if (lane == 31) sh.scan[warp] = make_float2(upto, upto2);
    __syncthreads();
    float beyond = upto - mass, beyond2 = fmaxf(upto2 - square, 0.0f);
    for (int w = 0; w < NW; ++w) {
      beyond += sh.fpart[w];
      if (w < warp) beyond += sh.scan[w].x, beyond2 += sh.scan[w].y;
    }
    // From the far end, the first bin with which the sum surely reaches the rest (a heavy entry
    // nearer by makes the sum less sure, but not less), and the first with which it may.
    int lo = -1, hi = -1;
    float in_lo = 1.0f, in_hi = 0.0f;  // which part of the bin, from its far end
    const float want = rest / factor;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int b = kBins - 1 - (tid * kEach + j);
      const float w = weight(b), x = w * (float)sh.count[b];
      beyond += x;
      beyond2 += x * w;
      const float slack = 2.4f * sqrtf(beyond2) + 0.002f * beyond;
      const float less = beyond - slack, more = beyond + slack;
      if (lo < 0 && less >= want) {
        lo = b;
        in_lo = less - want < x ? 1.0f - (less - want) / x : 0.0f;
      }
      if (hi < 0 && more >= want) {
        hi = b;
        in_hi = more - want < x ? 1.0f - (more - want) / x : 0.0f;
      }
    }
    if (lo >= 0) atomicMax(&sh.found, lo);
    if (hi >= 0) atomicMax(&sh.last, hi);
    __syncthreads();
    if (lo >= 0 && lo == sh.found)
      sh.search.d_lo = ((float)(lo + 1) - in_lo) * (1.0f / kBinsPerUnit);
    if (hi >= 0 && hi == sh.last)
      sh.search.d_hi = ((float)(hi + 1) - in_hi) * (1.0f / kBinsPerUnit);
  } else {
    uint32_t own = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) own += sh.count[tid * kEach + j];
    uint32_t upto = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t x = __shfl_up_sync(~0u, upto, off);
      if (lane >= off) upto += x;
    }
    if (lane == 31) sh.part2[warp] = upto;
    __syncthreads();
    upto -= own;
    for (int w = 0; w < warp; ++w) upto += (uint32_t)sh.part2[w];
    float before = (float)upto;
    const float want = (float)q.top_k / factor;
    int lo = kBins, hi = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int b = tid * kEach + j;
      before += (float)sh.count[b];
      const float slack = every > 1 ? 2.0f * sqrtf(before) + 2.0f : 0.0f;
      if (lo == kBins && before + slack >= want) lo = b;
      if (before - slack < want) hi = b + 1;  // after the last that surely lies before it
    }
    if (lo < kBins) atomicMin(&sh.found, lo);
    atomicMax(&sh.last, min(hi, kBins - 1));
  }
  __syncthreads();
  const int lo = max(0, sh.found), hi = sh.last;
  float d_lo = !by_mass         ? (float)lo * (1.0f / kBinsPerUnit)
               : sh.found < 0 ? 0.0f
                              : sh.search.d_lo;
  float d_hi = hi >= kBins - 1 ? INFINITY
               : by_mass       ? sh.search.d_hi
                               : fminf((float)(hi + 1) * (1.0f / kBinsPerUnit), limit);
  if constexpr (NT == 1024) {  // the sampled entries of the bracket
    static_assert(kBins == NT);
    if (tid >= lo && tid <= hi && sh.count[tid] > 0) atomicAdd(&sh.n, (int)sh.count[tid]);
  }
  __syncthreads();
  if (lo >= kBins || hi < lo || !(d_lo < d_hi)) return false;
  // A miss costs another pass over the row.  Where rows are few, the slowest decides, and the
  // bracket is made wider as long as its entries fit into the list twice and more.
  if constexpr (NT == 1024) {
    const float room = __fdiv_rn(0.8f * kList * (float)(hi - lo + 1),
                                 fmaxf(factor * (float)sh.n * kBinsPerUnit * (d_hi - d_lo), 1.0f));
    if (room > 2.0f) {
      const float more = fminf(0.5f * (fminf(0.5f * room, 2.0f) - 1.0f) * (d_hi - d_lo),
                               8.0f / kBinsPerUnit);
      d_lo = fmaxf(0.0f, d_lo - more);
      d_hi += more;
    }
  }
  for (int tries = 0; tries < 6; ++tries) {
    if (tid == 0) {
      sh.search.d_lo = d_lo;
      sh.search.d_hi = d_hi;
    }
    __syncthreads();
    const Found found = search_bracket<T, NT>();
    if (found == kFound) return true;
    __syncthreads();
    // as wide as what is missing asks for at the bracket's density
    const Search at = sh.search;
    const uint64_t reached = found == kNearer ? at.before : at.before + at.within;
    const float missing = (float)(found == kNearer ? at.before - at.target : at.target - reached);
    const float ratio = at.within > 0 ? fminf(missing / (float)at.within, 8.0f) : 8.0f;
    const float wide = fmaxf((d_hi - d_lo) * (1.4f * ratio + 0.1f), 0.25f / kBinsPerUnit);
    if (found == kCrowded) {
      if (!narrow_bracket<T, NT>()) return false;
      __syncthreads();
      d_lo = sh.search.d_lo;
      d_hi = sh.search.d_hi;
    } else if (found == kNearer) {
      if (d_lo <= 0.0f) return false;
      d_hi = d_lo;
      d_lo = wide < INFINITY ? fmaxf(0.0f, d_lo - wide) : 0.0f;
    } else {
      if (!(d_hi < INFINITY)) return false;
      d_lo = d_hi;
      d_hi += wide;
    }
    __syncthreads();
  }
  return false;
}

// The thresholds of top-k and top-p on any row, in passes over it.  `limit`: the first top_k
// entries have m - z below it (or +inf); `about`: the sum of all weights, where top-p stands
// alone.  Returns whether sh.part holds the runs' sums over the entries in order.
template <typename T, int NT>
__device__ __noinline__ bool cut_all(bool by_k, int top_k, float limit, bool by_p, float top_p,
                                     float about) {
  SampleShared<NT> &sh = shared_of<NT>();
  const RowVectors<T> &row = sh.template row<T>();
  if (by_k) {
    if (threadIdx.x == 0) sh.search = Search{false, true, (uint64_t)top_k, 0.0f, 0, 0.0f, 0.0f, 0, 0, 0};
    __syncthreads();
    const bool summed = cut_sampled<T, NT>(limit);
    __syncthreads();
    if (!summed) cut_order<T, NT>((uint64_t)top_k, false);
    if (!by_p) return summed;
    if (!summed) run_sums<T, NT>(sh, row, 0, row.count, OrderWeight(sh.params));
  }
  const uint64_t all = by_k ? total_of(sh) : __float2ull_rn(about * sh.params.scale);
  if (threadIdx.x == 0) sh.search = Search{true, by_k, 0, top_p, all, 0.0f, 0.0f, 0, 0, 0};
  __syncthreads();
  if (cut_sampled<T, NT>(INFINITY)) return true;
  __syncthreads();
  run_sums<T, NT>(sh, row, 0, row.count, OrderWeight(sh.params));
  const uint64_t exact = total_of(sh);
  __syncthreads();
  cut_order<T, NT>(share_of(top_p, exact), true);
  return false;
}

// The draw from the kept entries of any row: where it is, and in sh.before the kept sum.
// `summed`: sh.part holds the runs' sums.
template <typename T, int NT>
__device__ __noinline__ int draw_all(float u, bool summed) {
  SampleShared<NT> &sh = shared_of<NT>();
  const RowVectors<T> row = sh.template row<T>();
  const RowParams p = sh.params;
  auto draw = [&](const auto &kept) {
    if (!summed) run_sums<T, NT>(sh, row, 0, row.count, kept);
    const uint64_t all = total_of(sh);
    if (threadIdx.x == 0) sh.before = all;
    return locate<T, NT>(sh, row, 0, row.count, point_of(u, all), true, kept).index;
  };
  if (!p.cut() && p.min_p <= 0.0f) return draw(EveryWeight{p});
  return draw(KeptWeight(p));
}

// Writes value(z, index) of every entry to an output row.  From the row's end, which was
// read last and may still be in L2.
template <typename T, typename TO, int NT, typename F>
__device__ __forceinline__ void write_row(SampleShared<NT> &sh, const RowVectors<T> &row, TO *out,
                                          F value) {
  constexpr int VW = Elem<T>::kPerVec;
  // whole vectors where the output lies as the input against the 16-byte boundaries
  const bool alike = sizeof(T) == sizeof(TO) &&
                     reinterpret_cast<uint64_t>(out) % 16 == reinterpret_cast<uint64_t>(row.row) % 16;
  auto write = [&](const uint4 &v, int k) {
    if (sizeof(T) == sizeof(TO) && alike && k >= row.full_lo && k < row.full_hi) {
      uint4 y;
#pragma unroll
      for (int e = 0; e < VW / 2; ++e)
        put_pair<T>(y, e, value(Elem<T>::get(v, 2 * e), (int)row.index(k, 2 * e)),
                    value(Elem<T>::get(v, 2 * e + 1), (int)row.index(k, 2 * e + 1)));
      __stcs(reinterpret_cast<uint4 *>(out + row.index(k, 0)), y);
      return;
    }
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const int64_t i = row.index(k, e);
      if (i >= 0 && i < row.V) out[i] = narrow<TO>(value(Elem<T>::get(v, e), (int)i));
    }
  };
  for_vectors<T, NT, NT, true>(sh, row, 0, row.count, threadIdx.x, write);
}

// The filtered row by reading the row again: kept entries over the temperature, others -inf.
template <typename T, typename TO, int NT>
__device__ __noinline__ void write_filtered(bool greedy, TO *out) {
  SampleShared<NT> &sh = shared_of<NT>();
  const RowVectors<T> row = sh.template row<T>();
  const RowParams p = sh.params;
  if (p.min_p <= 0.0f && !greedy)
    write_row<T, TO, NT>(sh, row, out, [&](float z, int i) {
      return p.in_order(z, i) ? finite<TO>(__fmul_rn(z, p.r)) : -INFINITY;
    });
  else
    write_row<T, TO, NT>(sh, row, out, [&](float z, int i) {
      const bool kept = p.in_order(z, i) && p.weight(z) >= p.min_p;
      return kept ? (greedy ? 0.0f : finite<TO>(__fmul_rn(z, p.r))) : -INFINITY;
    });
}

// x in every entry of an output row.
template <typename TO, int NT>
__device__ __forceinline__ void fill_row(TO *out, int V, float x) {
  const Grid<TO> grid(out, V);
  uint4 v;
#pragma unroll
  for (int e = 0; e < Elem<TO>::kPerVec / 2; ++e) put_pair<TO>(v, e, x, x);
  for (int k = threadIdx.x; k < grid.count; k += NT) store_pack<TO>(out, grid, k, v);
}

// A row that nothing filters, over its temperature: one pass, unless it is no distribution.
template <typename T, typename TO, int NT>
__device__ __noinline__ void write_unfiltered(float r, TO *out) {
  SampleShared<NT> &sh = shared_of<NT>();
  const RowVectors<T> row = sh.template row<T>();
  float m = -INFINITY;
  write_row<T, TO, NT>(sh, row, out, [&](float z, int) {
    m = max_nan(m, z);
    return z > -INFINITY ? finite<TO>(__fmul_rn(z, r)) : -INFINITY;
  });
  if (__syncthreads_or(!(m < INFINITY))) fill_row<TO, NT>(out, row.V, quiet_nan());
}

// The draw from a row that nothing filters: the warp whose run holds u W by the first pass's
// sums, `about` in all and up to off_by off; exact within the run.  The index is -1 where
// those sums do not tell it from a neighbour.
template <typename T, int NT>
__device__ __noinline__ int draw_plain(float u, float about, float off_by) {
  SampleShared<NT> &sh = shared_of<NT>();
  const RowVectors<T> row = sh.template row<T>();
  const RowParams p = sh.params;
  const Deal<NT> deal(row.count);
  // every lane takes a run's sum: their running sums
  const int lane = threadIdx.x & 31;
  const float at = __fmul_rn(u, about), mine = lane < NT / 32 ? sh.fsum[lane] : 0.0f;
  float upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const float x = __shfl_up_sync(~0u, upto, off);
    if (lane >= off) upto = __fadd_rn(upto, x);
  }
  const uint32_t over = __ballot_sync(~0u, upto > at && lane < NT / 32);
  const int w = over != 0 ? __ffs(over) - 1 : NT / 32 - 1;
  const float before = __shfl_sync(~0u, upto, w > 0 ? w - 1 : 0) * (w > 0 ? 1.0f : 0.0f);
  const int lo = deal.lo(w, row.count), hi = deal.lo(w + 1, row.count);
  // u times the whole and what lies before the run, each off in proportion; and roundings
  const float t = __fsub_rn(at, before);
  const float off = __fmaf_rn(__fadd_rn(u, __fdiv_rn(before, about)), off_by, 5e-7f * about);
  const uint64_t t_at = __float2ull_rn(fmaxf(t, 0.0f) * p.scale), t_off = __float2ull_ru(off * p.scale);
  const EveryWeight every{p};
  run_sums<T, NT>(sh, row, lo, hi, every);
  const uint64_t all = total_of(sh);
  int index = -1;
  if (t_at >= t_off && t_at + t_off < all) {
    const Place x = locate<T, NT>(sh, row, lo, hi, t_at, true, every);
    if (t_at >= x.below + t_off && t_at + t_off < x.below + x.own) index = x.index;
  }
  __syncthreads();
  return index;
}

// What the first pass leaves to further ones.
struct Rest {
  bool by_k, by_p, plain, greedy;
  int top_k;
  float top_p, u, limit, about, off_by;
};
template <typename T, typename TO, int NT>
__device__ __noinline__ void by_passes(const SampleArgs &a, const Rest q) {
  SampleShared<NT> &sh = shared_of<NT>();
  const int64_t r = blockIdx.x;
  bool summed = false;
  if (q.by_k || q.by_p)
    summed = cut_all<T, NT>(q.by_k, q.top_k, q.limit > 0.0f ? q.limit : INFINITY, q.by_p, q.top_p,
                            q.about) &&
             sh.params.min_p <= 0.0f;
  if (a.u != nullptr) {
    int x = -1;
    float ln = 0.0f;
    if (q.plain) {
      x = draw_plain<T, NT>(q.u, q.about, q.off_by);
      ln = logf(q.about);
    }
    // (close to a weight of 1 the logarithm wants the exact sum)
    if (x < 0 || q.about < 1.05f) {
      // (within the row whatever happens: a caller may write it meanwhile)
      x = max(0, draw_all<T, NT>(q.u, summed));
      ln = ln_units(sh.before, sh.params.scale);
    }
    if (threadIdx.x == 0) {
      const RowParams p = sh.params;
      const float zx = widen(*(static_cast<const volatile T *>(sh.template row<T>().row) + x));
      a.tokens[r] = x;
      a.logprob[r] = __fmul_rn(__fsub_rn(zx, p.m), p.r) - ln;
      a.lse[r] = q.greedy ? 0.0f : finite<float>(__fmaf_rn(p.m, p.r, ln));
    }
    __syncthreads();  // zx is read: the row may be overwritten
  }
  if (a.filtered != nullptr)
    write_filtered<T, TO, NT>(q.greedy, static_cast<TO *>(a.filtered) + r * (int64_t)a.V);
}

template <typename T, typename TO, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) sample_kernel(
    const __grid_constant__ SampleArgs a) {
  SampleShared<NT> &sh = shared_of<NT>();
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T *first = static_cast<const T *>(a.logits) + row_offset(r, a.N, a.stride_b, a.stride_n);
  const RowVectors<T> row(first, a.V, Span{a.logits, a.logits_end});
  TO *out = a.filtered != nullptr ? static_cast<TO *>(a.filtered) + r * (int64_t)a.V : nullptr;

  // --------------------------------------------------------------- the parameters
  const Request q(a, r);
  const bool draw = a.u != nullptr, greedy = q.greedy, by_k = q.by_k, by_p = q.by_p, by_a = q.by_a;
  const bool plain = !by_k && !by_p && !by_a, no_params = q.bad;
  const int top_k = q.top_k;
  const float top_p = q.top_p, min_p = q.min_p, u = q.u;
  RowParams p;
  p.r = q.r;
  p.min_p = min_p;
  p.scale = a.scale;
  p.tau = -INFINITY;
  p.tie = -1;

  if (plain && !draw && !no_params) {
    if (tid == 0) sh.template row<T>() = row;
    __syncthreads();
    write_unfiltered<T, TO, NT>(p.r, out);
    return;
  }

  // ------------------------------------------------------------------ the first pass
  const Deal<NT> deal(row.count);
  float m, ref, s;
  const bool sums = by_p ? !by_k : plain && draw;
  if (sums)
    first_pass<T, NT, true>(sh, row, deal, p.r, m, ref, s);
  else
    first_pass<T, NT, false>(sh, row, deal, p.r, m, ref, s);
  float top = m;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, off));
  if (lane == 0) sh.fpart[warp] = top;
  __syncthreads();
  m = sh.fpart[0];
#pragma unroll 8
  for (int w = 1; w < NT / 32; ++w) m = max_nan(m, sh.fpart[w]);
  const bool bad = no_params || !(m < INFINITY);
  if (bad || m == -INFINITY) {  // no distribution
    if (draw && tid == 0) {
      a.tokens[r] = -1;
      a.logprob[r] = bad ? quiet_nan() : 0.0f;
      a.lse[r] = bad ? quiet_nan() : -INFINITY;
    }
    if (out != nullptr) fill_row<TO, NT>(out, a.V, bad ? quiet_nan() : -INFINITY);
    return;
  }
  p.m = m;
  float about = 0.0f, off_by = 0.0f;  // the sum of all weights, and how far it may be off
  if (sums) {
    if (s != 0.0f) s = __fmul_rn(s, ex2(fmaxf(__fmul_rn(__fsub_rn(ref, m), __fmul_rn(p.r, kLog2e)), kFarBelow)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s = __fadd_rn(s, __shfl_xor_sync(~0u, s, off));
    if (lane == 0) sh.fsum[warp] = s;
    __syncthreads();
#pragma unroll 8
    for (int w = 0; w < NT / 32; ++w) about = __fadd_rn(about, sh.fsum[w]);
    // In units of 2^-24 of the sum.  Additions: a strip's terms, the strips, the edges, the merges.
    // Weights, here and by their definition: four roundings each in proportion to the
    // exponent, whose weighted mean is at most ln V, to the 16 that the reference may be off,
    // and the exponentials.
    const int terms = deal.seg_batches * kUnroll * Elem<T>::kPerVec / 2 + deal.segs + NT / 32 + 10;
    off_by = __fmul_rn(about, (float)(terms + 6 * (32 - __clz(a.V)) + 80) * 5.9604645e-8f);
  }

  // --------------------------------------------------------- the list, where it holds all
  float limit = -1.0f;
  if (by_k || by_p) {
    // the strips' maxima alone reach the target in this bin: so does the row
    for (int b = tid; b < kBins; b += NT) sh.count[b] = sh.mass_lo[b] = sh.mass_hi[b] = 0;
    __syncthreads();
    for (int g = 0; g < deal.segs; ++g) {
      const float z = sh.strip[g * NT + tid];
      if (!(z > -INFINITY)) continue;
      if (by_k)
        atomicAdd(&sh.count[linear_bin(m, z)], 1u);
      else  // rounded down: 4096 strips stay below 2^32
        atomicAdd(&sh.mass_lo[linear_bin(m, z)], (uint32_t)(p.weight(z) * 524288.0f));
    }
    __syncthreads();
    const uint64_t target =
        by_k ? (uint64_t)top_k
             : __float2ull_ru(top_p * (about + 1.05f * off_by) * 524288.0f) + 1;
    find_bin(sh, 0, target, !by_k);
    const int b = sh.found;
    if (b < kBins - 1) limit = (float)(b + 1) * (1.0f / kBinsPerUnit);
    __syncthreads();
  } else if (by_a) {
    // w >= a: (m - z) / T is at most -ln a, up to roundings
    limit = __fmul_rn(__fdiv_rn(__fadd_rn(-logf(min_p), 1e-4f), p.r), 1.0001f);
  }
  int n = 0;  // entries of the list up to the cut
  bool listed = false;
  if (limit > 0.0f) {
    const int have = gather_strips<T, NT>(sh, row, deal, m, limit);
    listed = have <= kList && have > 0;
    if (listed) {
      if (by_k || by_p) sort_keys<NT>(sh.key, have);  // (min-p alone asks for no order)
      n = by_k ? min(top_k, have) : have;
      if (by_p) {
        scan_list<NT>(sh, n, [&](int i) { return p.units(p.weight(key_value(sh.key[i]))); });
        if (by_k) {
          n = min(n - 1, first_reaching(sh, n, share_of(top_p, sh.upto[n - 1]))) + 1;
        } else {
          // (a twentieth more for the roundings here)
          const uint64_t lo = __float2ull_rd(fmaxf(0.0f, top_p * (about - 1.05f * off_by)) * p.scale);
          const uint64_t hi = __float2ull_ru(top_p * (about + 1.05f * off_by) * p.scale);
          const int i = first_reaching(sh, n, lo > 0 ? lo : 1);
          listed = i < n && sh.upto[i] >= hi;  // wherever in between the share lies
          n = i + 1;
        }
      }
    }
    __syncthreads();
  }
  if (listed) {
    if (out != nullptr) {
      fill_row<TO, NT>(out, a.V, -INFINITY);  // (the row itself is not needed any more)
      __syncthreads();
      for (int i = tid; i < n; i += NT) {
        const float z = key_value(sh.key[i]);
        if (!by_a || p.weight(z) >= min_p)
          out[key_index(sh.key[i])] = narrow<TO>(greedy ? 0.0f : finite<TO>(__fmul_rn(z, p.r)));
      }
    }
    if (!draw) return;
    auto weight = [&](int i) -> uint64_t {
      const float w = p.weight(key_value(sh.key[i]));
      return w >= min_p || greedy ? p.units(w) : 0;
    };
    constexpr int kCount = NT < 256 ? NT : 256;
    if (n > kCount) {
      // by rising index
      __syncthreads();
      for (int i = tid; i < n; i += NT) {
        const uint64_t k = sh.key[i];
        sh.key[i] = ((uint64_t)~key_index(k) << 32) | __float_as_uint(key_value(k));
      }
      __syncthreads();
      sort_keys<NT>(sh.key, n);
      auto value = [&](int i) { return __uint_as_float((uint32_t)sh.key[i]); };
      scan_list<NT>(sh, n, [&](int i) -> uint64_t {
        const float w = p.weight(value(i));
        return w >= min_p ? p.units(w) : 0;
      });
      const uint64_t all = sh.upto[n - 1];
      const int i = min(n - 1, first_reaching(sh, n, point_of(u, all) + 1));
      if (tid == 0) {
        const float ln = ln_units(all, p.scale);
        a.tokens[r] = (int)~(uint32_t)(sh.key[i] >> 32);
        a.logprob[r] = __fmul_rn(__fsub_rn(value(i), m), p.r) - ln;
        a.lse[r] = finite<float>(__fmaf_rn(m, p.r, ln));
      }
      return;
    }
    scan_list<NT>(sh, n, weight);
    const uint64_t all = sh.upto[n - 1], t = point_of(u, all);
    if (tid < n) {
      const uint64_t k = sh.key[tid], own = sh.upto[tid] - (tid > 0 ? sh.upto[tid - 1] : 0);
      uint64_t below = 0, last = 0;
      for (int j = 0; j < n; ++j) {  // (key_index falls as the key's lower half rises)
        const uint64_t upto = sh.upto[j];
        if ((uint32_t)sh.key[j] > (uint32_t)k) below += upto - last;
        last = upto;
      }
      if (below <= t && below + own > t) {  // one thread
        const float ln = ln_units(all, p.scale);
        a.tokens[r] = (int)key_index(k);
        a.logprob[r] = __fmul_rn(__fsub_rn(key_value(k), m), p.r) - ln;
        a.lse[r] = greedy ? 0.0f : finite<float>(__fmaf_rn(m, p.r, ln));
      }
    }
    return;
  }

  if (tid == 0) {
    sh.template row<T>() = row;
    sh.params = p;
  }
  __syncthreads();
  by_passes<T, TO, NT>(a, Rest{by_k, by_p, plain, greedy, top_k, top_p, u, limit, about, off_by});
}

template <typename T, typename TO, int NT>
cudaError_t launch_nt(const SampleArgs &a, cudaStream_t stream) {
  sample_kernel<T, TO, NT><<<(unsigned)a.R, NT, sizeof(SampleShared<NT>), stream>>>(a);
  return cudaGetLastError();
}

// Threads per row.  A CTA of 1024 takes an SM, 512 half of one, 256 a quarter: many threads
// end a row's passes soon, few leave its barriers and its sorts less to wait for.
//
// Where top-p may need passes over whole rows, rows differ in work, and the slowest decide
// (us with 1024 / 512 / 256 threads; rows of bf16, three in four with likely entries, top-p
// 0.95): V = 128256, 152 rows 78 / 80 / 121, 608 rows 157 / 173 / 255, 2048 rows 468 / 366 /
// 440; V = 50000, 152 rows 66 / 63 / 83, 608 rows 111 / 76 / 90, 2048 rows 320 / 200 / 193;
// V = 20000, 304 rows 58 / 36 / 37, 608 rows 95 / 57 / 53; V = 5000, 152 rows 32 / 25 / 25, 608
// rows 89 / 44 / 27.
// Otherwise as many as let every row begin at once (top-k 50): V = 128256, 152 rows 16.2 / 15.8 /
// 18.4, 304 rows 26 / 15.6 / 15.1, 608 rows 61 / 41 / 33; V = 20000, 152 rows 9.2 / 7.8 / 7.7;
// min-p, V = 50001, 133 rows 14.1 with 1024 and 15.6 with 512.
int row_threads(const SampleArgs &a, int sms) {
  const bool listed = a.top_k == nullptr && a.top_k_all > 0 && a.top_k_all <= kList / 2;
  const bool passes = (a.top_p != nullptr || a.top_p_all < 1.0f) && !listed;
  const bool vast = a.V >= (passes ? 80000 : 30000);
  if (a.R <= (passes ? 4 : 1) * (int64_t)sms && vast) return 1024;
  if (passes && vast) return 512;
  const int waves = a.V < 10000 ? 1 : passes && a.V >= 30000 ? 4 : 2;
  return a.R <= waves * (int64_t)sms ? 512 : 256;
}

template <typename T, typename TO>
cudaError_t launch(const SampleArgs &a, int sms, cudaStream_t stream) {
  switch (row_threads(a, sms)) {
    case 1024: return launch_nt<T, TO, 1024>(a, stream);
    case 512: return launch_nt<T, TO, 512>(a, stream);
    default: return launch_nt<T, TO, 256>(a, stream);
  }
}

template <typename T, typename TO>
cudaError_t prepare() {
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<T, TO, 512>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(SampleShared<512>));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(sample_kernel<T, TO, 1024>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(SampleShared<1024>));
  return e;
}

}  // namespace

cudaError_t sample_prepare() {
  cudaError_t e = prepare<float, float>();
  if (e == cudaSuccess) e = prepare<uint16_t, uint16_t>();
  if (e == cudaSuccess) e = prepare<uint16_t, float>();
  return e;
}

cudaError_t sample_launch(const SampleArgs &a, int dtype_bf16, int out_bf16, int sms,
                          cudaStream_t stream) {
  // Rows that a warp can hold, wherever they begin.
  if (a.V <= kShortEntries - (dtype_bf16 ? 8 : 4))
    return sample_short_launch(a, dtype_bf16, out_bf16, stream);
  if (dtype_bf16)
    return out_bf16 ? launch<uint16_t, uint16_t>(a, sms, stream)
                    : launch<uint16_t, float>(a, sms, stream);
  return launch<float, float>(a, sms, stream);
}

}  // namespace specv
