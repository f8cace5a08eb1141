// nvfp4_sample.cu -- the next token of each row of logits, by a given random number:
//   w_i = exp((l_i - max) / temperature), 0 where masked;  the tokens in descending
//   order of l (equal ones by index);  top-k: the first k;  top-p: while the w
//   before a token are less than top_p of what top-k left;  min-p: w_i >= min_p;
//   token: the least i with sum_{j <= i, kept} w_j > u * sum_kept w.
//
// The result is a whole number that hangs on sums over a vocabulary, so those
// are exact: a weight is a whole number of 2^-42, off by 2^-30 of itself or a
// unit (its exponent in two fp32 numbers, 2^-x by a table of 256 and a
// polynomial), sums of them are 64-bit integers, whose order does not matter,
// and u times a sum is formed in 128 bits.
//
// Bound: latency, a dozen dependent phases of a cluster (reading and the largest, a
// histogram, its slices, the cut, the sum), and the instructions of a token: about 40 for
// its weight, 50 more for a cut by mass.  Measured (bytes are the logits'): 1 x 32000 bf16,
// top-k 50 and top-p 0.9: 15 us; 7 x 262144 fp32, top-p 0.9: 38 us; 61 x 128256 bf16,
// every row with cuts of its own: 65 us; 256 x 151003 fp32, min-p 0.02: 102 us, 1.5 TB/s.
// (Tried for the third: bf16 in shared memory and clusters of half the size, one wave
// instead of two, took 14 % longer; CTAs of 1024 threads 9 %; comparing values before bins
// are computed 7 %.)
//
// Work split: a cluster of 1 to 16 CTAs per row, each with its run of the row in
// shared memory as fp32 (what does not fit is read again), so a row is read
// once.  A thread owns a run of consecutive tokens, of odd length, which spreads
// its threads over the banks and keeps index order in thread order.
//
// A cut (the k-th token, or the one that reaches top_p) is found through a
// histogram of counts and masses over 2048 ranges of the exponent, whose
// slices the cluster's CTAs add up; the tokens of the range that holds the
// cut (a handful to some hundreds) meet in one CTA, which sorts them (each
// counts those before it) and sums in order.  A range with too many of them is
// split again, by value and index.  Without top-k and top-p there is no
// histogram: two passes.
#include <algorithm>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {

namespace cg = cooperative_groups;

constexpr int kSampleThreads = 512, kSampleWarps = kSampleThreads / 32;
constexpr int kSampleMaxCtas = 16;  // of a cluster (8 where a device cannot place more)
constexpr int kBins = 2048;
constexpr int kList = kSampleThreads;  // tokens that one CTA ranks
constexpr int kShortK = 256;           // top-k up to which one CTA finishes the row
constexpr int kOneBits = 42;      // a weight of 1
constexpr int kSampleSmem = 226 * 1024;
static_assert(kMaxVocabulary <= 1 << 20, "a sum of weights stays below 2^63, a bin's high words below 2^32");

// 2^(j / 256) in units of 2^-31, and as fp32.
struct Pow2Table {
  uint32_t q[256];
  float f[256];
};
constexpr double root(double v) {  // by Newton's method
  double r = v;
  for (int i = 0; i < 60; ++i) r = 0.5 * (r + v / r);
  return r;
}
constexpr Pow2Table make_pow2_table() {
  Pow2Table t = {};
  double step[8] = {};  // 2^(1/2), 2^(1/4), ..
  double v = 2.0;
  for (int i = 0; i < 8; ++i) step[i] = v = root(v);
  for (int j = 0; j < 256; ++j) {
    double p = 1.0;
    for (int i = 0; i < 8; ++i)
      if (j >> (7 - i) & 1) p *= step[i];
    t.q[j] = (uint32_t)(p * 2147483648.0 + 0.5);
    t.f[j] = (float)(p * 2147483648.0);
  }
  return t;
}
__device__ const Pow2Table kPow2 = make_pow2_table();

struct SampleLaunch {
  SampleArgs a;
  int seg;   // tokens of a CTA
  int run;   // of a thread (odd)
  int cap;   // of a CTA in shared memory
};

// floor or ceiling of m * f for 0 <= f < 1: f is 24 bits times a power of two.
__device__ __forceinline__ uint64_t share_of(uint64_t m, float f, bool ceiling) {
  const uint32_t b = __float_as_uint(f);
  const int e = (int)(b >> 23);
  const uint64_t man = e ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;
  const int s = e ? 150 - e : 149;  // f = man * 2^-s, s >= 24
  const uint64_t lo = man * m, hi = __umul64hi(man, m);
  uint64_t q, r;  // r: whether anything is cut off
  if (s < 64) q = lo >> s | hi << (64 - s), r = lo << (64 - s);
  else if (s < 128) q = s == 64 ? hi : hi >> (s - 64), r = lo | (s == 64 ? 0 : hi << (128 - s));
  else q = 0, r = lo | hi;
  return q + (ceiling && r != 0);
}

// Shared memory of a CTA before its tokens' values.
template <bool CUTS>
struct alignas(16) SampleShared {
  uint32_t hist[3][CUTS ? kBins : 4];  // counts; masses' low and high words.  CTA 0: also the list.
  uint2 pow2[256];
  uint64_t box[2][kSampleMaxCtas][4];  // what the cluster's CTAs tell each other, in turn
  uint64_t warp_sum[kSampleWarps];
  uint32_t warp_count[kSampleWarps];
  uint64_t found[4];
  uint64_t total_mass[2][kSampleMaxCtas];  // of the slices of a histogram, by CTA
  uint32_t total_count[2][kSampleMaxCtas];
  uint32_t listed;
  // of the row, by one thread (fp64 is slow): log2(e) / temperature in two parts, the
  // least weight that stays, and how far below the largest logit it lies at most
  float unit_hi, unit_lo, reach;
  uint64_t least;
};
struct SampleList {  // over the histogram
  uint64_t key[kList], mass[kList];
  uint64_t sorted_key[kList], sorted_mass[kList];
};
static_assert(sizeof(SampleList) <= sizeof(SampleShared<true>::hist), "the list lies over the histogram");
// The slices' totals (for the first histogram and for a finer one), then the values.
__host__ __device__ constexpr int64_t sample_slices(bool cuts, int ctas) { return cuts ? 2 * (int64_t)(kBins / ctas) * 12 : 0; }

constexpr uint64_t kNoCut = 0;  // keeps every token

// CUTS: some row may have a top_k or top_p.  Without (known from the values for
// all rows) the kernel is a third as long and needs no histogram.
// PER_SM: CTAs that may share an SM.  With cuts, two leave 64 registers a thread, which is
// too few (7 x 262144: 41.7 us, alone on an SM 39.1), but 61 rows of 128256 take 90 us
// instead of 66 with one CTA to an SM.
template <typename T, bool CUTS, int PER_SM>
__global__ void __launch_bounds__(kSampleThreads, PER_SM) k_sample(const __grid_constant__ SampleLaunch p) {
  constexpr int kVec = 16 / sizeof(T);
  extern __shared__ __align__(16) uint8_t dsm[];
  SampleShared<CUTS> &sh = *reinterpret_cast<SampleShared<CUTS> *>(dsm);
  const auto cluster = cg::this_cluster();
  const SampleArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), bins = kBins / ctas;
  uint64_t *slice_mass = reinterpret_cast<uint64_t *>(dsm + sizeof(sh));     // [2][bins]
  uint32_t *slice_count = reinterpret_cast<uint32_t *>(slice_mass + 2 * bins);         // [2][bins]
  float *vals = reinterpret_cast<float *>(CUTS ? (void *)(slice_count + 2 * bins) : (void *)slice_mass);
  const int row = blockIdx.x / ctas;
  cluster_begun();
  const int first = rank * p.seg, n = max(0, min(p.seg, a.vocabulary - first));
  const T *logits = static_cast<const T *>(a.logits) + (int64_t)row * a.stride + first;

  // values to vals[shift + i], so that 16-byte loads meet 16-byte places
  const int head = n > 0 ? (int)(((16 - (reinterpret_cast<uintptr_t>(logits) & 15u)) & 15u) / sizeof(T)) : 0;
  const int shift = (kVec - head) % kVec, kept = min(n, p.cap);
  auto as_float = [](T v) { return (float)v; };
  auto get = [&](int i) { return i < kept ? vals[shift + i] : as_float(logits[i]); };
  // an order of the alive tokens: by value, then by index; bigger is earlier
  auto key_of = [&](float v, int i) {
    const uint32_t b = __float_as_uint(v + 0.0f);  // (-0 is 0)
    return (uint64_t)(b >> 31 ? ~b : b | 0x80000000u) << 32 | (uint32_t)~(first + i);
  };
  auto alive = [](float v) { return v > -INFINITY; };  // (not NaN either)

  const float temperature = a.temperature ? a.temperature[row] : a.temperature_all;
  if (tid == kSampleThreads - 1 && temperature > 0.0f) {
    const float min_p = a.min_p ? a.min_p[row] : a.min_p_all;
    uint64_t least = 1;
    if (min_p > 0.0f) least = min_p < 1.0f ? max(uint64_t{1}, share_of(uint64_t{1} << kOneBits, min_p, true)) : uint64_t{1} << kOneBits;
    const double unit = fmin(1.4426950408889634 / (double)temperature, 1e38);
    sh.unit_hi = (float)unit;
    sh.unit_lo = (float)(unit - (double)(float)unit);
    sh.least = least;
    sh.reach = (float)((log2((double)least) - kOneBits - 0.01) / unit);  // (0.01: more than fp32 rounds)
  }

  // ---- the row into shared memory; its largest
  for (int i = tid; i < 256; i += kSampleThreads) sh.pow2[i] = make_uint2(kPow2.q[i], __float_as_uint(kPow2.f[i]));
  float most = -INFINITY;  // of this thread, first seen at `where` or in the kVec from there
  int where = -1;
  if (tid < head && tid < n) {
    const float v = as_float(logits[tid]);
    if (tid < kept) vals[shift + tid] = v;
    if (v > most) most = v, where = tid;
  }
  const int whole = max(0, n - head) / kVec;
#pragma unroll 4
  for (int v = tid; v < whole; v += kSampleThreads) {
    const uint4 r = __ldcs(reinterpret_cast<const uint4 *>(logits + head) + v);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    float x[kVec];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(w[i]);
      else x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    const int at = head + v * kVec;
    if (at + kVec <= kept) {
#pragma unroll
      for (int i = 0; i < kVec; i += 4) *reinterpret_cast<float4 *>(vals + shift + at + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (at + i < kept) vals[shift + at + i] = x[i];
    }
    float here = x[0];
#pragma unroll
    for (int i = 1; i < kVec; ++i) here = fmaxf(here, x[i]);  // (NaN gives way)
    if (here > most) most = here, where = at;
  }
  for (int i = head + whole * kVec + tid; i < n; i += kSampleThreads) {
    const float v = as_float(logits[i]);
    if (i < kept) vals[shift + i] = v;
    if (v > most) most = v, where = i;
  }
  uint64_t top = 0;
  if (where >= 0) {
    while (as_float(logits[where]) != most) ++where;
    top = key_of(most, where);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) sh.warp_sum[warp] = top;
  __syncthreads();

  // Tells every CTA of the cluster four numbers of this one; read at box[turn][rank].
  int turn = 1;
  auto tell = [&](uint64_t v0, uint64_t v1, uint64_t v2, uint64_t v3) {  // by threads 0 .. ctas - 1, of which each has them
    turn ^= 1;
    if (tid < ctas) {
      uint64_t *to = cluster.map_shared_rank(sh.box[turn][rank], tid);
      to[0] = v0, to[1] = v1, to[2] = v2, to[3] = v3;
    }
    cluster.sync();
  };
  top = 0;
  for (int w = 0; w < kSampleWarps; ++w) top = max(top, sh.warp_sum[w]);
  cluster_wait_begun();
  tell(top, 0, 0, 0);
  for (int r = 0; r < ctas; ++r) top = max(top, sh.box[turn][r][0]);
  const bool writes = rank == 0 && tid == 0;
  const int best = (int)~(uint32_t)top;
  if (top == 0 || !(temperature > 0.0f)) {  // nothing unmasked; or the largest is asked for
    if (writes) {
      a.token[row] = top == 0 ? -1 : best;
      if (a.logprob) a.logprob[row] = top == 0 ? -INFINITY : 0.0f;
    }
    return;
  }

  // ---- weights
  const uint32_t tb = (uint32_t)(top >> 32);
  const float m = __uint_as_float(tb >> 31 ? tb & 0x7FFFFFFFu : ~tb);
  const float ch = sh.unit_hi, cl = sh.unit_lo;
  const bool endless = m == INFINITY;  // then the infinite ones share the row
  // log2 of a weight, its larger part (in the order of the values: each operation keeps it)
  auto power = [&](float v) { return endless ? v == m ? 0.0f : -INFINITY : (v - m) * ch; };
  auto weight = [&](float v) -> uint64_t {
    if (!(v >= -3.4028235e38f)) return 0;  // masked
    if (endless) return v == m ? 1ull << kOneBits : 0;
    // v - m, and what its rounding lost; times log2(e) / T likewise
    const float d = v - m, b = v - d, dl = (v - (d + b)) - (m - b);
    const float h = d * ch;
    if (!(h > -64.0f)) return 0;
    float l = fmaf(d, ch, -h);
    l = fmaf(d, cl, l);
    l = fmaf(dl, ch, l);
    const float t = fmaf(h, 256.0f, 12582912.0f);
    const int k = __float_as_int(t) - 0x4B400000;
    const float r = fmaf(t - 12582912.0f, -0.00390625f, h) + l;  // |r| <= 2^-9
    const float z = r * fmaf(r, fmaf(r, 0.05550410866f, 0.24022650696f), 0.69314718056f);  // 2^r - 1
    const uint2 e = sh.pow2[k & 255];
    const uint32_t q = e.x + (uint32_t)__float2int_rn(__uint_as_float(e.y) * z);  // in units of 2^-31
    const int down = -(k >> 8);
    return down > kOneBits ? 0 : ((uint64_t)q << (kOneBits - 31)) >> down;
  };
  const int t0 = min(tid * p.run, n), t1 = min(t0 + p.run, n);  // this thread's tokens

  // ---- cuts
  int top_k = CUTS ? a.top_k ? a.top_k[row] : a.top_k_all : 0;
  if (top_k < 0 || top_k >= a.vocabulary) top_k = 0;
  const float top_p = CUTS ? a.top_p ? a.top_p[row] : a.top_p_all : 1.0f;
  const bool by_mass = top_p < 1.0f;
  uint64_t cut = kNoCut;

  // A histogram's totals in this CTA's slice of it, and those of every slice.
  auto add_slices = [&](int set, bool masses) {
    cluster.sync();
    uint64_t ms = 0;
    uint32_t cs = 0;
    for (int i = tid; i < bins; i += kSampleThreads) {
      uint64_t mass = 0;
      uint32_t count = 0;
#pragma unroll
      for (int r0 = 0; r0 < kSampleMaxCtas; r0 += 8) {  // (eight CTAs' words on their way at once)
        uint32_t w[8][3];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          w[r][0] = w[r][1] = w[r][2] = 0u;
          if (r0 + r < ctas) {
            const uint32_t *h = cluster.map_shared_rank(&sh.hist[0][0], r0 + r) + rank * bins + i;
            w[r][0] = h[0];
            if (masses) w[r][1] = h[kBins], w[r][2] = h[2 * kBins];
          }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) count += w[r][0], mass += (uint64_t)w[r][1] + ((uint64_t)w[r][2] << 32);
      }
      slice_mass[set * bins + i] = mass;
      slice_count[set * bins + i] = count;
      ms += mass, cs += count;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ms += __shfl_xor_sync(~0u, ms, o), cs += __shfl_xor_sync(~0u, cs, o);
    if (lane == 0) sh.warp_sum[warp] = ms, sh.warp_count[warp] = cs;
    __syncthreads();
    ms = 0, cs = 0;
    for (int w = 0; w < kSampleWarps; ++w) ms += sh.warp_sum[w], cs += sh.warp_count[w];
    tell(ms, cs, 0, 0);
    if (tid < ctas) sh.total_mass[set][tid] = sh.box[turn][tid][0], sh.total_count[set][tid] = (uint32_t)sh.box[turn][tid][1];
    __syncthreads();
  };
  auto clear = [&] {
    for (int i = tid; i < 3 * kBins; i += kSampleThreads) (&sh.hist[0][0])[i] = 0u;
    __syncthreads();
  };
  auto add = [&](int bin, uint64_t w) {
    atomicAdd(&sh.hist[0][bin], 1u);
    if (by_mass) {
      const uint32_t lo = (uint32_t)w, old = atomicAdd(&sh.hist[1][bin], lo);
      const uint32_t hi = (uint32_t)(w >> 32) + (old + lo < lo);
      if (hi) atomicAdd(&sh.hist[2][bin], hi);
    }
  };
  // Three quarters of the bins for the first 22 of the 44 octaves, where a cut by mass
  // lies: its weight is at least (1 - top_p) / vocabulary of the largest.
  auto bin_of = [&](float v) {
    const float x = -power(v);
    return (int)fminf(fminf(x * (0.75f * kBins / 22.0f), fmaf(x, 0.25f * kBins / 22.0f, 0.5f * kBins)), (float)(kBins - 1));
  };

  struct Totals {
    uint64_t mass;
    uint32_t count;
  };
  // The bin of histogram `set` in which the count or mass in order, with `before` ahead
  // of the histogram, reaches goal: everything up to it, and its own count.
  // (Some bin does: the caller has seen to it.)
  auto find_bin = [&](int set, Totals before, bool mass, uint64_t goal, int *bin, uint32_t *inside) {
    int owner = 0;
    for (; owner < ctas - 1; ++owner) {
      const Totals t = {sh.total_mass[set][owner], sh.total_count[set][owner]};
      if ((mass ? before.mass + t.mass : before.count + t.count) >= goal) break;
      before.mass += t.mass, before.count += t.count;
    }
    if (rank == owner) {  // each thread a run of bins
      const int per = (bins + kSampleThreads - 1) / kSampleThreads, b0 = min(tid * per, bins), b1 = min(b0 + per, bins);
      uint64_t ms = 0;
      uint32_t cs = 0;
      for (int i = b0; i < b1; ++i) ms += slice_mass[set * bins + i], cs += slice_count[set * bins + i];
      uint64_t im = ms;
      uint32_t ic = cs;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t um = __shfl_up_sync(~0u, im, o);
        const uint32_t uc = __shfl_up_sync(~0u, ic, o);
        if (lane >= o) im += um, ic += uc;
      }
      if (lane == 31) sh.warp_sum[warp] = im, sh.warp_count[warp] = ic;
      __syncthreads();
      Totals b = before;
      for (int w = 0; w < warp; ++w) b.mass += sh.warp_sum[w], b.count += sh.warp_count[w];
      b.mass += im - ms, b.count += ic - cs;
      if ((mass ? b.mass : b.count) < goal && (mass ? b.mass + ms : b.count + cs) >= goal) {  // one thread's
        for (int i = b0; i < b1; ++i) {
          const uint64_t wm = slice_mass[set * bins + i];
          const uint32_t wc = slice_count[set * bins + i];
          if ((mass ? b.mass + wm : b.count + wc) >= goal) {
            sh.found[0] = b.mass, sh.found[1] = b.count, sh.found[2] = (uint64_t)(rank * bins + i), sh.found[3] = wc;
            break;
          }
          b.mass += wm, b.count += wc;
        }
      }
      __syncthreads();
    }
    tell(sh.found[0], sh.found[1], sh.found[2], sh.found[3]);
    const uint64_t *f = sh.box[turn][owner];
    *bin = (int)f[2];
    *inside = (uint32_t)f[3];
    return Totals{f[0], (uint32_t)f[1]};
  };
  // Puts a list in descending order of its keys (all different): an element's place is the
  // number of larger ones, counted by as many threads as there are for each.
  auto sort_list = [&](SampleList &l, int count) {
    const int share = min(9 - (32 - __clz(max(count - 1, 0))), 5), e = tid >> share;  // log2 of an element's threads
    const bool there = e < count;
    const uint64_t key = there ? l.key[e] : 0;
    int place = 0;
    if (there) {
#pragma unroll 4
      for (int j = tid & ((1 << share) - 1); j < count; j += 1 << share) place += l.key[j] > key;
    }
    for (int o = 1; o < 1 << share; o <<= 1) place += __shfl_xor_sync(~0u, place, o);
    if (there && (tid & ((1 << share) - 1)) == 0) l.sorted_key[place] = key, l.sorted_mass[place] = l.mass[e];
    __syncthreads();
  };
  static_assert(kSampleThreads == 512 && kList == 512, "2^9 threads and elements");
  // The sum of the masses of the threads before this one, and of all.
  auto block_scan = [&](uint64_t v, uint64_t *all) {
    uint64_t in = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t up = __shfl_up_sync(~0u, in, o);
      if (lane >= o) in += up;
    }
    __syncthreads();
    if (lane == 31) sh.warp_sum[warp] = in;
    __syncthreads();
    uint64_t before = in - v, sum = 0;
    for (int w = 0; w < kSampleWarps; ++w) {
      if (w == warp) before += sum;
      sum += sh.warp_sum[w];
    }
    *all = sum;
    return before;
  };
  // This thread's tokens of which `is` holds to the list of CTA 0 (which lies over its histogram, by
  // then spent); what does not fit is left out.
  auto gather = [&](auto is) {
    if (rank == 0 && tid == 0) sh.listed = 0;
    cluster.sync();
    SampleList *list = reinterpret_cast<SampleList *>(cluster.map_shared_rank(&sh.hist[0][0], 0));
    uint32_t *listed = cluster.map_shared_rank(&sh.listed, 0);
#pragma unroll 4
    for (int i = t0; i < t1; ++i) {
      const float v = get(i);
      if (!is(v, i)) continue;
      const uint32_t at = atomicAdd(listed, 1u);
      if (at < kList) list->key[at] = key_of(v, i), list->mass[at] = weight(v);
    }
    cluster.sync();
  };
  // The first token in order with which the count or mass reaches goal, and both up to and with it.
  auto find = [&](bool mass, uint64_t goal, uint64_t *key) {
    int bin;
    uint32_t inside;
    Totals b = find_bin(0, Totals{0, 0}, mass, goal, &bin, &inside);
    uint64_t high = ~0ull, low = 0;  // the range's keys, once it is one of keys
    auto in_range = [&](float v, int i) {  // (the last bin's weights are 0: no cut lies there)
      if (!alive(v)) return false;
      if (low == 0) return bin_of(v) == bin;
      const uint64_t k = key_of(v, i);
      return k <= high && k >= low;
    };
    while (inside > kList) {
      uint64_t hk = 0, lk = ~0ull;  // the largest and smallest key inside
      for (int i = t0; i < t1; ++i) {
        const float v = get(i);
        if (in_range(v, i)) hk = max(hk, key_of(v, i)), lk = min(lk, key_of(v, i));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) hk = max(hk, __shfl_xor_sync(~0u, hk, o)), lk = min(lk, __shfl_xor_sync(~0u, lk, o));
      if (tid < 2) sh.found[tid] = tid ? ~0ull : 0;
      clear();
      if (lane == 0) atomicMax((unsigned long long *)&sh.found[0], (unsigned long long)hk), atomicMin((unsigned long long *)&sh.found[1], (unsigned long long)lk);
      __syncthreads();
      tell(sh.found[0], sh.found[1], 0, 0);
      for (int r = 0; r < ctas; ++r) hk = max(hk, sh.box[turn][r][0]), lk = min(lk, sh.box[turn][r][1]);
      const int width = 64 - __clzll((hk - lk) | 1), down = max(0, width - 11);  // (hk - lk) >> down < 2048
      for (int i = t0; i < t1; ++i) {
        const float v = get(i);
        if (in_range(v, i)) add((int)((hk - key_of(v, i)) >> down), by_mass ? weight(v) : 0);
      }
      add_slices(1, by_mass);
      int at;
      b = find_bin(1, b, mass, goal, &at, &inside);
      high = hk - ((uint64_t)at << down);  // (keys of finite values are above 2^54, a bin's width is at most 2^53)
      low = max(high - ((uint64_t{1} << down) - 1), lk);  // (the last bin reaches below lk, where the next range's tokens are)
    }
    gather(in_range);  // (there are `inside` of them)
    if (rank == 0) {
      const int count = min((int)inside, kList);
      SampleList &l = *reinterpret_cast<SampleList *>(&sh.hist[0][0]);
      sort_list(l, count);
      const uint64_t own = tid < count ? l.sorted_mass[tid] : 0;
      uint64_t all;
      const Totals ahead = {b.mass + block_scan(own, &all), b.count + (uint32_t)tid};
      const uint64_t upto = mass ? ahead.mass + own : (uint64_t)ahead.count + 1;
      if (tid < count && (mass ? ahead.mass : ahead.count) < goal && upto >= goal)
        sh.found[0] = l.sorted_key[tid], sh.found[1] = ahead.mass + own, sh.found[2] = ahead.count + 1;
      __syncthreads();
    }
    tell(sh.found[0], sh.found[1], sh.found[2], 0);
    *key = sh.box[turn][0][0];
    return Totals{sh.box[turn][0][1], (uint32_t)sh.box[turn][0][2]};
  };

  const uint64_t least = sh.least;
  float u = a.uniform[row];
  u = u > 0.0f ? u < 1.0f ? u : 0.99999994f : 0.0f;  // (NaN: 0)
  auto write = [&](int i, float v, uint64_t total) {
    a.token[row] = i;
    if (!a.logprob) return;
    const double l = endless ? 0.0 : ((double)v - (double)m) / (double)temperature;
    a.logprob[row] = (float)(l - log((double)total * (1.0 / (1ull << kOneBits))));
  };

  // ---- few tokens to choose from: a histogram of counts alone, and CTA 0 does the rest
  if (CUTS && top_k > 0 && top_k <= kShortK) {
    for (int i = tid; i < kBins; i += kSampleThreads) sh.hist[0][i] = 0u;
    __syncthreads();
    for (int i = t0; i < t1; ++i) {
      const float v = get(i);
      if (!alive(v)) continue;
      const int bin = bin_of(v);
      if (bin < kBins - 1) atomicAdd(&sh.hist[0][bin], 1u);  // (the last bin's weights are 0)
    }
    add_slices(0, false);
    uint32_t count = 0;
    for (int r = 0; r < ctas; ++r) count += sh.total_count[0][r];
    int last = kBins - 2;
    if (count > (uint32_t)top_k) {
      uint32_t inside;
      count = find_bin(0, Totals{0, 0}, false, (uint64_t)top_k, &last, &inside).count + inside;
    }
    if (count <= kList) {
      gather([&](float v, int) { return alive(v) && bin_of(v) <= last; });  // (there are `count` of them)
      if (rank > 0) return;
      SampleList &l = *reinterpret_cast<SampleList *>(&sh.hist[0][0]);
      sort_list(l, (int)count);
      // (top-k, top-p and min-p each keep the first in order)
      const int keep = min((int)count, top_k);
      const uint64_t key = tid < keep ? l.sorted_key[tid] : 0;
      uint64_t w = tid < keep ? l.sorted_mass[tid] : 0, total;
      const uint64_t ahead = block_scan(w, &total);
      if (by_mass && ahead >= max(uint64_t{1}, share_of(total, top_p > 0.0f ? top_p : 0.0f, true))) w = 0;  // (the largest stays)
      if (w < least) w = 0;
      // those that stay by index: their keys' halves change places
      if (tid < keep) l.key[tid] = key << 32 | key >> 32, l.mass[tid] = w;
      const int stay = __syncthreads_count(w != 0);
      sort_list(l, stay);
      w = tid < stay ? l.sorted_mass[tid] : 0;
      const uint64_t before = block_scan(w, &total), goal = share_of(total, u, false);
      if (w && before <= goal && before + w > goal) {
        const uint64_t k = l.sorted_key[tid];
        const uint32_t vb = (uint32_t)k;
        write((int)~(uint32_t)(k >> 32), __uint_as_float(vb >> 31 ? vb & 0x7FFFFFFFu : ~vb), total);
      }
      return;
    }
  }

  if (CUTS && (by_mass || top_k > 0)) {
    clear();
    for (int i = t0; i < t1; ++i) {
      const float v = get(i);
      if (!alive(v)) continue;
      const int bin = bin_of(v);
      if (bin < kBins - 1) add(bin, by_mass ? weight(v) : 0);
    }
    add_slices(0, by_mass);
    Totals whole_row = {0, 0};
    for (int r = 0; r < ctas; ++r) whole_row.mass += sh.total_mass[0][r], whole_row.count += sh.total_count[0][r];
    if (top_k > 0 && whole_row.count > (uint32_t)top_k) whole_row = find(false, (uint64_t)top_k, &cut);
    if (by_mass) {  // (the largest token stays whatever top_p)
      const uint64_t goal = max(uint64_t{1}, share_of(whole_row.mass, top_p > 0.0f ? top_p : 0.0f, true));
      if (goal < whole_row.mass) find(true, goal, &cut);
    }
  }

  // ---- the kept weights' sum, and the token
  // a value below which nothing stays: most tokens need no weight
  const float floor_v = endless ? m : __fadd_rd(m, sh.reach);
  const uint32_t cb = (uint32_t)(cut >> 32);
  const float cut_v = cut == kNoCut ? -INFINITY : __uint_as_float(cb >> 31 ? cb & 0x7FFFFFFFu : ~cb);
  const float low_v = fmaxf(floor_v, cut_v);
  auto stays = [&](float v, int i) -> uint64_t {
    const uint64_t w = weight(v);
    return w >= least && (cut == kNoCut || key_of(v, i) >= cut) ? w : 0;
  };
  uint64_t own = 0;
#pragma unroll 4
  for (int i = t0; i < t1; ++i) {
    const float v = get(i);
    if (v >= low_v) own += stays(v, i);
  }
  uint64_t sum;
  uint64_t before = block_scan(own, &sum);
  tell(sum, 0, 0, 0);
  uint64_t total = 0;
  for (int r = 0; r < ctas; ++r) {
    if (r < rank) before += sh.box[turn][r][0];
    total += sh.box[turn][r][0];
  }
  const uint64_t goal = share_of(total, u, false);  // a whole sum is above u * total where it is above this
  const uint32_t here = __ballot_sync(~0u, before <= goal && before + own > goal);
  if (here == 0) return;
  // one thread's run, of the whole cluster: its warp goes over it once more
  const int from = __ffs(here) - 1, first_of = __shfl_sync(~0u, t0, from), last_of = __shfl_sync(~0u, t1, from);
  before = __shfl_sync(~0u, before, from);
  for (int i0 = first_of; i0 < last_of; i0 += 32) {
    const int i = i0 + lane;
    const float v = i < last_of ? get(i) : -INFINITY;
    const uint64_t w = v >= low_v && i < last_of ? stays(v, i) : 0;
    uint64_t upto = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t up = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += up;
    }
    upto += before;
    if (upto - w <= goal && upto > goal) write(first + i, v, total);
    before = __shfl_sync(~0u, upto, 31);
    if (before > goal) break;
  }
}

namespace {

template <typename T, bool CUTS>
cudaError_t sample_launch(const SampleArgs &a, int sms, int most_ctas, cudaStream_t st) {
  // As few CTAs per row as let two of them share an SM (three, of twice as many, took 7 %
  // longer on 256 x 151003, half as many that read a third of their row again 58 %); more, down to 2048 tokens each, while that
  // leaves SMs idle.
  int ctas = 1;
  const int64_t share = 112 * 1024;
  auto fixed = [&](int c) { return (int64_t)sizeof(SampleShared<CUTS>) + sample_slices(CUTS, c); };
  auto seg = [&](int c) { return (a.vocabulary + c - 1) / c; };
  while (ctas < most_ctas && (seg(ctas) > (share - fixed(ctas)) / 4 - 8 || ((int64_t)a.rows * ctas < sms && seg(ctas) > 2048)))
    ctas *= 2;
  SampleLaunch p = {a, seg(ctas), 0, 0};
  p.run = (p.seg + kSampleThreads - 1) / kSampleThreads | 1;
  p.cap = (int)std::min<int64_t>(p.seg, (kSampleSmem - fixed(ctas)) / 4 - 8);
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)ctas;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows * ctas));
  cfg.blockDim = dim3(kSampleThreads);
  cfg.dynamicSmemBytes = (size_t)fixed(ctas) + 4 * ((size_t)p.cap + 8);
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if constexpr (CUTS)
    if ((int64_t)a.rows * ctas <= sms) return cudaLaunchKernelEx(&cfg, k_sample<T, CUTS, 1>, p);
  return cudaLaunchKernelEx(&cfg, k_sample<T, CUTS, 2>, p);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, int sms, int most_ctas, cudaStream_t st) {
  const bool cuts = a.top_k || a.top_p || (a.top_k_all > 0 && a.top_k_all < a.vocabulary) || a.top_p_all < 1.0f;
  if (a.fp32) return cuts ? sample_launch<float, true>(a, sms, most_ctas, st) : sample_launch<float, false>(a, sms, most_ctas, st);
  return cuts ? sample_launch<__nv_bfloat16, true>(a, sms, most_ctas, st) : sample_launch<__nv_bfloat16, false>(a, sms, most_ctas, st);
}

cudaError_t prepare_sample_kernels(int *ctas) {
  auto prepare = [](auto *k) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSampleSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
  };
  cudaError_t e = prepare(k_sample<float, true, 1>);
  if (e == cudaSuccess) e = prepare(k_sample<float, true, 2>);
  if (e == cudaSuccess) e = prepare(k_sample<float, false, 2>);
  if (e == cudaSuccess) e = prepare(k_sample<__nv_bfloat16, true, 1>);
  if (e == cudaSuccess) e = prepare(k_sample<__nv_bfloat16, true, 2>);
  if (e == cudaSuccess) e = prepare(k_sample<__nv_bfloat16, false, 2>);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = kSampleMaxCtas;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSampleMaxCtas);
  cfg.blockDim = dim3(kSampleThreads);
  cfg.dynamicSmemBytes = kSampleSmem;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, k_sample<float, true, 1>, &cfg) != cudaSuccess) cudaGetLastError();  // (8 then)
  *ctas = clusters > 0 ? kSampleMaxCtas : 8;
  return cudaSuccess;
}

}  // namespace nvfp4
