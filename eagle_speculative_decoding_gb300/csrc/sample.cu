// A token from each row of logits by temperature, top-k, top-p and min-p, or
// the logits that these leave.
//
// Source: "EAGLE: Speculative Sampling Requires Rethinking Feature
// Uncertainty", "Verification Phase: Multi-Round Speculative Sampling on Trees"
// (the token behind a prompt is drawn from the target's distribution, and a
// truncated distribution is verified like any other).
//
//   w_i = exp((x_i - max x) / T), entries ordered by (x descending, i ascending):
//   top-k keeps the first k; top-p keeps of these an entry while the weights
//   before it add up to less than p times their sum; min-p keeps w_i >= min_p;
//   the token is the first i, by index, whose running sum of kept weights
//   exceeds u times their sum.
//
// Where a sum passes a border (p times the sum, u times the sum) decides the
// result, and with 10^5 entries the borders lie closer than fp32's rounding of
// such sums.  So weights are whole numbers, w = round(2^44 e^((x - max) / T)), off by
// half a unit and 2^-36 of themselves at most (below 2^-9 of the largest the half unit is the
// larger part), and their sums are exact 64-bit integers: no order of summation, no
// atomics' order and no split of a row changes any result.
//
// A row belongs to a cluster of 1 to 8 CTAs: contiguous ranges by CTA and warp, so
// that running sums by index are sums over ranges.  Passes after the first read the
// row from L2.  What a row costs goes by what it keeps:
//   few entries  In the first pass every thread finds its largest entry.  With q = k / 8
//                of a CTA's at or above a value, k entries of the row are at or above
//                the least of the eight CTAs' values, and not many more: one comparison
//                each in the second pass collects them.  One CTA works out the order
//                of up to 256 by comparing all with all, sorts up to 1024, and
//                finishes the row with their exact weights.  Top-p without top-k needs
//                the sum over the whole row as well: the second pass adds it up in
//                fp32, which settles the border unless the sum's error reaches across
//                it; then the exact sum is taken.
//   many         For a cut, a histogram over the distance from the maximum (counts, or
//                weights to 16 bits of their bin's, one addition each) finds the bin that
//                it lies in, or the few that it may.  One pass with exact weights adds up
//                what lies in front of them and the whole, and collects their entries,
//                among which they are refined until they are few enough for one CTA, or
//                equal; equal entries are cut by their index.  What lies in front is kept,
//                so that a token's running sums need no further pass.  After a top-k the
//                CTAs go on with the entries that they collected, otherwise with the row.
//
// What bounds it: one row, the chain of loads, cluster barriers (1 us each) and first
// fetches of its code: 128,256 entries, bf16, top-k 50 and top-p 0.95 12 us in a graph
// (first pass 2.5, threshold and barrier 2.5, second pass 2.5, list 5).  Rows that
// keep many, the instructions of the exact weights (some 75 an entry, a third of the
// stalls waiting for instructions): a row of 128,256 whose top-p keeps half of it 55
// us, 64 of them 112.  Copies in flight to shared memory, rings of loads in registers
// and shorter loops changed none of that, and sums of exact weights in the bins, four
// additions an entry, took as long.
// Four CTAs an SM at 64 registers against three at 80: 64 rows of top-p 0.95 112 us and
// 156, of top-k 50 29 and 35, 256 rows of mixed settings truncated 134 and 152; 17 rows
// of 50,257 57.4 and 54.5.  Clusters of two or four CTAs serve many rows
// better, and take up to twice as long for one that keeps many (sample_launch).
#include <float.h>
#include <math.h>
#include <stddef.h>

#include <algorithm>

#include "common.cuh"

namespace eagle {
namespace {

// Table-driven exponential (P. Tang, "Table-driven implementation of the exponential
// function in IEEE floating-point arithmetic", 1989), here for 2^-y in fixed
// point: 2^(-i/64) in units of 2^-44, and 1 - 2^(-i/4096) in units of 2^-38.
__device__ __constant__ const unsigned long long kPow64[64] = {
    0x100000000000ull, 0xfd3e0c0cf48ull, 0xfa83b2db723ull, 0xf7d0df730adull, 0xf5257d15248ull, 0xf281773c5a0ull,
    0xefe4b99bdceull, 0xed4f301ed99ull, 0xeac0c6e7dd2ull, 0xe8396a503c5ull, 0xe5b906e77c8ull, 0xe33f8972be9ull,
    0xe0ccdeec2a9ull, 0xde60f4825e1ull, 0xdbfbb797dafull, 0xd99d15c278bull, 0xd744fccad6aull, 0xd4f35aabcffull,
    0xd2a81d91f13ull, 0xd06333daef3ull, 0xce248c151f8ull, 0xcbec14fef27ull, 0xc9b9bd866e3ull, 0xc78d74c8abcull,
    0xc5672a11550ull, 0xc346ccda249ull, 0xc12c4cca667ull, 0xbf1799b67a7ull, 0xbd08a39f581ull, 0xbaff5ab2134ull,
    0xb8fbaf47630ull, 0xb6fd91e328dull, 0xb504f333f9eull, 0xb311c412a91ull, 0xb123f581d2bull, 0xaf3b78ad691ull,
    0xad583eea42aull, 0xab7a39b5a94ull, 0xa9a15ab4ea8ull, 0xa7cd93b4e96ull, 0xa5fed6a9b15ull, 0xa43515ae09eull,
    0xa27043030c5ull, 0xa0b0510fb97ull, 0x9ef5326091aull, 0x9d3ed9a72d0ull, 0x9b8d39b9d55ull, 0x99e0459320bull,
    0x9837f0518dcull, 0x96942d37202ull, 0x94f4efa8fefull, 0x935a2b2f13eull, 0x91c3d373ab1ull, 0x9031dc43146ull,
    0x8ea4398b45dull, 0x8d1adf5b7e6ull, 0x8b95c1e3ea9ull, 0x8a14d575497ull, 0x88980e8092eull, 0x871f61969e9ull,
    0x85aac367cc5ull, 0x843a28c3aceull, 0x82cd8698ac3ull, 0x8164d1f3bc0ull};
__device__ __constant__ const uint32_t kPow4096[64] = {
    0u, 46512384u, 93016898u, 139513543u, 186002320u, 232483230u, 278956276u, 325421458u, 371878777u,
    418328235u, 464769834u, 511203574u, 557629456u, 604047484u, 650457656u, 696859976u, 743254444u, 789641061u,
    836019829u, 882390750u, 928753824u, 975109052u, 1021456437u, 1067795980u, 1114127681u, 1160451543u, 1206767566u,
    1253075751u, 1299376101u, 1345668617u, 1391953299u, 1438230149u, 1484499169u, 1530760360u, 1577013722u, 1623259258u,
    1669496969u, 1715726856u, 1761948920u, 1808163163u, 1854369586u, 1900568191u, 1946758978u, 1992941949u, 2039117105u,
    2085284448u, 2131443979u, 2177595699u, 2223739610u, 2269875713u, 2316004009u, 2362124500u, 2408237187u, 2454342070u,
    2500439153u, 2546528435u, 2592609919u, 2638683604u, 2684749494u, 2730807589u, 2776857890u, 2822900400u, 2868935118u,
    2914962046u};

constexpr int kNT = 256, kNW = kNT / 32;
constexpr int kBins = 512;       // of a bin that is refined
constexpr int kFine = 2048;      // of a whole row
constexpr int kCap = 1024;       // entries that one CTA sorts
constexpr int kLocal = 1536;     // entries that a CTA collects
constexpr int kMaxVocab = 1 << 18;
constexpr int kOne = 44;         // a weight of 1 is 2^kOne: 2^18 of them stay below 2^63
constexpr int kLimb = 15;        // a weight's limbs in the histogram: 2^16 of them stay below 2^32
constexpr int kMaxCluster = 8;
// Of the row's sum in fp32, relative: an entry's exponent y <= 45 in three roundings
// (0.7 * 3 * 45 * 2^-24), its exponential (2^-22), and up to 128 + 21 additions.
constexpr float kSumError = 3.0517578125e-5f;
// Of sums over the row's bins, relative: a weight is the bin's times 16 bits (2^-17, its
// exponential 2^-22), its place in units of the exponent up to 45 is off by 2^-22 of
// itself (2^-17), the bin's weight by 2^-24 of that exponent (2^-19).
constexpr double kBinError = 3.0517578125e-5;

struct SampleParams {
  const void* x;
  long long stride;  // elements from row to row
  int M, V, per;
  const float *temp, *top_p, *min_p, *u;
  const int32_t* top_k;
  int32_t* tokens;
  float* logprobs;
  int32_t* kept;
  void* out;  // the truncated logits (null: a token is drawn)
  long long out_stride;
  int units;  // 16-byte units of a warp's range
  int32_t* status;
};

struct Entry {  // of the sorted list
  unsigned long long key, w;
};
struct Part {  // what a CTA tells the others
  unsigned long long v;
  unsigned int n, flags;
  unsigned long long w;
};
struct Found {  // the bin that a search ends at
  unsigned long long before;  // measure before it
  unsigned int bin, before_n, n, pad;
};
struct Cut {  // entries behind (value, idx) in the order are dropped
  float value;
  int idx;
};
enum Outcome { kDone, kNeedSum, kNeedAll };  // of a list
enum Source { kList, kRow };                 // where a CTA's entries are

// Order-preserving key of a float that is no NaN; the two zeros are equal.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

struct Weigh {
  float xmax, ch, cl;  // log2(e) / T in two parts
  // round(2^44 2^-y), y = (xmax - x) log2(e) / T, the difference and the product
  // in two fp32 parts each: y to 2^-40 or better where the weight is not small.
  __device__ __forceinline__ unsigned long long operator()(float x, const unsigned long long* pow64,
                                                           const uint32_t* pow4096) const {
    const float dh = xmax - x, b = dh - xmax, dl = (xmax - (dh - b)) - (x + b);
    // (no branch, so that a thread's entries are worked out side by side; at 50 the
    // weight is zero, as it is from 45 on)
    const float yh = fminf(dh * ch, 50.f);
    const float yl = yh < 50.f ? fmaf(dh, ch, -yh) + fmaf(dh, cl, dl * ch) : 0.f;
    const float t = fmaf(yh, 4096.f, 12582912.f);  // rounds to a whole number in the low bits
    const int j = __float_as_int(t) - 0x4b400000;
    const float r = fmaf(t - 12582912.f, -1.f / 4096.f, yh) + yl;  // |r| <= 2^-13 and a little
    // 1 - 2^-r = g - g^2 / 2 (the next term is below 2^-43), times 2^38
    const float g = r * 0.6931471805599453f, e = fmaf(-0.5f * g, g, g);
    const unsigned long long a = pow64[(j >> 6) & 63];
    const uint32_t q = pow4096[j & 63], a31 = (uint32_t)(a >> (kOne - 31));
    const int s = __float2int_rn(fmaf(-e, (float)q, e * 274877906944.f));  // e - e q
    unsigned long long w = a - (((unsigned long long)a31 * q + (1u << 24)) >> (31 + 38 - kOne));
    w -= (unsigned long long)(((long long)(int)(a31 >> 1) * s) >> (30 + 38 - kOne));
    const int n = j >> 12;
    return (2 * w + (1ull << n)) >> (n + 1);  // rounded: 2 w < 2^46
  }
};


// What a CTA holds of a row.
struct alignas(16) Shared {
  // counts, and three limbs of sums of weights (a bin's four words apart: neighbouring
  // bins in all banks); or a word each of kFine bins
  uint32_t hist[4][kBins];
  uint2 local[kLocal];  // this CTA's collected entries: (order key, index)
  Entry list[kCap];     // the leader's list
  unsigned long long pow64[64], wv[kNW], wkey[kNW];
  unsigned long long kept_w[kNW];  // of the warps' ranges: what is kept, its weights and number
  uint32_t pow4096[64], wn[kNW], kept_n[kNW];
  float wsum[kNW];
  Part part[2][kMaxCluster];
  Found found;
  unsigned long long range[2];  // bins
  Cut cut;
  Weigh weigh;
  float bins, width, low, temp, top_p, u;  // bins per distance, and a bin's width in powers of two
  int top_k, n;
};

__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
  uint32_t ra;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(p)), "r"(rank));
  return ra;
}
__device__ __forceinline__ uint32_t ld_remote(const uint32_t* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
// whole 64-bit words to the same place in the shared memory of CTA `rank`
template <typename S>
__device__ __forceinline__ void st_remote(S* p, int rank, const S& v) {
  static_assert(sizeof(S) % 8 == 0, "whole 64-bit words");
  unsigned long long w[sizeof(S) / 8];
  memcpy(w, &v, sizeof(S));
  const uint32_t ra = remote(p, rank);
#pragma unroll
  for (int i = 0; i < (int)sizeof(S) / 8; ++i)
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(ra + 8 * i), "l"(w[i]) : "memory");
}
// barrier of the cluster after code that may have parted a warp
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  cluster_barrier();
}

// floor(f s), 0 <= f < 1 an fp32 number, exactly; `rest`: there is a fraction.
__device__ __forceinline__ unsigned long long scaled(float f, unsigned long long s, bool& rest) {
  const uint32_t b = __float_as_uint(f), ex = b >> 23;
  const uint32_t m = ex ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int sh = 150 - (int)max(ex, 1u);  // f = m 2^-sh, sh >= 24
  const unsigned long long lo = s * m, hi = __umul64hi(s, m);
  if (sh < 64) {
    rest = (lo & ((1ull << sh) - 1)) != 0;
    return hi << (64 - sh) | lo >> sh;
  }
  const int k = sh - 64;  // hi < 2^24
  rest = lo != 0 || (k >= 24 ? hi != 0 : (hi & ((1ull << k) - 1)) != 0);
  return k >= 24 ? 0 : hi >> k;
}

template <typename T>
struct Unit {
  static constexpr int E = 16 / sizeof(T);
};
__device__ __forceinline__ void open_unit(const uint4& u, float* f, const __nv_bfloat16*) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void open_unit(const uint4& u, float* f, const float*) {
  f[0] = __uint_as_float(u.x);
  f[1] = __uint_as_float(u.y);
  f[2] = __uint_as_float(u.z);
  f[3] = __uint_as_float(u.w);
}

template <typename V>
__device__ __forceinline__ V warp_scan(V v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const V x = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += x;
  }
  return v;
}
__device__ __forceinline__ unsigned long long warp_total(unsigned long long v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// A row's first or last unit, what is not the row's as -infinity.  (Rare steps are
// functions of their own: a row's code runs once or a few times on an SM, and fetching
// it takes longer than running it.)
template <typename T>
__device__ __noinline__ uint4 load_edge(const T* x, int i0, int V) {
  alignas(16) T e[Unit<T>::E];
  for (int k = 0; k < Unit<T>::E; ++k) e[k] = i0 + k >= 0 && i0 + k < V ? x[i0 + k] : (T)(-INFINITY);
  return *reinterpret_cast<const uint4*>(e);
}
template <typename T>
__device__ __noinline__ void store_edge(T* out, uint4 v, int i0, int V) {
  alignas(16) T e[Unit<T>::E];
  *reinterpret_cast<uint4*>(e) = v;
  for (int k = 0; k < Unit<T>::E; ++k)
    if (i0 + k >= 0 && i0 + k < V) out[i0 + k] = e[k];
}
// The entries of a unit within [from, to] to this CTA's local list.
template <typename T>
__device__ __noinline__ void collect_unit(Shared& sh, uint4 u, int i0, float from, float to) {
  float f[Unit<T>::E];
  open_unit(u, f, (const T*)nullptr);
  uint32_t n = 0;
#pragma unroll
  for (int k = 0; k < Unit<T>::E; ++k) n += (f[k] >= from) & (f[k] <= to);
  int at = atomicAdd(&sh.n, (int)n);
#pragma unroll
  for (int k = 0; k < Unit<T>::E; ++k)
    if ((f[k] >= from) & (f[k] <= to)) {
      if (at < kLocal) sh.local[at] = make_uint2(order_key(f[k]), (uint32_t)(i0 + k));
      ++at;
    }
}

// A row, a thread's place in it, and the steps that the paths share.  The cluster is
// the grid's x, the row its y.
template <typename T>
struct Row {
  static constexpr int E = Unit<T>::E;
  const SampleParams& p;
  Shared& sh;
  const T* x;
  int lead, u0, n_units;  // elements in front of the row in its first unit; the warp's units
  int phase;              // of sh.part: a CTA may write the next while another reads this one

  __device__ __forceinline__ Row(const SampleParams& p_, Shared& s, int phase_) : p(p_), sh(s), phase(phase_) {
    x = static_cast<const T*>(p.x) + (size_t)blockIdx.y * p.stride;
    lead = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    u0 = ((int)blockIdx.x * kNW + ((int)threadIdx.x >> 5)) * p.units;
    n_units = max(0, min(p.units, (p.V + lead + E - 1) / E - u0));
  }
  __device__ __forceinline__ int lane() const { return threadIdx.x & 31; }
  __device__ __forceinline__ int warp() const { return threadIdx.x >> 5; }
  __device__ __forceinline__ int C() const { return (int)gridDim.x; }
  __device__ __forceinline__ bool leader() const { return blockIdx.x == 0; }
  __device__ __forceinline__ int first_of(int j) const { return (u0 + j) * E - lead; }
  // unit j of the warp's range; what is not the row's counts as -infinity
  __device__ __forceinline__ uint4 load(int j) const {
    const int i0 = first_of(j);
    if (i0 >= 0 && i0 + E <= p.V) return *reinterpret_cast<const uint4*>(x + i0);
    return load_edge(x, i0, p.V);
  }
  // f(unit j, its values, index of its first entry) for this lane's units, in ascending
  // order, kUnits loads in flight
  template <int kUnits, typename F>
  __device__ __forceinline__ void sweep_units(F&& f) const {
    constexpr int U = kUnits;
#pragma unroll 1
    for (int j0 = lane(); j0 < n_units; j0 += 32 * U) {
      uint4 v[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (j0 + 32 * i < n_units) v[i] = load(j0 + 32 * i);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (j0 + 32 * i < n_units) f(v[i], first_of(j0 + 32 * i));
    }
  }
  // the same with one copy of f, the next load in flight meanwhile
  template <typename F>
  __device__ __forceinline__ void sweep_short(F&& f) const {
    uint4 next = lane() < n_units ? load(lane()) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
    for (int j = lane(); j < n_units; j += 32) {
      const uint4 v = next;
      if (j + 32 < n_units) next = load(j + 32);
      f(v, first_of(j));
    }
  }
  template <typename F>
  __device__ __forceinline__ void sweep(F&& f) const {  // f(value, index)
    sweep_short([&](const uint4& u, int i0) {
      float v[E];
      open_unit(u, v, (const T*)nullptr);
#pragma unroll
      for (int k = 0; k < E; ++k) f(v[k], i0 + k);
    });
  }
  // f(value, index, weight)
  template <typename F>
  __device__ __forceinline__ void sweep_weights(F&& f) const {
    sweep_short([&](const uint4& u, int i0) {
      float v[E];
      open_unit(u, v, (const T*)nullptr);
      unsigned long long w[E];
#pragma unroll
      for (int k = 0; k < E; ++k) w[k] = weight(v[k]);
#pragma unroll
      for (int k = 0; k < E; ++k) f(v[k], i0 + k, w[k]);
    });
  }
  // `mine`, the same in threads 0 .. C - 1, to all CTAs; returns where theirs are
  __device__ __forceinline__ const Part* tell(const Part& mine) {
    Part* to = sh.part[phase & 1];
    ++phase;
    if ((int)threadIdx.x < C()) st_remote(&to[blockIdx.x], threadIdx.x, mine);
    cluster_sync();
    return to;
  }
  __device__ __forceinline__ unsigned long long weight(float f) const { return sh.weigh(f, sh.pow64, sh.pow4096); }
  // place of an entry among the kFine bins by its distance from the maximum: in front of
  // the last up to where weights vanish
  __device__ __forceinline__ float place(float f) const { return fminf((sh.weigh.xmax - f) * sh.bins, (float)(kFine - 1)); }
  // keys that bin b's entries lie between, with room for the roundings
  __device__ __forceinline__ void keys_of(int b, uint32_t& lo, uint32_t& hi) const {
    const float xmax = sh.weigh.xmax;
    float from = -FLT_MAX, to = xmax;
    if (sh.bins > 0.f) {
      const float d0 = (float)b / sh.bins, d1 = (float)(b + 1) / sh.bins;
      to = fminf(to, xmax - d0 + 1e-6f * (fabsf(xmax) + d0));
      if (b < kFine - 1) from = fmaxf(from, xmax - d1 - 1e-6f * (fabsf(xmax) + d1));
    }
    lo = order_key(from);
    hi = order_key(to);
  }
  // Exclusive prefixes over the threads of the CTA, and the sums over all.
  __device__ __forceinline__ void block_scan(unsigned long long v, uint32_t n, unsigned long long& before, uint32_t& before_n,
                                             unsigned long long& all, uint32_t& all_n) {
    const unsigned long long iv = warp_scan(v);
    const uint32_t in = warp_scan(n);
    __syncthreads();  // sh.wv, sh.wn are free
    if (lane() == 31) sh.wv[warp()] = iv, sh.wn[warp()] = in;
    __syncthreads();
    unsigned long long o = 0, a = 0;
    uint32_t on = 0, an = 0;
#pragma unroll
    for (int w = 0; w < kNW; ++w) {
      if (w < warp()) o += sh.wv[w], on += sh.wn[w];
      a += sh.wv[w], an += sh.wn[w];
    }
    before = o + iv - v;
    before_n = on + in - n;
    all = a;
    all_n = an;
  }
  __device__ __forceinline__ void clear() {
    static_assert(alignof(Shared) >= 16 && offsetof(Shared, hist) % 16 == 0 && sizeof(sh.hist) == 16 * kBins, "16 bytes a store");
    for (int i = threadIdx.x; i < kBins; i += kNT) reinterpret_cast<uint4*>(sh.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
  }
  __device__ __forceinline__ void add(int b, bool weighted, unsigned long long w) {
    atomicAdd(&sh.hist[0][b], 1u);
    if (weighted) {
      constexpr uint32_t mask = (1u << kLimb) - 1;
      const uint32_t w0 = (uint32_t)w & mask, w1 = (uint32_t)(w >> kLimb) & mask, w2 = (uint32_t)(w >> (2 * kLimb));
      if (w0) atomicAdd(&sh.hist[1][b], w0);
      if (w1) atomicAdd(&sh.hist[2][b], w1);
      if (w2) atomicAdd(&sh.hist[3][b], w2);
    }
  }
  __device__ __forceinline__ unsigned long long block_sum(unsigned long long v) {
    v = warp_total(v);
    __syncthreads();
    if (lane() == 0) sh.wv[warp()] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kNW; ++w) v += sh.wv[w];
    return v;
  }
  // Of the kBins bins the one at which the cluster's running measure (counts, or sums of
  // weights) reaches goal (which some bin does): before < goal <= before + the bin's.  A
  // CTA adds up an eighth of the bins over all the histograms.
  __device__ __forceinline__ Found find_bin(bool weighted, unsigned long long goal) {
    cluster_sync();  // the histograms are complete
    constexpr int B = kBins / kNT;
    const int nb = kBins / C(), per = max(1, nb / kNT);
    // every word of this CTA's bins over all CTAs
    static_assert(sizeof(sh.list) >= 4 * kBins * sizeof(unsigned long long), "their sums are where the list will be");
    unsigned long long* sums = reinterpret_cast<unsigned long long*>(sh.list);
    for (int x = threadIdx.x; x < (weighted ? 4 : 1) * nb; x += kNT) {
      const uint32_t* word = &sh.hist[x / nb][blockIdx.x * nb + x % nb];
      uint32_t h[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) h[r] = r < C() ? ld_remote(word, r) : 0u;
      unsigned long long a = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) a += h[r];
      sums[x] = a;
    }
    __syncthreads();
    unsigned long long v[B], mine = 0;
    uint32_t n[B], mine_n = 0;
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int b = (int)threadIdx.x * per + i;
      const bool has = i < per && b < nb;
      n[i] = has ? (uint32_t)sums[b] : 0u;
      v[i] = !has ? 0 : weighted ? sums[nb + b] + (sums[2 * nb + b] << kLimb) + (sums[3 * nb + b] << (2 * kLimb)) : n[i];
      mine += v[i];
      mine_n += n[i];
    }
    unsigned long long before, sum;
    uint32_t before_n, all_n;
    block_scan(mine, mine_n, before, before_n, sum, all_n);
    const Part* parts = tell(Part{sum, all_n, 0});
    for (int r = 0; r < (int)blockIdx.x; ++r) before += parts[r].v, before_n += parts[r].n;
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (before < goal && goal <= before + v[i]) {
        const Found f{before, (uint32_t)(blockIdx.x * nb + threadIdx.x * per + i), before_n, n[i], 0};
        for (int r = 0; r < C(); ++r) st_remote(&sh.found, r, f);
      }
      before += v[i];
      before_n += n[i];
    }
    cluster_sync();
    return sh.found;
  }
  // Of the kFine bins those in which the cluster's running measure passes the goal, top_k
  // or top_p's part of the sum, whose sums of weights are within kBinError of the true
  // ones.  False if there are fewer than top_k entries.
  __device__ __forceinline__ bool find_range(bool weighted, int& first, int& last) {
    cluster_sync();  // the histograms are complete
    const int nb = kFine / C(), per = nb / kNT, b0 = (int)blockIdx.x * nb;
    static_assert(kFine % (kMaxCluster * kNT) == 0 && sizeof(sh.hist) >= 4 * kFine && sizeof(sh.list) >= 8 * kFine, "a CTA's bins");
    unsigned long long* sums = reinterpret_cast<unsigned long long*>(sh.list);
    const Weigh edge{0.f, sh.width, 0.f};
#pragma unroll 1
    for (int x = threadIdx.x; x < nb; x += kNT) {
      const uint32_t* word = sh.hist[0] + b0 + x;
      uint32_t h[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) h[r] = r < C() ? ld_remote(word, r) : 0u;
      unsigned long long a = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) a += h[r];
      if (weighted) a = __double2ull_rn((double)a * (double)edge(-(float)(b0 + x), sh.pow64, sh.pow4096) * 0x1p-16);
      sums[x] = a;
    }
    __syncthreads();
    unsigned long long mine = 0, before, sum;
    uint32_t bn, an;
    for (int i = 0; i < per; ++i) mine += sums[(int)threadIdx.x * per + i];
    block_scan(mine, 0, before, bn, sum, an);
    const Part* parts = tell(Part{sum, 0, 0, 0});
    sum = 0;
    for (int r = 0; r < C(); ++r) {
      if (r < (int)blockIdx.x) before += parts[r].v;
      sum += parts[r].v;
    }
    unsigned long long from = (unsigned long long)sh.top_k, to = from;
    if (weighted) {
      const double g = (double)sh.top_p * (double)sum;
      from = max(1ull, __double2ull_rd(g * (1.0 - 2 * kBinError)));
      to = __double2ull_ru(g * (1.0 + 2 * kBinError)) + 1;
    } else if (to > sum) {
      return false;
    }
    for (int i = 0; i < per; ++i) {
      const int x = (int)threadIdx.x * per + i;
      const unsigned long long end = before + sums[x];
      for (int r = 0; r < C(); ++r) {
        if (before < from && from <= end) st_remote(&sh.range[0], r, (unsigned long long)(b0 + x));
        if (before < to && to <= end) st_remote(&sh.range[1], r, (unsigned long long)(b0 + x));
      }
      before = end;
    }
    cluster_sync();
    first = (int)sh.range[0];
    last = to > sum ? kFine - 1 : (int)sh.range[1];
    return true;
  }
  // list[0 .. n) of the leader by key ascending
  __device__ __forceinline__ void sort_list(int n) {
    int n2 = 32;
    while (n2 < n) n2 <<= 1;
    for (int i = n + threadIdx.x; i < n2; i += kNT) sh.list[i] = Entry{~0ull, 0};
    __syncthreads();
    // up to 64 entries one warp does it, without the CTA's barriers
    const bool alone = n2 <= 64;
    if (!alone || warp() == 0) {
      const int step = alone ? 32 : kNT;
      for (int k = 2; k <= n2; k <<= 1)
        for (int j = k >> 1; j; j >>= 1) {
          for (int i = threadIdx.x; i < n2 / 2; i += step) {
            const int a = 2 * i - (i & (j - 1)), b = a + j;
            const Entry ea = sh.list[a], eb = sh.list[b];
            if ((ea.key > eb.key) == ((a & k) == 0)) sh.list[a] = eb, sh.list[b] = ea;
          }
          if (alone)
            __syncwarp();
          else
            __syncthreads();
        }
    }
    __syncthreads();
  }
  // All CTAs' local lists (sh.n entries each) in the leader's: the number of entries,
  // in all CTAs; over kCap nothing is sent (most: the largest local list).  Whole CTAs
  // call it.  The entries go with the counts, to a stretch of the list for each CTA,
  // where that holds them; otherwise behind another barrier.
  __device__ __forceinline__ int gather(unsigned long long v, unsigned long long& sum, int& most) {
    __syncthreads();
    const int mine = sh.n, stretch = kCap / C();
    auto send = [&](int to) {
      for (int i = threadIdx.x; i < mine; i += kNT) {
        const uint2 e = sh.local[i];
        st_remote(&sh.list[to + i], 0, Entry{(unsigned long long)~e.x << 32 | e.y, weight(key_value(e.x))});
      }
    };
    if (mine <= stretch) send((int)blockIdx.x * stretch);
    const Part* parts = tell(Part{v, (unsigned)mine, 0});
    int n = 0, at = 0;
    sum = 0;
    most = 0;
    for (int r = 0; r < C(); ++r) {
      const int m = (int)parts[r].n;
      if (r < (int)blockIdx.x) at += m;
      most = max(most, m);
      n += m;  // (262144 at most)
      sum += parts[r].v;
    }
    if (n > kCap) return n;
    if (most > stretch) {
      send(at);
      cluster_sync();
    } else if (leader()) {
      // close the gaps: entry i of all is entry i - at of CTA r
      constexpr int K = kCap / kNT;
      Entry e[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int i = (int)threadIdx.x + k * kNT;
        if (i >= n) continue;
        int r = 0, from = 0;
        while (i >= from + (int)parts[r].n) from += (int)parts[r++].n;
        e[k] = sh.list[r * stretch + i - from];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k)
        if ((int)threadIdx.x + k * kNT < n) sh.list[threadIdx.x + k * kNT] = e[k];
      __syncthreads();
    }
    return n;
  }
  // The leader, of a list of at most kNT entries: `lanes` neighbouring threads have entry
  // i (< n), and compare it with all.  key is its key with `turn` applied; before: the
  // measure of the entries of lower keys, rank: their number.
  template <typename K, typename W>
  __device__ __forceinline__ void among(int n, int lanes, int i, unsigned long long key, K&& key_of, W&& measure, uint32_t& rank,
                                        unsigned long long& before) const {
    rank = 0;
    before = 0;
    for (int j = (int)threadIdx.x & (lanes - 1); j < n; j += lanes) {
      const Entry e = sh.list[j];
      if (key_of(e.key) < key) {
        ++rank;
        before += measure(e);
      }
    }
    for (int d = 1; d < lanes; d <<= 1) {
      rank += __shfl_xor_sync(0xffffffffu, rank, d);
      before += __shfl_xor_sync(0xffffffffu, before, d);
    }
  }
  __device__ __forceinline__ int lanes_of(int n) const { return n <= kNT / 8 ? 8 : n <= kNT / 4 ? 4 : n <= kNT / 2 ? 2 : 1; }
  __device__ __forceinline__ Cut cut_of(unsigned long long key) const {
    return Cut{key_value(~(uint32_t)(key >> 32)), (int)(uint32_t)key};
  }
  __device__ __forceinline__ void send_cut(const Cut& c) {
    for (int r = 0; r < C(); ++r) st_remote(&sh.cut, r, c);
  }
  // The leader: the entry of its list of at most kNT at which the measure, from `before` on, reaches
  // goal, as the cut in all CTAs.
  __device__ __forceinline__ void cut_list(int n, bool weighted, unsigned long long before, unsigned long long goal) {
    const int lanes = lanes_of(n), i = (int)threadIdx.x / lanes;
    const Entry e = i < n ? sh.list[i] : Entry{0, 0};
    uint32_t rank;
    unsigned long long b;
    among(n, lanes, i, e.key, [](unsigned long long k) { return k; },
          [&](const Entry& x) { return weighted ? x.w : 1ull; }, rank, b);
    b += before;
    if (i < n && threadIdx.x % lanes == 0 && b < goal && goal <= b + (weighted ? e.w : 1ull)) send_cut(cut_of(e.key));
  }
  // one thread: the drawn token
  __device__ __forceinline__ void finish(float f, int i, unsigned long long sum, uint32_t kept) const {
    const int row = blockIdx.y;
    p.tokens[row] = i;
    if (p.kept) p.kept[row] = (int)kept;
    // -(xmax - x) / T - log(sum), the sum as 1 (the largest entry, which is always kept) and the rest
    if (p.logprobs)
      p.logprobs[row] = -(sh.weigh.xmax - f) / sh.temp - log1pf((float)(sum - (1ull << kOne)) * 5.684341886080802e-14f);
  }
  __device__ __forceinline__ unsigned long long part_of(unsigned long long sum) const {
    bool rest;  // kept while before < p sum: up to the entry that reaches ceil(p sum), the first at least
    const unsigned long long g = scaled(sh.top_p, sum, rest);
    return max(1ull, g + (rest ? 1 : 0));
  }
  // The leader: what is kept of its list, which holds all that may be, cut by top_k (0:
  // no cut) and top-p between the limits lo and hi (0: of the list's own sum; ~0: no
  // cut).  Draws the token, or leaves the cut in all CTAs' sh.cut.
  __device__ __forceinline__ Outcome use_list(int n, int top_k, unsigned long long lo, unsigned long long hi) {
    return n <= kNT ? use_short_list(n, top_k, lo, hi) : use_long_list(n, top_k, lo, hi);
  }
  __device__ __forceinline__ Outcome use_short_list(int n, int top_k, unsigned long long lo, unsigned long long hi) {
    const int lanes = lanes_of(n), i = (int)threadIdx.x / lanes;
    const bool mine = i < n && threadIdx.x % lanes == 0;
    const Entry e = i < n ? sh.list[i] : Entry{0, 0};
    uint32_t rank;
    unsigned long long before;
    among(n, lanes, i, e.key, [](unsigned long long k) { return k; }, [](const Entry& x) { return x.w; }, rank, before);
    const bool in = mine && (top_k == 0 || (int)rank < top_k);
    unsigned long long all = 0;
    if (hi != ~0ull) {
      all = block_sum(in ? e.w : 0);
      if (lo == 0) lo = hi = part_of(all);
      if (all < hi) return kNeedAll;
    }
    const bool above = cut_of(e.key).value >= sh.low;
    const bool k_lo = in && above && before < lo, k_hi = in && above && before < hi;
    unsigned long long none, sum;
    uint32_t bn, an;
    block_scan(k_lo ? e.w : 0, (k_lo ? 1u : 0u) + (k_hi ? 0x10000u : 0u), none, bn, sum, an);
    const int m = (int)(an & 0xffffu);
    if (m != (int)(an >> 16)) return kNeedSum;
    if (p.out) {
      if (k_lo && (int)rank == m - 1) {
        send_cut(cut_of(e.key));
        if (p.kept) p.kept[blockIdx.y] = m;
      }
      return kDone;
    }
    // the kept entries by index
    if (mine && !k_lo) sh.list[i].w = 0;
    __syncthreads();
    bool rest;
    const unsigned long long t = scaled(sh.u, sum, rest);
    auto index = [](unsigned long long k) { return (unsigned long long)(uint32_t)k; };
    among(n, lanes, i, index(e.key), index, [](const Entry& x) { return x.w; }, rank, before);
    if (k_lo && before <= t && t < before + e.w) finish(cut_of(e.key).value, (int)(uint32_t)e.key, sum, (uint32_t)m);
    return kDone;
  }
  __device__ __forceinline__ Outcome use_long_list(int n, int top_k, unsigned long long lo, unsigned long long hi) {
    sort_list(n);
    constexpr int K = kCap / kNT;  // neighbours of the list, a thread's
    unsigned long long w[K], mine = 0, before, all;
    uint32_t bn, an;
    const int i0 = (int)threadIdx.x * K;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      w[k] = i0 + k < n && (top_k == 0 || i0 + k < top_k) ? sh.list[i0 + k].w : 0;
      mine += w[k];
    }
    block_scan(mine, 0, before, bn, all, an);
    if (lo == 0) lo = hi = part_of(all);
    if (hi != ~0ull && all < hi) return kNeedAll;
    // kept by the lower and by the upper limit
    uint32_t m_lo = 0, m_hi = 0;
    unsigned long long v = 0, b = before;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (i0 + k < n && (top_k == 0 || i0 + k < top_k)) {
        const bool above = key_value(~(uint32_t)(sh.list[i0 + k].key >> 32)) >= sh.low;
        if (b < lo && above) ++m_lo, v += w[k];
        if (b < hi && above) ++m_hi;
      }
      b += w[k];
    }
    unsigned long long sum, none;
    block_scan(v, m_lo | m_hi << 16, none, bn, sum, an);
    const int m = (int)(an & 0xffffu);  // the first m of the list are kept
    if (m != (int)(an >> 16)) return kNeedSum;
    if (p.out) {
      if (threadIdx.x == 0) {
        send_cut(cut_of(sh.list[m - 1].key));
        if (p.kept) p.kept[blockIdx.y] = m;
      }
      return kDone;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < m; i += kNT) sh.list[i].key = sh.list[i].key << 32 | sh.list[i].key >> 32;  // by index
    sort_list(m);
    bool rest;
    const unsigned long long t = scaled(sh.u, sum, rest);
    mine = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      w[k] = i0 + k < m ? sh.list[i0 + k].w : 0;
      mine += w[k];
    }
    block_scan(mine, 0, before, bn, all, an);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (before <= t && t < before + w[k]) {
        const Entry e = sh.list[i0 + k];
        finish(key_value(~(uint32_t)e.key), (int)(e.key >> 32), sum, (uint32_t)m);
      }
      before += w[k];
    }
    return kDone;
  }
  // an entry that the cut, and min-p's border, leave
  __device__ __forceinline__ bool inside(float f, int i, const Cut& cut) const {
    return (f > cut.value) | ((f == cut.value) & (i <= cut.idx));
  }
  // out = the entries that `cut` leaves
  __device__ __forceinline__ uint32_t write(const Cut& cut) const {
    uint32_t n = 0;
    T* out = static_cast<T*>(p.out) + (size_t)blockIdx.y * p.out_stride;
    const bool whole = (reinterpret_cast<uintptr_t>(out) & 15u) == (reinterpret_cast<uintptr_t>(x) & 15u);
    const float low = sh.low;
    sweep_units<4>([&](const uint4& raw, int i0) {
      float v[E];
      open_unit(raw, v, (const T*)nullptr);
      alignas(16) T e[E];
      *reinterpret_cast<uint4*>(e) = raw;
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const bool in = (v[k] >= low) & inside(v[k], i0 + k, cut);
        n += in;
        e[k] = in ? e[k] : (T)(-INFINITY);
      }
      if (whole && i0 >= 0 && i0 + E <= p.V) {
        *reinterpret_cast<uint4*>(out + i0) = *reinterpret_cast<const uint4*>(e);
      } else {
        store_edge(out, *reinterpret_cast<const uint4*>(e), i0, p.V);
      }
    });
    return n;
  }
};

// Rows that keep many entries, from what the CTAs have collected (which holds all that
// may be kept) or from the whole row.  (Out of line: its registers and code are none
// of the others'.)
template <typename T, Source kFrom>
__device__ __noinline__ void many_kept(const SampleParams& p, Shared& sh, int phase) {
  constexpr int E = Row<T>::E;
  Row<T> row(p, sh, phase);
  const int lane = row.lane(), warp = row.warp(), C = row.C(), tid = threadIdx.x;
  int n_local = sh.n;
  Cut cut{-FLT_MAX, 0x7fffffff};
  auto sweep_local = [&](auto&& f) {
    for (int i = tid; i < n_local; i += kNT) {
      const uint2 e = sh.local[i];
      f(key_value(e.x), (int)e.y);
    }
  };
  auto sweep_weights = [&](auto&& f) {  // f(value, index, weight)
    if (kFrom == kRow)
      row.sweep_weights(f);
    else
      sweep_local([&](float x, int i) { f(x, i, row.weight(x)); });
  };
  // the sum of the cluster, and this warp's prefix in it by CTA and warp
  auto total = [&](unsigned long long v, uint32_t n, unsigned long long& off, uint32_t& off_n, unsigned long long& all,
                   uint32_t& all_n) {  // v, n: the warp's
    __syncthreads();
    if (lane == 0) sh.wv[warp] = v, sh.wn[warp] = n;
    __syncthreads();
    off = all = 0;
    off_n = all_n = 0;
    for (int w = 0; w < kNW; ++w) {
      if (w < warp) off += sh.wv[w], off_n += sh.wn[w];
      all += sh.wv[w];
      all_n += sh.wn[w];
    }
    const Part* parts = row.tell(Part{all, all_n, 0});
    all = 0;
    all_n = 0;
    for (int r = 0; r < C; ++r) {
      if (r < (int)blockIdx.x) off += parts[r].v, off_n += parts[r].n;
      all += parts[r].v;
      all_n += parts[r].n;
    }
  };
  const bool use_k = sh.top_k > 0 && sh.top_k < p.V, use_p = sh.top_p < 1.f;
  // the values between which a stage by weights has collected the row's entries, with the
  // sums over those in front in kept_w and kept_n (none: from > to)
  float col_from = 1.f, col_to = 0.f;
#pragma unroll 1
  for (int stage = 0; stage < 2; ++stage) {
    const bool by_w = stage == 1;
    if (by_w ? !use_p : !use_k) continue;
    cluster_sync();  // (the histogram, and what else the CTAs read of one another, is free)
    row.clear();
    {
      uint32_t far = 0;  // of the last bin, which may be most entries: they weigh nothing
      uint32_t* hist = sh.hist[0];
      auto put = [&](float f, int i) {
        const float at = row.place(f);
        const int b = (int)at;
        const bool in = row.inside(f, i, cut), last = b == kFine - 1;
        far += in & last;
        // (2^16 entries of a CTA at most)
        if (in & !last) atomicAdd(&hist[b], by_w ? __float2uint_rn(ex2_approx(((float)b - at) * sh.width) * 65535.f) : 1u);
      };
      if (kFrom == kRow)
        row.sweep(put);
      else
        sweep_local(put);
      far = __reduce_add_sync(0xffffffffu, far);
      if (!by_w && lane == 0 && far) atomicAdd(&hist[kFine - 1], far);
    }
    int b0, b1;
    if (!row.find_range(by_w, b0, b1)) continue;  // fewer than k entries
    // Exactly, then: what lies in front of those bins, the sum of all, and the entries
    // between (the row's are collected once, if they have room).
    uint32_t lo, hi, none;
    row.keys_of(b0, none, hi);
    row.keys_of(b1, lo, none);
    const float from = key_value(lo), to = key_value(hi);
    unsigned long long front = 0, sum = 0;
    uint32_t n_bin = 0, n_front = 0;
    auto measure = [&](float f, int i, unsigned long long w) {
      const bool in = row.inside(f, i, cut);
      front += in & (f > to) ? w : 0;
      n_front += in & (f > to);
      sum += in ? w : 0;
      n_bin += in & (f >= from) & (f <= to);
    };
    if (kFrom == kRow) {
      __syncthreads();
      if (tid == 0) sh.n = 0;
      __syncthreads();
      row.sweep_short([&](const uint4& raw, int i0) {
        float v[E];
        open_unit(raw, v, (const T*)nullptr);
        unsigned long long w[E];
#pragma unroll
        for (int k = 0; k < E; ++k) w[k] = by_w ? row.weight(v[k]) : (unsigned long long)(v[k] > -INFINITY);
        const uint32_t n = n_bin;
#pragma unroll
        for (int k = 0; k < E; ++k) measure(v[k], i0 + k, w[k]);
        if (n_bin != n) collect_unit<T>(sh, raw, i0, from, to);
      });
    } else {
      sweep_local([&](float f, int i) { measure(f, i, by_w ? row.weight(f) : 1ull); });
    }
    front = warp_total(front);
    n_bin = __reduce_add_sync(0xffffffffu, n_bin);
    n_front = __reduce_add_sync(0xffffffffu, n_front);
    if (lane == 0) sh.kept_w[warp] = front, sh.kept_n[warp] = n_front;
    sum = row.block_sum(sum);  // (and all of the row's are collected)
    if (kFrom == kRow) n_local = sh.n;
    __syncthreads();
    if (lane == 0) sh.wv[warp] = front, sh.wn[warp] = n_bin;
    __syncthreads();
    front = 0;
    n_bin = 0;
#pragma unroll
    for (int w = 0; w < kNW; ++w) front += sh.wv[w], n_bin += sh.wn[w];
    const Part* parts = row.tell(Part{front, n_bin, n_local > kLocal, sum});
    unsigned long long before = 0;
    sum = 0;
    n_bin = 0;
    bool collected = true;
    for (int r = 0; r < C; ++r) {
      before += parts[r].v;
      n_bin += parts[r].n;
      sum += parts[r].w;
      collected = collected && !parts[r].flags;
    }
    if (kFrom == kRow && by_w && collected) col_from = from, col_to = to;
    const unsigned long long goal = by_w ? row.part_of(sum) : (unsigned long long)sh.top_k;
    auto member = [&](float f, int i) {
      const uint32_t k = order_key(f);
      return (k >= lo) & (k <= hi) & row.inside(f, i, cut);
    };
    auto members = [&](auto&& f) {  // f(value, index) of the bin's entries
      auto if_member = [&](float x, int i) {
        if (member(x, i)) f(x, i);
      };
      if (kFrom == kRow && !collected)
        row.sweep(if_member);
      else
        sweep_local(if_member);
    };
    while (n_bin > kNT && lo < hi) {
      const int shift = max(0, 32 - __clz((int)(hi - lo)) - 9);
      row.clear();
      members([&](float f, int i) { row.add((int)((hi - order_key(f)) >> shift), by_w, row.weight(f)); });
      const Found in = row.find_bin(by_w, goal - before);
      before += in.before;
      n_bin = in.n;
      const uint32_t top = hi - (in.bin << shift), width = (1u << shift) - 1;
      lo = top - lo > width ? top - width : lo;
      hi = top;
    }
    if (n_bin <= kNT) {
      // to the leader, by their places in order of CTAs
      uint32_t n = 0;
      members([&](float, int) { ++n; });
      const uint32_t in = warp_scan(n);
      unsigned long long x, y;
      uint32_t off, all;
      total(0, __shfl_sync(0xffffffffu, in, 31), x, off, y, all);
      off += in - n;
      if (n)
        members([&](float f, int i) {
          st_remote(&sh.list[off++], 0, Entry{(unsigned long long)~order_key(f) << 32 | (uint32_t)i, row.weight(f)});
        });
      cluster_sync();
      if (row.leader()) row.cut_list((int)all, by_w, before, goal);
    } else {
      // equal entries: the c-th by index is the last
      const unsigned long long each = by_w ? row.weight(key_value(lo)) : 1ull;
      const unsigned long long c = (goal - before + each - 1) / each;
      uint32_t n = 0;
      row.sweep([&](float f, int i) { n += member(f, i) ? 1u : 0u; });  // (ranges by index: the row's)
      n = __reduce_add_sync(0xffffffffu, n);
      unsigned long long x, y;
      uint32_t off, all;
      total(0, n, x, off, y, all);
      if (off < c && c <= (unsigned long long)off + n) {  // this warp's range holds it
#pragma unroll 1
        for (int j0 = 0; j0 < row.n_units; j0 += 32) {
          const int j = j0 + lane, i0 = row.first_of(j);
          float v[E];
          uint32_t m = 0;
          if (j < row.n_units) {
            open_unit(row.load(j), v, (const T*)nullptr);
#pragma unroll
            for (int k = 0; k < E; ++k) m += member(v[k], i0 + k) ? 1u : 0u;
          }
          const uint32_t in = warp_scan(m);
          uint32_t nth = off + in - m;
          if (j < row.n_units && nth < c && c <= (unsigned long long)nth + m) {
#pragma unroll
            for (int k = 0; k < E; ++k)
              if (member(v[k], i0 + k) && ++nth == c) row.send_cut(Cut{key_value(lo), i0 + k});
          }
          off += __shfl_sync(0xffffffffu, in, 31);
        }
      }
    }
    cluster_sync();
    cut = sh.cut;
  }

  // ---- what is kept
  const float low = sh.low;
  uint32_t n = 0;
  unsigned long long v = 0;
  if (!p.out && col_from <= col_to && low <= col_to) {
    // those in front of what was collected are summed up already
    __syncthreads();
    sweep_local([&](float f, int i) {
      if ((f >= col_from) & (f >= low) & row.inside(f, i, cut)) {
        const int w = (i + row.lead) / E / p.units - (int)blockIdx.x * kNW;
        atomicAdd(&sh.kept_w[w], row.weight(f));
        atomicAdd(&sh.kept_n[w], 1u);
      }
    });
    __syncthreads();
    v = sh.kept_w[warp];
    n = sh.kept_n[warp];
  } else {
    if (p.out)
      n = row.write(cut);
    else
      sweep_weights([&](float f, int i, unsigned long long w) {
        const bool in = (f >= low) & row.inside(f, i, cut);
        v += in ? w : 0;
        n += in;
      });
    v = warp_total(v);
    n = __reduce_add_sync(0xffffffffu, n);
  }
  unsigned long long off, all;
  uint32_t off_n, all_n;
  total(v, n, off, off_n, all, all_n);
  if (p.out) {
    if (p.kept && row.leader() && tid == 0) p.kept[blockIdx.y] = (int)all_n;
    return;
  }
  bool rest;
  const unsigned long long t = scaled(sh.u, all, rest);
  if (kFrom == kList) {
    // the CTA whose range of indices holds the token: its entries by index
    unsigned long long mine = 0;
    for (int w = 0; w < kNW; ++w) mine += sh.wv[w];
    off = 0;
    for (int r = 0; r < (int)blockIdx.x; ++r) off += sh.part[(row.phase - 1) & 1][r].v;
    if (!(off <= t && t < off + mine)) return;
    // their sums over stretches of indices find a stretch of few entries
    unsigned long long from = (unsigned long long)max(0, ((int)blockIdx.x * kNW) * p.units * E - row.lead);
    uint32_t width = (uint32_t)kNW * p.units * E;
    // (a stretch of 1 / kNT of the range at a time: the CTA's threads hold one each)
    unsigned long long* sums = reinterpret_cast<unsigned long long*>(sh.list);  // [kNT], not the leader's list any more
    while (width > 1) {
      const uint32_t step = (width + kNT - 1) / kNT;
      __syncthreads();
      sums[tid] = 0;
      __syncthreads();
      for (int i = tid; i < n_local; i += kNT) {
        const uint2 e = sh.local[i];
        const float f = key_value(e.x);
        if (f >= low && row.inside(f, (int)e.y, cut) && e.y >= from && e.y - from < width)
          atomicAdd(&sums[(uint32_t)(e.y - from) / step], row.weight(f));
      }
      __syncthreads();
      unsigned long long before, s;
      uint32_t bn, an;
      const unsigned long long w = sums[tid];
      row.block_scan(w, 0, before, bn, s, an);
      before += off;
      if (before <= t && t < before + w) sh.found = Found{before, (uint32_t)tid, 0, 0, 0};
      __syncthreads();
      off = sh.found.before;
      from += (unsigned long long)sh.found.bin * step;
      width = step;
    }
    for (int i = tid; i < n_local; i += kNT)
      if (sh.local[i].y == (uint32_t)from) row.finish(key_value(sh.local[i].x), (int)from, all, all_n);
    return;
  }
  if (!(off <= t && t < off + v)) return;
#pragma unroll 1
  for (int j0 = 0; j0 < row.n_units; j0 += 32) {
    const int j = j0 + lane, i0 = row.first_of(j);
    float f[E];
    unsigned long long w[E], mine = 0;
#pragma unroll
    for (int k = 0; k < E; ++k) w[k] = 0;
    if (j < row.n_units) {
      open_unit(row.load(j), f, (const T*)nullptr);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const unsigned long long x = row.weight(f[k]);
        w[k] = (f[k] >= low) & row.inside(f[k], i0 + k, cut) ? x : 0;
        mine += w[k];
      }
    }
    const unsigned long long in = warp_scan(mine);
    unsigned long long at = off + in - mine;
    if (at <= t && t < at + mine) {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        if (at <= t && t < at + w[k]) row.finish(f[k], i0 + k, all, all_n);
        at += w[k];
      }
    }
    off += __shfl_sync(0xffffffffu, in, 31);
    if (off > t) break;
  }
}

template <typename T>
__global__ void __launch_bounds__(kNT, 4) sample_kernel(const SampleParams p) {
  constexpr int E = Unit<T>::E;
  __shared__ Shared sh;
  const int tid = threadIdx.x, at_row = blockIdx.y;
  if (tid < 64) {
    sh.pow64[tid] = kPow64[tid];
    sh.pow4096[tid] = kPow4096[tid];
  }
  if (tid == 0) sh.n = 0;
  // no CTA writes to another's shared memory before that one runs: waited for below
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  pdl_trigger();
  Row<T> row(p, sh, 0);
  const int lane = row.lane(), warp = row.warp();
  const int rq = at_row / p.per;
  const float temp = p.temp ? p.temp[rq] : 1.f, top_p = p.top_p ? p.top_p[rq] : 1.f, min_p = p.min_p ? p.min_p[rq] : 0.f;
  const int top_k = p.top_k ? p.top_k[rq] : 0;
  const float u = p.out ? 0.f : p.u[at_row];
  const bool bad_args = !(temp >= 0.f && temp <= FLT_MAX) || !(top_p >= 0.f) || !(min_p >= 0.f && min_p <= 1.f) ||
                        top_k < 0 || !(u >= 0.f && u < 1.f);

  // ---- first pass: the largest, and what is no logit
  const bool use_k = top_k > 0 && top_k < p.V, use_p = top_p < 1.f, small = p.V <= kCap;
  // What may be kept is collected from the q-th largest of a CTA's threads' largest on:
  // their largest of all entries, or, for a large k, of so many that about half of
  // them reach the value looked for.  q k-ths of the CTAs' are k entries at least; a
  // large k's is an estimate, and the entries are counted.
  int q = 0, group = 0x7fffffff;
  if (!small && temp != 0.f) {
    if (use_k) {
      q = (top_k + row.C() - 1) / row.C();
      if (q > kNT / 4) {
        const float share = (1.25f * (float)top_k + 32.f) / (float)p.V, units = (float)((p.units + 31) / 32);
        const float g = fmaxf(1.f, fminf(units, floorf(1.2f / (share * (float)E))));
        group = (int)g;
        q = share < 0.2f ? min(kNT, (int)((1.f - __expf(-share * g * (float)E)) * (float)kNT) + 8) : 0;
      }
    } else if (use_p) {
      q = 128 / row.C();  // (a nucleus of more takes the row's sums)
    }
  }
  float top = -INFINITY, group_top = -INFINITY;
  int at = 0x7fffffff, units = 0;
  bool odd = false;  // NaN or +infinity
  row.template sweep_units<8>([&](const uint4& v, int i0) {
    float f[E];
    open_unit(v, f, (const T*)nullptr);
#pragma unroll
    for (int k = 0; k < E; ++k) {
      odd = odd || !(f[k] <= FLT_MAX);
      if (f[k] > top) top = f[k], at = i0 + k;
    }
    if (units++ < group) group_top = top;
  });
  unsigned long long best = (unsigned long long)order_key(top) << 32 | (uint32_t)~at;
#pragma unroll
  for (int d = 16; d; d >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
  if (lane == 0) sh.wkey[warp] = best;
  const bool any_odd = __syncthreads_or(odd);
  best = sh.wkey[lane % kNW];
#pragma unroll
  for (int d = kNW / 2; d; d >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
  uint32_t from_key = 0xffffffffu;  // a value that q of this CTA's threads reach, to 2^-11
  if (q) {
    const uint32_t mine = order_key(group_top);
    from_key = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 12; --bit) {
      const uint32_t key = from_key | 1u << bit;
      if (__syncthreads_count(mine >= key) >= q) from_key = key;
    }
  }
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  {
    const Part* all = row.tell(Part{best, from_key, any_odd});
    odd = false;
    for (int r = 0; r < row.C(); ++r) {
      best = max(best, all[r].v);
      from_key = min(from_key, all[r].n);
      odd = odd || all[r].flags;
    }
  }
  const float xmax = key_value((uint32_t)(best >> 32));
  const int first = (int)~(uint32_t)best;
  if (bad_args || odd || xmax == -INFINITY) {
    if (row.leader() && tid == 0) {
      set_status(p.status, bad_args ? EAGLE_ERR_INVALID_ARG : EAGLE_ERR_NONFINITE);
      if (p.tokens) p.tokens[at_row] = -1;
      if (p.logprobs) p.logprobs[at_row] = -INFINITY;
      if (p.kept) p.kept[at_row] = 0;
    }
    return;
  }
  if (temp == 0.f) {
    if (row.leader() && tid == 0) {
      if (p.tokens) p.tokens[at_row] = first;
      if (p.logprobs) p.logprobs[at_row] = 0.f;
      if (p.kept) p.kept[at_row] = 1;
    }
    if (!p.out) return;
    if (tid == 0) sh.low = -FLT_MAX;
    __syncthreads();
    row.write(Cut{xmax, first});
    return;
  }
  if (tid == 0) {
    // log2(e) / T in two parts, the second from the remainder (a temperature so small
    // that its reciprocal overflows leaves the largest alone)
    const float ch = fminf(1.44269502f / temp, 3.0e38f);
    const float cl = ch < 3.0e38f ? (fmaf(-ch, temp, 1.44269502f) + 1.92596303e-8f) / temp : 0.f;
    sh.weigh = Weigh{xmax, ch, isfinite(cl) ? cl : 0.f};
    sh.bins = fminf((float)(kFine - 1) / ((float)(kOne + 1) + 0.01f) * ch, 3.0e38f);
    sh.width = ch / sh.bins;
    // w >= min_p as a border of x: the smallest fp32 number not below max + T log(min_p)
    float low = -FLT_MAX;
    if (min_p > 0.f) {
      const double b = (double)xmax + (double)temp * log((double)min_p);
      low = b <= -(double)FLT_MAX ? -FLT_MAX : __double2float_ru(b);
    }
    sh.low = low;
    sh.temp = temp;
    sh.top_p = top_p;
    sh.u = u;
    sh.top_k = top_k;
  }
  __syncthreads();

  // ---- the entries that may be kept, when they are few
  const bool by_sum = !use_k && use_p && !small;
  if (small || q || (!use_k && !use_p && min_p > 0.f)) {
    const float from = q ? (from_key > order_key(-FLT_MAX) ? key_value(from_key) : -FLT_MAX) : small ? -FLT_MAX : sh.low;
    const bool all_of_them = from == -FLT_MAX;
    const float c = by_sum ? sh.weigh.ch : 0.f;
    float sum = 0.f;
    row.template sweep_units<8>([&](const uint4& raw, int i0) {
      float v[E];
      open_unit(raw, v, (const T*)nullptr);
      float most = v[0];
#pragma unroll
      for (int k = 1; k < E; ++k) most = fmaxf(most, v[k]);
      if (by_sum) {
#pragma unroll
        for (int k = 0; k < E; ++k) sum += ex2_approx((v[k] - xmax) * c);
      }
      if (most >= from) collect_unit<T>(sh, raw, i0, from, xmax);
    });
    if (by_sum) {
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) sh.wsum[warp] = sum;
      __syncthreads();
      sum = 0.f;
#pragma unroll
      for (int w = 0; w < kNW; ++w) sum += sh.wsum[w];
    }
    unsigned long long around;  // the CTAs' sums, in units of 2^-40
    int most;
    const int n = row.gather(by_sum ? __float2ull_rn(sum * 1.099511627776e12f) : 0ull, around, most);
    const bool enough = all_of_them || !use_k || n >= top_k;
    if (n <= kCap && enough) {
      unsigned long long lo = ~0ull, hi = ~0ull;  // top-p's limits
      if (use_p) lo = hi = 0;
      if (by_sum && !all_of_them) {
        const float s = (float)around * 16.f;
        lo = row.part_of(__float2ull_rd(s * (1.f - kSumError)));
        hi = row.part_of(__float2ull_ru(s * (1.f + kSumError)));
      }
      Outcome result = kDone;
      if (row.leader()) result = row.use_list(n, use_k ? top_k : 0, lo, hi);
      if (by_sum && !all_of_them) {
        result = (Outcome)row.tell(Part{0, (unsigned)result, 0})[0].n;
        if (result == kNeedSum) {
          // the border lies within the sum's error: the exact sum
          unsigned long long v = 0;
          row.sweep_weights([&](float, int, unsigned long long w) { v += w; });
          const Part* parts = row.tell(Part{row.block_sum(v), 0, 0});
          v = 0;
          for (int r = 0; r < row.C(); ++r) v += parts[r].v;
          lo = row.part_of(v);
          result = kDone;
          if (row.leader()) result = row.use_list(n, 0, lo, lo);
          result = (Outcome)row.tell(Part{0, (unsigned)result, 0})[0].n;
        }
      } else if (p.out) {
        cluster_sync();
      }
      if (result == kDone) {
        if (p.out) row.write(sh.cut);
        return;
      }
    } else if (use_k && enough && most <= kLocal) {
      many_kept<T, kList>(p, sh, row.phase);
      return;
    }
  }
  many_kept<T, kRow>(p, sh, row.phase);
}

template <typename T>
int sample_launch(SampleParams p, void* stream) {
  if (p.M == 0) return EAGLE_OK;
  const int total = (p.V + Unit<T>::E - 1) / Unit<T>::E + 1;  // and one for a start off its boundary
  int C = 1;
  while (C < kMaxCluster && total > C * kNT * 2) C *= 2;
  // Many rows: two or four CTAs a row where a thread has 16 units at most then, for fewer
  // barriers and first fetches a row; from four waves of CTAs on, or two where it has 8 (one
  // row that keeps many takes longer).  bf16, mixed settings, fewer / eight: 256 rows of
  // 32,000 104 us and 142, 512 147 and 264, 4,096 792 and 1,970 (one CTA a row 1,070);
  // 512 rows of 128,256 332 and 402; 256 rows of 128,256 in fp32, of top-k up to 5,000,
  // which four CTAs cannot hold, 190 and 133.
  const long long slots = 4ll * std::max(1, sm_count());
  while (C > 2 && total <= C / 2 * kNT * 16 && (long long)p.M * C > slots * (total <= C / 2 * kNT * 8 ? 2 : 4)) C /= 2;
  p.units = (total + C * kNW - 1) / (C * kNW);
  launch_cluster(sample_kernel<T>, dim3(C, p.M), dim3(kNT), dim3(C, 1, 1), 0, static_cast<cudaStream_t>(stream), p);
  note_launch();
  return last_launch_status();
}

int sample_check(const SampleParams& p, int dtype, size_t es) {
  if (dtype != EAGLE_BF16 && dtype != EAGLE_FP32) return EAGLE_ERR_INVALID_ARG;
  if (p.M < 0 || p.V < 1 || p.per < 1 || (p.M > 0 && !p.x)) return EAGLE_ERR_INVALID_ARG;
  if (p.M > 65535 || p.V > kMaxVocab) return EAGLE_ERR_UNSUPPORTED;
  if (p.stride < p.V || (reinterpret_cast<uintptr_t>(p.x) & (es - 1))) return EAGLE_ERR_INVALID_ARG;
  return EAGLE_OK;
}

}  // namespace
}  // namespace eagle

using namespace eagle;

extern "C" int eagle_sample(const void* logits, long long row_stride, int M, int V, int dtype, const float* temperature,
                            const int32_t* top_k, const float* top_p, const float* min_p, int rows_per_request,
                            const float* uniforms, int32_t* tokens, float* logprobs, int32_t* n_kept,
                            int32_t* dev_status, void* stream) {
  const SampleParams p = {logits, row_stride, M, V, rows_per_request, temperature, top_p, min_p, uniforms, top_k, tokens,
                          logprobs, n_kept, nullptr, 0, 0, dev_status};
  const int rc = sample_check(p, dtype, dtype == EAGLE_BF16 ? 2 : 4);
  if (rc != EAGLE_OK) return rc;
  if (M > 0 && (!uniforms || !tokens)) return EAGLE_ERR_INVALID_ARG;
  return dtype == EAGLE_BF16 ? sample_launch<__nv_bfloat16>(p, stream) : sample_launch<float>(p, stream);
}

extern "C" int eagle_truncate_logits(const void* logits, long long row_stride, int M, int V, int dtype,
                                     const float* temperature, const int32_t* top_k, const float* top_p,
                                     const float* min_p, int rows_per_request, void* out, long long out_stride,
                                     int32_t* n_kept, int32_t* dev_status, void* stream) {
  const SampleParams p = {logits, row_stride, M, V, rows_per_request, temperature, top_p, min_p, nullptr, top_k, nullptr,
                          nullptr, n_kept, out, out_stride, 0, dev_status};
  const size_t es = dtype == EAGLE_BF16 ? 2 : 4;
  const int rc = sample_check(p, dtype, es);
  if (rc != EAGLE_OK) return rc;
  if (M > 0 && !out) return EAGLE_ERR_INVALID_ARG;
  if (out_stride < V || (reinterpret_cast<uintptr_t>(out) & (es - 1)) || (out == logits && out_stride != row_stride))
    return EAGLE_ERR_INVALID_ARG;
  return dtype == EAGLE_BF16 ? sample_launch<__nv_bfloat16>(p, stream) : sample_launch<float>(p, stream);
}
