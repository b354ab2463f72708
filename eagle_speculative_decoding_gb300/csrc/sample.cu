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
// such sums.  So weights are whole numbers, w = round(2^44 e^((x - max) / T)), good
// to 2^-37 of themselves, and their sums are exact 64-bit integers: no order of
// summation, no atomics' order and no split of a row changes any result.
//
// A row belongs to a cluster of 1 to 8 CTAs, which read it once and keep it in
// shared memory: contiguous ranges by CTA and warp, so that running sums by index
// are sums over ranges.  The order is never sorted as a whole.  A histogram over
// the distance from the maximum (64 bins per octave; counts, and for top-p sums of
// weights) finds the bin in which the k-th entry or the p-th part lies; the entries
// up to it, when they are at most 1024, are sorted by one CTA, which finishes the
// row.  Otherwise that bin alone is refined, until its entries are few enough to be
// sorted or all equal; equal entries are cut by their index.
#include <float.h>
#include <math.h>

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

constexpr int kNT = 512, kNW = kNT / 32;
constexpr int kBins = 2048;
constexpr int kCap = 1024;       // entries that one CTA sorts
constexpr int kMaxVocab = 1 << 18;
constexpr int kOne = 44;         // a weight of 1 is 2^kOne: 2^18 of them stay below 2^63
constexpr int kLimb = 15;        // a weight's limbs in the histogram: 2^16 of them stay below 2^32
constexpr int kMaxCluster = 8;

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
  unsigned long long v, key;
  unsigned int n, flags;
};
struct Found {  // the bin or entry that a search ends at
  unsigned long long before;  // measure before it
  unsigned int bin, before_n, n, pad;
};
struct Cut {  // entries behind (key, idx) in the order are dropped
  uint32_t key;
  int idx;
};

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
    const float yh = dh * ch;
    if (!(yh < (float)kOne + 1.f)) return 0;  // below half a unit (or no difference at all)
    const float yl = fmaf(dh, ch, -yh) + fmaf(dh, cl, dl * ch);
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
    return n ? (w + (1ull << (n - 1))) >> n : w;
  }
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
__device__ __forceinline__ uint2 ld_remote2(const uint2* p, int rank) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(remote(p, rank)) : "memory");
  return v;
}
// 24 or 32 bytes to the same place in the shared memory of CTA `rank`.
template <typename S>
__device__ __forceinline__ void st_remote(S* p, int rank, const S& v) {
  static_assert(sizeof(S) % 8 == 0, "whole 64-bit words");
  const unsigned long long* w = reinterpret_cast<const unsigned long long*>(&v);
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

template <typename T>
__global__ void __launch_bounds__(kNT) sample_kernel(const SampleParams p) {
  constexpr int E = Unit<T>::E;
  extern __shared__ __align__(16) unsigned char sm[];  // histogram, then the row's slice
  uint32_t* hist_n = reinterpret_cast<uint32_t*>(sm);
  uint32_t* hist_w = hist_n + kBins;                    // three limbs
  uint2* local = reinterpret_cast<uint2*>(sm);          // this CTA's entries of the list (over hist_n)
  Entry* list = reinterpret_cast<Entry*>(hist_w);       // the leader's sorted list
  const uint4* slice = reinterpret_cast<const uint4*>(sm + 4 * kBins * 4);
  static_assert(kCap * sizeof(uint2) <= 4 * kBins && kCap * sizeof(Entry) <= 12 * kBins, "the lists lie over the histogram");
  __shared__ unsigned long long s_pow64[64], s_wv[kNW];
  __shared__ uint32_t s_pow4096[64], s_wn[kNW];
  __shared__ Part s_part[2][kMaxCluster];
  __shared__ Found s_found;
  __shared__ float s_ch, s_cl, s_low;
  __shared__ int s_local;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)gridDim.x, rank = (int)blockIdx.x, row = blockIdx.y;  // the cluster is the grid's x
  const T* tag = nullptr;
  if (tid < 64) {
    s_pow64[tid] = kPow64[tid];
    s_pow4096[tid] = kPow4096[tid];
  }
  // no CTA writes to another's shared memory before that one runs: waited for below
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  pdl_trigger();

  const int rq = row / p.per;
  const float temp = p.temp ? p.temp[rq] : 1.f, top_p = p.top_p ? p.top_p[rq] : 1.f, min_p = p.min_p ? p.min_p[rq] : 0.f;
  const int top_k = p.top_k ? p.top_k[rq] : 0;
  const float u = p.out ? 0.f : p.u[row];
  const bool bad_args = !(temp >= 0.f && temp <= FLT_MAX) || !(top_p >= 0.f) || !(min_p >= 0.f && min_p <= 1.f) ||
                        top_k < 0 || !(u >= 0.f && u < 1.f);

  // ------------------------------------------------------------ the row, once
  // 16-byte units of the row, counted from the boundary at or before it
  const T* x = static_cast<const T*>(p.x) + (size_t)row * p.stride;
  const int lead = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const int u0 = (rank * kNW + warp) * p.units, ul = warp * p.units;  // the warp's first unit: of the row, of the slice
  const int n_units = max(0, min(p.units, (p.V + lead + E - 1) / E - u0));
  unsigned long long best = 0;  // (order key, ~index) of the largest
  bool odd = false;             // NaN or +infinity
  {
    uint4* to = const_cast<uint4*>(slice) + ul;
    float top = -INFINITY;
    int at = 0x7fffffff;
#pragma unroll 4
    for (int j = lane; j < n_units; j += 32) {
      const int i0 = (u0 + j) * E - lead;
      uint4 v;
      float f[E];
      if (i0 >= 0 && i0 + E <= p.V) {
        v = __ldcs(reinterpret_cast<const uint4*>(x + i0));
        open_unit(v, f, tag);
      } else {  // the row's first or last unit: what is not the row's counts as -infinity
        alignas(16) T e[E];
#pragma unroll
        for (int k = 0; k < E; ++k) {
          e[k] = i0 + k >= 0 && i0 + k < p.V ? x[i0 + k] : (T)(-INFINITY);
          f[k] = (float)e[k];
        }
        v = *reinterpret_cast<const uint4*>(e);
      }
      to[j] = v;
#pragma unroll
      for (int k = 0; k < E; ++k) {
        odd = odd || !(f[k] <= FLT_MAX);
        if (f[k] > top) top = f[k], at = i0 + k;
      }
    }
    best = (unsigned long long)order_key(top) << 32 | (uint32_t)~at;
  }
  int phase = 0;  // of s_part: a CTA may write the next while another reads this one
  // Every CTA's part in s_part[..][rank] of all; returns where they are.  A barrier of the cluster.
  auto tell = [&](const Part& mine) -> const Part* {  // the same value in threads 0 .. C - 1
    Part* to = s_part[phase & 1];
    ++phase;
    if (tid < C) st_remote(&to[rank], tid, mine);
    cluster_sync();
    return to;
  };
#pragma unroll
  for (int d = 16; d; d >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
  if (lane == 0) s_wv[warp] = best;
  const bool any_odd = __syncthreads_or(odd);
  {
    best = s_wv[lane % kNW];
#pragma unroll
    for (int d = kNW / 2; d; d >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const Part* all = tell(Part{0, best, 0, any_odd});
    odd = false;
    for (int r = 0; r < C; ++r) {
      best = max(best, all[r].key);
      odd = odd || all[r].flags;
    }
  }
  const uint32_t max_key = (uint32_t)(best >> 32);
  const float xmax = key_value(max_key);
  const bool leader = rank == 0;
  if (bad_args || odd || xmax == -INFINITY) {
    if (leader && tid == 0) {
      set_status(p.status, bad_args ? EAGLE_ERR_INVALID_ARG : EAGLE_ERR_NONFINITE);
      if (p.tokens) p.tokens[row] = -1;
      if (p.logprobs) p.logprobs[row] = -INFINITY;
      if (p.kept) p.kept[row] = 0;
    }
    return;
  }
  const bool greedy = temp == 0.f;
  if (greedy && !p.out) {
    if (leader && tid == 0) {
      p.tokens[row] = (int)~(uint32_t)best;
      if (p.logprobs) p.logprobs[row] = 0.f;
      if (p.kept) p.kept[row] = 1;
    }
    return;
  }
  if (tid == 0) {
    // (a temperature so small that its reciprocal overflows leaves the largest alone)
    const double c = fmin(1.4426950408889634 / (double)(greedy ? 1.f : temp), 3.0e38);
    s_ch = (float)c;
    s_cl = (float)(c - (double)s_ch);
    // w >= min_p as a border of x: the smallest fp32 number not below max + T log(min_p)
    float low = -FLT_MAX;
    if (min_p > 0.f) {
      const double b = (double)xmax + (double)temp * log((double)min_p);
      low = b <= -(double)FLT_MAX ? -FLT_MAX : __double2float_ru(b);
    }
    s_low = low;
  }
  __syncthreads();
  const Weigh weigh{xmax, s_ch, s_cl};
  const float low = s_low;
  Cut cut{0u, 0x7fffffff};
  if (greedy) cut = Cut{max_key, (int)~(uint32_t)best};

  auto weight = [&](float f) { return weigh(f, s_pow64, s_pow4096); };
  auto inside = [&](float f, int i) {  // not cut so far
    const uint32_t k = order_key(f);
    return f > -INFINITY && (k > cut.key || (k == cut.key && i <= cut.idx));
  };
  // f(value, index) for this thread's entries, in the order of indices within a lane
  auto sweep = [&](auto&& f) {
#pragma unroll 1
    for (int j = lane; j < n_units; j += 32) {
      float v[E];
      open_unit(slice[ul + j], v, tag);
      const int i0 = (u0 + j) * E - lead;
#pragma unroll
      for (int k = 0; k < E; ++k) f(v[k], i0 + k);
    }
  };
  // bin of an entry by its distance d from the maximum: 64 per octave from 2^-10 to 2^22
  auto octave_bin = [&](float f) {
    const int b = (int)(__float_as_uint(xmax - f) >> 17) - ((127 - 10) << 6);
    return min(max(b, 0), kBins - 1);
  };
  auto clear = [&]() {
    uint4* h = reinterpret_cast<uint4*>(hist_n);
    for (int i = tid; i < kBins; i += kNT) h[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
  };
  auto add = [&](int b, bool weighted, float f) {
    atomicAdd(&hist_n[b], 1u);
    if (weighted) {
      const unsigned long long w = weight(f);
      constexpr uint32_t mask = (1u << kLimb) - 1;
      const uint32_t w0 = (uint32_t)w & mask, w1 = (uint32_t)(w >> kLimb) & mask, w2 = (uint32_t)(w >> (2 * kLimb));
      if (w0) atomicAdd(&hist_w[b], w0);
      if (w1) atomicAdd(&hist_w[kBins + b], w1);
      if (w2) atomicAdd(&hist_w[2 * kBins + b], w2);
    }
  };
  // Exclusive prefixes over the threads of the CTA, and the sums over all.
  auto block_scan = [&](unsigned long long v, uint32_t n, unsigned long long& before, uint32_t& before_n,
                        unsigned long long& all, uint32_t& all_n) {
    const unsigned long long iv = warp_scan(v);
    const uint32_t in = warp_scan(n);
    __syncthreads();  // s_wv, s_wn are free
    if (lane == 31) s_wv[warp] = iv, s_wn[warp] = in;
    __syncthreads();
    unsigned long long o = 0, a = 0;
    uint32_t on = 0, an = 0;
#pragma unroll
    for (int x = 0; x < kNW; ++x) {
      if (x < warp) o += s_wv[x], on += s_wn[x];
      a += s_wv[x], an += s_wn[x];
    }
    before = o + iv - v;
    before_n = on + in - n;
    all = a;
    all_n = an;
  };
  // The bin at which the histogram's running measure (counts, or sums of weights)
  // reaches a target: before < target <= before + bin.  target(sum) gives it from
  // the sum of all; returns false where that is not reached.  Everyone calls it.
  auto find_bin = [&](bool weighted, auto&& target, unsigned long long& goal, unsigned long long& sum, Found& at) -> bool {
    cluster_sync();  // the histograms are complete
    const int nb = kBins / C, per = max(1, nb / kNT);
    unsigned long long v[kBins / kNT], mine = 0;
    uint32_t n[kBins / kNT], mine_n = 0;
#pragma unroll
    for (int i = 0; i < kBins / kNT; ++i) {
      v[i] = 0;
      n[i] = 0;
      const int b = tid * per + i;
      if (i >= per || b >= nb) continue;
      for (int r = 0; r < C; ++r) {
        const uint32_t* h = hist_n + rank * nb + b;
        n[i] += ld_remote(h, r);
        if (weighted)
          v[i] += ld_remote(h + kBins, r) + ((unsigned long long)ld_remote(h + 2 * kBins, r) << kLimb) +
                  ((unsigned long long)ld_remote(h + 3 * kBins, r) << (2 * kLimb));
      }
      if (!weighted) v[i] = n[i];
      mine += v[i];
      mine_n += n[i];
    }
    unsigned long long before, all;
    uint32_t before_n, all_n;
    block_scan(mine, mine_n, before, before_n, all, all_n);
    const Part* parts = tell(Part{all, 0, all_n, 0});
    sum = 0;
    for (int r = 0; r < C; ++r) {
      if (r < rank) before += parts[r].v, before_n += parts[r].n;
      sum += parts[r].v;
    }
    goal = target(sum);
    if (goal > sum) return false;
#pragma unroll
    for (int i = 0; i < kBins / kNT; ++i) {
      if (before < goal && goal <= before + v[i]) {
        const Found f{before, (uint32_t)(rank * nb + tid * per + i), before_n, n[i], 0};
        for (int r = 0; r < C; ++r) st_remote(&s_found, r, f);
      }
      before += v[i];
      before_n += n[i];
    }
    cluster_sync();
    at = s_found;
    return true;
  };
  auto sort_list = [&](int n) {  // the leader's list[0 .. n), by key ascending
    int n2 = 32;
    while (n2 < n) n2 <<= 1;
    for (int i = n + tid; i < n2; i += kNT) list[i] = Entry{~0ull, 0};
    __syncthreads();
    for (int k = 2; k <= n2; k <<= 1)
      for (int j = k >> 1; j; j >>= 1) {
        for (int i = tid; i < n2 / 2; i += kNT) {
          const int a = 2 * i - (i & (j - 1)), b = a + j;
          const Entry ea = list[a], eb = list[b];
          if ((ea.key > eb.key) == ((a & k) == 0)) list[a] = eb, list[b] = ea;
        }
        __syncthreads();
      }
  };
  // The entries with take(value, index), at most kCap, in this CTA's local list and
  // then all CTAs' in the leader's, best first.  Everyone calls it; the leader's
  // result is their number.
  auto gather = [&](auto&& take) -> int {
    __syncthreads();
    if (tid == 0) s_local = 0;
    __syncthreads();
    sweep([&](float f, int i) {
      if (take(f, i)) {
        const int at = atomicAdd(&s_local, 1);
        if (at < kCap) local[at] = make_uint2(order_key(f), (uint32_t)i);
      }
    });
    __syncthreads();
    const Part* parts = tell(Part{0, 0, (unsigned)min(s_local, kCap), 0});
    int n = 0;
    if (leader) {
      for (int r = 0; r < C; ++r) {
        const int m = (int)parts[r].n;
        for (int i = tid; i < m && n + i < kCap; i += kNT) {
          const uint2 e = ld_remote2(&local[i], r);
          list[n + i] = Entry{(unsigned long long)~e.x << 32 | e.y, weight(key_value(e.x))};
        }
        n = min(n + m, kCap);
      }
    }
    cluster_sync();
    if (leader) sort_list(n);
    return n;
  };
  auto entry_value = [&](const Entry& e) { return key_value(~(uint32_t)(e.key >> 32)); };
  auto finish = [&](float f, int i, unsigned long long sum, uint32_t kept) {  // one thread: the drawn token
    p.tokens[row] = i;
    if (p.kept) p.kept[row] = (int)kept;
    if (p.logprobs) {
      // -(xmax - x) / T - log(sum), the sum as 1 (the largest entry, which is always kept) and the rest
      p.logprobs[row] = -(xmax - f) / temp - log1pf((float)(sum - (1ull << kOne)) * 5.684341886080802e-14f);
    }
  };

  // ------------------------------------------------------------ top-k, top-p
  bool done = false;     // the leader has drawn the token
  bool settled = false;  // the cut is final
  const bool use_k = !greedy && top_k > 0 && top_k < p.V, use_p = !greedy && top_p < 1.f;
#pragma unroll 1
  for (int stage = 0; stage < 2 && !done && !settled; ++stage) {
    const bool by_w = stage == 1;
    if (by_w ? !use_p : !use_k) continue;
    clear();
    sweep([&](float f, int i) {
      if (inside(f, i)) add(octave_bin(f), by_w, f);
    });
    unsigned long long goal = 0, sum = 0;
    Found at;
    auto target = [&](unsigned long long s) -> unsigned long long {
      if (!by_w) return (unsigned long long)top_k;
      bool rest;  // kept while before < p s: up to the entry that reaches ceil(p s), the first at least
      const unsigned long long g = scaled(top_p, s, rest);
      return max(1ull, g + (rest ? 1 : 0));
    };
    if (!find_bin(by_w, target, goal, sum, at)) continue;  // fewer than k entries
    const int bin1 = (int)at.bin;
    if (at.before_n + at.n <= kCap) {
      // the list holds all that is kept: the leader finishes the row
      const int n = gather([&](float f, int i) { return inside(f, i) && octave_bin(f) <= bin1; });
      if (leader) {
        // each thread has two neighbours of the sorted list
        static_assert(kCap == 2 * kNT, "two entries a thread");
        unsigned long long w0, w1, before, all;
        uint32_t bn, an;
        const bool h0 = 2 * tid < n, h1 = 2 * tid + 1 < n;
        const float f0 = h0 ? entry_value(list[2 * tid]) : 0.f, f1 = h1 ? entry_value(list[2 * tid + 1]) : 0.f;
        const bool k0 = h0 && (by_w || 2 * tid < top_k), k1 = h1 && (by_w || 2 * tid + 1 < top_k);
        w0 = k0 ? list[2 * tid].w : 0;
        w1 = k1 ? list[2 * tid + 1].w : 0;
        block_scan(w0 + w1, 0, before, bn, all, an);
        unsigned long long lim = ~0ull;
        if (by_w)
          lim = goal;
        else if (use_p) {
          bool rest;
          const unsigned long long g = scaled(top_p, all, rest);
          lim = max(1ull, g + (rest ? 1 : 0));
        }
        const bool y0 = k0 && before < lim && f0 >= low, y1 = k1 && before + w0 < lim && f1 >= low;
        block_scan((y0 ? w0 : 0) + (y1 ? w1 : 0), (y0 ? 1u : 0u) + (y1 ? 1u : 0u), before, bn, all, an);
        const int m = (int)an;  // the first m of the list are kept
        if (p.out) {
          if (tid == 0) {
            const Entry e = list[m - 1];
            const Cut c{~(uint32_t)(e.key >> 32), (int)(uint32_t)e.key};
            const Found f{0, c.key, (uint32_t)c.idx, (uint32_t)m, 0};
            for (int r = 0; r < C; ++r) st_remote(&s_found, r, f);
          }
        } else {
          __syncthreads();
          for (int i = tid; i < m; i += kNT) list[i].key = list[i].key << 32 | list[i].key >> 32;  // by index
          sort_list(m);
          bool rest;
          const unsigned long long t = scaled(u, all, rest);
          const unsigned long long a = 2 * tid < m ? list[2 * tid].w : 0, b = 2 * tid + 1 < m ? list[2 * tid + 1].w : 0;
          unsigned long long s;
          block_scan(a + b, 0, before, bn, s, an);
          int hit = -1;
          if (before <= t && t < before + a) hit = 2 * tid;
          if (before + a <= t && t < before + a + b) hit = 2 * tid + 1;
          if (hit >= 0) {
            const Entry e = list[hit];
            finish(key_value(~(uint32_t)e.key), (int)(e.key >> 32), all, (uint32_t)m);
          }
        }
      }
      if (!p.out) {
        done = true;
      } else {
        cluster_sync();
        cut = Cut{s_found.bin, (int)s_found.before_n};
        settled = true;
      }
      continue;
    }
    // refine the bin: keys of its entries lie in [lo, hi], with room for the
    // rounding of the distance
    const float d0 = bin1 ? __uint_as_float((uint32_t)(bin1 + ((127 - 10) << 6)) << 17) : 0.f;
    const float d1 = bin1 < kBins - 1 ? __uint_as_float((uint32_t)(bin1 + 1 + ((127 - 10) << 6)) << 17) : INFINITY;
    const float slack = (fabsf(xmax) + d0) * 2.4e-7f;
    uint32_t hi = min(max_key, order_key(fminf(xmax - d0 + slack, FLT_MAX)));
    uint32_t lo = order_key(fmaxf(xmax - d1 - 2.f * slack, -FLT_MAX));
    unsigned long long before = at.before;
    uint32_t n_bin = at.n;
    auto member = [&](float f, int i) {
      const uint32_t k = order_key(f);
      return k >= lo && k <= hi && octave_bin(f) == bin1 && inside(f, i);
    };
    while (n_bin > kCap && lo < hi) {
      const int shift = max(0, 32 - __clz((int)(hi - lo)) - 11);
      clear();
      sweep([&](float f, int i) {
        if (member(f, i)) add((int)((hi - order_key(f)) >> shift), by_w, f);
      });
      unsigned long long s;
      auto rest = [&](unsigned long long) { return goal - before; };
      unsigned long long g;
      Found in;
      find_bin(by_w, rest, g, s, in);
      before += in.before;
      n_bin = in.n;
      const uint32_t top = hi - (in.bin << shift);
      const uint32_t width = (1u << shift) - 1;
      lo = top - lo > width ? top - width : lo;
      hi = top;
    }
    if (n_bin <= kCap) {
      const int n = gather(member);
      if (leader) {
        const unsigned long long w0 = 2 * tid < n ? (by_w ? list[2 * tid].w : 1) : 0;
        const unsigned long long w1 = 2 * tid + 1 < n ? (by_w ? list[2 * tid + 1].w : 1) : 0;
        unsigned long long b, all;
        uint32_t bn, an;
        block_scan(w0 + w1, 0, b, bn, all, an);
        b += before;
        int hit = -1;
        if (b < goal && goal <= b + w0) hit = 2 * tid;
        if (b + w0 < goal && goal <= b + w0 + w1) hit = 2 * tid + 1;
        if (hit >= 0) {
          const Entry e = list[hit];
          const Found f{0, ~(uint32_t)(e.key >> 32), (uint32_t)e.key, 0, 0};
          for (int r = 0; r < C; ++r) st_remote(&s_found, r, f);
        }
      }
      cluster_sync();
      cut = Cut{s_found.bin, (int)s_found.before_n};
    } else {
      // equal entries: the c-th by index is the last
      const unsigned long long each = by_w ? weight(key_value(lo)) : 1ull;
      const unsigned long long c = (goal - before + each - 1) / each;
      uint32_t n = 0;
      sweep([&](float f, int i) { n += member(f, i) ? 1u : 0u; });
      n = __reduce_add_sync(0xffffffffu, n);
      __syncthreads();
      if (lane == 0) s_wn[warp] = n;
      __syncthreads();
      uint32_t all = 0, off = 0;
      for (int x = 0; x < kNW; ++x) {
        if (x < warp) off += s_wn[x];
        all += s_wn[x];
      }
      const Part* parts = tell(Part{0, 0, all, 0});
      for (int r = 0; r < rank; ++r) off += parts[r].n;
      if (off < c && c <= (unsigned long long)off + n) {  // this warp's range holds it
#pragma unroll 1
        for (int j0 = 0; j0 < n_units; j0 += 32) {
          const int j = j0 + lane;
          float v[E];
          uint32_t m = 0;
          const int i0 = (u0 + j) * E - lead;
          if (j < n_units) {
            open_unit(slice[ul + j], v, tag);
#pragma unroll
            for (int k = 0; k < E; ++k) m += member(v[k], i0 + k) ? 1u : 0u;
          }
          const uint32_t in = warp_scan(m);
          uint32_t at_ = off + in - m;
          if (j < n_units && at_ < c && c <= (unsigned long long)at_ + m) {
#pragma unroll
            for (int k = 0; k < E; ++k)
              if (member(v[k], i0 + k) && ++at_ == c) {
                const Found f{0, lo, (uint32_t)(i0 + k), 0, 0};
                for (int r = 0; r < C; ++r) st_remote(&s_found, r, f);
              }
          }
          off += __shfl_sync(0xffffffffu, in, 31);
        }
      }
      cluster_sync();
      cut = Cut{s_found.bin, (int)s_found.before_n};
    }
  }
  if (done) return;

  // ------------------------------------------------------------ the whole row
  auto keep = [&](float f, int i) { return f >= low && inside(f, i); };
  if (p.out) {
    uint32_t n = 0;
    T* out = static_cast<T*>(p.out) + (size_t)row * p.out_stride;
    const bool whole = (reinterpret_cast<uintptr_t>(out) & 15u) == (reinterpret_cast<uintptr_t>(x) & 15u);
#pragma unroll 2
    for (int j = lane; j < n_units; j += 32) {
      const int i0 = (u0 + j) * E - lead;
      const uint4 raw = slice[ul + j];
      float v[E];
      open_unit(raw, v, tag);
      alignas(16) T e[E];
      *reinterpret_cast<uint4*>(e) = raw;
#pragma unroll
      for (int k = 0; k < E; ++k) {
        if (keep(v[k], i0 + k))
          ++n;
        else
          e[k] = (T)(-INFINITY);
      }
      if (whole && i0 >= 0 && i0 + E <= p.V) {
        *reinterpret_cast<uint4*>(out + i0) = *reinterpret_cast<const uint4*>(e);
      } else {
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (i0 + k >= 0 && i0 + k < p.V) out[i0 + k] = e[k];
      }
    }
    if (!p.kept) return;
    n = __reduce_add_sync(0xffffffffu, n);
    __syncthreads();
    if (lane == 0) s_wn[warp] = n;
    __syncthreads();
    uint32_t all = 0;
    for (int x = 0; x < kNW; ++x) all += s_wn[x];
    const Part* parts = tell(Part{0, 0, all, 0});
    if (leader && tid == 0) {
      for (int r = 1; r < C; ++r) all += parts[r].n;
      p.kept[row] = (int)all;
    }
    return;
  }
  unsigned long long v = 0;
  uint32_t n = 0;
  sweep([&](float f, int i) {
    if (keep(f, i)) {
      v += weight(f);
      ++n;
    }
  });
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  n = __reduce_add_sync(0xffffffffu, n);
  __syncthreads();
  if (lane == 0) s_wv[warp] = v, s_wn[warp] = n;
  __syncthreads();
  unsigned long long off = 0, all = 0;
  uint32_t all_n = 0;
  for (int x = 0; x < kNW; ++x) {
    if (x < warp) off += s_wv[x];
    all += s_wv[x];
    all_n += s_wn[x];
  }
  const Part* parts = tell(Part{all, 0, all_n, 0});
  all = 0;
  all_n = 0;
  for (int r = 0; r < C; ++r) {
    if (r < rank) off += parts[r].v;
    all += parts[r].v;
    all_n += parts[r].n;
  }
  bool rest;
  const unsigned long long t = scaled(u, all, rest);
  if (!(off <= t && t < off + v)) return;
#pragma unroll 1
  for (int j0 = 0; j0 < n_units; j0 += 32) {
    const int j = j0 + lane;
    float f[E];
    unsigned long long w[E], mine = 0;
    const int i0 = (u0 + j) * E - lead;
#pragma unroll
    for (int k = 0; k < E; ++k) w[k] = 0;
    if (j < n_units) {
      open_unit(slice[ul + j], f, tag);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        w[k] = keep(f[k], i0 + k) ? weight(f[k]) : 0;
        mine += w[k];
      }
    }
    const unsigned long long in = warp_scan(mine);
    unsigned long long at = off + in - mine;
    if (at <= t && t < at + mine) {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        if (at <= t && t < at + w[k]) finish(f[k], i0 + k, all, all_n);
        at += w[k];
      }
    }
    off += __shfl_sync(0xffffffffu, in, 31);
    if (off > t) break;
  }
}

template <typename T>
int sample_launch(SampleParams p, void* stream) {
  if (p.M == 0) return EAGLE_OK;
  const int total = (p.V + Unit<T>::E - 1) / Unit<T>::E + 1;  // and one for a start off its boundary
  int C = 1;
  while (C < kMaxCluster && total > C * kNT * 2) C *= 2;
  p.units = (total + C * kNW - 1) / (C * kNW);
  const size_t smem = 16 * kBins + 16 * (size_t)p.units * kNW;
  if (cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
    cudaGetLastError();
    return EAGLE_ERR_CUDA;
  }
  launch_cluster(sample_kernel<T>, dim3(C, p.M), dim3(kNT), dim3(C, 1, 1), smem, static_cast<cudaStream_t>(stream), p);
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
