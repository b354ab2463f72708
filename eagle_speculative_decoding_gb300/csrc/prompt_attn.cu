// Causal attention of the packed rows of many requests over the paged cache,
// in 16-bit, 32-bit or 4-bit pages.
//
// Source: "M7.5 - EAGLE Feature Drafting: Uncertainty, Dynamic Trees, HASS, and
// EAGLE-3", section 0x03C (the drafter's committed prefix) and 0x05D (rows go
// to the cache by position).
//
//   out = sum_k 2^(z_k - m) v_k / sum_k 2^(z_k - m),
//   z_k = scale log2(e) q . k_k over the keys k up to the row's position,
// for any reference m; one pass over the keys keeps m, l = sum_k 2^(z_k - m) and
// O = sum_k 2^(z_k - m) v_k in fp32 and rescales the two when m changes.  The
// weights 2^(z - m) are rounded to the operand type for the product with V (l
// sums them unrounded): bf16 for 16-bit pages, whose values bf16 holds, and
// fp16 for 4-bit pages, whose values fp16 holds exactly.
//
// bf16 rows (16- and 4-bit pages): tensor cores.  The rows of a kv head are
// the (token, grouped query head) pairs of a request in that order, so that
// all of them share the K/V a CTA stages and a row's last key moves by one
// every Hq / Hkv rows.  A unit is two tiles of up to 128 such rows of one
// request and kv head against its 128-key blocks.  Three kernels:
//   plan    one CTA lists the units from the real lengths; units longer than
//           a CTA's fair share are cut along the keys; longest pieces first
//   main    persistent CTAs take pieces from that list: the two-tile kernel
//           (one CTA per SM, tcgen05), or for single tokens the few-rows kernel
//   merge   joins the pieces of cut units (few rows: their last CTA does)
// fp32 rows: the same list and merge around a kernel on the CUDA cores.
//
// Rows that share a prefix (FLAT): the two-tile and the fp32 kernel without a plan in
// front, and a join that brings in the rows' own attention (below).
#include <float.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kv4.cuh"

namespace eagle {
namespace {

constexpr int kBlk = 128;        // keys per block
constexpr int kTileRows = 128;   // query rows per tile
constexpr int kMaxPages = 1 << 26;  // of a cache, and of a request
constexpr int kF32Rows = 64, kF32Few = 16;  // query rows per unit of the fp32 path, and when they are few
constexpr int kF32FewCtas = 2;               // CTAs per SM then
// A row's reference lies kBelow under the maximum that it is taken from, and holds
// until a block's weights add up to more than kSumLimit.  fp16 (4-bit pages) ends
// at 65504 and loses bits below 2^-14: references 7 under the maximum put those
// at 2^-21 of the largest weight and the smallest step's half at 2^-32, so that a
// long tail of small weights behind one large key still counts (with kBelow 0 and
// a limit of 256, weights under 2^-25 were zeros beside a sum that had them).
// 128 first weights add up to 2^14 at most.  bf16 keeps its 8 bits anywhere.
template <bool F16>
constexpr float kBelow = F16 ? 7.f : 0.f;
template <bool F16>
constexpr float kSumLimit = F16 ? 32768.f : 256.f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxGroups = 1024;  // that share prefixes

struct AttnParams {
  const void* q;
  long long q_stride;
  const void *kc, *vc;     // 4-bit: the codes
  const uint8_t *ks, *vs;  // 4-bit: the scales
  float k_scale, v_scale;
  int num_pages, max_pages, B, T, Hq, Hkv;
  const int32_t *table, *cu, *ctx;
  void* out;
  float* lse;
  float scale;
  int32_t* status;
};

// ------------------------------------------------------------------- plan
// A piece: key blocks [k0, k1) of unit u of (request b, kv head h); slot >= 0
// when the unit is cut (its partial result goes there).
struct __align__(16) Piece {
  int b, h, u, k0, k1, slot, c0, n, ctx;
  int cut, first, pieces;  // of a cut unit: its index, its pieces' first slot and their number
};
struct __align__(16) Cut {  // a cut unit: its pieces are slots slot .. slot + pieces - 1
  int h, u, slot, pieces, c0, n;
  int done, pad;  // pieces whose results are written (few rows)
};
struct PlanHeader {
  int pieces, cuts, next, most;  // most: pieces of the most cut unit
};

constexpr int kCand = 6;       // candidate cuts of the plan
constexpr int kMaxShare = 6;   // pieces per CTA at the finest cut
// In sixteenths of a piece per CTA (0: no unit is cut); a little under whole
// numbers, so that rounding a unit's pieces up does not start another wave.
__device__ __constant__ const int kShares[kCand] = {0, 14, 29, 45, 62, 96};

struct Shape {
  int g, tpt, tpu, rows;  // heads per kv head, tokens per tile and unit, rows per slot
  int ctas, cap_units, cap_pieces, cap_slots;
  size_t off_pieces, off_cuts, off_ml, off_o, total;
};
// CTAs per SM of the few-rows kernel with NG groups of eight rows: as many as
// the registers allow (4-bit, one group: 4 CTAs 62 us, 3 71 us, 5 69 us)
constexpr int few_ctas(bool kv4, int ng) { return kv4 ? (ng == 1 ? 4 : 3) : 2; }
enum Path { kTensor, kFew, kFew4, kFp32, kFp32Few };
Shape attn_shape(int B, int T, int Hq, int Hkv, int D, Path path) {
  Shape s;
  s.g = Hq / Hkv;
  s.tpt = path == kTensor ? kTileRows / s.g : path == kFp32 ? kF32Rows / s.g : path == kFp32Few ? std::max(1, kF32Few / s.g) : 1;
  s.tpu = path == kTensor ? 2 * s.tpt : s.tpt;
  s.rows = std::min(s.tpu, T) * s.g;
  const int sms = sm_count();
  s.ctas = (sms > 0 ? sms : 152) * (path == kFew4 || path == kFew ? few_ctas(path == kFew4, s.g > 8 ? 2 : 1) : path == kFp32Few ? kF32FewCtas : 1);
  s.cap_units = T / s.tpu + std::min(B, T);
  // a unit of L > C blocks makes ceil(L / C) < 2 L / C pieces and the finest C
  // is total / (kMaxShare * ctas)
  s.cap_slots = 2 * kMaxShare * s.ctas;
  s.cap_pieces = s.cap_units * Hkv + s.cap_slots;
  s.off_pieces = 256;
  s.off_cuts = round_up(s.off_pieces + sizeof(Piece) * (size_t)s.cap_pieces, 256);
  s.off_ml = round_up(s.off_cuts + sizeof(Cut) * (size_t)s.cap_slots, 256);
  s.off_o = round_up(s.off_ml + sizeof(float2) * (size_t)s.cap_slots * s.rows, 256);
  s.total = s.off_o + sizeof(float) * (size_t)s.cap_slots * s.rows * D + 256;
  return s;
}
// Single tokens take the few-rows kernel, everything else the two-tile kernel.
// The host does not know the lengths, so the rule goes by their mean, and a
// batch of unlike requests has one kernel for all of them.  What that costs, us,
// 32 heads over 8, D 128, one call from a cold L2: a chunk of 512 rows beside 63
// single tokens 158 on 16-bit pages (the parts alone 67 and 133) and 198 on 4-bit
// (97 and 74); a chunk of 60 rows among 63 empty requests 70 on 16-bit pages, where
// each row reads the whole context (30 as a call of its own), 43 on 4-bit (58).
// Requests of one kind, us,
// few rows / two tiles, 64 requests over 1024 .. 4096 keys, D 128:
//   16-bit, 32 heads over 8: 1 token 121 / 130, 2 tokens 195 / 131;
//     64 over 8: 122 / 130; 64 over 4 (16 rows): 84 / 76
//   4-bit, 32 over 8: 1 token 62 / 140, 2 tokens 88 / 143, 3 tokens 121 / 143,
//     4 tokens 159 / 146; 64 over 4: 1 token 50 / 86, 2 tokens 89 / 90, 3 tokens 99 / 97
bool few_rows(bool kv4, int B, int T, int Hq, int Hkv) {
  return kv4 ? T <= 2 * B && Hq / Hkv <= 16 : T <= B && Hq / Hkv <= 8;
}
// fp32: at most 16 rows per request and kv head on average take units of 16.
// us, 16 / 64 rows a unit, 32 heads over 8, D 128, 64 requests over 1024 ..
// 4096 keys: 1 to 4 tokens 800 / 1,200, 6 tokens 1,680 / 985; 8 heads of 16
// requests over 300 .. 500 keys, D 64: 16 tokens 36 / 48, 20 tokens 57 / 40.
bool few_rows_f32(int B, int T, int Hq, int Hkv) {
  return Hq / Hkv <= kF32Few && (long long)T * (Hq / Hkv) <= (long long)kF32Few * B;
}

struct PlanParams {
  const int32_t *cu, *ctx;
  int B, T, Hkv, max_pages, tpu, g, ctas, cap_pieces, cap_slots;
  int min_cut, min_cut_short;  // blocks of a piece at least; the latter if no unit has over 16 blocks
  PlanHeader* hdr;
  Piece* pieces;
  Cut* cuts;
  int32_t* status;
};

constexpr int kPlanThreads = 512;

// One CTA.  The requests are taken 512 at a time (up to that many are loaded
// once): a block scan of their unit counts, then every thread finds the request
// of its units by bisection.  Sweeps over all units: the total of key blocks,
// the cost of each candidate cut, the lengths' histogram, and the list.  It is
// bound by its chain of block-wide steps: 8.5 us from cold caches for one
// prompt, 12.7 us for 64 requests cut into some 1,700 pieces.
__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const PlanParams p) {
  __shared__ unsigned long long s_total;
  __shared__ int s_longest, s_C[kCand], s_n[kCand], s_cut[kCand], s_hist[32], s_cursor[32], s_c, s_slots, s_cuts, s_most, s_falls;
  __shared__ int s_c0[kPlanThreads], s_len[kPlanThreads], s_ctx[kPlanThreads], s_end[kPlanThreads], s_warp[kPlanThreads / 32];
  struct Unit {
    int at, k, slot, cut, o, u, len, extra;
  };
  __shared__ Unit s_unit[kPlanThreads];
  __shared__ int s_pend[kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 32) s_hist[tid] = 0;
  if (tid < kCand) s_n[tid] = s_cut[tid] = 0;
  if (tid == 0) {
    s_total = 0;
    s_longest = s_slots = s_cuts = s_most = s_falls = 0;
  }
  pdl_wait();
  pdl_trigger();

  // requests base .. base + 511 into shared memory; s_end: inclusive prefix of their units
  auto load = [&](int base, bool report) {
    int c0 = 0, n = 0, ctx = 0;
    bool falls = false;
    const int b = base + tid;
    if (b < p.B) {
      c0 = p.cu[b];
      const int c1 = p.cu[b + 1];
      ctx = p.ctx[b];
      n = c1 - c0;
      falls = c1 < c0;
      if (c0 < 0 || falls || c1 > p.T || ctx < 0) {
        if (report) set_status(p.status, EAGLE_ERR_INVALID_ARG);
        n = 0;
      } else if ((long long)ctx + n > 16ll * p.max_pages) {
        if (report) set_status(p.status, EAGLE_ERR_BAD_KV);
        n = 0;
      }
      // rows in front of the first request or behind the last belong to none
      if (report && ((b == 0 && c0 != 0) || (b == p.B - 1 && c1 != p.T))) set_status(p.status, EAGLE_ERR_INVALID_ARG);
    }
    int end = (n + p.tpu - 1) / p.tpu;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, end, d);
      if (lane >= d) end += x;
    }
    if (lane == 31) s_warp[warp] = end;
    // where cu_seqlens falls, requests may claim the same rows again and again:
    // no room is laid out for that, and nothing is listed
    if (__syncthreads_or(falls) && tid == 0) s_falls = 1;
    int before = lane < warp ? s_warp[lane] : 0;  // warps are fewer than lanes
    before = (int)__reduce_add_sync(0xffffffffu, (unsigned)before);
    s_c0[tid] = c0;
    s_len[tid] = n;
    s_ctx[tid] = ctx;
    s_end[tid] = end + before;
    __syncthreads();
  };
  const bool once = p.B <= kPlanThreads;
  if (once) load(0, true);

  // unit i of the loaded requests: its request's place o, its index u there; returns its key blocks
  auto find = [&](int i, int& o, int& u) -> int {
    o = 0;  // the first request with s_end > i
#pragma unroll
    for (int d = kPlanThreads / 2; d; d >>= 1)
      if (s_end[o + d - 1] <= i) o += d;
    const int n = s_len[o];
    u = i - (s_end[o] - (n + p.tpu - 1) / p.tpu);
    return (s_ctx[o] + min(n, (u + 1) * p.tpu) + kBlk - 1) / kBlk;
  };
  // f(live, key blocks) for every unit: whole warps call it, `live` lanes have one
  auto sweep = [&](bool report, auto&& f) {
#pragma unroll 1
    for (int base = 0; base < p.B; base += kPlanThreads) {
      if (!once) {
        __syncthreads();
        load(base, report);
      }
      const int total = s_end[kPlanThreads - 1];
#pragma unroll 1
      for (int i0 = warp * 32; i0 < total; i0 += kPlanThreads) {
        int o, u;
        f(i0 + lane < total, find(min(i0 + lane, total - 1), o, u));
      }
    }
  };

  {
    unsigned sum = 0;  // of this lane's units: below 2^32 key blocks
    int longest = 0;
    sweep(true, [&](bool live, int L) {
      if (!live) return;
      sum += (unsigned)L;
      longest = max(longest, L);
    });
    longest = __reduce_max_sync(0xffffffffu, longest);
    unsigned long long all = sum;
#pragma unroll
    for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
    if (lane == 0 && longest) {
      atomicAdd(&s_total, all);
      atomicMax(&s_longest, longest);
    }
  }
  __syncthreads();
  if (s_falls) {
    if (tid == 0) *p.hdr = PlanHeader{0, 0, p.ctas, 0};
    return;
  }
  const long long all = (long long)s_total * p.Hkv;  // key blocks of all units
  const int longest = s_longest;
  // candidate x cuts units longer than C_x = all / (share x ctas)
  if (tid < kCand) {
    const long long f = (long long)kShares[tid] * p.ctas;
    s_C[tid] = f ? (int)max((long long)(longest > 16 ? p.min_cut : p.min_cut_short), (16 * all + f - 1) / f) : 0x7fffffff;
  }
  __syncthreads();
  {
    int C[kCand], n[kCand], cut[kCand];
#pragma unroll
    for (int x = 0; x < kCand; ++x) {
      C[x] = s_C[x];
      n[x] = cut[x] = 0;
    }
    sweep(false, [&](bool live, int L) {
      if (!live) return;
#pragma unroll
      for (int x = 0; x < kCand; ++x) {
        const int k = L > C[x] ? (L + C[x] - 1) / C[x] : 1;
        n[x] += k;
        cut[x] += k > 1 ? k : 0;
      }
    });
#pragma unroll
    for (int x = 0; x < kCand; ++x) {
      const int a = __reduce_add_sync(0xffffffffu, n[x]), b = __reduce_add_sync(0xffffffffu, cut[x]);
      if (lane == 0 && a) {
        atomicAdd(&s_n[x], a);
        atomicAdd(&s_cut[x], b);
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    // estimated time in blocks per CTA: whole waves of pieces of the mean
    // length (at least the longest piece), and for each cut piece its
    // partial result (a block's worth of traffic per 64 rows, written and
    // read) and a block for its start; a lane per candidate, the least wins
    // (the lower candidate of equals)
    const int x = min(lane, kCand - 1), C = s_C[x];
    const float per_cut = 1.f + (float)min(p.tpu, p.T) * (float)p.g / 64.f;
    const float N = (float)s_n[x] * p.Hkv;
    float t = 3e38f;
    if (lane < kCand && N >= 1.f && (long long)s_cut[x] * p.Hkv <= p.cap_slots)
      t = fmaxf(ceilf(N / p.ctas) * ((float)all / N), (float)min(longest, C)) + (float)s_cut[x] * p.Hkv * per_cut / p.ctas;
    const unsigned best = __reduce_min_sync(0xffffffffu, __float_as_uint(t));  // non-negative: ordered as integers
    const int who = __ffs(__ballot_sync(0xffffffffu, __float_as_uint(t) == best)) - 1;
    if (lane == who) s_c = C;
  }
  __syncthreads();
  const int C = s_c, top = max(1, min(longest, C));
  const float per_class = 32.f / (float)top;
  auto klass = [&](int len) { return 31 - min(31, (int)((float)(len - 1) * per_class)); };  // 0: the longest
  sweep(false, [&](bool live, int L) {
    if (!live) return;
    const int k = L > C ? (L + C - 1) / C : 1;
    atomicAdd(&s_hist[klass((L + k - 1) / k)], k * p.Hkv);
  });
  __syncthreads();
  if (warp == 0) {
    const int v = s_hist[lane];
    int end = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, end, d);
      if (lane >= d) end += x;
    }
    s_cursor[lane] = end - v;
    if (lane == 31) {
      p.hdr->pieces = min(end, p.cap_pieces);
      p.hdr->next = p.ctas;  // the first piece of each CTA is its own index
    }
  }
  __syncthreads();
  // the list: 512 units at a time into shared memory, then their pieces over
  // all threads, each finding its unit by bisection
#pragma unroll 1
  for (int base = 0; base < p.B; base += kPlanThreads) {
    if (!once) {
      __syncthreads();
      load(base, false);
    }
    const int total = s_end[kPlanThreads - 1];
#pragma unroll 1
    for (int i0 = 0; i0 < total; i0 += kPlanThreads) {
      int k = 0;
      if (i0 + tid < total) {
        int o, u;
        const int L = find(i0 + tid, o, u);
        k = 1;
        int slot = -1, cut = 0, len = L, extra = 0;  // the first `extra` pieces have len + 1 blocks
        if (L > C) {
          k = (L + C - 1) / C;
          len = L / k;
          extra = L - len * k;
          slot = atomicAdd(&s_slots, k * p.Hkv);
          cut = atomicAdd(&s_cuts, p.Hkv);
          atomicMax(&s_most, k);
        }
        s_unit[tid] = Unit{atomicAdd(&s_cursor[klass((L + k - 1) / k)], k * p.Hkv), k, slot, cut, o, u, len, extra};
      }
      int end = k * p.Hkv;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, end, d);
        if (lane >= d) end += x;
      }
      if (lane == 31) s_warp[warp] = end;
      __syncthreads();
      const int before = (int)__reduce_add_sync(0xffffffffu, (unsigned)(lane < warp ? s_warp[lane] : 0));
      s_pend[tid] = end + before;
      __syncthreads();
      const int pieces = s_pend[kPlanThreads - 1];
      for (int q = tid; q < pieces; q += kPlanThreads) {
        int i = 0;  // the first unit with s_pend > q
#pragma unroll
        for (int d = kPlanThreads / 2; d; d >>= 1)
          if (s_pend[i + d - 1] <= q) i += d;
        const Unit w = s_unit[i];
        const int j = q - (s_pend[i] - w.k * p.Hkv), h = w.k > 1 ? j / w.k : j, x = j - h * w.k;
        const int k0 = x * w.len + min(x, w.extra), c0 = s_c0[w.o], n = s_len[w.o];
        // (the list has room for every cu_seqlens that does not fall; this is for
        // one that is overwritten during the call)
        if ((unsigned)(w.at + j) < (unsigned)p.cap_pieces)
          p.pieces[w.at + j] = Piece{base + w.o, h, w.u, k0, k0 + w.len + (x < w.extra ? 1 : 0), w.k > 1 ? w.slot + j : -1,
                                     c0, n, s_ctx[w.o], w.cut + h, w.slot + h * w.k, w.k};
        if (w.k > 1 && x == 0) p.cuts[w.cut + h] = Cut{h, w.u, w.slot + j, w.k, c0, n, 0, 0};
      }
      __syncthreads();
    }
  }
  __syncthreads();
  if (tid == 0) {
    p.hdr->cuts = s_cuts;
    p.hdr->most = s_most;
  }
}

// ---------------------------------------------------------- shared prefixes
// FLAT kernels: attention of groups of rows over a prefix that the group shares
// (B groups, cu their rows, ctx their prefix's keys, table its pages), every key
// visible to every row.  A unit's key blocks are all known from a group's two
// numbers, so nothing is planned in front: the blocks of all units (by group, kv
// head and unit) are one line, of which CTA c takes blocks c per .. c per + per - 1,
// and each CTA finds its own part.  Where the units are few, `per` is such that
// units, rounded up to a multiple of it, have a CTA for every part, and no CTA has
// parts of two units (a second piece's start costs 3 us: its pages, keys and rows
// are only then known).
// A unit that lies in one CTA's part is finished there; of the others each CTA
// leaves a partial result (slot 2 c + 1 for the piece that a unit starts with, at
// most one per CTA, 2 c for one that it goes on with), and the CTA that it starts in
// describes it to flat_join_kernel, which joins them.
//
// What bounds it (32 + 8 heads, D 128, in a graph): few rows, the chain of a start and
// two key blocks a CTA, and the join behind it: 64 tokens over 8,000 keys 20 us, of which
// the pieces are known after 1.6, S of the first block after 3.6, a block takes 2, the
// last piece ends at 13 and the join takes 5 (the plan and merge of eagle_prompt_attn
// would be 12 in front and behind; the keys' bytes are 5 us).  4 tokens over 32,768 keys
// 36 us, 3.8 TB/s.  Many rows, the chain S - softmax - P V: 1,885 rows of two
// groups over 3,808 and 4,333 keys 128 us, 0.98 PFLOP/s (main kernel 115 from a cold L2,
// join 24, of which half shows).
struct __align__(16) Split {  // a unit that starts in a CTA's part and ends in CTA `last`'s
  int rows, last, h, tok0;   // rows: 0 if there is none
};
// (A part has one block at least.  With two at least, calls of 300 to 1,000 keys and
// up to 128 tokens took 0.3 to 2 us more; only units of two blocks, which nobody joins
// then, 1.2 less.)
// By how many blocks a part may grow for whole units.  32 + 8 heads, D 128, 3 / none:
// 64 and 256 tokens over 2,400 keys 15.9 / 17.5 and 26 / 28.5 us, 1,024 over 2,000
// 41 / 55; with 8, 1,024 over 4,800 is 76 and not 86, but 400 over 8,000 71 and not 64.
constexpr int kFlatMore = 3;
struct Groups {  // a warp's view: lane i holds group base + i (of one group, all lanes have it)
  int c0, n, len;     // first row, rows, keys (0 if the group is in error)
  int units, blocks;  // units: of all kv heads
  bool falls;
};
__device__ __forceinline__ Groups load_groups(const AttnParams& a, int base, int tpu, bool report) {
  Groups g = {0, 0, 0, 0, 0, false};
  const int i = a.B == 1 ? 0 : base + (int)(threadIdx.x & 31);
  if (i >= a.B) return g;
  g.c0 = a.cu[i];
  const int c1 = a.cu[i + 1], len = a.ctx[i];
  g.falls = c1 < g.c0;
  if (g.c0 < 0 || g.falls || c1 > a.T || len < 0) {
    if (report) set_status(a.status, EAGLE_ERR_INVALID_ARG);
  } else if (len > 16ll * min(a.max_pages, kMaxPages)) {
    if (report) set_status(a.status, EAGLE_ERR_BAD_KV);
  } else {
    g.n = c1 - g.c0;
    g.len = len;
    g.units = (g.n + tpu - 1) / tpu * a.Hkv;
    g.blocks = (len + kBlk - 1) / kBlk;
  }
  // rows in front of the first group or behind the last belong to none
  if (report && ((i == 0 && g.c0 != 0) || (i == a.B - 1 && c1 != a.T))) set_status(a.status, EAGLE_ERR_INVALID_ARG);
  return g;
}
// a / b, 0 <= a < 2^24, 0 < b: the quotient of floats, put right by the remainder
__device__ __forceinline__ int quotient(int a, int b) {
  const int q = (int)__fdividef((float)a, (float)b), r = a - q * b;
  return q + (r >= b ? 1 : 0) - (r < 0 ? 1 : 0);
}
__device__ __forceinline__ long long quotient(long long a, int b) {
  return a < (1 << 24) && b < (1 << 24) ? quotient((int)a, b) : a / b;
}
// The sum of f(group) over all groups; one warp calls it.
template <typename F>
__device__ __forceinline__ long long sum_groups(const AttnParams& a, int tpu, const Groups& first, F&& f) {
  if (a.B == 1) return f(first);
  long long v = f(first);
  for (int base = 32; base < a.B; base += 32) v += f(load_groups(a, base, tpu, false));
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
// A CTA's part, piece by piece; one warp has it.
struct FlatWalk {
  int per;         // blocks of a part
  bool snap;       // units are rounded up to whole parts
  long long left;  // blocks still to be given out
  int base, src, h, u, k;
  Groups g;
  __device__ __forceinline__ int take(int x) const { return __shfl_sync(0xffffffffu, x, src); }
  __device__ __forceinline__ long long line(const Groups& x) const {  // a group's stretch of it
    return (long long)x.units * (snap ? (x.blocks + per - 1) / per * per : x.blocks);
  }
  __device__ __forceinline__ void start(const AttnParams& a, int tpu, bool report) {
    const int ctas = (int)gridDim.x;
    g = load_groups(a, 0, tpu, report);
    left = 0;
    per = 1;
    snap = false;
    bool falls = g.falls;
    if (a.B > 1) {
      for (base = 32; base < a.B; base += 32) falls = load_groups(a, base, tpu, report).falls || falls;
      falls = __any_sync(0xffffffffu, falls);
    }
    if (falls) return;  // rows might have two prefixes: nothing is done
    const int limit = 1 << 23;
    if (a.B == 1 && g.units < limit && g.blocks < limit && (long long)g.units * g.blocks < limit) {
      // one group and a short line, as in most calls: the same in plain ints (a CTA's
      // first loads wait for this: 0.9 us the other way)
      const int units = g.units, blocks = g.blocks, all = units * blocks;
      const int even = max(1, quotient(all + ctas - 1, ctas));
      per = even;
      int parts = 0;
      for (int more = 0; more <= kFlatMore && !snap; ++more) {
        parts = quotient(blocks + even + more - 1, even + more);
        if (units * (long long)parts <= ctas) snap = true, per = even + more;
      }
      base = src = 0;
      const int c = (int)blockIdx.x, at = c * per;
      if (snap ? c >= units * parts : at >= all) return;
      const int unit = snap ? quotient(c, parts) : quotient(at, blocks);
      k = snap ? (c - unit * parts) * per : at - unit * blocks;
      const int of_head = units / a.Hkv;
      h = of_head == 1 ? unit : quotient(unit, of_head);
      u = unit - h * of_head;
      left = snap ? min(per, blocks - k) : min(per, all - at);
      return;
    }
    const long long all = sum_groups(a, tpu, g, [](const Groups& x) { return (long long)x.units * x.blocks; });
    const int even = (int)max(1ll, quotient(all + ctas - 1, ctas));  // (lines of 2^31 blocks would be 2^38 keys)
    per = even;
    for (int more = 0; more <= kFlatMore && !snap; ++more) {
      const int p = even + more;
      snap = sum_groups(a, tpu, g, [&](const Groups& x) { return x.units * quotient((long long)x.blocks + p - 1, p); }) <= ctas;
      if (snap) per = p;
    }
    long long at = (long long)blockIdx.x * per;
    base = src = 0;
    if (a.B == 1) {
      if (at >= line(g)) return;
    } else {
      for (;; base += 32) {
        if (base >= a.B) return;
        if (base) g = load_groups(a, base, tpu, false);
        const long long mine = line(g);
        long long end = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, end, d);
          if ((int)(threadIdx.x & 31) >= d) end += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, end > at);
        if (past) {
          src = __ffs((int)past) - 1;
          at -= __shfl_sync(0xffffffffu, end - mine, src);
          break;
        }
        at -= __shfl_sync(0xffffffffu, end, 31);
      }
    }
    const int blocks = take(g.blocks), units = take(g.units), len = snap ? (blocks + per - 1) / per * per : blocks;
    const int unit = (int)quotient(at, len), of_head = units / a.Hkv;  // (at: within the group)
    k = (int)(at - (long long)unit * len);
    h = (int)quotient((long long)unit, of_head);
    u = unit - h * of_head;
    left = snap ? min(per, blocks - k) : min((long long)per, all - (long long)blockIdx.x * per);
  }
  __device__ __forceinline__ bool next(const AttnParams& a, int tpu, Piece& w) {
    if (left <= 0) return false;
    const int blocks = take(g.blocks), n = take(g.n);
    const int k1 = (int)min((long long)blocks, k + left), c = (int)blockIdx.x;
    w = Piece{base + src, h, u, k, k1, k1 - k == blocks ? -1 : 2 * c + (k == 0 ? 1 : 0), take(g.c0), n, take(g.len), 0, 0, 1};
    left -= k1 - k;
    k = 0;
    if (left > 0 && ++u * tpu >= n) {
      u = 0;
      if (++h == a.Hkv) {
        h = 0;
        unsigned more = a.B == 1 ? 0u : __ballot_sync(0xffffffffu, g.blocks > 0 && g.units > 0) & (src == 31 ? 0u : ~0u << (src + 1));
        while (!more) {  // (blocks are left, so some later group has them)
          base += 32;
          if (base >= a.B) {
            left = 0;
            return true;
          }
          g = load_groups(a, base, tpu, false);
          more = __ballot_sync(0xffffffffu, g.blocks > 0 && g.units > 0);
        }
        src = __ffs((int)more) - 1;
      }
    }
    return true;
  }
  // what the join needs of the part's last piece w, whose unit may go on in the next parts
  __device__ __forceinline__ Split split(const Piece& w, int tpu, int of_token) const {
    Split s = {0, 0, 0, 0};
    if (w.slot < 0 || w.k0 > 0) return s;
    s.rows = min(tpu, w.n - w.u * tpu) * of_token;
    s.last = (int)blockIdx.x + 1 + ((w.ctx + kBlk - 1) / kBlk - w.k1 - 1) / per;
    s.h = w.h;
    s.tok0 = w.c0 + w.u * tpu;
    return s;
  }
};
// A row's own keys as one more term of its sums: their log-sum-exp L becomes the
// weight 2^(L log2(e) - M) beside the prefix's sum l 2^(m - M), M the larger of the two
// references.  L log2(e) is kept in two parts (as one it is off by 2^-24 of itself,
// which is 2^-20 of a weight).  A side whose weight is zero does not count, whatever its
// values are: with `prefix` 0 the own result is left as it is.
struct OwnWeight {
  float prefix, own, lse;  // factors of O and of own_out, and the joined log-sum-exp
  __device__ __forceinline__ float of_prefix(float o, float by) const { return prefix == 0.f ? 0.f : o * by; }
};
__device__ __forceinline__ OwnWeight own_weight(float m, float l, float L) {
  if (l == 0.f) return {0.f, L == -INFINITY ? 0.f : 1.f, L};  // the own result as it is
  const float hi = L * 1.44269502f, lo = fmaf(L, 1.44269502f, -hi) + L * 1.92596303e-8f, M = fmaxf(m, hi);
  // (past fp32's range, as for a mask of the type's lowest value: nothing beside the other side)
  if (isinf(hi)) return hi < 0.f ? OwnWeight{1.f / l, 0.f, (m + log2f(l)) * kLn2} : OwnWeight{0.f, 1.f, L};
  const float p = ex2_approx(m - M), o = ex2_approx((hi - M) + lo), total = fmaf(l, p, o), f = 1.f / total;
  if (l * p == 0.f) return {0.f, 1.f, L};
  return {p * f, o * f, (M + log2f(total)) * kLn2};
}

// ------------------------------------------------------------------- main
// 512 threads, one CTA per SM:
//   warps 0-3    K/V producers: 16-byte asynchronous copies from the pages to
//                128-byte-swizzled stages (16 tokens of a page are 16 rows
//                Hkv D apart: copies by threads reach what boxes of a tensor
//                map, 2 KB each, do not), or, for 4-bit pages, copies of
//                the codes to a raw ring and from there exact fp16 values to
//                the stages
//   warps 4, 5   issue the MMAs of tile 0 and 1
//   warp 6       takes pieces from the list, ahead of the others
//   warp 7       loads Q: TMA boxes of tokens x grouped heads, or, for 4-bit
//                pages, whose MMAs are fp16, loads and converts it
//   warps 8-11   softmax of tile 0, warps 12-15 of tile 1: a thread is a row
//                (a TMEM lane) and holds the block's 128 scores
// S of a tile (fp32, 128 columns), its weights P (16-bit, over S) and O (D
// columns) live in TMEM; P is the A operand of P V from there.  Per tile the
// issuing warp issues P V(i), then S(i + 1): while one tile's softmax runs, the
// other tile's MMAs do.  S(i + 1) follows P V(i) in the pipe, so that the
// softmax that sees S(i + 1) complete may rescale O.
// A unit of at most 128 rows (single tokens, short chunks) would leave one
// tile idle and the chain S - softmax - P V exposed: then both tiles hold the
// same rows, tile 0 takes the even blocks and tile 1 the odd ones, and tile
// 0's warps join the two at the end (same TMEM lanes).
//
// Bound by each tile's chain S - softmax - P V: about 3,300 cycles per block
// and two tiles (D 128), while the MMAs take 2,048 and the exponentials, at 32
// a cycle and SM, 1,024 beside them.  Causal FLOPs at
// 64 heads over 8, 8192 tokens: 830 us, 1.32 PFLOP/s; chunks of 256 .. 512
// tokens over 32k keys, 32 over 8: 656 us, 1.21 PFLOP/s; one prompt of 2048
// tokens: 50-56 us.  On 4-bit pages the producers' conversions take issue slots
// from the softmax: chunks over 8k keys 272 us, 205 us on 16-bit pages.
constexpr int kThreads = 512;
constexpr int kSlots = 4;  // pieces known ahead
constexpr int kNoPage = -0x7fffffff - 1;  // past the keys (or found out of range): reads as zeros

template <int D, bool KV4>
struct Cfg {
  static constexpr uint32_t kHalf = kTileRows * 128u;        // 64 columns of 128 rows
  static constexpr uint32_t kTile = kHalf * (D / 64);         // one Q, K or V tile
  static constexpr int kStages = KV4 ? (D == 128 ? 4 : 6) : (D == 128 ? 5 : 8);
  static constexpr uint32_t kRawCodes = kBlk * D / 2, kRaw = kRawCodes + kBlk * D / 16;
  static constexpr int kRawRing = 3;
  static constexpr uint32_t kSmem = 2 * kTile + kStages * kTile + (KV4 ? kRawRing * kRaw : 0) + 1024;
  static constexpr uint32_t kColO = 256;  // S of tile t at t * 128, O at kColO + t * D
};

struct MainParams {
  AttnParams a;
  float scale_log2;
  int g, tpt, tpu, slot_rows;
  const PlanHeader* hdr;
  int* next;
  const Piece* pieces;
  float2* part_ml;
  float* part_o;
  const void* own_out;  // FLAT: what the rows' own keys gave, or null
  const float* own_lse;
  Split* splits;  // one per CTA
};

template <int ST, bool KV4>
struct Bars {
  uint64_t kv_full[ST], kv_empty[ST], q_full[2], q_empty[2], o_full[2], x_stat, x_back, x_done, s_full[2];
  uint64_t turn[2][4];  // by tile and quarter: the other tile's softmax has done its block
  uint64_t p_full[2];
  uint64_t slot_full[kSlots], slot_empty[kSlots], drain[2];
  uint32_t tmem_base;
  int abort_flag;
  Piece piece[kSlots];      // b < 0: no more work
  int bad_v[kSlots];        // a masked block of the piece holds non-finite values
  float q_fac[2][2][KV4 ? kTileRows : 1];  // 4-bit: the rows' powers of two, by a tile's use parity and tile
  float2 x_ml[kTileRows];
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// This thread's arrival on `bar` once all its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}
// at most n (0 .. 2) of the newest groups may still be in flight
__device__ __forceinline__ void cp_async_wait_n(int n) {
  switch (n) {
    case 0: cp_async_wait<0>(); break;
    case 1: cp_async_wait<1>(); break;
    default: cp_async_wait<2>(); break;
  }
}
// The bounded wait of this file's kernel: a failed try suspends the thread for
// about 4 us, so 2^19 of them are the 2 s of mbar_wait, without its clock
// reads (some thirty waits are in line here, and the roles share an
// instruction cache).
__device__ __forceinline__ bool mbar_wait_short(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (int i = 0; i < (1 << 19); ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = 1;
  return false;
}
// 1 in one lane of the converged warp, 0 in the others.  MMAs are predicated
// on it: a predicate by elect.sync lets the compiler issue them once (64.5
// cycles per M 128 N 128 K 16, the tensor core's own rate, 10-30 to issue),
// any other predicate or a one-lane branch makes it loop over the lanes
// (100-135 cycles per MMA, 65-82 to issue).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// MMAs and commits predicated on `one` (elect_one).
// D += A B, both operands in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(one)
      : "memory");
}
// The same with A in tensor memory (16 keys = 8 columns of pairs).
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                       bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(one)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t one, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(one)
      : "memory");
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Stores 16 fp32 columns of this warp's 32 TMEM lanes (complete after tmem_wait_st()).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
template <int N, bool INC>
__device__ __forceinline__ void set_max_regs() {
  if (INC)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 4-bit pages: a row of q goes to fp16 divided by 2^row_exponent, which brings
// its largest magnitude (the bits `mx` of a bf16) to [1, 2); 0 for a row of zeros.
__device__ __forceinline__ int row_exponent(uint32_t mx) {
  return mx ? min(126, max(-126, (int)(mx >> 7) - 127)) : 0;
}
// What its scores are then multiplied by: never 0, which would make NaN of a
// masked score (no score of a row with a factor this small leaves a weight of 1),
// and never infinite, which would make NaN of a score of 0.
__device__ __forceinline__ float row_factor(float scale_log2, float power) {
  return fminf(fmaxf(scale_log2 * power, 1.17549435e-38f), 3.40282347e38f);
}

// Eight 4-bit codes as four fp16 pairs times the pair `s`.
__device__ __forceinline__ void kv4_expand(uint32_t w, uint32_t s, uint32_t* v) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
#pragma unroll
  for (int y = 0; y < 4; ++y)  // exact: at most six significant bits, all multiples of 2^-10
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(v[y]) : "r"(s));
}
__device__ __forceinline__ uint32_t e4m3_pair_as_f16(uint32_t two) {
  uint32_t s2;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(s2) : "r"(two));
  return s2;
}

// Blocks of a piece that tile t takes, and the block its i-th one is.
struct TileWork {
  int rows0, rows1;  // valid rows of the tiles
  int n0, n1;        // blocks of the tiles
  bool twin;         // both tiles hold the same rows and take alternate blocks
  __device__ __forceinline__ int n(int t) const { return t ? n1 : n0; }
  __device__ __forceinline__ int rows(int t) const { return t ? rows1 : rows0; }
  __device__ __forceinline__ int blk(int t, int i) const { return twin ? 2 * i + t : i; }
};
template <bool FLAT>
__device__ __forceinline__ TileWork tile_work(const Piece& w, int tpt, int tpu, int g) {
  TileWork r;
  const int t0 = w.u * tpu, left = FLAT ? min(w.n - t0, tpu) : w.n - t0, nblk = w.k1 - w.k0;
  r.twin = left <= tpt;
  r.rows0 = min(left, tpt) * g;
  if (r.twin) {
    r.rows1 = r.rows0;
    r.n0 = (nblk + 1) / 2;
    r.n1 = nblk / 2;
  } else {
    r.rows1 = min(left - tpt, tpt) * g;
    // tile 0's last token may need fewer blocks than tile 1's
    r.n0 = FLAT ? nblk : max(0, min(nblk, (w.ctx + t0 + tpt - 1) / kBlk + 1 - w.k0));
    r.n1 = nblk;
  }
  return r;
}

// Adds to a row's written result the non-finite values it sees in the masked
// blocks, which the stages held as zeros (cold: only when there are any).
template <int D, bool KV4, typename T>
__device__ __noinline__ void add_nonfinite(const AttnParams& a, int req, int h, int first, int last, T* row) {
  for (int k = first; k <= last; ++k) {
    const int page = a.table[(size_t)req * a.max_pages + k / 16];
    if (page < 0 || page >= a.num_pages) continue;
    for (int d = 0; d < D; ++d) {
      float v;
      if (KV4)
        v = kv4_scale_value(a.vs[(((size_t)page * a.Hkv + h) * 16 + (k & 15)) * (D / 16) + d / 16]);
      else
        v = __bfloat162float(
            static_cast<const __nv_bfloat16*>(a.vc)[(((size_t)page * 16 + (k & 15)) * a.Hkv + h) * D + d]);
      if (!isfinite(v)) row[d] = (T)((float)row[d] + v);
    }
  }
}

template <int D, bool KV4, bool FLAT>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attn_tc_kernel(const __grid_constant__ CUtensorMap map_q, const MainParams p) {
  using C = Cfg<D, KV4>;
  using Sb = Bars<C::kStages, KV4>;
  constexpr int ST = C::kStages;
  constexpr uint32_t kFmt = KV4 ? 0u : 1u;  // fp16 or bf16 operands
  static_assert(C::kSmem + sizeof(Sb) <= 232448, "shared memory of a CTA");
  __shared__ Sb sb;
  extern __shared__ unsigned char dsm[];
  const uint32_t base = (smem_u32(dsm) + 1023u) & ~1023u;
  unsigned char* gbase = dsm + (base - smem_u32(dsm));
  const uint32_t sQ = 0, sKV = 2 * C::kTile, sRaw = sKV + ST * C::kTile;  // offsets from base
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sb.abort_flag;
  const AttnParams& a = p.a;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(smem_u32(&sb.kv_full[i]), KV4 ? 4 : 128);
      mbar_init(smem_u32(&sb.kv_empty[i]), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&sb.q_full[t]), KV4 && FLAT ? 4 : 1);
      mbar_init(smem_u32(&sb.q_empty[t]), 1);
      mbar_init(smem_u32(&sb.s_full[t]), 1);
      mbar_init(smem_u32(&sb.p_full[t]), 4);
      for (int q = 0; q < 4; ++q) mbar_init(smem_u32(&sb.turn[t][q]), 1);
      mbar_init(smem_u32(&sb.o_full[t]), 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&sb.slot_full[i]), 1);
      mbar_init(smem_u32(&sb.slot_empty[i]), 15);  // warps 0-5 and 7-15
    }
    mbar_init(smem_u32(&sb.x_stat), 4);
    mbar_init(smem_u32(&sb.x_back), 4);
    mbar_init(smem_u32(&sb.x_done), FLAT ? 8 : 4);
    mbar_init(smem_u32(&sb.drain[0]), 1);
    mbar_init(smem_u32(&sb.drain[1]), 1);
    sb.abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();  // the plan is complete, and the previous grid's TMEM is free
  if (warp == 4) {
    tmem_alloc(smem_u32(&sb.tmem_base), 512u);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  // all 512 columns are this CTA's: its tensor memory starts at 0
  constexpr uint32_t tmem = 0;

  auto warp_wait = [&](uint64_t& bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_short(smem_u32(&bar), parity, abort_flag)) != 0;
  };
  // The ps-th piece: false at the end of the list (or on abort).
  auto get_piece = [&](int ps, Piece& w) -> bool {
    if (!warp_wait(sb.slot_full[ps % kSlots], (uint32_t)(ps / kSlots) & 1u)) return false;
    w = sb.piece[ps % kSlots];
    return w.b >= 0;
  };
  auto release_piece = [&](int ps) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sb.slot_empty[ps % kSlots]));
  };

  if (warp < 4) {
    // ------------------------------------------------------ K/V producers
    // registers move from the copying and issuing warps to the softmax:
    // 256 x 56 + 256 x 200 (4-bit, whose producers convert: 64 and 192) = the
    // 512 x 128 of the launch
    set_max_regs<KV4 ? 64 : 56, false>();
    const int tid = threadIdx.x;
    int st = 0;
    uint32_t ph = 0;  // stage and phase of the next tile to be filled
    bool ok = true;
    if constexpr (!KV4) {
      constexpr int CPR = D / 8, RPI = 128 / CPR, IT = kBlk / RPI;  // chunks per row, rows per iteration
      const int row0 = tid / CPR, c = tid % CPR;
      const uint32_t dst0 = (uint32_t)(c / 8) * C::kHalf + (uint32_t)row0 * 128u + (uint32_t)(((c % 8) ^ (row0 & 7)) << 4);
      const size_t tok_bytes = (size_t)a.Hkv * D * 2, page_bytes = tok_bytes * 16;
      // V of a masked block: a weight of zero does not silence a NaN or an
      // infinity in the matrix product, so they are taken out of the stage
      // and added at the end to the rows that see them
      auto take_out_nonfinite = [&](int slot) {
        bool found = false;
#pragma unroll 4
        for (int i = 0; i < IT; ++i) {
          uint4* q = reinterpret_cast<uint4*>(gbase + sKV + st * C::kTile + dst0 + (uint32_t)i * (RPI * 128u));
          uint4 v = *q;
          uint32_t e[4] = {v.x, v.y, v.z, v.w};
          bool hit = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if ((e[k] & 0x7f80u) == 0x7f80u) e[k] &= 0xffff0000u, hit = true;
            if ((e[k] & 0x7f800000u) == 0x7f800000u) e[k] &= 0x0000ffffu, hit = true;
          }
          if (hit) *q = make_uint4(e[0], e[1], e[2], e[3]), found = true;
        }
        if (found) *(volatile int*)&sb.bad_v[slot] = 1;
      };
      Piece w;
      for (int ps = 0;; ++ps) {
        if (!get_piece(ps, w)) break;
        const int n_keys = w.ctx + (FLAT ? 0 : w.n), masked_from = w.ctx + w.u * p.tpu;  // the first row's position
        const char* kb_ = static_cast<const char*>(a.kc) + (size_t)w.h * D * 2 + c * 16;
        const char* vb_ = static_cast<const char*>(a.vc) + (size_t)w.h * D * 2 + c * 16;
        const int32_t* tab = a.table + (size_t)w.b * a.max_pages;
        // page ids of four blocks at a time, lane 8 j + q: page q of block j;
        // the next four are loaded one group ahead (a wait for a load is also
        // one for the copies in flight)
        auto pages_of = [&](int blk) -> int {
          const int pi = blk * 8 + lane;
          return pi < w.k1 * 8 && pi * 16 < n_keys ? tab[pi] : kNoPage;
        };
        int pg = kNoPage, pg_next = pages_of(w.k0);
        for (int blk = w.k0; ok && blk < w.k1; ++blk) {
          const int j = (blk - w.k0) & 3;
          if (j == 0) {
            pg = pg_next;
            pg_next = pages_of(blk + 4);
            if (pg != kNoPage && (pg < 0 || pg >= a.num_pages)) {
              set_status(a.status, EAGLE_ERR_BAD_KV);
              pg = kNoPage;
            }
          }
          const int key0 = blk * kBlk;
          const bool masked = !FLAT && key0 + kBlk - 1 > masked_from;
          // the block's pages, all before the first copy: a copy that waits
          // for a shuffle of its own cost 89 cycles each
          int pq[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) pq[q] = __shfl_sync(0xffffffffu, pg, j * 8 + q);
          const bool whole = __all_sync(0xffffffffu, pg >= 0 || (lane >> 3) != j) && key0 + kBlk <= n_keys;
#pragma unroll 1
          for (int o = 0; o < 2; ++o) {
            ok = warp_wait(sb.kv_empty[st], ph ^ 1u);
            if (!ok) break;
            const uint32_t dst = base + sKV + st * C::kTile + dst0;
            const char* src = (o ? vb_ : kb_) + (size_t)(row0 & 15) * tok_bytes;
            if (whole) {
#pragma unroll
              for (int i = 0; i < IT; ++i)
                cp_async16(dst + (uint32_t)i * (RPI * 128u),
                           src + (size_t)pq[i * RPI / 16] * page_bytes + (size_t)(i * RPI & 15) * tok_bytes);
            } else {
#pragma unroll
              for (int i = 0; i < IT; ++i) {  // a block with a tail or a page out of range
                const int q = pq[i * RPI / 16];
                const bool live = q >= 0 && key0 + i * RPI + row0 < n_keys;
                cp_async16_or_zero(dst + (uint32_t)i * (RPI * 128u),
                                   live ? src + (size_t)q * page_bytes + (size_t)(i * RPI & 15) * tok_bytes : src, live);
              }
            }
            if (o && masked) {
              cp_async_commit();
              cp_async_wait<0>();
              take_out_nonfinite(ps % kSlots);
              mbar_arrive(smem_u32(&sb.kv_full[st]));
            } else {
              cp_async_arrive(smem_u32(&sb.kv_full[st]));
            }
            if (++st == ST) {
              st = 0;
              ph ^= 1u;
            }
          }
        }
        if (!ok) break;
        release_piece(ps);
      }
      cp_async_wait_all();
    } else {
      constexpr int R = C::kRawRing;
      static_assert(R <= 3, "cp_async_wait_n");
      constexpr int CP = 16 * (D / 2) / 16 / 32;  // code copies per lane and page (16 tokens of a head)
      constexpr int SP = 16 * (D / 16) / 16;      // 16-byte scale copies per page
      int issued = 0, consumed = 0, islot = 0, cslot = 0;  // tiles, and their raw slots
      // the cursor of the copies runs ahead of that of the conversion
      int ips = 0, iblk = 0, ik1 = 0, ikeys = 0, iop = 0, igrp = 0, ipg = kNoPage, ipg_next = kNoPage;
      const int32_t* itab = nullptr;
      size_t ihead = 0;  // the kv head's 16 x D channels in a page
      bool have = false, last = false;
      const size_t page_ch = (size_t)a.Hkv * 16 * D;  // channels of a page
      const uint32_t raw0 = base + sRaw + (uint32_t)(warp * 32 * (D / 2) + lane * 16);
      const uint32_t raws0 = base + sRaw + C::kRawCodes + (uint32_t)(warp * 32 * (D / 16) + lane * 16);
      // page ids of 16 blocks at a time, lane 2 j + q: page q of this warp's 32
      // keys of block j; the next are loaded one group ahead (a wait for a
      // load is also one for the copies in flight)
      auto pages_of = [&](int blk) -> int {
        const int bl = blk + (lane >> 1), pi = bl * 8 + warp * 2 + (lane & 1);
        return bl < ik1 && pi * 16 < ikeys ? itab[pi] : kNoPage;
      };
      int ip0 = kNoPage, ip1 = kNoPage;
      auto issue = [&](bool must) -> bool {
        if (!have) {
          if (last) return false;
          if (!must && !__all_sync(0xffffffffu, mbar_try_wait(smem_u32(&sb.slot_full[ips % kSlots]),
                                                              (uint32_t)(ips / kSlots) & 1u)))
            return false;
          Piece w;
          if (!get_piece(ips, w)) {
            last = true;
            return false;
          }
          have = true;
          itab = a.table + (size_t)w.b * a.max_pages;
          ihead = (size_t)w.h * (16 * D);
          ik1 = w.k1;
          ikeys = w.ctx + (FLAT ? 0 : w.n);
          iblk = w.k0;
          iop = 0;
          igrp = 0;
          ipg_next = pages_of(iblk);
        }
        if (iop == 0) {
          if (igrp == 0) {
            ipg = ipg_next;
            ipg_next = pages_of(iblk + 16);
            if (ipg != kNoPage && (ipg < 0 || ipg >= a.num_pages)) {
              set_status(a.status, EAGLE_ERR_BAD_KV);
              ipg = kNoPage;
            }
          }
          ip0 = __shfl_sync(0xffffffffu, ipg, 2 * igrp);
          ip1 = __shfl_sync(0xffffffffu, ipg, 2 * igrp + 1);
          igrp = (igrp + 1) & 15;
        }
        const uint8_t* codes = static_cast<const uint8_t*>(iop ? a.vc : a.kc) + lane * 16;
        const uint8_t* scales = iop ? a.vs : a.ks;
        const uint32_t slot_off = (uint32_t)islot * C::kRaw;
        if (++islot == R) islot = 0;
        const bool live0 = ip0 >= 0, live1 = ip1 >= 0;
        const size_t ch0 = live0 ? (size_t)ip0 * page_ch + ihead : 0, ch1 = live1 ? (size_t)ip1 * page_ch + ihead : 0;
#pragma unroll
        for (int i = 0; i < CP; ++i) cp_async16_or_zero(raw0 + slot_off + i * 512u, codes + (ch0 >> 1) + i * 512, live0);
#pragma unroll
        for (int i = 0; i < CP; ++i)
          cp_async16_or_zero(raw0 + slot_off + (CP + i) * 512u, codes + (ch1 >> 1) + i * 512, live1);
        if (lane < 2 * SP) {
          const bool second = lane >= SP;
          cp_async16_or_zero(raws0 + slot_off, scales + ((second ? ch1 : ch0) >> 4) + (lane & (SP - 1)) * 16,
                             second ? live1 : live0);
        }
        cp_async_commit();
        ++issued;
        if (++iop == 2) {
          iop = 0;
          if (++iblk == ik1) {
            have = false;
            ++ips;
          }
        }
        return true;
      };
      Piece w;
      for (int ps = 0; ok; ++ps) {
        if (!get_piece(ps, w)) break;
        const int n_keys = w.ctx + (FLAT ? 0 : w.n), masked_from = w.ctx + w.u * p.tpu;
        for (int blk = w.k0; ok && blk < w.k1; ++blk) {
          const int key0 = blk * kBlk;
          const bool masked = !FLAT && key0 + kBlk - 1 > masked_from;
#pragma unroll 1
          for (int o = 0; o < 2; ++o) {
            while (issued - consumed < R && issue(issued == consumed)) {
            }
            cp_async_wait_n(issued - consumed - 1);
            __syncwarp();
            ok = warp_wait(sb.kv_empty[st], ph ^ 1u);
            if (!ok) break;
            const unsigned char* raw = gbase + sRaw + (uint32_t)cslot * C::kRaw;
            if (++cslot == R) cslot = 0;
            unsigned char* stage = gbase + sKV + st * C::kTile;
            bool found = false;
            // a lane takes 32 channels of a row: eight lanes at a time write
            // 4 rows x 2 chunks, whose swizzled places are all different
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              const int r = warp * 32 + (D == 128 ? (i >> 1) * 16 : i * 16) + (lane >> 1);
              const int ch = (D == 128 ? (i & 1) * 2 : 0) + (lane & 1);
              const uint4 cw = *reinterpret_cast<const uint4*>(raw + r * (D / 2) + ch * 16);
              uint32_t sc = *reinterpret_cast<const uint16_t*>(raw + C::kRawCodes + r * (D / 16) + ch * 2);
              if (key0 + r >= n_keys) sc = 0;
              if (o && masked) {
                if ((sc & 0x7fu) == 0x7fu) sc &= 0xff00u, found = true;
                if ((sc & 0x7f00u) == 0x7f00u) sc &= 0x00ffu, found = true;
              }
              const uint32_t s2 = e4m3_pair_as_f16(sc);
              const uint32_t sl = __byte_perm(s2, s2, 0x1010), sh = __byte_perm(s2, s2, 0x3232);
              const uint32_t cwv[4] = {cw.x, cw.y, cw.z, cw.w};
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                uint32_t v[4];
                kv4_expand(cwv[x], x < 2 ? sl : sh, v);
                *reinterpret_cast<uint4*>(stage + (uint32_t)(ch / 2) * C::kHalf + r * 128 +
                                          ((((ch & 1) * 4 + x) ^ (r & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
              }
            }
            if (found) *(volatile int*)&sb.bad_v[ps % kSlots] = 1;
            __syncwarp();  // also: the raw slot may be filled again
            if (lane == 0) mbar_arrive(smem_u32(&sb.kv_full[st]));
            ++consumed;
            if (++st == ST) {
              st = 0;
              ph ^= 1u;
            }
          }
        }
        if (!ok) break;
        release_piece(ps);
      }
      cp_async_wait_all();
    }
  } else if (warp < 8) {
    set_max_regs<KV4 ? 64 : 56, false>();
    if (warp < 6) {
      // ------------------------------------------------------- MMA issuers
      // One warp per tile, so that one's waits and commits stand beside the
      // other's MMAs.  Each runs converged, every value the same in its lanes
      // (descriptors and addresses stay in uniform registers), only the MMAs
      // and commits predicated on the elected lane.
      constexpr uint32_t idesc_s = mma_idesc(kFmt, 128, kBlk), idesc_pv = mma_idesc_bmn(kFmt, 128, D);
      const int t = __shfl_sync(0xffffffffu, warp - 4, 0);
      const uint64_t dq = smem_desc_sw128(base + sQ + t * C::kTile), dk0 = smem_desc_sw128(base + sKV);
      const uint64_t dv0 = smem_desc_sw128_mn(base + sKV, C::kHalf);
      const uint32_t s_col = (uint32_t)(t * kBlk), o_col = C::kColO + (uint32_t)(t * D);
      uint32_t pph = 0, qph = 0;
      int st = 0;  // stage and phase of the next K/V tile
      uint32_t ph = 0;
      bool ok = true;
      auto next_tile = [&]() {
        if (++st == ST) {
          st = 0;
          ph ^= 1u;
        }
      };
      // both warps free every K/V tile; this one does not read this one
      auto skip = [&](int tiles) {
#pragma unroll 1
        for (int x = 0; x < tiles && ok; ++x) {
          ok = warp_wait(sb.kv_full[st], ph);
          if (ok && lane == 0) mbar_arrive(smem_u32(&sb.kv_empty[st]));
          next_tile();
        }
      };
      // the next K/V tile, written by the copying threads, becomes the tensor
      // core's: the fence stands on this side because in a copying thread it
      // would wait for all its copies in flight
      auto take = [&]() {
        ok = ok && warp_wait(sb.kv_full[st], ph);
        fence_proxy_async_smem();
        tc_fence_after();
      };
      for (int ps = 0; ok; ++ps) {
        Piece w;
        if (!get_piece(ps, w)) break;
        const TileWork tw = tile_work<FLAT>(w, p.tpt, p.tpu, p.g);
        const int n = __shfl_sync(0xffffffffu, tw.n(t), 0), nblk = __shfl_sync(0xffffffffu, w.k1 - w.k0, 0);
        const int twin = __shfl_sync(0xffffffffu, (int)tw.twin, 0);
        if (n == 0) {
          skip(2 * nblk);
        } else {
          if (twin && t) skip(2);  // the other tile's block
          ok = ok && warp_wait(sb.q_full[t], qph);
          qph ^= 1u;
          int kst = 0, vst = 0;
          auto take_k = [&]() {
            take();
            kst = st;
            next_tile();
          };
          // Block i: P V(i), then S(i + 1) over the P just read (one loop with
          // one place for each, started a step early, keeps the code small).
#pragma unroll 1
          for (int i = -1; i < n && ok; ++i) {
            const bool more = i + 1 < n;
            if (i >= 0) {
              take();
              vst = st;
              next_tile();
              // with alternate blocks the next K tile lies past the other
              // tile's two and may need this V tile's stage: V goes first
              if (more && !twin) take_k();
              ok = ok && warp_wait(sb.p_full[t], pph);
              if (!ok) break;
              pph ^= 1u;
              tc_fence_after();
              const uint64_t dv = dv0 + (uint64_t)((uint32_t)(vst * C::kTile) >> 4);
              const uint32_t one = elect_one();
#pragma unroll
              for (int k = 0; k < kBlk / 16; ++k)
                mma_ts(one, o_col, s_col + (uint32_t)(k * 8), dv + (uint32_t)k * 128u, idesc_pv, i > 0 || k > 0);
              commit(one, smem_u32(&sb.kv_empty[vst]));
              if (!more) commit(one, smem_u32(&sb.o_full[t]));
            }
            if (more) {
              if (twin || i < 0) {
                if (i >= 0) skip(2);
                if (ok) take_k();
              }
              if (!ok) break;
              const uint64_t dk = dk0 + (uint64_t)((uint32_t)(kst * C::kTile) >> 4);
              const uint32_t one = elect_one();
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = ((uint32_t)(k >> 2) * C::kHalf + (uint32_t)(k & 3) * 32u) >> 4;
                mma_ss(one, s_col, dq + off, dk + off, idesc_s, k > 0);
              }
              commit(one, smem_u32(&sb.s_full[t]));
              commit(one, smem_u32(&sb.kv_empty[kst]));
              if (i + 2 == n) commit(one, smem_u32(&sb.q_empty[t]));
            }
          }
          // what follows this tile's last block in the piece
          if (ok) skip(2 * (twin ? nblk - (2 * (n - 1) + t + 1) : nblk - n));
        }
        if (!ok) break;
        release_piece(ps);
      }
      // every MMA completes before tensor memory is freed
      commit(elect_one(), smem_u32(&sb.drain[t]));
      const unsigned long long t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(&sb.drain[t]), 0) && globaltimer_ns() - t0 < 100000000ull) {
      }
      __syncwarp();
    } else if (warp == 6) {
      // ----------------------------------------------------------- scheduler
      if constexpr (FLAT) {
        FlatWalk walk;
        walk.start(a, p.tpu, blockIdx.x == 0);
        Piece w;
        w.slot = -1;
        for (int ps = 0;; ++ps) {
          const int slot = ps % kSlots;
          const bool more = walk.next(a, p.tpu, w);
          if (!warp_wait(sb.slot_empty[slot], ((uint32_t)(ps / kSlots) & 1u) ^ 1u)) break;
          if (lane == 0) {
            if (more)
              sb.piece[slot] = w;
            else
              sb.piece[slot].b = -1;
            sb.bad_v[slot] = 0;
            mbar_arrive(smem_u32(&sb.slot_full[slot]));
          }
          __syncwarp();
          if (!more) break;
        }
        const Split x = walk.split(w, p.tpu, p.g);
        if (lane == 0) p.splits[blockIdx.x] = x;
      } else if (lane == 0) {
        const int total = p.hdr->pieces;
        for (int ps = 0;; ++ps) {
          const int slot = ps % kSlots;
          if (!mbar_wait_short(smem_u32(&sb.slot_empty[slot]), ((uint32_t)(ps / kSlots) & 1u) ^ 1u, abort_flag)) break;
          const int i = ps == 0 ? (int)blockIdx.x : atomicAdd(p.next, 1);
          if (i < total)
            sb.piece[slot] = p.pieces[i];
          else
            sb.piece[slot].b = -1;
          sb.bad_v[slot] = 0;
          mbar_arrive(smem_u32(&sb.slot_full[slot]));
          if (i >= total) break;
        }
      }
      __syncwarp();
    } else {
      // ----------------------------------------------------------- Q loader
      constexpr int CPR = D / 8, RPI = 32 / CPR;  // rows per iteration of the warp
      constexpr int QU = 8;                       // rows a lane has in flight
      const int row0 = lane / CPR, c = lane % CPR;
      const uint32_t g_inv = (65536u + (uint32_t)p.g - 1) / (uint32_t)p.g;  // r / g = r * g_inv >> 16 for r < 128
      const uint64_t pol = l2_policy_evict_first();
      int uses[2] = {0, 0};
      bool ok = true;
      Piece w;
      for (int ps = 0; ok; ++ps) {
        if (!get_piece(ps, w)) break;
        const TileWork tw = tile_work<FLAT>(w, p.tpt, p.tpu, p.g);
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          if (tw.n(t) == 0 || (KV4 && FLAT)) continue;
          ok = warp_wait(sb.q_empty[t], ((uint32_t)uses[t] & 1u) ^ 1u);
          if (!ok) break;
          const int tok0 = w.c0 + w.u * p.tpu + (tw.twin ? 0 : t * p.tpt);
          if constexpr (!KV4) {
            // one box per 64 columns: tokens x the kv head's query heads, in
            // the tile's row order (rows past the request's end are another's
            // or zeros: nothing of them is written)
            if (lane == 0) {
              const uint32_t bar = smem_u32(&sb.q_full[t]);
              mbar_arrive_expect_tx(bar, (uint32_t)(p.tpt * p.g) * 128u * (D / 64));
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_load_3d(base + sQ + t * C::kTile + h * C::kHalf, &map_q, bar, h * 64, w.h * p.g, tok0, pol);
            }
            __syncwarp();
          } else {
            // rows as fp16, each scaled by a power of two to [1, 2) at its
            // largest: bf16's 8 bits fit fp16's 11, and what is below 2^-14
            // of the row's largest keeps an absolute error of 2^-25 of it
            const int rows = tw.rows(t);
            const __nv_bfloat16* q =
                static_cast<const __nv_bfloat16*>(a.q) + (size_t)tok0 * a.q_stride + (size_t)w.h * p.g * D + c * 8;
#pragma unroll 1
            for (int r0 = row0; r0 < rows + row0; r0 += QU * RPI) {
              uint4 v[QU];
#pragma unroll
              for (int x = 0; x < QU; ++x) {
                const int r = r0 + x * RPI, tk = (int)((uint32_t)r * g_inv >> 16);
                v[x] = r < rows ? *reinterpret_cast<const uint4*>(q + (size_t)tk * a.q_stride + (size_t)(r - tk * p.g) * D)
                                : make_uint4(0u, 0u, 0u, 0u);
              }
#pragma unroll
              for (int x = 0; x < QU; ++x) {
                const int r = r0 + x * RPI;
                const uint32_t e[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
                uint32_t mx = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) mx = max(mx, max(e[k] & 0x7fffu, (e[k] >> 16) & 0x7fffu));
#pragma unroll
                for (int d = CPR / 2; d; d >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const int k2 = row_exponent(mx);
                const float down = __uint_as_float((uint32_t)(127 - k2) << 23);
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  h[k] = pack16<true>(__uint_as_float(e[k] << 16) * down, __uint_as_float(e[k] & 0xffff0000u) * down);
                if (r < rows) {
                  *reinterpret_cast<uint4*>(gbase + sQ + t * C::kTile + (uint32_t)(c / 8) * C::kHalf + (uint32_t)r * 128u +
                                            (uint32_t)(((c % 8) ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                  if (c == 0) sb.q_fac[uses[t] & 1][t][r] = __uint_as_float((uint32_t)(127 + k2) << 23);
                }
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sb.q_full[t]));
          }
          ++uses[t];
        }
        if (!ok) break;
        release_piece(ps);
      }
      // no box may land in the memory of the SM's next CTA: done already, but
      // after an abort, which may show as a failed wait here or as a list
      // that ends early
      if (!KV4) {
        const unsigned long long t0 = globaltimer_ns();
        for (int t = 0; t < 2; ++t)
          while (uses[t] && !mbar_try_wait(smem_u32(&sb.q_full[t]), (uint32_t)(uses[t] - 1) & 1u) &&
                 globaltimer_ns() - t0 < 100000000ull) {
          }
        __syncwarp();
      }
    }
  } else {
    // ------------------------------------------------------------- softmax
    set_max_regs<KV4 ? 192 : 200, true>();
    const int t = (warp - 8) >> 2, q4 = warp & 3, row = q4 * 32 + lane;
    const uint32_t lane_addr = (uint32_t)(q4 * 32) << 16;
    const uint32_t s_addr = tmem + lane_addr + (uint32_t)(t * kBlk);
    const uint32_t o_addr = tmem + lane_addr + C::kColO + (uint32_t)(t * D);
    uint32_t sph = 0, oph = 0, xph = 0, tph = 0;
    bool my_turn_comes = t != 0;  // the other tile's warp passes before this one's next turn (not before tile 0's first)
    int uses = 0;
    bool ok = true;
    Piece w;
    for (int ps = 0; ok; ++ps) {
      if (!get_piece(ps, w)) break;
      const TileWork tw = tile_work<FLAT>(w, p.tpt, p.tpu, p.g);
      const int n = tw.n(t), rows = tw.rows(t);
      const bool quad_live = q4 * 32 < rows, row_ok = row < rows;
      const int tok = w.u * p.tpu + (tw.twin ? 0 : t * p.tpt) + row / p.g;
      const int pos = row_ok ? (FLAT ? w.ctx - 1 : w.ctx + tok) : 0x7fffffff;
      // Two warps of a scheduler, one per tile, take turns at a block's
      // softmax: left alone the tiles fall into step, both in their softmax
      // and then both waiting for their MMAs.  (Not with alternate blocks,
      // where the MMAs are few.)  Tile 0 goes first, and the turns run on
      // from piece to piece: each warp waits for the other's last pass before
      // it passes again, so that no barrier is ever two phases ahead of the
      // warp that waits on it by parity.  (With a waiting of its own in every
      // piece, tile 0 could pass at the last block of a piece and at the first
      // of the next before tile 1 had seen either.)
      const int turns = !tw.twin && q4 * 32 < min(tw.rows0, tw.rows1) ? min(tw.n0, tw.n1) : 0;
      const int pos0 = __shfl_sync(0xffffffffu, pos, 0);  // the warp's first row sees least
      float m = -INFINITY, l = 0.f, sl2 = p.scale_log2;
      bool fresh = true;  // some row has seen no key yet
      if constexpr (KV4 && FLAT) {
        // Pieces are short here, and one warp that brings 256 rows of Q to fp16
        // would hold up the first block of each: a row's thread does it (as the
        // Q loader's warp does otherwise).
        if (n > 0) {
          ok = warp_wait(sb.q_empty[t], ((uint32_t)uses & 1u) ^ 1u);
          if (!ok) break;
          if (row_ok) {
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                              ((size_t)w.c0 + tok) * a.q_stride + (size_t)(w.h * p.g + row % p.g) * D);
            uint4 v[D / 8];
#pragma unroll
            for (int c = 0; c < D / 8; ++c) v[c] = src[c];
            uint32_t mx = 0;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              const uint32_t e[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) mx = max(mx, max(e[k] & 0x7fffu, (e[k] >> 16) & 0x7fffu));
            }
            const int k2 = row_exponent(mx);
            const float down = __uint_as_float((uint32_t)(127 - k2) << 23);
            sl2 = row_factor(sl2, __uint_as_float((uint32_t)(127 + k2) << 23));
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              const uint32_t e[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
              uint32_t x[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                x[k] = pack16<true>(__uint_as_float(e[k] << 16) * down, __uint_as_float(e[k] & 0xffff0000u) * down);
              *reinterpret_cast<uint4*>(gbase + sQ + t * C::kTile + (uint32_t)(c / 8) * C::kHalf + (uint32_t)row * 128u +
                                        (uint32_t)(((c % 8) ^ (row & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sb.q_full[t]));
        }
      }
      int key0 = (w.k0 + tw.blk(t, 0)) * kBlk;
      const int key_step = tw.twin ? 2 * kBlk : kBlk;
#pragma unroll 1
      for (int i = 0; i < n; ++i, key0 += key_step) {
        ok = warp_wait(sb.s_full[t], sph);
        if (!ok) break;
        sph ^= 1u;
        tc_fence_after();
        if (quad_live) {
          if (KV4 && !FLAT && i == 0) sl2 = row_factor(sl2, row_ok ? sb.q_fac[uses & 1][t][row] : 1.f);
          if (i < turns && my_turn_comes) {
            ok = warp_wait(sb.turn[t][q4], tph);
            if (!ok) break;
            tph ^= 1u;
          }
          my_turn_comes = my_turn_comes || i < turns;
          // m is the reference of O and l.  It need not be the maximum: the
          // weights' type only has to hold 2^(z - m).  So a row takes (kBelow
          // under) the maximum of the first keys it sees and keeps it until a block's
          // weights add up to more than kSumLimit; then (and for NaN) the
          // block's maximum is looked for, and O and l are rescaled.  (Only
          // the row itself decides, so its result does not depend on the rows
          // beside it.)
          bool mine = row_ok && m == -INFINITY, renew = fresh;
          uint32_t pk[64];
          float l0;
#pragma unroll 1
          for (int pass = 0;; ++pass) {
            uint32_t r[kBlk];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32_issue(s_addr + (uint32_t)(c * 32), r + c * 32);
            tmem_wait_ld();
            if (__builtin_expect(key0 + kBlk - 1 > pos0, 0)) {
              const int lim = pos - key0;  // the last visible column
#pragma unroll
              for (int c = 0; c < kBlk; ++c) r[c] = c <= lim ? r[c] : 0xff800000u;
            }
            if (__builtin_expect(renew, 0)) {
              float mx[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) mx[c] = fmaxf(__uint_as_float(r[c]), __uint_as_float(r[c + 4]));
#pragma unroll
              for (int c = 8; c < kBlk; c += 8)
#pragma unroll
                for (int y = 0; y < 4; ++y) mx[y] = max3(mx[y], __uint_as_float(r[c + y]), __uint_as_float(r[c + y + 4]));
              const float bm = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sl2 - kBelow<KV4>;
              const bool resc = mine && bm > m && m != -INFINITY;
              if (__any_sync(0xffffffffu, resc)) {
                // S(i) was issued after P V(i - 1): O is still
                const float alpha = resc ? ex2_approx(m - bm) : 1.f;
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                  float o[16];
                  tmem_ld16(o_addr + (uint32_t)(c * 16), o);
#pragma unroll
                  for (int k = 0; k < 16; ++k) o[k] *= alpha;
                  tmem_st16(o_addr + (uint32_t)(c * 16), o);
                }
                l *= alpha;
              }
              if (mine && bm > m) m = bm;
              if (fresh) fresh = __any_sync(0xffffffffu, row_ok && m == -INFINITY);
            }
            const float neg_m = m == -INFINITY ? 0.f : -m;
            const uint64_t sc2 = pack2(sl2, sl2), nm2 = pack2(neg_m, neg_m);
            uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int k = 0; k < 64; ++k) {
              // half of them issued: the other tile's may start to fill the gaps
              if (k == 32 && !pass && i < turns && lane == 0) mbar_arrive(smem_u32(&sb.turn[t ^ 1][q4]));
              float e0, e1;
              unpack2(fma2(pack2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])), sc2, nm2), e0, e1);
              e0 = ex2_approx(e0);
              e1 = ex2_approx(e1);
              ls[k & 3] = add2(ls[k & 3], pack2(e0, e1));
              pk[k] = pack16<KV4>(e0, e1);
            }
            float l1;
            unpack2(add2(add2(ls[0], ls[1]), add2(ls[2], ls[3])), l0, l1);
            l0 += l1;
            if (pass) break;
            mine = row_ok && !(l0 <= kSumLimit<KV4>);
            renew = __any_sync(0xffffffffu, mine);
            if (!renew) break;
          }
          tmem_st32(s_addr, pk);
          tmem_st32(s_addr + 32u, pk + 32);
          l += l0;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sb.p_full[t]));
      }
      if (!ok) break;
      if (n > 0) {
        ++uses;
        ok = warp_wait(sb.o_full[t], oph);
        if (!ok) break;
        oph ^= 1u;
        tc_fence_after();
      }
      const bool whole = w.slot < 0;
      const size_t orow = ((size_t)w.c0 + tok) * a.Hq + w.h * p.g + row % p.g;
      float w0 = 1.f, w1 = 0.f;  // weights of this tile's O and of the other's
      const bool join = tw.twin && tw.n1 > 0;
      const bool halves = FLAT && join;  // of the channels, one for each tile's warps
      const bool writes = quad_live && (halves || !(tw.twin && t == 1));
      // A row's own log-sum-exp, in whose place lse may be written.  With `halves` both tiles'
      // warps read it, and tile 0's write lse: tile 1's read it in front of their arrivals
      // on x_stat, all of which tile 0's have waited for by then, so that no read comes
      // behind a write.  (Otherwise a row is one thread's.)
      float own_lse = -INFINITY;
      if (FLAT && writes && whole && row_ok && p.own_lse) own_lse = p.own_lse[orow];
      if (join) {
        if (t == 1) {
          sb.x_ml[row] = make_float2(m, l);
          tc_fence_before();  // tile 0's warps read this tile's O after their fence
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sb.x_stat));
        } else {
          ok = warp_wait(sb.x_stat, xph);
          if (!ok) break;
          tc_fence_after();
          const float2 x = sb.x_ml[row];
          if (FLAT) {
            sb.x_ml[row] = make_float2(m, l);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sb.x_back));
          }
          const float mm = fmaxf(m, x.x);
          w0 = mm == -INFINITY ? 1.f : ex2_approx(m - mm);
          w1 = mm == -INFINITY ? 1.f : ex2_approx(x.x - mm);
          l = l * w0 + x.y * w1;
          m = mm;
        }
        if (FLAT && t == 1) {
          // (pieces are short here, and writing their results a good part of them:
          // tile 1's warps take the upper half of the channels)
          ok = warp_wait(sb.x_back, xph);
          if (!ok) break;
          tc_fence_after();
          const float2 x = sb.x_ml[row];
          const float mm = fmaxf(m, x.x);
          w1 = mm == -INFINITY ? 1.f : ex2_approx(m - mm);
          w0 = mm == -INFINITY ? 1.f : ex2_approx(x.x - mm);
          l = x.y * w0 + l * w1;
          m = mm;
        }
      }
      if (writes) {
        const int urow = (tw.twin ? 0 : t * p.tpt * p.g) + row;
        const size_t prow = (size_t)max(w.slot, 0) * p.slot_rows + urow;
        const float inv = whole ? (l == 0.f ? 0.f : a.v_scale / l) : 1.f;
        OwnWeight x = {};
        if constexpr (FLAT) {
          if (whole && row_ok) x = own_weight(m, l, own_lse);
        }
        const uint32_t o_first = halves ? tmem + lane_addr + C::kColO : o_addr;
#pragma unroll 1
        for (int c = halves ? t * (D / 64) : 0; c < (halves && t == 0 ? D / 64 : D / 32); ++c) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32_issue(o_first + (uint32_t)(c * 32), o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          if (join) {
            uint32_t o2[32];
            tmem_ld32_issue(o_first + (uint32_t)(D + c * 32), o2);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k)
              o[k] = __float_as_uint(__uint_as_float(o[k]) * w0 + __uint_as_float(o2[k]) * w1);
          }
          if (!row_ok) continue;
          float* f = reinterpret_cast<float*>(o);
          if (whole) {
            if constexpr (FLAT) {
#pragma unroll
              for (int k = 0; k < 32; ++k) f[k] = x.of_prefix(f[k], x.prefix * a.v_scale);
              // (a row without keys of its own may hold anything)
              if (p.own_out && !(x.own == 0.f)) {
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.own_out) + orow * D + c * 32);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  const uint4 v = src[u];
                  const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    f[8 * u + 2 * k] = fmaf(__uint_as_float(e[k] << 16), x.own, f[8 * u + 2 * k]);
                    f[8 * u + 2 * k + 1] = fmaf(__uint_as_float(e[k] & 0xffff0000u), x.own, f[8 * u + 2 * k + 1]);
                  }
                }
              }
            }
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + orow * D + c * 32);
            const float by = FLAT ? 1.f : inv;
#pragma unroll
            for (int u = 0; u < 4; ++u)
              dst[u] = make_uint4(pack16<false>(f[8 * u] * by, f[8 * u + 1] * by),
                                  pack16<false>(f[8 * u + 2] * by, f[8 * u + 3] * by),
                                  pack16<false>(f[8 * u + 4] * by, f[8 * u + 5] * by),
                                  pack16<false>(f[8 * u + 6] * by, f[8 * u + 7] * by));
          } else if constexpr (FLAT) {
            // eight rows by channel: whole sectors (a row's 16 bytes each, 32 rows
            // apart, took 5,900 cycles a tile)
            float* dst = p.part_o + (((size_t)w.slot * p.slot_rows + (urow & ~7)) * D + c * 256) + (urow & 7);
#pragma unroll
            for (int k = 0; k < 32; ++k) dst[k * 8] = f[k];
          } else {
            float4* dst = reinterpret_cast<float4*>(p.part_o + prow * D + c * 32);
#pragma unroll
            for (int u = 0; u < 8; ++u) dst[u] = make_float4(f[4 * u], f[4 * u + 1], f[4 * u + 2], f[4 * u + 3]);
          }
        }
        if (row_ok && !(halves && t == 1)) {
          if (whole) {
            if (a.lse) a.lse[orow] = FLAT ? x.lse : l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
          } else {
            p.part_ml[prow] = make_float2(m, l);
          }
          if (!FLAT && *(volatile int*)&sb.bad_v[ps % kSlots]) {
            // the keys it sees from the first masked block on, in this piece
            const int first = max((w.ctx + w.u * p.tpu) / kBlk, w.k0) * kBlk, last = min(pos, w.k1 * kBlk - 1);
            if (whole)
              add_nonfinite<D, KV4>(a, w.b, w.h, first, last, static_cast<__nv_bfloat16*>(a.out) + orow * D);
            else
              add_nonfinite<D, KV4>(a, w.b, w.h, first, last, p.part_o + prow * D);
          }
        }
      }
      if (join) {
        // tile 1's O may be overwritten once tile 0's warps have read it
        // (where both read both, neither's may before both have)
        tc_fence_before();
        __syncwarp();
        if (FLAT || t == 0) {
          if (lane == 0) mbar_arrive(smem_u32(&sb.x_done));
        }
        if (FLAT || t == 1) {
          ok = warp_wait(sb.x_done, xph);
          if (!ok) break;
        }
        xph ^= 1u;
      }
      release_piece(ps);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (sb.abort_flag && threadIdx.x == 0) set_status(a.status, EAGLE_ERR_TIMEOUT);
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, 512u);
  }
}

// ------------------------------------------------------------------ merge
// out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s over the pieces s of a
// cut unit.  A CTA takes eight rows, a warp each, or, of a unit with many pieces,
// one row with all its warps (128 rows of some 50 pieces: 6.4 us, 15 us with a
// warp each).  Bound by latency: 2.5-5.5 us.
struct MergeParams {
  const PlanHeader* hdr;
  const Cut* cuts;
  const float2* ml;
  const float* o;
  void* out;
  float* lse;
  float v_scale;
  int Hq, g, tpu, slot_rows;
};
// A warp sums the pieces s0, s0 + step, .. of the row at row0 (its next piece
// slot_rows further on), a lane D / 32 channels; returns the maximum M over all.
template <int D>
__device__ __forceinline__ float merge_row(const float2* ml, const float* part, size_t row0, int slot_rows, int pieces,
                                           int s0, int step, float& l, float* o) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  float M = -INFINITY;
  for (int s = lane; s < pieces; s += 32) M = fmaxf(M, __ldcg(ml + row0 + (size_t)s * slot_rows).x);
#pragma unroll
  for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
  for (int s = s0; s < pieces; s += step) {
    const size_t row = row0 + (size_t)s * slot_rows;
    const float2 x = __ldcg(ml + row);
    const float w = M == -INFINITY ? 1.f : ex2_approx(x.x - M);
    l = fmaf(w, x.y, l);
    float f[E];
    if constexpr (E == 4)
      *reinterpret_cast<float4*>(f) = __ldcg(reinterpret_cast<const float4*>(part + row * D + lane * 4));
    else
      *reinterpret_cast<float2*>(f) = __ldcg(reinterpret_cast<const float2*>(part + row * D + lane * 2));
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(w, f[e], o[e]);
  }
  return M;
}
template <int D, typename T>
__device__ __forceinline__ void merge_store(T* out, float* lse, size_t orow, float M, float l, const float* o,
                                            float v_scale) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const float inv = l == 0.f ? 0.f : v_scale / l;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    T* dst = out + orow * D + lane * E + e;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float2*>(dst) = make_float2(o[e] * inv, o[e + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(dst) = pack16<false>(o[e] * inv, o[e + 1] * inv);
  }
  if (lse && lane == 0) lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}
// Few rows: the last CTA of a cut unit to write its partial result joins them
// all, in the pieces' order, which saves the merge's launch: one token over 100
// keys takes 9.8 us from the host, 12.1 with a merge kernel (10.4 and 11.1 in a
// graph); 64 requests 119 and 121 us, on 4-bit pages 62.5 and 61.5.  Not for
// fp32's 64 rows (166 rows: 30 us, with the merge kernel 23).  The whole CTA
// calls it.
template <int D>
__device__ __forceinline__ void join_if_last(const AttnParams& a, const Piece& w, int g, int tpu, int slot_rows, Cut* cuts,
                                             const float2* ml, const float* part, int* s_last) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    *s_last = atomicAdd(&cuts[w.cut].done, 1) == w.pieces - 1;
    __threadfence();
  }
  __syncthreads();
  if (!*s_last) return;
  const int rows = min(tpu, w.n - w.u * tpu) * g;
  for (int r = threadIdx.x >> 5; r < rows; r += blockDim.x >> 5) {
    float l, o[D / 32];
    const float M = merge_row<D>(ml, part, (size_t)w.first * slot_rows + r, slot_rows, w.pieces, 0, 1, l, o);
    merge_store<D>(static_cast<__nv_bfloat16*>(a.out), a.lse, ((size_t)w.c0 + w.u * tpu + r / g) * a.Hq + w.h * g + r % g, M, l, o,
                   a.v_scale);
  }
}
template <int D, typename T>
__global__ void __launch_bounds__(256) prompt_merge_kernel(const MergeParams p) {
  constexpr int E = D / 32;
  __shared__ float s_o[8][D], s_l[8];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, groups = (p.slot_rows + 7) / 8;
  const int per = p.hdr->most > 8 ? 8 : 1;  // items per eight rows
  const long long items = (long long)p.hdr->cuts * groups * per;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int i = (int)(it / per), y = (int)(it % per);
    const Cut c = p.cuts[i / groups];
    const bool shared = c.pieces > 8;  // the warps share row y's pieces
    if (!shared && y) continue;
    const int r = i % groups * 8 + (shared ? y : warp), tok = c.u * p.tpu + r / p.g;
    if (r >= min(min(p.tpu, c.n - c.u * p.tpu) * p.g, p.slot_rows)) continue;  // shared: the whole CTA
    float l, o[E];
    const float M = merge_row<D>(p.ml, p.o, (size_t)c.slot * p.slot_rows + r, p.slot_rows, c.pieces, shared ? warp : 0,
                                 shared ? 8 : 1, l, o);
    if (shared) {
#pragma unroll
      for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
      if (lane == 0) s_l[warp] = l;
      __syncthreads();
      if (warp == 0) {
        for (int x = 1; x < 8; ++x) {
          l += s_l[x];
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] += s_o[x][lane * E + e];
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    merge_store<D>(static_cast<T*>(p.out), p.lse, ((size_t)c.c0 + tok) * p.Hq + c.h * p.g + r % p.g, M, l, o,
                   p.v_scale);
  }
}

// --------------------------------------------------------------- few rows
// Single tokens: one unit per (token, kv head), its at most 16 rows the
// query heads of the group, every key up to the token's own visible to all of
// them.  The call is bound by the cache's bytes, and the path through stages
// above costs more than they do (4-bit pages: staging and converting a 128-key
// tile takes four warps 1,700 cycles, its bytes arrive in 400), so here a warp
// takes a page at a time to the fragments of mma.sync: no stage that others
// wait for, no barrier.  128 threads; warp w takes pages w and w + 4 of each
// 128-key block, with its own m, l and O; the warps are joined in shared memory
// at the end of a piece.
//
// The products are transposed, S^T = K Q^T and O^T = V^T P^T: an m16n8k16 MMA
// then has 16 keys or channels and eight rows, so that a group of eight heads or
// fewer costs half of what it did as 16 rows (4-bit pages: 62 us as one group
// of eight, 80 us as two), and an 8 x 8 transpose turns the weights' layout
// into an operand's.  The channels of a fragment may stand in any order, as
// long as Q's and K's agree and O is stored by V's: a lane's registers are then
// consecutive channels in memory.  With t = lane % 4, j = lane / 4:
//   K (A operand of S^T): keys j and j + 8; 16-bit: 16-byte loads
//     i = 0 .. D/32 - 1 at channel 32 i + 8 t; 4-bit: D/4 channels at t D/4
//   V (A operand of O^T): keys 2t, 2t + 1, 2t + 8, 2t + 9; 16-bit: loads
//     i = 0 .. D/64 - 1 at channel 64 i + 8 j; 4-bit: D/8 channels at j D/8
//
// 64 requests over 1024 .. 4096 keys, 32 heads over 8, D 128, with the plan:
// 16-bit pages 120 us, 5.6 TB/s of K and V (bound by HBM: the copy rate
// here is 6.7); 4-bit pages 62.5 us, 3.0 TB/s: neither issue slots (55-59 %, some
// 370 instructions a page and head) nor the integer pipe (46-51 %) nor HBM are
// full in this kernel, 16 warps an SM leave the latencies of a step's chain
// uncovered, and the plan in front takes 12.7 us.  Four requests over 32k keys,
// 4-bit: 49.6 us.
constexpr int kFewThreads = 128;

struct FewParams {
  AttnParams a;
  float scale_log2;
  int g, slot_rows;
  const PlanHeader* hdr;
  int* next;
  const Piece* pieces;
  Cut* cuts;
  float2* part_ml;
  float* part_o;
};

template <bool F16>
__device__ __forceinline__ void mma_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transposed 8 x 8 of 16-bit elements (a lane holds elements 2 (lane % 4),
// + 1 of row lane / 4).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(v));
  return v;
}
template <int D, bool KV4, int NG>
struct CfgFew {
  // pages per step (their chains of latencies run side by side)
  static constexpr int NP = KV4 ? 2 : 1, kRows = 8 * NG;
  // 4-bit: steps in flight per warp, copied to shared memory (2.3 KB a page:
  // held in registers, three pages a warp left the loads' latency exposed).
  // Two pages a step, two steps: 62 us; three steps 64, one page a step 68.
  static constexpr int kRing = 2;
  static constexpr int kCodes = 16 * D / 2, kPage = 2 * (kCodes + D);  // bytes: K and V codes, K and V scales
  static constexpr int kJoin = 4 * kRows * (D * 4 + 8);             // the warps' O, m and l at the end (over the ring)
  static constexpr int kSmem = KV4 && 4 * kRing * NP * kPage > kJoin ? 4 * kRing * NP * kPage : kJoin;
};
template <int D, bool KV4, int NG>
__global__ void __launch_bounds__(kFewThreads, few_ctas(KV4, NG)) prompt_attn_few_kernel(const FewParams p) {
  using C = CfgFew<D, KV4, NG>;
  constexpr int KS = D / 16, NT = D / 16;  // k steps of S, 16-channel tiles of O
  constexpr int KW = KV4 ? D / 32 : D / 8;   // 32-bit words of K per key and lane
  constexpr int VW = KV4 ? D / 64 : D / 16;  // of V
  constexpr int NP = C::NP, R = C::kRows;
  extern __shared__ __align__(16) float fm[];  // [4 warps][R rows][D], then [4][R] (m, l)
  float2* s_ml = reinterpret_cast<float2*>(fm + 4 * R * D);
  __shared__ int s_piece, s_last;
  pdl_wait();
  pdl_trigger();
  const AttnParams& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = lane & 3, j = lane >> 2;
  for (bool first = true;; first = false) {
    __syncthreads();
    if (tid == 0) s_piece = first ? (int)blockIdx.x : atomicAdd(p.next, 1);
    __syncthreads();
    if (s_piece >= p.hdr->pieces) break;
    const Piece w = p.pieces[s_piece];
    const int tok = w.c0 + w.u, pos = w.ctx + w.u, n_keys = pos + 1;
    const int lim = min(n_keys, w.k1 * kBlk), page_end = (lim + 15) / 16;  // the piece's keys end at lim
    const int32_t* tab = a.table + (size_t)w.b * a.max_pages;
    // Q as the B operand of each k step: rows j of the NG groups
    uint32_t q[NG][D / 8];
    float fac[NG][2];  // of rows 2 t, 2 t + 1 of each group
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const int row = j + 8 * n;
      const __nv_bfloat16* src =
          static_cast<const __nv_bfloat16*>(a.q) + (size_t)tok * a.q_stride + (size_t)(w.h * p.g + row) * D;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        // 16-bit: channels 32 i + 8 t ..; 4-bit: t D/4 + 8 i ..
        const uint4 v = row < p.g ? *reinterpret_cast<const uint4*>(src + (KV4 ? t * (D / 4) + 8 * i : 32 * i + 8 * t))
                                  : make_uint4(0u, 0u, 0u, 0u);
        q[n][4 * i] = v.x, q[n][4 * i + 1] = v.y, q[n][4 * i + 2] = v.z, q[n][4 * i + 3] = v.w;
      }
      float up = p.scale_log2;
      if constexpr (KV4) {
        // fp16, scaled by a power of two to [1, 2) at the row's largest
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) mx = max(mx, max(q[n][i] & 0x7fffu, (q[n][i] >> 16) & 0x7fffu));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int k2 = row_exponent(mx);
        const float down = __uint_as_float((uint32_t)(127 - k2) << 23);
        up = row_factor(up, __uint_as_float((uint32_t)(127 + k2) << 23));
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          q[n][i] = pack16<true>(__uint_as_float(q[n][i] << 16) * down, __uint_as_float(q[n][i] & 0xffff0000u) * down);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) fac[n][e] = __shfl_sync(0xffffffffu, up, 4 * (2 * t + e));
    }
    float o[NG][NT][4], m[NG][2], l[NG][2];  // row 2 t + e of group n: o[n][..][e], o[n][..][2 + e]
    bool fresh = true;                       // some row has no reference yet
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < NT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    }

    struct Page {
      uint32_t k[2][KW], v[4][VW];
    };
    // page ids of this warp, 32 at a time: lane x holds page k0 * 8 + warp + 4 (32 G + x)
    int ids = 0, group = -1;
    const int page0 = w.k0 * 8 + warp;
    auto page_id = [&](int i) -> int {  // the i-th page of this warp (in order)
      if ((i >> 5) != group) {
        group = i >> 5;
        const int pi = page0 + 4 * (group * 32 + lane);
        ids = pi < page_end ? tab[pi] : -1;
      }
      int id = __shfl_sync(0xffffffffu, ids, i & 31);
      if (id < 0 || id >= a.num_pages) {
        if (page0 + 4 * i < page_end) set_status(a.status, EAGLE_ERR_BAD_KV);
        id = -1;
      }
      return id;
    };
    unsigned char* wring = reinterpret_cast<unsigned char*>(fm) + warp * C::kRing * NP * C::kPage;
    // 4-bit: page i of this warp to its ring, a 16-byte chunk c of V's key r at
    // chunk c ^ (r / 2 & 3), so that the reads below meet fewer bank conflicts
    constexpr int CK = D / 32, CX = 16 * CK / 32;  // chunks per key, and per lane
    const uint8_t *lane_k, *lane_v, *lane_s;       // of page 0
    uint32_t to_v;
    if constexpr (KV4) {
      const int r = lane / CK;  // chunk lane + 32 x: key r + 32 x / CK
      lane_k = static_cast<const uint8_t*>(a.kc) + (size_t)w.h * (8 * D) + lane * 16;
      lane_v = static_cast<const uint8_t*>(a.vc) + (size_t)w.h * (8 * D) + lane * 16;
      lane_s = (lane < D / 16 ? a.ks : a.vs) + (size_t)w.h * D + (lane & (D / 16 - 1)) * 16;
      to_v = C::kCodes + (r * CK + ((lane % CK) ^ ((r >> 1) & (CK - 1)))) * 16;
    }
    auto copy_page = [&](unsigned char* to, int i) {
      const int id = page_id(i), key0 = (page0 + 4 * i) * 16;
      const size_t page = (size_t)max(id, 0) * ((size_t)a.Hkv * D);  // scales before the page
      const uint32_t dst = smem_u32(to);
#pragma unroll
      for (int x = 0; x < CX; ++x) {
        const bool live = id >= 0 && key0 + (lane + 32 * x) / CK < lim;
        cp_async16_or_zero(dst + lane * 16 + x * 512, lane_k + page * 8 + x * 512, live);
        cp_async16_or_zero(dst + to_v + x * 512, lane_v + page * 8 + x * 512, live);
      }
      if (lane < 2 * D / 16) cp_async16_or_zero(dst + 2 * C::kCodes + lane * 16, lane_s + page, id >= 0);
    };
    auto load = [&](Page& g, int i) {
      const int id = page_id(i), key0 = (page0 + 4 * i) * 16;
      if constexpr (!KV4) {
        const size_t tok_ch = (size_t)a.Hkv * D, at0 = (size_t)max(id, 0) * 16 * tok_ch + (size_t)w.h * D;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = j + 8 * x;
          const bool live = id >= 0 && key0 + r < lim;
          const __nv_bfloat16* c = static_cast<const __nv_bfloat16*>(a.kc) + at0 + r * tok_ch + 8 * t;
#pragma unroll
          for (int y = 0; y < D / 32; ++y) {
            const uint4 v = live ? __ldg(reinterpret_cast<const uint4*>(c + 32 * y)) : make_uint4(0u, 0u, 0u, 0u);
            g.k[x][4 * y] = v.x, g.k[x][4 * y + 1] = v.y, g.k[x][4 * y + 2] = v.z, g.k[x][4 * y + 3] = v.w;
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = 2 * t + (x & 1) + 8 * (x >> 1);
          const bool live = id >= 0 && key0 + r < lim;
          const __nv_bfloat16* c = static_cast<const __nv_bfloat16*>(a.vc) + at0 + r * tok_ch + 8 * j;
#pragma unroll
          for (int y = 0; y < D / 64; ++y) {
            const uint4 v = live ? __ldg(reinterpret_cast<const uint4*>(c + 64 * y)) : make_uint4(0u, 0u, 0u, 0u);
            g.v[x][4 * y] = v.x, g.v[x][4 * y + 1] = v.y, g.v[x][4 * y + 2] = v.z, g.v[x][4 * y + 3] = v.w;
          }
        }
      }
    };
    // the step of pages i .. i + NP - 1
    auto use = [&](const Page* pg, const unsigned char* raw, int i) {
      const bool tail = (page0 + 4 * (i + NP - 1)) * 16 + 16 > lim;
      float s[NP][NG][4];  // s[z][n][2 x + e]: key j + 8 x of page z, row 2 t + e of group n
#pragma unroll
      for (int z = 0; z < NP; ++z) {
        float part[NG][2][4] = {};  // two chains of MMAs each
        if constexpr (KV4) {
          const unsigned char* pr = raw + z * C::kPage;
          uint32_t kw[2][KW], sl[2], sh[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = j + 8 * x;
            uint32_t sb;
            if constexpr (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(pr + r * 64 + t * 16);
              kw[x][0] = v.x, kw[x][1] = v.y, kw[x][2] = v.z, kw[x][3] = v.w;
              sb = *reinterpret_cast<const uint16_t*>(pr + 2 * C::kCodes + r * 8 + 2 * t);
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(pr + r * 32 + t * 8);
              kw[x][0] = v.x, kw[x][1] = v.y;
              sb = pr[2 * C::kCodes + r * 4 + t] * 0x101u;
            }
            // (a dead key's score is masked below, whatever its scale)
            const uint32_t s2 = e4m3_pair_as_f16(sb);
            sl[x] = __byte_perm(s2, s2, 0x1010), sh[x] = __byte_perm(s2, s2, 0x3232);
          }
#pragma unroll
          for (int y = 0; y < KW; ++y) {
            uint32_t e[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x) kv4_expand(kw[x][y], y < KW / 2 ? sl[x] : sh[x], e[x]);
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                mma_16816<true>(part[n][c], e[0][2 * c], e[1][2 * c], e[0][2 * c + 1], e[1][2 * c + 1], q[n][4 * y + 2 * c],
                                q[n][4 * y + 2 * c + 1]);
          }
        } else {
#pragma unroll
          for (int y = 0; y < KS; ++y)
#pragma unroll
            for (int n = 0; n < NG; ++n)
              mma_16816<false>(part[n][y & 1], pg[z].k[0][2 * y], pg[z].k[1][2 * y], pg[z].k[0][2 * y + 1],
                               pg[z].k[1][2 * y + 1], q[n][2 * y], q[n][2 * y + 1]);
        }
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[z][n][e] = part[n][0][e] + part[n][1][e];
      }
      if (tail) {
#pragma unroll
        for (int z = 0; z < NP; ++z)
#pragma unroll
          for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((page0 + 4 * (i + z)) * 16 + 8 * (e >> 1) + j >= lim) s[z][n][e] = -INFINITY;
      }
      // the reference of a row is the maximum of the first step that has a
      // finite score for it; it is renewed when a step's weights pass kSumLimit
      // (or are NaN), see the kernel above
      float wt[NP][NG][4];
      bool renew = fresh, mine[NG][2];  // by row, the same in its eight lanes
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) mine[n][e] = m[n][e] == -INFINITY;
#pragma unroll 1
      for (int pass = 0;; ++pass) {
        if (renew) {
#pragma unroll
          for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float bm = -INFINITY;
#pragma unroll
              for (int z = 0; z < NP; ++z) bm = fmaxf(bm, fmaxf(s[z][n][e], s[z][n][2 + e]));
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, d));
              bm = bm * fac[n][e] - kBelow<KV4>;
              if (mine[n][e] && bm > m[n][e]) {
                if (m[n][e] != -INFINITY) {
                  const float alpha = ex2_approx(m[n][e] - bm);
                  l[n][e] *= alpha;
#pragma unroll
                  for (int y = 0; y < NT; ++y) {
                    o[n][y][e] *= alpha;
                    o[n][y][2 + e] *= alpha;
                  }
                }
                m[n][e] = bm;
              }
            }
          if (fresh) {
            bool none = false;
#pragma unroll
            for (int n = 0; n < NG; ++n) none = none || m[n][0] == -INFINITY || m[n][1] == -INFINITY;
            fresh = __any_sync(0xffffffffu, none);
          }
        }
        float sum[NG][2];
        bool over = false;
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float ref = m[n][e] == -INFINITY ? 0.f : -m[n][e];
            sum[n][e] = 0.f;
#pragma unroll
            for (int z = 0; z < NP; ++z)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float f = ex2_approx(fmaf(s[z][n][2 * x + e], fac[n][e], ref));
                wt[z][n][2 * x + e] = f;
                sum[n][e] += f;
              }
            over = over || !(sum[n][e] <= kSumLimit<KV4>);
          }
        if (pass || !__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            l[n][0] += sum[n][0];
            l[n][1] += sum[n][1];
          }
          break;
        }
        renew = true;
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            mine[n][e] = (__ballot_sync(0xffffffffu, !(sum[n][e] <= kSumLimit<KV4>)) >> t & 0x11111111u) != 0;
      }
#pragma unroll
      for (int z = 0; z < NP; ++z) {
        uint32_t pb[NG][2];  // the weights as the B operand: keys 2 t, 2 t + 1 (+ 8) of row j
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          pb[n][0] = transpose8(pack16<KV4>(wt[z][n][0], wt[z][n][1]));
          pb[n][1] = transpose8(pack16<KV4>(wt[z][n][2], wt[z][n][3]));
        }
        // V: pairs of keys (2t, 2t + 1) and (2t + 8, 2t + 9) of each channel
        if constexpr (KV4) {
          const unsigned char* pr = raw + z * C::kPage;
          uint32_t vw[4][VW], vs[4], sc[2];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = 2 * t + (x & 1) + 8 * (x >> 1), at = (r >> 1) & (D / 32 - 1);
            if constexpr (D == 128) {
              const uint2 v = *reinterpret_cast<const uint2*>(pr + C::kCodes + r * 64 + (((j >> 1) ^ at) << 4) + (j & 1) * 8);
              vw[x][0] = v.x, vw[x][1] = v.y;
              vs[x] = pr[2 * C::kCodes + D + r * 8 + j];
            } else {
              vw[x][0] = *reinterpret_cast<const uint32_t*>(pr + C::kCodes + r * 32 + (((j >> 2) ^ at) << 4) + (j & 3) * 4);
              vs[x] = pr[2 * C::kCodes + D + r * 4 + (j >> 1)];
            }
            // a dead key's scale may be anything; its codes are zeros
            if (tail && (page0 + 4 * (i + z)) * 16 + r >= lim) vs[x] = 0;
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) sc[x] = e4m3_pair_as_f16(vs[2 * x] | vs[2 * x + 1] << 8);
#pragma unroll
          for (int y = 0; y < VW; ++y) {
            uint32_t e[2][2][4];  // [pair of keys][channel's parity]
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t lo = vw[2 * x][y], hi = vw[2 * x + 1][y];  // a byte: the pair's codes of one channel
              kv4_expand((lo & 0x0f0f0f0fu) | (hi << 4 & 0xf0f0f0f0u), sc[x], e[x][0]);
              kv4_expand((lo >> 4 & 0x0f0f0f0fu) | (hi & 0xf0f0f0f0u), sc[x], e[x][1]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int n = 0; n < NG; ++n)
                mma_16816<true>(o[n][4 * y + c], e[0][0][c], e[0][1][c], e[1][0][c], e[1][1][c], pb[n][0], pb[n][1]);
          }
        } else {
#pragma unroll
          for (int y = 0; y < VW; ++y) {
            uint32_t e[2][2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              e[x][0] = __byte_perm(pg[z].v[2 * x][y], pg[z].v[2 * x + 1][y], 0x5410u);
              e[x][1] = __byte_perm(pg[z].v[2 * x][y], pg[z].v[2 * x + 1][y], 0x7632u);
            }
#pragma unroll
            for (int n = 0; n < NG; ++n) mma_16816<false>(o[n][y], e[0][0], e[0][1], e[1][0], e[1][1], pb[n][0], pb[n][1]);
          }
        }
      }
    };
    const int n_pages = page0 < page_end ? (page_end - page0 + 3) / 4 : 0;
    if constexpr (KV4) {
      auto copy_step = [&](int slot, int i) {  // a page past the end is masked: its slot's old bytes do
        if (i < n_pages) {
#pragma unroll
          for (int z = 0; z < NP; ++z) copy_page(wring + (slot * NP + z) * C::kPage, i + z);
        }
        cp_async_commit();
      };
#pragma unroll
      for (int x = 0; x < C::kRing; ++x) copy_step(x, x * NP);
      int slot = 0;
#pragma unroll 1
      for (int i = 0; i < n_pages; i += NP) {
        cp_async_wait<C::kRing - 1>();
        __syncwarp();
        use(nullptr, wring + slot * NP * C::kPage, i);
        __syncwarp();
        copy_step(slot, i + C::kRing * NP);
        if (++slot == C::kRing) slot = 0;
      }
      cp_async_wait_all();
      __syncthreads();  // the join below takes the rings' place
    } else {
      // the next page's loads are issued as soon as this one's have been taken
      Page next;
      if (n_pages > 0) load(next, 0);
#pragma unroll 1
      for (int i = 0; i < n_pages; ++i) {
        const Page cur = next;
        if (i + 1 < n_pages) load(next, i + 1);
        use(&cur, nullptr, i);
      }
    }
    // join the warps: rows < g of (m, l) and O
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * n + 2 * t + e;
        float sum = l[n][e];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (j == 0) s_ml[warp * R + row] = make_float2(m[n][e], sum);
        if (row < p.g) {
          float* dst = fm + (warp * R + row) * D;
#pragma unroll
          for (int y = 0; y < NT; ++y)  // the lane's channels 2 y, 2 y + 1 in V's order
            *reinterpret_cast<float2*>(dst + (KV4 ? j * (D / 8) + 2 * y : 64 * (y / 4) + 8 * j + 2 * (y & 3))) =
                make_float2(o[n][y][e], o[n][y][2 + e]);
        }
      }
    __syncthreads();
    const bool whole = w.slot < 0;
    for (int i = tid; i < p.g * (D / 4); i += kFewThreads) {
      const int row = i / (D / 4), c = (i % (D / 4)) * 4;
      float mm = -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x) mm = fmaxf(mm, s_ml[x * R + row].x);
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      float ll = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 ml = s_ml[x * R + row];
        const float wt = mm == -INFINITY ? 1.f : ex2_approx(ml.x - mm);
        const float4 v = *reinterpret_cast<const float4*>(fm + (x * R + row) * D + c);
        ll = fmaf(wt, ml.y, ll);
        f = make_float4(fmaf(wt, v.x, f.x), fmaf(wt, v.y, f.y), fmaf(wt, v.z, f.z), fmaf(wt, v.w, f.w));
      }
      const size_t orow = (size_t)tok * a.Hq + w.h * p.g + row, prow = (size_t)max(w.slot, 0) * p.slot_rows + row;
      if (whole) {
        const float inv = ll == 0.f ? 0.f : a.v_scale / ll;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * D + c) =
            make_uint2(pack16<false>(f.x * inv, f.y * inv), pack16<false>(f.z * inv, f.w * inv));
        if (c == 0 && a.lse) a.lse[orow] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(p.part_o + prow * D + c) = f;
        if (c == 0) p.part_ml[prow] = make_float2(mm, ll);
      }
    }
    if (!whole) join_if_last<D>(a, w, p.g, 1, p.slot_rows, p.cuts, p.part_ml, p.part_o, &s_last);
  }
}

// ------------------------------------------------------------------- fp32
// Units of 64 rows against 128-key blocks on the CUDA cores, from the same
// list of pieces.  256 threads: thread (ty, tx) holds scores of RT = 4 rows,
// ty + 16 i, against keys tx + 16 j, and of O the same rows' columns 4 tx ..
// (and 64 + 4 tx ..): 128 FMAs for every 12 16-byte shared loads, rows padded
// so that 16 keys' loads touch all banks evenly.  K of the next block is copied
// while the weights and P V of this one are computed, V of the next during its
// scores.  Units of at most 32 rows compute those alone (64 requests of 8
// tokens, 32 rows each: 988 us, 1,203 with all 64; a long prompt pays 4 % for
// the larger kernel).  Few rows: units of 16, one row per thread, and half
// blocks, so that two CTAs fit an SM (64 single tokens 800 us; whole blocks, one
// CTA 902).  Bound by the FMA and shared-memory pipes: a prompt of 2048 tokens,
// 32 heads over 8, D 128: 1,027 us, 33 TFLOP/s causal; 64 single tokens over
// 1024 .. 4096 keys 800 us, 1.7 TB/s (a key's shared loads serve one row).  Three
// prompts of up to 130 tokens, 4 heads over 2, D 64: 24 us, 17.5 in this kernel.
template <int D, int RT>
struct CfgF32 {
  static constexpr int kRows = 16 * RT, kKeys = RT == 1 ? 64 : 128;  // per unit, per step
  static constexpr int kCtas = RT == 1 ? kF32FewCtas : 1;            // per SM
  static constexpr int kLd = D + 4, kLdP = kKeys + 4;  // floats per shared row
  static constexpr int kSmem = (kRows * kLd + 2 * kKeys * kLd + kRows * kLdP) * 4;
};
struct F32Params {
  AttnParams a;
  float scale_log2;
  int g, tpu, slot_rows;
  const PlanHeader* hdr;
  int* next;
  const Piece* pieces;
  float2* part_ml;
  float* part_o;
  const float *own_out, *own_lse;  // FLAT
  Split* splits;
};
template <int D, int RT, bool FLAT>
__global__ void __launch_bounds__(256, (CfgF32<D, RT>::kCtas)) prompt_attn_f32_kernel(const F32Params p) {
  using C = CfgF32<D, RT>;
  constexpr int CPR = D / 4, NC = D / 64;  // 16-byte chunks per row, 64-column groups
  constexpr int KB = C::kKeys, NJ = KB / 16;
  extern __shared__ __align__(16) float sm[];
  float *sq = sm, *sk = sq + C::kRows * C::kLd, *sv = sk + KB * C::kLd, *sp = sv + KB * C::kLd;
  __shared__ int s_piece;
  pdl_wait();
  pdl_trigger();
  const AttnParams& a = p.a;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  __shared__ Piece s_w;  // FLAT
  FlatWalk walk;
  if (FLAT && tid < 32) {
    // (walked twice: what the join needs is in the part's last piece)
    walk.start(a, p.tpu, blockIdx.x == 0);
    const FlatWalk from = walk;
    Piece w;
    w.slot = -1;
    while (walk.next(a, p.tpu, w)) {
    }
    const Split x = walk.split(w, p.tpu, p.g);
    if (tid == 0) p.splits[blockIdx.x] = x;
    walk = from;
  }
  for (bool first = true;; first = false) {
    __syncthreads();
    if (FLAT) {
      if (tid < 32) {
        Piece w;
        const bool more = walk.next(a, p.tpu, w);
        if (tid == 0) s_piece = more, s_w = w;
      }
    } else if (tid == 0) {
      s_piece = first ? (int)blockIdx.x : atomicAdd(p.next, 1);
    }
    __syncthreads();
    if (FLAT ? !s_piece : s_piece >= p.hdr->pieces) break;
    const Piece w = FLAT ? s_w : p.pieces[s_piece];
    const int rows = min(w.n - w.u * p.tpu, p.tpu) * p.g, n_keys = w.ctx + (FLAT ? 0 : w.n);
    const int32_t* tab = a.table + (size_t)w.b * a.max_pages;
    const int b0 = w.k0 * (kBlk / KB), b1 = min(w.k1 * (kBlk / KB), (n_keys + KB - 1) / KB);  // in steps
    auto copy = [&](float* dst, const void* src, int blk) {
      if (blk < b1) {
#pragma unroll 8
        for (int i = tid; i < KB * CPR; i += 256) {
          const int r = i / CPR, c = i % CPR, k = blk * KB + r;
          const int pg = k < n_keys ? tab[k / 16] : -1;
          const bool live = pg >= 0 && pg < a.num_pages;
          if (k < n_keys && !live) set_status(a.status, EAGLE_ERR_BAD_KV);
          const float* from = static_cast<const float*>(src) +
                              (live ? (((size_t)pg * 16 + (k & 15)) * a.Hkv + w.h) * D + c * 4 : 0);
          cp_async16_or_zero(smem_u32(dst + r * C::kLd + c * 4), from, live);
        }
      }
      cp_async_commit();
    };
    copy(sk, a.kc, b0);
    copy(sv, a.vc, b0);
    for (int i = tid; i < C::kRows * CPR; i += 256) {
      const int r = i / CPR, c = i % CPR;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                             ((size_t)w.c0 + w.u * p.tpu + r / p.g) * a.q_stride +
                                             (size_t)(w.h * p.g + r % p.g) * D + c * 4);
      *reinterpret_cast<float4*>(sq + r * C::kLd + c * 4) = v;
    }
    int pos[RT];
    float m[RT], l[RT], o[RT][4 * NC];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = ty + 16 * i;
      pos[i] = r < rows ? (FLAT ? w.ctx - 1 : w.ctx + w.u * p.tpu + r / p.g) : 0x7fffffff;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < 4 * NC; ++c) o[i][c] = 0.f;
    }
    // a block for the first 16 R rows
    auto step = [&](int blk, auto r_) {
      constexpr int R = decltype(r_)::value;
      const bool masked = blk * KB + KB - 1 > w.ctx + (FLAT ? -1 : w.u * p.tpu);
      cp_async_wait<1>();
      __syncthreads();
      float z[R][NJ];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) z[i][j] = 0.f;
#pragma unroll 4
      for (int c = 0; c < CPR; ++c) {
        float4 q[R];
#pragma unroll
        for (int i = 0; i < R; ++i) q[i] = *reinterpret_cast<const float4*>(sq + (ty + 16 * i) * C::kLd + c * 4);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const float4 k = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * C::kLd + c * 4);
#pragma unroll
          for (int i = 0; i < R; ++i)
            z[i][j] = fmaf(q[i].x, k.x, fmaf(q[i].y, k.y, fmaf(q[i].z, k.z, fmaf(q[i].w, k.w, z[i][j]))));
        }
      }
      __syncthreads();
      copy(sk, a.kc, blk + 1);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float bm = -INFINITY;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          z[i][j] = blk * KB + tx + 16 * j <= pos[i] ? z[i][j] * p.scale_log2 : -INFINITY;
          bm = fmaxf(bm, z[i][j]);
        }
#pragma unroll
        for (int d = 8; d; d >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, d));
        const float mn = fmaxf(m[i], bm), ref = mn == -INFINITY ? 0.f : mn;
        const float al = ex2_approx(m[i] - ref);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const float e = ex2_approx(z[i][j] - ref);
          sum += e;
          sp[(ty + 16 * i) * C::kLdP + tx + 16 * j] = e;
        }
#pragma unroll
        for (int d = 8; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l[i] = fmaf(l[i], al, sum);
        m[i] = mn;
#pragma unroll
        for (int c = 0; c < 4 * NC; ++c) o[i][c] *= al;
      }
      cp_async_wait<1>();
      __syncthreads();
      // in a masked block a key adds only to the rows that see it: a weight
      // of zero would not silence a NaN or an infinity
      auto weigh = [&](auto keep) {
#pragma unroll 2
        for (int k = 0; k < KB; k += 4) {
          float4 e[R];
#pragma unroll
          for (int i = 0; i < R; ++i) e[i] = *reinterpret_cast<const float4*>(sp + (ty + 16 * i) * C::kLdP + k);
#pragma unroll
          for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const float4 v = *reinterpret_cast<const float4*>(sv + (k + y) * C::kLd + c * 64 + tx * 4);
#pragma unroll
              for (int i = 0; i < R; ++i) {
                const float ey = y == 0 ? e[i].x : y == 1 ? e[i].y : y == 2 ? e[i].z : e[i].w;
                if (!keep(i, k + y)) continue;
                o[i][4 * c] = fmaf(ey, v.x, o[i][4 * c]);
                o[i][4 * c + 1] = fmaf(ey, v.y, o[i][4 * c + 1]);
                o[i][4 * c + 2] = fmaf(ey, v.z, o[i][4 * c + 2]);
                o[i][4 * c + 3] = fmaf(ey, v.w, o[i][4 * c + 3]);
              }
            }
        }
      };
      if (masked)
        weigh([&](int i, int k) { return blk * KB + k <= pos[i]; });
      else
        weigh([](int, int) { return true; });
      __syncthreads();
      copy(sv, a.vc, blk + 1);
    };
    for (int blk = b0; blk < b1; ++blk) {
      if (RT > 1 && rows <= 32)
        step(blk, std::integral_constant<int, (RT + 1) / 2>());
      else
        step(blk, std::integral_constant<int, RT>());
    }
    cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = ty + 16 * i;
      if (r >= rows) continue;
      const bool whole = w.slot < 0;
      const size_t orow = ((size_t)w.c0 + w.u * p.tpu + r / p.g) * a.Hq + w.h * p.g + r % p.g;
      const size_t prow = (size_t)max(w.slot, 0) * p.slot_rows + r;
      float f = whole ? (l[i] == 0.f ? 0.f : 1.f / l[i]) : 1.f;
      float* dst = whole ? static_cast<float*>(a.out) + orow * D : p.part_o + prow * D;
      if (FLAT && whole) {
        const OwnWeight x = own_weight(m[i], l[i], p.own_lse ? p.own_lse[orow] : -INFINITY);
        const float own = x.own;
        f = 1.f;
        m[i] = x.lse;
#pragma unroll
        for (int c = 0; c < 4 * NC; ++c) o[i][c] = x.of_prefix(o[i][c], x.prefix);
        if (p.own_out && !(own == 0.f)) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float4 v = *reinterpret_cast<const float4*>(p.own_out + orow * D + c * 64 + tx * 4);
            o[i][4 * c] = fmaf(v.x, own, o[i][4 * c]);
            o[i][4 * c + 1] = fmaf(v.y, own, o[i][4 * c + 1]);
            o[i][4 * c + 2] = fmaf(v.z, own, o[i][4 * c + 2]);
            o[i][4 * c + 3] = fmaf(v.w, own, o[i][4 * c + 3]);
          }
        }
        __syncwarp(0xffffu << (tid & 16));  // own_lse, which lse may be, is read by the row's threads
      }
#pragma unroll
      for (int c = 0; c < NC; ++c)
        *reinterpret_cast<float4*>(dst + c * 64 + tx * 4) =
            make_float4(o[i][4 * c] * f, o[i][4 * c + 1] * f, o[i][4 * c + 2] * f, o[i][4 * c + 3] * f);
      if (tx == 0) {
        if (!whole)
          p.part_ml[prow] = make_float2(m[i], l[i]);
        else if (a.lse)
          a.lse[orow] = FLAT ? m[i] : l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
      }
    }
  }
}

// ----------------------------------------------- shared prefixes: the join
// The units that several CTAs shared, as those CTAs described them.  A CTA of 2 D
// threads takes eight rows of a unit at a time, whose partial results are 32 D
// contiguous bytes of each piece: 16 bytes a thread, of 16-bit rows four rows of a
// channel, of fp32 rows four channels of a row.  The pieces' weights are worked out
// once, a thread a piece and row, while those are on their way.  CTAs
// that have none of that let rows of empty prefixes take their own result over.
struct JoinParams {
  AttnParams a;
  int g, tpu, slot_rows, ctas;
  const Split* splits;
  const float2* ml;
  const float* o;
  const void* own_out;
  const float* own_lse;
};
// Rows of empty prefixes, a warp a row; CTA c of `ctas`.
template <int D, typename T>
__device__ __forceinline__ void take_over(const JoinParams& p, int c, int ctas) {
  const AttnParams& a = p.a;
  using V = typename std::conditional<sizeof(T) * D == 512, uint4, typename std::conditional<sizeof(T) * D == 256, uint2, uint32_t>::type>::type;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  bool falls = false;
  for (int base = 0; base < a.B; base += 32) falls = __any_sync(0xffffffffu, load_groups(a, base, p.tpu, false).falls) || falls;
  if (falls) return;
  for (int base = 0; base < a.B; base += 32) {
    const Groups g = load_groups(a, base, p.tpu, false);
    unsigned m = __ballot_sync(0xffffffffu, g.n > 0 && g.len == 0);
    if (a.B == 1) m &= 1u;
    for (; m; m &= m - 1) {
      const int src = __ffs((int)m) - 1;
      const size_t r0 = (size_t)__shfl_sync(0xffffffffu, g.c0, src) * a.Hq, n = (size_t)__shfl_sync(0xffffffffu, g.n, src) * a.Hq;
      for (size_t r = r0 + c * warps + warp; r < r0 + n; r += ctas * warps) {
        const float L = p.own_lse ? p.own_lse[r] : -INFINITY;
        const size_t at = r * (sizeof(T) * D / sizeof(V)) + lane;
        V v = {};
        if (L != -INFINITY) v = static_cast<const V*>(p.own_out)[at];
        static_cast<V*>(a.out)[at] = v;
        __syncwarp();  // lse may be own_lse
        if (a.lse && lane == 0) a.lse[r] = L;
      }
    }
  }
}
constexpr int kMaxParts = 320;  // CTAs of a main kernel at most
template <int D, typename T, int kBatch, int kCtas, bool kSpare>
__global__ void __launch_bounds__(2 * D, kCtas) flat_join_kernel(const JoinParams p) {
  constexpr bool kByRow = sizeof(T) == 4;
  constexpr int kThreads_ = 2 * D, kWarps = kThreads_ / 32;
  __shared__ Split s_split[kMaxParts];
  __shared__ int s_first[kMaxParts], s_count[kMaxParts / 32];  // the CTAs that left one, in order
  __shared__ float s_w[kMaxParts][8];  // the pieces' weights
  __shared__ float s_top[kWarps][8], s_sum[kWarps][8];
  __shared__ OwnWeight s_own[8];
  const AttnParams& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // element e of this thread's four: row and channel
  auto row_of = [&](int e) { return kByRow ? tid / (D / 4) : (tid & 1) * 4 + e; };
  auto chan_of = [&](int e) { return kByRow ? tid % (D / 4) * 4 + e : tid >> 1; };
  // the eight rows from `first` of a unit, whose row 0 is row r0 of the arrays and row
  // x at(x) rows further; O in o; s_own holds their factors
  auto load_own = [&](size_t r0, int first, int rows, auto&& at, float* own) {
    const T* src = static_cast<const T*>(p.own_out) + r0 * D;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      own[e] = p.own_out && first + row_of(e) < rows ? (float)src[at(first + row_of(e)) * D + chan_of(e)] : 0.f;
  };
  auto store = [&](size_t r0, int first, int rows, auto&& at, const float* o, const float* own) {
    T* dst = static_cast<T*>(a.out) + r0 * D;
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = row_of(e);
      if (first + row >= rows) continue;
      const OwnWeight w = s_own[row];
      y[e] = w.of_prefix(o[e], w.prefix * a.v_scale);
      if (w.own != 0.f) y[e] = fmaf(own[e], w.own, y[e]);
      if constexpr (!kByRow) dst[at(first + row) * D + chan_of(e)] = (T)y[e];
    }
    if constexpr (kByRow) {
      if (first + row_of(0) < rows)
        *reinterpret_cast<float4*>(dst + at(first + row_of(0)) * D + chan_of(0)) = make_float4(y[0], y[1], y[2], y[3]);
    }
  };
  pdl_wait();
  pdl_trigger();
  // this CTA's chunks of eight rows, of slot_rows / 8 of each split: numbers
  // blockIdx.x, + stride, ..
  const int of_split = p.slot_rows / 8, stride = (int)gridDim.x - (kSpare ? p.ctas : 1);
  const int sets = (p.ctas + 31) / 32;
  for (int x = warp; x < sets; x += kWarps) {
    const int c = x * 32 + lane;
    Split u = {0, 0, 0, 0};
    if (c < p.ctas) {
      const int4 v = __ldcg(reinterpret_cast<const int4*>(p.splits + c));
      u = Split{v.x, v.y, v.z, v.w};
    }
    s_split[c] = u;
    const unsigned has = __ballot_sync(0xffffffffu, u.rows > 0);
    s_w[x][0] = __uint_as_float(has);
    if (lane == 0) s_count[x] = __popc(has);
  }
  __syncthreads();
  int splits = 0;
  for (int x = 0; x < sets; ++x) {
    if (x % kWarps == warp) {
      const unsigned has = __float_as_uint(s_w[x][0]);
      if (has >> lane & 1u) s_first[splits + __popc(has & ((1u << lane) - 1u))] = x * 32 + lane;
    }
    splits += s_count[x];
  }
  __syncthreads();
  // CTAs without a chunk, one at least, let rows of empty prefixes take their own result
  // over (64 tokens of which 32 have one 21 us, 4,096 tokens 21; with one CTA for them 106
  // and 14,400)
  const int joining = min(splits * of_split, stride);
  if ((int)blockIdx.x >= joining) {
    take_over<D, T>(p, (int)blockIdx.x - joining, (int)gridDim.x - joining);
    return;
  }
  const uint32_t g_inv = (65536u + (uint32_t)p.g - 1) / (uint32_t)p.g;
#pragma unroll 1
  for (int it = (int)blockIdx.x; it < splits * of_split; it += stride) {
    const int n = it / of_split, chunk = it - n * of_split, c0 = s_first[n];
    const Split u = s_split[c0];
    const int rows = u.rows, pieces = u.last - c0 + 1, h = u.h, tok0 = u.tok0;
    const int row0 = chunk * 8;
    if (row0 >= rows) continue;
    // (rows of a unit are fewer than 2^9, groups of heads no more than 2^6: x / g is
    // x g_inv >> 16)
    const size_t r0 = (size_t)tok0 * a.Hq + h * p.g;
    auto to = [&](int row) {
      const int of_token = (int)((uint32_t)row * g_inv >> 16);
      return of_token * a.Hq + (row - of_token * p.g);
    };
    // the unit's first piece is in slot 2 c0 + 1, the others in 2 (c0 + 1), 2 (c0 + 2), ..
    auto slot = [&](int x) { return (size_t)(2 * (c0 + x) + (x == 0 ? 1 : 0)) * p.slot_rows + row0; };
    float4 f[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i < pieces) f[i] = __ldcg(reinterpret_cast<const float4*>(p.o + slot(i) * D) + tid);
    float L = -INFINITY, own[4];
    load_own(r0, row0, rows, to, own);
    if (tid < 8 && row0 + tid < rows && p.own_lse) L = p.own_lse[r0 + to(row0 + tid)];
    // the weights: thread (x, row) = (tid / 8, tid % 8) of pieces x, x + 2 D / 8, ..
    const int row = tid & 7;
    float sum = 0.f;
    const bool mine = tid >> 3 < pieces;
    const float2 ml = mine ? __ldcg(p.ml + slot(tid >> 3) + row) : make_float2(-INFINITY, 0.f);
    float top = ml.x;
    for (int x = (tid >> 3) + 2 * D / 8; x < pieces; x += 2 * D / 8) top = fmaxf(top, __ldcg(p.ml + slot(x) + row).x);
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
    if (lane < 8) s_top[warp][lane] = top;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kWarps; ++x) top = fmaxf(top, s_top[x][row]);
    auto weigh = [&](int x, float2 v) {
      // a piece without a key that counts has zeros, or a NaN to pass on
      const float w = v.x == -INFINITY ? 1.f : ex2_approx(v.x - top);
      s_w[x][row] = w;
      sum = fmaf(w, v.y, sum);
    };
    if (mine) weigh(tid >> 3, ml);
    for (int x = (tid >> 3) + 2 * D / 8; x < pieces; x += 2 * D / 8) weigh(x, __ldcg(p.ml + slot(x) + row));
    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    if (lane < 8) s_sum[warp][lane] = sum;
    __syncthreads();
    if (tid < 8 && row0 + tid < rows) {
      sum = s_sum[0][tid];
#pragma unroll
      for (int x = 1; x < kWarps; ++x) sum += s_sum[x][tid];
      s_own[tid] = own_weight(top, sum, L);
      if (a.lse) a.lse[r0 + to(row0 + tid)] = s_own[tid].lse;  // (this thread alone read own_lse, which it may be)
    }
    float o[4] = {};
    for (int x0 = 0; x0 < pieces; x0 += kBatch) {
      if (x0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (x0 + i < pieces) f[i] = __ldcg(reinterpret_cast<const float4*>(p.o + slot(x0 + i) * D) + tid);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (x0 + i < pieces) {
          const float v[4] = {f[i].x, f[i].y, f[i].z, f[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = fmaf(s_w[x0 + i][row_of(e)], v[e], o[e]);
        }
    }
    __syncthreads();
    store(r0, row0, rows, to, o, own);
  }
}

int attn_check(const AttnParams& p, int D, int page_size, size_t es) {
  if (p.B <= 0 || p.T < 0 || p.Hq <= 0 || p.Hkv <= 0 || p.num_pages <= 0 || p.max_pages <= 0 || p.Hq % p.Hkv)
    return EAGLE_ERR_INVALID_ARG;
  if (!p.kc || !p.vc || !p.table || !p.cu || !p.ctx) return EAGLE_ERR_INVALID_ARG;
  if (p.T > 0 && (!p.q || !p.out)) return EAGLE_ERR_INVALID_ARG;  // (arrays of no rows may have no address)
  if (!(p.scale > 0.f) || !isfinite(p.scale) || !(p.k_scale > 0.f) || !(p.v_scale > 0.f) || !isfinite(p.k_scale) ||
      !isfinite(p.v_scale))
    return EAGLE_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || page_size != 16 || p.Hq / p.Hkv > 64 || p.B > 65535 || p.num_pages > kMaxPages)
    return EAGLE_ERR_UNSUPPORTED;
  if (p.q_stride < (long long)p.Hq * D || p.q_stride % (long long)(16 / es)) return EAGLE_ERR_INVALID_ARG;
  if (!aligned16(p.q) || !aligned16(p.kc) || !aligned16(p.vc) || !aligned16(p.out)) return EAGLE_ERR_INVALID_ARG;
  return EAGLE_OK;
}

struct Ws {
  PlanHeader* hdr;
  Piece* pieces;
  Cut* cuts;
  float2* ml;
  float* po;
};
Ws attn_ws(const Shape& sh, void* ws) {
  char* w = reinterpret_cast<char*>(round_up(reinterpret_cast<size_t>(ws), 256));
  return {reinterpret_cast<PlanHeader*>(w), reinterpret_cast<Piece*>(w + sh.off_pieces),
          reinterpret_cast<Cut*>(w + sh.off_cuts), reinterpret_cast<float2*>(w + sh.off_ml),
          reinterpret_cast<float*>(w + sh.off_o)};
}
void launch_plan(const AttnParams& a, const Shape& sh, const Ws& w, int min_cut, int min_cut_short, cudaStream_t s) {
  // a request ends at 2^30 tokens (the pages that ids can name), so that
  // positions and their blocks' ends stay below 2^31
  const int max_pages = std::min(a.max_pages, kMaxPages);
  const PlanParams pp = {a.cu, a.ctx, a.B, a.T, a.Hkv, max_pages, sh.tpu, sh.g, sh.ctas, sh.cap_pieces, sh.cap_slots, min_cut, min_cut_short,
                         w.hdr, w.pieces, w.cuts, a.status};
  launch(prompt_plan_kernel, 1, kPlanThreads, 0, s, pp);
}
template <int D, typename T>
int launch_merge(const AttnParams& a, const Shape& sh, const Ws& w, cudaStream_t s) {
  const MergeParams gp = {w.hdr, w.cuts, w.ml, w.po, a.out, a.lse, a.v_scale, a.Hq, sh.g, sh.tpu, sh.rows};
  launch(prompt_merge_kernel<D, T>, 2 * sh.ctas, 256, 0, s, gp);
  note_launch(3);
  return last_launch_status();
}
// The factor of the scores, in fp32's range (as row_factor).
float scale_log2(const AttnParams& a) {
  const double f = (double)a.scale * a.k_scale * 1.4426950408889634;
  return (float)std::min(std::max(f, (double)FLT_MIN), (double)FLT_MAX);
}
template <typename K>
bool allow_smem(K kern, int bytes) {
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess) return true;
  cudaGetLastError();
  return false;
}

template <int D, bool KV4, int NG>
int attn_launch_few(const AttnParams& a, void* ws, cudaStream_t s) {
  const Shape sh = attn_shape(a.B, a.T, a.Hq, a.Hkv, D, KV4 ? kFew4 : kFew);
  const Ws w = attn_ws(sh, ws);
  constexpr int smem = CfgFew<D, KV4, NG>::kSmem;
  if (!allow_smem(prompt_attn_few_kernel<D, KV4, NG>, smem)) return EAGLE_ERR_CUDA;
  // a token over 300 keys: 13.7 us in single blocks, 15.2 in pairs; over 1000:
  // 13.9, 14.9; over 4000, whose 32 pieces are joined: 18.4, 17.5
  launch_plan(a, sh, w, 2, 1, s);
  const FewParams fp = {a, scale_log2(a), sh.g, sh.rows, w.hdr, &w.hdr->next, w.pieces, w.cuts, w.ml, w.po};
  launch(prompt_attn_few_kernel<D, KV4, NG>, sh.ctas, kFewThreads, smem, s, fp);
  note_launch(2);
  return last_launch_status();
}
template <int D, bool KV4>
int attn_launch_tc(const AttnParams& a, void* ws, cudaStream_t s) {
  using C = Cfg<D, KV4>;
  if (few_rows(KV4, a.B, a.T, a.Hq, a.Hkv)) {
    if constexpr (KV4) {
      if (a.Hq / a.Hkv > 8) return attn_launch_few<D, KV4, 2>(a, ws, s);
    }
    return attn_launch_few<D, KV4, 1>(a, ws, s);
  }
  const Shape sh = attn_shape(a.B, a.T, a.Hq, a.Hkv, D, kTensor);
  const Ws w = attn_ws(sh, ws);
  CUtensorMap map_q = {};
  if (!KV4 && !make_tmap_3d_bf16(&map_q, a.q, D, (uint64_t)a.Hq, (uint64_t)a.T, (uint64_t)D * 2, (uint64_t)a.q_stride * 2,
                                 64, (uint32_t)sh.g, (uint32_t)sh.tpt))
    return EAGLE_ERR_CUDA;
  if (!allow_smem(prompt_attn_tc_kernel<D, KV4, false>, (int)C::kSmem)) return EAGLE_ERR_CUDA;
  launch_plan(a, sh, w, 2, 2, s);
  const MainParams mp = {a, scale_log2(a), sh.g, sh.tpt, sh.tpu, sh.rows, w.hdr, &w.hdr->next, w.pieces,
                         w.ml, w.po, nullptr, nullptr, nullptr};
  launch(prompt_attn_tc_kernel<D, KV4, false>, sh.ctas, kThreads, C::kSmem, s, map_q, mp);
  return launch_merge<D, __nv_bfloat16>(a, sh, w, s);
}
template <int D, int RT>
int attn_launch_f32(const AttnParams& a, void* ws, cudaStream_t s) {
  const Shape sh = attn_shape(a.B, a.T, a.Hq, a.Hkv, D, RT == 1 ? kFp32Few : kFp32);
  const Ws w = attn_ws(sh, ws);
  constexpr int smem = CfgF32<D, RT>::kSmem;
  if (!allow_smem(prompt_attn_f32_kernel<D, RT, false>, smem)) return EAGLE_ERR_CUDA;
  launch_plan(a, sh, w, 1, 1, s);
  const F32Params fp = {a, scale_log2(a), sh.g, sh.tpu, sh.rows, w.hdr, &w.hdr->next, w.pieces, w.ml, w.po, nullptr, nullptr, nullptr};
  launch(prompt_attn_f32_kernel<D, RT, false>, sh.ctas, 256, smem, s, fp);
  return launch_merge<D, float>(a, sh, w, s);
}
template <int D>
int attn_launch_f32(const AttnParams& a, void* ws, cudaStream_t s) {
  return few_rows_f32(a.B, a.T, a.Hq, a.Hkv) ? attn_launch_f32<D, 1>(a, ws, s) : attn_launch_f32<D, 4>(a, ws, s);
}

// Shared prefixes.  Units are those of the tensor-core or the fp32 path, or of one
// tile of the former.
struct FlatShape {
  int g, tpt, tpu, rows, ctas;
  size_t off_ml, off_o, total;  // the splits first
};
FlatShape flat_shape(int T, int Hq, int Hkv, int D, Path path, bool one_tile = false) {
  FlatShape s;
  const Shape x = attn_shape(1, T, Hq, Hkv, D, path);
  s.g = x.g, s.tpt = x.tpt, s.ctas = x.ctas;
  s.tpu = one_tile ? x.tpt : x.tpu;
  s.rows = (int)round_up(std::min(s.tpu, T) * s.g, 8);  // (the join takes eight at a time)
  s.off_ml = round_up(sizeof(Split) * (size_t)s.ctas, 256);
  s.off_o = round_up(s.off_ml + sizeof(float2) * 2 * (size_t)s.ctas * s.rows, 256);
  s.total = s.off_o + sizeof(float) * 2 * (size_t)s.ctas * s.rows * D + 256;
  return s;
}
struct FlatWs {
  Split* splits;
  float2* ml;
  float* o;
};
FlatWs flat_ws(const FlatShape& sh, void* ws) {
  char* w = reinterpret_cast<char*>(round_up(reinterpret_cast<size_t>(ws), 256));
  return {reinterpret_cast<Split*>(w), reinterpret_cast<float2*>(w + sh.off_ml), reinterpret_cast<float*>(w + sh.off_o)};
}
// Few rows of all groups together: units of one tile, whose key blocks both tiles'
// warps share, so that there are twice as many, shorter pieces.  32 + 8 heads, D 128,
// one tile / two, us: 64 tokens (256 rows of a kv head) over 500, 2,000 and 8,000 keys
// 13.4 / 15.7, 14.3 / 16.3, 19.9 / 20.5, in 4-bit pages 16.9 / 20.0, 17.8 / 21.1, 25.4 /
// 26.5; 128 tokens 14.8 / 16.9, 17.6 / 18.8, 28.9 / 27.2; 256 tokens over 8,000 46.7 /
// 44.1, 1,024 over 500 34.6 / 21.2 (keys are read and brought to shared memory twice as
// often).
constexpr int kOneTileRows = 256;
bool flat_one_tile(int T, int Hq, int Hkv) { return (long long)T * (Hq / Hkv) <= kOneTileRows; }
struct Own {
  const void* out;
  const float* lse;
};
template <int D, typename T>
int flat_join(const AttnParams& a, const Own& own, const FlatShape& sh, const FlatWs& w, cudaStream_t s) {
  // CTAs for the chunks of eight rows that there can be, and one more (where they are more
  // than the CTAs, one an SM more)
  const int sms = std::max(1, sm_count());
  const JoinParams jp = {a, sh.g, sh.tpu, sh.rows, sh.ctas, w.splits, w.ml, w.o, own.out, own.lse};
  const long long units = ((long long)a.T + (long long)std::min(a.B, a.T) * (sh.tpu - 1)) / sh.tpu * a.Hkv;
  const long long chunks = std::min<long long>(units, sh.ctas) * (sh.rows / 8);
  // Few chunks, two a SM at most: 20 pieces' loads at a time and all their CTAs at once,
  // since the chain of loads is what they wait for (64 tokens over 8,000 keys 20.0 us,
  // 4 over 32,768 35.3; the other way 22.0 and 38.6).  More: two pieces at a time, for
  // more CTAs a SM (1,885 rows in two groups 128 us, 158 the first way).
  constexpr int kFew = 2, kMany = 640 / D;
  if (chunks <= (long long)kFew * sms)
    launch(flat_join_kernel<D, T, 20, 256 / D, false>, (int)chunks + 1, 2 * D, 0, s, jp);
  else
    launch(flat_join_kernel<D, T, 2, kMany, true>, (int)std::min<long long>(chunks, kMany * sms) + sh.ctas, 2 * D, 0, s, jp);
  note_launch(2);
  return last_launch_status();
}
template <int D, bool KV4>
int flat_launch_tc(const AttnParams& a, const Own& own, void* ws, cudaStream_t s) {
  using C = Cfg<D, KV4>;
  const FlatShape sh = flat_shape(a.T, a.Hq, a.Hkv, D, kTensor, flat_one_tile(a.T, a.Hq, a.Hkv));
  const FlatWs w = flat_ws(sh, ws);
  if (sh.ctas > kMaxParts) return EAGLE_ERR_UNSUPPORTED;
  CUtensorMap map_q = {};
  if (!KV4 && !make_tmap_3d_bf16(&map_q, a.q, D, (uint64_t)a.Hq, (uint64_t)a.T, (uint64_t)D * 2, (uint64_t)a.q_stride * 2,
                                 64, (uint32_t)sh.g, (uint32_t)sh.tpt))
    return EAGLE_ERR_CUDA;
  if (!allow_smem(prompt_attn_tc_kernel<D, KV4, true>, (int)C::kSmem)) return EAGLE_ERR_CUDA;
  const MainParams mp = {a, scale_log2(a), sh.g, sh.tpt, sh.tpu, sh.rows, nullptr, nullptr, nullptr, w.ml, w.o, own.out, own.lse, w.splits};
  launch(prompt_attn_tc_kernel<D, KV4, true>, sh.ctas, kThreads, C::kSmem, s, map_q, mp);
  return flat_join<D, __nv_bfloat16>(a, own, sh, w, s);
}
template <int D, int RT>
int flat_launch_f32(const AttnParams& a, const Own& own, void* ws, cudaStream_t s) {
  const FlatShape sh = flat_shape(a.T, a.Hq, a.Hkv, D, RT == 1 ? kFp32Few : kFp32);
  const FlatWs w = flat_ws(sh, ws);
  if (sh.ctas > kMaxParts) return EAGLE_ERR_UNSUPPORTED;
  constexpr int smem = CfgF32<D, RT>::kSmem;
  if (!allow_smem(prompt_attn_f32_kernel<D, RT, true>, smem)) return EAGLE_ERR_CUDA;
  const F32Params fp = {a, scale_log2(a), sh.g, sh.tpu, sh.rows, nullptr, nullptr, nullptr, w.ml, w.o,
                        static_cast<const float*>(own.out), own.lse, w.splits};
  launch(prompt_attn_f32_kernel<D, RT, true>, sh.ctas, 256, smem, s, fp);
  return flat_join<D, float>(a, own, sh, w, s);
}
template <int D>
int flat_launch_f32(const AttnParams& a, const Own& own, void* ws, cudaStream_t s) {
  return few_rows_f32(a.B, a.T, a.Hq, a.Hkv) ? flat_launch_f32<D, 1>(a, own, ws, s) : flat_launch_f32<D, 4>(a, own, ws, s);
}
// What a shared prefix needs beside attn_check().
int flat_check(const AttnParams& a, const Own& own, int D, void* ws, size_t ws_bytes) {
  if (a.B > kMaxGroups) return EAGLE_ERR_UNSUPPORTED;
  if ((own.out != nullptr) != (own.lse != nullptr) && a.T > 0) return EAGLE_ERR_INVALID_ARG;
  if (!aligned16(own.out)) return EAGLE_ERR_INVALID_ARG;
  if (a.T > 0 && (!ws || ws_bytes < eagle_prefix_attn_workspace_size(a.B, a.T, a.Hq, a.Hkv, D))) return EAGLE_ERR_WORKSPACE;
  return EAGLE_OK;
}

int attn_ws_check(const AttnParams& a, int D, void* ws, size_t ws_bytes) {
  return !ws || ws_bytes < eagle_prompt_attn_workspace_size(a.B, a.T, a.Hq, a.Hkv, D) ? EAGLE_ERR_WORKSPACE : EAGLE_OK;
}

}  // namespace
}  // namespace eagle

using namespace eagle;

extern "C" size_t eagle_prompt_attn_workspace_size(int B, int T, int Hq, int Hkv, int D) {
  if (B <= 0 || T < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hq / Hkv > 64 || (D != 64 && D != 128)) return 0;
  // the largest of the paths that some call of at most these B and T takes, each
  // at the most rows that it takes: a workspace serves all those calls
  const long long g = Hq / Hkv;
  auto rows = [&](long long limit) { return (int)std::min<long long>(T, limit); };
  const struct {
    Path path;
    int T;
  } calls[] = {{kTensor, T}, {kFew, rows(B)}, {kFew4, rows(2ll * B)}, {kFp32, T}, {kFp32Few, rows((long long)kF32Few * B / g)}};
  size_t most = 0;
  for (const auto& c : calls) most = std::max(most, attn_shape(B, c.T, Hq, Hkv, D, c.path).total);
  return most + 256;
}

extern "C" int eagle_prompt_attn(const void* q, long long q_stride, const void* k_cache, const void* v_cache,
                                 int num_pages, const int32_t* block_table, int max_pages, const int32_t* cu_seqlens,
                                 const int32_t* ctx_lens, void* out, float* lse, int B, int T, int Hq, int Hkv, int D,
                                 int page_size, float scale, int dtype, void* ws, size_t ws_bytes,
                                 int32_t* dev_status, void* stream) {
  if (dtype != EAGLE_BF16 && dtype != EAGLE_FP32) return EAGLE_ERR_INVALID_ARG;
  const AttnParams p = {q, q_stride, k_cache, v_cache, nullptr, nullptr, 1.f, 1.f, num_pages, max_pages, B, T, Hq, Hkv,
                        block_table, cu_seqlens, ctx_lens, out, lse, scale, dev_status};
  const int rc = attn_check(p, D, page_size, dtype == EAGLE_BF16 ? 2 : 4);
  if (rc != EAGLE_OK) return rc;
  if (T == 0) return EAGLE_OK;
  const int wrc = attn_ws_check(p, D, ws, ws_bytes);
  if (wrc != EAGLE_OK) return wrc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == EAGLE_BF16) return D == 128 ? attn_launch_tc<128, false>(p, ws, s) : attn_launch_tc<64, false>(p, ws, s);
  return D == 128 ? attn_launch_f32<128>(p, ws, s) : attn_launch_f32<64>(p, ws, s);
}

extern "C" int eagle_prompt_attn_kv4(const void* q, long long q_stride, const uint8_t* k_codes,
                                     const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales,
                                     float k_scale, float v_scale, int num_pages, const int32_t* block_table,
                                     int max_pages, const int32_t* cu_seqlens, const int32_t* ctx_lens, void* out,
                                     float* lse, int B, int T, int Hq, int Hkv, int D, int page_size, float scale,
                                     void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  const AttnParams p = {q, q_stride, k_codes, v_codes, k_scales, v_scales, k_scale, v_scale, num_pages, max_pages, B, T,
                        Hq, Hkv, block_table, cu_seqlens, ctx_lens, out, lse, scale, dev_status};
  if (!k_scales || !v_scales || !aligned16(k_scales) || !aligned16(v_scales)) return EAGLE_ERR_INVALID_ARG;
  const int rc = attn_check(p, D, page_size, 2);
  if (rc != EAGLE_OK) return rc;
  if (T == 0) return EAGLE_OK;
  const int wrc = attn_ws_check(p, D, ws, ws_bytes);
  if (wrc != EAGLE_OK) return wrc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return D == 128 ? attn_launch_tc<128, true>(p, ws, s) : attn_launch_tc<64, true>(p, ws, s);
}

extern "C" size_t eagle_prefix_attn_workspace_size(int G, int T, int Hq, int Hkv, int D) {
  if (G <= 0 || G > kMaxGroups || T < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hq / Hkv > 64 || (D != 64 && D != 128)) return 0;
  const int few = (int)std::min<long long>(T, (long long)kF32Few * G / (Hq / Hkv));
  size_t most = 0;
  for (const Path path : {kTensor, kFp32}) most = std::max(most, flat_shape(T, Hq, Hkv, D, path).total);
  return std::max(most, flat_shape(few, Hq, Hkv, D, kFp32Few).total) + 256;
}

extern "C" int eagle_prefix_attn(const void* q, long long q_stride, const void* k_cache, const void* v_cache, int num_pages,
                                 const int32_t* prefix_table, int max_pages, const int32_t* cu_rows,
                                 const int32_t* prefix_lens, const void* own_out, const float* own_lse, void* out,
                                 float* lse, int G, int T, int Hq, int Hkv, int D, int page_size, float scale, int dtype,
                                 void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (dtype != EAGLE_BF16 && dtype != EAGLE_FP32) return EAGLE_ERR_INVALID_ARG;
  const AttnParams p = {q, q_stride, k_cache, v_cache, nullptr, nullptr, 1.f, 1.f, num_pages, max_pages, G, T, Hq, Hkv,
                        prefix_table, cu_rows, prefix_lens, out, lse, scale, dev_status};
  const Own own = {own_out, own_lse};
  int rc = attn_check(p, D, page_size, dtype == EAGLE_BF16 ? 2 : 4);
  if (rc == EAGLE_OK) rc = flat_check(p, own, D, ws, ws_bytes);
  if (rc != EAGLE_OK || T == 0) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == EAGLE_BF16)
    return D == 128 ? flat_launch_tc<128, false>(p, own, ws, s) : flat_launch_tc<64, false>(p, own, ws, s);
  return D == 128 ? flat_launch_f32<128>(p, own, ws, s) : flat_launch_f32<64>(p, own, ws, s);
}

extern "C" int eagle_prefix_attn_kv4(const void* q, long long q_stride, const uint8_t* k_codes, const uint8_t* k_scales,
                                     const uint8_t* v_codes, const uint8_t* v_scales, float k_scale, float v_scale,
                                     int num_pages, const int32_t* prefix_table, int max_pages, const int32_t* cu_rows,
                                     const int32_t* prefix_lens, const void* own_out, const float* own_lse, void* out,
                                     float* lse, int G, int T, int Hq, int Hkv, int D, int page_size, float scale,
                                     void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  const AttnParams p = {q, q_stride, k_codes, v_codes, k_scales, v_scales, k_scale, v_scale, num_pages, max_pages, G, T,
                        Hq, Hkv, prefix_table, cu_rows, prefix_lens, out, lse, scale, dev_status};
  if (!k_scales || !v_scales || !aligned16(k_scales) || !aligned16(v_scales)) return EAGLE_ERR_INVALID_ARG;
  const Own own = {own_out, own_lse};
  int rc = attn_check(p, D, page_size, 2);
  if (rc == EAGLE_OK) rc = flat_check(p, own, D, ws, ws_bytes);
  if (rc != EAGLE_OK || T == 0) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return D == 128 ? flat_launch_tc<128, true>(p, own, ws, s) : flat_launch_tc<64, true>(p, own, ws, s);
}
