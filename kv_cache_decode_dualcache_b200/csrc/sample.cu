// fdllm_sample: one token per row of logits with temperature, top-k, top-p
// and min-p, drawn with a given uniform number.
//
// A row is split over the CTAs of a thread-block cluster and read from
// memory once, into their shared memories (or, with many long rows, into L2);
// everything else happens there and over distributed shared memory, in one
// launch without a workspace.
//
// The kept tokens are a prefix of the row sorted by (falling logit, rising
// id).  Usually a small superset of them is known early: min-p bounds
// z = (m - l) / T; the top_k-th largest of the threads' own maxima bounds the
// top_k-th token; a histogram of the weights bounds the nucleus.  Then the
// superset is gathered (at most CAP tokens), ordered by one CTA (by counting,
// or a sort if it is large), and the filters and the draw are prefix sums.  Larger kept sets are described by
// a cut, the last kept token, found on counts (top-k) or weight sums (top-p)
// by a histogram over 256 linear bins of z in [0, 32) (a token beyond weighs
// under 2^-45 and cannot be drawn), one over 256 bins of the bin the cut
// falls into, and the exact order of the few tokens of that small bin; if
// even that holds more than CAP tokens (thousands of equal logits), by
// bisection over the logit's bits.  The draw then walks the ids in order.
// Bins are linear in z and not in the logit's bits because that spreads a
// row's tokens evenly: the shared-memory atomics of a warp then rarely meet.
//
// Weights are held as integers, w = rint(exp(-z) 2^44) with the exponential
// in float64: sums of up to 2^18 weights are exact in 64 bits, so no order
// of additions can change a cut or a token.
//
// Bound: for few rows the chain of cluster barriers (one row of 152064 float32
// logits, all filters: 12 us); for many rows too, for a row's chain (maximum,
// bound, gathered tokens, their order) takes 15 to 25 us of a CTA and an SM holds
// two or three (512 rows of 126464 bf16 logits: 130 us, 1.0 TB/s, the last rows
// being wide nuclei of 60 us each; 32 rows of float32 with wide nuclei: 35 us).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "kv8.h"

namespace fd {
namespace {

constexpr int ST = 512;                      // threads of a CTA
constexpr int SW = ST / 32;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_VOCAB = 1 << 18;
constexpr int MAX_SLICE = 1 << 16;           // tokens of a CTA (histogram words hold 2^16 x 2^15)
constexpr int SLICE_BYTES = 78 << 10;        // two CTAs and their lists fit on an SM
constexpr int BINS = 256;
constexpr float Z_BINS = 8.0f;               // bins per unit of z: 256 / 32
constexpr int CAP = 1024;                    // tokens that are gathered and sorted
// Tokens whose order is taken by counting, which keeps all warps busy where the
// steps of a sort wait for one another: 37 rows with about 250 tokens 31 us, 36 us
// sorted; no gain above.
constexpr int DIRECT = 384;
constexpr double W_ONE = 17592186044416.0;   // 2^44

typedef unsigned long long u64;

// Order-preserving key of a live logit (> -inf).
FD_DEV uint32_t logit_key(float l) {
  const uint32_t u = __float_as_uint(l + 0.0f);   // -0 and +0 are equal logits
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
FD_DEV float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// A token's place in the order: larger first; equal logits, the lower id.
FD_DEV u64 order_of(float l, int id) { return ((u64)logit_key(l) << 32) | (uint32_t)~(uint32_t)id; }
FD_DEV float order_logit(u64 o) { return key_logit((uint32_t)(o >> 32)); }
FD_DEV int order_id(u64 o) { return (int)~(uint32_t)o; }

struct __align__(16) Shared {
  double exp2_64[64];          // 2^(j / 64)
  uint32_t hist[2][3][BINS];   // weights in words of 15, 15 and 15 bits, or counts
  u64 red[SW];
  u64 part[2];                 // this CTA's share of a cluster sum (by parity of use)
  u64 before, upto;
  float top;                   // this CTA's largest logit
  int bin, n_hot, n_list, n_sub, cut_id, cut_ties, pick;
  int run0, run1;              // the run of ids that holds the drawn token
  uint32_t cut_key;
  uint16_t hot[ST];            // threads that hold a token within the bound
  u64 list[CAP];               // this CTA's gathered tokens (order_of)
  u64 all[CAP];                // the cluster's
  u64 w[CAP];                  // their weights
  u64 sub[CAP];                // this CTA's tokens of the smaller bin
};

// 2^(j / 64)
__device__ const double EXP2_64[64] = {
    1.0, 1.0108892860517005, 1.0218971486541166, 1.0330248790212284,
    1.0442737824274138, 1.0556451783605572, 1.0671404006768237, 1.0787607977571199,
    1.0905077326652577, 1.102382583307841, 1.1143867425958924, 1.1265216186082418,
    1.1387886347566916, 1.1511892299529827, 1.1637248587775775, 1.1763969916502812,
    1.189207115002721, 1.202156731452703, 1.215247359980469, 1.22848053610687,
    1.241857812073484, 1.255380757024691, 1.2690509571917332, 1.2828700160787783,
    1.2968395546510096, 1.3109612115247644, 1.3252366431597413, 1.339667524053303,
    1.3542555469368927, 1.3690024229745905, 1.383909881963832, 1.3989796725383112,
    1.4142135623730951, 1.42961333839197, 1.4451808069770467, 1.460917794180647,
    1.4768261459394993, 1.4929077282912648, 1.5091644275934228, 1.5255981507445384,
    1.5422108254079407, 1.559004400237837, 1.5759808451078865, 1.593142151342267,
    1.6104903319492543, 1.6280274218573478, 1.645755478153965, 1.6636765803267364,
    1.681792830507429, 1.7001063537185235, 1.718619298122478, 1.7373338352737062,
    1.7562521603732995, 1.7753764925265212, 1.7947090750031072, 1.8142521755003989,
    1.8340080864093424, 1.8539791250833855, 1.8741676341103, 1.8945759815869656,
    1.9152065613971474, 1.9360617934922943, 1.9571441241754002, 1.978456026387951};

FD_DEV uint32_t ld_remote32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_map(smem_u32(p), rank)) : "memory");
  return v;
}
FD_DEV u64 ld_remote64(const void* p, uint32_t rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_map(smem_u32(p), rank)) : "memory");
  return v;
}

// The row's state that every thread of the cluster knows.
struct Row {
  float m;          // largest logit
  float zs;         // bins per unit of logit
  double md, y;     // m; 64 log2(e) / T
  const double* exp2_64;
  // the cut: kept are key > cut_key, and key == cut_key with id <= cut_id
  uint32_t cut_key;
  int cut_id;
  int ties;         // kept tokens with key == cut_key
  bool has_cut, listed;   // listed: the class of cut_key is in Shared::all[0 .. n_list)
};

// exp((l - m) / T) = 2^((n + f) / 64) of a token with z < BINS (anything for
// others): 2^(n / 64) from the table and the exponent, 2^(f / 64), |f| <= 1/2,
// by its Taylor polynomial (error below (ln 2 / 128)^5 / 120 = 4e-14).
// Without a branch, so that the chains of several tokens overlap.
FD_DEV double weight(const Row& r, float l) {
  const double y = ((double)l - r.md) * r.y;   // 64 log2 of the weight
  const double magic = 6755399441055744.0;     // 1.5 2^52: its sum with y is an integer
  const double t = y + magic;
  const int n = __double2loint(t);
  const double f = y - (t - magic);
  constexpr double c = 0.010830424696249145;   // ln 2 / 64
  double p = fma(f, c * c * c * c / 24.0, c * c * c / 6.0);
  p = fma(f, p, c * c / 2.0);
  p = fma(f, p, c);
  const double s = r.exp2_64[n & 63];
  const double w = fma(f * p, s, s);
  return __hiloint2double(__double2hiint(w) + ((n >> 6) << 20), __double2loint(w));
}
// rint(w 2^44): the sum with 2^52 is an integer in the low bits.
FD_DEV u64 fixed(double w) {
  return (u64)__double_as_longlong(fma(w, W_ONE, 4503599627370496.0)) & 0xfffffffffffffull;
}

// Place of a token among the bins; not below BINS: not live (-inf, NaN), or
// too light to be drawn.  Rounded on its own (no fused z - bin), so that every
// pass puts a token into the same bin.
FD_DEV float z_of(const Row& r, float l) { return __fmul_rn(r.m - l, r.zs); }
FD_DEV bool below_cut(const Row& r, float l) { return r.has_cut && logit_key(l) <= r.cut_key; }

// A CTA's tokens: a copy in shared memory, prepared when it was made, or the
// logits themselves (16-byte aligned), prepared when they are read.
template <typename T, bool STAGED>
struct Slice {
  static constexpr int VEC = 16 / sizeof(T);
  const T* p;
  int n, mask;    // mask: index of the masked token, out of [0, n) if it is not here
  bool inf;       // infinite logits count as equal ones, the rest as -inf
  FD_DEV float fix(float l, int i) const {
    if (STAGED) return l;
    if (i == mask) l = -INFINITY;
    if (inf) l = l == INFINITY ? 0.0f : -INFINITY;
    return l;
  }
  FD_DEV float at(int i) const { return fix(to_f<T>(p[i]), i); }
  // logits of tokens i VEC .. i VEC + VEC - 1, -inf behind the last one
  FD_DEV void vec(int i, float* l) const {
    uint4 u;
    T* e = reinterpret_cast<T*>(&u);
    if (STAGED || (i + 1) * VEC <= n) {
      u = reinterpret_cast<const uint4*>(p)[i];
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) e[j] = i * VEC + j < n ? p[i * VEC + j] : from_f<T>(-INFINITY);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) l[j] = fix(to_f<T>(e[j]), i * VEC + j);
  }
};

// Largest of two vectors element by element, in their type; NaN never wins.
template <typename T> FD_DEV uint4 max_vec(uint4 a, uint4 b) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&a);
  const uint32_t* y = reinterpret_cast<const uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same_v<T, float>)
      x[i] = __float_as_uint(fmaxf(__uint_as_float(x[i]), __uint_as_float(y[i])));
    else if constexpr (std::is_same_v<T, __half>)
      asm("max.f16x2 %0, %0, %1;" : "+r"(x[i]) : "r"(y[i]));
    else
      asm("max.bf16x2 %0, %0, %1;" : "+r"(x[i]) : "r"(y[i]));
  }
  return a;
}

// f(index, logits) for the slice's tokens, 16 bytes at a time.
template <typename X, typename F>
FD_DEV void for_vectors(const X& x, F f) {
  for (int i = threadIdx.x; i * X::VEC < x.n; i += ST) {
    float l[X::VEC];
    x.vec(i, l);
    f(i * X::VEC, l);
  }
}
// f(index, logit) for the slice's tokens with pred(logit), for rare ones: a
// thread first marks its hits among 32 tokens, then visits them, so that a
// warp runs f as often as its busiest lane has hits.
template <typename X, typename P, typename F>
FD_DEV void for_hits(const X& x, P pred, F f) {
  constexpr int VEC = X::VEC, G = 32 / VEC;
  for (int i0 = threadIdx.x; i0 * VEC < x.n; i0 += G * ST) {
    uint32_t hits = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int i = i0 + g * ST;
      if (i * VEC < x.n) {
        float l[VEC];
        x.vec(i, l);
#pragma unroll
        for (int j = 0; j < VEC; ++j) hits |= pred(l[j]) ? 1u << (g * VEC + j) : 0u;
      }
    }
    while (hits) {
      const int b = __ffs(hits) - 1;
      hits &= hits - 1;
      const int i = (i0 + (b / VEC) * ST) * VEC + b % VEC;
      f(i, x.at(i));
    }
  }
}

FD_DEV u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Every thread owns a run of ids, [tid run, tid run + run): an odd number of
// vectors, so that the threads' reads of shared memory meet no bank twice.
template <typename X>
FD_DEV int run_of(const X& x) { return ((x.n + ST * X::VEC - 1) / (ST * X::VEC) | 1) * X::VEC; }
// Sum of f(logit) over the thread's run, of tokens with pred(index, logit).
// They are marked first, so that a warp runs f as often as its busiest lane
// has them.
template <typename X, typename P, typename F>
FD_DEV u64 run_sum(const X& x, P pred, F f) {
  constexpr int VEC = X::VEC;
  const int run = run_of(x), i0 = threadIdx.x * run, i1 = min(i0 + run, x.n);
  u64 sum = 0;
  for (int j0 = i0; j0 < i1; j0 += 32) {
    uint32_t hits = 0;
#pragma unroll
    for (int g = 0; g < 32; g += VEC) {
      if (j0 + g >= i1) break;
      float l[VEC];
      x.vec((j0 + g) / VEC, l);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (pred(j0 + g + j, l[j])) hits |= 1u << (g + j);
    }
    while (hits) {
      const int j = __ffs(hits) - 1;
      hits &= hits - 1;
      sum += f(x.at(j0 + j));
    }
  }
  return sum;
}
// Inclusive prefix sum over the threads; *total over all of them.
template <typename U>
FD_DEV U block_scan(U v, Shared& s, U* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const U y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  U* red = reinterpret_cast<U*>(s.red);
  if (lane == 31) red[warp] = v;
  __syncthreads();
  U t = 0;
#pragma unroll
  for (int i = 0; i < SW; ++i) {
    const U x = red[i];
    if (i < warp) v += x;
    t += x;
  }
  *total = t;
  return v;
}
FD_DEV u64 block_sum(u64 v, Shared& s) {
  v = warp_sum64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 t = 0;
#pragma unroll
  for (int i = 0; i < SW; ++i) t += s.red[i];
  return t;
}
// Sum of v over the CTAs (v the same in all threads of a CTA), and over those
// of lower rank.  Alternate `use`: a part is rewritten two uses later.
FD_DEV u64 cluster_total(u64 v, Shared& s, int n_cta, int rank, int use, u64* lower) {
  if (threadIdx.x == 0) s.part[use & 1] = v;
  cluster_sync();
  u64 t = 0, lo = 0;
#pragma unroll
  for (int i = 0; i < MAX_CLUSTER; ++i) {
    const u64 x = i < n_cta ? ld_remote64(&s.part[use & 1], i) : 0;
    t += x;
    if (i < rank) lo += x;
  }
  if (lower) *lower = lo;
  return t;
}

FD_DEV void zero_hist(Shared& s, int h) {
  for (int i = threadIdx.x; i < 3 * BINS; i += ST) (&s.hist[h][0][0])[i] = 0;
}
template <bool MASS>
FD_DEV void hist_add(Shared& s, int h, int bin, u64 w) {
  if (MASS) {
    const uint32_t lo = (uint32_t)w, hi = (uint32_t)(w >> 30);
    atomicAdd(&s.hist[h][0][bin], lo & 0x7fff);
    atomicAdd(&s.hist[h][1][bin], (lo >> 15) & 0x7fff);
    if (hi) atomicAdd(&s.hist[h][2][bin], hi);
  } else {
    atomicAdd(&s.hist[h][0][bin], 1u);
  }
}

// The bin in which the running sum over the bins of all CTAs (weights, or
// counts) reaches `need` = need_of(sum of all bins) goes to s.bin, what lies
// before it to s.before, and up to its end to s.upto.  *above: the sum of
// all bins.
template <bool MASS, typename F>
FD_DEV u64 find_bin(Shared& s, int h, int n_cta, u64* above, F need_of) {
  // two threads a bin, each for half of the CTAs
  const int bin = threadIdx.x >> 1, half = threadIdx.x & 1;
  typedef std::conditional_t<MASS, u64, uint32_t> U;
  U v = 0, sum;
#pragma unroll
  for (int j = 0; j < MAX_CLUSTER / 2; ++j) {
    const int i = 2 * j + half;
    if (i >= n_cta) continue;
    v += ld_remote32(&s.hist[h][0][bin], i);
    if constexpr (MASS)
      v += ((u64)ld_remote32(&s.hist[h][1][bin], i) << 15) +
           ((u64)ld_remote32(&s.hist[h][2][bin], i) << 30);
  }
  const U upto = block_scan(v, s, &sum);
  *above = sum;
  const u64 need = need_of(*above);
  const U bin_sum = v + __shfl_xor_sync(0xffffffffu, v, 1);
  if (half == 1 && upto - bin_sum < need && need <= upto) {
    s.bin = bin;
    s.before = upto - bin_sum;
    s.upto = upto;
  }
  __syncthreads();
  return need;
}

// Sets the cut to the `ties`-th token (by id) of the class with key r.cut_key.
template <typename X>
FD_DEV void nth_tie(Shared& s, Row& r, int ties, const X& x, int id0, int n_cta, int rank,
                    int& use) {
  r.ties = ties;
  if (r.listed) {
    for (int j = threadIdx.x; j < s.n_list; j += ST) {
      if ((uint32_t)(s.all[j] >> 32) != r.cut_key) continue;
      int before = 0;
      for (int i = 0; i < s.n_list; ++i)
        before += (uint32_t)(s.all[i] >> 32) == r.cut_key && s.all[i] > s.all[j];
      if (before == ties - 1) s.cut_id = order_id(s.all[j]);
    }
    __syncthreads();
    r.cut_id = s.cut_id;
    __syncthreads();
    return;
  }
  const float lc = key_logit(r.cut_key);
  u64 lower, cta;
  const u64 mine = run_sum(x, [&](int, float l) { return l == lc; }, [](float) { return (u64)1; });
  u64 before = block_scan(mine, s, &cta) - mine;
  cluster_total(cta, s, n_cta, rank, use++, &lower);
  before += lower;
  if (threadIdx.x == 0) s.cut_id = -1;
  __syncthreads();
  if (before < (u64)ties && (u64)ties <= before + mine) {
    const int run = run_of(x), i0 = threadIdx.x * run;
    for (int i = i0; i < min(i0 + run, x.n); ++i)
      if (x.at(i) == lc && ++before == (u64)ties) s.cut_id = id0 + i;
  }
  __syncthreads();
  // the CTA that holds it tells the others (ids as id + 1, none = 0)
  r.cut_id = (int)cluster_total((u64)(s.cut_id + 1), s, n_cta, rank, use++, nullptr) - 1;
}

// First step of a search: the bin of z in which the sum over the kept tokens
// reaches need_of(all of it).
struct Level {
  u64 need, above, before, upto;   // above: strictly above the cut
  int bin;                         // valid if 0 < need <= above
};
template <bool MASS, typename X, typename F>
FD_DEV Level level1(Shared& s, const Row& r, const X& x, int n_cta, F need_of) {
  const u64 at_cut = r.has_cut ? (u64)r.ties * (MASS ? fixed(weight(r, key_logit(r.cut_key))) : 1) : 0;
  for_vectors(x, [&](int, const float* l) {
    constexpr int VEC = X::VEC;
    u64 w[VEC];
    if (MASS) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) w[j] = fixed(weight(r, l[j]));   // chains side by side
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float z = z_of(r, l[j]);
      if (z < (float)BINS && !below_cut(r, l[j])) hist_add<MASS>(s, 0, (int)z, MASS ? w[j] : 0);
    }
  });
  cluster_sync();
  Level v;
  v.need = find_bin<MASS>(s, 0, n_cta, &v.above, [&](u64 t) { return need_of(t + at_cut); });
  v.bin = s.bin;
  v.before = s.before;
  v.upto = s.upto;
  return v;
}

// Moves the cut to the token at which the sum reaches v.need.
template <bool MASS, typename X>
FD_DEV void refine(Shared& s, Row& r, const Level& v, const X& x, int id0, int n_cta, int rank,
                   int& use) {
  const int tid = threadIdx.x;
  auto unit = [&](float l) { return MASS ? fixed(weight(r, l)) : (u64)1; };
  if (v.need == 0 || v.need > v.above) {
    const bool first = v.need == 0;   // only the first token
    int ties = 1;
    if (!first && r.has_cut) {
      const u64 w = unit(key_logit(r.cut_key));
      ties = w ? (int)min((v.need - v.above + w - 1) / w, (u64)r.ties) : r.ties;
    }
    // the first histogram is free again once every CTA has read it
    cluster_sync();
    zero_hist(s, 0);
    __syncthreads();
    if (first) {
      r.cut_key = logit_key(r.m);
      r.has_cut = true;
      r.listed = false;
      nth_tie(s, r, 1, x, id0, n_cta, rank, use);
    } else if (r.has_cut && ties < r.ties) {
      nth_tie(s, r, ties, x, id0, n_cta, rank, use);
    }
    return;
  }
  // this CTA's tokens of the bin as a list; a list that overflows is replaced
  // by passes over the slice
  const float lo = (float)v.bin;
  auto in_bin1 = [&](float l) {
    const float z = z_of(r, l) - lo;
    return z >= 0.0f && z < 1.0f && !below_cut(r, l);
  };
  auto bin2 = [&](float l) { return (int)((z_of(r, l) - lo) * BINS); };
  if (tid == 0) s.n_list = s.n_sub = 0;
  __syncthreads();
  for_hits(x, in_bin1, [&](int i, float l) {
    const int at = atomicAdd(&s.n_list, 1);
    if (at < CAP) s.list[at] = order_of(l, id0 + i);
  });
  __syncthreads();
  const int n1 = s.n_list;
  auto for_bin = [&](auto f) {
    if (n1 <= CAP)
      for (int j = tid; j < n1; j += ST) f(s.list[j]);
    else
      for_hits(x, in_bin1, [&](int i, float l) { f(order_of(l, id0 + i)); });
  };
  for_bin([&](u64 o) {
    const float l = order_logit(o);
    hist_add<MASS>(s, 1, bin2(l), MASS ? unit(l) : 0);
  });
  cluster_sync();
  zero_hist(s, 0);   // every CTA has read it
  u64 total;
  find_bin<MASS>(s, 1, n_cta, &total, [&](u64) { return v.need - v.before; });
  const int b2 = s.bin;
  const u64 before = v.before + s.before;
  auto in_bin = [&](float l) { return in_bin1(l) && bin2(l) == b2; };
  for_bin([&](u64 o) {
    if (bin2(order_logit(o)) == b2) {
      const int at = atomicAdd(&s.n_sub, 1);
      if (at < CAP) s.sub[at] = o;
    }
  });
  cluster_sync();
  zero_hist(s, 1);
  int n_all = 0;
#pragma unroll
  for (int c = 0; c < MAX_CLUSTER; ++c) {
    const int nc = c < n_cta ? (int)ld_remote32(&s.n_sub, c) : 0;
    if (n_all + nc <= CAP)
      for (int j = tid; j < nc; j += ST) {
        const u64 o = ld_remote64(&s.sub[j], c);
        s.all[n_all + j] = o;
        s.w[n_all + j] = unit(order_logit(o));
      }
    n_all += nc;
  }
  cluster_sync();   // every CTA has read the lists and their lengths
  if (n_all <= CAP) {
    for (int j = tid; j < n_all; j += ST) {
      const u64 o = s.all[j];
      u64 sum = before;
      int ties = 1;
      for (int i = 0; i < n_all; ++i) {
        const bool over = s.all[i] > o;
        if (over) sum += s.w[i];
        ties += over && (s.all[i] >> 32) == (o >> 32);
      }
      if (sum < v.need && v.need <= sum + s.w[j]) {
        s.cut_key = (uint32_t)(o >> 32);
        s.cut_id = order_id(o);
        s.cut_ties = ties;
      }
    }
    if (tid == 0) s.n_list = n_all;
    __syncthreads();
    r.cut_key = s.cut_key;
    r.cut_id = s.cut_id;
    r.ties = s.cut_ties;
    r.has_cut = r.listed = true;
    __syncthreads();
    return;
  }
  // too many: bisect over the keys for the largest one that reaches need
  uint32_t k0 = r.has_cut ? r.cut_key + 1 : 1, k1 = logit_key(r.m);
  const uint32_t kmax = k1;
  auto upto = [&](uint32_t k) {   // sum up to and over the bin's tokens with key >= k
    u64 t = 0;
    for_hits(x, [&](float l) { return in_bin(l) && logit_key(l) >= k; },
             [&](int, float l) { t += unit(l); });
    return before + cluster_total(block_sum(t, s), s, n_cta, rank, use++, nullptr);
  };
  while (k0 < k1) {
    const uint32_t mid = k0 + (k1 - k0) / 2 + 1;
    if (upto(mid) >= v.need) k0 = mid; else k1 = mid - 1;
  }
  const u64 over = k0 == kmax ? before : upto(k0 + 1);
  const u64 w = unit(key_logit(k0));
  r.cut_key = k0;
  r.has_cut = true;
  r.listed = false;
  nth_tie(s, r, (int)((v.need - over + w - 1) / w), x, id0, n_cta, rank, use);
}

// Sorts a[0 .. n) (n a power of two, at most 2 ST), largest first.
FD_DEV void sort_desc(u64* a, int n) {
  for (int size = 2; size <= n; size *= 2)
    for (int d = size / 2; d > 0; d /= 2) {
      // pairs of a distance up to 32 stay in the 64 elements of a warp
      if (d >= 32) __syncthreads(); else __syncwarp();
      const int p = threadIdx.x;
      if (p < n / 2) {
        const int i = 2 * d * (p / d) + p % d;
        const u64 u = a[i], v = a[i + d];
        const bool down = (i & size) == 0;
        if ((u < v) == down) {
          a[i] = v;
          a[i + d] = u;
        }
      }
      if (d >= 32) __syncthreads();
    }
  __syncthreads();
}

struct Filters {
  int top_k;
  double top_p, min_p;
  bool greedy;
};

// The filters and the draw on s.all[0 .. n), by one CTA: all tokens down to
// some place of the order behind the last kept one, and, unless top-p's goal
// `need` is given (not 0), behind the last one that top-k keeps.
FD_DEV void draw_sorted(Shared& s, const Row& r, const Filters& f, int n, u64 need, double u,
                        int32_t* tok, float* prob) {
  const int tid = threadIdx.x;
  if (n <= DIRECT) {
    // `per` threads a token count its rank and the weight before it
    int per = 1;
    while (2 * per * n <= ST && per < 8) per *= 2;
    const int t = tid / per, part = tid % per;
    const bool have = t < n;
    const u64 o = have ? s.all[t] : 0;
    const double wd = weight(r, have ? order_logit(o) : r.m);
    u64 w = have ? fixed(wd) : 0;
    if (have && part == 0) s.w[t] = w;
    if (tid == 0) s.pick = 0;
    __syncthreads();
    int rank = 0;
    u64 before = 0;
    if (have)
#pragma unroll 4
      for (int i = part; i < n; i += per)
        if (s.all[i] > o) {
          ++rank;
          before += s.w[i];
        }
    for (int d = per / 2; d > 0; d /= 2) {
      rank += __shfl_xor_sync(0xffffffffu, rank, d);
      before += __shfl_xor_sync(0xffffffffu, before, d);
    }
    if (part > 0) w = 0;   // the first of a token's threads stands for it in the sums
    if (f.top_k > 0 && rank >= f.top_k) w = 0;
    if (!(f.top_p >= 1.0)) {
      const u64 total = need ? 0 : block_sum(w, s);
      if (need == 0) need = (u64)ceil(fmax(f.top_p * (double)total, 0.0));
      if (rank > 0 && before >= need) w = 0;
    }
    if (f.min_p > 0.0 && wd < f.min_p) w = 0;
    const u64 all = block_sum(w, s);   // every thread has read s.w
    if (f.greedy) {
      if (have && part == 0 && rank == 0) {
        *tok = order_id(o);
        if (prob) *prob = (float)(wd / ((double)all / W_ONE));
      }
      return;
    }
    // the tokens up to the last kept one once more, by rank: the weight of lower
    // ids (nearly all of them are kept; weights that differ by a rounding may
    // lie on either side of min_p)
    if (have && part == 0) {
      s.list[rank] = o;
      s.w[rank] = w;
      if (w) atomicMax(&s.pick, rank + 1);
    }
    __syncthreads();
    const int kept = s.pick;
    per = 1;
    while (2 * per * kept <= ST && per < 32) per *= 2;
    const int t2 = tid / per, part2 = tid % per;
    const u64 target = min((u64)(fmax(u, 0.0) * (double)all), all - 1);
    const uint32_t low = t2 < kept ? (uint32_t)s.list[t2] : 0;   // ~id
    u64 lower = 0;
    if (t2 < kept)
#pragma unroll 4
      for (int i = part2; i < kept; i += per)
        if ((uint32_t)s.list[i] > low) lower += s.w[i];
    for (int d = per / 2; d > 0; d /= 2) lower += __shfl_xor_sync(0xffffffffu, lower, d);
    if (t2 < kept && part2 == 0 && lower <= target && target < lower + s.w[t2]) {
      *tok = order_id(s.list[t2]);
      if (prob) *prob = (float)(weight(r, order_logit(s.list[t2])) / ((double)all / W_ONE));
    }
    return;
  }
  int size = 64;
  while (size < n) size *= 2;
  for (int i = n + tid; i < size; i += ST) s.all[i] = 0;
  __syncthreads();
  sort_desc(s.all, size);
  if (f.top_k > 0) n = min(n, f.top_k);
  // thread t takes tokens 2t and 2t + 1 of the order
  u64 w[2], total;
  double wd[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * tid + j;
    wd[j] = i < n ? weight(r, order_logit(s.all[i])) : 0.0;
    w[j] = fixed(wd[j]);
  }
  u64 upto = block_scan(w[0] + w[1], s, &total);
  if (!(f.top_p >= 1.0)) {
    // kept while the weight before is below top_p total
    if (need == 0) need = (u64)ceil(fmax(f.top_p * (double)total, 0.0));
    const u64 b1 = upto - w[1], b0 = b1 - w[0];
    if (2 * tid > 0 && b0 >= need) w[0] = 0;
    if (b1 >= need) w[1] = 0;
  }
  if (f.min_p > 0.0) {
    if (wd[0] < f.min_p) w[0] = 0;
    if (wd[1] < f.min_p) w[1] = 0;
  }
  const u64 all = block_sum(w[0] + w[1], s);
  if (f.greedy) {
    if (tid == 0) {
      *tok = order_id(s.all[0]);
      if (prob) *prob = (float)(W_ONE / (double)all);
    }
    return;
  }
  // the kept ones by rising id (those without weight last); the low word finds the weight again
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * tid + j;
    if (i < size) {
      s.list[i] = w[j] ? ((u64)(uint32_t)~(uint32_t)order_id(s.all[i]) << 32) | (uint32_t)i : 0;
      s.w[i] = w[j];
    }
  }
  const int kept = __syncthreads_count(w[0] > 0) + __syncthreads_count(w[1] > 0);
  if (kept < size) {   // kept tokens are a prefix of the order: sort no more than them
    int small = 64;
    while (small < kept) small *= 2;
    size = small;
  }
  sort_desc(s.list, size);
  u64 v[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (2 * tid + j < size && s.list[2 * tid + j]) v[j] = s.w[(uint32_t)s.list[2 * tid + j]];
  upto = block_scan(v[0] + v[1], s, &total);
  const u64 target = min((u64)(fmax(u, 0.0) * (double)all), all - 1);
  const u64 b0 = upto - v[1] - v[0], b1 = upto - v[1];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const u64 lo = j ? b1 : b0;
    if (lo <= target && target < lo + v[j]) {
      const u64 e = s.list[2 * tid + j];
      *tok = (int)~(uint32_t)(e >> 32);
      if (prob)
        *prob = (float)(weight(r, order_logit(s.all[(uint32_t)e])) / ((double)all / W_ONE));
    }
  }
}

template <typename T, bool STAGED>
__global__ void __launch_bounds__(ST, STAGED ? 2 : 3) sample_kernel(const fdllm_sample_args a, int slice, int n_cta) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  static_assert(sizeof(Shared) % 16 == 0, "the slice is read 16 bytes at a time");
  const int tid = threadIdx.x, row = blockIdx.x / n_cta, rank = blockIdx.x % n_cta;
  const int id0 = rank * slice, n = max(0, min(slice, a.vocab - id0));
  const T* src = reinterpret_cast<const T*>(a.logits) + (int64_t)row * a.row_stride + id0;
  int use = 0;
  T* copy = reinterpret_cast<T*>(smem + sizeof(Shared));
  Slice<T, STAGED> x{STAGED ? copy : src, n, a.mask_id - id0, false};

  // ---- the slice (the masked token and the last vector's rest as -inf), and
  // every thread's largest logit
  constexpr int VEC = 16 / sizeof(T);
  const T none = from_f<T>(-INFINITY);
  float top = -INFINITY;
  {
    const bool wide = !STAGED || (reinterpret_cast<uintptr_t>(src) & 15) == 0;
    const int mask = a.mask_id - id0;
    uint4 tops;
#pragma unroll
    for (int j = 0; j < VEC; ++j) reinterpret_cast<T*>(&tops)[j] = none;
#pragma unroll 4
    for (int i = tid; i * VEC < n; i += ST) {
      uint4 u;
      T* e = reinterpret_cast<T*>(&u);
      if (wide && (i + 1) * VEC <= n) {
        u = STAGED ? __ldcs(reinterpret_cast<const uint4*>(src) + i) : reinterpret_cast<const uint4*>(src)[i];
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) e[j] = i * VEC + j < n ? src[i * VEC + j] : none;
      }
      if ((uint32_t)(mask - i * VEC) < (uint32_t)VEC) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (i * VEC + j == mask) e[j] = none;
      }
      if (STAGED) reinterpret_cast<uint4*>(copy)[i] = u;
      tops = max_vec<T>(tops, u);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) top = fmaxf(top, to_f<T>(reinterpret_cast<const T*>(&tops)[j]));
  }
  zero_hist(s, 0);
  zero_hist(s, 1);
  if (tid < 64) s.exp2_64[tid] = EXP2_64[tid];
  if (tid == 0) s.n_list = s.n_hot = 0;
  {
    const float w = warp_max(top);
    if ((tid & 31) == 0) s.red[tid >> 5] = __float_as_uint(w);
  }
  __syncthreads();
  if (tid == 0) {
    float t = -INFINITY;
#pragma unroll
    for (int i = 0; i < SW; ++i) t = fmaxf(t, __uint_as_float((uint32_t)s.red[i]));
    s.top = t;
  }
  cluster_sync();
  Row r{};
  r.m = -INFINITY;
#pragma unroll
  for (int i = 0; i < MAX_CLUSTER; ++i)
    if (i < n_cta) r.m = fmaxf(r.m, __uint_as_float(ld_remote32(&s.top, i)));

  if (r.m == INFINITY) {   // they share all the weight: equal logits, the rest is out
    if (STAGED) {
      for (int i = tid; i < n; i += ST)
        copy[i] = from_f<T>(to_f<T>(copy[i]) == INFINITY ? 0.0f : -INFINITY);
    }
    x.inf = true;
    r.m = 0.0f;
    top = top == INFINITY ? 0.0f : -INFINITY;
    __syncthreads();
  }
  if (r.m == -INFINITY) {
    if (rank == 0 && tid == 0) {
      a.tok[row] = -1;
      if (a.prob) a.prob[row] = 0.0f;
    }
  } else {
    Filters f;
    double temp = a.temperature ? (double)a.temperature[row] : 1.0;
    f.greedy = !(temp > 0.0);
    if (f.greedy) temp = 1.0;
    temp = fmin(fmax(temp, 1e-29), 1e30);
    f.top_k = a.top_k ? max(a.top_k[row], 0) : 0;
    f.top_p = a.top_p ? (double)a.top_p[row] : 1.0;
    f.min_p = a.min_p ? fmin((double)a.min_p[row], 1.0) : 0.0;
    const bool has_p = !(f.top_p >= 1.0);
    const double u = a.u[row];
    r.md = r.m;
    r.y = 64.0 * 1.4426950408889634 / temp;
    r.zs = (float)((double)Z_BINS / temp);
    r.exp2_64 = s.exp2_64;
    auto need_p = [&](u64 t) { return (u64)ceil(fmax(f.top_p * (double)t, 0.0)); };

    // ---- a bound on the kept tokens' z
    float z_end = (float)BINS;
    bool gather = a.vocab <= CAP;
    bool used = false;   // hist[0] holds the threads' maxima
    Level lp{};
    if (f.min_p > 0.0 && !(has_p && f.top_k > 0)) {   // top-p's goal counts what top-k keeps
      z_end = fminf(z_end, (float)(-log(f.min_p)) * (Z_BINS * 1.00001f) + 0.001f);
      gather = true;
    }
    if (a.vocab <= CAP) {
      if (has_p) z_end = (float)BINS;
    } else if (f.top_k > 0 && f.top_k <= ST * n_cta / 2) {
      const float z = z_of(r, top);
      if (z < (float)BINS) atomicAdd(&s.hist[0][0][(int)z], 1u);
      cluster_sync();
      u64 above;
      const u64 need = find_bin<false>(s, 0, n_cta, &above, [&](u64) { return (u64)f.top_k; });
      if (need <= above) {
        z_end = fminf(z_end, (float)(s.bin + 1));
        gather = true;
      }
      used = true;
    } else if (f.top_k == 0 && has_p) {
      lp = level1<true>(s, r, x, n_cta, need_p);
      if (lp.need > 0 && lp.need <= lp.above) {
        // none of the tokens up to the bin's end is lighter than its end
        gather |= (double)lp.upto / W_ONE * exp((lp.bin + 1) / (double)Z_BINS) <= CAP;
        z_end = fminf(z_end, (float)(lp.bin + 1));
      } else {
        gather = false;
      }
    }
    // ---- the tokens within the bound, if they are few
    bool drawn = false;
    if (gather) {
      // only threads whose largest logit is within it have any: their tokens
      // are spread over all threads again
      __syncthreads();
      if (z_of(r, top) < z_end) s.hot[atomicAdd(&s.n_hot, 1)] = (uint16_t)tid;
      __syncthreads();
      const int per = ((n + VEC - 1) / VEC + ST - 1) / ST, items = s.n_hot * per;
      for (int j = tid; j < items; j += ST) {
        const int i = s.hot[j / per] + (j % per) * ST;
        if (i * VEC >= n) continue;
        float l[VEC];
        x.vec(i, l);
#pragma unroll
        for (int q = 0; q < VEC; ++q)
          if (z_of(r, l[q]) < z_end) {
            const int at = atomicAdd(&s.n_list, 1);
            if (at < CAP) s.list[at] = order_of(l[q], id0 + i * VEC + q);
          }
      }
      cluster_sync();
      int n_all = 0;
#pragma unroll
      for (int c = 0; c < MAX_CLUSTER; ++c) {
        const int nc = c < n_cta ? (int)ld_remote32(&s.n_list, c) : 0;
        if (rank == 0 && n_all + nc <= CAP)
          for (int j = tid; j < nc; j += ST) s.all[n_all + j] = ld_remote64(&s.list[j], c);
        n_all += nc;
      }
      drawn = n_all <= CAP;
      cluster_sync();   // every CTA has read the lists and their lengths
      if (drawn) {
        if (rank == 0) draw_sorted(s, r, f, n_all, lp.need, u, a.tok + row, a.prob ? a.prob + row : nullptr);
        return;
      }
    }
    if (!drawn) {
      if (used) {
        if (!gather) cluster_sync();   // every CTA has read the histogram
        zero_hist(s, 0);
      }
      if (f.top_k > 0) {
        __syncthreads();
        const Level v = level1<false>(s, r, x, n_cta, [&](u64) { return (u64)f.top_k; });
        refine<false>(s, r, v, x, id0, n_cta, rank, use);
        if (has_p) lp = level1<true>(s, r, x, n_cta, need_p);
      }
      if (has_p) refine<true>(s, r, lp, x, id0, n_cta, rank, use);

      // ---- the draw: every thread has a run of ids
      auto kept = [&](int i, float l) {
        bool in = z_of(r, l) < z_end;
        if (r.has_cut) {
          const uint32_t k = logit_key(l);
          in = in && (k > r.cut_key || (k == r.cut_key && id0 + i <= r.cut_id));
        }
        return in;
      };
      auto weigh = [&](float l) {
        const double wd = weight(r, l);
        return f.min_p > 0.0 && wd < f.min_p ? (u64)0 : fixed(wd);
      };
      u64 lower, mine;
      int first = 0x7fffffff;
      const u64 sum = run_sum(x, kept, weigh);
      if (f.greedy)
        for (int i = tid; i < n && first == 0x7fffffff; i += ST)
          if (x.at(i) == r.m) first = id0 + i;
      u64 before = block_scan(sum, s, &mine) - sum;
      const u64 all = cluster_total(mine, s, n_cta, rank, use++, &lower);
      if (f.greedy) {
        if (tid == 0) s.pick = 0x7fffffff;
        __syncthreads();
        atomicMin(&s.pick, first);
        cluster_sync();
        if (rank == 0 && tid == 0) {
          int t = 0x7fffffff;
          for (int c = 0; c < n_cta; ++c) t = min(t, (int)ld_remote32(&s.pick, c));
          a.tok[row] = t;
          if (a.prob) a.prob[row] = (float)(W_ONE / (double)all);
        }
      } else {
        // first id whose running sum passes u all: integers, so passes its floor
        const u64 target = min((u64)(fmax(u, 0.0) * (double)all), all - 1);
        before += lower;
        if (tid == 0) s.run1 = -1;
        __syncthreads();
        if (before <= target && target < before + sum) {   // this thread's run: a warp walks it
          s.run0 = tid * run_of(x);
          s.run1 = min(s.run0 + run_of(x), n);
          s.before = before;
        }
        __syncthreads();
        if (s.run1 >= 0 && tid < 32) {
          u64 base = s.before;
          for (int i = s.run0; i < s.run1; i += 32) {
            const float l = i + tid < s.run1 ? x.at(i + tid) : -INFINITY;
            const u64 w = i + tid < s.run1 && kept(i + tid, l) ? weigh(l) : 0;
            u64 upto = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const u64 y = __shfl_up_sync(0xffffffffu, upto, o);
              if (tid >= o) upto += y;
            }
            upto += base;
            if (upto - w <= target && target < upto) {
              a.tok[row] = id0 + i + tid;
              if (a.prob)
                a.prob[row] = (float)(weight(r, l) / ((double)all / W_ONE));
            }
            base = __shfl_sync(0xffffffffu, upto, 31);
          }
        }
      }
    }
  }
  cluster_sync();   // no CTA leaves while another may read its shared memory
}

template <typename T>
cudaError_t launch_sample(const fdllm_sample_args& a, cudaStream_t st) {
  // The smallest cluster whose slices let two CTAs share an SM, and a larger
  // one while the rows leave SMs idle and slices stay worth a CTA.
  int c = 1;
  auto slice_of = [&](int n) { return ((a.vocab + n - 1) / n + 15) / 16 * 16; };
  while (c < MAX_CLUSTER && (slice_of(c) * (int)sizeof(T) > SLICE_BYTES || slice_of(c) > MAX_SLICE)) c *= 2;
  while (c < MAX_CLUSTER && (int64_t)a.rows * c * 2 <= 296 && slice_of(c) >= 4096) c *= 2;
  // Slices that need a cluster are so large that two CTAs fill an SM's shared
  // memory.  Rows for more than two waves of those leave the logits where they
  // are: the copy of the first pass in L2 serves the later ones, and a third CTA
  // fits on the SM.  bf16, 126464 tokens, top_k 200, top_p 0.95, min_p 0.01: 512 rows 165 -> 131 us, 256 rows 94 -> 88, but 75 rows
  // 46 -> 55; wide nuclei (top_p 0.9 alone), which read the slice most often, 5 to
  // 7% slower.  32000 tokens (one CTA a row): 78 -> 98 us, so not there.
  const bool aligned = kv8::aligned16(a.logits) && a.row_stride * (int64_t)sizeof(T) % 16 == 0;
  const bool staged = c == 1 || (int64_t)a.rows * c <= 592 || !aligned;
  const int slice = slice_of(c);
  const int smem = (int)sizeof(Shared) + (staged ? slice * (int)sizeof(T) : 0);
  auto kern = staged ? sample_kernel<T, true> : sample_kernel<T, false>;
  static std::atomic<uint64_t> ready[2];   // devices whose limit is set
  const cudaError_t e = kv8::allow_smem(kern, 227 << 10, ready[staged]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.rows * c));
  cfg.blockDim = dim3(ST);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, slice, c);
}

}  // namespace
}  // namespace fd

extern "C" int fdllm_sample(const fdllm_sample_args* args, void* cuda_stream) {
  using namespace fd;
  const char* call = "fdllm_sample";
  if (!args) return kv8::fail(call, FDLLM_ERR_ARG, "args is NULL");
  const fdllm_sample_args& a = *args;
  const int esz = kv8::elem_bytes(a.dtype);
  if (!esz) return kv8::fail(call, FDLLM_ERR_ARG, "unknown dtype");
  if (a.rows < 0 || a.rows > (1 << 27))
    return kv8::fail(call, FDLLM_ERR_ARG, "rows must be in [0, 2^27]");
  if (a.vocab < 1 || a.vocab > MAX_VOCAB)
    return kv8::fail(call, FDLLM_ERR_ARG, "vocab must be in [1, 2^18]");
  if (a.row_stride < a.vocab) return kv8::fail(call, FDLLM_ERR_ARG, "row_stride must be >= vocab");
  if (a.mask_id < -1 || a.mask_id >= a.vocab)
    return kv8::fail(call, FDLLM_ERR_ARG, "mask_id must be -1 or in [0, vocab)");
  if (a.rows == 0) return FDLLM_OK;
  if (!a.logits || !a.u || !a.tok) return kv8::fail(call, FDLLM_ERR_ARG, "logits, u or tok is NULL");
  if (reinterpret_cast<uintptr_t>(a.logits) % esz || reinterpret_cast<uintptr_t>(a.u) % 8 ||
      !kv8::aligned4({a.temperature, a.top_k, a.top_p, a.min_p, a.tok, a.prob}))
    return kv8::fail(call, FDLLM_ERR_ARG, "arrays must be aligned to their elements");
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = a.dtype == FDLLM_DTYPE_F32    ? launch_sample<float>(a, st)
                        : a.dtype == FDLLM_DTYPE_BF16 ? launch_sample<__nv_bfloat16>(a, st)
                                                      : launch_sample<__half>(a, st);
  if (e != cudaSuccess) return kv8::fail(call, FDLLM_ERR_CUDA, cudaGetErrorString(e));
  return FDLLM_OK;
}
