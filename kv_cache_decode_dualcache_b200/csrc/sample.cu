// fdllm_sample: one token per row of logits with temperature, top-k, top-p
// and min-p, drawn with a given uniform number.
//
// A row is split over the CTAs of a thread-block cluster and read from
// memory once, into their shared memories; everything else happens there and
// over distributed shared memory, in one launch without a workspace.
//
// The kept tokens are a prefix of the row sorted by (falling logit, rising
// id), so they are described by a cut, the last kept token, and nothing is
// sorted.  top-k looks for its cut on counts, top-p on weight sums, both in
// three steps: a histogram of z = (m - l) / T over 256 linear bins of [0, 32)
// (a token beyond weighs under 2^-45 and cannot be drawn), one over 256
// bins of the bin the cut falls into, and the exact order of the few tokens
// of that small bin.  Bins are linear in z and not in the logit's bits
// because that spreads a row's tokens evenly: the shared-memory atomics of a
// warp then rarely meet.  A small bin with more tokens than the list holds
// (thousands of equal logits) is searched by bisection over the logit's bits.
// The draw walks the ids in order.
//
// Weights are held as integers, w = rint(exp(-z) 2^44) with the exponential
// in float64: sums of up to 2^18 weights are exact in 64 bits, so no order
// of additions can change a cut or a token.
//
// Bound: the logits' bytes for many rows; for few rows the chain of cluster
// barriers (one for the maximum, three for each search, one for the draw).
#include <algorithm>

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
constexpr int CAP = 1024;                    // tokens of a small bin whose order is taken directly
constexpr double W_ONE = 17592186044416.0;   // 2^44
constexpr uint32_t KEY_NONE = 0;             // a token that cannot be drawn

typedef unsigned long long u64;

// Order-preserving key of a logit; NaN and -inf give KEY_NONE.
FD_DEV uint32_t logit_key(float l) {
  if (!(l > -INFINITY)) return KEY_NONE;
  const uint32_t u = __float_as_uint(l + 0.0f);   // -0 and +0 are equal logits
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
FD_DEV float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

struct Shared {
  uint32_t hist[2][4][BINS];   // counts, or weights in words of 15, 15 and 15 bits
  u64 red[SW];
  u64 scan[SW];
  u64 part[2];                 // this CTA's share of a cluster sum (by parity of use)
  u64 best;                    // largest (key, lowest id)
  u64 before;
  int bin;
  int n_list;
  uint32_t list_key[CAP];      // this CTA's tokens of the small bin
  int list_id[CAP];
  uint32_t all_key[CAP];       // the cluster's
  int all_id[CAP];
  u64 all_w[CAP];
  uint32_t cut_key;
  int cut_id;
  int cut_ties;
};

template <typename U> FD_DEV U ld_remote(const U* p, uint32_t rank) {
  U v;
  const uint32_t a = cluster_map(smem_u32(p), rank);
  if constexpr (sizeof(U) == 8)
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  else
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// The row's state that every thread of the cluster knows.
struct Row {
  uint32_t kmax;
  float m;
  double temp;
  float zs;         // bins per unit of logit
  double min_w;     // min-p
  // the cut: kept are key > cut_key, and key == cut_key with id <= cut_id
  uint32_t cut_key;
  int cut_id;
  int ties;         // kept tokens with key == cut_key (valid once a cut was set)
  bool has_cut, listed;   // listed: the class of cut_key is in Shared::all_*
};

// exp((l - m) / T) of a live token.
FD_DEV double weight(const Row& r, uint32_t key) {
  if (key == r.kmax) return 1.0;
  if (r.m == INFINITY) return 0.0;
  return exp(((double)key_logit(key) - (double)r.m) / r.temp);
}
FD_DEV u64 fixed(double w) { return __double2ull_rn(w * W_ONE); }

// Place of a token among the bins; >= BINS: too light to be drawn.
FD_DEV float z_of(const Row& r, uint32_t key) {
  if (key == r.kmax) return 0.0f;
  if (r.m == INFINITY) return (float)BINS;
  return fminf(r.m - key_logit(key), 3.402823466e38f) * r.zs;
}

FD_DEV u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
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
// Exclusive prefix sum over the threads.
FD_DEV u64 block_scan(u64 v, Shared& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s.scan[warp] = x;
  __syncthreads();
  u64 before = 0;
  for (int i = 0; i < warp; ++i) before += s.scan[i];
  return before + x - v;
}
// Sum of v over the CTAs (v the same in all threads of a CTA), and over those
// of lower rank.  Alternate `use`: a part is rewritten two uses later.
FD_DEV u64 cluster_total(u64 v, Shared& s, int n_cta, int rank, int use, u64* lower) {
  if (threadIdx.x == 0) s.part[use & 1] = v;
  cluster_sync();
  u64 t = 0, lo = 0;
#pragma unroll
  for (int i = 0; i < MAX_CLUSTER; ++i) {
    const u64 x = i < n_cta ? ld_remote(&s.part[use & 1], i) : 0;
    t += x;
    if (i < rank) lo += x;
  }
  if (lower) *lower = lo;
  return t;
}

// Bins of all CTAs; the bin in which the running sum reaches `need` (set by
// the caller from the sum of all bins) goes to s.bin, what is before it to
// s.before.
template <bool MASS, typename F>
FD_DEV u64 find_bin(Shared& s, int h, int n_cta, F need_of) {
  u64 v = 0;
  if (threadIdx.x < BINS) {
#pragma unroll
    for (int i = 0; i < MAX_CLUSTER; ++i) {
      if (i >= n_cta) continue;
      if (MASS)
        v += (u64)ld_remote(&s.hist[h][0][threadIdx.x], i) +
             ((u64)ld_remote(&s.hist[h][1][threadIdx.x], i) << 15) +
             ((u64)ld_remote(&s.hist[h][2][threadIdx.x], i) << 30);
      else
        v += ld_remote(&s.hist[h][0][threadIdx.x], i);
    }
  }
  const u64 total = block_sum(v, s);
  const u64 need = need_of(total);
  const u64 before = block_scan(v, s);
  if (threadIdx.x < BINS && before < need && need <= before + v) {
    s.bin = threadIdx.x;
    s.before = before;
  }
  __syncthreads();
  return need;
}

FD_DEV void zero_hist(Shared& s, int h) {
  for (int i = threadIdx.x; i < 4 * BINS; i += ST) (&s.hist[h][0][0])[i] = 0;
}

template <bool MASS>
FD_DEV void hist_add(Shared& s, int h, int bin, const Row& r, uint32_t key) {
  if (MASS) {
    const u64 w = fixed(weight(r, key));
    if (w & 0x7fff) atomicAdd(&s.hist[h][0][bin], (uint32_t)w & 0x7fff);
    if (w & 0x3fff8000) atomicAdd(&s.hist[h][1][bin], (uint32_t)(w >> 15) & 0x7fff);
    if (w >> 30) atomicAdd(&s.hist[h][2][bin], (uint32_t)(w >> 30));
  } else {
    atomicAdd(&s.hist[h][0][bin], 1u);
  }
}

// Sets the cut to the `ties`-th token (by id) of the class with key r.cut_key.
template <typename K>
FD_DEV void nth_tie(Shared& s, Row& r, int ties, K key_at, int n, int id0, int n_cta, int rank,
                    int& use) {
  r.ties = ties;
  if (r.listed) {
    for (int j = threadIdx.x; j < s.n_list; j += ST) {
      if (s.all_key[j] != r.cut_key) continue;
      int before = 0;
      for (int i = 0; i < s.n_list; ++i)
        before += s.all_key[i] == r.cut_key && s.all_id[i] < s.all_id[j];
      if (before == ties - 1) s.cut_id = s.all_id[j];
    }
    __syncthreads();
    r.cut_id = s.cut_id;
    return;
  }
  const int run = ((n + ST - 1) / ST) | 1;
  const int i0 = min((int)threadIdx.x * run, n), i1 = min(i0 + run, n);
  u64 mine = 0, lower;
  for (int i = i0; i < i1; ++i) mine += key_at(i) == r.cut_key;
  const u64 cta = block_sum(mine, s);
  cluster_total(cta, s, n_cta, rank, use++, &lower);
  u64 before = lower + block_scan(mine, s);
  if (threadIdx.x == 0) s.cut_id = -1;
  __syncthreads();
  if (before < (u64)ties && (u64)ties <= before + mine)
    for (int i = i0; i < i1; ++i)
      if (key_at(i) == r.cut_key && ++before == (u64)ties) s.cut_id = id0 + i;
  __syncthreads();
  // the CTA that holds it tells the others (ids as id + 1, none = 0)
  r.cut_id = (int)cluster_total((u64)(s.cut_id + 1), s, n_cta, rank, use++, nullptr) - 1;
}

// Moves the cut to where the sum over the kept tokens, in order, reaches
// `need` = need_of(sum of all kept).  MASS: weights, else counts (of tokens
// that are not too light; no cut when need exceeds their number).
template <bool MASS, typename K, typename F>
FD_DEV void search(Shared& s, Row& r, K key_at, int n, int id0, int n_cta, int rank, int& use,
                   F need_of) {
  const int tid = threadIdx.x;
  const u64 w_cut = r.has_cut && MASS ? fixed(weight(r, r.cut_key)) : 0;
  const u64 at_cut = r.has_cut ? (u64)r.ties * w_cut : 0;
  // strictly above the cut; its class is a sum of its own
  for (int i = tid; i < n; i += ST) {
    const uint32_t k = key_at(i);
    if (k == KEY_NONE || (r.has_cut && k <= r.cut_key)) continue;
    const float z = z_of(r, k);
    if (z < (float)BINS) hist_add<MASS>(s, 0, (int)z, r, k);
  }
  cluster_sync();
  u64 above = 0;
  const u64 need = find_bin<MASS>(s, 0, n_cta, [&](u64 t) { above = t; return need_of(t + at_cut); });
  if (need == 0) {   // only the first token
    r.cut_key = r.kmax;
    r.cut_id = (int)~(uint32_t)s.best;
    r.ties = 1;
    r.has_cut = true;
    r.listed = false;
  } else if (need > above) {
    if (r.has_cut) {
      const u64 t = w_cut ? (need - above + w_cut - 1) / w_cut : r.ties;
      if (t < (u64)r.ties) nth_tie(s, r, (int)t, key_at, n, id0, n_cta, rank, use);
    }
  } else {
    const int b1 = s.bin;
    const u64 before1 = s.before;
    const float lo1 = (float)b1;
    __syncthreads();
    for (int i = tid; i < n; i += ST) {
      const uint32_t k = key_at(i);
      if (k == KEY_NONE || (r.has_cut && k <= r.cut_key)) continue;
      const float z = z_of(r, k) - lo1;
      if (z >= 0.0f && z < 1.0f) hist_add<MASS>(s, 1, (int)(z * BINS), r, k);
    }
    cluster_sync();
    zero_hist(s, 0);   // every CTA has read it
    find_bin<MASS>(s, 1, n_cta, [&](u64) { return need - before1; });
    const int b2 = s.bin;
    const u64 before2 = before1 + s.before;
    if (tid == 0) s.n_list = 0;
    __syncthreads();
    auto in_bin = [&](uint32_t k) {
      if (k == KEY_NONE || (r.has_cut && k <= r.cut_key)) return false;
      const float z = z_of(r, k) - lo1;
      return z >= 0.0f && z < 1.0f && (int)(z * BINS) == b2;
    };
    for (int i = tid; i < n; i += ST) {
      const uint32_t k = key_at(i);
      if (in_bin(k)) {
        const int at = atomicAdd(&s.n_list, 1);
        if (at < CAP) {
          s.list_key[at] = k;
          s.list_id[at] = id0 + i;
        }
      }
    }
    cluster_sync();
    zero_hist(s, 1);
    int n_all = 0;
    for (int c = 0; c < n_cta; ++c) {
      const int nc = ld_remote(&s.n_list, c);
      if (n_all + nc <= CAP)
        for (int j = tid; j < nc; j += ST) {
          const uint32_t k = ld_remote(&s.list_key[j], c);
          s.all_key[n_all + j] = k;
          s.all_id[n_all + j] = ld_remote(&s.list_id[j], c);
          s.all_w[n_all + j] = MASS ? fixed(weight(r, k)) : 1;
        }
      n_all += nc;
    }
    if (n_all <= CAP) {
      __syncthreads();
      for (int j = tid; j < n_all; j += ST) {
        const uint32_t kj = s.all_key[j];
        const int idj = s.all_id[j];
        u64 before = before2;
        int ties = 1;
        for (int i = 0; i < n_all; ++i) {
          const bool tie = s.all_key[i] == kj && s.all_id[i] < idj;
          ties += tie;
          if (tie || s.all_key[i] > kj) before += s.all_w[i];
        }
        if (before < need && need <= before + s.all_w[j]) {
          s.cut_key = kj;
          s.cut_id = idj;
          s.cut_ties = ties;
        }
      }
      __syncthreads();
      r.cut_key = s.cut_key;
      r.cut_id = s.cut_id;
      r.ties = s.cut_ties;
      r.has_cut = r.listed = true;
      cluster_sync();   // every CTA has read the lists' lengths
      if (tid == 0) s.n_list = n_all;
      __syncthreads();
    } else {
      // too many: bisect over the keys for the largest one that reaches need
      uint32_t lo = r.has_cut ? r.cut_key + 1 : 1, hi = r.kmax;
      auto upto = [&](uint32_t k0) {   // sum over the bin's tokens with key >= k0
        u64 v = 0;
        for (int i = tid; i < n; i += ST) {
          const uint32_t k = key_at(i);
          if (k >= k0 && in_bin(k)) v += MASS ? fixed(weight(r, k)) : 1;
        }
        return before2 + cluster_total(block_sum(v, s), s, n_cta, rank, use++, nullptr);
      };
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2 + 1;
        if (upto(mid) >= need) lo = mid; else hi = mid - 1;
      }
      const u64 over = lo == r.kmax ? before2 : upto(lo + 1);
      const u64 w = MASS ? fixed(weight(r, lo)) : 1;
      r.cut_key = lo;
      r.has_cut = true;
      r.listed = false;
      nth_tie(s, r, (int)((need - over + w - 1) / w), key_at, n, id0, n_cta, rank, use);
    }
    return;
  }
  // the first histogram is free again once every CTA has read it
  cluster_sync();
  zero_hist(s, 0);
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(ST, 2) sample_kernel(const fdllm_sample_args a, int slice, int n_cta) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  T* x = reinterpret_cast<T*>(smem + sizeof(Shared));
  const int tid = threadIdx.x, row = blockIdx.x / n_cta, rank = blockIdx.x % n_cta;
  const int id0 = rank * slice, n = max(0, min(slice, a.vocab - id0));
  const T* src = reinterpret_cast<const T*>(a.logits) + (int64_t)row * a.row_stride + id0;
  const int mask = a.mask_id - id0;
  auto key_at = [&](int i) { return i == mask ? KEY_NONE : logit_key(to_f<T>(x[i])); };
  int use = 0;

  // ---- the slice, and the row's largest logit
  constexpr int VEC = 16 / sizeof(T);
  u64 best = 0;
  auto see = [&](int i, T v) {
    x[i] = v;
    const uint32_t k = i == mask ? KEY_NONE : logit_key(to_f<T>(v));
    const u64 c = ((u64)k << 32) | (uint32_t)~(uint32_t)(id0 + i);   // equal keys: the lowest id
    if (k != KEY_NONE && c > best) best = c;
  };
  if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
    const int nv = n / VEC;
#pragma unroll 4
    for (int i = tid; i < nv; i += ST) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src) + i);
      const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) see(i * VEC + j, e[j]);
    }
    for (int i = nv * VEC + tid; i < n; i += ST) see(i, src[i]);
  } else {
    for (int i = tid; i < n; i += ST) see(i, src[i]);
  }
  zero_hist(s, 0);
  zero_hist(s, 1);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if ((tid & 31) == 0) s.red[tid >> 5] = best;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < SW; ++i) best = max(best, s.red[i]);
  if (tid == 0) s.part[1] = best;
  cluster_sync();
  for (int i = 0; i < n_cta; ++i) best = max(best, ld_remote(&s.part[1], i));
  if (tid == 0) s.best = best;
  __syncthreads();

  Row r{};
  r.kmax = (uint32_t)(best >> 32);
  bool done = false;
  if (r.kmax == KEY_NONE) {
    if (rank == 0 && tid == 0) {
      a.tok[row] = -1;
      if (a.prob) a.prob[row] = 0.0f;
    }
    done = true;
  }
  if (!done) {
    r.m = key_logit(r.kmax);
    r.temp = a.temperature ? (double)a.temperature[row] : 1.0;
    const bool greedy = !(r.temp > 0.0);
    if (greedy) r.temp = 1.0;
    r.zs = (float)fmin((double)Z_BINS / r.temp, 1e30);
    const int top_k = a.top_k ? a.top_k[row] : 0;
    const double top_p = a.top_p ? (double)a.top_p[row] : 1.0;
    const double min_p = a.min_p ? fmin((double)a.min_p[row], 1.0) : 0.0;
    if (top_k > 0)
      search<false>(s, r, key_at, n, id0, n_cta, rank, use, [&](u64) { return (u64)top_k; });
    if (!(top_p >= 1.0))
      search<true>(s, r, key_at, n, id0, n_cta, rank, use,
                   [&](u64 t) { return (u64)ceil(fmax(top_p * (double)t, 0.0)); });

    // ---- the draw: every thread takes a run of ids (odd: no bank conflicts)
    const int run = ((n + ST - 1) / ST) | 1;
    const int i0 = min(tid * run, n), i1 = min(i0 + run, n);
    auto kept_w = [&](int i) {
      const uint32_t k = key_at(i);
      if (k == KEY_NONE || (r.has_cut && (k < r.cut_key || (k == r.cut_key && id0 + i > r.cut_id))))
        return (u64)0;
      if (!(z_of(r, k) < (float)BINS)) return (u64)0;
      const double w = weight(r, k);
      return min_p > 0.0 && w < min_p ? (u64)0 : fixed(w);
    };
    u64 sum = 0, lower;
    for (int i = i0; i < i1; ++i) sum += kept_w(i);
    const u64 mine = block_sum(sum, s);
    const u64 all = cluster_total(mine, s, n_cta, rank, use++, &lower);
    if (greedy) {
      if (rank == 0 && tid == 0) {
        a.tok[row] = (int)~(uint32_t)s.best;
        if (a.prob) a.prob[row] = (float)(W_ONE / (double)all);
      }
    } else {
      // first id whose running sum passes u all: integers, so passes its floor
      const u64 target = min((u64)(fmax(a.u[row], 0.0) * (double)all), all - 1);
      if (lower <= target && target < lower + mine) {
        u64 before = lower + block_scan(sum, s);
        if (before <= target && target < before + sum) {
          int i = i0;
          for (;; ++i) {
            before += kept_w(i);
            if (before > target) break;
          }
          a.tok[row] = id0 + i;
          if (a.prob) a.prob[row] = (float)(weight(r, key_at(i)) / ((double)all / W_ONE));
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
  const int slice = slice_of(c);
  const int smem = (int)sizeof(Shared) + slice * (int)sizeof(T);
  auto kern = sample_kernel<T>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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
