// fdllm_sample: one token per row of logits with temperature, top-k, top-p
// and min-p, drawn with a given uniform number.
//
// The kept tokens are a prefix of the row sorted by (falling logit, rising
// id), so they are described by a cut: every token above a logit and the
// first `ties` tokens (by id) at it.  Nothing is sorted: top-k and top-p
// look for their cut by its logit's bits, on counts and on weight sums, and
// the draw walks the ids in order.
//
// Weights are held as integers, w = rint(exp((l - m) / T) 2^44) with the
// exponential in float64: sums of up to 2^18 weights are exact in 64 bits,
// so no order of additions can change a cut or a token.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv8.h"

namespace fd {
namespace {

constexpr int SAMPLE_THREADS = 1024;
constexpr int SAMPLE_WARPS = SAMPLE_THREADS / 32;
constexpr int MAX_VOCAB = 1 << 18;
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

// exp((l - m) / T) of a live token.
FD_DEV double weight(uint32_t key, uint32_t key_max, double m, double temp) {
  if (key == key_max) return 1.0;
  if (m == (double)INFINITY) return 0.0;
  return exp(((double)key_logit(key) - m) / temp);
}
FD_DEV u64 fixed(double w) { return __double2ull_rn(w * W_ONE); }

FD_DEV u64 block_sum(u64 v, u64* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 s = 0;
  for (int i = 0; i < SAMPLE_WARPS; ++i) s += red[i];
  return s;
}

// Exclusive prefix sum over the threads.
FD_DEV u64 block_scan(u64 v, u64* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) red[warp] = x;
  __syncthreads();
  u64 before = 0;
  for (int i = 0; i < warp; ++i) before += red[i];
  return before + x - v;
}

template <typename T>
__global__ void __launch_bounds__(SAMPLE_THREADS) sample_kernel(const fdllm_sample_args a) {
  __shared__ u64 red[SAMPLE_WARPS];
  __shared__ int s_last, s_pick;
  const int row = blockIdx.x, tid = threadIdx.x, V = a.vocab;
  const T* x = reinterpret_cast<const T*>(a.logits) + (int64_t)row * a.row_stride;
  auto key_at = [&](int i) { return i == a.mask_id ? KEY_NONE : logit_key(to_f<T>(x[i])); };
  if (tid == 0) {
    s_last = -1;
    s_pick = 0x7fffffff;
  }

  uint32_t kmax = KEY_NONE;
  for (int i = tid; i < V; i += SAMPLE_THREADS) kmax = max(kmax, key_at(i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) kmax = max(kmax, __shfl_xor_sync(0xffffffffu, kmax, o));
  if ((tid & 31) == 0) red[tid >> 5] = kmax;
  __syncthreads();
  for (int i = 0; i < SAMPLE_WARPS; ++i) kmax = max(kmax, (uint32_t)red[i]);
  if (kmax == KEY_NONE) {
    if (tid == 0) {
      a.tok[row] = -1;
      if (a.prob) a.prob[row] = 0.0f;
    }
    return;
  }
  const double m = (double)key_logit(kmax);
  double temp = a.temperature ? (double)a.temperature[row] : 1.0;
  const bool greedy = !(temp > 0.0);
  if (greedy) temp = 1.0;
  const int top_k = a.top_k ? a.top_k[row] : 0;
  const double top_p = a.top_p ? (double)a.top_p[row] : 1.0;
  const double min_p = a.min_p ? fmin((double)a.min_p[row], 1.0) : 0.0;

  auto wt = [&](uint32_t k) { return fixed(weight(k, kmax, m, temp)); };
  // sum over tokens with key >= lo of f(key)
  auto total = [&](uint32_t lo, auto f) {
    u64 s = 0;
    for (int i = tid; i < V; i += SAMPLE_THREADS) {
      const uint32_t k = key_at(i);
      if (k != KEY_NONE && k >= lo) s += f(k);
    }
    return block_sum(s, red);
  };
  auto one = [](uint32_t) { return (u64)1; };

  // the cut: tokens with key > cut, and the first `ties` with key == cut
  uint32_t cut = 1;
  u64 ties = MAX_VOCAB;
  if (top_k > 0 && total(1, one) > (u64)top_k) {
    uint32_t lo = 1, hi = kmax;   // largest cut with at least top_k tokens at or above it
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2 + 1;
      if (total(mid, one) >= (u64)top_k) lo = mid; else hi = mid - 1;
    }
    cut = lo;
    ties = top_k - (cut == 0xffffffffu ? 0 : total(cut + 1, one));
  }
  if (!(top_p >= 1.0)) {
    auto mass = [&](uint32_t lo) {   // kept so far, key >= lo
      u64 s = total(max(lo, cut + 1), wt);
      if (lo <= cut && ties < (u64)MAX_VOCAB) s += ties * wt(cut);
      else if (lo <= cut) s += total(cut, [&](uint32_t k) { return k == cut ? wt(k) : (u64)0; });
      return s;
    };
    const u64 need = (u64)ceil(fmax(top_p * (double)mass(cut), 0.0));
    if (need == 0) {
      cut = kmax;
      ties = 1;
    } else {
      uint32_t lo = cut, hi = kmax;
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2 + 1;
        if (mass(mid) >= need) lo = mid; else hi = mid - 1;
      }
      const u64 above = lo == kmax ? 0 : mass(lo + 1), w = wt(lo);
      u64 t = (need - above + w - 1) / w;
      if (lo == cut) t = min(t, ties);
      cut = lo;
      ties = t;
    }
  }

  // the draw: every thread takes a run of ids
  const int run = (V + SAMPLE_THREADS - 1) / SAMPLE_THREADS;
  const int i0 = min(tid * run, V), i1 = min(i0 + run, V);
  u64 mine = 0;
  for (int i = i0; i < i1; ++i) mine += key_at(i) == cut;
  const u64 tie0 = block_scan(mine, red);
  auto kept_w = [&](int i, u64& tie) {
    const uint32_t k = key_at(i);
    if (k == KEY_NONE || k < cut) return (u64)0;
    if (k == cut && tie++ >= ties) return (u64)0;
    const double w = weight(k, kmax, m, temp);
    return min_p > 0.0 && w < min_p ? (u64)0 : fixed(w);
  };
  u64 sum = 0, tie = tie0;
  int last = -1, first_max = 0x7fffffff;
  for (int i = i0; i < i1; ++i) {
    const u64 w = kept_w(i, tie);
    if (w) last = i;
    if (key_at(i) == kmax) first_max = min(first_max, i);
    sum += w;
  }
  atomicMax(&s_last, last);
  if (greedy) atomicMin(&s_pick, first_max);
  const u64 all = block_sum(sum, red);
  u64 before = block_scan(sum, red);
  if (!greedy) {
    const double target = fmax(a.u[row], 0.0) * (double)all;
    if ((double)before <= target && (double)(before + sum) > target) {
      tie = tie0;
      for (int i = i0; i < i1; ++i) {
        before += kept_w(i, tie);
        if ((double)before > target) {
          s_pick = i;
          break;
        }
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    const int t = min(s_pick, s_last);
    a.tok[row] = t;
    if (a.prob) a.prob[row] = (float)(weight(key_at(t), kmax, m, temp) / ((double)all / W_ONE));
  }
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
  if (a.rows < 0) return kv8::fail(call, FDLLM_ERR_ARG, "rows must be >= 0");
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
  const dim3 grid(a.rows), block(SAMPLE_THREADS);
  const cudaError_t e =
      a.dtype == FDLLM_DTYPE_F32 ? launch_k(false, sample_kernel<float>, grid, block, 0, st, a)
      : a.dtype == FDLLM_DTYPE_BF16
          ? launch_k(false, sample_kernel<__nv_bfloat16>, grid, block, 0, st, a)
          : launch_k(false, sample_kernel<__half>, grid, block, 0, st, a);
  if (e != cudaSuccess) return kv8::fail(call, FDLLM_ERR_CUDA, cudaGetErrorString(e));
  return FDLLM_OK;
}
