// fdllm_kv8_append: rotation, 8-bit rounding and storing of new keys and
// values into the paged cache, one launch.
//
// A warp takes one block of 16 positions of a head: K (rotated, rounded,
// stored), V (rounded, stored) or q (rotated, written back in its type).  A
// lane holds 8 dims and their 8 rotation partners (d + head_dim / 2) of
// head_dim / 32 tokens in registers, so a block is read once, its maximum is
// one warp reduction and its codes leave in 8-byte stores.  The (cos, sin) rows
// lie in shared memory for all heads of the CTA, and a warp with several heads
// loads the next one's rows while it works on one.
//
// Bound: the bytes of the rows (read), the codes and the optional outputs
// (written).  A prompt of 8191 tokens with 32 K/V heads and 32 heads of q of 128
// dims (474 MB, bf16): 85 us, 5.6 TB/s; 101 us with a head a warp (all of a warp's
// loads then wait at once), 141 us with the (cos, sin) rows read through L1 by
// every warp.  With few blocks a warp has one head: 16 blocks of 32 tokens take
// 8.7 us so and 11.4 us with 4 heads a warp, for their loads then wait in turn.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv8.h"

namespace fd {
namespace {

constexpr int BLK = FDLLM_KV8_BLOCK;
constexpr int APP_WARPS = 8;
constexpr float TINY_SCALE = 7.888609052210118e-31f;  // 2^-100

struct AppendP {
  fdllm_kv8 c;
  fdllm_kv8_append_args a;
  int per_warp;   // heads of a warp
};

// 8 consecutive elements as they lie in memory (16-byte aligned; plain loads,
// q_out may be q itself), and as float.
template <typename T> struct Raw8 {
  uint4 u[sizeof(T) / 2];
};
template <typename T> FD_DEV Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
FD_DEV void floats8(const Raw8<float>& r, float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(r.u[i].x);
    x[4 * i + 1] = __uint_as_float(r.u[i].y);
    x[4 * i + 2] = __uint_as_float(r.u[i].z);
    x[4 * i + 3] = __uint_as_float(r.u[i].w);
  }
}
FD_DEV void floats8(const Raw8<__half>& r, float* x) {
  const __half2* h = reinterpret_cast<const __half2*>(&r.u[0]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
FD_DEV void floats8(const Raw8<__nv_bfloat16>& r, float* x) {
  const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

template <typename T> FD_DEV void store8(T* p, const float* x) {
  T v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = from_f<T>(x[i]);
#pragma unroll
  for (int i = 0; i < (int)sizeof(v) / 16; ++i)
    reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(v)[i];
}

FD_DEV float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.0f;   // inf and NaN do not count
}

// clamp(rint(y), -127, 127), NaN -> 0 (the conversion saturates and maps NaN
// to 0).
FD_DEV int to_code(float y) { return max(-127, min(127, __float2int_rn(y))); }

// max(a, |b|), NaN if either is.
FD_DEV float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(fabsf(b)));
  return y;
}

// Codes of 8 finite values that the scale covers (|x inv| < 127.5): added to
// 1.5 2^23, a value is rounded to an integer (halves to even), whose low byte
// is the code.  deq: the codes as floats.
FD_DEV uint2 codes8(const float* x, float inv, float* deq) {
  constexpr float MAGIC = 12582912.0f;
  uint32_t m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = __fadd_rn(__fmul_rn(x[i], inv), MAGIC);
    deq[i] = __fsub_rn(y, MAGIC);
    m[i] = __float_as_uint(y);
  }
  return make_uint2(__byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(m[4], m[5], 0x0040), __byte_perm(m[6], m[7], 0x0040), 0x5410));
}

FD_DEV uint2 pack8(const int* q) {
  uint2 r;
  r.x = (q[0] & 255) | ((q[1] & 255) << 8) | ((q[2] & 255) << 16) | ((uint32_t)q[3] << 24);
  r.y = (q[4] & 255) | ((q[5] & 255) << 8) | ((q[6] & 255) << 16) | ((uint32_t)q[7] << 24);
  return r;
}

FD_DEV uint2 rescale8(uint2 w, float ratio) {
  int q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = i < 4 ? w.x : w.y;
    const int code = (int)(int8_t)(u >> (8 * (i & 3)));
    q[i] = __float2int_rn(__fmul_rn((float)code, ratio));
  }
  return pack8(q);
}

template <typename T, int HD>
__global__ void __launch_bounds__(APP_WARPS * 32, 2) kv8_append_kernel(const AppendP P) {
  constexpr int LPT = HD / 16;      // lanes per token
  constexpr int TPP = 32 / LPT;     // tokens per pass
  constexpr int NP = BLK / TPP;     // passes over the block
  constexpr int H2 = HD / 2;
  constexpr bool AHEAD = sizeof(T) * HD <= 256;   // a head ahead, where registers allow it
  const fdllm_kv8& c = P.c;
  const fdllm_kv8_append_args& a = P.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seq = blockIdx.z;
  const int Hkv = c.n_kv_heads, heads = 2 * Hkv + (a.q ? a.n_heads : 0);
  // the CTA's heads, of K, V, q in a row; a warp takes every APP_WARPS-th
  const int h_lo = blockIdx.x * APP_WARPS * P.per_warp, h_hi = min(h_lo + APP_WARPS * P.per_warp, heads);
  __shared__ float4 rope_s[BLK][H2 / 2];   // the block's (cos, sin) rows, a lane's four chunks apart

  const int r_lo = min(max(a.starts[seq], 0), a.n_tokens);
  const int r_hi = min(max(a.starts[seq + 1], r_lo), a.n_tokens);
  const int len_in = a.lens[seq];
  const int w0 = a.pos ? a.pos[seq] : len_in;
  int n = r_hi - r_lo;
  int bad = kv8::starts_ok(a.starts, seq, a.n_tokens) ? 0 : FDLLM_KV8_BAD_RANGE;
  int limit = c.max_pages * FDLLM_KV8_PAGE;
  const int len = min(max(len_in, 0), limit);
  if (len != len_in) bad |= FDLLM_KV8_BAD_RANGE;
  if (a.rope) limit = min(limit, a.rope_len);
  if (n > 0 && (w0 < 0 || w0 > limit - n)) {
    bad |= FDLLM_KV8_BAD_RANGE;
    n = w0 < 0 ? 0 : max(limit - w0, 0);
  }
  const int w1 = w0 + n;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    if (bad && a.status) atomicOr(a.status, bad);
    if (a.lens_out) a.lens_out[seq] = n > 0 ? max(len, w1) : len;
  }
  if (n == 0) return;

  const int sub = lane % LPT, tk = lane / LPT;
  const int d0 = 8 * sub;

  const bool any_rope = a.rope != nullptr && (h_lo < Hkv || h_hi > 2 * Hkv);
  const int b_lo = w0 / BLK, b_hi = (w1 - 1) / BLK;
  for (int b = b_lo + blockIdx.y; b <= b_hi; b += gridDim.y) {
    const int base = b * BLK;
    Raw8<T> raw[NP][2];   // dims d0 .. d0 + 7, then their partners
    auto load = [&](int head) {
      const bool is_q = head >= 2 * Hkv, is_v = !is_q && head >= Hkv;
      const T* src = reinterpret_cast<const T*>(is_q ? a.q : is_v ? a.v : a.k);
      const int64_t* st = is_q ? a.q_strides : is_v ? a.v_strides : a.k_strides;
      src += (int64_t)(is_q ? head - 2 * Hkv : is_v ? head - Hkv : head) * st[1] + d0;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int at = base + p * TPP + tk;
        if (at >= w0 && at < w1 && head < h_hi) {
          const T* row = src + (int64_t)(r_lo + at - w0) * st[0];
          raw[p][0] = load8<T>(row);
          raw[p][1] = load8<T>(row + H2);
        } else {
          raw[p][0] = raw[p][1] = Raw8<T>{};
        }
      }
    };
    if (AHEAD) load(h_lo + warp);
    const int page = h_lo >= 2 * Hkv ? 0 : c.page_table[(int64_t)seq * c.table_stride + base / FDLLM_KV8_PAGE];
    if (any_rope) {
      const float4* src = reinterpret_cast<const float4*>(a.rope + (int64_t)base * HD);
      __syncthreads();   // the rows of the block before have been used
      for (int i = threadIdx.x; i < BLK * H2 / 2; i += APP_WARPS * 32) {
        const int t = i / (H2 / 2), ch = i % (H2 / 2);
        if (base + t >= w0 && base + t < w1) rope_s[t][ch % 4 * LPT + ch / 4] = __ldg(src + i);
      }
      __syncthreads();
    }
#pragma unroll 1
    for (int head = h_lo + warp; head < h_hi; head += APP_WARPS) {
      const bool is_q = head >= 2 * Hkv, is_v = !is_q && head >= Hkv;
      const int g = is_q ? head - 2 * Hkv : is_v ? head - Hkv : head;
      T* out = reinterpret_cast<T*>(is_q ? a.q_out : is_v ? a.v_out : a.k_out);
      const int out_heads = is_q ? a.n_heads : Hkv;
      float x[NP][16];
      if (!AHEAD) load(head);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        floats8(raw[p][0], x[p]);
        floats8(raw[p][1], x[p] + 8);
      }
      if (AHEAD) load(head + APP_WARPS);   // on its way while this head is worked on
      if (a.rope != nullptr && !is_v) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int at = base + p * TPP + tk;
          if (at >= w0 && at < w1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 w = rope_s[p * TPP + tk][i * LPT + sub];
              const float cw[2] = {w.x, w.z}, sw[2] = {w.y, w.w};
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float lo = x[p][2 * i + j], hi = x[p][8 + 2 * i + j];
                x[p][2 * i + j] = __fsub_rn(__fmul_rn(lo, cw[j]), __fmul_rn(hi, sw[j]));
                x[p][8 + 2 * i + j] = __fadd_rn(__fmul_rn(hi, cw[j]), __fmul_rn(lo, sw[j]));
              }
            }
          }
        }
      }
      if (is_q) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int at = base + p * TPP + tk;
          if (at >= w0 && at < w1) {
            T* o = out + ((int64_t)(r_lo + at - w0) * out_heads + g) * HD + d0;
            store8<T>(o, x[p]);
            store8<T>(o + H2, x[p] + 8);
          }
        }
        continue;
      }
      if (page < 0 || page >= c.n_pages) {
        if (lane == 0 && a.status) atomicOr(a.status, FDLLM_KV8_BAD_PAGE);
        continue;
      }
      const int sb = base % FDLLM_KV8_PAGE / BLK;
      float* sp = (is_v ? c.v_scale : c.k_scale) + (int64_t)page * c.scale_stride + g * 4 + sb;
      int8_t* codes = (is_v ? c.v : c.k) + (int64_t)page * c.page_stride +
                      ((int64_t)g * FDLLM_KV8_PAGE + sb * BLK) * HD + d0;
      // old tokens of the block that stay: before w0, or behind the new rows
      const bool any_kept = base < min(len, w0) || w1 < min(len, base + BLK);
      const float old = any_kept ? *sp : 0.0f;
      float top = 0.0f;
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max_nan(top, x[p][i]);
      const bool finite = __all_sync(0xffffffffu, top <= 3.402823466e38f);
      if (!finite) {
        top = 0.0f;
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int i = 0; i < 16; ++i) top = fmaxf(top, finite_abs(x[p][i]));
      }
      top = warp_max(top);
      float scale = fmaxf(old, __fmul_rn(top, 1.0f / 127.0f));
      if (!(scale >= TINY_SCALE)) scale = 0.0f;
      const float inv = scale > 0.0f ? __fdiv_rn(1.0f, scale) : 0.0f;
      const bool regrid = any_kept && scale != old;
      const float ratio = regrid && scale > 0.0f ? __fdiv_rn(old, scale) : 0.0f;
      __syncwarp();   // every lane has read the old scale
      if (lane == 0) *sp = scale;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int slot = p * TPP + tk, at = base + slot;
        uint2* lo = reinterpret_cast<uint2*>(codes + slot * HD);
        uint2* hi = reinterpret_cast<uint2*>(codes + slot * HD + H2);
        if (at >= w0 && at < w1) {
          float y[16];
          if (!finite) {   // infinities end at +-127, NaN at 0
#pragma unroll
            for (int i = 0; i < 16; ++i) x[p][i] = (float)to_code(__fmul_rn(x[p][i], inv));
          }
          const float by = finite ? inv : 1.0f;
          *lo = codes8(x[p], by, y);
          *hi = codes8(x[p] + 8, by, y + 8);
          if (out) {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(y[i], scale);
            T* o = out + ((int64_t)(r_lo + at - w0) * out_heads + g) * HD + d0;
            store8<T>(o, y);
            store8<T>(o + H2, y + 8);
          }
        } else if (regrid && at < len) {
          *lo = rescale8(*lo, ratio);
          *hi = rescale8(*hi, ratio);
        }
      }
    }
  }
}

template <typename T>
cudaError_t launch_append_t(const AppendP& P, dim3 grid, cudaStream_t st) {
  const dim3 block(APP_WARPS * 32);
  switch (P.c.head_dim) {
    case 128: return launch_k(false, kv8_append_kernel<T, 128>, grid, block, 0, st, P);
    case 64: return launch_k(false, kv8_append_kernel<T, 64>, grid, block, 0, st, P);
    default: return launch_k(false, kv8_append_kernel<T, 32>, grid, block, 0, st, P);
  }
}

}  // namespace
}  // namespace fd

extern "C" int fdllm_kv8_append(const fdllm_kv8* cache, const fdllm_kv8_append_args* args,
                                void* cuda_stream) {
  using namespace fd;
  const char* call = "fdllm_kv8_append";
  AppendP P{};
  if (const char* why = kv8::check_cache(cache, &P.c)) return kv8::fail(call, FDLLM_ERR_ARG, why);
  if (!args) return kv8::fail(call, FDLLM_ERR_ARG, "args is NULL");
  P.a = *args;
  const fdllm_kv8_append_args& a = P.a;
  const int esz = kv8::elem_bytes(a.dtype);
  if (!esz) return kv8::fail(call, FDLLM_ERR_ARG, "unknown dtype");
  if (a.n_tokens < 0 || a.max_new < 0 || a.reserved)
    return kv8::fail(call, FDLLM_ERR_ARG, "n_tokens and max_new must be >= 0, reserved 0");
  if (!a.starts || !a.lens) return kv8::fail(call, FDLLM_ERR_ARG, "starts or lens is NULL");
  if (!kv8::aligned4({a.starts, a.lens, a.pos, a.lens_out, a.status}))
    return kv8::fail(call, FDLLM_ERR_ARG, "int32 arrays must be 4-byte aligned");
  const int64_t seqs = P.c.n_seqs;
  if (a.lens_out && (kv8::overlap(a.lens_out, seqs, a.starts, seqs + 1) ||
                     kv8::overlap(a.lens_out, seqs, a.lens, seqs) || kv8::overlap(a.lens_out, seqs, a.pos, seqs)))
    return kv8::fail(call, FDLLM_ERR_ARG, "lens_out must not overlap starts, lens or pos");
  if (a.rope && (a.rope_len < 1 || !kv8::aligned16(a.rope)))
    return kv8::fail(call, FDLLM_ERR_ARG, "rope needs rope_len >= 1 and 16-byte alignment");
  if (a.n_tokens > 0) {
    if (!a.k || !a.v) return kv8::fail(call, FDLLM_ERR_ARG, "k or v is NULL");
    if (!kv8::rows_ok(a.k, a.k_strides, esz) || !kv8::rows_ok(a.v, a.v_strides, esz) ||
        (a.q && !kv8::rows_ok(a.q, a.q_strides, esz)))
      return kv8::fail(call, FDLLM_ERR_ARG, "rows and heads of k, v and q must be 16-byte aligned");
  }
  if ((a.q != nullptr) != (a.q_out != nullptr))
    return kv8::fail(call, FDLLM_ERR_ARG, "q and q_out go together");
  if (a.q && (a.n_heads < 1 || a.n_heads > 65535))
    return kv8::fail(call, FDLLM_ERR_ARG, "n_heads must be in [1, 65535]");
  if (!kv8::aligned16(a.k_out) || !kv8::aligned16(a.v_out) || !kv8::aligned16(a.q_out))
    return kv8::fail(call, FDLLM_ERR_ARG, "outputs must be 16-byte aligned");

  // Blocks of 16 that a run of max_new rows can touch; the kernel strides
  // over whatever a sequence has beyond that.
  const int rows = a.max_new > 0 ? std::min(a.max_new, a.n_tokens) : a.n_tokens;
  const int64_t blocks = std::max<int64_t>(1, ((int64_t)rows + 2 * BLK - 2) / BLK);
  const int heads = 2 * P.c.n_kv_heads + (a.q ? a.n_heads : 0);
  // Many CTAs' worth of heads: 4 to a warp, each loaded while the one before is
  // worked on.  Few: one each, all in flight at once.
  int sms = 0;
  if (cudaError_t e = kv8::sm_count(&sms)) return kv8::fail(call, FDLLM_ERR_CUDA, cudaGetErrorString(e));
  const int64_t groups = (heads + APP_WARPS - 1) / APP_WARPS;
  P.per_warp = groups * blocks * P.c.n_seqs > 8 * (int64_t)sms ? 4 : 1;
  const dim3 grid((unsigned)((groups + P.per_warp - 1) / P.per_warp),
                  (unsigned)std::min<int64_t>(blocks, 65535), P.c.n_seqs);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = a.dtype == FDLLM_DTYPE_F32    ? launch_append_t<float>(P, grid, st)
                        : a.dtype == FDLLM_DTYPE_BF16 ? launch_append_t<__nv_bfloat16>(P, grid, st)
                                                      : launch_append_t<__half>(P, grid, st);
  if (e != cudaSuccess) return kv8::fail(call, FDLLM_ERR_CUDA, cudaGetErrorString(e));
  return FDLLM_OK;
}
