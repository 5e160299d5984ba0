// fdllm_kv8_attention: attention of a few query rows per sequence over the
// 8-bit paged K/V cache.
//
// A query row is a (token, head-in-group) pair, so that the query heads of a
// K/V head share every cached byte.  CTA = (tile of 16 RT rows, K/V head,
// sequence, key split); its 8 warps take the split's keys in tiles of 32,
// every warp with a ring of cp.async stages, softmax statistics and an
// output accumulator of its own, so the loop has no barrier beyond the
// warp's; the warps' results meet in shared memory at the end, the splits'
// in a second kernel.
//
// Codes are exact in fp16 and become matrix operands on the way from shared
// memory to registers (sign bit flipped, byte put under the exponent of
// 1024, 1152 subtracted).  The products run on mma.sync m16n8k16: with few
// rows the kernel streams the cache, and operands that go straight to
// registers spare the round trip through shared memory that a converted tile
// would take.  Both contractions are free in the order of their index, and
// so every lane reads 16 consecutive bytes: in Q K^T the dims are permuted
// alike in q and k, in P V the output columns.
//
//   S = Q K^T, q scaled per row by a power of two to |q| < 2^9;
//   t = S f + log2(vs), f = scale log2(e) ks 2^-e   (ks, vs: the block's scales)
//   M = running max of t, w = 2^(t - M + 8) rounded to fp16
//   O = sum_j w_j V_j (V: codes), l = sum_j w_j / vs_j
// The value scale is part of the softmax weight, so that w spans the
// contributions to the output and not the probabilities: its largest is
// near 2^8 and 2^-22 of it is still a normal fp16 number.  float32 q and w are
// carried as two fp16 terms, and vs enters as its exponent (in t) and its
// mantissa (a factor of w).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "kv8.h"

namespace fd {
namespace {

constexpr int AT_WARPS = 8;
constexpr int TILE = 32;      // keys of a warp's tile
constexpr int STAGES = 3;
constexpr int PAGE = FDLLM_KV8_PAGE;
constexpr float W_EXP = 8.0f;        // largest weights are about 2^W_EXP
constexpr float M_SLACK = 7.0f;      // the reference moves when the max passes it by this
constexpr float LOG2E = 1.4426950408889634f;
constexpr float VS_MIN = 7.888609052210118e-31f;  // 2^-100: an all-zero block still counts in l

struct AttnP {
  fdllm_kv8 c;
  fdllm_kv8_attention_args a;
  int n_split;       // most splits of a sequence
  int keys;          // keys of a split, a multiple of 64
  float* part_o;     // [split][n_tokens][n_heads][head_dim]
  float2* part_ml;   // [split][n_tokens][n_heads] (reference max, weight sum)
};

// Split length of a sequence of L keys: P.keys unless that makes more splits
// than there is room for.
FD_DEV int split_keys(const AttnP& P, int L) {
  const int least = ((L + P.n_split - 1) / P.n_split + PAGE - 1) / PAGE * PAGE;
  return max(P.keys, least);
}

FD_DEV void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
FD_DEV void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
FD_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> FD_DEV void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

FD_DEV void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two of the four offset-binary bytes of x (selector) as exact fp16 codes.
template <uint32_t SEL> FD_DEV uint32_t codes_h2(uint32_t x) {
  const uint32_t u = __byte_perm(x, 0x64646464u, SEL);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __float2half2_rn(1152.0f));
  return *reinterpret_cast<const uint32_t*>(&h);
}
FD_DEV uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
FD_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int B> FD_DEV void lds(uint32_t addr, uint32_t* w) {
  if constexpr (B == 16)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
  else if constexpr (B == 8)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
}

template <int HD, int RT, bool TWO>
struct Lay {
  static constexpr int R = 16 * RT;
  static constexpr int TILE_BYTES = TILE * HD;             // codes of K (or V) of a tile
  static constexpr int STAGE = 2 * TILE_BYTES + 32;        // K, V, 2 + 2 scales, flag
  static constexpr int RING = AT_WARPS * STAGES * STAGE;
  static constexpr int XROW = HD + 4;                      // exchange row (floats)
  static constexpr int XCH = AT_WARPS * R * XROW * 4;
  static constexpr int Q_OFF = RING > XCH ? RING : XCH;    // the exchange reuses the ring
  static constexpr int Q_TERM = R * HD * 2;
  static constexpr int FAC_OFF = Q_OFF + Q_TERM * (TWO ? 2 : 1);
  static constexpr int ML_OFF = FAC_OFF + R * 4;
  static constexpr int SMEM = ML_OFF + 2 * AT_WARPS * R * 4;
  static constexpr int CB = HD / 4 < 16 ? HD / 4 : 16;     // bytes of a key's row per lane and load
  static constexpr int NH = HD / (4 * CB);
  static constexpr int NW = CB / 4;
  static_assert(STAGE % 16 == 0 && SMEM <= 232448, "shared memory layout");
};

// Offset of 16-byte chunk c of row `row` in a staged tile: chunks are
// swizzled so that the fragment reads of K (two rows, all chunks of a half)
// and of V (four even or odd rows, two chunks) touch every bank once.
template <int HD> FD_DEV int k_off(int row, int c) {
  if constexpr (HD == 128) return row * 128 + ((c ^ (((row & 1) << 2) | ((row >> 1) & 3))) << 4);
  return row * HD + (c << 4);
}
template <int HD> FD_DEV int v_off(int row, int c) {
  if constexpr (HD == 128) return row * 128 + ((c ^ (row & 7)) << 4);
  if constexpr (HD == 64) {
    const int line = row >> 1, p = (row & 1) * 4 + c;
    return line * 128 + ((p ^ ((line & 3) << 1)) << 4);
  }
  return row * HD + (c << 4);
}

template <typename T, int HD, int RT, bool TWO>
__global__ void __launch_bounds__(AT_WARPS * 32, 1) kv8_attn_kernel(const AttnP P) {
  using L_ = Lay<HD, RT, TWO>;
  constexpr int R = L_::R, NH = L_::NH, NW = L_::NW, CB = L_::CB, NTERM = TWO ? 2 : 1;
  extern __shared__ __align__(16) uint8_t smem[];
  const fdllm_kv8& c = P.c;
  const fdllm_kv8_attention_args& a = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, t = lane & 3;
  const int rep = a.n_heads / c.n_kv_heads;
  const int g = blockIdx.y % c.n_kv_heads, seq = blockIdx.z;

  const int r_lo = min(max(a.starts[seq], 0), a.n_tokens);
  const int r_hi = min(max(a.starts[seq + 1], r_lo), a.n_tokens);
  const int rows = (r_hi - r_lo) * rep;
  const int len_in = a.lens[seq];
  const int L = min(max(len_in, 0), c.max_pages * PAGE);
  const bool first_cta = blockIdx.x == 0 && blockIdx.y == 0;
  if (first_cta && tid == 0 && L != len_in && a.status) atomicOr(a.status, FDLLM_KV8_BAD_RANGE);
  const int keys = split_keys(P, L);
  const int n_split = max(1, (L + keys - 1) / keys);
  const int z = blockIdx.x;
  if (z >= n_split) return;
  const int k_lo = z * keys, k_hi = min(L, k_lo + keys);

  const uint32_t sbase = smem_u32(smem);
  const uint32_t ring = sbase + warp * STAGES * L_::STAGE;
  float* fac = reinterpret_cast<float*>(smem + L_::FAC_OFF);
  float* xm = reinterpret_cast<float*>(smem + L_::ML_OFF);   // [warp][R]
  float* xl = xm + AT_WARPS * R;
  float* xo = reinterpret_cast<float*>(smem);                // [warp][R][XROW]

  const int n_tiles = (k_hi - k_lo + TILE - 1) / TILE;
  const int my = n_tiles > warp ? (n_tiles - warp + AT_WARPS - 1) / AT_WARPS : 0;
  const int32_t* table = c.page_table + (int64_t)seq * c.table_stride;

  for (int row0 = (blockIdx.y / c.n_kv_heads) * R; row0 < rows;
       row0 += (gridDim.y / c.n_kv_heads) * R) {
    // ---- q: a warp per row, lanes with 4 dims each; fragment order in shared memory
    for (int r = warp; r < R; r += AT_WARPS) {
      const int rr = row0 + r;
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (rr < rows && lane < HD / 4) {
        const T* src = reinterpret_cast<const T*>(a.q) + (int64_t)(r_lo + rr / rep) * a.q_strides[0] +
                       (int64_t)(g * rep + rr % rep) * a.q_strides[1] + lane * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = to_f<T>(src[i]);
      }
      const float top = warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
      // 2^up brings the row's largest |q| into [2^8, 2^9)
      const int e = (int)((__float_as_uint(top) >> 23) & 255);
      const int up = e == 0 || e == 255 ? 0 : min(135 - e, 120);
      const float mul = __uint_as_float((uint32_t)(up + 127) << 23);
      if (lane < HD / 4) {
        const int d = lane * 4, ct = d / CB, s = (ct / 4) * NW + (d % CB) / 4;
        const int mt = r >> 4, half = (r >> 3) & 1;
        uint8_t* dst = smem + L_::Q_OFF +
                       (((mt * 2 + half) * (HD / 32) + s / 2) * 32 + (r & 7) * 4 + ct % 4) * 16 +
                       (s & 1) * 8;
        __half hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_f16(x[i] * mul, hi[i], lo[i]);
        *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(hi);
        if (TWO) *reinterpret_cast<uint2*>(dst + L_::Q_TERM) = *reinterpret_cast<const uint2*>(lo);
      }
      if (lane == 0) fac[r] = a.scale * LOG2E * __uint_as_float((uint32_t)(127 - up) << 23);
    }
    __syncthreads();

    float o[RT][HD / 8][4];
    float M[RT][2], l[RT][2];
#pragma unroll
    for (int m = 0; m < RT; ++m) {
#pragma unroll
      for (int i = 0; i < HD / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[m][i][j] = 0.0f;
      M[m][0] = M[m][1] = -INFINITY;
      l[m][0] = l[m][1] = 0.0f;
    }

    int pages = 0;   // lane i: page of the warp's tile (issued & ~31) + i
    auto issue = [&](int i) {
      if (i < my) {
        if ((i & 31) == 0) {
          const int k = k_lo + TILE * (warp + AT_WARPS * (i + lane));
          pages = k < k_hi ? table[k / PAGE] : 0;
        }
        const int page = __shfl_sync(0xffffffffu, pages, i & 31);
        const int k0 = k_lo + TILE * (warp + AT_WARPS * i);
        const uint32_t st = ring + (i % STAGES) * L_::STAGE;
        const bool ok = page >= 0 && page < c.n_pages;
        if (ok) {
          const int64_t off = (int64_t)page * c.page_stride +
                              ((int64_t)g * PAGE + k0 % PAGE) * HD + lane * 16;
          const int8_t* ks = c.k + off;
          const int8_t* vs = c.v + off;
#pragma unroll
          for (int j = 0; j < HD / 16; ++j) {
            const int id = j * 32 + lane, row = id / (HD / 16), ch = id % (HD / 16);
            cp16(st + k_off<HD>(row, ch), ks + j * 512);
            cp16(st + L_::TILE_BYTES + v_off<HD>(row, ch), vs + j * 512);
          }
          const int64_t so = (int64_t)page * c.scale_stride + g * 4 + (k0 % PAGE) / 16;
          if (lane < 4)
            cp4(st + 2 * L_::TILE_BYTES + lane * 4, (lane < 2 ? c.k_scale : c.v_scale) + so + (lane & 1));
        } else if (lane == 0 && a.status) {
          atomicOr(a.status, FDLLM_KV8_BAD_PAGE);
        }
        if (lane == 0)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(st + 2 * L_::TILE_BYTES + 16), "r"((int)ok) : "memory");
      }
      cp_commit();
    };

#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue(i);
    for (int it = 0; it < my; ++it) {
      issue(it + STAGES - 1);
      cp_wait<STAGES - 1>();
      __syncwarp();
      const uint32_t st = ring + (it % STAGES) * L_::STAGE;
      const uint32_t vt = st + L_::TILE_BYTES, sc = vt + L_::TILE_BYTES;
      const int k0 = k_lo + TILE * (warp + AT_WARPS * it);
      uint32_t flag[1];
      lds<4>(sc + 16, flag);
      if (flag[0]) {
        // ---- S = Q K^T
        float s[RT][4][4];
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[m][j][e] = 0.0f;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          uint32_t kw[4][NW];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = 8 * j + gid;
            if constexpr (CB == 16) lds<16>(st + k_off<HD>(row, t + 4 * h), kw[j]);
            else lds<CB>(st + row * HD + t * CB, kw[j]);
          }
#pragma unroll
          for (int w2 = 0; w2 < NW; w2 += 2) {
            uint32_t qa[NTERM][RT][2][4];   // [half of the rows]: two k-steps, 2 registers each
            const int sp = (h * NW + w2) / 2;
#pragma unroll
            for (int tm = 0; tm < NTERM; ++tm)
#pragma unroll
              for (int m = 0; m < RT; ++m)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                  lds<16>(sbase + L_::Q_OFF + tm * L_::Q_TERM +
                              (((m * 2 + hf) * (HD / 32) + sp) * 32 + lane) * 16, qa[tm][m][hf]);
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t x = kw[j][w2 + w] ^ 0x80808080u;
                const uint32_t b0 = codes_h2<0x4140>(x), b1 = codes_h2<0x4342>(x);
#pragma unroll
                for (int tm = 0; tm < NTERM; ++tm)
#pragma unroll
                  for (int m = 0; m < RT; ++m) {
                    const uint32_t af[4] = {qa[tm][m][0][2 * w], qa[tm][m][1][2 * w],
                                            qa[tm][m][0][2 * w + 1], qa[tm][m][1][2 * w + 1]};
                    mma16816(s[m][j], af, b0, b1);
                  }
              }
          }
        }
        // ---- softmax weights
        float ks[2], lv[2], iv[2], mn[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float raw[2];
          lds<4>(sc + b * 4, reinterpret_cast<uint32_t*>(&raw[0]));
          lds<4>(sc + 8 + b * 4, reinterpret_cast<uint32_t*>(&raw[1]));
          const bool live = k0 + 16 * b < k_hi;   // else the scales may be anything
          ks[b] = live ? raw[0] : 0.0f;
          const float vs = live ? (raw[1] < VS_MIN ? VS_MIN : raw[1]) : 1.0f;
          if (TWO) {   // vs = mn 2^lv exactly: no rounding of a logarithm reaches a weight
            const int e = (int)(__float_as_uint(vs) >> 23) - 127;
            lv[b] = (float)e;
            iv[b] = __uint_as_float((uint32_t)(127 - e) << 23);
            mn[b] = vs * iv[b];
          } else {
            lv[b] = __log2f(vs);
            iv[b] = __fdividef(1.0f, vs);
            mn[b] = 1.0f;
          }
        }
        const bool tail = k0 + TILE > k_hi;
        bool moved = false;
        float alpha[RT][2];
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float rf = fac[m * 16 + hf * 8 + gid];
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float f = rf * ks[j >> 1];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& v = s[m][j][2 * hf + e];
                v = fmaf(v, f, lv[j >> 1]);
                if (tail && k0 + 8 * j + 2 * t + e >= k_hi) v = -INFINITY;
                mx = fmaxf(mx, v);
              }
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            alpha[m][hf] = 1.0f;
            if (mx > M[m][hf] + M_SLACK || (M[m][hf] == -INFINITY && mx > -INFINITY)) {
              alpha[m][hf] = ex2(M[m][hf] - mx);
              M[m][hf] = mx;
              moved = true;
            }
            const float ref = W_EXP - (M[m][hf] == -INFINITY ? 0.0f : M[m][hf]);
            float sum = 0.0f;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              float part = 0.0f;
#pragma unroll
              for (int j = 2 * b; j < 2 * b + 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float& v = s[m][j][2 * hf + e];
                  v = ex2(v + ref);
                  part += v;
                  if (TWO) v *= mn[b];
                }
              sum = fmaf(part, iv[b], sum);
            }
            l[m][hf] = fmaf(l[m][hf], alpha[m][hf], sum);
          }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int m = 0; m < RT; ++m)
#pragma unroll
            for (int i = 0; i < HD / 8; ++i) {
              o[m][i][0] *= alpha[m][0];
              o[m][i][1] *= alpha[m][0];
              o[m][i][2] *= alpha[m][1];
              o[m][i][3] *= alpha[m][1];
            }
        }
        // ---- O += w V
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t pa[NTERM][RT][4];
#pragma unroll
          for (int m = 0; m < RT; ++m)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float* v = &s[m][2 * b + (q >> 1)][2 * (q & 1)];
              pa[0][m][q] = pack_h2(v[0], v[1]);
              if (TWO) {
                const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&pa[0][m][q]));
                pa[NTERM - 1][m][q] = pack_h2(v[0] - hi.x, v[1] - hi.y);
              }
            }
          uint32_t vw[4][HD / 32];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int row = 16 * b + 2 * t + (q & 1) + 8 * (q >> 1);
            if constexpr (HD == 128) lds<16>(vt + v_off<128>(row, gid), vw[q]);
            else if constexpr (HD == 64) lds<8>(vt + v_off<64>(row, gid >> 1) + (gid & 1) * 8, vw[q]);
            else lds<4>(vt + row * 32 + gid * 4, vw[q]);
          }
#pragma unroll
          for (int i = 0; i < HD / 32; ++i) {
            const uint32_t x0 = vw[0][i] ^ 0x80808080u, x1 = vw[1][i] ^ 0x80808080u;
            const uint32_t x2 = vw[2][i] ^ 0x80808080u, x3 = vw[3][i] ^ 0x80808080u;
            // bytes (row 2t, row 2t + 1) of dims 0, 1 and of dims 2, 3
            const uint32_t a01 = __byte_perm(x0, x1, 0x5140), a23 = __byte_perm(x0, x1, 0x7362);
            const uint32_t b01 = __byte_perm(x2, x3, 0x5140), b23 = __byte_perm(x2, x3, 0x7362);
            const uint32_t f0[4] = {codes_h2<0x4140>(a01), codes_h2<0x4342>(a01),
                                    codes_h2<0x4140>(a23), codes_h2<0x4342>(a23)};
            const uint32_t f1[4] = {codes_h2<0x4140>(b01), codes_h2<0x4342>(b01),
                                    codes_h2<0x4140>(b23), codes_h2<0x4342>(b23)};
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int tm = 0; tm < NTERM; ++tm)
#pragma unroll
                for (int m = 0; m < RT; ++m) mma16816(o[m][4 * i + q], pa[tm][m], f0[q], f1[q]);
          }
        }
      }
      __syncwarp();   // the stage may be refilled
    }
    cp_wait<0>();
    __syncthreads();   // every ring is free: exchange the warps' results

#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float v = l[m][hf];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        const int r = m * 16 + hf * 8 + gid;
        if (t == 0) {
          xm[warp * R + r] = M[m][hf];
          xl[warp * R + r] = v;
        }
        // column n of n-tile i holds dim n * (HD / 8) + i
        float* dst = xo + (warp * R + r) * L_::XROW + 2 * t * (HD / 8);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < HD / 8; i += 4)
            *reinterpret_cast<float4*>(dst + e * (HD / 8) + i) =
                make_float4(o[m][i][2 * hf + e], o[m][i + 1][2 * hf + e], o[m][i + 2][2 * hf + e],
                            o[m][i + 3][2 * hf + e]);
      }
    __syncthreads();
    for (int idx = tid; idx < R * (HD / 4); idx += AT_WARPS * 32) {
      const int r = idx / (HD / 4), d = idx % (HD / 4) * 4, rr = row0 + r;
      if (rr >= rows) continue;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) mx = fmaxf(mx, xm[w * R + r]);
      float sum = 0.0f;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) {
        const float mw = xm[w * R + r];
        const float f = mw == -INFINITY ? 0.0f : ex2(mw - mx);
        const float4 v = *reinterpret_cast<const float4*>(xo + (w * R + r) * L_::XROW + d);
        sum = fmaf(xl[w * R + r], f, sum);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      const int tok = r_lo + rr / rep, head = g * rep + rr % rep;
      if (n_split > 1) {
        const int64_t at = ((int64_t)z * a.n_tokens + tok) * a.n_heads + head;
        *reinterpret_cast<float4*>(P.part_o + at * HD + d) = acc;
        if (d == 0) P.part_ml[at] = make_float2(mx, sum);
      } else {
        const float inv = mx == -INFINITY ? 0.0f : 1.0f / sum;
        T* dst = reinterpret_cast<T*>(a.out) + (int64_t)tok * a.out_strides[0] +
                 (int64_t)head * a.out_strides[1] + d;
        dst[0] = from_f<T>(acc.x * inv);
        dst[1] = from_f<T>(acc.y * inv);
        dst[2] = from_f<T>(acc.z * inv);
        dst[3] = from_f<T>(acc.w * inv);
      }
    }
    __syncthreads();   // exchange area and fac are rewritten by the next row tile
  }
}

// Join the splits of a row: one warp per (token, head), lanes over the dims.
template <typename T, int HD>
__global__ void __launch_bounds__(AT_WARPS * 32) kv8_join_kernel(const AttnP P) {
  const fdllm_kv8_attention_args& a = P.a;
  const int lane = threadIdx.x & 31, seq = blockIdx.y;
  const int r_lo = min(max(a.starts[seq], 0), a.n_tokens);
  const int r_hi = min(max(a.starts[seq + 1], r_lo), a.n_tokens);
  const int L = min(max(a.lens[seq], 0), P.c.max_pages * PAGE);
  const int keys = split_keys(P, L), n_split = (L + keys - 1) / keys;
  if (n_split <= 1) return;
  const int64_t rows = (int64_t)(r_hi - r_lo) * a.n_heads;
  for (int64_t r = blockIdx.x * AT_WARPS + (threadIdx.x >> 5); r < rows;
       r += (int64_t)gridDim.x * AT_WARPS) {
    const int tok = r_lo + (int)(r / a.n_heads), head = (int)(r % a.n_heads);
    const int64_t row = (int64_t)tok * a.n_heads + head, step = (int64_t)a.n_tokens * a.n_heads;
    float mx = -INFINITY;
    for (int z = lane; z < n_split; z += 32) mx = fmaxf(mx, P.part_ml[z * step + row].x);
    mx = warp_max(mx);
    float sum = 0.0f, acc[HD / 32];
#pragma unroll
    for (int i = 0; i < HD / 32; ++i) acc[i] = 0.0f;
    for (int z = 0; z < n_split; ++z) {
      const float2 ml = P.part_ml[z * step + row];
      const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - mx);
      sum = fmaf(ml.y, f, sum);
      const float* po = P.part_o + (z * step + row) * HD;
#pragma unroll
      for (int i = 0; i < HD / 32; ++i) acc[i] = fmaf(po[i * 32 + lane], f, acc[i]);
    }
    const float inv = mx == -INFINITY ? 0.0f : 1.0f / sum;
    T* dst = reinterpret_cast<T*>(a.out) + (int64_t)tok * a.out_strides[0] +
             (int64_t)head * a.out_strides[1];
#pragma unroll
    for (int i = 0; i < HD / 32; ++i) dst[i * 32 + lane] = from_f<T>(acc[i] * inv);
  }
}

struct Plan {
  int rt, row_tiles, n_split, keys;
  size_t bytes;
};

// Rows of a CTA and the key split.  Splits are chosen for the fewest key
// tiles on the busiest SM, a split costing as much as 256 more keys (its
// start, its exchange and its part of the join).
Plan plan(const fdllm_kv8& c, const fdllm_kv8_attention_args& a, int num_sms) {
  Plan p{};
  const int64_t most_q = a.max_q > 0 ? std::min(a.max_q, a.n_tokens) : a.n_tokens;
  const int64_t rows = std::max<int64_t>(1, most_q * (a.n_heads / c.n_kv_heads));
  p.rt = a.dtype != FDLLM_DTYPE_F32 && rows > 16 ? 2 : 1;
  p.row_tiles = (int)std::min<int64_t>((rows + 16 * p.rt - 1) / (16 * p.rt), 65535 / c.n_kv_heads);
  const int64_t table = (int64_t)c.max_pages * PAGE;
  const int64_t len = std::max<int64_t>(1, a.max_len > 0 ? std::min<int64_t>(a.max_len, table) : table);
  const int64_t units = (int64_t)c.n_seqs * c.n_kv_heads * p.row_tiles;
  int64_t best = 0, best_cost = -1;
  for (int64_t s = 1; s <= 256; ++s) {
    const int64_t keys = ((len + s - 1) / s + PAGE - 1) / PAGE * PAGE;
    if (s > 1 && keys < 256) break;
    const int64_t cost = (units * s + num_sms - 1) / num_sms * (keys + 256);
    if (best_cost < 0 || cost < best_cost) best = s, best_cost = cost;
  }
  p.keys = (int)(((len + best - 1) / best + PAGE - 1) / PAGE * PAGE);
  p.n_split = (int)((len + p.keys - 1) / p.keys);
  p.bytes = p.n_split > 1
                ? (size_t)p.n_split * a.n_tokens * a.n_heads * (c.head_dim + 2) * sizeof(float) : 0;
  return p;
}

template <typename K>
cudaError_t big_smem(K kern, int bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, int HD, int RT, bool TWO>
cudaError_t launch_attn_rt(const AttnP& P, dim3 grid, cudaStream_t st) {
  auto kern = kv8_attn_kernel<T, HD, RT, TWO>;
  constexpr int smem = Lay<HD, RT, TWO>::SMEM;
  cudaError_t e = big_smem(kern, smem);
  if (e == cudaSuccess) e = launch_k(false, kern, grid, dim3(AT_WARPS * 32), smem, st, P);
  return e;
}

template <typename T, int HD>
cudaError_t launch_attn_hd(const AttnP& P, const Plan& p, cudaStream_t st) {
  const dim3 grid(p.n_split, P.c.n_kv_heads * p.row_tiles, P.c.n_seqs);
  cudaError_t e;
  if constexpr (std::is_same_v<T, float>)
    e = launch_attn_rt<T, HD, 1, true>(P, grid, st);
  else
    e = p.rt == 1 ? launch_attn_rt<T, HD, 1, false>(P, grid, st)
                  : launch_attn_rt<T, HD, 2, false>(P, grid, st);
  if (e != cudaSuccess || p.n_split == 1) return e;
  const int64_t most_q = P.a.max_q > 0 ? std::min(P.a.max_q, P.a.n_tokens) : P.a.n_tokens;
  const dim3 jgrid((unsigned)std::min<int64_t>((most_q * P.a.n_heads + AT_WARPS - 1) / AT_WARPS, 1 << 20),
                   P.c.n_seqs);
  return launch_k(false, kv8_join_kernel<T, HD>, jgrid, dim3(AT_WARPS * 32), 0, st, P);
}

template <typename T>
cudaError_t launch_attn_t(const AttnP& P, const Plan& p, cudaStream_t st) {
  switch (P.c.head_dim) {
    case 128: return launch_attn_hd<T, 128>(P, p, st);
    case 64: return launch_attn_hd<T, 64>(P, p, st);
    default: return launch_attn_hd<T, 32>(P, p, st);
  }
}

const char* check_args(const fdllm_kv8_attention_args* args, const fdllm_kv8& c) {
  if (!args) return "args is NULL";
  const fdllm_kv8_attention_args& a = *args;
  if (!kv8::elem_bytes(a.dtype)) return "unknown dtype";
  if (a.n_tokens < 0 || a.max_q < 0 || a.max_len < 0) return "n_tokens, max_q and max_len must be >= 0";
  if (a.n_heads < 1 || a.n_heads > 65535 || a.n_heads % c.n_kv_heads)
    return "n_heads must be a multiple of n_kv_heads in [1, 65535]";
  if ((int64_t)a.n_tokens * (a.n_heads / c.n_kv_heads) > 0x7fffffff) return "too many query rows";
  if (!std::isfinite(a.scale)) return "scale must be finite";
  return nullptr;
}

cudaError_t sm_count(int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  return e;
}

}  // namespace
}  // namespace fd

extern "C" int fdllm_kv8_attention_workspace(const fdllm_kv8* cache,
                                             const fdllm_kv8_attention_args* args, size_t* bytes) {
  using namespace fd;
  const char* call = "fdllm_kv8_attention_workspace";
  fdllm_kv8 c;
  if (!cache || !args || !bytes) return kv8::fail(call, FDLLM_ERR_ARG, "NULL argument");
  fdllm_kv8 shape = *cache;   // pointers are not looked at
  shape.k = shape.v = reinterpret_cast<int8_t*>(16);
  shape.k_scale = shape.v_scale = reinterpret_cast<float*>(16);
  shape.page_table = reinterpret_cast<const int32_t*>(16);
  if (const char* why = kv8::check_cache(&shape, &c)) return kv8::fail(call, FDLLM_ERR_ARG, why);
  if (const char* why = check_args(args, c)) return kv8::fail(call, FDLLM_ERR_ARG, why);
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return kv8::fail(call, FDLLM_ERR_CUDA, cudaGetErrorString(e));
  *bytes = plan(c, *args, sms).bytes;
  return FDLLM_OK;
}

extern "C" int fdllm_kv8_attention(const fdllm_kv8* cache, const fdllm_kv8_attention_args* args,
                                   void* cuda_stream) {
  using namespace fd;
  const char* call = "fdllm_kv8_attention";
  AttnP P{};
  if (const char* why = kv8::check_cache(cache, &P.c)) return kv8::fail(call, FDLLM_ERR_ARG, why);
  if (const char* why = check_args(args, P.c)) return kv8::fail(call, FDLLM_ERR_ARG, why);
  P.a = *args;
  const fdllm_kv8_attention_args& a = P.a;
  if (!a.starts || !a.lens) return kv8::fail(call, FDLLM_ERR_ARG, "starts or lens is NULL");
  if (!kv8::aligned4({a.starts, a.lens, a.status}))
    return kv8::fail(call, FDLLM_ERR_ARG, "int32 arrays must be 4-byte aligned");
  if (a.n_tokens == 0) return FDLLM_OK;
  if (!a.q || !a.out) return kv8::fail(call, FDLLM_ERR_ARG, "q or out is NULL");
  const int esz = kv8::elem_bytes(a.dtype);
  if (!kv8::rows_ok(a.q, a.q_strides, esz) || !kv8::rows_ok(a.out, a.out_strides, esz))
    return kv8::fail(call, FDLLM_ERR_ARG, "rows and heads of q and out must be 16-byte aligned");
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return kv8::fail(call, FDLLM_ERR_CUDA, cudaGetErrorString(e));
  Plan p = plan(P.c, a, sms);
  if (!a.workspace && p.n_split > 1) {
    p.n_split = 1;
    p.keys = P.c.max_pages * PAGE;
  }
  if (p.n_split > 1) {
    if (a.workspace_bytes < p.bytes || !kv8::aligned16(a.workspace))
      return kv8::fail(call, FDLLM_ERR_ARG, "workspace needs " + std::to_string(p.bytes) +
                                                " bytes, 16-byte aligned");
    P.part_o = static_cast<float*>(a.workspace);
    P.part_ml = reinterpret_cast<float2*>(
        P.part_o + (size_t)p.n_split * a.n_tokens * a.n_heads * P.c.head_dim);
  }
  P.n_split = p.n_split;
  P.keys = p.keys;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  e = a.dtype == FDLLM_DTYPE_F32    ? launch_attn_t<float>(P, p, st)
      : a.dtype == FDLLM_DTYPE_BF16 ? launch_attn_t<__nv_bfloat16>(P, p, st)
                                    : launch_attn_t<__half>(P, p, st);
  if (e != cudaSuccess) return kv8::fail(call, FDLLM_ERR_CUDA, cudaGetErrorString(e));
  return FDLLM_OK;
}
