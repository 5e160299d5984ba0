// fdllm_kv8_attention: attention of a few query rows per sequence over the
// 8-bit paged K/V cache.
//
// A query row is a (token, head-in-group) pair, so that the query heads of a
// K/V head share every cached byte.  A run is a tile of 16 RT rows, a K/V head
// and a sequence with all its pages; the pages of all runs, laid end to end,
// are shared out evenly over the CTAs (two an SM), whatever the lengths are.
// They are known on the device only, so every CTA sums them up for itself.
// A CTA's 4 warps take its part of a run in tiles of 32 keys, every warp with
// a ring of cp.async stages, softmax statistics and an output accumulator of
// its own, so the loop has no barrier beyond the warp's; the warps' results
// meet in shared memory.  A run that a CTA does not hold whole leaves a
// partial result in the workspace (at most two a CTA: the end of one run and
// the start of another), and a second kernel joins those, one block for the
// first share boundary inside a run.
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

constexpr int AT_WARPS = 4;    // two CTAs an SM: one's start and end hide behind the other's loop
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
  int n_cta;         // shares (the grid)
  float* part_o;     // [share][2][rows of a tile][head_dim]; NULL: runs are not split
  float2* part_ml;   // [share][2][rows of a tile] (reference max, weight sum)
};

// A sequence's rows and runs.
struct Seq {
  int r_lo, rows, len, pages, tiles;   // rows: (token, head) pairs of a K/V head
  int64_t work;                        // pages of all its runs
};
FD_DEV Seq seq_of(const AttnP& P, int i, int tile_rows) {
  const fdllm_kv8_attention_args& a = P.a;
  Seq s;
  s.r_lo = min(max(a.starts[i], 0), a.n_tokens);
  const int r_hi = min(max(a.starts[i + 1], s.r_lo), a.n_tokens);
  s.rows = (r_hi - s.r_lo) * (a.n_heads / P.c.n_kv_heads);
  s.len = min(max(a.lens[i], 0), P.c.max_pages * PAGE);
  s.pages = max(1, (s.len + PAGE - 1) / PAGE);   // a run without keys still writes its zeros
  s.tiles = (s.rows + tile_rows - 1) / tile_rows;
  s.work = (int64_t)s.tiles * P.c.n_kv_heads * s.pages;
  return s;
}
// Sum of all sequences' work, by a warp.
FD_DEV int64_t total_work(const AttnP& P, int tile_rows) {
  const int lane = threadIdx.x & 31;
  int64_t t = 0;
  for (int i = lane; i < P.c.n_seqs; i += 32) t += seq_of(P, i, tile_rows).work;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}
// The sequence that holds position x < total of the pages laid end to end,
// by a warp; *off: the place within it.
FD_DEV int find_seq(const AttnP& P, int tile_rows, int64_t x, int64_t* off) {
  const int lane = threadIdx.x & 31;
  int64_t base = 0;
  for (int i0 = 0;; i0 += 32) {
    const int64_t w = i0 + lane < P.c.n_seqs ? seq_of(P, i0 + lane, tile_rows).work : 0;
    int64_t upto = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, base + upto > x);
    if (hit || i0 + 32 >= P.c.n_seqs) {
      const int l = hit ? __ffs(hit) - 1 : 0;
      *off = x - base - __shfl_sync(0xffffffffu, upto - w, l);
      return i0 + l;
    }
    base += __shfl_sync(0xffffffffu, upto, 31);
  }
}
// Shares in use: at least MIN_PAGES pages each.
constexpr int MIN_PAGES = 2;
FD_DEV int64_t shares(const AttnP& P, int64_t total) {
  return max((int64_t)1, min((int64_t)P.n_cta, (total + MIN_PAGES - 1) / MIN_PAGES));
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

// 4 consecutive elements of a row (aligned to their size).
template <typename T> FD_DEV void load4(const T* p, float* x) {
  if constexpr (sizeof(T) == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = to_f<T>(e[i]);
  }
}
template <typename T> FD_DEV void store4(T* p, float a, float b, float c, float d) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
  } else {
    const T e[4] = {from_f<T>(a), from_f<T>(b), from_f<T>(c), from_f<T>(d)};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(e);
  }
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
  static_assert(STAGE % 16 == 0 && SMEM <= 115712, "shared memory layout");
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
__global__ void __launch_bounds__(AT_WARPS * 32, 2) kv8_attn_kernel(const AttnP P) {
  using L_ = Lay<HD, RT, TWO>;
  constexpr int R = L_::R, NH = L_::NH, NW = L_::NW, CB = L_::CB, NTERM = TWO ? 2 : 1;
  extern __shared__ __align__(16) uint8_t smem[];
  const fdllm_kv8& c = P.c;
  const fdllm_kv8_attention_args& a = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, t = lane & 3;
  const int rep = a.n_heads / c.n_kv_heads;
  pdl_trigger();   // the join may be set up; it waits for this grid's end
  if (blockIdx.x == 0 && a.status)
    for (int i = tid; i < c.n_seqs; i += AT_WARPS * 32)
      if (a.lens[i] < 0 || a.lens[i] > c.max_pages * PAGE) atomicOr(a.status, FDLLM_KV8_BAD_RANGE);

  // ---- this CTA's share [x, x_end) of all runs' pages
  const int64_t total = total_work(P, R), n_cta = shares(P, total);
  if (blockIdx.x >= n_cta) return;
  int64_t x = total * blockIdx.x / n_cta, off = 0;
  const int64_t x_end = total * (blockIdx.x + 1) / n_cta;
  if (x >= x_end) return;
  int seq = find_seq(P, R, x, &off);
  Seq sq = seq_of(P, seq, R);

  const uint32_t sbase = smem_u32(smem);
  const uint32_t ring = sbase + warp * STAGES * L_::STAGE;
  float* fac = reinterpret_cast<float*>(smem + L_::FAC_OFF);
  float* xm = reinterpret_cast<float*>(smem + L_::ML_OFF);   // [warp][R]
  float* xl = xm + AT_WARPS * R;
  float* xo = reinterpret_cast<float*>(smem);                // [warp][R][XROW]

  while (x < x_end) {
    while (off >= sq.work) {
      off -= sq.work;
      sq = seq_of(P, ++seq, R);
    }
    const int run = (int)(off / sq.pages), p_lo = (int)(off % sq.pages);
    int p_hi = (int)min((int64_t)sq.pages, p_lo + (x_end - x));
    if (!P.part_o) {   // whole runs: those that start in the share
      if (p_lo > 0) {
        x += sq.pages - p_lo;
        off += sq.pages - p_lo;
        continue;
      }
      p_hi = sq.pages;
    }
    x += p_hi - p_lo;
    off += p_hi - p_lo;
    const bool whole = p_lo == 0 && p_hi == sq.pages;
    const int g = run / sq.tiles, row0 = run % sq.tiles * R, rows = sq.rows, r_lo = sq.r_lo;
    const int k_lo = p_lo * PAGE, k_hi = min(sq.len, p_hi * PAGE);
    const int n_tiles = (k_hi - k_lo + TILE - 1) / TILE;
    const int my = n_tiles > warp ? (n_tiles - warp + AT_WARPS - 1) / AT_WARPS : 0;
    const int32_t* table = c.page_table + (int64_t)seq * c.table_stride;

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

    // ---- q: a warp per row, lanes with 4 dims each; fragment order in shared memory
    float qx[R / AT_WARPS][4];
#pragma unroll
    for (int j = 0; j < R / AT_WARPS; ++j) {
      const int rr = row0 + warp + j * AT_WARPS;
#pragma unroll
      for (int i = 0; i < 4; ++i) qx[j][i] = 0.0f;
      if (rr < rows && lane < HD / 4)
        load4(reinterpret_cast<const T*>(a.q) + (int64_t)(r_lo + rr / rep) * a.q_strides[0] +
                  (int64_t)(g * rep + rr % rep) * a.q_strides[1] + lane * 4, qx[j]);
    }
#pragma unroll
    for (int j = 0; j < R / AT_WARPS; ++j) {
      const int r = warp + j * AT_WARPS;
      const float* x = qx[j];
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
      if (!whole) {
        const int64_t at = ((int64_t)blockIdx.x * 2 + (p_lo == 0)) * R + r;
        *reinterpret_cast<float4*>(P.part_o + at * HD + d) = acc;
        if (d == 0) P.part_ml[at] = make_float2(mx, sum);
      } else {
        const int tok = r_lo + rr / rep, head = g * rep + rr % rep;
        const float inv = mx == -INFINITY ? 0.0f : 1.0f / sum;
        T* dst = reinterpret_cast<T*>(a.out) + (int64_t)tok * a.out_strides[0] +
                 (int64_t)head * a.out_strides[1] + d;
        store4(dst, acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      }
    }
    __syncthreads();   // exchange area and fac are rewritten by the next run
  }
}

// Joins the partial results of the run around share boundary blockIdx.x + 1,
// if that is the first boundary inside it: the end of the share before (its
// slot 1, the run's start), and slot 0 of the shares that follow.  A warp per
// row, lanes over the dims.
template <typename T, int HD, int R>
__global__ void __launch_bounds__(AT_WARPS * 32) kv8_join_kernel(const AttnP P) {
  const fdllm_kv8_attention_args& a = P.a;
  const int lane = threadIdx.x & 31;
  const int64_t total = total_work(P, R), n_cta = shares(P, total), c = blockIdx.x + 1;
  bool mine = c < n_cta;
  int64_t off = 0;
  const int64_t x = mine ? total * c / n_cta : 0;
  const int seq = mine ? find_seq(P, R, x, &off) : 0;
  const Seq sq = seq_of(P, seq, R);
  const int p = (int)(off % sq.pages), run = (int)(off / sq.pages);
  mine = mine && p != 0 && total * (c - 1) / n_cta <= x - p;
  const int64_t run_end = x - p + sq.pages;
  int n = 1;   // pieces
  if (mine)
    while (c + n - 1 < n_cta && total * (c + n - 1) / n_cta < run_end) ++n;
  const int rep = a.n_heads / P.c.n_kv_heads, g = mine ? run / sq.tiles : 0;
  const int r = blockIdx.y * AT_WARPS + (threadIdx.x >> 5), rr = mine ? run % sq.tiles * R + r : 0;
  pdl_wait();   // by every block: this grid must not end before the one that feeds it
  if (!mine || rr >= sq.rows) return;
  auto piece = [&](int i) { return ((c - 1 + i) * 2 + (i == 0)) * R + r; };
  float mx = -INFINITY;
  for (int i = lane; i < n; i += 32) mx = fmaxf(mx, P.part_ml[piece(i)].x);
  mx = warp_max(mx);
  float sum = 0.0f, acc[HD / 32];
#pragma unroll
  for (int i = 0; i < HD / 32; ++i) acc[i] = 0.0f;
#pragma unroll 8
  for (int i = 0; i < n; ++i) {
    const float2 ml = P.part_ml[piece(i)];
    const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - mx);
    sum = fmaf(ml.y, f, sum);
    const float* po = P.part_o + piece(i) * HD;
#pragma unroll
    for (int j = 0; j < HD / 32; ++j) acc[j] = fmaf(po[j * 32 + lane], f, acc[j]);
  }
  const float inv = mx == -INFINITY ? 0.0f : 1.0f / sum;
  T* dst = reinterpret_cast<T*>(a.out) + (int64_t)(sq.r_lo + rr / rep) * a.out_strides[0] +
           (int64_t)(g * rep + rr % rep) * a.out_strides[1];
#pragma unroll
  for (int j = 0; j < HD / 32; ++j) dst[j * 32 + lane] = from_f<T>(acc[j] * inv);
}

struct Plan {
  int rt, n_cta;
  size_t bytes;
};

// Rows of a tile and the number of shares: two CTAs an SM, fewer when the
// hints say that there are not MIN_PAGES pages for each.
Plan plan(const fdllm_kv8& c, const fdllm_kv8_attention_args& a, int num_sms) {
  Plan p{};
  const int64_t most_q = a.max_q > 0 ? std::min(a.max_q, a.n_tokens) : a.n_tokens;
  const int64_t rows = std::max<int64_t>(1, most_q * (a.n_heads / c.n_kv_heads));
  p.rt = a.dtype != FDLLM_DTYPE_F32 && rows > 16 ? 2 : 1;
  const int64_t table = (int64_t)c.max_pages * PAGE;
  const int64_t len = std::max<int64_t>(1, a.max_len > 0 ? std::min<int64_t>(a.max_len, table) : table);
  const double pages = (double)c.n_seqs * c.n_kv_heads * ((rows + 16 * p.rt - 1) / (16 * p.rt)) *
                       ((len + PAGE - 1) / PAGE);
  p.n_cta = (int)std::min<double>(2.0 * num_sms, std::ceil(pages / MIN_PAGES));
  p.bytes = p.n_cta > 1 ? (size_t)p.n_cta * 2 * 16 * p.rt * (c.head_dim + 2) * sizeof(float) : 0;
  return p;
}

template <typename T, int HD, int RT, bool TWO>
cudaError_t launch_attn_rt(const AttnP& P, dim3 grid, cudaStream_t st) {
  auto kern = kv8_attn_kernel<T, HD, RT, TWO>;
  constexpr int smem = Lay<HD, RT, TWO>::SMEM;
  static std::atomic<uint64_t> ready{0};   // devices whose limit is set
  cudaError_t e = kv8::allow_smem(kern, smem, ready);
  if (e == cudaSuccess) e = launch_k(false, kern, grid, dim3(AT_WARPS * 32), smem, st, P);
  return e;
}

template <typename T, int HD>
cudaError_t launch_attn_hd(const AttnP& P, const Plan& p, cudaStream_t st) {
  const dim3 grid(p.n_cta);
  cudaError_t e;
  if constexpr (std::is_same_v<T, float>)
    e = launch_attn_rt<T, HD, 1, true>(P, grid, st);
  else
    e = p.rt == 1 ? launch_attn_rt<T, HD, 1, false>(P, grid, st)
                  : launch_attn_rt<T, HD, 2, false>(P, grid, st);
  if (e != cudaSuccess || !P.part_o) return e;
  const dim3 jgrid(p.n_cta - 1, 16 * p.rt / AT_WARPS), block(AT_WARPS * 32);
  return p.rt == 1 ? launch_k(true, kv8_join_kernel<T, HD, 16>, jgrid, block, 0, st, P)
                   : launch_k(true, kv8_join_kernel<T, HD, 32>, jgrid, block, 0, st, P);
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
  const cudaError_t e = kv8::sm_count(&sms);
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
  cudaError_t e = kv8::sm_count(&sms);
  if (e != cudaSuccess) return kv8::fail(call, FDLLM_ERR_CUDA, cudaGetErrorString(e));
  const Plan p = plan(P.c, a, sms);
  P.n_cta = p.n_cta;
  if (p.bytes > 0 && a.workspace) {
    if (a.workspace_bytes < p.bytes || !kv8::aligned16(a.workspace))
      return kv8::fail(call, FDLLM_ERR_ARG, "workspace needs " + std::to_string(p.bytes) +
                                                " bytes, 16-byte aligned");
    P.part_o = static_cast<float*>(a.workspace);
    P.part_ml = reinterpret_cast<float2*>(P.part_o + (size_t)p.n_cta * 2 * 16 * p.rt * P.c.head_dim);
  }
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  e = a.dtype == FDLLM_DTYPE_F32    ? launch_attn_t<float>(P, p, st)
      : a.dtype == FDLLM_DTYPE_BF16 ? launch_attn_t<__nv_bfloat16>(P, p, st)
                                    : launch_attn_t<__half>(P, p, st);
  if (e != cudaSuccess) return kv8::fail(call, FDLLM_ERR_CUDA, cudaGetErrorString(e));
  return FDLLM_OK;
}
