// fdllm_kv8_attention, and its kernel for up to 64 query rows a K/V head, 16 a
// run (and for more rows of short work, see plan): attention over the 8-bit paged
// K/V cache on mma.sync.
//
// With few rows the kernel streams the cache, and operands that go straight
// to registers spare the round trip through shared memory and TMEM that a
// converted tile would take (kv8_attn_tc.cu takes it for more rows).  A CTA's
// 4 warps take its part of a run in tiles of 32 keys, every warp with a ring
// of cp.async stages, softmax statistics and an output accumulator of its
// own, so the loop has no barrier beyond the warp's; the warps' results meet
// in shared memory.  Two CTAs an SM: one's start and end hide behind the
// other's loop.
//
// Bound: 64 sequences' tokens over up to 8192 keys (4 K/V heads of 128 dims, 281
// MB) take 68 us, 4.2 TB/s: 8 warps an SM with 2 stages in flight each wait for
// instructions of their own chain (933 a tile of 32 keys) as much as for memory;
// more warps do not fit the accumulators' registers (234 a thread), half of
// which are idle rows when a K/V head has 8 query rows or fewer.  A lone token
// over 512 keys takes 8.9 us, a chain of latencies: the lengths (1.2), page ids
// (0.8), q (0.8), the tile (1.3), the warps' exchange (0.8), the join's launch.
//
// Codes are exact in fp16 and become matrix operands on the way from shared
// memory to registers.  Both contractions are free in the order of their
// index, and so every lane reads 16 consecutive bytes: in Q K^T the dims are
// permuted alike in q and k, in P V the output columns.
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
#include <cstdlib>

#include "kv8_attn.cuh"

namespace fd {
namespace {

using namespace kv8;

constexpr int AT_WARPS = 4;
constexpr int TILE = 32;      // keys of a warp's tile
constexpr int STAGES = 3;
constexpr int R = 16;         // rows of a run

FD_DEV void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
FD_DEV void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
FD_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> FD_DEV void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

FD_DEV void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// N bytes of shared memory as words.
template <int N> FD_DEV void lds(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (N == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

template <int HD, bool TWO>
struct Lay {
  static constexpr int TILE_BYTES = TILE * HD;             // codes of K (or V) of a tile
  static constexpr int STAGE = 2 * TILE_BYTES + 32;        // K, V, 2 + 2 scales, flag
  static constexpr int RING = AT_WARPS * STAGES * STAGE;
  static constexpr int XROW = HD + 4;                      // exchange row (floats)
  static constexpr int XCH = AT_WARPS * R * XROW * 4;
  static constexpr int Q_OFF = RING > XCH ? RING : XCH;    // the exchange reuses the ring
  static constexpr int Q_TERM = R * HD * 2;
  static constexpr int FAC_OFF = Q_OFF + Q_TERM * (TWO ? 2 : 1);
  static constexpr int ML_OFF = FAC_OFF + R * 4;
  static constexpr int WALK_OFF = ML_OFF + (2 * AT_WARPS + 1) * R * 4;
  static constexpr int SMEM = WALK_OFF + AT_WARPS * (int)sizeof(Walk);
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

template <typename T, int HD, bool TWO>
__global__ void __launch_bounds__(AT_WARPS * 32, 2) kv8_attn_kernel(const AttnP P) {
  using L_ = Lay<HD, TWO>;
  constexpr int NH = L_::NH, NW = L_::NW, CB = L_::CB, NTERM = TWO ? 2 : 1;
  // With the mantissa of vs a factor of the weight, which may then be twice as
  // large: 2^(W_EXP + SLACK) 2 stays below fp16's 65504.
  constexpr float SLACK = TWO ? M_SLACK - 1.0f : M_SLACK;
  extern __shared__ __align__(16) uint8_t smem[];
  const fdllm_kv8& c = P.c;
  const fdllm_kv8_attention_args& a = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, t = lane & 3;
  const int rep = a.n_heads / c.n_kv_heads;
  uint8_t* ring = smem + warp * STAGES * L_::STAGE;
  float* fac = reinterpret_cast<float*>(smem + L_::FAC_OFF);
  float* xf = reinterpret_cast<float*>(smem + L_::ML_OFF);   // [warp][R] reference max, then factor
  float* xl = xf + AT_WARPS * R;                             // [warp][R] weight sum
  float* xi = xl + AT_WARPS * R;                             // [R] 1 / sum of all
  float* xo = reinterpret_cast<float*>(smem);                // [warp][R][XROW]

  pdl_trigger();   // the join may be set up; it waits for this grid's end
  report_range(P);
  Walk* walk = reinterpret_cast<Walk*>(smem + L_::WALK_OFF) + warp;
  walk_start(walk, P, R);
  Segment sg;
  while (walk_next(walk, P, R, &sg)) {
    const int g = sg.g, rows = sg.rows, r_lo = sg.r_lo;
    const int k_lo = sg.p_lo * PAGE, k_hi = min(sg.len, sg.p_hi * PAGE);
    const int n_tiles = (k_hi - k_lo + TILE - 1) / TILE;
    const int my = n_tiles > warp ? (n_tiles - warp + AT_WARPS - 1) / AT_WARPS : 0;
    const int32_t* table = c.page_table + (int64_t)sg.seq * c.table_stride;

    // ---- q: a warp per row, lanes with 4 dims each, on its way while the page
    // table is read; then in fragment order to shared memory
    float qx[R / AT_WARPS][4];
    {
      int token = (sg.row0 + warp) / rep, head = (sg.row0 + warp) % rep;
#pragma unroll
      for (int j = 0; j < R / AT_WARPS; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) qx[j][i] = 0.0f;
        if (sg.row0 + warp + j * AT_WARPS < rows && lane < HD / 4)
          load4(reinterpret_cast<const T*>(a.q) + (int64_t)(r_lo + token) * a.q_strides[0] +
                    (int64_t)(g * rep + head) * a.q_strides[1] + lane * 4, qx[j]);
        for (head += AT_WARPS; head >= rep; head -= rep) ++token;
      }
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
        uint8_t* stage = ring + (i % STAGES) * L_::STAGE;
        const uint32_t st = smem_u32(stage);
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
        if (lane == 0) *reinterpret_cast<int*>(stage + 2 * L_::TILE_BYTES + 16) = ok;
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue(i);
#pragma unroll
    for (int j = 0; j < R / AT_WARPS; ++j) {
      const int r = warp + j * AT_WARPS;
      const float* x = qx[j];
      const int up = q_shift(warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])))));
      const float mul = exp2_int(up);
      if (lane < HD / 4) {
        const int d = lane * 4, ct = d / CB, s = (ct / 4) * NW + (d % CB) / 4;
        uint8_t* dst = smem + L_::Q_OFF +
                       (((r >> 3) * (HD / 32) + s / 2) * 32 + (r & 7) * 4 + ct % 4) * 16 + (s & 1) * 8;
        __half hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_f16(x[i] * mul, hi[i], lo[i]);
        *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(hi);
        if (TWO) *reinterpret_cast<uint2*>(dst + L_::Q_TERM) = *reinterpret_cast<const uint2*>(lo);
      }
      if (lane == 0) fac[r] = a.scale * LOG2E * exp2_int(-up);
    }
    __syncthreads();

    float o[HD / 8][4];
#pragma unroll
    for (int i = 0; i < HD / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
    float M[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const float rf[2] = {fac[gid], fac[8 + gid]};

    for (int it = 0; it < my; ++it) {
      issue(it + STAGES - 1);
      cp_wait<STAGES - 1>();
      __syncwarp();
      const uint8_t* kt = ring + (it % STAGES) * L_::STAGE;
      const uint8_t* vt = kt + L_::TILE_BYTES;
      const float* sc = reinterpret_cast<const float*>(vt + L_::TILE_BYTES);
      const int k0 = k_lo + TILE * (warp + AT_WARPS * it);
      if (*reinterpret_cast<const int*>(sc + 4)) {
        // ---- S = Q K^T
        float s[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[j][e] = 0.0f;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          uint32_t kw[4][NW];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = 8 * j + gid;
            if constexpr (CB == 16) lds<16>(kt + k_off<HD>(row, t + 4 * h), kw[j]);
            else lds<CB>(kt + row * HD + t * CB, kw[j]);
          }
#pragma unroll
          for (int w2 = 0; w2 < NW; w2 += 2) {
            uint32_t qa[NTERM][2][4];   // [half of the rows]: two k-steps, 2 registers each
            const int sp = (h * NW + w2) / 2;
#pragma unroll
            for (int tm = 0; tm < NTERM; ++tm)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
                lds<16>(smem + L_::Q_OFF + tm * L_::Q_TERM + ((hf * (HD / 32) + sp) * 32 + lane) * 16,
                        qa[tm][hf]);
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t x = kw[j][w2 + w] ^ 0x80808080u;
                const uint32_t b0 = codes_h2<0x4140>(x), b1 = codes_h2<0x4342>(x);
#pragma unroll
                for (int tm = 0; tm < NTERM; ++tm) {
                  const uint32_t af[4] = {qa[tm][0][2 * w], qa[tm][1][2 * w], qa[tm][0][2 * w + 1],
                                          qa[tm][1][2 * w + 1]};
                  mma16816(s[j], af, b0, b1);
                }
              }
          }
        }
        // ---- softmax weights
        float ks[2], lv[2], iv[2], mn[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const bool live = k0 + 16 * b < k_hi;   // else the scales may be anything
          ks[b] = live ? sc[b] : 0.0f;
          const float raw = sc[2 + b], vs = live ? (raw < VS_MIN ? VS_MIN : raw) : 1.0f;
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
        float alpha[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float mx = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float f = rf[hf] * ks[j >> 1];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& v = s[j][2 * hf + e];
              v = fmaf(v, f, lv[j >> 1]);
              if (tail && k0 + 8 * j + 2 * t + e >= k_hi) v = -INFINITY;
              mx = fmaxf(mx, v);
            }
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          alpha[hf] = 1.0f;
          if (passes(mx, M[hf], SLACK)) {
            alpha[hf] = ex2(M[hf] - mx);
            M[hf] = mx;
            moved = true;
          }
          const float ref = weight_ref(M[hf]);
          float sum = 0.0f;
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float part = 0.0f;
#pragma unroll
            for (int j = 2 * b; j < 2 * b + 2; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& v = s[j][2 * hf + e];
                v = ex2(v + ref);
                part += v;
                if (TWO) v *= mn[b];
              }
            sum = fmaf(part, iv[b], sum);
          }
          l[hf] = fmaf(l[hf], alpha[hf], sum);
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int i = 0; i < HD / 8; ++i) {
            o[i][0] *= alpha[0];
            o[i][1] *= alpha[0];
            o[i][2] *= alpha[1];
            o[i][3] *= alpha[1];
          }
        }
        // ---- O += w V
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t pa[NTERM][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float* v = &s[2 * b + (q >> 1)][2 * (q & 1)];
            pa[0][q] = pack_h2(v[0], v[1]);
            if (TWO) {
              const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&pa[0][q]));
              pa[NTERM - 1][q] = pack_h2(v[0] - hi.x, v[1] - hi.y);
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
              for (int tm = 0; tm < NTERM; ++tm) mma16816(o[4 * i + q], pa[tm], f0[q], f1[q]);
          }
        }
      }
      __syncwarp();   // the stage may be refilled
    }
    cp_wait<0>();
    __syncthreads();   // every ring is free: exchange the warps' results

#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float v = l[hf];
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      const int r = hf * 8 + gid;
      if (t == 0) {
        xf[warp * R + r] = M[hf];
        xl[warp * R + r] = v;
      }
      // column n of n-tile i holds dim n * (HD / 8) + i
      float* dst = xo + (warp * R + r) * L_::XROW + 2 * t * (HD / 8);
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < HD / 8; i += 4)
          *reinterpret_cast<float4*>(dst + e * (HD / 8) + i) =
              make_float4(o[i][2 * hf + e], o[i + 1][2 * hf + e], o[i + 2][2 * hf + e], o[i + 3][2 * hf + e]);
    }
    __syncthreads();
    if (tid < R) {
      float mw[AT_WARPS], mx = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) mx = fmaxf(mx, mw[w] = xf[w * R + tid]);
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) {
        const float f = mw[w] == -INFINITY ? 0.0f : ex2(mw[w] - mx);
        xf[w * R + tid] = f;
        sum = fmaf(xl[w * R + tid], f, sum);
      }
      xi[tid] = mx == -INFINITY ? 0.0f : 1.0f / sum;
      if (!sg.whole)
        P.part_ml[((int64_t)blockIdx.x * 2 + (sg.p_lo == 0)) * R + tid] = make_float2(mx, sum);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < R * HD / (4 * AT_WARPS * 32); ++j) {
      const int idx = j * AT_WARPS * 32 + tid, r = idx / (HD / 4), d = idx % (HD / 4) * 4;
      const int rr = sg.row0 + r;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) {
        const float f = xf[w * R + r];
        const float4 v = *reinterpret_cast<const float4*>(xo + (w * R + r) * L_::XROW + d);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      if (rr < rows) {
        if (!sg.whole) {
          const int64_t at = ((int64_t)blockIdx.x * 2 + (sg.p_lo == 0)) * R + r;
          *reinterpret_cast<float4*>(P.part_o + at * HD + d) = acc;
        } else {
          const float inv = xi[r];
          T* dst = reinterpret_cast<T*>(a.out) + (int64_t)(r_lo + rr / rep) * a.out_strides[0] +
                   (int64_t)(g * rep + rr % rep) * a.out_strides[1] + d;
          store4(dst, acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        }
      }
    }
    __syncthreads();   // the exchange area and fac are rewritten by the next run
  }
}

struct Plan {
  int tile_rows, n_cta;   // tile_rows R: the kernel above
  size_t bytes;
};

// The kernel, the rows of its tile and the number of shares.  Up to 64 rows a
// K/V head, for float32 and for heads of 32 dims: the kernel above.  For more
// rows, kv8_attn_tc.cu takes a page once for all of them but starts and ends
// more slowly; a share of w pages (run starts counted in) takes about 12 + w
// us above and 20 + 1.5 w us there.  Measured here / there: 112 rows, 4 K/V heads,
// 2048 keys 16 / 22 us; 224 rows, 1024 keys 16 / 24 us, and 131072 keys, where
// the kernel above would read every page 14 times, 122 us there.  Tiles of 32
// and 64 rows there took 53 us for 16 blocks of 32, which is 54 above.
Plan plan(const fdllm_kv8& c, const fdllm_kv8_attention_args& a, int num_sms) {
  // rows of a sequence; without a hint those of an even batch, not all of them
  const int64_t most_q = a.max_q > 0 ? std::min(a.max_q, a.n_tokens)
                                     : ((int64_t)a.n_tokens + c.n_seqs - 1) / c.n_seqs;
  const int64_t rows = std::max<int64_t>(1, most_q * (a.n_heads / c.n_kv_heads));
  const int64_t table = (int64_t)c.max_pages * PAGE;
  const int64_t len = std::max<int64_t>(1, a.max_len > 0 ? std::min<int64_t>(a.max_len, table) : table);
  double pages = 0, share = 0;
  Plan p{};
  auto with = [&](int tile_rows, int ctas) {
    pages = (double)c.n_seqs * c.n_kv_heads * ((rows + tile_rows - 1) / tile_rows) *
            (RUN_START + (len + PAGE - 1) / PAGE);
    p.tile_rows = tile_rows;
    p.n_cta = (int)std::min(ctas * (double)num_sms, std::ceil(pages / MIN_PAGES));
    share = pages / p.n_cta;
  };
  with(R, 2);
  if (rows > 64 && a.dtype != FDLLM_DTYPE_F32 && c.head_dim >= 64) {
    const double mma = 12.0 + share;
    const int tile_rows = tc_tile_rows(rows);
    with(tile_rows, 1);
    if (mma < 20.0 + 1.5 * share) with(R, 2);
  }
  p.bytes = p.n_cta > 1 ? (size_t)p.n_cta * 2 * p.tile_rows * (c.head_dim + 2) * sizeof(float) : 0;
  return p;
}

template <typename T, int HD>
cudaError_t launch_attn_hd(const AttnP& P, cudaStream_t st) {
  constexpr bool two = std::is_same_v<T, float>;
  auto kern = kv8_attn_kernel<T, HD, two>;
  constexpr int smem = Lay<HD, two>::SMEM;
  static std::atomic<uint64_t> ready{0};   // devices whose limit is set
  cudaError_t e = allow_smem(kern, smem, ready);
  if (e == cudaSuccess) e = launch_k(false, kern, dim3(P.n_cta), dim3(AT_WARPS * 32), smem, st, P);
  if (e == cudaSuccess) e = launch_join<T, HD, R>(P, st);
  return e;
}

template <typename T>
cudaError_t launch_attn_t(const AttnP& P, cudaStream_t st) {
  switch (P.c.head_dim) {
    case 128: return launch_attn_hd<T, 128>(P, st);
    case 64: return launch_attn_hd<T, 64>(P, st);
    default: return launch_attn_hd<T, 32>(P, st);
  }
}

const char* check_args(const fdllm_kv8_attention_args* args, const fdllm_kv8& c) {
  if (!args) return "args is NULL";
  const fdllm_kv8_attention_args& a = *args;
  if (!kv8::elem_bytes(a.dtype)) return "unknown dtype";
  if (a.n_tokens < 0 || a.max_q < 0 || a.max_len < 0) return "n_tokens, max_q and max_len must be >= 0";
  if (a.n_heads < 1 || a.n_heads > 65535 || a.n_heads % c.n_kv_heads)
    return "n_heads must be a multiple of n_kv_heads in [1, 65535]";
  // rows are counted in 32 bits, up to a tile's end
  if ((int64_t)a.n_tokens * (a.n_heads / c.n_kv_heads) > 0x7fffff00) return "too many query rows";
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
  kv8::AttnP P{};
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
  if (a.out == a.q || (a.n_tokens > 1 && std::abs(a.out_strides[0]) < P.c.head_dim) ||
      (a.n_heads > 1 && std::abs(a.out_strides[1]) < P.c.head_dim))
    return kv8::fail(call, FDLLM_ERR_ARG, "out must not overlap q, nor its rows and heads one another");
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
    P.part_ml = reinterpret_cast<float2*>(P.part_o + (size_t)p.n_cta * 2 * p.tile_rows * P.c.head_dim);
  }
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  e = p.tile_rows != R                ? kv8::launch_attn_tc(P, p.tile_rows, st)
      : a.dtype == FDLLM_DTYPE_F32    ? launch_attn_t<float>(P, st)
      : a.dtype == FDLLM_DTYPE_BF16   ? launch_attn_t<__nv_bfloat16>(P, st)
                                      : launch_attn_t<__half>(P, st);
  if (e != cudaSuccess) return kv8::fail(call, FDLLM_ERR_CUDA, cudaGetErrorString(e));
  return FDLLM_OK;
}
