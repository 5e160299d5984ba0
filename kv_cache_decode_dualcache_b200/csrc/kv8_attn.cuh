// What the kernels of fdllm_kv8_attention share: how the work is shared out,
// number formats, rows in global memory.
//
// A query row is a (token, head-in-group) pair, so that the query heads of a
// K/V head share every cached byte.  A run is a tile of R rows, a K/V head
// and a sequence with all its pages.  The pages of all runs, laid end to end,
// are shared out evenly over the CTAs, whatever the lengths are; they are
// known on the device only, so every CTA sums them up for itself.  Starting a
// run costs a CTA about as much as RUN_START pages: a run is laid out that
// much longer, and a share boundary within its first RUN_START + 1 pages
// moves back to its start.  A run that a CTA does not hold whole leaves a
// partial result in the workspace (at most two a CTA: the end of one run,
// slot 0, and the start of another, slot 1), and a second kernel joins those.
// RUN_START 3 / 4 / 6 / 8: 64 sequences' tokens over up to 8192 keys 77 / 72 / 70
// / 70 us, one block of 32 over 2048 keys 19.7 / 19.3 / 19.8 / 19.8.
#pragma once

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "kv8.h"

namespace fd {
namespace kv8 {

constexpr int PAGE = FDLLM_KV8_PAGE;
constexpr int RUN_START = 6;
constexpr int MIN_PAGES = 2;         // of a share, at least (counting run starts)
constexpr float W_EXP = 8.0f;        // largest softmax weights are about 2^W_EXP
constexpr float M_SLACK = 7.0f;      // the reference moves when the max passes it by this
constexpr float LOG2E = 1.4426950408889634f;
constexpr float VS_MIN = 7.888609052210118e-31f;  // 2^-100: an all-zero block still counts in l

struct AttnP {
  fdllm_kv8 c;
  fdllm_kv8_attention_args a;
  int n_cta;         // shares (the grid)
  float* part_o;     // [share][2][R][head_dim]; NULL: runs are not split
  float2* part_ml;   // [share][2][R] (reference max, weight sum)
};

// A sequence's rows and runs.
struct Seq {
  int r_lo, rows, len, pages, tiles;   // rows: (token, head) pairs of a K/V head
  int span;                            // RUN_START + pages
  int64_t work;                        // spans of all its runs
};
FD_DEV Seq seq_of(const AttnP& P, int i, int tile_rows) {
  const fdllm_kv8_attention_args& a = P.a;
  Seq s;
  s.r_lo = min(max(a.starts[i], 0), a.n_tokens);
  const int r_hi = min(max(a.starts[i + 1], s.r_lo), a.n_tokens);
  s.rows = (r_hi - s.r_lo) * (a.n_heads / P.c.n_kv_heads);
  s.len = min(max(a.lens[i], 0), P.c.max_pages * PAGE);
  s.pages = (s.len + PAGE - 1) / PAGE;
  s.span = RUN_START + max(1, s.pages);   // a run without keys still writes its zeros
  s.tiles = (s.rows + tile_rows - 1) / tile_rows;
  s.work = (int64_t)s.tiles * P.c.n_kv_heads * s.span;
  return s;
}
// The work of sequences i0 + lane, summed up to each lane, by a warp.
FD_DEV int64_t scan_work(const AttnP& P, int tile_rows, int i0, int64_t* own) {
  const int lane = threadIdx.x & 31;
  int64_t w = i0 + lane < P.c.n_seqs ? seq_of(P, i0 + lane, tile_rows).work : 0;
  *own = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  return w;
}
// All sequences' work; the first 32 sequences' scan stays in upto, own.
FD_DEV int64_t total_work(const AttnP& P, int tile_rows, int64_t* upto, int64_t* own) {
  *upto = scan_work(P, tile_rows, 0, own);
  int64_t t = __shfl_sync(0xffffffffu, *upto, 31);
  for (int i0 = 32; i0 < P.c.n_seqs; i0 += 32) {
    int64_t w;
    t += __shfl_sync(0xffffffffu, scan_work(P, tile_rows, i0, &w), 31);
  }
  return t;
}
// The sequence that holds position x < total, by a warp; *off: the place
// within it.  upto, own: from total_work.
FD_DEV int find_seq(const AttnP& P, int tile_rows, int64_t x, int64_t upto, int64_t own, int64_t* off) {
  int64_t base = 0;
  for (int i0 = 0;;) {
    const uint32_t hit = __ballot_sync(0xffffffffu, base + upto > x);
    if (hit || i0 + 32 >= P.c.n_seqs) {
      const int l = hit ? __ffs(hit) - 1 : 0;
      *off = x - base - __shfl_sync(0xffffffffu, upto - own, l);
      return i0 + l;
    }
    base += __shfl_sync(0xffffffffu, upto, 31);
    upto = scan_work(P, tile_rows, i0 += 32, &own);
  }
}
// Division of what nearly always fits 32 bits.
FD_DEV int64_t div64(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// Shares in use, and where share i begins.
struct Shares {
  int64_t n, each, rest;
  FD_DEV int64_t begin(int64_t i) const { return each * i + min(i, rest); }
};
FD_DEV Shares shares_of(const AttnP& P, int64_t total) {
  Shares s;
  s.n = max((int64_t)1, min((int64_t)P.n_cta, total / MIN_PAGES));
  s.each = div64(total, s.n);
  s.rest = total - s.each * s.n;
  return s;
}

// One CTA's part of a run: pages [p_lo, p_hi) of sequence seq, whose rows
// start at token r_lo.
struct Segment {
  int seq, g, row0, p_lo, p_hi, r_lo, rows, len;
  bool whole;
};
// Walks a share: in shared memory, one for each warp that needs the segments
// (its state would cost the loops' registers).
struct Walk {
  int64_t x, x_end, off;
  int seq;
  Seq sq;
  Segment sg;
};
// By a warp, with start and next.
FD_DEV void walk_start(Walk* w, const AttnP& P, int tile_rows) {
  int64_t upto, own, x = 0, x_end = 0, off = 0;
  const int64_t total = total_work(P, tile_rows, &upto, &own);
  const Shares sh = shares_of(P, total);
  int seq = 0;
  Seq sq{};
  if (blockIdx.x < sh.n) {
    x = sh.begin(blockIdx.x);
    x_end = sh.begin(blockIdx.x + 1);
  }
  if (x < x_end) {
    seq = find_seq(P, tile_rows, x, upto, own, &off);
    sq = seq_of(P, seq, tile_rows);
    const int p = (int)(off - div64(off, sq.span) * sq.span);
    if (!P.part_o && p > 0) {   // whole runs: those that start in the share
      x += sq.span - p;
      off += sq.span - p;
    } else if (p <= RUN_START) {
      x -= p;
      off -= p;
    }
  }
  if ((threadIdx.x & 31) == 0) {
    w->x = x;
    w->x_end = x_end;
    w->off = off;
    w->seq = seq;
    w->sq = sq;
  }
  __syncwarp();
}
// The next segment, or false at the share's end.
FD_DEV bool walk_next(Walk* w, const AttnP& P, int tile_rows, Segment* s) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    int64_t x = w->x, off = w->off;
    Seq sq = w->sq;
    Segment n{};
    n.seq = -1;
    if (x < w->x_end) {
      while (off >= sq.work) {
        off -= sq.work;
        sq = seq_of(P, ++w->seq, tile_rows);
      }
      const int run = (int)div64(off, sq.span), p = (int)(off - (int64_t)run * sq.span);
      int q = sq.span;
      if (P.part_o && w->x_end - x < sq.span - p) q = p + (int)(w->x_end - x);
      x += q - p;
      off += q - p;
      if (q > RUN_START) {   // else the next share takes the run from its start
        n.seq = w->seq;
        n.g = run / sq.tiles;
        n.row0 = run % sq.tiles * tile_rows;
        n.p_lo = max(0, p - RUN_START);
        n.p_hi = min(sq.pages, q - RUN_START);
        n.r_lo = sq.r_lo;
        n.rows = sq.rows;
        n.len = sq.len;
        n.whole = p == 0 && q == sq.span;
      }
    }
    w->x = x;
    w->off = off;
    w->sq = sq;
    w->sg = n;
  }
  __syncwarp();
  *s = w->sg;
  return s->seq >= 0;
}

FD_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Whether a row's reference M moves to its new maximum mx (M = -inf: to any that
// is above).  The difference of two near numbers is exact; M + slack would round
// up from 2^24 on.
FD_DEV bool passes(float mx, float M, float slack) { return mx - M > slack; }
// What is added to t to give a weight's exponent, at most W_EXP + M_SLACK.
// Rounded down, for where 16 lies between the numbers around M (2^27), half of
// the sums W_EXP - M would round up by 8.
FD_DEV float weight_ref(float M) { return __fadd_rd(W_EXP, M == -INFINITY ? 0.0f : -M); }
// Two of the four offset-binary bytes of x (selector) as exact fp16 codes:
// the byte under the exponent of 1024, minus 1024 + 128.
template <uint32_t SEL> FD_DEV uint32_t codes_h2(uint32_t x) {
  const uint32_t u = __byte_perm(x, 0x64646464u, SEL);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __float2half2_rn(1152.0f));
  return *reinterpret_cast<const uint32_t*>(&h);
}
FD_DEV uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^up brings a row's largest |q| into [2^8, 2^9) (0 and non-finite: as it is).
FD_DEV int q_shift(float top) {
  const int e = (int)((__float_as_uint(top) >> 23) & 255);
  return e == 0 || e == 255 ? 0 : min(135 - e, 120);
}
FD_DEV float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

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

// Block 0 reports lengths and starts out of range.
FD_DEV void report_range(const AttnP& P) {
  if (blockIdx.x == 0 && P.a.status)
    for (int i = threadIdx.x; i < P.c.n_seqs; i += blockDim.x)
      if (P.a.lens[i] < 0 || P.a.lens[i] > P.c.max_pages * PAGE || !starts_ok(P.a.starts, i, P.a.n_tokens))
        atomicOr(P.a.status, FDLLM_KV8_BAD_RANGE);
}

// Joins the partial results of the run around the start of share blockIdx.x +
// 1, if that is the first share start inside it: slot 1 of the share before
// (the run's start), and slot 0 of the shares that follow.  A warp per row,
// lanes over the dims.
constexpr int JOIN_WARPS = 4;
template <typename T, int HD, int R>
__global__ void __launch_bounds__(JOIN_WARPS * 32) kv8_join_kernel(const AttnP P) {
  const fdllm_kv8_attention_args& a = P.a;
  const int lane = threadIdx.x & 31;
  int64_t upto, own;
  const Shares sh = shares_of(P, total_work(P, R, &upto, &own));
  const int64_t c = blockIdx.x + 1;
  bool mine = c < sh.n;
  int64_t off = 0;
  const int64_t x = mine ? sh.begin(c) : 0;
  const int seq = mine ? find_seq(P, R, x, upto, own, &off) : 0;
  const Seq sq = seq_of(P, seq, R);
  const int run = (int)div64(off, sq.span), p = (int)(off - (int64_t)run * sq.span);
  mine = mine && p > RUN_START && sh.begin(c - 1) <= x - p + RUN_START;
  int n = 1;   // pieces
  if (mine)
    while (c + n - 1 < sh.n && sh.begin(c + n - 1) < x - p + sq.span) ++n;
  const int rep = a.n_heads / P.c.n_kv_heads, g = mine ? run / sq.tiles : 0;
  const int r = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5);
  const int rr = mine ? run % sq.tiles * R + r : 0;
  pdl_wait();   // by every block: this grid must not end before the one that feeds it
  if (!mine || rr >= sq.rows) return;
  auto piece = [&](int i) { return ((c - 1 + i) * 2 + (i == 0)) * R + r; };
  // a lane holds the (max, sum) of one of 32 pieces, and V consecutive dims
  constexpr int V = HD / 32;
  float mx = -INFINITY;
  for (int i = lane; i < n; i += 32) mx = fmaxf(mx, P.part_ml[piece(i)].x);
  mx = warp_max(mx);
  float sum = 0.0f, acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.0f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float f = 0.0f;
    if (i0 + lane < n) {
      const float2 ml = P.part_ml[piece(i0 + lane)];
      f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - mx);
      sum = fmaf(ml.y, f, sum);
    }
    const int m = min(32, n - i0);
#pragma unroll 1
    for (int i = 0; i < m; i += 8) {   // 8 loads in flight
      float x[8][V];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (i + k >= m) break;
        const float* po = P.part_o + piece(i0 + i + k) * HD + lane * V;
        if constexpr (V == 4) {
          load4(po, x[k]);
        } else if constexpr (V == 2) {
          const float2 u = *reinterpret_cast<const float2*>(po);
          x[k][0] = u.x;
          x[k][1] = u.y;
        } else {
          x[k][0] = *po;
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (i + k >= m) break;
        const float w = __shfl_sync(0xffffffffu, f, i + k);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = fmaf(x[k][j], w, acc[j]);
      }
    }
  }
  sum = warp_sum(sum);
  const float inv = mx == -INFINITY ? 0.0f : 1.0f / sum;
  T* dst = reinterpret_cast<T*>(a.out) + (int64_t)(sq.r_lo + rr / rep) * a.out_strides[0] +
           (int64_t)(g * rep + rr % rep) * a.out_strides[1] + lane * V;
  if constexpr (V == 4) {
    store4(dst, acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) dst[j] = from_f<T>(acc[j] * inv);
  }
}

template <typename T, int HD, int R>
cudaError_t launch_join(const AttnP& P, cudaStream_t st) {
  if (!P.part_o) return cudaSuccess;
  return launch_k(true, kv8_join_kernel<T, HD, R>, dim3(P.n_cta - 1, R / JOIN_WARPS),
                  dim3(JOIN_WARPS * 32), 0, st, P);
}

// The kernel for more than 64 rows (kv8_attn_tc.cu): rows of its tile for
// runs of at most `rows` rows, and the launch with its join.
int tc_tile_rows(int64_t rows);
cudaError_t launch_attn_tc(const AttnP& P, int tile_rows, cudaStream_t st);

}  // namespace kv8
}  // namespace fd
