// fdllm_kv8_attention for more than 16 query rows a K/V head (diffusion
// blocks, grouped heads, chunks of a prompt) with 16-bit q: both products on
// the 5th-generation tensor cores, the codes converted to fp16 tiles once per
// CTA for all of its rows.
//
// The CTA's MMA tile has NQ x 128 rows.  Tiles of up to 32 (64) query rows
// fill 128 rows with 4 (2) copies: copy i of a row takes columns [128 / C i,
// 128 / C (i + 1)) of every 128-key tile, with statistics of its own, and
// leaves zero weights in the others' columns, so that the softmax runs on all
// four warps and the copies' outputs add up at the end.  The idle part of
// the MMAs costs nothing: with so few rows the kernel waits for the cache.
//
// Roles: 4 warps a row tile for the softmax (a thread per MMA row: q, weights,
// output; the first one's lane 0 issues the tile's MMAs), 4 converter warps (K
// and V codes from global memory through registers into 128-byte-swizzled
// fp16 tiles, the blocks' scales beside them).  Per tile of 128 keys:
//   S = Q K^T        tcgen05, Q and K in shared memory, S in TMEM
//   w = 2^(S f + log2 vs - M + 8), written over S as packed fp16
//   O += w V         tcgen05, w from TMEM, V MN-major from shared memory
// with the statistics of kv8_attn.cu.  A tile's w V and the next tile's S are
// issued together; with two row tiles (NQ = 2) one tile's softmax runs behind
// the other's products, with one two CTAs share an SM and hide each other's.
//
// Every wait is bounded (WAIT_LIMIT_NS); a role whose wait ran out keeps
// walking its loops without waiting or touching TMEM, so that all barriers
// are still met, and FDLLM_KV8_TIMEOUT is reported.
#include <algorithm>

#include "kv8_attn.cuh"

namespace fd {
namespace {

using namespace kv8;

constexpr int KEYS = 128;            // keys of a tile: two pages
constexpr int NB = KEYS / FDLLM_KV8_BLOCK;
constexpr int CONV = 128;            // converter threads

template <int HD, int NQ>
struct TcLay {
  static constexpr int KH = HD / 64;                  // 64-dim sub-tiles (128-byte rows)
  static constexpr int SUB = KEYS * 128;              // [128 rows][64 dims] fp16
  static constexpr int MAT = KH * SUB;                // K, V or 128 rows of Q
  static constexpr int STAGES = NQ;
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = K_OFF + STAGES * MAT;
  static constexpr int Q_OFF = V_OFF + STAGES * MAT;
  // scales of a tile, by its parity: ks, log2 vs, 1 / vs of 8 blocks
  static constexpr int SC_OFF = Q_OFF + NQ * MAT;
  static constexpr int ML_OFF = SC_OFF + 2 * 3 * NB * 4;   // copies' (max, sum) [128]
  static constexpr int RF_OFF = ML_OFF + 128 * 8;          // row factors
  static constexpr int BAR_OFF = RF_OFF + NQ * 128 * 4;
  static constexpr int MISC_OFF = BAR_OFF + 32 * 8;
  static constexpr int SMEM = MISC_OFF + 16 + 1024;   // slack for 1024-byte alignment
  static constexpr int THREADS = 128 * NQ + CONV;
  static constexpr uint32_t TMEM_COLS = 256 * NQ;     // S: 128, O: 128 columns a row tile
  static_assert(SMEM <= (NQ == 1 ? 115712 : 232448), "shared memory layout");
};

// D (+)= A B with A in TMEM (row i in lane i, two fp16 a column).
FD_DEV void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                      uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// (a, b) = (a, b) * f + g, one instruction.
FD_DEV void fma2(float& a, float& b, float f, float g) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(f), "f"(g));
}
// 16 TMEM columns of this warp's lanes.
FD_DEV void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
FD_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <typename T, int HD, int NQ, int C>
__global__ void __launch_bounds__(TcLay<HD, NQ>::THREADS, NQ == 1 ? 2 : 1)
    kv8_attn_tc_kernel(const AttnP P) {
  using L = TcLay<HD, NQ>;
  constexpr int R = NQ * 128 / C;      // query rows of a run
  constexpr int NC = KEYS / C;         // key columns of a thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  uint64_t* k_full = bars;             // [STAGES]
  uint64_t* k_free = bars + 2;
  uint64_t* v_full = bars + 4;
  uint64_t* v_free = bars + 6;
  uint64_t* s_full = bars + 8;         // [NQ]
  uint64_t* o_full = bars + 10;        // [NQ]
  uint64_t* sc_full = bars + 12;       // [2]: by tile parity
  uint64_t* sc_free = bars + 14;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
  int* err = reinterpret_cast<int*>(misc + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 2);
  const fdllm_kv8& c = P.c;
  const fdllm_kv8_attention_args& a = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rep = a.n_heads / c.n_kv_heads;

  pdl_trigger();   // the join may be set up; it waits for this grid's end
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], CONV);
      mbar_init(&k_free[i], NQ);
      mbar_init(&v_full[i], CONV);
      mbar_init(&v_free[i], NQ);
      mbar_init(&s_full[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&sc_full[i], NB);
      mbar_init(&sc_free[i], 128 * NQ);
    }
    *err = 0;
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(misc, L::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  report_lengths(P);
  Walk walk;
  walk.start(P, R);
  Segment sg;
  bool ok = true;
  // a warp's wait: all lanes agree
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, err, abort_flag)) != 0;
    return ok;
  };

  if (warp < 4 * NQ) {
    // ================================================== softmax
    const int q = warp >> 2, quad = warp & 3, i = quad * 32 + lane;   // MMA row of tile q
    const int r = q * 128 + i % R, copy = NQ == 1 ? i / R : 0;        // row of the run, its copy
    const uint32_t s_col = tmem + ((uint32_t)(quad * 32) << 16) + q * 128;
    const uint32_t o_col = s_col + NQ * 128;
    uint8_t* qs = smem + L::Q_OFF + q * L::MAT;
    float2* ml = reinterpret_cast<float2*>(smem + L::ML_OFF);
    float* rfs = reinterpret_cast<float*>(smem + L::RF_OFF);
    const uint32_t kb = smem_u32(smem + L::K_OFF), vb = smem_u32(smem + L::V_OFF), qb = smem_u32(qs);
    // the MMAs of this row tile, by warp 0 of its four: S of tile n; w V of tile n
    auto scores = [&](int n) {
      const int st = n % L::STAGES;
      wait(&k_full[st], (n / L::STAGES) & 1);
      if (ok && lane == 0) {
        tc_fence_after();
        // a step along K moves the descriptors' start address (in 16 bytes)
        const uint64_t qd = smem_desc_sw128(qb), kd = smem_desc_sw128(kb + st * L::MAT);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t off = ((k >> 2) * L::SUB + (k & 3) * 32) >> 4;
          tc_mma(tmem + q * 128, qd + off, kd + off, idesc_f32acc(KEYS, true), k > 0);
        }
        tc_commit(&s_full[q]);
        tc_commit(&k_free[st]);
      }
      __syncwarp();
    };
    auto products = [&](int n, bool first, bool last) {
      const int st = n % L::STAGES;
      wait(&v_full[st], (n / L::STAGES) & 1);
      if (ok && lane == 0) {
        tc_fence_after();
        const uint64_t vd = smem_desc_sw128_mn(vb + st * L::MAT, L::SUB, 1024);
#pragma unroll
        for (int k = 0; k < KEYS / 16; ++k)
          tc_mma_ts(tmem + (NQ + q) * 128, tmem + q * 128 + k * 8, vd + (k * 2048 >> 4),
                    idesc_f32acc_bmn(HD, true), !first || k > 0);
        tc_commit(&v_free[st]);
        if (last) tc_commit(&o_full[q]);
      }
      __syncwarp();
    };
    int n_tile = 0, n_seg = 0;
    while (walk.next(P, &sg)) {
      const int rows = walk.sq.rows, rr = sg.row0 + r;
      const int k_lo = sg.p_lo * PAGE, k_hi = min(walk.sq.len, sg.p_hi * PAGE);
      const int tiles = (k_hi - k_lo + KEYS - 1) / KEYS;
      // ---- q, scaled per row by a power of two, into the swizzled A tile: HD / 8
      // lanes a row, 16 bytes each; every warp a quarter of the rows, all copies
      {
        constexpr int LR = HD / 8, RPW = 128 / C / 4, STEP = 32 / LR, N = RPW / STEP;
        const int ch = lane % LR, row_a = quad * RPW + lane / LR;   // row of the MMA tile
        const int first = sg.row0 + q * 128 + row_a;
        int token = first / rep, head = first % rep;
        uint4 raw[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          raw[j] = make_uint4(0, 0, 0, 0);
          if (first + j * STEP < rows)
            raw[j] = *reinterpret_cast<const uint4*>(
                reinterpret_cast<const T*>(a.q) + (int64_t)(walk.sq.r_lo + token) * a.q_strides[0] +
                (int64_t)(sg.g * rep + head) * a.q_strides[1] + ch * 8);
          for (head += STEP; head >= rep; head -= rep) ++token;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const T* e = reinterpret_cast<const T*>(&raw[j]);
          float top = 0.0f;
#pragma unroll
          for (int m = 0; m < 8; ++m) top = fmaxf(top, fabsf(to_f<T>(e[m])));
#pragma unroll
          for (int o = LR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const int up = q_shift(top), row = row_a + j * STEP;
          const float mul = exp2_int(up);
          uint32_t h[4];
#pragma unroll
          for (int m = 0; m < 4; ++m)
            h[m] = pack_h2(to_f<T>(e[2 * m]) * mul, to_f<T>(e[2 * m + 1]) * mul);
#pragma unroll
          for (int k = 0; k < C; ++k) {
            const int at = k * (128 / C) + row;
            *reinterpret_cast<uint4*>(qs + (ch >> 3) * L::SUB + at * 128 + (((ch & 7) ^ (at & 7)) << 4)) =
                make_uint4(h[0], h[1], h[2], h[3]);
          }
          if (ch == 0) rfs[q * 128 + row] = a.scale * LOG2E * exp2_int(-up);
        }
        fence_proxy_async_smem();
        named_bar(1 + q, 128);
        if (quad == 0 && tiles > 0) scores(n_tile);
      }
      const float rf = rfs[r];
      float M = -INFINITY, l = 0.0f;
      for (int t = 0; t < tiles; ++t, ++n_tile) {
        const int k0 = k_lo + t * KEYS + copy * NC;   // first key of this thread's columns
        const float* sc = reinterpret_cast<const float*>(smem + L::SC_OFF) + (n_tile & 1) * 3 * NB +
                          copy * (NC / 16);
        wait(&s_full[q], n_tile & 1);
        wait(&sc_full[n_tile & 1], (n_tile >> 1) & 1);
        if (ok) {
          tc_fence_after();
          const bool tail = k0 + NC > k_hi;
          const uint32_t col = s_col + copy * NC;
          float v[32], mx = -INFINITY;
          // t of 32 columns from c0 on, shifted by add; columns behind the run's
          // last key are -inf
          auto read = [&](int c0, float add) {
            tmem_ld32(col + c0, v);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float f = rf * sc[c0 / 16 + b], g = sc[NB + c0 / 16 + b] + add;
#pragma unroll
              for (int j = 16 * b; j < 16 * b + 16; j += 2) fma2(v[j], v[j + 1], f, g);
            }
            if (tail) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (k0 + c0 + j >= k_hi) v[j] = -INFINITY;
            }
          };
#pragma unroll
          for (int c0 = 0; c0 < NC; c0 += 32) {
            read(c0, 0.0f);
#pragma unroll
            for (int j = 0; j < 32; j += 2) mx = fmaxf(fmaxf(mx, v[j]), v[j + 1]);
          }
          float alpha = 1.0f;
          const bool move = mx > M + M_SLACK || (M == -INFINITY && mx > -INFINITY);
          if (move) {
            alpha = ex2(M - mx);
            M = mx;
          }
          const float ref = W_EXP - (M == -INFINITY ? 0.0f : M);
          float sum = 0.0f;
#pragma unroll
          for (int c0 = 0; c0 < NC; c0 += 32) {
            uint32_t w[16];
            if (NC > 32) {   // the registers hold one chunk only: read the scores again
              read(c0, ref);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] += ref;
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              float part = 0.0f;
#pragma unroll
              for (int j = 16 * b; j < 16 * b + 16; j += 2) {
                const float e0 = ex2(v[j]), e1 = ex2(v[j + 1]);
                part += e0 + e1;
                w[j / 2] = pack_h2(e0, e1);
              }
              sum = fmaf(part, sc[2 * NB + c0 / 16 + b], sum);
            }
            // w goes over the scores' first 64 columns, which chunks c0 / 2
            // and below of this row have been read by now
            tmem_st16(s_col + (copy * NC + c0) / 2, w);
          }
          if constexpr (C > 1) {
            const uint32_t zero[16] = {};
#pragma unroll
            for (int o = 0; o < 64; o += 16)
              if (o / (NC / 2) != copy) tmem_st16(s_col + o, zero);
          }
          l = fmaf(l, alpha, sum);
          if (t > 0 && __any_sync(0xffffffffu, move)) {
            // S of this tile came after the products before it: O is still
#pragma unroll
            for (int c0 = 0; c0 < HD; c0 += 32) {
              tmem_ld32(o_col + c0, v);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] *= alpha;
              tmem_st32(o_col + c0, v);
            }
          }
          tmem_wait_st();
          tc_fence_before();
        }
        mbar_arrive(&sc_free[n_tile & 1]);
        named_bar(1 + q, 128);   // the tile's weights are written, O is rescaled
        if (quad == 0) {
          products(n_tile, t == 0, t + 1 == tiles);
          if (t + 1 < tiles) scores(n_tile + 1);
        }
      }
      // ---- the run's output, or its part
      const bool have_o = tiles > 0 && wait(&o_full[q], n_seg & 1);
      tc_fence_after();
      if (tiles > 0) ++n_seg;
      const int64_t slot = ((int64_t)blockIdx.x * 2 + (sg.p_lo == 0)) * R;
      auto emit = [&](int row, int d, const float* x, float inv) {   // 8 dims of a row
        const int rw = sg.row0 + row;
        if (rw >= rows) return;
        if (!sg.whole) {
          float* dst = P.part_o + (slot + row) * HD + d;
          *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<float4*>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
        } else {
          T* dst = reinterpret_cast<T*>(a.out) + (int64_t)(walk.sq.r_lo + rw / rep) * a.out_strides[0] +
                   (int64_t)(sg.g * rep + rw % rep) * a.out_strides[1] + d;
          uint4 u;
          T* e = reinterpret_cast<T*>(&u);
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = from_f<T>(x[j] * inv);
          *reinterpret_cast<uint4*>(dst) = u;
        }
      };
      if constexpr (C == 1) {
        const float inv = M == -INFINITY ? 0.0f : 1.0f / l;
        if (!sg.whole && rr < rows) P.part_ml[slot + r] = make_float2(M, l);
#pragma unroll
        for (int c0 = 0; c0 < HD; c0 += 32) {
          float v[32];
          if (have_o) tmem_ld32(o_col + c0, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = have_o ? v[j] : 0.0f;
#pragma unroll
          for (int j = 0; j < 32; j += 8) emit(r, c0 + j, v + j, inv);
        }
      } else {
        // the copies of a row add up, scaled to their common reference, DIMS
        // dims at a time through the area of Q (no product reads it any more)
        constexpr int DIMS = HD / 4, XROW = DIMS + 4;
        static_assert(128 * XROW * 4 <= L::MAT, "the exchange exceeds the Q area");
        float* xo = reinterpret_cast<float*>(qs);
        ml[i] = make_float2(M, l);
        named_bar(1, 128);
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < C; ++k) mx = fmaxf(mx, ml[k * R + r].x);
        const float fac = M == -INFINITY ? 0.0f : ex2(M - mx);
        // this thread adds up 8 dims of row orow
        constexpr int PER = 128 / R;                 // threads a row
        const int orow = i / PER;
        float omx = -INFINITY, osum = 0.0f;
#pragma unroll
        for (int k = 0; k < C; ++k) omx = fmaxf(omx, ml[k * R + orow].x);
#pragma unroll
        for (int k = 0; k < C; ++k) {
          const float2 m = ml[k * R + orow];
          osum += m.x == -INFINITY ? 0.0f : m.y * ex2(m.x - omx);
        }
        const float inv = omx == -INFINITY ? 0.0f : 1.0f / osum;
        if (!sg.whole && i % PER == 0 && sg.row0 + orow < rows)
          P.part_ml[slot + orow] = make_float2(omx, osum);
#pragma unroll
        for (int c0 = 0; c0 < HD; c0 += 32) {
          float v[32];
          if (have_o) tmem_ld32(o_col + c0, v);
#pragma unroll
          for (int s0 = 0; s0 < 32; s0 += DIMS) {
#pragma unroll
            for (int j = 0; j < DIMS; j += 4)
              *reinterpret_cast<float4*>(xo + i * XROW + j) =
                  have_o ? make_float4(v[s0 + j] * fac, v[s0 + j + 1] * fac, v[s0 + j + 2] * fac,
                                       v[s0 + j + 3] * fac)
                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            named_bar(1, 128);
            for (int d = i % PER * 8; d < DIMS; d += PER * 8) {
              float x[8] = {};
#pragma unroll
              for (int k = 0; k < C; ++k)
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                  const float4 u = *reinterpret_cast<const float4*>(xo + (k * R + orow) * XROW + d + j);
                  x[j] += u.x;
                  x[j + 1] += u.y;
                  x[j + 2] += u.z;
                  x[j + 3] += u.w;
                }
              emit(orow, c0 + s0 + d, x, inv);
            }
            named_bar(1, 128);
          }
        }
      }
      tc_fence_before();   // O has been read before the next run's first product
    }
  } else {
    // ================================================== converters
    const int ct = tid - 128 * NQ;
    constexpr int HALVES = HD / 64;            // 64-byte halves of a key
    constexpr int PER = KEYS / 32 * HALVES;    // 16-byte chunks of a thread
    // 4 lanes take 64 bytes of a key: the 8 lanes of a store then have an
    // even and an odd row, whose swizzled chunks are on different banks
    const int row0 = ct >> 2, ch = ct & 3;
    int n_tile = 0;
    while (walk.next(P, &sg)) {
      const int32_t* table = c.page_table + (int64_t)sg.seq * c.table_stride;
      const int k_lo = sg.p_lo * PAGE, k_hi = min(walk.sq.len, sg.p_hi * PAGE);
      const int tiles = (k_hi - k_lo + KEYS - 1) / KEYS;
      uint4 kr[PER], vr[PER];
      float ks = 0.0f, vs = -1.0f;             // scales of block ct (vs < 0: no key)
      int page0 = -1, page1 = -1, next0 = -1, next1 = -1;
      // page id of key k, as the table has it; -1 behind the run's end
      auto page_at = [&](int k) { return k < k_hi ? table[k / PAGE] : -1; };
      auto next_pages = [&](int t) {   // of tile t, from the ids asked for one tile before
        page0 = next0;
        page1 = next1;
        const int k = k_lo + t * KEYS;
        if (k < k_hi && (page0 < 0 || page0 >= c.n_pages || (k + PAGE < k_hi && (page1 < 0 || page1 >= c.n_pages)))) {
          if (ct == 0 && a.status) atomicOr(a.status, FDLLM_KV8_BAD_PAGE);
        }
        if (page0 >= c.n_pages) page0 = -1;
        if (page1 >= c.n_pages) page1 = -1;
        next0 = page_at(k + KEYS);
        next1 = page_at(k + KEYS + PAGE);
      };
      auto load = [&](const int8_t* pool, uint4* x) {
        const int8_t* base = pool + ((int64_t)sg.g * PAGE + row0) * HD + ch * 16;
        const int8_t* p0 = base + (int64_t)page0 * c.page_stride;
        const int8_t* p1 = base + (int64_t)page1 * c.page_stride;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int rg = j / HALVES, h = j % HALVES;   // rows 32 rg + row0
          const bool have = (rg < 2 ? page0 : page1) >= 0;
          x[j] = make_uint4(0, 0, 0, 0);
          if (have)
            x[j] = __ldg(reinterpret_cast<const uint4*>((rg < 2 ? p0 : p1) + (rg & 1) * 32 * HD + h * 64));
        }
      };
      auto load_scales = [&](int t) {
        if (ct < NB) {
          const int pg = ct < NB / 2 ? page0 : page1;
          ks = 0.0f;
          vs = -1.0f;
          if (pg >= 0 && k_lo + t * KEYS + ct * 16 < k_hi) {
            const int64_t so = (int64_t)pg * c.scale_stride + sg.g * 4 + ct % 4;
            ks = c.k_scale[so];
            vs = fmaxf(c.v_scale[so], 0.0f);
          }
        }
      };
      auto put = [&](uint8_t* mat, const uint4* x) {   // 16 codes: two 16-byte chunks
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int row = j / HALVES * 32 + row0;
          const uint32_t u[4] = {x[j].x ^ 0x80808080u, x[j].y ^ 0x80808080u, x[j].z ^ 0x80808080u,
                                 x[j].w ^ 0x80808080u};
          uint32_t h[8];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            h[2 * m] = codes_h2<0x4140>(u[m]);
            h[2 * m + 1] = codes_h2<0x4342>(u[m]);
          }
          uint8_t* dst = mat + j % HALVES * L::SUB + row * 128;
          *reinterpret_cast<uint4*>(dst + ((2 * ch ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(dst + (((2 * ch + 1) ^ (row & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
      };
      if (tiles > 0) {
        next0 = page_at(k_lo);
        next1 = page_at(k_lo + PAGE);
        next_pages(0);
        load(c.k, kr);
        load_scales(0);
        load(c.v, vr);
      }
      for (int t = 0; t < tiles; ++t, ++n_tile) {
        const int st = n_tile % L::STAGES, use = n_tile / L::STAGES;
        if (use > 0) wait(&k_free[st], (use - 1) & 1);
        put(smem + L::K_OFF + st * L::MAT, kr);
        fence_proxy_async_smem();
        mbar_arrive(&k_full[st]);
        if (n_tile >= 2) wait(&sc_free[n_tile & 1], (n_tile / 2 - 1) & 1);
        if (ct < NB) {
          float* sc = reinterpret_cast<float*>(smem + L::SC_OFF) + (n_tile & 1) * 3 * NB + ct;
          const float v = fmaxf(vs, VS_MIN);
          sc[0] = ks;
          sc[NB] = vs < 0.0f ? -INFINITY : __log2f(v);
          sc[2 * NB] = vs < 0.0f ? 0.0f : __fdividef(1.0f, v);
          mbar_arrive(&sc_full[n_tile & 1]);
        }
        // the next tile's loads; V's registers hold this one's until it is stored
        if (t + 1 < tiles) {
          next_pages(t + 1);
          load(c.k, kr);
          load_scales(t + 1);
        }
        if (use > 0) wait(&v_free[st], (use - 1) & 1);
        put(smem + L::V_OFF + st * L::MAT, vr);
        fence_proxy_async_smem();
        mbar_arrive(&v_full[st]);
        if (t + 1 < tiles) load(c.v, vr);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, L::TMEM_COLS);
  if (tid == 0 && *err && a.status) atomicOr(a.status, FDLLM_KV8_TIMEOUT);
}

template <typename T, int HD, int NQ, int C>
cudaError_t launch_tc(const AttnP& P, cudaStream_t st) {
  using L = TcLay<HD, NQ>;
  auto kern = kv8_attn_tc_kernel<T, HD, NQ, C>;
  static std::atomic<uint64_t> ready{0};   // devices whose limit is set
  cudaError_t e = allow_smem(kern, L::SMEM, ready);
  if (e == cudaSuccess) e = launch_k(false, kern, dim3(P.n_cta), dim3(L::THREADS), L::SMEM, st, P);
  if (e == cudaSuccess) e = launch_join<T, HD, NQ * 128 / C>(P, st);
  return e;
}

template <typename T, int HD>
cudaError_t launch_tc_hd(const AttnP& P, int rows, cudaStream_t st) {
  switch (rows) {
    case 32: return launch_tc<T, HD, 1, 4>(P, st);
    case 64: return launch_tc<T, HD, 1, 2>(P, st);
    case 128: return launch_tc<T, HD, 1, 1>(P, st);
    default: return launch_tc<T, HD, 2, 1>(P, st);
  }
}

}  // namespace

namespace kv8 {

int tc_tile_rows(int64_t rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256; }
int tc_ctas_per_sm(int tile_rows) { return tile_rows == 256 ? 1 : 2; }

cudaError_t launch_attn_tc(const AttnP& P, int rows, cudaStream_t st) {
  if (P.a.dtype == FDLLM_DTYPE_BF16)
    return P.c.head_dim == 128 ? launch_tc_hd<__nv_bfloat16, 128>(P, rows, st)
                               : launch_tc_hd<__nv_bfloat16, 64>(P, rows, st);
  return P.c.head_dim == 128 ? launch_tc_hd<__half, 128>(P, rows, st)
                             : launch_tc_hd<__half, 64>(P, rows, st);
}

}  // namespace kv8
}  // namespace fd
