// fdllm_kv8_attention for more than 64 query rows a K/V head (blocks of grouped
// heads, chunks of a prompt) with 16-bit q: both products on the 5th-generation
// tensor cores, the codes converted to fp16 tiles once per CTA for all of its
// rows.  The CTA's MMA tile has NQ x 128 rows.
//
// Roles: 4 warps a row tile for the softmax (a thread per MMA row: q, weights,
// output), 2 converter warps for K and 2 for V, one copy warp, an MMA warp a
// row tile.  A page is a tile:
// its codes of K (and V) of a head are contiguous and come by one bulk copy
// each into a ring of int8 units; the converters turn them into
// 128-byte-swizzled fp16 tiles, and the copy warp fetches the blocks' scales.
//   S = Q K^T        tcgen05, Q and K in shared memory, S in TMEM (two buffers)
//   w = 2^(S f + log2 vs - M + 8), written over S as packed fp16
//   O += w V         tcgen05, w in TMEM, V MN-major from shared memory
// with the statistics of kv8_attn.cu.  S of tile t + 1 is done before the softmax
// of tile t is, so that the chain from tile to tile is the softmax alone.
// What shaped this: with shared memory in use there is next to no L1, so
// loads through registers and spilled registers both starve (loads in flight
// need L1 lines, spills go to L2); hence the bulk copies, and 64-key tiles,
// whose scores fit a thread's registers.
//
// Bound: 224 rows (32 tokens, 28 heads on 4) over 131072 keys take 122 us, 493
// TF/s: 1.4 us for a tile's 64 keys, of which its products are 0.73 at the rate of
// a large library product (the tensor pipe is active for 33% of the cycles); the
// rest is the softmax's chain (scores out of TMEM, weights back, barriers).
//
// Orderings.  Who waits for whom (n: the CTA's running tile, a barrier's phase
// is the n-th use of its slot, and none can be two phases ahead of a waiter):
//   unit_full   codes of n have landed            -> converter reads them
//   unit_free   converted and stored, proxy fence -> copy of tile n + DEPTH
//   k/v_full    fp16 tile written, proxy fence    -> S (n), w V (n)
//   k/v_free    commit after S (n), w V (n)       -> converter writes n + STAGES
//   q_full      Q written, proxy fence            -> first S of the run
//   s_full      commit after S (n)                -> softmax reads S
//   p_full      w stored, O rescaled, TMEM fence  -> w V (n)
//   pv_done     commit after w V (n)              -> S (n + 2), whose buffer holds the
//               weights of n; O's rescale for n + 1; O's and Q's last use of a run
//   sc_full/free  the scales of n                 -> softmax; scales of n + 4
// A commit follows all earlier products of its warp, so s_full (n) also says
// that w V (n - 2) is done, and a pv_done that nobody waited for is no phase
// behind.  Products of different shape or accumulator have no order of their own
// in the PTX model, so S (n + 2) waits for pv_done (n); only products into the
// same accumulator follow one another without a wait.  A converter's reads of
// a unit (generic proxy) and the copy that refills it (async proxy) need the
// proxy fence between them: with the unit released as soon as its loads were
// issued, a tile's last keys were now and then those of the tile after next.
//
// Every wait is bounded (WAIT_LIMIT_NS); a role whose wait ran out keeps
// walking its loops without waiting or touching TMEM, so that all barriers
// are still met.  The rows of that run and of the CTA's later ones are then NaN,
// and FDLLM_KV8_TIMEOUT is reported.  Before the CTA frees TMEM and ends, its
// copies and products in flight are waited for, on every path.
#include <algorithm>

#include "kv8_attn.cuh"

namespace fd {
namespace {

using namespace kv8;

constexpr int KEYS = PAGE;           // keys of a tile
constexpr int NB = KEYS / FDLLM_KV8_BLOCK;
constexpr int CONV = 64;             // converter threads of K, and of V

template <int HD, int NQ>
struct TcLay {
  static constexpr int KH = HD / 64;                  // 64-dim sub-tiles (128-byte rows)
  static constexpr int SUB = KEYS * 128;              // [64 keys][64 dims] fp16
  static constexpr int MAT = KH * SUB;                // fp16 K or V of a tile
  static constexpr int UNIT = KEYS * HD;              // int8 K or V of a tile
  static constexpr int DEPTH = 4;                     // tiles in the ring, K and V a unit each
  static constexpr int RING = 2 * DEPTH;
  static constexpr int STAGES = NQ;                   // fp16 tiles of K, and of V
  static constexpr int Q_SUB = 128 * 128;             // [128 rows][64 dims] fp16
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = K_OFF + STAGES * MAT;
  static constexpr int Q_OFF = V_OFF + STAGES * MAT;
  static constexpr int RING_OFF = Q_OFF + NQ * KH * Q_SUB;
  static constexpr int DIMS = 16;                     // dims of an exchange round
  static constexpr int XROW = DIMS + 4;
  static constexpr int X_OFF = RING_OFF + RING * UNIT;
  // scales of four tiles: ks, log2 vs, 1 / vs of 4 blocks
  static constexpr int SC_OFF = X_OFF + NQ * 128 * XROW * 4;
  static constexpr int RF_OFF = SC_OFF + 4 * 3 * NB * 4;   // row factors
  static constexpr int BAR_OFF = RF_OFF + NQ * 128 * 4;
  static constexpr int MISC_OFF = BAR_OFF + (31 + 2 * RING) * 8;
  static constexpr int PAGE_OFF = MISC_OFF + 16;           // the units' pages
  static constexpr int THREADS = 128 * NQ + 2 * CONV + 32 + 32 * NQ;
  static constexpr int WALK_OFF = (PAGE_OFF + RING * 4 + 15) / 16 * 16;
  static constexpr int SMEM = WALK_OFF + THREADS / 32 * (int)sizeof(Walk) + 1024;   // slack for
                                                                                    // 1024-byte alignment
  static constexpr uint32_t TMEM_COLS = 256 * NQ;     // a row tile: S 2 x 64, O 128
  static_assert(SMEM <= 232448, "shared memory layout");
};

// bytes (a multiple of 16) from global to shared memory, both 16-byte aligned.
FD_DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
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
// TMEM columns of this warp's lanes: 16 loaded, 32 stored (tmem_wait_st follows).
FD_DEV void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
FD_DEV void tmem_st32u(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
      "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31])
      : "memory");
}
FD_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <typename T, int HD, int NQ>
__global__ void __launch_bounds__(TcLay<HD, NQ>::THREADS, 1)
    kv8_attn_tc_kernel(const AttnP P) {
  using L = TcLay<HD, NQ>;
  constexpr int R = NQ * 128;          // query rows of a run
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  uint64_t* k_full = bars;             // [STAGES]: fp16 tiles
  uint64_t* k_free = bars + 2;
  uint64_t* v_full = bars + 4;
  uint64_t* v_free = bars + 6;
  uint64_t* s_full = bars + 8;         // [NQ][2], by tile parity
  uint64_t* drained = bars + 12;       // [NQ]: all products of the CTA
  uint64_t* pv_done = bars + 27;       // [NQ][2], by tile parity
  uint64_t* sc_full = bars + 14;       // [4]: scales
  uint64_t* sc_free = bars + 18;
  // [NQ][2], by tile parity (the softmax may be a tile ahead of the products):
  // weights written, O rescaled
  uint64_t* p_full = bars + 22;
  uint64_t* q_full = bars + 26;
  uint64_t* unit_full = bars + 31;     // [RING]
  uint64_t* unit_free = unit_full + L::RING;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
  int* err = reinterpret_cast<int*>(misc + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 2);
  volatile int* unit_page = reinterpret_cast<volatile int*>(smem + L::PAGE_OFF);   // -1: none
  const fdllm_kv8& c = P.c;
  const fdllm_kv8_attention_args& a = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_trigger();   // the join may be set up; it waits for this grid's end
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], CONV);
      mbar_init(&k_free[i], NQ);
      mbar_init(&v_full[i], CONV);
      mbar_init(&v_free[i], NQ);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_full[2 + i], 1);
      mbar_init(&pv_done[i], 1);
      mbar_init(&pv_done[2 + i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&p_full[2 + i], 128);
      mbar_init(&drained[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sc_full[i], NB);
      mbar_init(&sc_free[i], 128 * NQ);
    }
    mbar_init(q_full, 128 * NQ);
    for (int i = 0; i < L::RING; ++i) {
      mbar_init(&unit_full[i], 1);
      mbar_init(&unit_free[i], CONV);
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
  report_range(P);
  Walk* walk = reinterpret_cast<Walk*>(smem + L::WALK_OFF) + warp;
  walk_start(walk, P, R);
  Segment sg;
  bool ok = true;
  // a warp's wait: all lanes agree
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, err, abort_flag)) != 0;
    return ok;
  };

  if (warp < 4 * NQ) {
    // ================================================== softmax
    const int rep = a.n_heads / c.n_kv_heads;
    const int q = warp >> 2, quad = warp & 3, i = quad * 32 + lane;   // MMA row of tile q
    const int r = q * 128 + i;                                        // row of the run
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t s_col = tmem + q * 128 + lanes, o_col = s_col + NQ * 128;   // S: two buffers
    uint8_t* qs = smem + L::Q_OFF + q * L::KH * L::Q_SUB;
    float* rfs = reinterpret_cast<float*>(smem + L::RF_OFF) + q * 128;
    auto pv_wait = [&](int n) { return wait(&pv_done[2 * q + (n & 1)], (n >> 1) & 1); };
    int n_tile = 0;
    while (walk_next(walk, P, R, &sg)) {
      const int rr = sg.row0 + r;
      const int k_lo = sg.p_lo * PAGE, k_hi = min(sg.len, sg.p_hi * PAGE);
      const int tiles = (k_hi - k_lo + KEYS - 1) / KEYS;
      // ---- q, scaled per row by a power of two, into the swizzled A tile: HD / 8
      // lanes a row, 16 bytes each; every warp a quarter of the rows
      {
        constexpr int LR = HD / 8, RPW = 128 / 4, STEP = 32 / LR, N = RPW / STEP;
        constexpr int B = N < 8 ? N : 8;   // rows of a lane that are loaded at once
        const int ch = lane % LR, row_a = quad * RPW + lane / LR;   // row of the MMA tile
        const int first = sg.row0 + q * 128 + row_a;
        int token = first / rep, head = first % rep;
#pragma unroll 1
        for (int j0 = 0; j0 < N; j0 += B) {
          uint4 raw[B];
#pragma unroll
          for (int j = 0; j < B; ++j) {
            raw[j] = make_uint4(0, 0, 0, 0);
            if (first + (j0 + j) * STEP < sg.rows)
              raw[j] = *reinterpret_cast<const uint4*>(
                  reinterpret_cast<const T*>(a.q) + (int64_t)(sg.r_lo + token) * a.q_strides[0] +
                  (int64_t)(sg.g * rep + head) * a.q_strides[1] + ch * 8);
            for (head += STEP; head >= rep; head -= rep) ++token;
          }
#pragma unroll
          for (int j = 0; j < B; ++j) {
            const T* e = reinterpret_cast<const T*>(&raw[j]);
            float top = 0.0f;
#pragma unroll
            for (int m = 0; m < 8; ++m) top = fmaxf(top, fabsf(to_f<T>(e[m])));
#pragma unroll
            for (int o = LR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int up = q_shift(top), row = row_a + (j0 + j) * STEP;
            const float mul = exp2_int(up);
            uint32_t h[4];
#pragma unroll
            for (int m = 0; m < 4; ++m)
              h[m] = pack_h2(to_f<T>(e[2 * m]) * mul, to_f<T>(e[2 * m + 1]) * mul);
            *reinterpret_cast<uint4*>(qs + (ch >> 3) * L::Q_SUB + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) =
                make_uint4(h[0], h[1], h[2], h[3]);
            if (ch == 0) rfs[row] = a.scale * LOG2E * exp2_int(-up);
          }
        }
        fence_proxy_async_smem();
        if (tiles > 0) mbar_arrive(q_full);   // runs without keys have no MMAs
        named_bar(1 + q, 128);   // rfs
      }
      const float rf = rfs[i];
      float M = -INFINITY, l = 0.0f;
      for (int t = 0; t < tiles; ++t, ++n_tile) {
        const int k0 = k_lo + t * KEYS;
        const float* sc = reinterpret_cast<const float*>(smem + L::SC_OFF) + (n_tile & 3) * 3 * NB;
        wait(&s_full[2 * q + (n_tile & 1)], (n_tile >> 1) & 1);
        wait(&sc_full[n_tile & 3], (n_tile >> 2) & 1);
        if (ok) {
          tc_fence_after();
          float v[KEYS], mx = -INFINITY;
          const uint32_t buf = s_col + (n_tile & 1) * 64;
          tmem_ld64(buf, v);
#pragma unroll
          for (int b = 0; b < KEYS / 16; ++b) {
            const float f = rf * sc[b], g = sc[NB + b];
#pragma unroll
            for (int j = 16 * b; j < 16 * b + 16; j += 2) fma2(v[j], v[j + 1], f, g);
          }
          if (k0 + KEYS > k_hi) {
#pragma unroll
            for (int j = 0; j < KEYS; ++j)
              if (k0 + j >= k_hi) v[j] = -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < KEYS; j += 2) mx = fmaxf(fmaxf(mx, v[j]), v[j + 1]);
          float alpha = 1.0f;
          const bool move = passes(mx, M, M_SLACK);
          if (move) {
            alpha = ex2(M - mx);
            M = mx;
          }
          const float ref = weight_ref(M);
          float sum = 0.0f;
          uint32_t w[KEYS / 2];
#pragma unroll
          for (int b = 0; b < KEYS / 16; ++b) {
            float part[2] = {0.0f, 0.0f};
#pragma unroll
            for (int j = 16 * b; j < 16 * b + 16; j += 2) {
              const float e0 = ex2(v[j] + ref), e1 = ex2(v[j + 1] + ref);
              part[0] += e0;
              part[1] += e1;
              w[j / 2] = pack_h2(e0, e1);
            }
            sum = fmaf(part[0] + part[1], sc[2 * NB + b], sum);
          }
          // over the scores' first 32 columns (this warp has read its lanes)
          tmem_st32u(buf, w);
          l = fmaf(l, alpha, sum);
          if (t > 0 && __any_sync(0xffffffffu, move) && pv_wait(n_tile - 1)) {
            tc_fence_after();   // the products before are done: O is still
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 32) {
              float o[32];
              tmem_ld32(o_col + c0, o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] *= alpha;
              tmem_st32(o_col + c0, o);
            }
          }
          tmem_wait_st();
          tc_fence_before();
        }
        mbar_arrive(&sc_free[n_tile & 3]);
        mbar_arrive(&p_full[2 * q + (n_tile & 1)]);
      }
      // ---- the run's output, or its part, DIMS dims at a time through shared memory
      // (a role whose wait ran out has said so before it went on)
      const bool have_o = tiles > 0 && pv_wait(n_tile - 1) && !__any_sync(0xffffffffu, *abort_flag);
      const float none = tiles > 0 ? __int_as_float(0x7fffffff) : 0.0f;
      tc_fence_after();
      {
        constexpr int DIMS = L::DIMS, XROW = L::XROW, LR = DIMS / 4;
        const int64_t slot = ((int64_t)blockIdx.x * 2 + (sg.p_lo == 0)) * R;
        float* xo = reinterpret_cast<float*>(smem + L::X_OFF) + q * 128 * XROW;
        // a whole row is divided by its sum here, a partial one by the join
        float fac = 1.0f;
        if (sg.whole) fac = M == -INFINITY ? 0.0f : 1.0f / l;
        else if (rr < sg.rows) P.part_ml[slot + r] = make_float2(M, l);
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += DIMS) {
          float v[DIMS];
          if (have_o) tmem_ld16(o_col + c0, v);
#pragma unroll
          for (int j = 0; j < DIMS; j += 4)
            *reinterpret_cast<float4*>(xo + i * XROW + j) =
                have_o ? make_float4(v[j] * fac, v[j + 1] * fac, v[j + 2] * fac, v[j + 3] * fac)
                       : make_float4(none, none, none, none);
          named_bar(1 + q, 128);
          // LR lanes a row
          for (int at = i / LR; at < 128; at += 128 / LR) {
            const int d = i % LR * 4, rw = sg.row0 + q * 128 + at;
            if (rw >= sg.rows) break;
            const float4 x = *reinterpret_cast<const float4*>(xo + at * XROW + d);
            if (sg.whole)
              store4(reinterpret_cast<T*>(a.out) + (int64_t)(sg.r_lo + rw / rep) * a.out_strides[0] +
                         (int64_t)(sg.g * rep + rw % rep) * a.out_strides[1] + c0 + d,
                     x.x, x.y, x.z, x.w);
            else
              *reinterpret_cast<float4*>(P.part_o + (slot + q * 128 + at) * HD + c0 + d) = x;
          }
          named_bar(1 + q, 128);
        }
      }
      tc_fence_before();   // O has been read before the next run's first product
    }
  } else if (warp < 4 * NQ + 2 * CONV / 32) {
    // ================================================== converters
    const int is_v = tid >= 128 * NQ + CONV, ct = tid - 128 * NQ - (is_v ? CONV : 0);
    constexpr int HALVES = HD / 64;                // 64-byte halves of a key
    constexpr int ROWS = CONV / 4;
    constexpr int PER = KEYS / ROWS * HALVES;      // 16-byte chunks of a thread and unit
    // 4 lanes take 64 bytes of a key: the 8 lanes of a store then have an
    // even and an odd row, whose swizzled chunks are on different banks
    const int row0 = ct >> 2, ch = ct & 3;
    const uint8_t* ring = smem + L::RING_OFF;
    uint64_t *full = is_v ? v_full : k_full, *free = is_v ? v_free : k_free;
    int n_tile = 0;                                // tiles of the runs before
    while (walk_next(walk, P, R, &sg)) {
      const int end = n_tile + max(0, sg.p_hi - sg.p_lo);
      auto put = [&](uint8_t* mat, const uint4* x) {   // 16 codes: two 16-byte chunks
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int row = j / HALVES * ROWS + row0;
          const uint32_t y[4] = {x[j].x ^ 0x80808080u, x[j].y ^ 0x80808080u, x[j].z ^ 0x80808080u,
                                 x[j].w ^ 0x80808080u};
          uint32_t h[8];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            h[2 * m] = codes_h2<0x4140>(y[m]);
            h[2 * m + 1] = codes_h2<0x4342>(y[m]);
          }
          uint8_t* dst = mat + j % HALVES * L::SUB + row * 128;
          *reinterpret_cast<uint4*>(dst + ((2 * ch ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(dst + (((2 * ch + 1) ^ (row & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
      };
      for (; n_tile < end; ++n_tile) {
        const int st = n_tile % L::STAGES, use = n_tile / L::STAGES;
        const int slot = n_tile % L::DEPTH * 2 + is_v;
        wait(&unit_full[slot], (n_tile / L::DEPTH) & 1);
        const bool none = unit_page[slot] < 0;
        uint4 x[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j)
          x[j] = none ? make_uint4(0, 0, 0, 0)
                      : *reinterpret_cast<const uint4*>(ring + slot * L::UNIT + (j / HALVES * ROWS + row0) * HD +
                                                        j % HALVES * 64 + ch * 16);
        if (use > 0) wait(&free[st], (use - 1) & 1);
        put(smem + (is_v ? L::V_OFF : L::K_OFF) + st * L::MAT, x);
        // behind the stores, which need all that was loaded, and their proxy fence
        mbar_arrive(&unit_free[slot]);
        mbar_arrive(&full[st]);
      }
    }
  } else if (warp == 4 * NQ + 2 * CONV / 32) {
    // ================================================== copies
    uint8_t* ring = smem + L::RING_OFF;
    int n_tile = 0;
    // scales of block `lane` of the last tile asked for, on their way
    float ks = 0.0f, vs = 0.0f;
    bool live = false;
    int issued[2] = {0, 0};   // tiles whose units of K, of V were asked for
    auto store_scales = [&](int n) {
      const int at = n & 3;
      if (n >= 4) wait(&sc_free[at], (n / 4 - 1) & 1);
      if (lane < NB) {
        float* sc = reinterpret_cast<float*>(smem + L::SC_OFF) + at * 3 * NB + lane;
        const float v = fmaxf(vs, VS_MIN);
        sc[0] = live ? ks : 0.0f;
        sc[NB] = live ? __log2f(v) : -INFINITY;
        sc[2 * NB] = live ? __fdividef(1.0f, v) : 0.0f;
        mbar_arrive(&sc_full[at]);
      }
      __syncwarp();
    };
    while (walk_next(walk, P, R, &sg)) {
      const int32_t* table = c.page_table + (int64_t)sg.seq * c.table_stride;
      const int tiles = max(0, sg.p_hi - sg.p_lo);
      int ids = -1;                            // page ids of 32 tiles, one a lane
      for (int t = 0; t < tiles; ++t) {
        if ((t & 31) == 0) {
          const int at = sg.p_lo + t + lane;
          ids = at < sg.p_hi ? table[at] : -1;
          if (at < sg.p_hi && (ids < 0 || ids >= c.n_pages)) {
            ids = -1;
            if (a.status) atomicOr(a.status, FDLLM_KV8_BAD_PAGE);
          }
        }
        const int page = __shfl_sync(0xffffffffu, ids, t & 31), n = n_tile + t;
#pragma unroll
        for (int is_v = 0; is_v < 2; ++is_v) {
          const int slot = n % L::DEPTH * 2 + is_v;
          if (n >= L::DEPTH) wait(&unit_free[slot], (n / L::DEPTH - 1) & 1);
          if (ok) issued[is_v] = n + 1;
          if (ok && lane == 0) {
            unit_page[slot] = page;
            if (page < 0) {
              mbar_arrive(&unit_full[slot]);
            } else {
              mbar_arrive_expect_tx(&unit_full[slot], L::UNIT);
              bulk_load(ring + slot * L::UNIT,
                        (is_v ? c.v : c.k) + (int64_t)page * c.page_stride + (int64_t)sg.g * L::UNIT,
                        L::UNIT, &unit_full[slot]);
            }
          }
          __syncwarp();
        }
        // the scales of the tile before have arrived by now
        if (t > 0) store_scales(n - 1);
        live = lane < NB && page >= 0 && (sg.p_lo + t) * PAGE + lane * 16 < sg.len;
        if (live) {
          const int64_t so = (int64_t)page * c.scale_stride + sg.g * 4 + lane;
          ks = c.k_scale[so];
          vs = c.v_scale[so];
        }
      }
      if (tiles > 0) store_scales(n_tile + tiles - 1);
      n_tile += tiles;
    }
    // no copy may land in shared memory that the CTA has given back
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v)
      for (int n = max(0, issued[is_v] - L::DEPTH); n < issued[is_v]; ++n)
        mbar_wait(&unit_full[n % L::DEPTH * 2 + is_v], (n / L::DEPTH) & 1, err, nullptr);
  } else {
    // ================================================== MMA, a warp a row tile
    const int q = warp - (4 * NQ + 2 * CONV / 32 + 1);
    const uint32_t kb = smem_u32(smem + L::K_OFF), vb = smem_u32(smem + L::V_OFF);
    const uint64_t qd = smem_desc_sw128(smem_u32(smem + L::Q_OFF) + q * L::KH * L::Q_SUB);
    int n_tile = 0, n_seg = 0;
    while (walk_next(walk, P, R, &sg)) {
      const int tiles = max(0, sg.p_hi - sg.p_lo);
      if (tiles > 0) wait(q_full, n_seg++ & 1);
      for (int t = 0; tiles > 0 && t <= tiles; ++t) {
        // S of tile t, then w V of tile t - 1 (whose weights lie in S's other buffer)
        if (t < tiles) {
          const int n = n_tile + t, st = n % L::STAGES;
          wait(&k_full[st], (n / L::STAGES) & 1);
          // the weights of tile n - 2 lie where S goes
          if (n >= 2) wait(&pv_done[2 * q + (n & 1)], ((n >> 1) - 1) & 1);
          if (ok && lane == 0) {
            tc_fence_after();
            // a step along K moves the descriptors' start address (in 16 bytes)
            const uint64_t kd = smem_desc_sw128(kb + st * L::MAT);
#pragma unroll
            for (int k = 0; k < HD / 16; ++k)
              tc_mma(tmem + q * 128 + (n & 1) * 64, qd + (((k >> 2) * L::Q_SUB + (k & 3) * 32) >> 4),
                     kd + (((k >> 2) * L::SUB + (k & 3) * 32) >> 4), idesc_f32acc(KEYS, true), k > 0);
            tc_commit(&s_full[2 * q + (n & 1)]);
            tc_commit(&k_free[st]);
          }
          __syncwarp();
        }
        if (t > 0) {
          const int n = n_tile + t - 1, st = n % L::STAGES;
          wait(&v_full[st], (n / L::STAGES) & 1);
          wait(&p_full[2 * q + (n & 1)], (n >> 1) & 1);
          if (ok && lane == 0) {
            tc_fence_after();
            const uint64_t vd = smem_desc_sw128_mn(vb + st * L::MAT, L::SUB, 1024);
#pragma unroll
            for (int k = 0; k < KEYS / 16; ++k)
              tc_mma_ts(tmem + NQ * 128 + q * 128, tmem + q * 128 + (n & 1) * 64 + k * 8,
                        vd + (k * 2048 >> 4), idesc_f32acc_bmn(HD, true), t > 1 || k > 0);
            tc_commit(&pv_done[2 * q + (n & 1)]);
            tc_commit(&v_free[st]);
          }
          __syncwarp();
        }
      }
      n_tile += tiles;
    }
    // no product may touch TMEM or shared memory that the CTA has given back
    if (lane == 0) tc_commit(&drained[q]);
    mbar_wait(&drained[q], 0, err, nullptr);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, L::TMEM_COLS);
  if (tid == 0 && *err && a.status) atomicOr(a.status, FDLLM_KV8_TIMEOUT);
}

template <typename T, int HD, int NQ>
cudaError_t launch_tc(const AttnP& P, cudaStream_t st) {
  using L = TcLay<HD, NQ>;
  auto kern = kv8_attn_tc_kernel<T, HD, NQ>;
  static std::atomic<uint64_t> ready{0};   // devices whose limit is set
  cudaError_t e = allow_smem(kern, L::SMEM, ready);
  if (e == cudaSuccess) e = launch_k(false, kern, dim3(P.n_cta), dim3(L::THREADS), L::SMEM, st, P);
  if (e == cudaSuccess) e = launch_join<T, HD, NQ * 128>(P, st);
  return e;
}

template <typename T, int HD>
cudaError_t launch_tc_hd(const AttnP& P, int rows, cudaStream_t st) {
  return rows == 128 ? launch_tc<T, HD, 1>(P, st) : launch_tc<T, HD, 2>(P, st);
}

}  // namespace

namespace kv8 {

int tc_tile_rows(int64_t rows) { return rows <= 128 ? 128 : 256; }

cudaError_t launch_attn_tc(const AttnP& P, int rows, cudaStream_t st) {
  if (P.a.dtype == FDLLM_DTYPE_BF16)
    return P.c.head_dim == 128 ? launch_tc_hd<__nv_bfloat16, 128>(P, rows, st)
                               : launch_tc_hd<__nv_bfloat16, 64>(P, rows, st);
  return P.c.head_dim == 128 ? launch_tc_hd<__half, 128>(P, rows, st)
                             : launch_tc_hd<__half, 64>(P, rows, st);
}

}  // namespace kv8
}  // namespace fd
