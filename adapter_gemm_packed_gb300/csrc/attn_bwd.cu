// Windowed attention backward on the tensor cores (bf16): one kernel for dQ, then one for dK and dV.
//
// Both hold two tiles of 128 rows in shared memory and stream pairs of 64-row tiles of the other side past them:
//                rows (128)    streamed (64)   S               T                sums in TMEM
//   dQ           Q,  dO        K,  V           Q K^T           dO V^T           dQ += dS K
//   dK and dV    K,  V         Q,  dO          K Q^T           V dO^T           dV += P^T dO, dK += dS^T Q
// with P = 2^(|scale| log2(e) S - L2) and dS = P (T - delta), of which the dK / dV kernel holds the transposes: its
// threads own keys, so P^T and dS^T are TMEM operands of the second products just as they come out of the
// first, and nothing of a score tile goes through shared memory.  P and dS are rounded to bf16 as operands;
// all sums are fp32.  Computing S and T twice (seven products instead of five) buys sums without atomics:
// dQ belongs to one block, and so do dK and dV, whose block adds up the query heads of the group in order.
//
// delta_i = sum_d dO_id O_id is made by the dQ kernel and left for the other next to the softmax statistics.  O is
// completed by the bits that its rounding to bf16 cut off: with the rounded O alone, delta would cost dQ and dK as
// much accuracy as the rounding of dS does.
//
// What bounds these kernels is shared memory: a score product of 128 x 64 x 128 out of shared memory reads 48 KB,
// 384 cycles of its bandwidth for 256 cycles of tensor work, and the streamed tiles are written there too.  The dQ
// kernel has TMEM to spare and keeps Q and dO in it as operands (its steps took 1290 cycles from shared memory);
// the dK / dV kernel has not.  16,384 tokens, window 4096, 64 first tokens, 16 heads of 128 on 4: 452 and 648
// microseconds, 1.6 and 1.5 PFLOP/s of the three and four products that each does (a plain large product of the
// library: 1.9); 9 sequences of 97 to 2501, 32 heads on 8: 133 and 178, where pieces are short.
//
// One block per SM walks over its share of the work list; the next piece's loads and first products run under this
// one's last tiles and its output.
//
// Warps 0-3 and 4-7 take the even and the odd streamed tiles (S, T in buffers of their own), so that one set
// computes while the products of the other run.  Warp 8: TMA loads.  Warp 9: products.  Warp 10: zeros
// behind the sequence's end.  In the dQ kernel, warps 12-15 prepare the next piece (delta, TMEM operands).
#include "attn_tc.cuh"

namespace mlora {
namespace {

template <bool KEYS>
constexpr int THREADS = KEYS ? 352 : 512;
constexpr int STAGES = 4;

template <int DS>
constexpr int OWN = 128 * 128 * DS;         // bytes of a tile of the block's own rows
template <int DS>
constexpr int STR = 64 * 128 * DS;          // bytes of a streamed tile (two make a ring entry)
template <int DS, bool KEYS>
constexpr int SMEM = 2 * OWN<DS> + STAGES * (2 * STR<DS> + STAT_BLOCK * 4) + 8 * OUT_WARP + 256;

struct BwdArgs {
  AttnArgs a;
  TileMap x0, x1, y0, y1, g0, g1;      // g0, g1: dQ, or dV and dK
};

// A piece of work: 128 rows of a head and the tiles streamed past them, in order.
struct Work {
  int h, r0;
  KeyTiles kt;          // dQ: key tiles of 64
  int q_first, q_n;     // dK / dV: query tiles of 64 per query head
  int n0;               // first of them (counting through the query heads) that this part does
  int count;            // 0: rows that belong to no sequence
};

template <bool KEYS>
__device__ __forceinline__ Work decode(const AttnArgs& A, const AttnItem& it) {
  Work w{};
  w.h = it.sub;
  w.r0 = it.i0;
  if (it.len == 0) return w;
  const int r1 = min(it.i0 + 128, it.len);
  if (KEYS) {
    int lo, hi;
    query_rows(it.i0, r1, it.len, A.window, A.n_sink, lo, hi);
    w.q_first = lo / 64;
    w.q_n = (hi + 63) / 64 - w.q_first;
    w.count = w.q_n * A.group;
    if (it.parts > 1) {
      w.n0 = static_cast<int>(static_cast<long long>(w.count) * it.part / it.parts);
      w.count = static_cast<int>(static_cast<long long>(w.count) * (it.part + 1) / it.parts) - w.n0;
    }
  } else {
    w.kt = key_tiles(it.i0, r1, A.window, A.n_sink, 64);
    w.count = w.kt.count();
  }
  return w;
}

// head and first row (within the sequence) of streamed tile n
template <bool KEYS>
__device__ __forceinline__ void streamed(const AttnArgs& A, const Work& w, int n, int& head, int& row) {
  if (KEYS) {
    n += w.n0;
    const int g = n / w.q_n;
    head = w.h * A.group + g;
    row = (w.q_first + n - g * w.q_n) * 64;
  } else {
    head = w.h / A.group;
    row = w.kt.tile(n) * 64;
  }
}

// Eight columns of dO O, O completed by its low bytes
__device__ __forceinline__ float dot8(const uint4& x, const uint2& l, const uint4& y) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w}, lw[2] = {l.x, l.y};
  float t = 0.f, v = 0.f;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    t = fmaf(out_whole(xs[u] << 16, lw[u / 2], u % 2 * 2), __uint_as_float(ys[u] << 16), t);
    v = fmaf(out_whole(xs[u] & 0xffff0000u, lw[u / 2], u % 2 * 2 + 1), __uint_as_float(ys[u] & 0xffff0000u), v);
  }
  return t + v;
}

// delta of a warp's 32 rows (from row i0 of the sequence on) into d[0, 32) and the statistics: half a warp per row
// and eight columns a lane, eight pairs of rows at a time.  These warps share their schedulers with the softmax,
// so instructions are what counts: addresses advance by additions, and the eight sums of a lane are spread over
// the half-warp as they are added up (8 shuffles for 8 rows).
template <int DS>
__device__ __forceinline__ void warp_delta(const AttnArgs& A, const AttnItem& it, int h, int i0, float* d, int lane) {
  const int half = lane >> 4, col = 8 * (lane & 15);
  const bool on = col < A.D;
  const long long first = static_cast<long long>(it.seq0) + i0 + half;
  const __nv_bfloat16* o = head_row<__nv_bfloat16>(A.o, first, h) + (on ? col : 0);
  const __nv_bfloat16* g = head_row<__nv_bfloat16>(A.dout, first, h) + (on ? col : 0);
  const uint8_t* low = out_low_at(A, 4 * DS, h, it.stat0 + i0) + half * 16 + (on ? col / 16 * 512 + col % 16 : 0);
  const long long so = 2 * A.o.row_stride, sg = 2 * A.dout.row_stride;
  const int rows = it.len - i0 - half;      // rows of this half's parity count while 2 n < rows
#pragma unroll 1
  for (int n0 = 0; n0 < 16; n0 += 8) {
    uint4 x[8], y[8];
    uint2 l[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const bool real = 2 * (n0 + n) < rows;
      x[n] = y[n] = make_uint4(0, 0, 0, 0);
      l[n] = make_uint2(0, 0);
      if (real) {
        x[n] = *reinterpret_cast<const uint4*>(o);
        y[n] = *reinterpret_cast<const uint4*>(g);
        l[n] = *reinterpret_cast<const uint2*>(low + (n0 + n) * 32);
      }
      o += so;
      g += sg;
    }
    float t[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) t[n] = on ? dot8(x[n], l[n], y[n]) : 0.f;
#pragma unroll
    for (int w = 4; w; w /= 2) {      // a lane keeps w of the 2 w rows it holds and adds the other's share of them
      const bool up = lane & (2 * w);
#pragma unroll
      for (int n = 0; n < w; ++n) {
        const float keep = up ? t[n + w] : t[n], send = up ? t[n] : t[n + w];
        t[n] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * w);
      }
    }
    t[0] += __shfl_xor_sync(0xffffffffu, t[0], 1);
    const int r = 2 * (n0 + (lane >> 1 & 7)) + half;
    if (!(lane & 1)) {
      d[r] = t[0];
      A.saved[stat_at(A.n_stat, h, it.stat0 + i0 + r) + STAT_ROWS] = t[0];
    }
  }
}

// A warp's sums of a cut piece: into the scratch, and if all parts' are there, their sum in order into o.  No warp
// waits for another.  (The dQ kernel, which has ended, has set the counters to zero.)
template <int DS, int NQ>
__device__ __forceinline__ bool join_parts(const AttnArgs& A, const AttnItem& it, int warp, int lane, uint32_t (&o)[NQ][32]) {
  constexpr int SET = 8 * 32 * 64 * DS;      // floats of one part: eight warps, 32 rows, 64 DS columns
  float* sums = A.partials + static_cast<long long>(it.pbase) * SET + warp * (32 * 64 * DS) + lane * 4;
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int u = 0; u < 8; ++u)
      *reinterpret_cast<uint4*>(sums + static_cast<long long>(it.part) * SET + (8 * q + u) * 128) =
          make_uint4(o[q][4 * u], o[q][4 * u + 1], o[q][4 * u + 2], o[q][4 * u + 3]);
  __threadfence();
  __syncwarp();
  int* cnt = A.part_cnt + it.slot * 8 + warp;
  int last = 0;
  if (lane == 0) last = atomicAdd(cnt, 1) == it.parts - 1;
  if (!__shfl_sync(0xffffffffu, last, 0)) return false;
  __threadfence();
#pragma unroll 1
  for (int p = 0; p < it.parts; ++p)
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(sums + static_cast<long long>(p) * SET + (8 * q + u) * 128));
        const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[q][4 * u + e] = __float_as_uint(p == 0 ? a[e] : __uint_as_float(o[q][4 * u + e]) + a[e]);
      }
  return true;
}

template <int DS, bool KEYS>
__global__ void __launch_bounds__(THREADS<KEYS>, 1) k_attn_bwd(const __grid_constant__ BwdArgs F) {
  griddep_wait();
  extern __shared__ __align__(1024) uint8_t smem[];
  const AttnArgs& A = F.a;
  const int k_first = A.first[blockIdx.x], k_end = A.first[blockIdx.x + 1];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (!smem_aligned(smem, A.err)) return;
  uint8_t* sX0 = smem;
  uint8_t* sX1 = smem + OWN<DS>;
  uint8_t* sY = smem + 2 * OWN<DS>;                 // per stage: Y0, Y1
  uint8_t* sOut = sY + STAGES * 2 * STR<DS>;
  // dK / dV: L2 and delta per stage; dQ: of the block's own rows, [piece's parity][L2 or delta][row]
  float* sStat = reinterpret_cast<float*>(sOut + 8 * OUT_WARP);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sStat + STAGES * STAT_BLOCK);
  uint64_t *x_full = bars, *x_empty = bars + 1, *y_full = bars + 2, *y_empty = y_full + STAGES,
           *y_clean = y_empty + STAGES, *s_full = y_clean + STAGES, *p_full = s_full + 2, *acc_done = p_full + 2,
           *acc_free = acc_done + 1, *x_ready = acc_free + 1, *sc_done = x_ready + 1,
           *d_ready = sc_done + 1, *d_free = d_ready + 2, *done = d_free + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(slot + 1);
  if (tid == 0) {
    mbar_init(x_full, 1);
    mbar_init(x_empty, KEYS ? 1 : 4);
    for (int i = 0; i < STAGES; ++i) mbar_init(&y_full[i], 1), mbar_init(&y_empty[i], 1), mbar_init(&y_clean[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_full[i], 4);
    mbar_init(acc_free, 8);
    mbar_init(x_ready, 4);
    for (int i = 0; i < 2; ++i) mbar_init(&d_ready[i], 4), mbar_init(&d_free[i], 8);
    mbar_init(sc_done, 1);
    mbar_init(acc_done, 1);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(slot, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  // columns: S of buffer b at 64 b, T at 128 + 64 b; dV at 256 and dK at 384, or dQ at 256, Q at 384 and dO at 448

  AttnItem it = A.items[k_first];
  auto next_item = [&](int k) { return k + 1 < k_end ? A.items[k + 1] : it; };

  if (warp < 8) {
    const int b = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lanes + 64 * b, tT = tS + 128;
    const float c = A.scale_log2;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return warp_wait(bar, parity, abort_flag, A.err, DEV_ERR_TIMEOUT_EPILOGUE, A.timeout_ns, lane);
    };
    int pos = 0, tiles = 0, piece = 0;
    bool ok = true;
    // the counters that the cut pieces of the kernel after this one start from
    if (!KEYS && blockIdx.x == 0)
      for (int e = tid; e < A.n_cnt; e += 256) A.part_cnt[e] = 0;
    for (int k = k_first; ok && k < k_end; ++k) {
      const AttnItem nx = next_item(k);
      const Work w = decode<KEYS>(A, it);
      if (w.count == 0) {
        zero_out_rows(KEYS ? A.dk : A.dq, it, KEYS ? A.hk : A.hq, A.D, tid, 256);
        if (KEYS) zero_out_rows(A.dv, it, A.hk, A.D, tid, 256);
        it = nx;
        continue;
      }
      const int r0 = w.r0;
      float l2 = 0.f, delta = 0.f;
      if constexpr (!KEYS) {
        ok = wait(&d_ready[piece & 1], (piece >> 1) & 1);
        if (!ok) break;
        l2 = sStat[(piece & 1) * 256 + r];
        delta = sStat[(piece & 1) * 256 + 128 + r];
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_free[piece & 1]);
      }
      for (int n = (b ^ tiles) & 1; n < w.count; n += 2) {
        const int at = pos + n, sl = at % STAGES;
        int head, row;
        streamed<KEYS>(A, w, n, head, row);
        // dK / dV: the tile's statistics came with it, 16 columns of L2 and delta at a time (the same for all rows)
        float4 l4[4], d4[4];
        const float4* st4 = reinterpret_cast<const float4*>(sStat + sl * STAT_BLOCK);
        auto stats = [&](int c16) {
#pragma unroll
          for (int u = 0; u < 4; ++u) l4[u] = st4[4 * c16 + u], d4[u] = st4[16 + 4 * c16 + u];
        };
        if (KEYS) {
          ok = wait(&y_full[sl], (at / STAGES) & 1);
          if (!ok) break;
          stats(0);
        }
        uint32_t seen[2] = {0xffffffffu, 0xffffffffu};
        if (KEYS) {
          const int j = r0 + r;
          if (!(row >= r0 + 127 && (row + 63 - r0 < A.window || r0 + 127 < A.n_sink))) {
            // query column i = row + col sees key j: j <= i, and i < j + window unless j is a first token
#pragma unroll
            for (int q = 0; q < 2; ++q)
              seen[q] = ~bits_below(j - row, 32 * q) &
                        (j < A.n_sink ? 0xffffffffu
                                      : bits_below(static_cast<int>(min(static_cast<long long>(j) + A.window - row, 64ll)), 32 * q));
          }
        } else {
          const int i = r0 + r;
          if (!(row + 63 <= r0 && (r0 + 127 - row < A.window || row + 63 < A.n_sink))) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
              seen[q] = bits_below(i - row + 1, 32 * q) & (~bits_below(i - A.window + 1 - row, 32 * q) | bits_below(A.n_sink - row, 32 * q));
            // (a tile that such a row takes part in is never one that all rows see all of)
            if (sees_one(i, A.window, A.n_sink)) seen[0] = seen[1] = 0;
          }
        }
        const bool all = __all_sync(0xffffffffu, (seen[0] & seen[1]) == 0xffffffffu);
        ok = wait(&s_full[b], ((tiles + n) >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t s[32], t[32], p[16], ds[16];
          tmem_ld32(tS + 32 * q, s);
          tmem_ld32(tT + 32 * q, t);
          tmem_ld_wait();
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float ll[16], dd[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) ll[u] = l2, dd[u] = delta;
            if (KEYS) {
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                ll[4 * u] = l4[u].x, ll[4 * u + 1] = l4[u].y, ll[4 * u + 2] = l4[u].z, ll[4 * u + 3] = l4[u].w;
                dd[4 * u] = d4[u].x, dd[4 * u + 1] = d4[u].y, dd[4 * u + 2] = d4[u].z, dd[4 * u + 3] = d4[u].w;
              }
              if (2 * q + hf < 3) stats(2 * q + hf + 1);
            }
#pragma unroll
            for (int u = 0; u < 16; u += 2) {
              const int e = 16 * hf + u;
              float x0 = __uint_as_float(s[e]), x1 = __uint_as_float(s[e + 1]);
              float y0 = __uint_as_float(t[e]), y1 = __uint_as_float(t[e + 1]);
              fma2(x0, x1, c, c, -ll[u], -ll[u + 1]);
              x0 = ex2(x0), x1 = ex2(x1);
              add2(y0, y1, -dd[u], -dd[u + 1]);
              mul2(y0, y1, x0, x1);
              if (!all) {
                if (!(seen[q] >> e & 1)) x0 = y0 = 0.f;
                if (!(seen[q] >> (e + 1) & 1)) x1 = y1 = 0.f;
                if (KEYS && q == 0 && e == 0 && row == 0) y0 = 0.f;      // a sequence's first token sees one key
              }
              p[e / 2] = pack_bf16x2(x0, x1);
              ds[e / 2] = pack_bf16x2(y0, y1);
            }
          }
          // P goes over S, dS over T: onto columns whose values are in registers
          if (KEYS) tmem_st16(tS + 16 * q, p);
          tmem_st16(tT + 16 * q, ds);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[b]);
      }
      if (!ok) break;
      pos += w.count;
      tiles += w.count;
      // the sums: set 0 writes dV, set 1 dK; or each half the columns of dQ
      ok = wait(acc_done, piece & 1);
      if (!ok) break;
      tc_fence_after();
      constexpr int NQ = KEYS ? 2 * DS : DS;
      const int q0 = KEYS ? 0 : b * DS;
      const uint32_t acc = tmem + lanes + (KEYS ? 256 + 128 * b : 256) + 32 * q0;
      uint32_t o[NQ][32];
#pragma unroll
      for (int q = 0; q < NQ; ++q) tmem_ld32(acc + 32 * q, o[q]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_free);
      if (KEYS && it.parts > 1 && !join_parts<DS>(A, it, warp, lane, o)) {
        ++piece;
        it = nx;
        continue;
      }
      const int first = r0 + quarter * 32;
      OutWarp out{KEYS && b ? &F.g1 : &F.g0, KEYS ? (b ? &A.dk : &A.dv) : &A.dq, sOut + warp * OUT_WARP,
                  it.seq0 + first, w.h, max(0, min(32, it.len - first)), A.D, lane};
      if (!KEYS || b == 1) {
        // (zero where no token sees more than one key)
        const float f = KEYS && sees_one(1, A.window, A.n_sink) ? 0.f : A.scale;
#pragma unroll
        for (int q = 0; q < NQ; ++q) scale32(o[q], f);
      }
      if constexpr (NQ == 1) {
        if (32 * q0 < A.D) out.put<1>(32 * q0, &o[0]);
      } else {
#pragma unroll
        for (int q = 0; q < NQ; q += 2) out.put<2>(32 * (q0 + q), &o[q]);
      }
      ++piece;
      it = nx;
    }
    if (elect_lane()) bulk_wait_all();      // no store may still be reading shared memory when the block ends
    __syncwarp();
  } else if (warp == 8) {
    if (elect_lane()) {
      int pos = 0, piece = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait(bar, parity, abort_flag, A.err, DEV_ERR_TIMEOUT_PRODUCER, A.timeout_ns);
      };
      for (int k = k_first; ok && k < k_end; ++k) {
        const AttnItem nx = next_item(k);
        const Work w = decode<KEYS>(A, it);
        if (w.count) {
          ok = piece == 0 || wait(x_empty, (piece - 1) & 1);
          if (!ok) break;
          mbar_arrive_expect_tx(x_full, 2 * OWN<DS>);
          load_tile<DS, 128>(sX0, F.x0, x_full, it.seq0 + w.r0, w.h);
          load_tile<DS, 128>(sX1, F.x1, x_full, it.seq0 + w.r0, w.h);
          ++piece;
          // what the next piece starts with, towards L2
          if (k + 1 < k_end && nx.len) {
            const Work v = decode<KEYS>(A, nx);
            int head, row;
            streamed<KEYS>(A, v, 0, head, row);
            prefetch_tile<DS, 128>(F.x0, nx.seq0 + v.r0, v.h);
            prefetch_tile<DS, 128>(F.x1, nx.seq0 + v.r0, v.h);
            prefetch_tile<DS, 64>(F.y0, nx.seq0 + row, head);
            prefetch_tile<DS, 64>(F.y1, nx.seq0 + row, head);
          }
          for (int n = 0; n < w.count; ++n) {
            const int sl = pos % STAGES;
            ok = wait(&y_empty[sl], ((pos / STAGES) & 1) ^ 1u);
            if (!ok) break;
            uint8_t* y = sY + sl * 2 * STR<DS>;
            int head, row;
            streamed<KEYS>(A, w, n, head, row);
            mbar_arrive_expect_tx(&y_full[sl], 2 * STR<DS> + (KEYS ? STAT_BLOCK * 4 : 0));
            load_tile<DS, 64>(y, F.y0, &y_full[sl], it.seq0 + row, head);
            load_tile<DS, 64>(y + STR<DS>, F.y1, &y_full[sl], it.seq0 + row, head);
            if (KEYS)
              bulk_load(sStat + sl * STAT_BLOCK, A.saved + stat_at(A.n_stat, head, it.stat0 + row), STAT_BLOCK * 4, &y_full[sl]);
            ++pos;
          }
        }
        it = nx;
      }
      // bounded: no copy may still be writing shared memory when the block ends, whoever gave up and whenever
      volatile int no_abort = 0;
      if (piece) mbar_wait(x_full, (piece - 1) & 1, &no_abort, A.err, DEV_ERR_TIMEOUT_TEARDOWN, A.timeout_ns);
      for (int q = pos > STAGES ? pos - STAGES : 0; q < pos; ++q)
        mbar_wait(&y_full[q % STAGES], (q / STAGES) & 1, &no_abort, A.err, DEV_ERR_TIMEOUT_TEARDOWN, A.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 10) {
    // The last streamed tile may reach past the sequence's end: what lies there becomes zero before any product
    // reads it (zero times NaN is NaN).  Every entry goes through here, which keeps the warp in step.
    int pos = 0;
    bool ok = true;
    for (int k = k_first; ok && k < k_end; ++k) {
      const AttnItem nx = next_item(k);
      const Work w = decode<KEYS>(A, it);
      if (w.count)
        for (int n = 0; n < w.count; ++n, ++pos) {
          const int sl = pos % STAGES;
          ok = warp_wait(&y_full[sl], (pos / STAGES) & 1, abort_flag, A.err, DEV_ERR_TIMEOUT_PRODUCER, A.timeout_ns, lane);
          if (!ok) break;
          int head, row;
          streamed<KEYS>(A, w, n, head, row);
          if (row + 64 > it.len) {
            zero_rows_from<DS, 64>(sY + sl * 2 * STR<DS>, it.len - row, lane);
            if (KEYS) zero_rows_from<DS, 64>(sY + sl * 2 * STR<DS> + STR<DS>, it.len - row, lane);
          }
          if (lane == 0) mbar_arrive(&y_clean[sl]);
        }
      it = nx;
    }
  } else if (warp >= 12) {
    // dQ: what a piece needs besides its streamed tiles, a row per thread, while the piece before it is under way:
    // delta and L2 of its rows, and as soon as the score products before have read theirs, Q and dO into TMEM.
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t flip = A.scale < 0.f ? 0x80008000u : 0u;      // a negative scale negates Q
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return warp_wait(bar, parity, abort_flag, A.err, DEV_ERR_TIMEOUT_EPILOGUE, A.timeout_ns, lane);
    };
    int piece = 0;
    bool ok = !KEYS;
    for (int k = k_first; ok && k < k_end; ++k) {
      const AttnItem nx = next_item(k);
      const Work w = decode<KEYS>(A, it);
      if (w.count) {
        ok = piece < 2 || wait(&d_free[piece & 1], ((piece >> 1) - 1) & 1);
        if (!ok) break;
        float* own = sStat + (piece & 1) * 256;
        const long long at = stat_at(A.n_stat, w.h, it.stat0 + w.r0 + r);
        own[r] = A.saved[at];
        warp_delta<DS>(A, it, w.h, w.r0 + quarter * 32, own + 128 + quarter * 32, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_ready[piece & 1]);
        ok = wait(x_full, piece & 1);
        if (!ok) break;
        if (piece) {
          ok = wait(sc_done, (piece - 1) & 1);
          if (!ok) break;
          tc_fence_after();
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int s = 0; s < DS; ++s) {
            uint32_t v[32];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const uint4 t = *reinterpret_cast<const uint4*>((x ? sX1 : sX0) + s * 128 * 128 + r * 128 + ((c ^ (r & 7)) << 4));
              const uint32_t f = x ? 0u : flip;
              v[4 * c] = t.x ^ f, v[4 * c + 1] = t.y ^ f, v[4 * c + 2] = t.z ^ f, v[4 * c + 3] = t.w ^ f;
            }
            tmem_st32(tmem + lanes + 384 + 64 * x + 32 * s, v);
          }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(x_ready);
          mbar_arrive(x_empty);
        }
        ++piece;
      }
      it = nx;
    }
  } else if (warp == 9) {
    if (elect_lane()) {
      constexpr uint32_t idesc = idesc_bf16(128, 64, false, false);
      [[maybe_unused]] const uint32_t idesc_s = idesc | (A.scale < 0.f ? IDESC_NEG_A : 0u);
      [[maybe_unused]] const uint64_t dx0 = desc_rows(sX0), dx1 = desc_rows(sX1);
      const uint64_t dy = desc_rows(sY), dy_cols = desc_cols<64>(sY);
      constexpr uint64_t ONE = STR<DS> / 16;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait(bar, parity, abort_flag, A.err, DEV_ERR_TIMEOUT_MMA, A.timeout_ns);
      };
      int pos = 0, tiles = 0, piece = 0;
      bool ok = true;
      for (int k = k_first; ok && k < k_end; ++k) {
        const AttnItem nx = next_item(k);
        const int count = decode<KEYS>(A, it).count;
        if (count) {
          // S and T of tile n into the buffer of its turn
          auto scores = [&](int n) {
            const int at = pos + n, sl = at % STAGES, buf = (tiles + n) & 1;
            if (!wait(&y_clean[sl], (at / STAGES) & 1)) return false;
            const uint64_t y = dy + sl * 2 * ONE;
            if (KEYS) {
              mma_scores<DS, 128, 64>(tmem + 64 * buf, dx0, y, idesc_s);
              mma_scores<DS, 128, 64>(tmem + 128 + 64 * buf, dx1, y + ONE, idesc);
            } else {
              mma_scores_ts<DS, 64>(tmem + 64 * buf, tmem + 384, y, idesc);
              mma_scores_ts<DS, 64>(tmem + 128 + 64 * buf, tmem + 448, y + ONE, idesc);
            }
            umma_commit(&s_full[buf]);
            if (n + 1 == count) umma_commit(KEYS ? x_empty : sc_done);
            return true;
          };
          ok = wait(KEYS ? x_full : x_ready, piece & 1);
          if (!KEYS) tc_fence_after();
          ok = ok && scores(0) && (count < 2 || scores(1));
          const uint32_t acc = tmem + (KEYS ? 384 : 256);
          for (int n = 0; ok && n < count; ++n) {
            const int at = pos + n, sl = at % STAGES, buf = (tiles + n) & 1;
            // the sums of the piece before must have been read
            if (n == 0) ok = piece == 0 || wait(acc_free, (piece - 1) & 1);
            ok = ok && wait(&p_full[buf], ((tiles + n) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t y = dy_cols + sl * 2 * ONE;
            if (KEYS) mma_rows<DS, 64>(tmem + 256, tmem + 64 * buf, y + ONE, n > 0 ? 1u : 0u);
            mma_rows<DS, 64>(acc, tmem + 128 + 64 * buf, y, n > 0 ? 1u : 0u);
            umma_commit(&y_empty[sl]);
            if (n + 2 < count) ok = scores(n + 2);
          }
          umma_commit(acc_done);
          pos += count;
          tiles += count;
          ++piece;
        }
        it = nx;
      }
      // every product issued has completed once `done` flips
      umma_commit(done);
      volatile int no_abort = 0;
      mbar_wait(done, 0, &no_abort, A.err, DEV_ERR_TIMEOUT_TEARDOWN, A.timeout_ns);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int DS, bool KEYS>
cudaError_t go(const BwdArgs& F, int blocks, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  if (blocks == 0) return cudaSuccess;
  cudaError_t e = ensure_smem_attr(k_attn_bwd<DS, KEYS>, SMEM<DS, KEYS>, done);
  if (e != cudaSuccess) return e;
  // the second kernel's launch goes under the end of the first
  e = launch_k(k_attn_bwd<DS, KEYS>, dim3(blocks), dim3(THREADS<KEYS>), SMEM<DS, KEYS>, s, KEYS, F);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

mlora_status launch_attn_bwd(const AttnArgs& Aq, int q_blocks, const AttnArgs& Ak, int k_blocks, int64_t n_tokens,
                             cudaStream_t s) {
  BwdArgs Q{}, K{};
  const AttnArgs& A = Aq;
  Q.a = Aq;
  K.a = Ak;
  Q.a.scale_log2 = K.a.scale_log2 = fabsf(A.scale_log2);
  const struct { TileMap* m; const mlora_heads* t; int heads, cols, rows; } maps[] = {
      {&Q.x0, &A.q, A.hq, 64, 128}, {&Q.x1, &A.dout, A.hq, 64, 128}, {&Q.y0, &A.k, A.hk, 64, 64},
      {&Q.y1, &A.v, A.hk, 64, 64},  {&Q.g0, &A.dq, A.hq, 32, 32},
      {&K.x0, &A.k, A.hk, 64, 128}, {&K.x1, &A.v, A.hk, 64, 128},    {&K.y0, &A.q, A.hq, 64, 64},
      {&K.y1, &A.dout, A.hq, 64, 64}, {&K.g0, &A.dv, A.hk, 32, 32},  {&K.g1, &A.dk, A.hk, 32, 32}};
  for (const auto& m : maps) {
    const mlora_status st = make_tile_map(m.m, *m.t, n_tokens, m.heads, A.D, m.cols, m.rows);
    if (st != MLORA_OK) return st;
  }
  cudaError_t e = A.D <= 64 ? go<1, false>(Q, q_blocks, s) : go<2, false>(Q, q_blocks, s);
  if (e == cudaSuccess) e = A.D <= 64 ? go<1, true>(K, k_blocks, s) : go<2, true>(K, k_blocks, s);
  return e == cudaSuccess ? MLORA_OK : op_cuda_fail(e, "attention backward launch");
}

}  // namespace mlora
