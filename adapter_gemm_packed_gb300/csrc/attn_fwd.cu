// Windowed attention forward on the tensor cores (bf16).
//
// One block per SM walks over its share of the work list.  A piece of work is two query tiles of 128 rows that read
// the same keys ("streams"): two query heads of a group on the same tokens, or, where each query head has keys of
// its own, two neighbouring tiles of one head.  Per key tile of 128 rows and stream:  S = Q K^T (into TMEM),
// softmax (four warps, one row per thread), O += P V with P as the TMEM operand, written over S.  While one stream
// is in its softmax the tensor cores work on the other.  The next piece's loads and first products run under this
// one's last softmax and its output: a block of its own for each piece spent 10,000 of 21,700 cycles on its start,
// first loads and output with four key tiles a piece (sequences of 1024, window 512).
//
// Softmax in base 2: y = |scale| log2(e) S; P = 2^(y - m), l = sum P (fp32).  m is not the running maximum but a
// reference that follows it once it has fallen 32 behind, so that O is rescaled seldom: P is at most 2^32, which
// fp32 and bf16 hold as well as numbers up to 1, and y - m is rounded at 2^-19 at worst.  (Eight behind: 142
// microseconds for 16 sequences of 1024, window 512, 32 heads of 128 on 8, 139 with 32.)  A row that has seen nothing
// keeps m = -inf, l = 0.  P is rounded to bf16 (the tensor cores' operand type; fp32 sums), l sums the values before
// that rounding.
// A negative scale negates Q inside the score product.
//
// 16,384 tokens, window 4096, 64 first tokens, 16 heads of 128 on 4: 324 microseconds, 1.5 PFLOP/s (a plain large product
// of the library: 1.9).  Two streams' tile takes 2870 cycles, 2056 of products at the pipe's nominal rate, which the
// library's product does not reach either.  16 sequences of 1024: 137, 0.8 PFLOP/s, bound by starts, outputs and the
// hidden parts of tiles.
//
// Warps 0-3 and 4-7: the softmax of streams 0 and 1 and their outputs.  Warp 8: TMA loads.  Warp 9: products.
// Warp 10: zeros behind the sequence's end in V, between the load and the product.
#include "attn_tc.cuh"

namespace mlora {
namespace {

constexpr int THREADS = 352;
constexpr int STAGES = 4;          // key and value tiles in flight
constexpr float RESCALE = 32.f;    // how far the reference may fall behind the maximum, in base 2

template <int DS>
constexpr int TILE = 128 * 128 * DS;
template <int DS>
constexpr int SMEM = (2 + STAGES) * TILE<DS> + 8 * OUT_WARP + 256;

struct FwdArgs {
  AttnArgs a;
  TileMap q, k, v, o;
  int pair_heads;      // streams are two heads (else two tiles) ...
  int pairs;           // ... and a group of query heads makes this many pieces of work
};

struct Stream {
  bool on;
  int h, i0;
  KeyTiles kt;
  __device__ __forceinline__ bool active(int t) const {
    return on && t < kt.hi && (t < kt.sink || t >= kt.lo);
  }
};

struct Work {
  int kvh, cnt;      // cnt 0: rows that belong to no sequence
  Stream st[2];
  KeyTiles kt;       // of both streams
};

__device__ __forceinline__ Work decode(const FwdArgs& F, const AttnItem& it) {
  const AttnArgs& A = F.a;
  const int pair = it.sub % F.pairs;
  Work w;
  w.kvh = it.sub / F.pairs;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int g = F.pair_heads ? 2 * pair + s : pair;
    w.st[s].h = w.kvh * A.group + g;
    w.st[s].i0 = it.i0 + (F.pair_heads ? 0 : 128 * s);
    w.st[s].on = g < A.group && w.st[s].i0 < it.len;
    w.st[s].kt = key_tiles(w.st[s].i0, min(w.st[s].i0 + 128, it.len), A.window, A.n_sink, 128);
  }
  w.kt = key_tiles(it.i0, min((w.st[1].on ? w.st[1].i0 : it.i0) + 128, it.len), A.window, A.n_sink, 128);
  w.cnt = it.len ? w.kt.count() : 0;
  return w;
}

struct Bars {
  uint64_t *q_full, *q_empty, *kv_full, *kv_empty, *v_clean, *s_full, *p_full, *o_done, *o_free, *done;
};

// One stream's part of a piece of work, by its four warps.  `tiles` counts the stream's tiles since the start.
// False: a wait has given up.
template <int DS>
__device__ __forceinline__ bool softmax_stream(const FwdArgs& F, const AttnItem& it, const Stream& st, const KeyTiles& kt,
                                               uint32_t tS, uint32_t tO, uint64_t* s_full, uint64_t* p_full,
                                               uint64_t* o_done, uint64_t* o_free, int& tiles, uint8_t* out_buf,
                                               volatile int* abort_flag, int quarter, int lane) {
  const AttnArgs& A = F.a;
  const float c = A.scale_log2;      // > 0 here
  const int r = quarter * 32 + lane, i = st.i0 + r;
  float m = -INFINITY, l = 0.f;
  const int cnt = kt.count();
  for (int n = 0; n < cnt; ++n) {
    const int t = kt.tile(n);
    if (!st.active(t)) continue;
    if (!warp_wait(s_full, tiles & 1, abort_flag, A.err, DEV_ERR_TIMEOUT_EPILOGUE, A.timeout_ns, lane)) return false;
    tc_fence_after();
    uint32_t s[128];
#pragma unroll
    for (int q = 0; q < 4; ++q) tmem_ld32(tS + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * q]));
    tmem_ld_wait();
    const int j0 = t * 128;
    const bool all = j0 + 127 <= st.i0 && (st.i0 + 127 - j0 < A.window || j0 + 127 < A.n_sink);
    if (!all) {
      const int lo = i - A.window + 1 - j0;      // the window's first key
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t seen = bits_below(i - j0 + 1, 32 * q) & (~bits_below(lo, 32 * q) | bits_below(A.n_sink - j0, 32 * q));
#pragma unroll
        for (int u = 0; u < 32; ++u)
          if (!(seen >> u & 1)) s[32 * q + u] = 0xff800000u;      // -inf
      }
    }
    float top4[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      top4[q] = fmaxf(__uint_as_float(s[q]), __uint_as_float(s[4 + q]));
#pragma unroll
      for (int u = 8 + q; u < 128; u += 8) top4[q] = max3(top4[q], __uint_as_float(s[u]), __uint_as_float(s[u + 4]));
    }
    const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * c;
    const bool move = m != -INFINITY && top > m + RESCALE;
    if (__any_sync(0xffffffffu, move)) {
      const float f = move ? ex2(m - top) : 1.f;
      if (!warp_wait(o_done, (tiles - 1) & 1, abort_flag, A.err, DEV_ERR_TIMEOUT_EPILOGUE, A.timeout_ns, lane)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int q = 0; q < 2 * DS; ++q) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * q, o);
        tmem_ld_wait();
#pragma unroll
        for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
        tmem_st32(tO + 32 * q, o);
      }
      tmem_st_wait();
      l *= f;
    }
    if (move || m == -INFINITY) m = top;
    const float ref = m == -INFINITY ? 0.f : m;
    // two halves of 64 keys, so that the product with V starts on the first
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t p[32];
#pragma unroll
      for (int u = 0; u < 64; u += 2) {
        float a = __uint_as_float(s[64 * hf + u]), b = __uint_as_float(s[64 * hf + u + 1]);
        fma2(a, b, c, c, -ref, -ref);
        a = ex2(a), b = ex2(b);
        s[64 * hf + u] = __float_as_uint(a), s[64 * hf + u + 1] = __float_as_uint(b);
        p[u / 2] = pack_bf16x2(a, b);
      }
      tmem_st32(tS + 32 * hf, p);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + hf);
    }
    float sum[4] = {};
#pragma unroll
    for (int u = 0; u < 128; u += 4) {
      add2(sum[0], sum[1], __uint_as_float(s[u]), __uint_as_float(s[u + 1]));
      add2(sum[2], sum[3], __uint_as_float(s[u + 2]), __uint_as_float(s[u + 3]));
    }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    ++tiles;
  }
  if (!warp_wait(o_done, (tiles - 1) & 1, abort_flag, A.err, DEV_ERR_TIMEOUT_EPILOGUE, A.timeout_ns, lane)) return false;
  tc_fence_after();
  uint32_t o[2 * DS][32];
#pragma unroll
  for (int q = 0; q < 2 * DS; ++q) tmem_ld32(tO + 32 * q, o[q]);
  tmem_ld_wait();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(o_free);
  A.saved[stat_at(A.n_stat, st.h, it.stat0 + i)] = i < it.len ? m + log2f(l) : INFINITY;
  const float f = 1.f / l;
  const int first = st.i0 + quarter * 32;
  OutWarp out{&F.o, &A.o, out_buf, it.seq0 + first, st.h, max(0, min(32, it.len - first)), A.D, lane};
#pragma unroll
  for (int q = 0; q < 2 * DS; ++q) scale32(o[q], f);
  // the low bits of the warp's 32 rows, which lie in one piece: through the buffer that the outputs take after them (16
  // sequences of 1024: 132 microseconds, 140 with each lane storing its own)
  if (elect_lane()) bulk_wait_read();
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 2 * DS; ++q) stage_out_low(out_buf, 2 * q, o[q], lane);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (elect_lane()) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                     out_low_at(A, 4 * DS, st.h, it.stat0 + first)),
                 "r"(smem_u32(out_buf)), "r"(DS * 2048)
                 : "memory");
    bulk_commit();
  }
#pragma unroll
  for (int q = 0; q < 2 * DS; q += 2) out.put<2, true>(32 * q, &o[q]);
  return true;
}

template <int DS>
__global__ void __launch_bounds__(THREADS, 1) k_attn_fwd(const __grid_constant__ FwdArgs F) {
  griddep_wait();
  extern __shared__ __align__(1024) uint8_t smem[];
  const AttnArgs& A = F.a;
  const int k_first = A.first[blockIdx.x], k_end = A.first[blockIdx.x + 1];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (!smem_aligned(smem, A.err)) return;
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * TILE<DS>;
  uint8_t* sOut = sKV + STAGES * TILE<DS>;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sOut + 8 * OUT_WARP);
  Bars B;
  B.q_full = bars, B.q_empty = bars + 1, B.kv_full = bars + 2, B.kv_empty = B.kv_full + STAGES;
  B.v_clean = B.kv_empty + STAGES, B.s_full = B.v_clean + STAGES, B.p_full = B.s_full + 2, B.o_done = B.p_full + 4;
  B.o_free = B.o_done + 2, B.done = B.o_free + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(B.done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(slot + 1);
  if (tid == 0) {
    mbar_init(B.q_full, 1);
    mbar_init(B.q_empty, 1);
    for (int i = 0; i < STAGES; ++i) mbar_init(&B.kv_full[i], 1), mbar_init(&B.kv_empty[i], 1), mbar_init(&B.v_clean[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&B.s_full[i], 1), mbar_init(&B.o_done[i], 1), mbar_init(&B.o_free[i], 4);
    for (int i = 0; i < 4; ++i) mbar_init(&B.p_full[i], 4);
    mbar_init(B.done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(slot, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  // columns: S of stream s at 128 s, O at 256 + 128 s

  AttnItem it = A.items[k_first];
  auto next_item = [&](int k) { return k + 1 < k_end ? A.items[k + 1] : it; };

  if (warp < 8) {
    const int s = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    int tiles = 0;
    for (int k = k_first; k < k_end; ++k) {
      const AttnItem nx = next_item(k);
      const Work w = decode(F, it);
      const Stream mine = s ? w.st[1] : w.st[0];
      if (w.cnt == 0)
        zero_out_rows(A.o, it, A.hq, A.D, tid, 256);
      else if (mine.on && !softmax_stream<DS>(F, it, mine, w.kt, tmem + 128 * s + lanes, tmem + 256 + 128 * s + lanes,
                                              &B.s_full[s], &B.p_full[2 * s], &B.o_done[s], &B.o_free[s], tiles,
                                              sOut + warp * OUT_WARP, abort_flag, quarter, lane))
        break;
      it = nx;
    }
    if (elect_lane()) bulk_wait_all();      // no store may still be reading shared memory when the block ends
    __syncwarp();
  } else if (warp == 8) {
    if (elect_lane()) {
      int pos = 0, nq = 0;
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t parity) {
        return mbar_wait(b, parity, abort_flag, A.err, DEV_ERR_TIMEOUT_PRODUCER, A.timeout_ns);
      };
      for (int k = k_first; ok && k < k_end; ++k) {
        const AttnItem nx = next_item(k);
        const Work w = decode(F, it);
        if (w.cnt) {
          ok = nq == 0 || wait(B.q_empty, (nq - 1) & 1);
          if (!ok) break;
          mbar_arrive_expect_tx(B.q_full, (w.st[1].on ? 2 : 1) * TILE<DS>);
#pragma unroll
          for (int s = 0; s < 2; ++s)
            if (w.st[s].on) load_tile<DS, 128>(sQ + s * TILE<DS>, F.q, B.q_full, it.seq0 + w.st[s].i0, w.st[s].h);
          ++nq;
          // the next piece's queries, and its keys and values from the first on, towards L2
          if (k + 1 < k_end && nx.len) {
            const Work v = decode(F, nx);
#pragma unroll
            for (int s = 0; s < 2; ++s)
              if (v.st[s].on) prefetch_tile<DS, 128>(F.q, nx.seq0 + v.st[s].i0, v.st[s].h);
            prefetch_tile<DS, 128>(F.k, nx.seq0 + v.kt.tile(0) * 128, v.kvh);
            prefetch_tile<DS, 128>(F.v, nx.seq0 + v.kt.tile(0) * 128, v.kvh);
          }
          for (int n = 0; ok && n < w.cnt; ++n) {
            const int row = it.seq0 + w.kt.tile(n) * 128;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              const int sl = pos % STAGES;
              ok = ok && wait(&B.kv_empty[sl], ((pos / STAGES) & 1) ^ 1u);
              if (!ok) break;
              mbar_arrive_expect_tx(&B.kv_full[sl], TILE<DS>);
              load_tile<DS, 128>(sKV + sl * TILE<DS>, kv ? F.v : F.k, &B.kv_full[sl], row, w.kvh);
              ++pos;
            }
          }
        }
        it = nx;
      }
      // bounded: no copy may still be writing shared memory when the block ends, whoever gave up and whenever
      volatile int no_abort = 0;
      if (nq) mbar_wait(B.q_full, (nq - 1) & 1, &no_abort, A.err, DEV_ERR_TIMEOUT_TEARDOWN, A.timeout_ns);
      for (int q = pos > STAGES ? pos - STAGES : 0; q < pos; ++q)
        mbar_wait(&B.kv_full[q % STAGES], (q / STAGES) & 1, &no_abort, A.err, DEV_ERR_TIMEOUT_TEARDOWN, A.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 10) {
    // The last key tile may reach past the sequence's end: what lies there becomes zero in V before the product
    // sums over it (zero times NaN is NaN).  Every V tile goes through here, which keeps the warp in step.
    int pos = 0;
    bool ok = true;
    for (int k = k_first; ok && k < k_end; ++k) {
      const AttnItem nx = next_item(k);
      const Work w = decode(F, it);
      for (int n = 0; n < w.cnt; ++n, pos += 2) {
        const int vp = pos + 1, vs = vp % STAGES, row = w.kt.tile(n) * 128;
        ok = warp_wait(&B.kv_full[vs], (vp / STAGES) & 1, abort_flag, A.err, DEV_ERR_TIMEOUT_PRODUCER, A.timeout_ns, lane);
        if (!ok) break;
        if (row + 128 > it.len) zero_rows_from<DS, 128>(sKV + vs * TILE<DS>, it.len - row, lane);
        if (lane == 0) mbar_arrive(&B.v_clean[vs]);
      }
      it = nx;
    }
  } else {
    if (elect_lane()) {
      const uint32_t idesc_s = idesc_bf16(128, 128, false, false) | (A.scale < 0.f ? IDESC_NEG_A : 0u);
      const uint64_t dq = desc_rows(sQ), dk = desc_rows(sKV), dv = desc_cols<128>(sKV);
      constexpr uint64_t STEP = TILE<DS> / 16;
      auto wait = [&](uint64_t* b, uint32_t parity) {
        return mbar_wait(b, parity, abort_flag, A.err, DEV_ERR_TIMEOUT_MMA, A.timeout_ns);
      };
      int pos = 0, nq = 0;
      int ps[2] = {0, 0};        // tiles done, per stream
      int outs[2] = {0, 0};      // pieces of work, per stream
      bool ok = true;
      for (int k = k_first; ok && k < k_end; ++k) {
        const AttnItem nx = next_item(k);
        const Work w = decode(F, it);
        const int cnt = w.cnt;
        if (cnt) {
          const int k0 = pos % STAGES;
          bool act[2] = {w.st[0].active(w.kt.tile(0)), w.st[1].active(w.kt.tile(0))};
          bool first[2] = {true, true};
          ok = wait(B.q_full, nq & 1) && wait(&B.kv_full[k0], (pos / STAGES) & 1);
          if (!ok) break;
          ++nq;
#pragma unroll
          for (int s = 0; s < 2; ++s)
            if (act[s]) {
              mma_scores<DS, 128, 128>(tmem + 128 * s, dq + s * STEP, dk + k0 * STEP, idesc_s);
              umma_commit(&B.s_full[s]);
            }
          umma_commit(&B.kv_empty[k0]);
          if (cnt == 1) umma_commit(B.q_empty);
          for (int n = 0; n < cnt; ++n, pos += 2) {
            const int vp = pos + 1, kp = pos + 2, vs = vp % STAGES, ks = kp % STAGES;
            const bool more = n + 1 < cnt;
            const int t1 = w.kt.tile(n + 1);
            const bool next[2] = {more && w.st[0].active(t1), more && w.st[1].active(t1)};
            ok = wait(&B.v_clean[vs], (vp / STAGES) & 1) && (!more || wait(&B.kv_full[ks], (kp / STAGES) & 1));
            if (!ok) break;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              if (act[s]) {
                // O of the piece before must have been read
                ok = (!first[s] || outs[s] == 0 || wait(&B.o_free[s], (outs[s] - 1) & 1)) && wait(&B.p_full[2 * s], ps[s] & 1);
                if (!ok) break;
                tc_fence_after();
                mma_rows<DS, 128, 0, 4>(tmem + 256 + 128 * s, tmem + 128 * s, dv + vs * STEP, first[s] ? 0u : 1u);
                ok = wait(&B.p_full[2 * s + 1], ps[s] & 1);
                if (!ok) break;
                tc_fence_after();
                mma_rows<DS, 128, 4, 8>(tmem + 256 + 128 * s, tmem + 128 * s, dv + vs * STEP, 1u);
                umma_commit(&B.o_done[s]);
                if (first[s]) ++outs[s];
                first[s] = false;
                ++ps[s];
              }
              if (s == 1) umma_commit(&B.kv_empty[vs]);
              if (next[s]) {
                mma_scores<DS, 128, 128>(tmem + 128 * s, dq + s * STEP, dk + ks * STEP, idesc_s);
                umma_commit(&B.s_full[s]);
              }
            }
            if (!ok) break;
            if (more) umma_commit(&B.kv_empty[ks]);
            if (n + 2 == cnt) umma_commit(B.q_empty);      // the last score products are under way
            act[0] = next[0], act[1] = next[1];
          }
        }
        it = nx;
      }
      // every product issued has completed once `done` flips
      umma_commit(B.done);
      volatile int no_abort = 0;
      mbar_wait(B.done, 0, &no_abort, A.err, DEV_ERR_TIMEOUT_TEARDOWN, A.timeout_ns);
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

template <int DS>
cudaError_t go(const FwdArgs& F, int blocks, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = ensure_smem_attr(k_attn_fwd<DS>, SMEM<DS>, done);
  if (e != cudaSuccess) return e;
  return launch_k(k_attn_fwd<DS>, dim3(blocks), dim3(THREADS), SMEM<DS>, s, false, F);
}

}  // namespace

// Rows per item of the forward's work list: two streams of 128 rows, side by side or on the same rows.
int attn_fwd_rows(int group) { return group > 1 ? 128 : 256; }
// Pieces of work that a group of query heads makes on a tile.
int attn_fwd_pairs(int group) { return group > 1 ? (group + 1) / 2 : 1; }

mlora_status launch_attn_fwd(const AttnArgs& A, int blocks, int64_t n_tokens, cudaStream_t s) {
  FwdArgs F{};
  F.a = A;
  // a scale of zero would make 0 * -inf of a hidden key; with 2^-100 every visible key weighs the same too
  F.a.scale_log2 = A.scale == 0.f ? 0x1p-100f : fabsf(A.scale_log2);
  F.pair_heads = A.group > 1;
  F.pairs = attn_fwd_pairs(A.group);
  mlora_status st = make_tile_map(&F.q, A.q, n_tokens, A.hq, A.D, 64, 128);
  if (st == MLORA_OK) st = make_tile_map(&F.k, A.k, n_tokens, A.hk, A.D, 64, 128);
  if (st == MLORA_OK) st = make_tile_map(&F.v, A.v, n_tokens, A.hk, A.D, 64, 128);
  if (st == MLORA_OK) st = make_tile_map(&F.o, A.o, n_tokens, A.hq, A.D, 32, 32);
  if (st != MLORA_OK || blocks == 0) return st;
  const cudaError_t e = A.D <= 64 ? go<1>(F, blocks, s) : go<2>(F, blocks, s);
  if (e != cudaSuccess) return op_cuda_fail(e, "attention forward launch");
  count_launches(1);
  return MLORA_OK;
}

}  // namespace mlora
