// Pieces of the tensor-core attention kernels (bf16): tensor maps of head tensors, operand descriptors,
// tcgen05 products whose first operand lies in TMEM, and the zero fill behind a sequence's end.
//
// A tile is R rows of one head, in DS slices of 64 columns: slice s at s * R * 128 bytes, each a stack of
// 128-byte-swizzled 8-row atoms, which is what a TMA box of 64 columns x R rows writes.  The same bytes serve as
// a K-major operand (rows x head_dim, for the score products) and as an MN-major one (head_dim x rows, for the
// products that sum over the rows).  Columns past head_dim are zero (outside of the tensor map).
#pragma once
#include "attention.cuh"

namespace mlora {

struct TileMap {
  CUtensorMap map;
  int by_head;      // coordinates are (column, token, head) instead of (column, head, token)
};

// 3-D map of a head tensor with a box of `cols` columns (64, 128-byte swizzle, or 32, 64-byte swizzle) and `rows`
// tokens of one head; the two outer dimensions are ordered by their strides.
inline mlora_status make_tile_map(TileMap* out, const mlora_heads& t, int64_t n_tokens, int n_heads, int head_dim,
                                  int cols, int rows) {
  auto fn = encode_fn();
  if (!fn) return op_fail(MLORA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  // the stride of a dimension with one element is never used
  uint64_t rs = static_cast<uint64_t>(t.row_stride) * 2, hs = static_cast<uint64_t>(t.head_stride) * 2;
  if (n_heads == 1) hs = static_cast<uint64_t>((head_dim + 7) / 8) * 16;
  if (n_tokens == 1) rs = hs * n_heads;
  out->by_head = hs > rs;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(n_heads),
                        static_cast<cuuint64_t>(n_tokens)};
  cuuint64_t strides[2] = {hs, rs};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(cols), 1, static_cast<cuuint32_t>(rows)};
  if (out->by_head) {
    std::swap(dims[1], dims[2]);
    std::swap(strides[0], strides[1]);
    std::swap(box[1], box[2]);
  }
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(&out->map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, t.data, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE,
                        cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    char buf[160];
    snprintf(buf, sizeof buf, "cuTensorMapEncodeTiled failed (%d) for a head tensor", static_cast<int>(r));
    return op_fail(MLORA_ERR_CUDA, buf);
  }
  return MLORA_OK;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// A tile of R rows from token `row` on of head h (rows past the tensor's end arrive as zero).
template <int DS, int R>
__device__ __forceinline__ void load_tile(uint8_t* dst, const TileMap& m, uint64_t* bar, int row, int h) {
  const int y = m.by_head ? row : h, z = m.by_head ? h : row;
#pragma unroll
  for (int s = 0; s < DS; ++s) tma_load_3d(dst + s * R * 128, &m.map, bar, s * 64, y, z);
}

// The same tile into L2 only, ahead of its load.
template <int DS, int R>
__device__ __forceinline__ void prefetch_tile(const TileMap& m, int row, int h) {
  const int y = m.by_head ? row : h, z = m.by_head ? h : row;
#pragma unroll
  for (int s = 0; s < DS; ++s)
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(&m.map)),
                 "r"(s * 64), "r"(y), "r"(z)
                 : "memory");
}

// The dynamic shared memory of the attention kernels holds 1024-byte swizzle atoms from its first byte on; they
// declare that alignment, and do nothing but say so should it not be given.
__device__ __forceinline__ bool smem_aligned(const uint8_t* smem, int* err) {
  if ((smem_u32(smem) & 1023) == 0) return true;
  atomicCAS(err, 0, DEV_ERR_TIMEOUT_TEARDOWN);
  return false;
}

// Rows [from, R) of a tile to zero, by one warp, before an MMA sums over them: behind a sequence's end there may
// be anything, and zero times NaN is NaN.
template <int DS, int R>
__device__ __forceinline__ void zero_rows_from(uint8_t* tile, int from, int lane) {
#pragma unroll
  for (int s = 0; s < DS; ++s)
    for (int o = from * 128 + lane * 16; o < R * 128; o += 512)
      *reinterpret_cast<uint4*>(tile + s * R * 128 + o) = make_uint4(0, 0, 0, 0);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// D[tmem] (+)= A[tmem] * B[smem desc]: A is 128 rows (lanes) of bf16 pairs, one 32-bit column per two k.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

constexpr uint32_t IDESC_NEG_A = 1u << 13;      // the product with A negated

// The products are issued by one thread, whose warp shares its scheduler with two warps of the softmax; the tensor
// cores hold only a few products in their queue, so every instruction between two of them counts.  The thread is
// the one that elect.sync names: only then does the compiler know that a branch has one thread, and keeps the
// products' operands in uniform registers without asking.  (A dQ step's 20 products with both other warps of
// the scheduler always ready to issue: 5419 cycles from a branch on lane 0, 1091 from an elected one; 1042 with
// nothing else running.)  Descriptors are made once, and a step inside a tile is an addition to the address
// field (in units of 16 bytes).
__device__ __forceinline__ bool elect_lane() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// Descriptors of a tile of R rows: as rows of a score product, and as what the rows are summed into.
__device__ __forceinline__ uint64_t desc_rows(const void* tile) { return smem_desc(smem_u32(tile), 16, 1024); }
template <int R>
__device__ __forceinline__ uint64_t desc_cols(const void* tile) { return smem_desc(smem_u32(tile), R * 128, 1024); }

// D (128 x N) = A (128 rows, RA-row tile) B^T (N rows, RB-row tile), summed over head_dim.
template <int DS, int RA, int RB>
__device__ __forceinline__ void mma_scores(uint32_t d_tmem, uint64_t da, uint64_t db, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < DS * 4; ++k)
    umma_bf16(d_tmem, da + (k / 4) * RA * 8 + (k % 4) * 2, db + (k / 4) * RB * 8 + (k % 4) * 2, idesc, k > 0 ? 1u : 0u);
}

// The same with A in TMEM (a row per lane, 32 DS columns).
template <int DS, int RB>
__device__ __forceinline__ void mma_scores_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t db, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < DS * 4; ++k)
    umma_bf16_ts(d_tmem, a_tmem + k * 8, db + (k / 4) * RB * 8 + (k % 4) * 2, idesc, k > 0 ? 1u : 0u);
}

// D (128 x 64 DS) (+)= P (128 x R, bf16 in TMEM) B (R-row tile), summed over the tile's rows [16 K0, 16 K1).
template <int DS, int R, int K0 = 0, int K1 = R / 16>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint32_t p_tmem, uint64_t db, uint32_t accumulate) {
  constexpr uint32_t idesc = idesc_bf16(128, 64 * DS, false, true);
#pragma unroll
  for (int k = K0; k < K1; ++k)
    umma_bf16_ts(d_tmem, p_tmem + k * 8, db + k * 128, idesc, k > 0 ? 1u : accumulate);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]),
      "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// (x, y) = (x, y) * (a, b) + (c, d), two products in one instruction
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float c, float d) {
  asm("{\n\t.reg .b64 u, v, w;\n\t"
      "mov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tmov.b64 w, {%4, %5};\n\t"
      "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b), "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 u, v;\n\t"
      "mov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
      "add.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ void mul2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 u, v;\n\t"
      "mov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
      "mul.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

// bits c of [0, 32) with base + c < n
__device__ __forceinline__ uint32_t bits_below(int n, int base) {
  const int k = n - base;
  return k <= 0 ? 0u : (k >= 32 ? 0xffffffffu : (1u << k) - 1u);
}

// A whole warp waits for a barrier and agrees on the outcome (after a first look, one lane polls).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err, int code,
                                          unsigned long long timeout_ns, int lane) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  int ok = 1;
  if (lane == 0) ok = mbar_wait(bar, parity, abort_flag, err, code, timeout_ns);
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// v * f for 32 values
__device__ __forceinline__ void scale32(uint32_t (&v)[32], float f) {
#pragma unroll
  for (int u = 0; u < 32; u += 2) {
    float a = __uint_as_float(v[u]), b = __uint_as_float(v[u + 1]);
    mul2(a, b, f, f);
    v[u] = __float_as_uint(a), v[u + 1] = __float_as_uint(b);
  }
}
// Two values as bf16, to the nearest; AWAY: ties away from zero, otherwise to even.  (Rounding by adding given bits below
// the last place and cutting off: with half a place for those bits it is rounding to the nearest.)
template <bool AWAY>
__device__ __forceinline__ uint32_t pack2(uint32_t lo, uint32_t hi) {
  if constexpr (!AWAY) return pack_bf16x2(__uint_as_float(lo), __uint_as_float(hi));
  uint32_t p;
  asm("cvt.rs.bf16x2.f32 %0, %1, %2, %3;" : "=r"(p) : "f"(__uint_as_float(hi)), "f"(__uint_as_float(lo)), "r"(0x80008000u));
  return p;
}
// columns [u, u + 8) of 32 as bf16
template <bool AWAY>
__device__ __forceinline__ uint4 pack8(const uint32_t (&v)[32], int u) {
  return make_uint4(pack2<AWAY>(v[u], v[u + 1]), pack2<AWAY>(v[u + 2], v[u + 3]), pack2<AWAY>(v[u + 4], v[u + 5]),
                    pack2<AWAY>(v[u + 6], v[u + 7]));
}

// A warp's 32 rows of an output tile (a row per lane), 32 columns at a time: through two buffers of 2 KB in shared
// memory (64-byte swizzle: the lanes' 16-byte stores hit every bank once) and TMA stores of 32 x 32, which
// write whole lines where a lane storing its own row would touch 32 of them with each instruction.  Columns past
// head_dim are clipped by the map.  Rows past the sequence's end must not be written: a warp with such rows
// stores the others itself.
constexpr int OUT_BUF = 32 * 64, OUT_WARP = 2 * OUT_BUF;
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

struct OutWarp {
  const TileMap* map;
  const mlora_heads* t;
  uint8_t* buf;
  int row0, h, rows, D, lane;      // the warp's first token, its head, rows that exist (32 or fewer)
  // N (one or two) runs of 32 columns from c0 on
  template <int N, bool AWAY = false>
  __device__ __forceinline__ void put(int c0, const uint32_t (*v)[32]) {
    if (rows < 32) {
      if (lane < rows) {
        __nv_bfloat16* y = head_row<__nv_bfloat16>(*t, row0 + lane, h) + c0;
#pragma unroll
        for (int u = 0; u < 32 * N; u += 8)
          if (c0 + u < D) *reinterpret_cast<uint4*>(y + u) = pack8<AWAY>(v[u / 32], u % 32);      // D is a multiple of 8
      }
      return;
    }
    if (elect_lane()) bulk_wait_read();      // the stores before this one have read the buffers
    __syncwarp();
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(buf + k * OUT_BUF + lane * 64 + ((c ^ (lane >> 1 & 3)) << 4)) = pack8<AWAY>(v[k], 8 * c);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (elect_lane()) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (c0 + 32 * k < D)
          asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                           reinterpret_cast<uint64_t>(&map->map)),
                       "r"(smem_u32(buf + k * OUT_BUF)), "r"(c0 + 32 * k), "r"(map->by_head ? row0 : h),
                       "r"(map->by_head ? h : row0)
                       : "memory");
      bulk_commit();
    }
  }
};

// The outputs' low bits.  delta = rowsum(dO O) wants O as the fp32 sums gave it: the error of a rounded O is the
// same for all of a row's score gradients and does not average out.  Beside each bf16 output the forward keeps a byte:
// the difference of its fp32 pattern to the rounded one's in units of 2^8 of the last place, to the nearest, 127 at most.
// That leaves an error of either sign, at most 2^-16 of the output (2^-15 just below a tie), and an output that lies
// within half a unit of a bf16 number comes back as that number (a peaked row's dP and delta nearly cancel).  Rows as in the statistics, 32 rows x 16 columns (bytes)
// a run, so that a warp's rows are read and written in whole lines.
__device__ __forceinline__ uint8_t* out_low_at(const AttnArgs& A, int chunks, int h, long long s) {
  const long long r = h * A.n_stat + s;
  return A.out_low + (r / 32) * chunks * 512 + (r % 32) * 16;      // + 512 per 16 columns
}
// the value of a rounded output (its bits in the upper half of hi) with byte k of l: the byte in its place, its sign
// above it
__device__ __forceinline__ float out_whole(uint32_t hi, uint32_t l, int k) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(l), "r"(0u), "r"((8 + k) * 0x1100 + k * 0x10 + 4));
  return __uint_as_float(hi + d);
}
// The bytes of 32 outputs, two runs from run c on, of this lane's row, into the warp's buffer in shared memory: the
// differences of two outputs (l), half a unit added, the upper byte kept; differences that this would carry past 127 units
// stop there (0x7f7e: the lower one's sum may carry into the upper one).  Outputs round ties away from zero: with ties to
// even a lower half of 0x8000 would not say which way.  16 sequences of 1024: 142.3 microseconds with the bytes cut off
// and ties to even, 143.8 so (the same box in turn).
__device__ __forceinline__ void stage_out_low(uint8_t* buf, int c, const uint32_t (&v)[32], int lane) {
  const auto bytes = [&](int e) {
    const uint32_t l = __byte_perm(v[e], v[e + 1], 0x5410);
    return __vmins2(l, 0x7f7e7f7fu) + 0x00800080u;
  };
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = __byte_perm(bytes(16 * k + 4 * u), bytes(16 * k + 4 * u + 2), 0x7531);
    *reinterpret_cast<uint4*>(buf + (c + k) * 512 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Zeros into a run of rows that belong to no sequence, for all heads.
__device__ __forceinline__ void zero_out_rows(const mlora_heads& t, const AttnItem& it, int heads, int D, int tid,
                                              int threads) {
  const int per = D / 8, row = per * heads;
  for (int e = tid; e < it.i0 * row; e += threads)
    *reinterpret_cast<uint4*>(head_row<__nv_bfloat16>(t, static_cast<long long>(it.seq0) + e / row, e % row / per) +
                              e % per * 8) = make_uint4(0, 0, 0, 0);
}

}  // namespace mlora
