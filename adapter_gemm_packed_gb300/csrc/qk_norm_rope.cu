// Norms of queries and keys for each head, with the position rotation in the same pass, and the
// gradient of both.
//
// For a head vector x of D elements with weight w:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = n w,
//   out = R(pos) y: pair (a, b) of the first rot_dim elements -> (a c - b s, b c + a s).
// Backward, given g_out: g = R(pos)^T g_out (the rotation by the opposite angle), h = g w,
//   dx = r (h - n mean(h n)),  dw = sum over tokens and heads of g n.
// Both sums of the backward (x^2 and h x) come from x itself, so the forward saves nothing and the
// backward reads x and g_out once: mean(h n) = r sum(h x) / D.
//
// Everything between the loads and the stores is fp32; each output is rounded once to the tensors' type.
//
// Memory-bound: a lane holds two runs of a head vector, 16 bytes each where the sizes allow, and has several heads'
// runs of the next round on their way (asynchronous copies into shared memory) while it works on this one's, which is
// what keeps enough bytes in flight.  A block takes either queries or keys, so its lanes keep one set of weights (and,
// backward, of weight gradients) in registers.  71,680 tokens, 32 + 8 heads of 128 bf16: forward 230 microseconds, 6.4
// TB/s; backward 349, 6.3 TB/s (237 and 394 with the loads straight into registers).
#include "entry.cuh"

namespace mlora {
namespace {

constexpr int THREADS = 256;
constexpr int MAX_PART_BLOCKS = 1024;    // rows of partial weight gradients

struct Side {                // the queries, or the keys
  mlora_heads x, g, out;     // g: backward, the gradient of the output; out: the output, or dx
  const float* w;
  int H;
  int hb;                    // heads that a group of lanes has in flight at once
  int share;                 // groups of a block that share a token
  int blocks;
};

struct RopeArgs {
  long long n_tokens;
  int D, rot, max_pos;
  float eps;
  const float *cos, *sin;
  const int* pos;
  Side side[2];
  float* part;               // backward: [blocks][D] partial weight gradients, or null
};

// R elements in memory
template <typename T, int R>
struct Chunk;
template <>
struct Chunk<float, 4> {
  typedef float4 Raw;
  static __device__ __forceinline__ void unpack(const Raw& t, float (&v)[4]) { v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w; }
  static __device__ __forceinline__ Raw pack(const float (&v)[4]) { return make_float4(v[0], v[1], v[2], v[3]); }
};
__device__ __forceinline__ float bf16_low(uint32_t t) { return __uint_as_float(t << 16); }
__device__ __forceinline__ float bf16_high(uint32_t t) { return __uint_as_float(t & 0xffff0000u); }
template <>
struct Chunk<__nv_bfloat16, 4> {
  typedef uint2 Raw;
  static __device__ __forceinline__ void unpack(const Raw& t, float (&v)[4]) {
    v[0] = bf16_low(t.x), v[1] = bf16_high(t.x), v[2] = bf16_low(t.y), v[3] = bf16_high(t.y);
  }
  static __device__ __forceinline__ Raw pack(const float (&v)[4]) {
    return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
};
template <>
struct Chunk<__nv_bfloat16, 8> {
  typedef uint4 Raw;
  static __device__ __forceinline__ void unpack(const Raw& t, float (&v)[8]) {
    v[0] = bf16_low(t.x), v[1] = bf16_high(t.x), v[2] = bf16_low(t.y), v[3] = bf16_high(t.y);
    v[4] = bf16_low(t.z), v[5] = bf16_high(t.z), v[6] = bf16_low(t.w), v[7] = bf16_high(t.w);
  }
  static __device__ __forceinline__ Raw pack(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
};

template <int R>
__device__ __forceinline__ void load_f32(const float* p, float (&v)[R]) {
#pragma unroll
  for (int i = 0; i < R; i += 4) {
    const float4 t = *reinterpret_cast<const float4*>(p + i);
    v[i] = t.x, v[i + 1] = t.y, v[i + 2] = t.z, v[i + 3] = t.w;
  }
}

// A lane holds R pairs of one head vector, as a[R] and b[R].  Rotated pairs are (i, i + rot/2), or
// neighbours when INTER; the pairs past rot_dim (not rotated) split the rest of the vector the same way.
// Either way the 2 R elements are two runs of R: [oa, oa + R) and [ob, ob + R).
struct Lane {
  int oa, ob, ci;     // element offsets, and the first column of cos / sin (-1: not rotated)
  bool on;
};

template <int R, bool INTER>
__device__ __forceinline__ Lane lane_of(const RopeArgs& A, int l) {
  Lane L;
  const int p = R * l, half = A.rot / 2;
  L.on = 2 * p < A.D;
  L.ci = p < half ? p : -1;
  if (INTER) {
    L.oa = 2 * p, L.ob = 2 * p + R;
  } else if (p < half) {
    L.oa = p, L.ob = p + half;
  } else {
    L.oa = A.rot + (p - half), L.ob = L.oa + (A.D - A.rot) / 2;
  }
  if (!L.on) L.oa = L.ob = 0, L.ci = -1;
  return L;
}

// (run at oa, run at ob) turned by the angles (c, s), or back by them
template <int R, bool INTER, bool BACK>
__device__ __forceinline__ void rotate(float (&u)[R], float (&v)[R], const float (&c)[R], const float (&s)[R]) {
  float x[2 * R];
#pragma unroll
  for (int i = 0; i < R; ++i) x[i] = u[i], x[R + i] = v[i];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : R + i;
    const float a = x[ia], b = x[ib];
    x[ia] = BACK ? a * c[i] + b * s[i] : a * c[i] - b * s[i];
    x[ib] = BACK ? b * c[i] - a * s[i] : b * c[i] + a * s[i];
  }
#pragma unroll
  for (int i = 0; i < R; ++i) u[i] = x[i], v[i] = x[R + i];
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, L);
  return v;
}

template <int R>
__device__ __forceinline__ void load_table(const RopeArgs& A, const Lane& ln, int pos, float (&c)[R], float (&s)[R]) {
  // a position outside of the tables gives NaN in the whole head vector, never a read outside of them
  const bool ok = static_cast<unsigned>(pos) < static_cast<unsigned>(A.max_pos);
  if (ok && ln.ci >= 0) {
    const long long at = static_cast<long long>(pos) * (A.rot / 2) + ln.ci;
    load_f32(A.cos + at, c);
    load_f32(A.sin + at, s);
  } else {
    const float nan = __int_as_float(0x7fffffff);
#pragma unroll
    for (int i = 0; i < R; ++i) c[i] = ok ? 1.f : nan, s[i] = ok ? 0.f : nan;
  }
}

// One lane's own 8 or 16 bytes into shared memory; zeros where not ok.  Neighbouring pairs make a lane's two runs lie
// side by side, in one 32-byte sector: then by way of L1, which fetches it once.
template <bool INTER, typename Raw>
__device__ __forceinline__ void copy_own(Raw* dst, const void* src, bool ok) {
  if constexpr (sizeof(Raw) == 16 && INTER) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0) : "memory");
  } else if constexpr (sizeof(Raw) == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0) : "memory");
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 8 : 0) : "memory");
  }
}

template <bool BWD>
constexpr int HEADS = BWD ? 2 : 4;       // heads of a token that a group of lanes takes at once
constexpr int STAGES = 2;              // (three: no faster)
template <typename T, int R, bool BWD>
constexpr int RING = STAGES * HEADS<BWD> * (BWD ? 4 : 2) * THREADS * static_cast<int>(sizeof(typename Chunk<T, R>::Raw));

// One group of L lanes per head vector, HEADS heads of a token at a time; blocks walk over the tokens.  BWD: the gradient.
// A lane's elements come through a ring of its own in shared memory, a round ahead of their use: no other thread reads
// them, so its own wait for its copies is all the order there is.
template <typename T, int R, int L, bool INTER, bool BWD>
__global__ void __launch_bounds__(THREADS, 2) k_norm_rope(const RopeArgs A) {
  griddep_wait();
  typedef Chunk<T, R> Ch;
  typedef typename Ch::Raw Raw;
  extern __shared__ float4 smem4[];
  constexpr int GROUPS = THREADS / L, HB = HEADS<BWD>, RUNS = HB * (BWD ? 4 : 2);
  const int o = blockIdx.x >= A.side[0].blocks;      // the queries' blocks, then the keys'
  const Side& S = A.side[o];
  const int blk = blockIdx.x - (o ? A.side[0].blocks : 0);
  const int grp = threadIdx.x / L, per = GROUPS / S.share, slot = grp / S.share, turn = grp - slot * S.share;
  const Lane ln = lane_of<R, INTER>(A, threadIdx.x % L);
  const float inv = 1.f / A.D;
  float wu[R], wv[R], dwu[R] = {}, dwv[R] = {};
  load_f32(S.w + ln.oa, wu);
  load_f32(S.w + ln.ob, wv);
  const bool mine = ln.on && slot < per;
  const long long step = static_cast<long long>(S.blocks) * per;
  const T* const x = static_cast<const T*>(S.x.data);
  const T* const g = static_cast<const T*>(S.g.data);
  T* const out = static_cast<T*>(S.out.data);
  Raw* const ring = reinterpret_cast<Raw*>(smem4) + threadIdx.x;
  const long long base0 = static_cast<long long>(blk) * per;

  // rounds: the block's tokens, and for each the heads in turns (more than one only where there are more than a block
  // has groups for); the same number for every lane of a block
  const int wide = S.share * S.hb;
  struct At {
    long long base;
    int h;
  };
  auto next = [&](At& a) {
    a.h += wide;
    if (a.h >= S.H) a.h = 0, a.base += step;
  };
  auto issue = [&](const At& a, int stage) {
    const long long row = a.base + slot;
    const bool live = mine && row < A.n_tokens;
    Raw* const to = ring + stage * RUNS * THREADS;
#pragma unroll
    for (int i = 0; i < HB; ++i) {
      if (i >= S.hb) break;
      const int h = a.h + turn * S.hb + i;
      const bool ok = live && h < S.H;
      const T* p = ok ? x + row * S.x.row_stride + h * S.x.head_stride : x;
      copy_own<INTER>(to + (2 * i) * THREADS, p + ln.oa, ok);
      copy_own<INTER>(to + (2 * i + 1) * THREADS, p + ln.ob, ok);
      if (BWD) {
        const T* q = ok ? g + row * S.g.row_stride + h * S.g.head_stride : g;
        copy_own<INTER>(to + (2 * HB + 2 * i) * THREADS, q + ln.oa, ok);
        copy_own<INTER>(to + (2 * HB + 2 * i + 1) * THREADS, q + ln.ob, ok);
      }
    }
  };
  auto position = [&](long long base) { return mine && base + slot < A.n_tokens ? A.pos[base + slot] : 0; };
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

  At use{base0, 0}, ahead = use;
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) {
    if (ahead.base < A.n_tokens) issue(ahead, k), next(ahead);
    commit();
  }
  int pos = position(base0);
  float c[R], s[R];
  load_table(A, ln, pos, c, s);
  pos = position(base0 + step);
  for (int k = 0; use.base < A.n_tokens; ++k) {
    const long long row = use.base + slot;
    const bool live = mine && row < A.n_tokens;
    if (ahead.base < A.n_tokens) issue(ahead, (k + STAGES - 1) % STAGES), next(ahead);
    commit();
    const int h0 = use.h + turn * S.hb;
    const long long base = use.base;
    next(use);
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    const Raw* const from = ring + k % STAGES * RUNS * THREADS;
#pragma unroll
    for (int i = 0; i < HB; ++i) {
      if (i >= S.hb) break;
      float u[R], v[R], ss = 0.f;
      Ch::unpack(from[(2 * i) * THREADS], u);
      Ch::unpack(from[(2 * i + 1) * THREADS], v);
#pragma unroll
      for (int e = 0; e < R; ++e) ss += u[e] * u[e] + v[e] * v[e];
      if constexpr (!BWD) {
        const float r = rsqrtf(group_sum<L>(ss) * inv + A.eps);
#pragma unroll
        for (int e = 0; e < R; ++e) u[e] = u[e] * r * wu[e], v[e] = v[e] * r * wv[e];
        rotate<R, INTER, false>(u, v, c, s);
      } else {
        float hu[R], hv[R], hx = 0.f;
        Ch::unpack(from[(2 * HB + 2 * i) * THREADS], hu);
        Ch::unpack(from[(2 * HB + 2 * i + 1) * THREADS], hv);
        rotate<R, INTER, true>(hu, hv, c, s);
#pragma unroll
        for (int e = 0; e < R; ++e) hx += hu[e] * wu[e] * u[e] + hv[e] * wv[e] * v[e];
        ss = group_sum<L>(ss);
        hx = group_sum<L>(hx);
        const float r = rsqrtf(ss * inv + A.eps);
        const float t = r * r * hx * inv;      // r mean(h n): n mean(h n) = x t
        // (a lane or a head that is not there adds nothing: no 0 x NaN)
        if (live && h0 + i < S.H) {
#pragma unroll
          for (int e = 0; e < R; ++e) {
            dwu[e] += hu[e] * (u[e] * r);
            dwv[e] += hv[e] * (v[e] * r);
            u[e] = r * (hu[e] * wu[e] - u[e] * t);
            v[e] = r * (hv[e] * wv[e] - v[e] * t);
          }
        }
      }
      if (live && h0 + i < S.H) {
        T* y = out + row * S.out.row_stride + (h0 + i) * S.out.head_stride;
        *reinterpret_cast<Raw*>(y + ln.oa) = Ch::pack(u);
        *reinterpret_cast<Raw*>(y + ln.ob) = Ch::pack(v);
      }
    }
    if (use.base != base) {
      load_table(A, ln, pos, c, s);
      pos = position(use.base + step);
    }
  }
  if constexpr (BWD) {
    if (!A.part) return;
    // the block's sums, its groups in order
    float* const sh = reinterpret_cast<float*>(smem4);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int k = 0; k < R; ++k) sh[k * THREADS + threadIdx.x] = dwu[k], sh[(R + k) * THREADS + threadIdx.x] = dwv[k];
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * R * L; e += THREADS) {
      const int l = e % L, k = e / L;
      float t = 0.f;
      for (int q = 0; q < GROUPS; ++q) t += sh[k * THREADS + q * L + l];
      const Lane to = lane_of<R, INTER>(A, l);
      if (to.on) A.part[static_cast<long long>(blockIdx.x) * A.D + (k < R ? to.oa + k : to.ob + k - R)] = t;
    }
  }
}

// dw[d] = sum over the blocks' partial sums, in an order that depends on their number alone; queries, then keys.
__global__ void __launch_bounds__(1024) k_norm_dw(const float* part, int q_blocks, int k_blocks, int D, float* dwq,
                                                  float* dwk) {
  griddep_wait();
  __shared__ float sh[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  const int from = blockIdx.y ? q_blocks : 0, n = blockIdx.y ? k_blocks : q_blocks;
  float t = 0.f;
  if (col < D)
    for (int b = threadIdx.y; b < n; b += 32) t += part[static_cast<long long>(from + b) * D + col];
  sh[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0 && col < D) {
    t = 0.f;
    for (int i = 0; i < 32; ++i) t += sh[i][threadIdx.x];
    float* out = blockIdx.y ? dwk : dwq;
    if (out) out[col] = t;
  }
}

template <typename T, int R, int L, bool INTER, bool BWD>
cudaError_t launch(RopeArgs& A, int sms, cudaStream_t s) {
  constexpr int GROUPS = THREADS / L, HB = HEADS<BWD>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = ensure_smem_attr(k_norm_rope<T, R, L, INTER, BWD>, RING<T, R, BWD>, done);
  if (e != cudaSuccess) return e;
  const int room = sms * 2;                      // blocks that run at once
  const int heads = A.side[0].H + A.side[1].H;
  int hb = HB;
  // fewer heads at a time where the tokens' heads would not fill the device (13 tokens, 10 heads: 4.4 microseconds for
  // a launch with one head a group, 5.4 with four; 71,680 tokens forward and backward, loads straight into registers:
  // 894 with one, 625 with four and two)
  while (hb > 1 && A.n_tokens * heads < static_cast<long long>(room) * GROUPS * hb) hb /= 2;
  int total = 0;
  for (int o = 0; o < 2; ++o) {
    Side& S = A.side[o];
    S.hb = hb;
    const int want = (S.H + hb - 1) / hb;
    S.share = want < GROUPS ? want : GROUPS;
    const long long per = GROUPS / S.share, need = (A.n_tokens + per - 1) / per;
    // the device's blocks split by the work
    const int got = (room * S.H + heads / 2) / heads;
    S.blocks = static_cast<int>(need < got ? need : (got > 1 ? got : 1));
    if (S.blocks > MAX_PART_BLOCKS / 2) S.blocks = MAX_PART_BLOCKS / 2;
    total += S.blocks;
  }
  return launch_k(k_norm_rope<T, R, L, INTER, BWD>, dim3(total), dim3(THREADS), RING<T, R, BWD>, s, false, A);
}

template <typename T, int R, bool BWD>
cudaError_t by_lanes(RopeArgs& A, bool inter, int sms, cudaStream_t s) {
  // lanes per head vector, 2 R elements each
  const int lanes = A.D / (2 * R);
#define MLORA_GO(L) (inter ? launch<T, R, L, true, BWD>(A, sms, s) : launch<T, R, L, false, BWD>(A, sms, s))
  if (lanes <= 4) return MLORA_GO(4);
  if (lanes <= 8) return MLORA_GO(8);
  if constexpr (R == 8) {
    return MLORA_GO(16);
  } else {
    if (lanes <= 16) return MLORA_GO(16);
    return MLORA_GO(32);
  }
#undef MLORA_GO
}

template <bool BWD>
cudaError_t dispatch(RopeArgs& A, int esize, bool inter, int sms, cudaStream_t s) {
  if (esize == 4) return by_lanes<float, 4, BWD>(A, inter, sms, s);
  // runs of 16 bytes where both parts of the vector consist of them (71,680 tokens, loads straight into
  // registers: 625 microseconds, 882 with 8)
  if (A.rot % 16 == 0 && A.D % 16 == 0) return by_lanes<__nv_bfloat16, 8, BWD>(A, inter, sms, s);
  return by_lanes<__nv_bfloat16, 4, BWD>(A, inter, sms, s);
}

mlora_status check(const mlora_rope_problem* p) {
  if (!p) return op_fail(MLORA_ERR_INVALID, "null problem");
  if (p->dtype != MLORA_BF16 && p->dtype != MLORA_F32)
    return op_fail(MLORA_ERR_UNSUPPORTED, "queries and keys are bf16 or fp32");
  if (p->n_tokens < 1 || p->n_tokens > (1ll << 31) - 1 || p->n_q_heads < 1 || p->n_kv_heads < 1 ||
      p->n_q_heads > 4096 || p->n_kv_heads > 4096 || p->max_pos < 1)
    return op_fail(MLORA_ERR_INVALID, "tokens, heads and table rows must be positive (at most 4096 heads)");
  if (p->head_dim < 8 || p->head_dim > 256 || p->head_dim % 8)
    return op_fail(MLORA_ERR_UNSUPPORTED, "head_dim must be a multiple of 8, at most 256");
  if (p->rot_dim < 8 || p->rot_dim > p->head_dim || p->rot_dim % 8)
    return op_fail(MLORA_ERR_UNSUPPORTED, "rot_dim must be a multiple of 8, at most head_dim");
  if (p->flags & ~MLORA_ROPE_INTERLEAVED) return op_fail(MLORA_ERR_INVALID, "unknown flag");
  if (!(p->eps >= 0.f)) return op_fail(MLORA_ERR_INVALID, "eps must not be negative");
  return MLORA_OK;
}

mlora_status check_tables(const float* wq, const float* wk, const float* cosv,
                          const float* sinv, const int32_t* pos) {
  if (!wq || !wk || !cosv || !sinv || !pos) return op_fail(MLORA_ERR_INVALID, "null weight, table or position argument");
  if (!ptr_aligned(wq, 16) || !ptr_aligned(wk, 16) || !ptr_aligned(cosv, 16) || !ptr_aligned(sinv, 16) ||
      !ptr_aligned(pos, 4))
    return op_fail(MLORA_ERR_INVALID, "weights and tables must be 16-byte aligned");
  return MLORA_OK;
}

RopeArgs base(const mlora_rope_problem* p, const float* wq, const float* wk, const float* cosv, const float* sinv,
              const int32_t* pos) {
  RopeArgs A{};
  A.n_tokens = p->n_tokens;
  A.D = p->head_dim, A.rot = p->rot_dim, A.max_pos = p->max_pos;
  A.eps = p->eps;
  A.cos = cosv, A.sin = sinv, A.pos = pos;
  A.side[0].H = p->n_q_heads, A.side[0].w = wq;
  A.side[1].H = p->n_kv_heads, A.side[1].w = wk;
  return A;
}

}  // namespace
}  // namespace mlora

using namespace mlora;

extern "C" {

mlora_status mlora_qk_norm_rope(const mlora_rope_problem* p, const mlora_heads* q, const mlora_heads* k,
                                const float* wq, const float* wk, const float* cos_table, const float* sin_table,
                                const int32_t* positions, const mlora_heads* q_out, const mlora_heads* k_out,
                                void* stream) {
  mlora_status st = check(p);
  if (st == MLORA_OK) st = check_tables(wq, wk, cos_table, sin_table, positions);
  if (st != MLORA_OK) return st;
  const int es = p->dtype == MLORA_F32 ? 4 : 2;
  const struct { const mlora_heads* t; const char* name; int h; } all[] = {
      {q, "q", p->n_q_heads}, {k, "k", p->n_kv_heads}, {q_out, "q_out", p->n_q_heads}, {k_out, "k_out", p->n_kv_heads}};
  for (const auto& a : all)
    if ((st = check_heads(a.t, a.name, p->n_tokens, a.h, p->head_dim, es)) != MLORA_OK) return st;
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return op_cuda_fail(e, "querying the device");
  RopeArgs A = base(p, wq, wk, cos_table, sin_table, positions);
  A.side[0].x = *q, A.side[0].out = *q_out;
  A.side[1].x = *k, A.side[1].out = *k_out;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = dispatch<false>(A, es, p->flags & MLORA_ROPE_INTERLEAVED, sms, s);
  if (e != cudaSuccess) return op_cuda_fail(e, "norm and rotation launch");
  count_launches(1);
  return MLORA_OK;
}

size_t mlora_qk_norm_rope_workspace(const mlora_rope_problem* p) {
  return p && p->head_dim > 0 && p->head_dim <= 256 ? static_cast<size_t>(MAX_PART_BLOCKS) * p->head_dim * 4 : 0;
}

mlora_status mlora_qk_norm_rope_backward(const mlora_rope_problem* p, const mlora_heads* dq_out,
                                         const mlora_heads* dk_out, const mlora_heads* q, const mlora_heads* k,
                                         const float* wq, const float* wk, const float* cos_table,
                                         const float* sin_table, const int32_t* positions, const mlora_heads* dq,
                                         const mlora_heads* dk, float* dwq, float* dwk, void* workspace, void* stream) {
  mlora_status st = check(p);
  if (st == MLORA_OK) st = check_tables(wq, wk, cos_table, sin_table, positions);
  if (st != MLORA_OK) return st;
  const int es = p->dtype == MLORA_F32 ? 4 : 2;
  const struct { const mlora_heads* t; const char* name; int h; } all[] = {
      {dq_out, "dq_out", p->n_q_heads}, {dk_out, "dk_out", p->n_kv_heads}, {q, "q", p->n_q_heads},
      {k, "k", p->n_kv_heads}, {dq, "dq", p->n_q_heads}, {dk, "dk", p->n_kv_heads}};
  for (const auto& a : all)
    if ((st = check_heads(a.t, a.name, p->n_tokens, a.h, p->head_dim, es)) != MLORA_OK) return st;
  const bool want_dw = dwq || dwk;
  if (want_dw && (!workspace || !ptr_aligned(workspace, 16)))
    return op_fail(MLORA_ERR_INVALID, "weight gradients need a 16-byte aligned workspace");
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return op_cuda_fail(e, "querying the device");
  RopeArgs A = base(p, wq, wk, cos_table, sin_table, positions);
  A.side[0].x = *q, A.side[0].g = *dq_out, A.side[0].out = *dq;
  A.side[1].x = *k, A.side[1].g = *dk_out, A.side[1].out = *dk;
  A.part = want_dw ? static_cast<float*>(workspace) : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = dispatch<true>(A, es, p->flags & MLORA_ROPE_INTERLEAVED, sms, s);
  if (e != cudaSuccess) return op_cuda_fail(e, "norm and rotation gradient launch");
  count_launches(1);
  if (want_dw) {
    e = launch_k(k_norm_dw, dim3((p->head_dim + 31) / 32, 2), dim3(32, 32), 0, s, true,
                 static_cast<const float*>(A.part), A.side[0].blocks, A.side[1].blocks, p->head_dim, dwq, dwk);
    if (e != cudaSuccess) return op_cuda_fail(e, "weight gradient launch");
    count_launches(1);
  }
  return MLORA_OK;
}

}  // extern "C"
