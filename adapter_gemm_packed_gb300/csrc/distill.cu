// Distillation from a teacher's top logits: loss of every token and the gradient at the logits.
//
// A row of V student logits z and K teacher entries (id_k, t_k), temperature T, weight w:
//   p = softmax(t / T) over the row's entries, q = softmax(z / T) over the V logits,
//   loss = w T^2 sum_k p_k (log p_k - z_{id_k} / T + lse),   lse = log sum_v exp(z_v / T),
//   dz_v = w T (q_v - sum_{k: id_k = v} p_k).
// Entries whose id lies outside [0, V) are padding.  Rows of weight zero, and rows without an entry, have
// loss and gradient zero; their logits are not read.
//
// Memory-bound: z has to be read and dz written once.  A block goes over a row twice, for the sum (each thread keeps a
// running maximum and sum) and for the gradient.  The row comes through a ring of bulk copies in shared memory
// which keeps its last 108 KB for the second pass; what a longer row has before that is copied again, out of L2.
// As the second pass hands slots back, the next rows' copies fill them: reading runs under writing, and what is in
// flight does not depend on the threads.  What a copy brings for the last time is marked to leave L2 first, so that the
// parts of the 304 rows that come twice stay there.  8192 x 128,000 bf16 takes 720 microseconds, 5.8 TB/s of logits
// read and gradient written (820 without the marks, when almost half as much was read from memory again; 854 with two
// blocks an SM that load plainly and read the whole second pass out of L2); 2048 x 50,001, every fourth row without
// weight, 89.  A block's slots are full through its first pass and refill through its second, and rows are handed out
// whole: that is what is left above the copy rate, most where a block does few rows.
//
// In base 2: with k = log2(e) / T and the maximum M of z over what a thread or the block has seen,
// sum = sum_v 2^(k z_v - k M).  The product k M is rounded once and the rounded number is the reference for the sum
// and for the gradient alike, so its rounding cancels.  All sums are fp32, in an order that V alone fixes: not the
// other rows, not where a row starts in memory.  (Roundings are spelt out where the compiler might fuse one way here and
// another there; which thread adds what goes by an element's place in its row; in rows
// off a 16-byte boundary, a thread's 16 bytes are put together from two.)
//
// Waits have a limit.  Whether one has given up is settled by the computing threads together at the start of every row, so
// that they never part ways; a block's rows from there on, and the one before, get a loss and a gradient of NaN.
#include <climits>

#include "entry.cuh"

namespace mlora {
namespace {

constexpr int THREADS = 384;       // and a warp that fills the ring and one for the teacher's entries
constexpr int UNROLL = 3;          // 16-byte pieces of a slot per thread
constexpr int SLOT_VECS = THREADS * UNROLL, SLOT = SLOT_VECS * 16, SLOTS = 6;
constexpr int MAX_TOP = 256;
constexpr int NONE = 0x7fffffff;
constexpr int AHEAD = 4;           // rows whose teacher's softmax is known ahead of time

struct DistillArgs {
  const void* z;
  const int* ids;
  const float* teacher;
  const float* weight;      // null: 1 for every row
  float* loss;
  void* dz;
  long long n, z_stride, dz_stride;
  int V, K;
  float T, k2;              // temperature, log2(e) / T
  int same_align;           // rows of z and dz lie the same way to 16-byte boundaries
  int drop;                 // test hook: the place of a copy that every block leaves out, or -1
  unsigned long long timeout_ns;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Vec;      // 16 bytes of logits
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  static constexpr uint32_t NONE = 0xff800000u;      // -inf in every element
  // the larger of two, element by element; and the largest element
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ float top(uint32_t v) { return __uint_as_float(v); }
  static __device__ __forceinline__ float one(float v) { return v; }
  static __device__ __forceinline__ float round(float v) { return v; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
  static constexpr uint32_t NONE = 0xff80ff80u;
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ float top(uint32_t v) {
    return fmaxf(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  static __device__ __forceinline__ float one(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
};

// A running sum s of 2^(y - r): r is the reference, -inf while nothing but -inf has come (then s is 0, or NaN if a
// NaN has).
struct Run {
  float r, s;
};
// A warp's sum: the maximum of the references first, then each part at its weight.  (Sums by butterflies, which give
// every lane the same bits.)
__device__ __forceinline__ Run warp_sum(Run v) {
  float r = v.r;
#pragma unroll
  for (int o = 16; o; o >>= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, o));
  float s = r == -INFINITY ? v.s : __fmul_rn(v.s, v.r == -INFINITY ? 1.f : ex2(v.r - r));
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return Run{r, s};
}

// A barrier of the threads that compute.
__device__ __forceinline__ void sync_threads() { asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory"); }

// A barrier of theirs that tells each whether any of them says so.
__device__ __forceinline__ bool any_thread(bool v) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(v ? 1u : 0u), "n"(THREADS)
      : "memory");
  return any != 0;
}

// All computing threads get the block's sum.
__device__ __forceinline__ Run join(Run v, Run* sh) {
  v = warp_sum(v);
  const int lane = threadIdx.x & 31;
  if (lane == 0) sh[threadIdx.x >> 5] = v;
  sync_threads();
  return warp_sum(lane < THREADS / 32 ? sh[lane] : Run{-INFINITY, 0.f});
}

// How a row lies in memory: elements before its first 16-byte boundary, the whole vectors from there on (which go
// through the ring), the rest; and what that makes of the ring.
struct Row {
  int head, nvec, tail0;
  int chunks, again;      // slots the row takes, and how many of them have to be copied a second time
};
template <typename T>
__device__ __forceinline__ Row row_of(const T* z, int V, bool twice) {
  constexpr int N = Vec<T>::N;
  Row r;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
  r.head = min(V, off ? N - off : 0);
  r.nvec = (V - r.head) / N;
  r.tail0 = r.head + r.nvec * N;
  r.chunks = (r.nvec + SLOT_VECS - 1) / SLOT_VECS;
  r.again = twice ? max(0, r.chunks - SLOTS) : 0;
  return r;
}

// A row's elements N j .. N j + N, element by element where they are not all in the ring.
template <typename T>
__device__ __forceinline__ uint4 gather(const T* z, int j) {
  constexpr int N = Vec<T>::N;
  float x[N];
#pragma unroll
  for (int c = 0; c < N; ++c) x[c] = Vec<T>::one(z[static_cast<long long>(j) * N + c]);
  return Vec<T>::pack(x);
}

// 16 bytes from byte 16 - HB of (a, b) on
template <int HB>
__device__ __forceinline__ uint4 straddle(const uint4& a, const uint4& b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  constexpr int S = (16 - HB) / 4, B = (16 - HB) % 4 * 8;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = B ? __funnelshift_r(w[S + i], w[S + i + 1 < 8 ? S + i + 1 : 7], B) : w[S + i];
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// This thread's vectors of chunk c into its running sum: vectors j = SLOT_VECS c + tid + THREADS u of the row, counted
// from its first element.  HB: bytes before the row's first 16-byte boundary.  `first` and `last` are the row's
// first and last vector, where those are not whole in the ring (with their threads); `prev` the 16 bytes before the slot.
template <typename T, int HB>
__device__ __forceinline__ void sum_chunk(Run& r, const uint4& first, const uint4& last, const uint4* slot,
                                          const uint4* prev, int c, int nlog, int nvec, float k2) {
  typedef Vec<T> W;
  constexpr int N = W::N;
  uint4 v[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const int l = threadIdx.x + u * THREADS, j = c * SLOT_VECS + l;
    v[u] = make_uint4(W::NONE, W::NONE, W::NONE, W::NONE);
    if (j < nlog) {
      if (HB == 0) v[u] = slot[l];
      else if (j == 0) v[u] = first;
      else if (j >= nvec) v[u] = last;
      else v[u] = straddle<HB>(l ? slot[l - 1] : *prev, slot[l]);
    }
  }
  uint32_t most = W::NONE;
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) most = W::max(most, W::max(W::max(v[u].x, v[u].y), W::max(v[u].z, v[u].w)));
  const float ref = fmaxf(r.r, W::top(most) * k2), sub = ref == -INFINITY ? 0.f : ref;
  float s[4] = {__fmul_rn(r.s, r.r == -INFINITY ? 1.f : ex2(r.r - sub)), 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    float x[N];
    W::unpack(v[u], x);
#pragma unroll
    for (int e = 0; e < N; ++e) s[e % 4] = __fadd_rn(s[e % 4], ex2(fmaf(x[e], k2, -sub)));
  }
  r = Run{ref, __fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3]))};
}

__device__ __forceinline__ bool warp_ok(bool ok) { return __all_sync(0xffffffffu, ok); }

// What is known of a row ahead of time: the teacher's softmax in base 2 (sum 0: the row does not count), the weight.
struct Record {
  Run t;
  float w;
};

// What a thread of the first K holds of its row's teacher entries.
struct Entry {
  int id;        // -1: padding
  float u;       // t, then t / T in base 2
};

// The block's n-th row.  Each round starts 37 blocks further on: rows of weight zero at a regular distance do not all
// fall to the same blocks (2048 x 50,001, every fourth row: 100 microseconds without, 89 with).
__device__ __forceinline__ long long row_at(int n) {
  return static_cast<long long>(n) * gridDim.x + (blockIdx.x + 37ull * static_cast<unsigned>(n)) % gridDim.x;
}

template <typename T>
__global__ void __launch_bounds__(THREADS + 64, 2) k_distill(const DistillArgs A) {
  griddep_wait();
  typedef Vec<T> W;
  constexpr int N = W::N;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ Run sh[THREADS / 32];
  __shared__ Record rec[AHEAD];
  __shared__ uint64_t rec_full[AHEAD], rec_empty[AHEAD];
  __shared__ float p_sh[MAX_TOP], part_sh[MAX_TOP];
  __shared__ int id_sh[MAX_TOP];
  __shared__ uint64_t full[SLOTS], empty[SLOTS];
  __shared__ uint64_t ended;      // the computing warps are through
  __shared__ int abort_s, err_s;
  __shared__ int lost_s;          // which of its rows the block has lost, and those after it: a wait gave up
  volatile int* abort_flag = &abort_s;
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], THREADS / 32);
    for (int i = 0; i < AHEAD; ++i) mbar_init(&rec_full[i], 1), mbar_init(&rec_empty[i], THREADS / 32 + 1);
    mbar_init(&ended, THREADS / 32);
    abort_s = err_s = 0;
    lost_s = NONE;
    fence_mbar_init();
  }
  __syncthreads();
  // whether the second pass goes through the ring as well
  const bool twice = A.dz && A.same_align;

  if (tid >= THREADS + 32) {
    // the teacher's softmax of each row: its reference and sum (0: the row does not count)
    int n = 0;
    bool ok = true;
    auto term = [&](long long row, int k) {
      if (k >= A.K || row >= A.n) return -INFINITY;
      const int id = A.ids[row * A.K + k];
      return id >= 0 && id < A.V ? A.teacher[row * A.K + k] * A.k2 : -INFINITY;
    };
    auto weight = [&](long long row) { return A.weight && row < A.n ? A.weight[row] : 1.f; };
    float u = term(blockIdx.x, lane), w = weight(blockIdx.x);
    for (long long row = blockIdx.x, next; ok && row < A.n; row = next, ++n) {
      next = row_at(n + 1);
      Run t{u, u == -INFINITY ? 0.f : 1.f + (u - u)};
      const float wr = w;
      for (int k = lane + 32; k < A.K; k += 32) {
        const float x = term(row, k), r = fmaxf(t.r, x);
        if (x == -INFINITY) continue;
        // (a NaN reference does not come up: fmaxf drops it, the sum keeps it)
        t = Run{r, (t.r == -INFINITY ? t.s : __fmul_rn(t.s, ex2(t.r - r))) + (r == -INFINITY ? x - x : ex2(x - r))};
      }
      u = term(next, lane);      // the next row's, while this one is looked after
      w = weight(next);
      t = warp_sum(t);
      if (wr == 0.f) t.s = 0.f;
      if (lane == 0) {
        ok = mbar_wait(&rec_empty[n % AHEAD], ((n / AHEAD) & 1) ^ 1u, abort_flag, &err_s, 4, A.timeout_ns);
        if (ok) {
          rec[n % AHEAD] = Record{t, wr};
          mbar_arrive(&rec_full[n % AHEAD]);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    return;
  }
  if (tid >= THREADS) {
    // the ring: chunks of the rows that count, in order; those that come again behind the row's last
    const uint64_t once = l2_policy_evict_first();
    int pos = 0, n = 0;
    bool ok = true;
    for (long long row = blockIdx.x; ok && row < A.n; row = row_at(++n)) {
      ok = warp_ok(mbar_wait(&rec_full[n % AHEAD], (n / AHEAD) & 1, abort_flag, &err_s, 5, A.timeout_ns));
      if (!ok) break;
      const bool some = rec[n % AHEAD].t.s != 0.f;
      __syncwarp();
      if (lane == 0) mbar_arrive(&rec_empty[n % AHEAD]);
      if (!some) continue;
      const T* z = static_cast<const T*>(A.z) + row * A.z_stride;
      const Row R = row_of(z, A.V, twice);
      const uint8_t* from = reinterpret_cast<const uint8_t*>(z + R.head);
      if (lane == 0) {
        for (int i = 0; ok && i < R.chunks + R.again; ++i, ++pos) {
          const int c = i < R.chunks ? i : i - R.chunks, sl = pos % SLOTS;
          ok = mbar_wait(&empty[sl], ((pos / SLOTS) & 1) ^ 1u, abort_flag, &err_s, 1, A.timeout_ns);
          if (!ok) break;
          const uint32_t bytes = min(SLOT_VECS, R.nvec - c * SLOT_VECS) * 16;
          mbar_arrive_expect_tx(&full[sl], bytes);
          const uint8_t* src = from + static_cast<long long>(c) * SLOT;
          if (pos == A.drop) continue;
          // what will be read again stays in L2 if what will not leaves first
          if (i < R.again) bulk_load(ring + sl * SLOT, src, bytes, &full[sl]);
          else bulk_load_hint(ring + sl * SLOT, src, bytes, &full[sl], once);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0) {
      // bounded: no copy may still be writing shared memory when the block ends, whoever gave up
      volatile int no_abort = 0;
      for (int q = pos > SLOTS ? pos - SLOTS : 0; q < pos; ++q)
        mbar_wait(&full[q % SLOTS], (q / SLOTS) & 1, &no_abort, &err_s, 2, A.timeout_ns);
      // (a computing warp gives up once at most, and its row is bounded; no_abort is set where a copy is missing)
      no_abort = 0;
      if (!mbar_wait(&ended, 0, &no_abort, &err_s, 6, 4 * A.timeout_ns)) lost_s = 0;
    }
    __syncwarp();
    const float nan = __int_as_float(0x7fffffff);
    for (n = lost_s; n != NONE && (n == 0 || row_at(n) < A.n); ++n) {
      if (lane == 0) A.loss[row_at(n)] = nan;
      if (A.dz)
        for (long long i = lane; i < A.V; i += 32) (static_cast<T*>(A.dz) + row_at(n) * A.dz_stride)[i] = W::round(nan);
    }
    return;
  }

  // a row's entry of this thread, as it stands in memory
  auto entry = [&](long long row) {
    Entry e{-1, 0.f};
    if (tid < A.K && row < A.n) e.id = A.ids[row * A.K + tid], e.u = A.teacher[row * A.K + tid];
    return e;
  };
  int pos = 0, n = 0;
  auto slot_at = [&](int p) { return reinterpret_cast<const uint4*>(ring + p % SLOTS * SLOT); };
  // (one that gives up raises the abort flag, which is looked at once a row)
  auto arrived = [&](uint64_t* bar, int parity) { mbar_wait(bar, parity, abort_flag, &err_s, 3, A.timeout_ns); };
  auto release = [&](int p) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[p % SLOTS]);
  };

  long long row = blockIdx.x;
  Entry e = entry(row);
  for (long long next; row < A.n; row = next, ++n) {
    next = row_at(n + 1);
    const T* z = static_cast<const T*>(A.z) + row * A.z_stride;
    T* dz = A.dz ? static_cast<T*>(A.dz) + row * A.dz_stride : nullptr;
    const Row R = row_of(z, A.V, twice);
    // element of the row's ends that is this thread's in the second pass, or -1
    const int edge = tid < R.head ? tid : (tid >= 32 && tid - 32 < A.V - R.tail0 ? R.tail0 + tid - 32 : -1);

    arrived(&rec_full[n % AHEAD], (n / AHEAD) & 1);
    // (also: the row before is done with the shared arrays)
    if (any_thread(*abort_flag)) break;
    const Record known = rec[n % AHEAD];
    __syncwarp();
    if (lane == 0) mbar_arrive(&rec_empty[n % AHEAD]);
    const Run tr = known.t;
    const float wr = known.w;
    Entry mine{e.id >= 0 && e.id < A.V ? e.id : -1, e.u * A.k2};
    if (mine.id < 0) mine.u = -INFINITY;
    e = entry(next);
    const bool some = tr.s != 0.f;
    if (!some) {
      if (dz) {
        if (A.same_align) {
          uint4* out = reinterpret_cast<uint4*>(dz + R.head);
          for (int i = tid; i < R.nvec; i += THREADS) __stcs(out + i, make_uint4(0, 0, 0, 0));
          if (edge >= 0) dz[edge] = W::round(0.f);
        } else {
          for (int i = tid; i < A.V; i += THREADS) dz[i] = W::round(0.f);
        }
      }
      if (tid == 0) A.loss[row] = 0.f;
      continue;
    }
    const float zk = mine.id >= 0 ? W::one(z[mine.id]) : 0.f;

    // the student's sum
    const int nlog = A.V / N;
    Run r{-INFINITY, 0.f};
    if (tid < A.V - nlog * N) {
      r.r = W::one(z[nlog * N + tid]) * A.k2;
      r.s = r.r == -INFINITY ? 0.f : 1.f + (r.r - r.r);      // NaN for NaN and +inf
    }
    const int hb = R.head * static_cast<int>(sizeof(T));
    // in a row off a 16-byte boundary the first vector begins before the ring's part, and the last may end behind it
    uint4 first{}, last{};
    if (hb && nlog && tid == 0) first = gather(z, 0);
    if (hb && nlog > R.nvec && tid == (nlog - 1) % SLOT_VECS % THREADS) last = gather(z, nlog - 1);
    for (int c = 0; c < R.chunks; ++c) {
      arrived(&full[(pos + c) % SLOTS], ((pos + c) / SLOTS) & 1);
      const uint4* s = slot_at(pos + c);
      const uint4* prev = c ? slot_at(pos + c - 1) + SLOT_VECS - 1 : nullptr;
      switch (hb) {
        case 0: sum_chunk<T, 0>(r, first, last, s, prev, c, nlog, R.nvec, A.k2); break;
        case 4: sum_chunk<T, 4>(r, first, last, s, prev, c, nlog, R.nvec, A.k2); break;
        case 8: sum_chunk<T, 8>(r, first, last, s, prev, c, nlog, R.nvec, A.k2); break;
        case 12: sum_chunk<T, 12>(r, first, last, s, prev, c, nlog, R.nvec, A.k2); break;
        default:
          if constexpr (sizeof(T) == 2) {
            switch (hb) {
              case 2: sum_chunk<T, 2>(r, first, last, s, prev, c, nlog, R.nvec, A.k2); break;
              case 6: sum_chunk<T, 6>(r, first, last, s, prev, c, nlog, R.nvec, A.k2); break;
              case 10: sum_chunk<T, 10>(r, first, last, s, prev, c, nlog, R.nvec, A.k2); break;
              default: sum_chunk<T, 14>(r, first, last, s, prev, c, nlog, R.nvec, A.k2); break;
            }
          }
      }
      // (the next chunk's first vector begins in this one)
      if (c && (!twice || c - 1 < R.again)) release(pos + c - 1);
    }
    if (R.chunks && !twice) release(pos + R.chunks - 1);
    // a last vector of the row that has no chunk (its elements are the row's ends)
    if (R.chunks * SLOT_VECS < nlog) sum_chunk<T, 4>(r, first, last, nullptr, nullptr, R.chunks, nlog, 0, A.k2);
    r = join(r, sh);

    const float g = wr * A.T, inv = g / r.s;
    const float p = mine.id >= 0 && mine.u != -INFINITY ? ex2(mine.u - tr.r) / tr.s : 0.f;
    if (tid < A.K) {
      p_sh[tid] = p;
      id_sh[tid] = mine.id;
      // log p_k - log q_k, in base 2
      part_sh[tid] = p > 0.f || p != p ? p * (((mine.u - tr.r) - log2f(tr.s)) - (zk * A.k2 - r.r) + log2f(r.s)) : 0.f;
    }
    if (twice) {
      uint4* out = reinterpret_cast<uint4*>(dz + R.head);
      for (int i = R.again; i < R.chunks + R.again; ++i) {
        const int c = i < R.chunks ? i : i - R.chunks;
        if (i >= R.chunks) arrived(&full[(pos + i) % SLOTS], ((pos + i) / SLOTS) & 1);
        const uint4* s = slot_at(pos + i);
        const int n = min(SLOT_VECS, R.nvec - c * SLOT_VECS);
        uint4 v[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
          if (tid + u * THREADS < n) v[u] = s[tid + u * THREADS];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
          if (tid + u * THREADS < n) {
            float x[N];
            W::unpack(v[u], x);
#pragma unroll
            for (int k = 0; k < N; ++k) x[k] = __fmul_rn(inv, ex2(fmaf(x[k], A.k2, -r.r)));
            __stcs(out + static_cast<long long>(c) * SLOT_VECS + tid + u * THREADS, W::pack(x));
          }
        // only now: the loads must have returned, not just been issued, before a copy may overwrite the slot
        release(pos + i);
      }
      if (edge >= 0) dz[edge] = W::round(__fmul_rn(inv, ex2(fmaf(W::one(z[edge]), A.k2, -r.r))));
    } else if (dz) {
      for (int i = tid; i < A.V; i += THREADS)
        dz[i] = W::round(__fmul_rn(inv, ex2(fmaf(W::one(z[i]), A.k2, -r.r))));
    }
    pos += R.chunks + R.again;
    // the gradient is written and the entries are in shared memory
    sync_threads();
    if (tid < 32) {
      float t = 0.f;
      for (int k = tid; k < A.K; k += 32) t += part_sh[k];
#pragma unroll
      for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (tid == 0) A.loss[row] = wr * A.T * A.T * (t * 0.6931471805599453f);
    }
    // the entries' elements again; an id that comes twice by its first entry
    if (dz && tid < A.K && mine.id >= 0) {
      float sum = 0.f;
      bool first = true;
      for (int k = 0; k < A.K; ++k)
        if (id_sh[k] == mine.id) {
          if (k < tid) first = false;
          sum += p_sh[k];
        }
      if (first) dz[mine.id] = W::round(fmaf(-g, sum, __fmul_rn(inv, ex2(fmaf(zk, A.k2, -r.r)))));
    }
  }
  // the row before this one may be what a wait gave up in; none after it has been looked at
  __syncwarp();
  if (lane == 0) {
    if (*abort_flag) atomicMin(&lost_s, max(n - 1, 0));
    mbar_arrive(&ended);
  }
}

template <typename T>
cudaError_t launch(const DistillArgs& A, dim3 grid, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = ensure_smem_attr(k_distill<T>, SLOTS * SLOT, done);
  return e == cudaSuccess ? launch_k(k_distill<T>, grid, dim3(THREADS + 64), SLOTS * SLOT, s, false, A) : e;
}

}  // namespace
}  // namespace mlora

using namespace mlora;

extern "C" mlora_status mlora_distill_loss(const mlora_distill_problem* p, const void* logits, const int32_t* ids,
                                           const float* teacher, const float* weight, float* loss, void* dlogits,
                                           void* stream) {
  if (!p) return op_fail(MLORA_ERR_INVALID, "null problem");
  if (p->dtype != MLORA_BF16 && p->dtype != MLORA_F32)
    return op_fail(MLORA_ERR_UNSUPPORTED, "logits are bf16 or fp32");
  if (p->n_tokens < 1 || p->vocab < 1 || p->top < 1)
    return op_fail(MLORA_ERR_INVALID, "tokens, vocabulary and teacher entries must be positive");
  if (p->vocab > INT_MAX - 4096)      // places in a row, a step of all threads ahead, stay within 32 bits
    return op_fail(MLORA_ERR_UNSUPPORTED, "vocabulary out of range");
  if (p->top > MAX_TOP) return op_fail(MLORA_ERR_UNSUPPORTED, "at most 256 teacher entries a row");
  if (p->logits_stride < p->vocab || (dlogits && p->dlogits_stride < p->vocab))
    return op_fail(MLORA_ERR_INVALID, "rows of the logits or of their gradient overlap");
  if (!(p->temperature > 0.f) || !(p->temperature < INFINITY))
    return op_fail(MLORA_ERR_INVALID, "the temperature must be positive and finite");
  if (p->flags & ~(MLORA_DEBUG_SHORT_TIMEOUT | MLORA_DEBUG_DROP_COPY))
    return op_fail(MLORA_ERR_INVALID, "unknown flag");
  if (!logits || !ids || !teacher || !loss) return op_fail(MLORA_ERR_INVALID, "null tensor argument");
  const unsigned es = p->dtype == MLORA_F32 ? 4 : 2;
  if (!ptr_aligned(logits, es) || !ptr_aligned(dlogits, es) || !ptr_aligned(ids, 4) || !ptr_aligned(teacher, 4) ||
      !ptr_aligned(weight, 4) || !ptr_aligned(loss, 4))
    return op_fail(MLORA_ERR_INVALID, "a tensor is not aligned to its elements");
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return op_cuda_fail(e, "querying the device");
  DistillArgs A{logits, ids, teacher, weight, loss, dlogits, p->n_tokens, p->logits_stride, p->dlogits_stride,
                p->vocab, p->top, p->temperature, static_cast<float>(1.4426950408889634 / p->temperature), 0, 0,
                p->flags & MLORA_DEBUG_SHORT_TIMEOUT ? 1000000ull : 4000000000ull};
  A.drop = (p->flags & MLORA_DEBUG_SHORT_TIMEOUT) && (p->flags & MLORA_DEBUG_DROP_COPY) ? 2 : -1;
  A.same_align = (reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(dlogits)) % 16 == 0 &&
                 (p->logits_stride - p->dlogits_stride) * es % 16 == 0;
  const long long most = static_cast<long long>(sms) * 2;
  const dim3 grid(static_cast<unsigned>(p->n_tokens < most ? p->n_tokens : most));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = es == 4 ? launch<float>(A, grid, s) : launch<__nv_bfloat16>(A, grid, s);
  if (e != cudaSuccess) return op_cuda_fail(e, "distillation loss launch");
  count_launches(1);
  return MLORA_OK;
}
