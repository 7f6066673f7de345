// Windowed attention over packed sequences: what its kernels share.
//
// Token i of a sequence sees the tokens j <= i of it with i - j < window or j < n_sink.
//   S = scale Q K^T,  P = softmax of S over what is seen,  O = P V.
// The forward saves, for each query head and token, the softmax's logarithm of the sum in base 2,
//   L2 = log2(sum_j exp(S_ij)) = max + log2(sum), all of scale log2(e) S,
// from which the backward makes P again: P_ij = exp2(scale log2(e) q_i k_j - L2_i).
#pragma once
#include "entry.cuh"

namespace mlora {

constexpr int STAT_ROWS = 64;            // rows per block of the saved statistics
constexpr int STAT_BLOCK = 2 * STAT_ROWS;

// One piece of work: a tile of rows of a sequence and a head (or pair of heads) of it; with len 0, rows that
// belong to no sequence, for all heads.
struct AttnItem {
  int seq0;      // first token row of the sequence
  int len;       // its length
  int i0;        // the tile's first row within it; for a run without a sequence: its rows
  int stat0;     // the sequence's first row in the statistics' space
  int sub;       // forward: key head * pairs + pair; dQ: query head; dK and dV: key head
  // A dK / dV piece can be cut along its query tiles into `parts`, of which this is number `part`: each leaves its
  // sums in the scratch (set pbase + part) and counts itself on counter set `slot`; the last adds them up in order.
  short part, parts;
  int pbase, slot;
};

struct AttnArgs {
  const AttnItem* items;
  const int* first;          // block b of the persistent kernels does items [first[b], first[b + 1])
  int hq, hk, group, D;
  int window, n_sink;
  float scale, scale_log2;   // scale, and scale log2(e)
  long long n_stat;          // rows of the statistics' space per query head (a multiple of 128)
  mlora_heads q, k, v, o, dout, dq, dk, dv;
  float* saved;
  uint8_t* out_low;          // bf16: what the outputs' rounding cut off (see attn_tc.cuh), behind the statistics
  int* part_cnt;             // bf16 dK / dV, workspace: counters of cut pieces, and ...
  float* partials;           // ... their sums, behind that
  int n_cnt;
  int* err;
  unsigned long long timeout_ns;
};

// Where the statistics of row s (of n_stat) of query head h lie: blocks of 64 L2, then 64 delta.
__host__ __device__ __forceinline__ long long stat_at(long long n_stat, int h, long long s) {
  const long long r = h * n_stat + s;
  return (r / STAT_ROWS) * STAT_BLOCK + r % STAT_ROWS;
}

// The key tiles (of TK rows) that the query rows [i0, i1) see some key of: those of the window
// [lo, hi), after those of the first tokens that come before them, [0, sink).
struct KeyTiles {
  int sink, lo, hi;
  __host__ __device__ __forceinline__ int count() const { return sink + hi - lo; }
  __host__ __device__ __forceinline__ int tile(int n) const { return n < sink ? n : lo + (n - sink); }
};
__host__ __device__ __forceinline__ KeyTiles key_tiles(int i0, int i1, int window, int n_sink, int tk) {
  KeyTiles t;
  const int first = i0 >= window ? i0 - window + 1 : 0;
  t.lo = first / tk;
  t.hi = (i1 + tk - 1) / tk;
  const int s = (n_sink + tk - 1) / tk;
  t.sink = s < t.lo ? s : t.lo;
  return t;
}

// The query rows [lo, hi) that see some key of [j0, j1): from j0 on, to the window's end unless the
// keys include first tokens.
__host__ __device__ __forceinline__ void query_rows(int j0, int j1, int len, int window, int n_sink, int& lo, int& hi) {
  lo = j0;
  const long long end = static_cast<long long>(j1) + window - 1;
  hi = (j0 < n_sink || end > len) ? len : static_cast<int>(end);
}

__host__ __device__ __forceinline__ bool sees(int i, int j, int window, int n_sink) {
  return j <= i && (i - j < window || j < n_sink);
}

// Whether token i sees itself and no other key.  Its probability is then 1 whatever the score, and the score's gradient
// P (dP - delta) exactly zero; computed, dP and delta are two sums of the same numbers in different orders, and their
// difference is noise that would be all there is of dQ, and of dK where a key is seen by such rows alone.
__host__ __device__ __forceinline__ bool sees_one(int i, int window, int n_sink) {
  return i == 0 || (window == 1 && n_sink == 0);
}

template <typename T>
__device__ __forceinline__ T* head_row(const mlora_heads& t, long long row, int h) {
  return static_cast<T*>(t.data) + row * t.row_stride + h * t.head_stride;
}

cudaError_t launch_attn_simt_forward(const AttnArgs& A, int n_items, cudaStream_t s);
cudaError_t launch_attn_simt_backward(const AttnArgs& A, const AttnItem* q_items, int n_q, const AttnItem* k_items,
                                      int n_k, cudaStream_t s);
int attn_fwd_rows(int group);
int attn_fwd_pairs(int group);
mlora_status launch_attn_fwd(const AttnArgs& A, int blocks, int64_t n_tokens, cudaStream_t s);
// AttnArgs with the work list of the kernel that owns dQ, and of the one that owns dK and dV
mlora_status launch_attn_bwd(const AttnArgs& Q, int q_blocks, const AttnArgs& K, int k_blocks, int64_t n_tokens,
                             cudaStream_t s);

}  // namespace mlora
