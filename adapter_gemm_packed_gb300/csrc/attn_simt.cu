// Windowed attention, forward and backward, on the fp32 pipes: every product in true fp32.
//
// A block owns 32 rows (queries in the forward and for dQ, keys for dK and dV) of one head and walks over the 32-row
// tiles of the other side that see them; a piece of the plan, 64 rows, is two blocks' work.  Its two or four teams of
// 128 threads take turns at the tiles and add up at the end.  For dK and dV a cluster of two or four blocks shares half a
// piece or a piece, since a key tile meets the queries of every head of its group and, if it holds first tokens, all of
// the sequence's.
//
// Tiles come by asynchronous copies, each as soon as the last product that reads the one before has ended: the next
// tile's first operand travels under this one's last product.  They lie in rows of DP + 4 floats (so that 16 rows
// read at once start in different banks); a thread computes 4 x 2 elements of a score tile and 4 x DP/16 of an output
// tile, two at a time in packed operations.
//
// Bound by shared memory, which the 4 x 2 elements ask for eight passes per eight cycles of products (4 x 4 and 64-row
// tiles ask for less, but leave room for half the warps: 10 to 20 % slower), and by latency: 8 sequences of 1024, window
// 512, 8 heads of 64 on 2: forward 231 microseconds, 28 TFLOP/s of about 74; 4096 tokens without a window, 6 heads of
// 128: 702, 37 TFLOP/s, backward 27.  A small pack is bound by its longest piece: 4 sequences of 33 to 700, 6 heads of
// 80 on 3: 25 microseconds forward, 79 backward.
//
// Rows past a sequence's end are read as zero, so what lies behind them (another sequence, padding, NaN) takes no
// part.  Gradients of shared heads are summed by the block that owns the keys, in an order that the sequence alone
// fixes: no atomics, the same result each run.
#include "attention.cuh"

namespace mlora {
namespace {

constexpr int PIECE = 64;      // rows of a piece of the plan
constexpr int OWN = 32;        // rows that a team owns
constexpr int BT = 32;         // rows of a tile of the other side
constexpr int NB = BT / 16;
constexpr int TEAM = 128;
// Teams of a block.  Above 64 columns a block's registers leave room for one block an SM anyway, and four teams shorten
// the way through a short list of tiles: 4 sequences of 33 to 700, 6 heads of 80 on 3, 25 + 93 microseconds against 30 +
// 99 with two, 4096 tokens without a window, 6 heads of 128, 702 + 2366 against 710 + 2585.  At 64 and below more
// blocks of two teams fit: 8 sequences of 1024, 8 heads of 64 on 2, 231 + 802 against 300 + 970 with four.
template <int DP>
constexpr int TEAMS = DP > 64 ? 4 : 2;
template <int DP>
constexpr int THREADS = TEAMS<DP> * TEAM;
typedef unsigned long long f32x2;

template <int DP>
constexpr int ROW = DP + 4;
constexpr int PROW = BT + 4;

__device__ __forceinline__ void fma2(f32x2& d, f32x2 a, f32x2 b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ void add2(f32x2& d, f32x2 a) { asm("add.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(a)); }
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 both(f32x2 v) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
  return d;
}

__device__ __forceinline__ void copy16(float* dst, const float* src, bool ok) {      // zeros where not ok
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but this thread's N latest groups of copies have arrived
template <int N>
__device__ __forceinline__ void arrived() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// rows [r0, r0 + ROWS) of a sequence's head, zero past its end; by `threads` threads
template <int DP, int ROWS>
__device__ __forceinline__ void load_tile(float* dst, const mlora_heads& t, int seq0, int r0, int len, int h, int D,
                                          int tid, int threads) {
  for (int r = tid / 16; r < ROWS; r += threads / 16) {
    const bool ok = r0 + r < len;
    const float* src = ok ? head_row<float>(t, static_cast<long long>(seq0) + r0 + r, h) : static_cast<const float*>(t.data);
    for (int c = tid % 16 * 4; c < D; c += 64) copy16(dst + r * ROW<DP> + c, src + c, ok);
  }
}

// a barrier of one team
__device__ __forceinline__ void sync_team(int team) { asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(TEAM) : "memory"); }

// out[a][b] = sum_d A[4 ty + a][d] B[tx + 16 b][d]; even and odd d apart until the end
template <int DP>
__device__ __forceinline__ void scores(const float* A, const float* B, int D, int ty, int tx, float (&out)[4][NB]) {
  f32x2 acc[4][NB] = {};
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    ulonglong2 x[4], y[NB];
#pragma unroll
    for (int a = 0; a < 4; ++a) x[a] = *reinterpret_cast<const ulonglong2*>(A + (4 * ty + a) * ROW<DP> + d);
#pragma unroll
    for (int b = 0; b < NB; ++b) y[b] = *reinterpret_cast<const ulonglong2*>(B + (tx + 16 * b) * ROW<DP> + d);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        fma2(acc[a][b], x[a].x, y[b].x);
        fma2(acc[a][b], x[a].y, y[b].y);
      }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float2 v = both(acc[a][b]);
      out[a][b] = v.x + v.y;
    }
}

// out[a][.] += sum_r P[4 ty + a][r] B[r][.]; the thread's columns are 2 tx + 32 c + (0, 1)
template <int DP>
__device__ __forceinline__ void accumulate(const float* P, const float* B, int ty, int tx, f32x2 (&out)[4][DP / 32]) {
#pragma unroll 4
  for (int r = 0; r < BT; r += 4) {
    float p[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float4 v = *reinterpret_cast<const float4*>(P + (4 * ty + a) * PROW + r);
      p[a][0] = v.x, p[a][1] = v.y, p[a][2] = v.z, p[a][3] = v.w;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f32x2 y[DP / 32];
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) y[c] = *reinterpret_cast<const f32x2*>(B + (r + k) * ROW<DP> + 32 * c + 2 * tx);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const f32x2 pp = pair(p[a][k], p[a][k]);
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) fma2(out[a][c], pp, y[c]);
      }
    }
  }
}

template <int DP>
__device__ __forceinline__ void store_rows(const mlora_heads& t, int seq0, int r0, int len, int h, int D, int ty, int tx,
                                           const f32x2 (&out)[4][DP / 32], const float (&f)[4]) {
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int i = r0 + 4 * ty + a;
    if (i >= len) continue;
    float* y = head_row<float>(t, static_cast<long long>(seq0) + i, h);
#pragma unroll
    for (int c = 0; c < DP / 32; ++c) {
      const float2 v = both(out[a][c]);
      const int d = 32 * c + 2 * tx;
      if (d < D) *reinterpret_cast<float2*>(y + d) = make_float2(v.x * f[a], v.y * f[a]);
    }
  }
}

__device__ __forceinline__ void zero_rows(const mlora_heads& t, const AttnItem& it, int heads, int D) {
  for (int h = 0; h < heads; ++h)
    for (int e = threadIdx.x; e < it.i0 * D; e += blockDim.x)
      head_row<float>(t, static_cast<long long>(it.seq0) + e / D, h)[e % D] = 0.f;
}

// over the 16 threads of a row
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, 16);
  return v;
}
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o, 16));
  return v;
}

template <int DP>
__global__ void __launch_bounds__(THREADS<DP>, DP > 64 ? 1 : 3) k_attn_simt_fwd(const AttnArgs A) {
  griddep_wait();
  extern __shared__ float4 smem4[];
  float* Q = reinterpret_cast<float*>(smem4);
  const int team = threadIdx.x / TEAM, tid = threadIdx.x % TEAM, ty = tid / 16, tx = tid % 16;
  constexpr int MINE = 2 * BT * ROW<DP> + OWN * PROW;      // of a team
  float* K = Q + OWN * ROW<DP> + team * MINE;
  float* V = K + BT * ROW<DP>;
  float* P = V + BT * ROW<DP>;
  const AttnItem it = A.items[blockIdx.x / 2];
  const int half = blockIdx.x % 2, h = it.sub, hk = h / A.group;
  if (it.len == 0) {
    if (!half) zero_rows(A.o, it, A.hq, A.D);
    return;
  }
  const int own0 = it.i0 + OWN * half, i1 = min(own0 + OWN, it.len);
  if (own0 >= it.len) return;
  const KeyTiles kt = key_tiles(own0, i1, A.window, A.n_sink, BT);
  auto load = [&](float* dst, const mlora_heads& t, int n) {
    if (n < kt.count()) load_tile<DP, BT>(dst, t, it.seq0, kt.tile(n) * BT, it.len, hk, A.D, tid, TEAM);
    commit();
  };
  load_tile<DP, OWN>(Q, A.q, it.seq0, own0, it.len, h, A.D, threadIdx.x, THREADS<DP>);
  load(K, A.k, team);
  load(V, A.v, team);
  arrived<1>();
  __syncthreads();
  f32x2 out[4][DP / 32] = {};
  float m[4], l[4] = {};
#pragma unroll
  for (int a = 0; a < 4; ++a) m[a] = -INFINITY;
  for (int n = team; n < kt.count(); n += TEAMS<DP>) {
    const int j0 = kt.tile(n) * BT;
    float s[4][NB];
    scores<DP>(Q, K, A.D, ty, tx, s);
    arrived<0>();
    sync_team(team);      // V is there, K is done with
    load(K, A.k, n + TEAMS<DP>);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int i = own0 + 4 * ty + a;
      float top = -INFINITY;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int j = j0 + tx + 16 * b;
        s[a][b] = (i < it.len && sees(i, j, A.window, A.n_sink)) ? s[a][b] * A.scale_log2 : -INFINITY;
        top = fmaxf(top, s[a][b]);
      }
      top = fmaxf(m[a], row_max(top));
      const float ref = top == -INFINITY ? 0.f : top;      // a row that has seen nothing yet
      const float f = exp2f(m[a] - ref);
      float sum = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float p = exp2f(s[a][b] - ref);
        sum += p;
        P[(4 * ty + a) * PROW + tx + 16 * b] = p;
      }
      l[a] = l[a] * f + row_sum(sum);
      m[a] = top;
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) {
        const float2 v = both(out[a][c]);
        out[a][c] = pair(v.x * f, v.y * f);
      }
    }
    __syncwarp();      // a row's 16 threads are in one warp, and a warp reads only its own rows of P
    accumulate<DP>(P, V, ty, tx, out);
    arrived<0>();
    sync_team(team);      // the next K is there, V is done with
    load(V, A.v, n + TEAMS<DP>);
  }
  // the other teams' shares, through their tiles' memory, each at its weight
  f32x2* const shares = reinterpret_cast<f32x2*>(Q + OWN * ROW<DP>) + tid;
  if (team) {
    f32x2* mine = shares + team * (MINE / 2);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      mine[a * TEAM] = pair(m[a], l[a]);
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) mine[(4 + a * (DP / 32) + c) * TEAM] = out[a][c];
    }
  }
  __syncthreads();
  if (team) return;
  float f[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
#pragma unroll
    for (int t = 1; t < TEAMS<DP>; ++t) {
      const f32x2* theirs = shares + t * (MINE / 2);
      const float2 o = both(theirs[a * TEAM]);
      const float top = fmaxf(m[a], o.x), ref = top == -INFINITY ? 0.f : top;
      const float f0 = exp2f(m[a] - ref), f1 = exp2f(o.x - ref);
      l[a] = l[a] * f0 + o.y * f1;
      m[a] = top;
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) {
        const float2 v = both(out[a][c]), w = both(theirs[(4 + a * (DP / 32) + c) * TEAM]);
        out[a][c] = pair(v.x * f0 + w.x * f1, v.y * f0 + w.y * f1);
      }
    }
    const int i = own0 + 4 * ty + a;
    f[a] = 1.f / l[a];
    if (tx == 0 && i < it.len) A.saved[stat_at(A.n_stat, h, it.stat0 + i)] = m[a] + log2f(l[a]);
  }
  store_rows<DP>(A.o, it.seq0, own0, it.len, h, A.D, ty, tx, out, f);
}

// P = exp2(scale_log2 S - L2) and dS = P (dP - delta) of a tile for the thread's 4 x 2 elements, from S and dP.
__device__ __forceinline__ void grad_one(const AttnArgs& A, int len, int i, int j, float l2, float delta, float& p, float& ds) {
  const bool ok = i < len && sees(i, j, A.window, A.n_sink);
  p = ok ? exp2f(fmaf(p, A.scale_log2, -l2)) : 0.f;
  ds = ok && !sees_one(i, A.window, A.n_sink) ? p * (ds - delta) : 0.f;
}

// dQ; and delta_i = sum_d dO_id O_id on the way, which the kernel for dK and dV reads after it
template <int DP>
__global__ void __launch_bounds__(THREADS<DP>) k_attn_simt_dq(const AttnArgs A) {
  griddep_wait();
  extern __shared__ float4 smem4[];
  float* Q = reinterpret_cast<float*>(smem4);
  float* dO = Q + OWN * ROW<DP>;
  const int team = threadIdx.x / TEAM, tid = threadIdx.x % TEAM, ty = tid / 16, tx = tid % 16;
  constexpr int MINE = 2 * BT * ROW<DP> + OWN * PROW;      // of a team
  float* K = dO + OWN * ROW<DP> + team * MINE;
  float* V = K + BT * ROW<DP>;
  float* S = V + BT * ROW<DP>;
  const AttnItem it = A.items[blockIdx.x / 2];
  const int half = blockIdx.x % 2, h = it.sub, hk = h / A.group;
  if (it.len == 0) {
    if (!half) zero_rows(A.dq, it, A.hq, A.D);
    return;
  }
  const int own0 = it.i0 + OWN * half, i1 = min(own0 + OWN, it.len);
  if (own0 >= it.len) return;
  const KeyTiles kt = key_tiles(own0, i1, A.window, A.n_sink, BT);
  auto load = [&](float* dst, const mlora_heads& t, int n) {
    if (n < kt.count()) load_tile<DP, BT>(dst, t, it.seq0, kt.tile(n) * BT, it.len, hk, A.D, tid, TEAM);
    commit();
  };
  load_tile<DP, OWN>(dO, A.dout, it.seq0, own0, it.len, h, A.D, threadIdx.x, THREADS<DP>);
  load_tile<DP, OWN>(Q, A.q, it.seq0, own0, it.len, h, A.D, threadIdx.x, THREADS<DP>);
  load(V, A.v, team);
  load(K, A.k, team);
  float l2[4], delta[4];
  float4 o[4][DP > 64 ? 2 : 1];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int i = own0 + 4 * ty + a;
    l2[a] = i < it.len ? A.saved[stat_at(A.n_stat, h, it.stat0 + i)] : 0.f;
#pragma unroll
    for (int c = 0; c < (DP > 64 ? 2 : 1); ++c) {
      const int d = 4 * tx + 64 * c;
      o[a][c] = i < it.len && d < A.D
                    ? *reinterpret_cast<const float4*>(head_row<float>(A.o, static_cast<long long>(it.seq0) + i, h) + d)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  arrived<1>();
  __syncthreads();
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    float t = 0.f;
#pragma unroll
    for (int c = 0; c < (DP > 64 ? 2 : 1); ++c) {
      const int d = 4 * tx + 64 * c;
      if (d < A.D) {
        const float4 g = *reinterpret_cast<const float4*>(dO + (4 * ty + a) * ROW<DP> + d);
        t = fmaf(g.x, o[a][c].x, fmaf(g.y, o[a][c].y, fmaf(g.z, o[a][c].z, fmaf(g.w, o[a][c].w, t))));
      }
    }
    delta[a] = row_sum(t);
    const int i = own0 + 4 * ty + a;
    if (team == 0 && tx == 0 && i < it.len) A.saved[stat_at(A.n_stat, h, it.stat0 + i) + STAT_ROWS] = delta[a];
  }
  f32x2 out[4][DP / 32] = {};
  for (int n = team; n < kt.count(); n += TEAMS<DP>) {
    const int j0 = kt.tile(n) * BT;
    float p[4][NB], ds[4][NB];
    scores<DP>(dO, V, A.D, ty, tx, ds);
    arrived<0>();
    sync_team(team);      // K is there, V is done with
    load(V, A.v, n + TEAMS<DP>);
    scores<DP>(Q, K, A.D, ty, tx, p);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        grad_one(A, it.len, own0 + 4 * ty + a, j0 + tx + 16 * b, l2[a], delta[a], p[a][b], ds[a][b]);
        S[(4 * ty + a) * PROW + tx + 16 * b] = ds[a][b];
      }
    __syncwarp();
    accumulate<DP>(S, K, ty, tx, out);
    arrived<0>();
    sync_team(team);      // the next V is there, K is done with
    load(K, A.k, n + TEAMS<DP>);
  }
  f32x2* const shares = reinterpret_cast<f32x2*>(dO + OWN * ROW<DP>) + tid;
  if (team) {
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) shares[team * (MINE / 2) + (a * (DP / 32) + c) * TEAM] = out[a][c];
  }
  __syncthreads();
  if (team) return;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int t = 1; t < TEAMS<DP>; ++t)
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) add2(out[a][c], shares[t * (MINE / 2) + (a * (DP / 32) + c) * TEAM]);
  const float f[4] = {A.scale, A.scale, A.scale, A.scale};
  store_rows<DP>(A.dq, it.seq0, own0, it.len, h, A.D, ty, tx, out, f);
}

__device__ __forceinline__ void sync_cluster() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 8 bytes of another block of the cluster's shared memory, by their place in this block's
__device__ __forceinline__ f32x2 remote(const f32x2* p, int rank) {
  f32x2 v;
  asm volatile("{\n\t.reg .b32 at;\n\tmapa.shared::cluster.u32 at, %1, %2;\n\tld.shared::cluster.b64 %0, [at];\n\t}"
               : "=l"(v)
               : "r"(smem_u32(p)), "r"(rank)
               : "memory");
  return v;
}

template <int DP, int CLUSTER, bool SPLIT>
__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(THREADS<DP>) k_attn_simt_dkdv(const AttnArgs A) {
  griddep_wait();
  extern __shared__ float4 smem4[];
  const int team = threadIdx.x / TEAM, tid = threadIdx.x % TEAM, ty = tid / 16, tx = tid % 16;
  float* K = reinterpret_cast<float*>(smem4);
  float* V = K + OWN * ROW<DP>;
  constexpr int MINE = 2 * BT * ROW<DP> + 2 * OWN * PROW;      // of a team
  float* Q = V + OWN * ROW<DP> + team * MINE;
  float* dO = Q + BT * ROW<DP>;
  float* S = dO + BT * ROW<DP>;
  float* P = S + OWN * PROW;
  // Without first tokens a cluster for each half of a piece.  With them, a larger cluster for each half of a piece that
  // holds some, and one for both halves of any other: the grid's first clusters are for the second halves of the former.
  const int at = blockIdx.x / CLUSTER, pieces = gridDim.x / (2 * CLUSTER), rank = blockIdx.x % CLUSTER;
  const AttnItem it = A.items[SPLIT ? at % pieces : at / 2];
  const bool second = SPLIT ? at < pieces : at % 2;
  const int h = it.sub;
  if (it.len == 0) {
    if (!second && !rank) zero_rows(A.dk, it, A.hk, A.D), zero_rows(A.dv, it, A.hk, A.D);
    return;
  }
  const bool alone = !SPLIT || it.i0 < A.n_sink;
  if (!alone && second) return;
  const int half = alone ? second : rank / (CLUSTER / 2), share = alone ? CLUSTER : CLUSTER / 2;
  const int part = rank % share, rank0 = rank - part;
  // (a half behind the sequence's end has no tiles; as half of a cluster it takes part in the cluster's barriers)
  const int j0 = it.i0 + OWN * half, j1 = min(j0 + OWN, it.len);
  if (alone && j0 >= it.len) return;
  int lo = 0, hi = 0;
  if (j0 < it.len) query_rows(j0, j1, it.len, A.window, A.n_sink, lo, hi);
  const int from = lo / BT * BT, per = (hi - from + BT - 1) / BT, total = per * A.group;
  load_tile<DP, OWN>(K, A.k, it.seq0, j0, it.len, h, A.D, threadIdx.x, THREADS<DP>);
  load_tile<DP, OWN>(V, A.v, it.seq0, j0, it.len, h, A.D, threadIdx.x, THREADS<DP>);
  auto load = [&](float* dst, const mlora_heads& t, int n) {
    if (n < total) load_tile<DP, BT>(dst, t, it.seq0, from + n % per * BT, it.len, h * A.group + n / per, A.D, tid, TEAM);
    commit();
  };
  const int stride = TEAMS<DP> * share, turn = part * TEAMS<DP> + team;
  load(dO, A.dout, turn);
  load(Q, A.q, turn);
  arrived<1>();
  __syncthreads();
  f32x2 dk[4][DP / 32] = {}, dv[4][DP / 32] = {};
  for (int n = turn; n < total; n += stride) {
    const int i0 = from + n % per * BT;
    float l2[NB], delta[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int i = i0 + tx + 16 * b;
      const long long at = stat_at(A.n_stat, h * A.group + n / per, it.stat0 + i);
      l2[b] = i < it.len ? A.saved[at] : 0.f;
      delta[b] = i < it.len ? A.saved[at + STAT_ROWS] : 0.f;
    }
    float p[4][NB], ds[4][NB];
    scores<DP>(V, dO, A.D, ty, tx, ds);
    arrived<0>();
    sync_team(team);      // Q is there
    scores<DP>(K, Q, A.D, ty, tx, p);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        grad_one(A, it.len, i0 + tx + 16 * b, j0 + 4 * ty + a, l2[b], delta[b], p[a][b], ds[a][b]);
        P[(4 * ty + a) * PROW + tx + 16 * b] = p[a][b];
        S[(4 * ty + a) * PROW + tx + 16 * b] = ds[a][b];
      }
    __syncwarp();
    accumulate<DP>(P, dO, ty, tx, dv);
    sync_team(team);      // dO is done with
    load(dO, A.dout, n + stride);
    accumulate<DP>(S, Q, ty, tx, dk);
    arrived<0>();
    sync_team(team);      // the next dO is there, Q is done with
    load(Q, A.q, n + stride);
  }
  // every team's sums through its tiles' memory; each block adds up and stores its share of the rows, one team dK,
  // the other dV
  f32x2* const sums = reinterpret_cast<f32x2*>(V + OWN * ROW<DP>) + tid;
  constexpr int TEAM_FAR = MINE / 2, SUMS = 4 * (DP / 32) * TEAM;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int c = 0; c < DP / 32; ++c) {
      sums[team * TEAM_FAR + (a * (DP / 32) + c) * TEAM] = dk[a][c];
      sums[team * TEAM_FAR + SUMS + (a * (DP / 32) + c) * TEAM] = dv[a][c];
    }
  sync_cluster();
  if (team < 2) {
    const mlora_heads& to = team ? A.dv : A.dk;
    const float f = team ? 1.f : A.scale;
    for (int a = part; a < 4; a += share) {
      const int j = j0 + 4 * ty + a;
      f32x2 t[DP / 32] = {};
      for (int q = 0; q < share; ++q)
#pragma unroll
        for (int k = 0; k < TEAMS<DP>; ++k)
#pragma unroll
          for (int c = 0; c < DP / 32; ++c)
            add2(t[c], remote(sums + k * TEAM_FAR + team * SUMS + (a * (DP / 32) + c) * TEAM, rank0 + q));
      if (j < it.len) {
        float* y = head_row<float>(to, static_cast<long long>(it.seq0) + j, h);
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) {
          const float2 v = both(t[c]);
          const int d = 32 * c + 2 * tx;
          if (d < A.D) *reinterpret_cast<float2*>(y + d) = make_float2(v.x * f, v.y * f);
        }
      }
    }
  }
  sync_cluster();      // the others have read this block's memory
}

// pdl: the launch goes under the end of the kernel before
template <typename K>
cudaError_t go(K kernel, int blocks, int threads, int floats, std::atomic<unsigned long long>& done, cudaStream_t s,
               const AttnArgs& A, bool pdl = false) {
  if (blocks == 0) return cudaSuccess;
  cudaError_t e = ensure_smem_attr(kernel, floats * 4, done);
  if (e != cudaSuccess) return e;
  e = launch_k(kernel, dim3(blocks), dim3(threads), floats * 4, s, pdl, A);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

constexpr int HALVES = PIECE / OWN;

template <int DP>
cudaError_t forward(const AttnArgs& A, int n, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const int floats = (OWN + 2 * TEAMS<DP> * BT) * ROW<DP> + TEAMS<DP> * OWN * PROW;
  return go(k_attn_simt_fwd<DP>, n * HALVES, THREADS<DP>, floats, done, s, A);
}

template <int DP>
cudaError_t backward(AttnArgs A, const AttnItem* q, int nq, const AttnItem* k, int nk, cudaStream_t s) {
  static std::atomic<unsigned long long> done1{0}, done2{0}, done4{0};
  A.items = q;
  int floats = (2 * OWN + 2 * TEAMS<DP> * BT) * ROW<DP> + TEAMS<DP> * OWN * PROW;
  cudaError_t e = go(k_attn_simt_dq<DP>, nq * HALVES, THREADS<DP>, floats, done1, s, A);
  A.items = k;
  if (e != cudaSuccess) return e;
  // Key tiles with first tokens meet the queries of the whole sequence, others those of the window; by the plan's
  // parameters alone, so a sequence's gradients do not depend on the pack.  Four sequences of 33 to 700, window 200:
  // with a first token 82 microseconds for the backward with four blocks a cluster and pieces without first tokens in one
  // (93 with each half in one, 108 with two blocks a cluster); without, 79 with two, 85 with one.
  floats += TEAMS<DP> * OWN * PROW;
  return A.n_sink > 0 ? go(k_attn_simt_dkdv<DP, 4, true>, nk * HALVES * 4, THREADS<DP>, floats, done4, s, A, true)
                      : go(k_attn_simt_dkdv<DP, 2, false>, nk * HALVES * 2, THREADS<DP>, floats, done2, s, A, true);
}

}  // namespace

cudaError_t launch_attn_simt_forward(const AttnArgs& A, int n, cudaStream_t s) {
  if (A.D <= 32) return forward<32>(A, n, s);
  if (A.D <= 64) return forward<64>(A, n, s);
  return A.D <= 96 ? forward<96>(A, n, s) : forward<128>(A, n, s);
}

cudaError_t launch_attn_simt_backward(const AttnArgs& A, const AttnItem* q, int nq, const AttnItem* k, int nk,
                                      cudaStream_t s) {
  if (A.D <= 32) return backward<32>(A, q, nq, k, nk, s);
  if (A.D <= 64) return backward<64>(A, q, nq, k, nk, s);
  return A.D <= 96 ? backward<96>(A, q, nq, k, nk, s) : backward<128>(A, q, nq, k, nk, s);
}

}  // namespace mlora
