// Entry points of the windowed attention over packed sequences: the plan (sequence table, work lists,
// layout of the saved statistics), argument checks and launches.  See include/mlora.h for the contract.
//
// Work lists: one piece per tile of rows of a sequence and head (pair of heads in the forward), in one list for
// each of the kernels that own query rows (forward, dQ) and one for the kernel that owns keys.  A piece's work is
// the number of tiles of the other side that it meets, which the window bounds and the sequence's start (queries)
// or end (keys) cut short.  The fp32 kernels run one block per piece, in order of falling work.  The bf16 kernels
// run one block per SM with a list of its own, made by greedy longest-first list scheduling.  Pieces of the dK / dV
// kernel longer than what is usual in their sequence (first tokens, which every later query sees; early keys
// without a window) are cut along their query tiles.  The cut looks at nothing but the sequence itself, so a
// sequence's gradients do not depend, not in one bit, on what else is in the pack.  Rows that belong to no sequence
// are pieces too, which write zeros.
#include <algorithm>
#include <cmath>
#include <limits>
#include <new>
#include <queue>
#include <vector>

#include "attention.cuh"

using namespace mlora;

struct WorkList {
  std::vector<AttnItem> items;
  std::vector<int> first;      // block b does items [first[b], first[b + 1])
  AttnItem* d_items = nullptr;
  int* d_first = nullptr;
  int blocks() const { return static_cast<int>(first.size()) - 1; }
};

struct mlora_attention_plan_s {
  mlora_attention_problem prob;
  WorkList f, q, k;            // forward, dQ, dK / dV
  long long n_stat = 0;
  int n_slots = 0, n_parts = 0;      // cut dK / dV pieces, and their parts
  int device = -1, sms = 152;
  bool on_device = false;
  void* dev_block = nullptr;   // status word (256 bytes), then the lists
  int* d_err = nullptr;
  unsigned long long timeout_ns = 4000000000ull;
};

namespace {

constexpr int STAT_PAD = 128;     // a sequence's statistics start at a multiple of this many rows

mlora_status check_problem(const mlora_attention_problem* p) {
  if (!p) return op_fail(MLORA_ERR_INVALID, "null problem");
  if (p->dtype != MLORA_BF16 && p->dtype != MLORA_F32)
    return op_fail(MLORA_ERR_UNSUPPORTED, "queries, keys and values are bf16 or fp32");
  if (p->n_tokens < 1 || p->n_tokens > std::numeric_limits<int32_t>::max() - 2 * STAT_PAD)
    return op_fail(MLORA_ERR_INVALID, "n_tokens out of range");
  if (p->n_kv_heads < 1 || p->n_q_heads < 1 || p->n_q_heads > 4096 || p->n_q_heads % p->n_kv_heads)
    return op_fail(MLORA_ERR_INVALID, "n_q_heads must be a multiple of n_kv_heads (at most 4096)");
  if (p->head_dim < 8 || p->head_dim > 128 || p->head_dim % 8)
    return op_fail(MLORA_ERR_UNSUPPORTED, "head_dim must be a multiple of 8, at most 128");
  if (p->window < 1) return op_fail(MLORA_ERR_INVALID, "the window must hold at least the token itself");
  if (p->n_sink < 0) return op_fail(MLORA_ERR_INVALID, "n_sink must not be negative");
  if (!std::isfinite(p->scale)) return op_fail(MLORA_ERR_INVALID, "the scale must be finite");
  if (p->flags & ~(MLORA_PLAN_HOST_ONLY | MLORA_DEBUG_SHORT_TIMEOUT))
    return op_fail(MLORA_ERR_INVALID, "unknown flag");
  return MLORA_OK;
}

void build(mlora_attention_plan_s* P, const int64_t* starts, const int32_t* lens, int32_t n_seqs) {
  const mlora_attention_problem& pr = P->prob;
  const bool f32 = pr.dtype == MLORA_F32;
  const int group = pr.n_q_heads / pr.n_kv_heads;
  struct Cost { int64_t c; AttnItem it; };
  std::vector<AttnItem> gaps;
  auto gap = [&](int64_t from, int64_t to) {      // 64 rows a piece
    for (; from < to; from += 64)
      gaps.push_back(AttnItem{static_cast<int>(from), 0, static_cast<int>(std::min<int64_t>(64, to - from)), 0, 0, 0, 1, 0, 0});
  };
  int64_t at = 0, stat = 0;
  std::vector<int> stat0(n_seqs);
  for (int32_t i = 0; i < n_seqs; ++i) {
    gap(at, starts[i]);
    at = starts[i] + lens[i];
    stat0[i] = static_cast<int>(stat);
    stat += (static_cast<int64_t>(lens[i]) + STAT_PAD - 1) / STAT_PAD * STAT_PAD;
  }
  gap(at, pr.n_tokens);
  P->n_stat = stat;

  // rows: of a piece; subs: pieces per tile; over: a piece's cost besides its tiles, in tiles
  auto fill = [&](WorkList& to, int rows, int subs, bool keys, int tile, int over) {
    std::vector<Cost> list;
    // tiles that the piece of sequence i from row i0 on streams
    auto cost = [&](int32_t i, int64_t i0) {
      const int a = static_cast<int>(i0), b = static_cast<int>(std::min<int64_t>(i0 + rows, lens[i]));
      if (!keys) return static_cast<int64_t>(key_tiles(a, b, pr.window, pr.n_sink, tile).count());
      int lo, hi;
      query_rows(a, b, lens[i], pr.window, pr.n_sink, lo, hi);
      return static_cast<int64_t>((hi + tile - 1) / tile - lo / tile) * group;
    };
    for (int32_t i = 0; i < n_seqs; ++i) {
      // What an ordinary piece of this sequence streams: its window, or half the sequence where that is less; at least
      // 128 tiles.  Where so many keys are first tokens that their pieces would make more than two parts a piece, the
      // mean, which cannot: the sums of every part take a kilobyte a column of the workspace.
      int64_t usual = std::numeric_limits<int64_t>::max();
      if (keys && !f32) {
        usual = std::max<int64_t>(std::min<int64_t>((pr.window + 126) / 64 + 1, (lens[i] / 64 + 2) / 2) * group, 128);
        int64_t n = 0, sum = 0, parts = 0;
        for (int64_t i0 = 0; i0 < lens[i]; i0 += rows, ++n) sum += cost(i, i0), parts += (cost(i, i0) + usual - 1) / usual;
        if (parts > 2 * n) usual = std::max(usual, (sum + n - 1) / n);
      }
      for (int64_t i0 = 0; i0 < lens[i]; i0 += rows) {
        const int a = static_cast<int>(i0);
        const int64_t c = cost(i, i0), parts = keys && !f32 ? std::min<int64_t>((c + usual - 1) / usual, 4096) : 1;
        for (int h = 0; h < subs; ++h) {
          AttnItem it{static_cast<int>(starts[i]), lens[i], a, stat0[i], h, 0, static_cast<short>(parts), 0, 0};
          if (parts > 1) it.slot = P->n_slots++, it.pbase = P->n_parts, P->n_parts += static_cast<int>(parts);
          for (int64_t p = 0; p < parts; ++p) {
            it.part = static_cast<short>(p);
            list.push_back({c * (p + 1) / parts - c * p / parts + over, it});
          }
        }
      }
    }
    std::stable_sort(list.begin(), list.end(), [](const Cost& x, const Cost& y) { return x.c > y.c; });
    for (const AttnItem& g : gaps) list.push_back({1, g});
    const int n = static_cast<int>(list.size()), blocks = f32 ? n : std::min(n, P->sms);
    std::vector<std::vector<int>> of(blocks);
    typedef std::pair<int64_t, int> Load;
    std::priority_queue<Load, std::vector<Load>, std::greater<Load>> least;
    for (int b = 0; b < blocks; ++b) least.push({0, b});
    for (int e = 0; e < n; ++e) {
      Load l = least.top();
      least.pop();
      of[l.second].push_back(e);
      least.push({l.first + list[e].c, l.second});
    }
    to.first.push_back(0);
    for (const auto& mine : of) {
      for (int e : mine) to.items.push_back(list[e].it);
      to.first.push_back(static_cast<int>(to.items.size()));
    }
  };
  if (f32) {
    fill(P->f, 64, pr.n_q_heads, false, 64, 1);
    fill(P->q, 64, pr.n_q_heads, false, 64, 1);
    fill(P->k, 64, pr.n_kv_heads, true, 64, 1);
  } else {
    fill(P->f, attn_fwd_rows(group), pr.n_kv_heads * attn_fwd_pairs(group), false, 128, 2);
    fill(P->q, 128, pr.n_q_heads, false, 64, 3);
    fill(P->k, 128, pr.n_kv_heads, true, 64, 4);
  }
}

mlora_status upload(mlora_attention_plan_s* P) {
  WorkList* const lists[] = {&P->f, &P->q, &P->k};
  size_t bytes = 256;
  for (WorkList* l : lists) bytes += l->items.size() * sizeof(AttnItem) + (l->first.size() + 3) / 4 * 16;
  cudaError_t e = cudaMalloc(&P->dev_block, bytes);
  if (e == cudaErrorMemoryAllocation) {
    cudaGetLastError();
    return op_fail(MLORA_ERR_OOM, "the attention plan's device tables could not be allocated");
  }
  if (e != cudaSuccess) return op_cuda_fail(e, "allocating the attention plan's device tables");
  uint8_t* b = static_cast<uint8_t*>(P->dev_block);
  P->d_err = reinterpret_cast<int*>(b);
  e = cudaMemset(b, 0, 256);
  b += 256;
  for (WorkList* l : lists) {
    l->d_first = reinterpret_cast<int*>(b);
    if (e == cudaSuccess) e = cudaMemcpy(b, l->first.data(), l->first.size() * sizeof(int), cudaMemcpyHostToDevice);
    b += (l->first.size() + 3) / 4 * 16;
    l->d_items = reinterpret_cast<AttnItem*>(b);
    if (e == cudaSuccess && !l->items.empty())
      e = cudaMemcpy(b, l->items.data(), l->items.size() * sizeof(AttnItem), cudaMemcpyHostToDevice);
    b += l->items.size() * sizeof(AttnItem);
  }
  // the copies must have arrived before kernels of any other stream read the tables
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  if (e != cudaSuccess) return op_cuda_fail(e, "uploading the attention plan");
  P->on_device = true;
  return MLORA_OK;
}

mlora_status check_run(const mlora_attention_plan_t* P) {
  if (!P) return op_fail(MLORA_ERR_INVALID, "null plan");
  if (!P->on_device) return op_fail(MLORA_ERR_INVALID, "plan was built with MLORA_PLAN_HOST_ONLY");
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != P->device)
    return op_fail(MLORA_ERR_INVALID, "the current device is not the one the plan was built on");
  const cudaError_t e = cudaSetDevice(dev);      // makes the primary context current on this thread
  return e == cudaSuccess ? MLORA_OK : op_cuda_fail(e, "cudaSetDevice");
}

// `saved`: the statistics; then for bf16 the outputs' low bits.  The backward's workspace, there or elsewhere: the counters
// of cut dK / dV pieces and their sums.
struct SavedLayout {
  int64_t low, kept, sums, scratch;      // in floats
};
SavedLayout saved_layout(const mlora_attention_plan_t* P) {
  SavedLayout L{};
  const int64_t rows = P->n_stat * P->prob.n_q_heads, cols = P->prob.head_dim <= 64 ? 64 : 128;
  L.low = 2 * rows;
  L.kept = L.low;
  if (P->prob.dtype == MLORA_BF16) {
    L.kept += rows * cols / 4;
    L.sums = static_cast<int64_t>(P->n_slots) * 8;
    L.scratch = L.sums + static_cast<int64_t>(P->n_parts) * 2 * 128 * cols;
  }
  return L;
}

AttnArgs args_of(const mlora_attention_plan_t* P, float* saved, float* work, const WorkList& list) {
  AttnArgs A{};
  const SavedLayout L = saved_layout(P);
  A.saved = saved;
  A.out_low = reinterpret_cast<uint8_t*>(saved + L.low);
  A.part_cnt = reinterpret_cast<int*>(work);
  A.partials = work + L.sums;
  A.n_cnt = P->n_slots * 8;
  A.first = list.d_first;
  const mlora_attention_problem& p = P->prob;
  A.items = list.d_items;
  A.hq = p.n_q_heads, A.hk = p.n_kv_heads, A.group = p.n_q_heads / p.n_kv_heads, A.D = p.head_dim;
  A.window = p.window, A.n_sink = p.n_sink;
  A.scale = p.scale;
  A.scale_log2 = static_cast<float>(p.scale * 1.4426950408889634);
  A.n_stat = P->n_stat;
  A.err = P->d_err;
  A.timeout_ns = P->timeout_ns;
  return A;
}

mlora_status check_tensor(const mlora_attention_plan_t* P, const mlora_heads* t, const char* name, bool q) {
  const mlora_attention_problem& p = P->prob;
  return check_heads(t, name, p.n_tokens, q ? p.n_q_heads : p.n_kv_heads, p.head_dim, p.dtype == MLORA_F32 ? 4 : 2);
}

}  // namespace

extern "C" {

mlora_status mlora_attention_plan(const mlora_attention_problem* problem, const int64_t* seq_start,
                                  const int32_t* seq_len, int32_t n_seqs, mlora_attention_plan_t** out) {
  set_last_error("");
  if (!out) return op_fail(MLORA_ERR_INVALID, "null output pointer");
  *out = nullptr;
  mlora_status st = check_problem(problem);
  if (st != MLORA_OK) return st;
  if (n_seqs < 0 || (n_seqs > 0 && (!seq_start || !seq_len)))
    return op_fail(MLORA_ERR_INVALID, "null or negative sequence table");
  int64_t at = 0, stat = 0;
  for (int32_t i = 0; i < n_seqs; ++i) {
    if (seq_len[i] < 0 || seq_start[i] < at || seq_start[i] > problem->n_tokens - seq_len[i])
      return op_fail(MLORA_ERR_INVALID, "sequences must lie in [0, n_tokens) in order, without overlap");
    at = seq_start[i] + seq_len[i];
    stat += (static_cast<int64_t>(seq_len[i]) + STAT_PAD - 1) / STAT_PAD * STAT_PAD;
  }
  if (stat > std::numeric_limits<int32_t>::max())
    return op_fail(MLORA_ERR_UNSUPPORTED, "too many rows of statistics");
  mlora_attention_plan_s* P = new (std::nothrow) mlora_attention_plan_s();
  if (!P) return op_fail(MLORA_ERR_OOM, "host allocation failed");
  P->prob = *problem;
  if (problem->flags & MLORA_DEBUG_SHORT_TIMEOUT) P->timeout_ns = 1000000ull;
  // a window or a number of first tokens beyond the longest sequence changes nothing; cut to it, differences
  // of row numbers and either stay within 32 bits
  int32_t longest = 1;
  for (int32_t i = 0; i < n_seqs; ++i) longest = std::max(longest, seq_len[i]);
  P->prob.window = std::min(problem->window, longest);
  P->prob.n_sink = std::min(problem->n_sink, longest);
  // how many pieces there may be: two lists of tiles x query heads, and gaps
  if ((stat / 64 + problem->n_tokens / 64 + n_seqs) * problem->n_q_heads > (int64_t(1) << 28)) {
    delete P;
    return op_fail(MLORA_ERR_UNSUPPORTED, "too many pieces of work");
  }
  if (!(problem->flags & MLORA_PLAN_HOST_ONLY)) {
    cudaError_t e = cudaGetDevice(&P->device);
    if (e == cudaSuccess) e = device_sms(&P->sms);
    if (e != cudaSuccess) {
      delete P;
      return op_cuda_fail(e, "querying the device");
    }
  }
  try {
    build(P, seq_start, seq_len, n_seqs);
  } catch (...) {      // no exception crosses the ABI
    delete P;
    return op_fail(MLORA_ERR_OOM, "host allocation failed");
  }
  if (!(problem->flags & MLORA_PLAN_HOST_ONLY)) {
    st = upload(P);
    if (st != MLORA_OK) {
      mlora_attention_plan_destroy(P);
      return st;
    }
  }
  *out = P;
  return MLORA_OK;
}

void mlora_attention_plan_destroy(mlora_attention_plan_t* plan) {
  if (!plan) return;
  if (plan->dev_block) cudaFree(plan->dev_block);
  delete plan;
}

int64_t mlora_attention_saved_elems(const mlora_attention_plan_t* plan) {
  if (!plan) return -1;
  const SavedLayout L = saved_layout(plan);
  return L.kept + L.scratch;
}

int64_t mlora_attention_kept_elems(const mlora_attention_plan_t* plan) { return plan ? saved_layout(plan).kept : -1; }

int64_t mlora_attention_workspace_elems(const mlora_attention_plan_t* plan) {
  return plan ? saved_layout(plan).scratch : -1;
}

mlora_status mlora_attention_forward(const mlora_attention_plan_t* P, const mlora_heads* q, const mlora_heads* k,
                                     const mlora_heads* v, const mlora_heads* out, float* saved, void* stream) {
  mlora_status st = check_run(P);
  if (st == MLORA_OK) st = check_tensor(P, q, "q", true);
  if (st == MLORA_OK) st = check_tensor(P, k, "k", false);
  if (st == MLORA_OK) st = check_tensor(P, v, "v", false);
  if (st == MLORA_OK) st = check_tensor(P, out, "out", true);
  if (st != MLORA_OK) return st;
  if (!saved || !ptr_aligned(saved, 16)) return op_fail(MLORA_ERR_INVALID, "saved must be a 16-byte aligned buffer");
  AttnArgs A = args_of(P, saved, nullptr, P->f);
  A.q = *q, A.k = *k, A.v = *v, A.o = *out;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (P->prob.dtype == MLORA_BF16) return launch_attn_fwd(A, P->f.blocks(), P->prob.n_tokens, s);
  const cudaError_t e = launch_attn_simt_forward(A, P->f.blocks(), s);
  return e == cudaSuccess ? MLORA_OK : op_cuda_fail(e, "attention forward launch");
}

mlora_status mlora_attention_backward(const mlora_attention_plan_t* P, const mlora_heads* q, const mlora_heads* k,
                                      const mlora_heads* v, const mlora_heads* out, const mlora_heads* dout,
                                      float* saved, const mlora_heads* dq, const mlora_heads* dk,
                                      const mlora_heads* dv, void* stream) {
  return mlora_attention_backward_ws(P, q, k, v, out, dout, saved, P && saved ? saved + saved_layout(P).kept : nullptr, dq,
                                     dk, dv, stream);
}

mlora_status mlora_attention_backward_ws(const mlora_attention_plan_t* P, const mlora_heads* q, const mlora_heads* k,
                                         const mlora_heads* v, const mlora_heads* out, const mlora_heads* dout,
                                         float* saved, float* workspace, const mlora_heads* dq, const mlora_heads* dk,
                                         const mlora_heads* dv, void* stream) {
  mlora_status st = check_run(P);
  const struct { const mlora_heads* t; const char* name; bool q; } all[] = {
      {q, "q", true}, {k, "k", false}, {v, "v", false}, {out, "out", true}, {dout, "dout", true},
      {dq, "dq", true}, {dk, "dk", false}, {dv, "dv", false}};
  for (const auto& a : all)
    if (st == MLORA_OK) st = check_tensor(P, a.t, a.name, a.q);
  if (st != MLORA_OK) return st;
  if (!saved || !ptr_aligned(saved, 16)) return op_fail(MLORA_ERR_INVALID, "saved must be a 16-byte aligned buffer");
  if (saved_layout(P).scratch && (!workspace || !ptr_aligned(workspace, 16)))
    return op_fail(MLORA_ERR_INVALID, "the plan's cut pieces need a 16-byte aligned workspace");
  AttnArgs A = args_of(P, saved, workspace, P->q), K = args_of(P, saved, workspace, P->k);
  for (AttnArgs* a : {&A, &K})
    a->q = *q, a->k = *k, a->v = *v, a->o = *out, a->dout = *dout, a->dq = *dq, a->dk = *dk, a->dv = *dv;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (P->prob.dtype == MLORA_BF16) return launch_attn_bwd(A, P->q.blocks(), K, P->k.blocks(), P->prob.n_tokens, s);
  const cudaError_t e = launch_attn_simt_backward(A, P->q.d_items, P->q.blocks(), P->k.d_items, P->k.blocks(), s);
  return e == cudaSuccess ? MLORA_OK : op_cuda_fail(e, "attention backward launch");
}

mlora_status mlora_attention_sync_status(const mlora_attention_plan_t* P, void* stream) {
  mlora_status st = check_run(P);
  if (st != MLORA_OK) return st;
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return op_cuda_fail(e, "cudaStreamSynchronize");
  int v = 0;
  e = cudaMemcpy(&v, P->d_err, sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && v) e = cudaMemset(P->d_err, 0, sizeof(int));
  if (e != cudaSuccess) return op_cuda_fail(e, "reading the status word");
  if (v) {
    char buf[96];
    snprintf(buf, sizeof buf, "a device-side wait gave up (code 0x%x)", v);
    return op_fail(MLORA_ERR_TIMEOUT, buf);
  }
  return MLORA_OK;
}

mlora_status mlora_attention_describe(const mlora_attention_plan_t* P, int32_t what, int64_t* out, int64_t cap,
                                      int64_t* count) {
  if (!P || !count) return op_fail(MLORA_ERR_INVALID, "null plan or count");
  if (what < MLORA_ATTN_Q_QUERIES || what > MLORA_ATTN_Q_FORWARD) return op_fail(MLORA_ERR_INVALID, "unknown table");
  const WorkList& l = what == MLORA_ATTN_Q_FORWARD ? P->f : (what == MLORA_ATTN_Q_QUERIES ? P->q : P->k);
  *count = static_cast<int64_t>(l.items.size()) * 8;
  for (int b = 0; out && b < l.blocks(); ++b)
    for (int i = l.first[b]; i < l.first[b + 1]; ++i) {
      const AttnItem& t = l.items[i];
      const int64_t v[8] = {t.seq0, t.len, t.i0, t.stat0, t.sub, t.part, t.parts, b};
      for (int c = 0; c < 8; ++c)
        if (static_cast<int64_t>(8) * i + c < cap) out[8 * i + c] = v[c];
    }
  return MLORA_OK;
}

}  // extern "C"
