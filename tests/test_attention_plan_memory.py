"""How much memory the attention's plans ask for, without a GPU."""
import pytest

from adapter_gemm_packed_gb300 import _mlora as M


@pytest.fixture(scope="module", autouse=True)
def built():
    from adapter_gemm_packed_gb300 import build
    build.build()


def _plan(lens, hq, hk, d, window, sinks):
    p = M.mlora_attention_problem(sum(lens), hq, hk, d, window, sinks, M.MLORA_BF16, 0.1, M.MLORA_PLAN_HOST_ONLY)
    return M.mlora_attention_plan(p, [sum(lens[:i]) for i in range(len(lens))], lens)


@pytest.mark.parametrize("lens,window,sinks", [([131072], 128, 65536), ([131072], 128, 131072), ([40000, 300], 64, 20000),
                                               ([131072], 131072, 0), ([16384], 4096, 64), ([3000] * 4, 1, 2999)])
def test_sums_of_cut_pieces_are_bounded(lens, window, sinks):
    """At most two parts a piece on average, each with sums of 128 rows of dK and dV, whatever the mask: with a window of 128
    and 65,536 first tokens in 131,072 it was 64 parts for every second piece, 34 GB."""
    hq, hk, d = 32, 8, 128
    h = _plan(lens, hq, hk, d, window, sinks)
    rows = sum(-(-n // 128) * 128 for n in lens)
    pieces = sum(-(-n // 128) for n in lens) * hk
    parts = M.mlora_attention_describe(h, M.MLORA_ATTN_Q_KEYS)[6::8]
    assert len(parts) <= 2 * pieces
    fixed = 2 * rows * hq + rows * hq * d // 4 + pieces * 8      # statistics, low bytes, counters
    assert M.mlora_attention_saved_elems(h) <= fixed + 2 * pieces * 2 * 128 * d
    M.mlora_attention_plan_destroy(h)


@pytest.mark.parametrize("lens,window,sinks,group", [([16384], 4096, 64, 4), ([2600], 2600, 0, 4), ([4200, 30], 200, 70, 4),
                                                     ([97, 2501, 1300], 2048, 0, 4), ([131072], 131072, 0, 4)])
def test_ordinary_pieces_are_cut_as_before(lens, window, sinks, group):
    """Windows with few first tokens, and plain causal attention: parts as long as the window's tiles, or half the
    sequence's, or 128."""
    h = _plan(lens, 2 * group, 2, 64, window, sinks)
    t = M.mlora_attention_describe(h, M.MLORA_ATTN_Q_KEYS)
    for length, i0, parts in zip(t[1::8], t[2::8], t[6::8]):
        usual = max(128, min((window + 126) // 64 + 1, (length // 64 + 2) // 2) * group)
        hi = length if i0 < sinks else min(length, min(i0 + 128, length) + window - 1)
        assert parts == -(-((-(-hi // 64) - i0 // 64) * group) // usual)
    M.mlora_attention_plan_destroy(h)


def test_plans_of_many_samples_take_time_in_proportion():
    """60,000 samples: a fraction of a second (adding up the lengths before each one took nine)."""
    import time
    from adapter_gemm_packed_gb300.attention import WindowAttention
    t = time.perf_counter()
    attn = WindowAttention([1, 2] * 30000, 1, 1, 64, 8, flags=M.MLORA_PLAN_HOST_ONLY)
    assert time.perf_counter() - t < 5
    p = M.mlora_attention_describe(attn.plan, M.MLORA_ATTN_Q_QUERIES)
    assert attn.n == 90000 and sorted(p[0::8]) == sorted(x for i in range(30000) for x in (3 * i, 3 * i + 1))
    attn.close()


@pytest.mark.parametrize("dtype", [M.MLORA_BF16, M.MLORA_F32])
def test_what_a_graph_keeps_has_no_scratch_in_it(dtype):
    """Statistics, 8 bytes a row and head, and for bf16 a byte an output element; the sums of cut pieces are the backward's
    workspace."""
    from adapter_gemm_packed_gb300.attention import WindowAttention
    for lens, cut in (([131072], True), ([300, 50], False)):
        p = M.mlora_attention_problem(sum(lens), 32, 8, 128, 10**6, 0, dtype, 0.1, M.MLORA_PLAN_HOST_ONLY)
        h = M.mlora_attention_plan(p, [sum(lens[:i]) for i in range(len(lens))], lens)
        rows = sum(-(-n // 128) * 128 for n in lens)
        kept, work = M.mlora_attention_kept_elems(h), M.mlora_attention_workspace_elems(h)
        assert kept == rows * 32 * (2 + (128 // 4 if dtype == M.MLORA_BF16 else 0))
        assert (work > 0) == (cut and dtype == M.MLORA_BF16)
        assert M.mlora_attention_saved_elems(h) == kept + work
        M.mlora_attention_plan_destroy(h)
        attn = WindowAttention(lens, 32, 8, 128, 10**6, dtype="bf16" if dtype == M.MLORA_BF16 else "f32",
                               flags=M.MLORA_PLAN_HOST_ONLY)
        assert attn.saved_elems == kept
        attn.close()
