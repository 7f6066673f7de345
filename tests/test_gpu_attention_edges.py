"""Rows, sizes and arguments at which the attention and the norms can go wrong (needs a GB300)."""
import pytest
import torch

from adapter_gemm_packed_gb300 import _mlora as M
import op_reference as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adapter_gemm_packed_gb300 import build
    build.build()


def _draw(shape, seed, dt, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dt).cuda()


# ------------------------------------------------------------------ rows that see one key

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (3, 3, 128), (8, 1, 72)])
@pytest.mark.parametrize("lens,window,sinks", [([1] * 20, 1, 0), ([1] * 5, 40, 3), ([300, 1, 65, 129], 1, 0),
                                               ([200, 1, 64, 3], 50, 0), ([130, 1, 2], 1, 2), ([1, 400, 1], 10**6, 5)])
def test_gradients_of_rows_that_see_one_key_are_zero(lens, window, sinks, hq, hk, d, dtype):
    """The softmax of one score is 1 whatever the score: dq of such a row is zero, and dk of a key that only such rows
    see; exactly, at scores of any size.  Values and outputs pass through: dv is the rows' sum, the output v."""
    from adapter_gemm_packed_gb300.attention import WindowAttention
    attn = WindowAttention(lens, hq, hk, d, window, n_sink=sinks, dtype=dtype)
    q, k, v, do = (_draw((attn.n, h, d), i, DT[dtype], 3.0) for i, h in enumerate((hq, hk, hk, hq)))
    o = attn.forward(q, k, v)
    dq, dk, dv = attn.backward(q, k, v, o, do)
    alone_q, alone_k, at = [], [], 0
    for n in lens:
        rows = list(range(at, at + n))
        alone_q += rows if window == 1 and sinks == 0 else rows[:1]
        alone_k += rows if window == 1 and sinks == 0 or n == 1 else []
        at += n
    assert (dq[alone_q] == 0).all()
    assert (dk[alone_k] == 0).all()
    assert torch.equal(o[alone_k], v[alone_k].repeat_interleave(hq // hk, 1))
    terms = do[alone_k].double().view(-1, hk, hq // hk, d)
    want = terms.sum(2)      # one rounding, and fp32 sums of a few terms
    assert ((dv[alone_k].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * terms.abs().sum(2)).all()
    others = [r for r in range(attn.n) if r not in set(alone_q)]
    assert all((dq[r] != 0).any() for r in others)
    assert attn.sync_status() == M.MLORA_OK
    attn.close()


# ------------------------------------------------------------------ delta

def _delta(attn, lens, h):
    """delta of head h as the backward left it in `saved`: blocks of 64 rows, 64 logarithms of sums, then 64 delta; each
    sequence's rows from a multiple of 128 on."""
    pads = [-(-n // 128) * 128 for n in lens]
    rows = attn.saved[:2 * sum(pads) * attn.hq].view(attn.hq, -1, 2, 64)[h, :, 1].reshape(-1)
    return torch.cat([rows[sum(pads[:i]):sum(pads[:i]) + n] for i, n in enumerate(lens)]).double().cpu()


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (3, 3, 72), (2, 1, 128), (2, 2, 40)])
@pytest.mark.parametrize("lens", [[2] * 40, [1, 3, 4, 5, 8, 130, 257], [500, 31]])
def test_delta_is_made_of_outputs_to_16_bits(lens, hq, hk, d):
    """delta = rowsum(dO O) from bf16 outputs and the bytes kept beside them.  Queries of zero weigh all visible values
    the same, which bf16 holds, so that the outputs are known: the values' mean, with many ties between two bf16 numbers
    where a row sees two or four.  A byte is the difference to the rounded output in units of 2^-8 of its last place, to
    the nearest (a unit off where 128 of them would be needed): 2^-15 of the output, and fp32 sums."""
    from adapter_gemm_packed_gb300.attention import WindowAttention
    attn = WindowAttention(lens, hq, hk, d, 10**6)
    q, k, v, do = (_draw((attn.n, h, d), i, torch.bfloat16) for i, h in enumerate((hq, hk, hk, hq)))
    q.zero_()
    v += 1      # (outputs away from zero)
    o = attn.forward(q, k, v)
    attn.backward(q, k, v, o, do)
    mean = torch.cat([x.cumsum(0) / torch.arange(1, len(x) + 1)[:, None, None]
                      for x in v.double().cpu().split(lens)]).repeat_interleave(hq // hk, 1)
    for h in range(hq):
        terms = do.double().cpu()[:, h] * mean[:, h]
        err = (_delta(attn, lens, h) - terms.sum(1)).abs()
        lim = (2.0 ** -15 + 2.0 ** -19) * terms.abs().sum(1)
        assert (err <= lim).all(), float((err / lim).max())
    attn.close()


def test_delta_is_not_biased():
    """Gradients of the outputs' signs add up every output's magnitude.  Errors of either sign, half a unit of 2^-15 at
    most, average out over 128 columns x 900 rows (to 2^-8 of a unit); cut off instead, they would all point one way (a third
    of a unit and more)."""
    from adapter_gemm_packed_gb300.attention import WindowAttention
    attn = WindowAttention([900], 2, 1, 128, 10**6)
    q, k, v = (_draw((900, h, 128), i, torch.bfloat16) for i, h in enumerate((2, 1, 1)))
    q.zero_()
    o = attn.forward(q, k, v)
    attn.backward(q, k, v, o, torch.sign(o))
    mean = v.double().cpu().cumsum(0) / torch.arange(1, 901)[:, None, None]
    for h in range(2):
        want = (mean[:, 0] * torch.sign(o[:, h].double().cpu())).sum()
        assert abs(float(_delta(attn, [900], h).sum() - want)) <= 2.0 ** -19 * float(want)
    attn.close()


# ------------------------------------------------------------------ arguments

def test_buffers_for_the_statistics():
    """A buffer of the caller's gives what the object's own gives; one that the kernels would write past the end of, or
    in another type, is refused before anything runs."""
    from adapter_gemm_packed_gb300.attention import WindowAttention
    attn = WindowAttention([70, 40], 4, 2, 64, 30, n_sink=1)
    q, k, v, do = (_draw((attn.n, h, 64), i, torch.bfloat16) for i, h in enumerate((4, 2, 2, 4)))
    o = attn.forward(q, k, v)
    want = (o, *attn.backward(q, k, v, o, do))
    n = attn.saved_elems
    mine = torch.empty(n, device="cuda")
    o = attn.forward(q, k, v, saved=mine)
    got = (o, *attn.backward(q, k, v, o, do, saved=mine))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for bad in (torch.empty(n - 1, device="cuda"), torch.empty(n, dtype=torch.bfloat16, device="cuda"), torch.empty(n),
                torch.empty(2 * n, device="cuda")[::2], torch.empty(n + 1, device="cuda")[1:]):
        for call in (lambda: attn.forward(q, k, v, saved=bad), lambda: attn.backward(q, k, v, o, do, saved=bad)):
            with pytest.raises(M.MloraError) as e:
                call()
            assert e.value.status == M.MLORA_ERR_INVALID
    attn.close()


# ------------------------------------------------------------------ norms with rotation

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 16), (128, 64), (40, 24), (96, 96)])
def test_positions_outside_the_tables_give_nan_in_every_element(d, rot, inter, dtype):
    """Those that are not rotated as well, forward and backward; the other tokens are what they are without it."""
    from adapter_gemm_packed_gb300.attention import qk_norm_rope, qk_norm_rope_backward
    n, hq, hk = 9, 6, 2
    q, k, dq, dk = (_draw((n, h, d), i, DT[dtype]) for i, h in enumerate((hq, hk, hq, hk)))
    w = [1 + 0.1 * _draw((d,), 7 + i, torch.float32) for i in range(2)]
    ang = torch.rand((50, rot // 2), generator=torch.Generator().manual_seed(1)) * 6.28
    tab = (*w, ang.cos().cuda(), ang.sin().cuda())
    good = torch.arange(n, dtype=torch.int32, device="cuda") * 5
    call = lambda pos: (*qk_norm_rope(q, k, *tab, pos, interleaved=inter),
                        *qk_norm_rope_backward(dq, dk, q, k, *tab, pos, interleaved=inter))
    want = call(good)
    pos = good.clone()
    pos[1], pos[4], pos[8] = -1, 50, 2**31 - 1
    got = call(pos)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[[1, 4, 8]] = True
    for a, b in zip(got[:4], want[:4]):
        assert a[bad].isnan().all() and torch.equal(a[~bad], b[~bad])
    assert got[4].isnan().all() and got[5].isnan().all()


# ------------------------------------------------------------------ autograd

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_that_start_anywhere(dtype):
    """A gradient that is a slice of another starts at any element, a broadcast one has strides of zero: both give what a
    tensor of its own gives."""
    from adapter_gemm_packed_gb300.attention import QKNormRope, WindowAttention
    n, hq, hk, d, dt = 40, 4, 2, 64, DT[dtype]
    attn, norm = WindowAttention([n], hq, hk, d, 30, dtype=dtype), QKNormRope(d, 64)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    g = _draw((n * hq * d + 3,), 5, dt)
    leaves = lambda: [_draw((n, h, d), i, dt).requires_grad_() for i, h in enumerate((hq, hk, hk))]

    def grads(use):
        x = leaves()
        use(x).backward()
        return [t.grad for t in x[:2]]

    both = lambda x: norm(x[0], x[1], pos)
    kg = _draw((n, hk, d), 6, dt)
    for one, other in [
            (lambda x: (attn(*both(x), x[2]) * g[3:].view(n, hq, d)).sum(),
             lambda x: (torch.cat([x[0].flatten()[:3].detach(), attn(*both(x), x[2]).flatten()]) * g).sum()),
            (lambda x: (both(x)[0] * g[3:].view(n, hq, d)).sum() + (both(x)[1] * kg).sum(),
             lambda x: (torch.cat([x[0].flatten()[:3].detach(), both(x)[0].flatten()]) * g).sum() + (both(x)[1] * kg).sum()),
            (lambda x: (attn(*both(x), x[2]) * torch.ones((n, hq, d), dtype=dt, device="cuda")).sum(),
             lambda x: attn(*both(x), x[2]).sum())]:
        for a, b in zip(grads(one), grads(other)):
            assert torch.equal(a, b)
    attn.close()


# ------------------------------------------------------------------ strides

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_of_dimensions_of_one_element_are_not_looked_at(dtype):
    """A view of one token, or of one head, may carry any stride there: here odd ones."""
    from adapter_gemm_packed_gb300.attention import WindowAttention, qk_norm_rope, qk_norm_rope_backward
    d, dt = 64, DT[dtype]
    w = [1 + 0.1 * _draw((d,), 7 + i, torch.float32) for i in range(2)]
    ang = torch.rand((300, d // 2), generator=torch.Generator().manual_seed(1)) * 6.28
    for n, hq, hk in ((1, 4, 2), (1, 1, 1), (200, 1, 1), (1, 3, 1)):
        pos = torch.arange(n, dtype=torch.int32, device="cuda")
        tab = (*w, ang.cos().cuda(), ang.sin().cuda(), pos)
        q, k, v, do = (_draw((n, h, d), i, dt) for i, h in enumerate((hq, hk, hk, hq)))
        attn = WindowAttention([n], hq, hk, d, 50, n_sink=1, dtype=dtype)

        def all_of(q, k, v, do, *out):
            out = out or [None] * 4
            r = [*qk_norm_rope(q, k, *tab), *qk_norm_rope_backward(do, v, q, k, *tab)]
            o = attn.forward(q, k, v, out=out[0])
            return r + [o, *attn.backward(q, k, v, o, do, *out[1:])]

        odd = lambda t: t.as_strided(t.shape, [77 if n == 1 else t.stride(0), 33 if t.shape[1] == 1 else t.stride(1), 1])
        want = all_of(q, k, v, do)
        got = all_of(*map(odd, (q, k, v, do)), *(odd(torch.empty_like(t)) for t in (q, q, k, v)))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert attn.sync_status() == M.MLORA_OK
        attn.close()


# ------------------------------------------------------------------ pieces cut along their queries

CUT = {"causal": ([2600], 10**6, 0), "first_tokens": ([4200, 30], 200, 70), "wide": ([70, 3500, 1], 1500, 3)}


def _parts(attn):
    """The largest number of parts that a dK / dV piece of the plan is cut into."""
    t = M.mlora_attention_describe(attn.plan, M.MLORA_ATTN_Q_KEYS)
    return max(t[6::8])


@pytest.mark.parametrize("name", sorted(CUT))
@pytest.mark.parametrize("hq,hk,d", [(4, 1, 64), (4, 1, 128), (8, 2, 72)])
def test_cut_pieces(name, hq, hk, d):
    """dK and dV of long pieces are summed by several blocks: against 64 bits; the same bits in every backward on one
    buffer (the counters are back at zero), in a graph's replay, and with the sequences inside a larger pack.  Tolerance as
    for all bf16 attention: 2^-8 of the result and 2^-7 of the sum of absolute terms."""
    from adapter_gemm_packed_gb300.attention import WindowAttention
    lens, window, sinks = CUT[name]
    attn = WindowAttention(lens, hq, hk, d, window, n_sink=sinks)
    assert _parts(attn) > 1
    q, k, v, do = (_draw((attn.n, h, d), 50 + i, torch.bfloat16) for i, h in enumerate((hq, hk, hk, hq)))
    o = attn.forward(q, k, v)
    first = attn.backward(q, k, v, o, do)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(attn.backward(q, k, v, o, do), first))
    starts = [sum(lens[:i]) for i in range(len(lens))]
    ref = R.attention(q, k, v, lens, starts, window, sinks, attn.scale, do)
    for what, got in zip(("o", "dq", "dk", "dv"), (o, *first)):
        want, bound = ref[what]
        err = (got.double().cpu() - want).abs()
        assert (err <= 2.0 ** -8 * want.abs() + 2.0 ** -7 * bound + 1e-30).all(), what

    out = [torch.empty_like(t) for t in (o, *first)]
    step = lambda: (attn.forward(q, k, v, out=out[0]), attn.backward(q, k, v, out[0], do, *out[1:]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, (o, *first)))

    # behind other sequences, which are cut too, and before others
    others, after = [1000, 2900], [333]
    big = WindowAttention(others + lens + after, hq, hk, d, window, n_sink=sinks)
    pad = lambda t, s: torch.cat([_draw((sum(others), *t.shape[1:]), s, t.dtype), t, _draw((333, *t.shape[1:]), s + 1, t.dtype)])
    Q, K, V, G = (pad(t, 60 + 2 * i) for i, t in enumerate((q, k, v, do)))
    O = big.forward(Q, K, V)
    inside = slice(sum(others), sum(others) + attn.n)
    for a, b in zip((O, *big.backward(Q, K, V, O, G)), (o, *first)):
        assert torch.equal(a[inside], b)
    assert attn.sync_status() == M.MLORA_OK and big.sync_status() == M.MLORA_OK
    attn.close()
    big.close()


def test_autograd_with_cut_pieces_and_two_forwards():
    """Each graph has its own statistics and scratch: two forwards before the first backward, bf16."""
    from adapter_gemm_packed_gb300.attention import WindowAttention
    attn = WindowAttention([2600], 4, 1, 64, 10**6)
    assert _parts(attn) > 1
    x = [_draw((2600, h, 64), 70 + i, torch.bfloat16).requires_grad_() for i, h in enumerate((4, 1, 1))]
    y = [_draw((2600, h, 64), 80 + i, torch.bfloat16).requires_grad_() for i, h in enumerate((4, 1, 1))]
    do = _draw((2600, 4, 64), 90, torch.bfloat16)
    a, b = attn(*x), attn(*y)
    got = torch.autograd.grad(a, x, do) + torch.autograd.grad(b, y, 2 * do)
    want = ()
    for t, g in ((x, do), (y, 2 * do)):
        t = [u.detach() for u in t]
        o = attn.forward(*t)
        want += attn.backward(*t, o, g)
    assert all(torch.equal(u, w) for u, w in zip(got, want))
    attn.close()


def test_scratch_of_the_backward():
    """In a workspace of its own, whatever it holds, or behind what the forward left, in one buffer: the same bits.  Cut
    pieces without a workspace are refused."""
    from adapter_gemm_packed_gb300.attention import WindowAttention, _heads
    attn = WindowAttention([2600], 4, 1, 64, 10**6)
    assert attn.work_elems > 0
    q, k, v, do = (_draw((2600, h, 64), 50 + i, torch.bfloat16) for i, h in enumerate((4, 1, 1, 4)))
    o = attn.forward(q, k, v)
    want = attn.backward(q, k, v, o, do)
    both = torch.full((M.mlora_attention_saved_elems(attn.plan),), float("nan"), device="cuda")
    got = [torch.empty_like(t) for t in (q, k, v)]
    ins = [_heads(t, "", "", *s) for t, s in ((q, attn.qs), (k, attn.ks), (v, attn.ks), (o, attn.qs), (do, attn.qs))]
    outs = [_heads(t, "", "", *s) for t, s in zip(got, (attn.qs, attn.ks, attn.ks))]
    s = torch.cuda.current_stream().cuda_stream
    M.mlora_attention_forward(attn.plan, *ins[:4], both.data_ptr(), s)
    M.mlora_attention_backward(attn.plan, *ins, both.data_ptr(), *outs, s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    work = torch.full((attn.work_elems,), -1, dtype=torch.int32, device="cuda")
    for t in got:
        t.zero_()
    M.mlora_attention_backward_ws(attn.plan, *ins, both.data_ptr(), work.data_ptr(), *outs, s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for bad in (None, work.data_ptr() + 4):
        with pytest.raises(M.MloraError) as e:
            M.mlora_attention_backward_ws(attn.plan, *ins, both.data_ptr(), bad, *outs, s)
        assert e.value.status == M.MLORA_ERR_INVALID
    assert attn.sync_status() == M.MLORA_OK
    attn.close()
