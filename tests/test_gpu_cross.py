"""Cross attention parity (forward, backward, single tokens) against the float64
oracle on the same 16-bit values, element by element.

Tolerances.  u = 2^-8 (bfloat16) or 2^-11 (float16) bounds one rounding.
 O     = sum_j P~_j v_j / l with each P~ rounded once, then rounded itself:
         |dO| <= u (sum_j p_j |v_j|) + u |O|.
 dV    = sum_i P~_i dO_i, rounded:   u sum_i p_i |dO_i| + u |dV|.
 dS~   = rnd(P^ (dP - D~)), P^ to 2^-15:  p |dP - D| (u + 2^-14) + p |dD|, and D~ takes
         the rounded O:              |dD_i| <= sum_c |dO_ic| |dO-tolerance_ic|.
         Up to 16 keys: D = sum_j P_j dP_j in float32, as dP itself; d <= 128 terms each:
         |d(dP - D)| <= 2 (d + 2) 2^-24 |dO| |v| <= 2^-16 |dO| |v|.
 dQ    = scale sum_j dS~_j k_j, rounded:  scale sum_j |d dS_j| |k_j| + u |dQ|; dK likewise.
float16 probabilities and dS below 2^-14 are subnormal: each is off by at most
2^-25 more (the probabilities before the division by l >= 1).  A tenth on top
covers second-order terms and the float32 arithmetic (exponentials to 2^-21)."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from gpu_util import LSE_ABS, check_status, dev, guarded, lib

pytestmark = pytest.mark.gpu
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
SUB = {"bf16": 0.0, "fp16": 2.0 ** -25}


@pytest.fixture(scope="module")
def attn():
    return lib()


def _inputs(seed, B, H, H_kv, N_q, N_k, d, dtype):
    q, do = workloads.normal(seed, (B, H, N_q, d), 2)
    k, v = workloads.normal(seed + 1, (B, H_kv, N_k, d), 2)
    return tuple(workloads.round_to(x, dtype) for x in (q, k, v, do))


def _forward_bound(q, k, v, o, scale, lens, dtype):
    a, _ = oracle.attention_cross_forward(q, k, np.abs(v), scale, lens)
    return 1.1 * (U[dtype] * (a + np.abs(o)) + SUB[dtype] * k.shape[2] * np.abs(v).max()) + 1e-6


def _backward_bounds(q, k, v, do, o, o_tol, grads, scale, lens, dtype):
    u, sub = U[dtype], SUB[dtype]
    B, H = q.shape[:2]
    G = H // k.shape[1]
    tq, tk, tv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for b in range(B):
        n = k.shape[2] if lens is None else int(lens[b])
        if n == 0:
            continue
        for h in range(H):
            j = h // G
            p, _, _ = oracle.attention_probs(q[b, h], k[b, j, :n], scale)
            dp = do[b, h] @ v[b, j, :n].T
            gap = np.abs(dp - (do[b, h] * o[b, h]).sum(1, keepdims=True))
            if k.shape[2] <= 16:
                dD = 2.0 ** -16 * np.abs(do[b, h]) @ np.abs(v[b, j, :n]).T
            else:
                dD = (np.abs(do[b, h]) * o_tol[b, h]).sum(1, keepdims=True)
            eds = (u + 2.0 ** -14) * p * gap + p * dD + sub * (1 + gap)
            tq[b, h] = scale * eds @ np.abs(k[b, j, :n])
            tk[b, j, :n] += scale * eds.T @ np.abs(q[b, h])
            tv[b, j, :n] += (u * p + sub).T @ np.abs(do[b, h])
    return [1.1 * (t + u * np.abs(g)) + 1e-6 for t, g in zip((tq, tk, tv), grads)]


def _within(got, ref, tol, what):
    x = got.double().cpu().numpy()
    assert np.all(np.isfinite(x)), what
    over = np.abs(x - ref) - tol
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, (what, at, x[at], ref[at], tol[at])


def _lse_close(lse, ref):
    x = lse.double().cpu().numpy()
    seen = np.isfinite(ref)
    assert np.array_equal(np.isneginf(x), ~seen)
    assert np.abs(x[seen] - ref[seen]).max(initial=0.0) <= LSE_ABS


def _check(attn, B, H, H_kv, N_q, N_k, d, dtype="bf16", lens=None, seed=900, backward=True, dirty=True):
    q, k, v, do = _inputs(seed, B, H, H_kv, N_q, N_k, d, dtype)
    scale = 1 / np.sqrt(d)
    f = [workloads.as_f64(t) for t in (q, k, v, do)]
    o_ref, l_ref = oracle.attention_cross_forward(*f[:3], scale, lens)
    gq, gk, gv, gdo = (t.to(dev()) for t in (q, k, v, do))
    if lens is not None and dirty:
        # what stands behind the keys must not matter
        for b, n in enumerate(lens):
            gk[b, :, n:], gv[b, :, n:] = float("nan"), float("inf")
    tl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev())
    o, co = guarded((B, H, N_q, d), q.dtype, -7.0)
    lse, cl = guarded((B, H, N_q), torch.float32, -7.0)
    attn.attn_cross_fwd(gq, gk, gv, tl, softmax_scale=scale, o=o, lse=lse)
    check_status(attn)
    co()
    cl()
    tol = _forward_bound(*f[:3], o_ref, scale, lens, dtype)
    _within(o, o_ref, tol, "o")
    _lse_close(lse, l_ref)
    if not backward:
        return
    grads = oracle.attention_cross_backward(*f, scale, lens)
    outs = [guarded(t.shape, t.dtype, -7.0) for t in (q, k, v)]
    attn.attn_cross_bwd(gq, gk, gv, o, gdo, lse, tl, softmax_scale=scale, dq=outs[0][0], dk=outs[1][0], dv=outs[2][0])
    check_status(attn)
    tols = _backward_bounds(*f, o_ref, tol, grads, scale, lens, dtype)
    for (x, check), ref, t, what in zip(outs, grads, tols, ("dq", "dk", "dv")):
        check()
        _within(x, ref, t, what)
    if lens is not None:
        for b, n in enumerate(lens):
            assert not outs[1][0][b, :, n:].any() and not outs[2][0][b, :, n:].any()


@pytest.mark.parametrize("N_q,N_k", [(1, 1), (1, 129), (7, 128), (128, 1), (129, 127), (257, 300), (300, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths(attn, N_q, N_k, d):
    _check(attn, 1, 2, 2, N_q, N_k, d)


@pytest.mark.parametrize("N_k", [1, 2, 3, 8, 15, 16, 17])
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (128, "fp16")])
def test_few_keys(attn, N_k, d, dtype):
    """Where the rounding of O would weigh most in the gradients; one, some and no keys seen."""
    _check(attn, 2, 6, 2, 203, N_k, d, dtype, seed=905)
    _check(attn, 3, 4, 4, 70, N_k, d, dtype, lens=[N_k, 0, (N_k + 1) // 2], seed=906)


@pytest.mark.parametrize("H,H_kv", [(4, 1), (6, 3), (8, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_grouped_heads(attn, H, H_kv, dtype):
    _check(attn, 2, H, H_kv, 70, 200, 128, dtype, seed=910)
    _check(attn, 2, H, H_kv, 3, 333, 64, dtype, seed=911)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N_q", [1, 40, 300])
def test_key_lengths(attn, d, N_q):
    """Empty, one key, both sides of a tile's border, all: with NaN and infinities behind."""
    _check(attn, 8, 2, 1, N_q, 300, d, lens=[0, 1, 127, 128, 129, 256, 299, 300], seed=920)


@pytest.mark.parametrize("H_kv,N_k", [(4, 700), (7, 4096), (8, 1500), (10, 2500), (4, 500), (23, 1500),
                                      (30, 1500), (50, 800), (4, 8192)])
@pytest.mark.parametrize("N_q", [1, 40])
def test_segments_and_their_keys(attn, H_kv, N_k, N_q):
    """Few to many segments of few to many tiles: a cluster of each size per segment, and none."""
    _check(attn, 2, H_kv, H_kv, N_q, N_k, 64, lens=[N_k - 1, 130], seed=925, backward=False)
    _check(attn, 2, H_kv, H_kv, N_q, N_k, 64, "fp16", lens=[0, N_k], seed=926, backward=False)


def test_key_lengths_fp16_all_empty(attn):
    _check(attn, 2, 2, 2, 5, 130, 64, "fp16", lens=[0, 0], seed=930)
    _check(attn, 2, 2, 2, 200, 130, 128, "fp16", lens=[0, 77], seed=931)


@pytest.mark.parametrize("N_q", [1, 200])
def test_wide_head_forward(attn, N_q):
    _check(attn, 2, 4, 2, N_q, 333, 256, lens=[333, 100], backward=False, seed=940)


def test_split_key_ranges(attn):
    """One query over many keys: several ranges, some of them behind the keys."""
    _check(attn, 3, 4, 2, 1, 5000, 128, lens=[5000, 130, 0], backward=False, seed=950)
    _check(attn, 1, 8, 1, 16, 3333, 64, "fp16", backward=False, seed=951)


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_shares_over_several_query_tiles(attn, d, dtype):
    """A few hundred rows per key/value head over many keys: segments of several query
    tiles that begin and end inside shares, some batch entries without keys."""
    _check(attn, 3, 4, 2, 70, 2000, d, dtype, lens=[1999, 0, 700], backward=False, seed=952)
    _check(attn, 1, 2, 1, 130, 3000, d, dtype, backward=False, seed=953)


@pytest.mark.parametrize("H,H_kv,N_q,N_k,d", [(4, 1, 900, 40, 64), (4, 1, 600, 130, 128), (2, 2, 257, 513, 64)])
def test_backward_shares(attn, H, H_kv, N_q, N_k, d):
    """Few key tiles with many query tiles: a segment spread over many CTAs."""
    _check(attn, 2, H, H_kv, N_q, N_k, d, lens=[N_k, N_k // 3], seed=960)


def test_backward_many_entries_and_repeat(attn):
    """More batch entries than threads; dK and dV are the same bits every time."""
    B, lens = 700, [(b * 11) % 7 * 20 for b in range(700)]
    _check(attn, B, 2, 1, 3, 130, 64, lens=lens, seed=961)
    q, k, v, do = (t.to(dev()) for t in _inputs(962, 2, 6, 2, 700, 300, 128, "bf16"))
    o, lse = attn.attn_cross_fwd(q, k, v)
    first = attn.attn_cross_bwd(q, k, v, o, do, lse)
    for _ in range(3):
        again = attn.attn_cross_bwd(q, k, v, o, do, lse)
        assert torch.equal(first[1], again[1]) and torch.equal(first[2], again[2])
    check_status(attn)


def test_many_entries(attn):
    """More batch entries than threads, most of them short or empty; and more than the
    shared plan takes."""
    lens = [(7 * b) % 5 * 30 for b in range(600)]
    _check(attn, 600, 2, 1, 1, 400, 64, lens=lens, backward=False, seed=954)
    B = 2049
    q, k, v, _ = _inputs(955, B, 1, 1, 1, 3, 64, "bf16")
    o, lse = attn.attn_cross_fwd(q.to(dev()), k.to(dev()), v.to(dev()))
    check_status(attn)
    f = [workloads.as_f64(t) for t in (q, k, v)]
    ref, l = oracle.attention_cross_forward(*f, 64 ** -0.5)
    _within(o, ref, _forward_bound(*f, ref, 64 ** -0.5, None, "bf16"), "o")
    _lse_close(lse, l)


def test_large_scores(attn):
    """Scores that grow along the keys by far more than the lazy rescale's 2^8."""
    q, k, v, do = _inputs(960, 1, 2, 2, 130, 400, 64, "bf16")
    k = (k.float() * torch.linspace(0.1, 8, 400)[:, None]).to(torch.bfloat16)
    f = [workloads.as_f64(t) for t in (q, k, v)]
    ref, l = oracle.attention_cross_forward(*f, 0.5)
    for rows in (slice(0, 130), slice(0, 1)):
        o, lse = attn.attn_cross_fwd(q[:, :, rows].contiguous().to(dev()), k.to(dev()), v.to(dev()), softmax_scale=0.5)
        check_status(attn)
        _within(o, ref[:, :, rows], _forward_bound(*f, ref, 0.5, None, "bf16")[:, :, rows], "o")
        _lse_close(lse, l[:, :, rows])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gradient_by_differences(attn, dtype):
    """The kernel's gradients along random directions against central differences of
    sum(O dO) in float64 (step 1e-5: truncation below 1e-6 here); the sum of the
    elements' bounds bounds the error."""
    scale, lens = 0.2, [50]
    q, k, v, do = _inputs(970, 1, 2, 1, 40, 60, 64, dtype)
    f = [workloads.as_f64(t) for t in (q, k, v, do)]
    tl = torch.tensor(lens, dtype=torch.int32, device=dev())
    gq, gk, gv, gdo = (t.to(dev()) for t in (q, k, v, do))
    o, lse = attn.attn_cross_fwd(gq, gk, gv, tl, softmax_scale=scale)
    got = attn.attn_cross_bwd(gq, gk, gv, o, gdo, lse, tl, softmax_scale=scale)
    check_status(attn)
    o_ref, _ = oracle.attention_cross_forward(*f[:3], scale, lens)
    tols = _backward_bounds(*f, o_ref, _forward_bound(*f[:3], o_ref, scale, lens, dtype),
                            oracle.attention_cross_backward(*f, scale, lens), scale, lens, dtype)
    rng = np.random.default_rng(971)
    for i in range(3):
        way = np.where(rng.random(f[i].shape) < 0.5, -1.0, 1.0)
        ends = []
        for sign in (1e-5, -1e-5):
            moved = list(f)
            moved[i] = f[i] + sign * way
            ends.append((oracle.attention_cross_forward(*moved[:3], scale, lens)[0] * f[3]).sum())
        slope = (ends[0] - ends[1]) / 2e-5
        mine = (got[i].double().cpu().numpy() * way).sum()
        assert abs(mine - slope) <= tols[i].sum() + 1e-5, (i, mine, slope)


def test_bad_lengths_are_reported_and_count_as_empty(attn):
    q, k, v, do = (t.to(dev()) for t in _inputs(980, 3, 2, 2, 200, 150, 64, "bf16"))
    for rows in (1, 200):
        qq, dd = q[:, :, :rows].contiguous(), do[:, :, :rows].contiguous()
        lens = torch.tensor([-1, 151, 150], dtype=torch.int32, device=dev())
        o, lse = attn.attn_cross_fwd(qq, k, v, lens)
        assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
        assert not o[:2].any() and torch.isneginf(lse[:2]).all() and torch.isfinite(lse[2]).all()
        dq, dk, dv = attn.attn_cross_bwd(qq, k, v, o, dd, lse, lens)
        assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
        assert not dq[:2].any() and not dk[:2].any() and not dv[:2].any() and dk[2].any()
    assert attn.attn_get_device_status() == 0


@pytest.mark.parametrize("N_q", [1, 200])
def test_graph_replay_stream_and_repeat(attn, N_q):
    """Two captured graphs with their own workspaces, replayed on two streams with new
    inputs, give the eager call's bits."""
    B, H, H_kv, N_k, d = 2, 4, 2, 1500, 64
    runs = []
    for i in range(2):
        q, k, v, _ = (t.to(dev()) for t in _inputs(990 + 2 * i, B, H, H_kv, N_q, N_k, d, "bf16"))
        lens = torch.tensor([N_k - i, 700], dtype=torch.int32, device=dev())
        need = attn.attn_cross_workspace_size(B, H, H_kv, N_q, N_k, d)
        ws = torch.empty(need, dtype=torch.uint8, device=dev()) if need else None
        o, lse = torch.empty_like(q), torch.empty(B, H, N_q, device=dev())
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            attn.attn_cross_fwd(q, k, v, lens, o=o, lse=lse, workspace=ws)
        runs.append((graph, stream, q, k, v, lens, o, lse))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream, q, *_ in runs:
            with torch.cuda.stream(stream):
                q.mul_(-1)
                graph.replay()
    torch.cuda.synchronize()
    for _, _, q, k, v, lens, o, lse in runs:
        ref_o, ref_l = attn.attn_cross_fwd(q, k, v, lens)
        assert torch.equal(o, ref_o) and torch.equal(lse, ref_l)
    check_status(attn)


@pytest.mark.parametrize("how", ["one stream", "two streams", "captured"])
@pytest.mark.parametrize("B,H_kv,N_k", [(1, 16, 1500), (24, 8, 700), (2, 2, 20000)])
def test_inputs_written_by_the_kernel_before(attn, B, H_kv, N_k, how):
    """Few-rows calls (a cluster per segment, shared tiles) start before the stream's previous
    kernel has ended.  Inputs, the lengths too, written right before each call, its output read
    and they overwritten right behind it, in a graph also from another stream and after a memset:
    the bits of calls with pauses between."""
    sets, want = [], []
    for i in range(3):
        q, k, v, _ = (t.to(dev()) for t in _inputs(1010 + 2 * i, B, H_kv, H_kv, 1, N_k, 64, "bf16"))
        lens = torch.tensor([(N_k - 37 * (b + 5 * i)) % (N_k + 1) for b in range(B)], dtype=torch.int32, device=dev())
        sets.append((q, k, v, lens))
        torch.cuda.synchronize()
        want.append(attn.attn_cross_fwd(q, k, v, lens))
        torch.cuda.synchronize()
    check_status(attn)
    now = [torch.zeros_like(t) for t in sets[0]]
    outs = [torch.zeros_like(t).expand(9, *t.shape).contiguous() for t in want[0]]
    need = attn.attn_cross_workspace_size(B, H_kv, H_kv, 1, N_k, 64)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev())
    o, lse = (torch.empty_like(t) for t in want[0])

    def run(side=None):
        here = torch.cuda.current_stream()
        for i in range(9):
            for to, source in zip(now, sets[i % 3]):
                if side is None:
                    to.copy_(source) if i % 2 else torch.mul(source, 1, out=to)
                    continue
                side.wait_stream(here)               # the next input from the other stream
                with torch.cuda.stream(side):
                    torch.mul(source, 1, out=to)
            if side is not None:
                ws.zero_()
                here.wait_stream(side)               # the call has to wait for both
            attn.attn_cross_fwd(*now, o=o, lse=lse, workspace=ws)
            for to, source in zip(outs, (o, lse)):
                torch.mul(source, 1, out=to[i])

    side = torch.cuda.Stream()
    if how == "captured":
        stream = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            run(side)
        for _ in range(3):
            graph.replay()
    else:
        run(side if how == "two streams" else None)
    torch.cuda.synchronize()
    check_status(attn)
    for i in range(9):
        for got, ref in zip(outs, want[i % 3]):
            assert torch.equal(got[i], ref), i


@pytest.mark.parametrize("captured", [False, True])
def test_training_inputs_written_by_the_kernel_before(attn, captured):
    """The same for forward and backward calls of many rows: tables of other inputs in the same
    memory, one set after the other."""
    B, H, H_kv, N_q, N_k, d = 2, 4, 2, 300, 400, 64
    sets, want = [], []
    for i in range(3):
        q, k, v, do = (t.to(dev()) for t in _inputs(1020 + 2 * i, B, H, H_kv, N_q, N_k, d, "bf16"))
        sets.append((q, k, v, torch.tensor([N_k - i, 130 * i], dtype=torch.int32, device=dev()), do))
        torch.cuda.synchronize()
        o, lse = attn.attn_cross_fwd(*sets[-1][:4])
        torch.cuda.synchronize()
        want.append((o, lse, *attn.attn_cross_bwd(q, k, v, o, do, lse, sets[-1][3])))
        torch.cuda.synchronize()
    q, k, v, lens, do = now = [torch.zeros_like(t) for t in sets[0]]
    outs = [t.expand(6, *t.shape).contiguous() for t in want[0]]
    o, lse, *grads = [torch.empty_like(t) for t in want[0]]

    def run():
        for i in range(6):
            for to, source in zip(now, sets[i % 3]):
                torch.mul(source, 1, out=to)
            attn.attn_cross_fwd(q, k, v, lens, o=o, lse=lse)
            attn.attn_cross_bwd(q, k, v, o, do, lse, lens, dq=grads[0], dk=grads[1], dv=grads[2])
            for to, source in zip(outs, (o, lse, *grads)):
                torch.mul(source, 1, out=to[i])

    if captured:
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            run()
        for _ in range(3):
            graph.replay()
    else:
        run()
    torch.cuda.synchronize()
    check_status(attn)
    for i in range(6):
        for got, ref, exact in zip(outs, want[i % 3], (True, True, False, True, True)):
            if exact:
                assert torch.equal(got[i], ref), i
            else:      # dQ: float32 sums in another order, then the same rounding
                assert torch.all((got[i].float() - ref.float()).abs() <= 2.0 ** -7 * ref.float().abs() + 1e-5), i


def test_host_tensors(attn):
    q, k, v, do = _inputs(995, 1, 2, 1, 20, 30, 64, "bf16")
    lens = torch.tensor([25], dtype=torch.int32)
    o, lse = attn.attn_cross_fwd(q, k, v, lens)
    dq, dk, dv = attn.attn_cross_bwd(q, k, v, o, do, lse, lens)
    assert all(t.device.type == "cpu" for t in (o, lse, dq, dk, dv))
    f = [workloads.as_f64(t) for t in (q, k, v)]
    ref, _ = oracle.attention_cross_forward(*f, 64 ** -0.5, [25])
    _within(o, ref, _forward_bound(*f, ref, 64 ** -0.5, [25], "bf16"), "o")
    with pytest.raises(ValueError, match="current CUDA device"):
        attn.attn_cross_fwd(q.to(dev()), k, v.to(dev()))
    with pytest.raises(ValueError, match="o must be"):
        attn.attn_cross_fwd(q.to(dev()), k.to(dev()), v.to(dev()), o=torch.empty(1, 2, 20, 32, device=dev()).bfloat16())


def test_self_attention_is_the_same_arithmetic(attn):
    """N_q = N_k without lengths, in a shape that the forward kernel takes: the plain forward's bits."""
    q, k, v, do = (t.to(dev()) for t in _inputs(997, 2, 16, 16, 700, 700, 128, "bf16"))
    o, lse = attn.attn_cross_fwd(q, k, v)
    ref = attn.attn_fwd(q, k, v)
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    grads = attn.attn_cross_bwd(q, k, v, o, do, lse)
    plain = attn.attn_bwd(q, k, v, o, do, lse)
    check_status(attn)
    # dV: float32 sums in another order, then one rounding to bfloat16 of each.  dQ, dK: attn_bwd
    # forms dS from P rounded to bfloat16, this one from P in 24 bits, both round dS: the two lie
    # at most (the bound of the one) + (that and u p |dP - D| more, below twice it) apart.
    assert torch.all((grads[2].float() - plain[2].float()).abs() <= 2.0 ** -7 * plain[2].float().abs() + 1e-5)
    one = [t[:1, :2].contiguous() for t in (q, k, v, do)]
    f = [workloads.as_f64(t.cpu()) for t in one]
    scale = 128 ** -0.5
    o_ref, _ = oracle.attention_cross_forward(*f[:3], scale)
    ref = oracle.attention_cross_backward(*f, scale)
    tols = _backward_bounds(*f, o_ref, _forward_bound(*f[:3], o_ref, scale, None, "bf16"), ref, scale, None, "bf16")
    for x, y, t in zip(grads[:2], plain[:2], tols):
        gap = (x[:1, :2].double() - y[:1, :2].double()).abs().cpu().numpy()
        assert np.all(gap <= 3 * t)


def test_explicit_stream(attn):
    """Calls on a stream that is not the current one, their scratch and outputs freed at once
    while the current stream allocates and writes: nothing of theirs is handed out early."""
    B, H, N_q, N_k, d = 2, 8, 96, 2000, 128
    q, k, v, do = (t.to(dev()) for t in _inputs(998, B, H, H, N_q, N_k, d, "bf16"))
    want = attn.attn_cross_fwd(q, k, v)
    grads = attn.attn_cross_bwd(q, k, v, want[0], do, want[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        o, lse = attn.attn_cross_fwd(q, k, v, stream=side)
        dq, dk, dv = attn.attn_cross_bwd(q, k, v, o, do, lse, stream=side)
        del dq
        for n in (q.numel() * 2, 1 << 20, attn.attn_cross_bwd_workspace_size(B, H, N_q, N_k, d)):
            torch.empty(n, dtype=torch.uint8, device=dev()).fill_(255)
        side.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(dk, grads[1]) and torch.equal(dv, grads[2])
    o, lse = attn.attn_cross_fwd(q.cpu(), k.cpu(), v.cpu(), stream=side)
    assert torch.equal(o, want[0].cpu())
    check_status(attn)


@pytest.mark.parametrize("H,H_kv,N_q", [(2, 2, 1), (16, 1, 1), (2, 2, 40), (2, 2, 300)])
@pytest.mark.parametrize("N_k,lens", [(300, None), (300, [300, 190]), (5000, [5000, 4900])])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (64, "fp16")])
def test_infinite_values_of_seen_keys(attn, H, H_kv, N_q, N_k, lens, d, dtype):
    """Columns with an infinity in some key's value are infinite, with both signs or a NaN they are
    NaN, the others as ever; whichever rows and keys share a tile."""
    q, k, v, _ = _inputs(1030, 2, H, H_kv, N_q, N_k, d, dtype)
    q = q * 0.5                                       # probabilities far from 0 in float16
    inf = float("inf")
    for j, c, x in ((0, 1, inf), (37, 2, -inf), (64, 3, inf), (127, 4, inf), (129, 5, -inf), (180, 6, inf),
                    (5, 7, inf), (100, 7, inf), (5, 8, inf), (70, 8, -inf), (33, 9, float("nan"))):
        v[:, :, j, c] = x
    tl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev())
    o, lse = attn.attn_cross_fwd(q.to(dev()), k.to(dev()), v.to(dev()), tl)
    check_status(attn)
    f = [workloads.as_f64(t) for t in (q, k, v)]
    with np.errstate(invalid="ignore"):
        ref, rl = oracle.attention_cross_forward(*f, d ** -0.5, lens)
    got = o.double().cpu().numpy()
    special = ~np.isfinite(ref)
    assert special[..., 1:10].all() and special.sum() == special[..., 1:10].sum()
    assert np.array_equal(got[..., 1:10], ref[..., 1:10], equal_nan=True)
    rest = np.r_[0, 10:d]
    f[2] = np.where(np.isfinite(f[2]), f[2], 0.0)
    ref, _ = oracle.attention_cross_forward(*f, d ** -0.5, lens)
    tol = _forward_bound(*f, ref, d ** -0.5, lens, dtype)
    assert np.all(np.abs(got - ref)[..., rest] <= tol[..., rest])
    _lse_close(lse, rl)


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "fp16"), (64, "bf16"), (128, "bf16")])
@pytest.mark.parametrize("N_k", [17, 300])
def test_few_seen_keys_of_a_padded_batch(attn, N_k, d, dtype):
    """Batch entries that see 1 to 17 keys beside one that sees all: the bounds of their own
    lengths, as if the batch were not padded."""
    B, H, H_kv, N_q, lens = 7, 6, 2, 203, [1, 2, 8, 16, 17, 0, N_k]
    q, k, v, do = _inputs(1040, B, H, H_kv, N_q, N_k, d, dtype)
    scale = d ** -0.5
    g = [t.to(dev()) for t in (q, k, v, do)]
    for b, n in enumerate(lens):
        g[1][b, :, n:], g[2][b, :, n:] = float("nan"), float("inf")
    tl = torch.tensor(lens, dtype=torch.int32, device=dev())
    o, lse = attn.attn_cross_fwd(*g[:3], tl)
    got = attn.attn_cross_bwd(*g[:3], o, g[3], lse, tl)
    check_status(attn)
    assert not any(x[5].any() for x in got)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        f = [workloads.as_f64(t[b:b + 1, :, :n] if t.shape[2] == N_k else t[b:b + 1]) for t in (q, k, v, do)]
        ref, _ = oracle.attention_cross_forward(*f[:3], scale)
        tol = _forward_bound(*f[:3], ref, scale, None, dtype)
        grads = oracle.attention_cross_backward(*f, scale)
        tols = _backward_bounds(*f, ref, tol, grads, scale, None, dtype)
        for x, r, t, what in zip(got, grads, tols, ("dq", "dk", "dv")):
            _within(x[b:b + 1, :, :r.shape[2]], r, t, (what, n))
