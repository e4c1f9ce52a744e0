"""Rotary tables and rotations against the float64 oracle.

Tolerances.  A table entry: the reduced angle in [-pi, pi] is rounded to float32
(2^-23 at most in absolute terms), sine and cosine are float32 functions (a few
2^-24), the product with attn_factor rounds once more, and the float64 angle is off
by 2^-52 of itself: attn_factor (2^-21 + p 2^-50).
A rotated value: two float32 products and a sum, 2^-22 (|x c| + |y s|), then one
rounding to 16 bits, u |result| (bfloat16 2^-8, float16 2^-11; subnormal float16
2^-25)."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from gpu_util import check_status, dev, guarded, lib

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def attn():
    return lib()


def _tables(n, rot):
    c, s = oracle.rope_table(n, rot)
    return torch.from_numpy(c).float().to(dev()), torch.from_numpy(s).float().to(dev())


def _check(got, x, at, cos, sin, interleaved, inverse):
    """got, x [..., tokens, d]-like with table rows cos[at] broadcast."""
    f = x.double().cpu().numpy()
    c, s = cos.double().cpu().numpy()[at], sin.double().cpu().numpy()[at]
    ref = oracle.rope_rotate(f, c, s, interleaved, inverse)
    mag = oracle.rope_rotate(np.abs(f), np.abs(c), -np.abs(s), interleaved) + oracle.rope_rotate(
        np.abs(f), np.abs(c), np.abs(s), interleaved)
    tol = U[x.dtype] * np.abs(ref) + 2.0 ** -22 * np.abs(mag) + 2.0 ** -25
    g = got.double().cpu().numpy()
    assert np.all(np.abs(g - ref) <= tol), np.abs(g - ref).max()
    rot = 2 * cos.shape[1]
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("n,rot,first", [(1, 16, 0), (257, 128, 0), (300, 96, 1000000), (5, 256, 2 ** 31 - 5), (9000, 64, 7)])
@pytest.mark.parametrize("kw", [dict(), dict(factor=8.0), dict(factor=4.0, orig_len=4096, low=1.0, high=32.0, attn_factor=1.3,
                                                               base=500000.0)])
def test_tables(attn, n, rot, first, kw):
    cos, cc = guarded((n, rot // 2), torch.float32, -7.0)
    sin, cs = guarded((n, rot // 2), torch.float32, -7.0)
    attn.attn_rope_table(n, rot, first=first, rope_cos=cos, rope_sin=sin, **kw)
    check_status(attn)
    cc()
    cs()
    rc, rs = oracle.rope_table(n, rot, first=first, **kw)
    tol = kw.get("attn_factor", 1.0) * (2.0 ** -21 + (first + n) * 2.0 ** -50)
    assert np.abs(cos.double().cpu().numpy() - rc).max() <= tol
    assert np.abs(sin.double().cpu().numpy() - rs).max() <= tol


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 256), (256, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_dense(attn, d, rot, interleaved, inverse):
    B, H, H_kv, N = 2, 5, 2, 37
    for dtype in (torch.bfloat16, torch.float16):
        q = torch.from_numpy(workloads.normal(d + rot, (B, H, N, d))).to(dev(), dtype)
        k = torch.from_numpy(workloads.normal(d + rot + 1, (B, H_kv, N, d))).to(dev(), dtype)
        cos, sin = _tables(N + 3, rot)
        qo, c1 = guarded(q.shape, dtype, -7.0)
        ko, c2 = guarded(k.shape, dtype, -7.0)
        attn.attn_rope(q, k, cos, sin, interleaved=interleaved, inverse=inverse, q_out=qo, k_out=ko)
        check_status(attn)
        c1()
        c2()
        _check(qo, q, np.arange(N), cos, sin, interleaved, inverse)
        _check(ko, k, np.arange(N), cos, sin, interleaved, inverse)
        # in place
        q2 = q.clone()
        attn.attn_rope(q2, None, cos, sin, interleaved=interleaved, inverse=inverse, q_out=q2)
        assert torch.equal(q2, qo)


@pytest.mark.parametrize("N", [1, 3, 130, 5000])
@pytest.mark.parametrize("interleaved", [False, True])
def test_packed_views_and_positions(attn, N, interleaved):
    """Rows of a fused projection, repeated and padded positions; in place the rest of
    the rows stays as it was."""
    H, H_kv, d, rot = 6, 3, 128, 96
    rows = torch.from_numpy(workloads.normal(N, (N, H + 2 * H_kv, d))).to(dev(), torch.bfloat16)
    before = rows.clone()
    cos, sin = _tables(64, rot)
    at = (np.arange(N) * 5) % 64
    pos = torch.from_numpy(at.astype(np.int32)).to(dev())
    pos[N // 2] = -1
    q, k = rows[:, :H], rows[:, H:H + H_kv]
    qo, ko = attn.attn_rope(q, k, cos, sin, positions=pos, interleaved=interleaved)
    check_status(attn)
    keep = np.arange(N) != N // 2
    for o, x in ((qo, q), (ko, k)):
        _check(o[keep], x[keep], at[keep][:, None], cos, sin, interleaved, False)
        assert torch.equal(o[~keep], x[~keep])
    attn.attn_rope(q, k, cos, sin, positions=pos, interleaved=interleaved, q_out=q, k_out=k)
    check_status(attn)
    assert torch.equal(rows[:, :H], qo) and torch.equal(rows[:, H:H + H_kv], ko)
    assert torch.equal(rows[:, H + H_kv:], before[:, H + H_kv:])


def test_positions_of_a_batch_and_broadcast_input(attn):
    B, H, N, d = 3, 2, 20, 64
    cos, sin = _tables(100, d)
    one = torch.from_numpy(workloads.normal(5, (1, H, N, d))).to(dev(), torch.float16)
    q = one.expand(B, H, N, d)                       # stride 0 over the batch
    pos = torch.randint(0, 100, (B, N), dtype=torch.int32, device=dev())
    qo, none = attn.attn_rope(q, None, cos, sin, positions=pos)
    check_status(attn)
    assert none is None
    _check(qo, q, pos.cpu().numpy()[:, None], cos, sin, False, False)
    with pytest.raises(attn.AttnError, match="strides"):
        attn.attn_rope(q, None, cos, sin, positions=pos, q_out=q)
    with pytest.raises(attn.AttnError, match="aligned"):
        attn.attn_rope(torch.zeros(N * d + 4, device=dev()).half()[4:].view(1, 1, N, d), None, cos, sin)


def test_positions_past_the_tables_are_copied_and_reported(attn):
    q = torch.from_numpy(workloads.normal(6, (4, 3, 64))).to(dev(), torch.bfloat16)
    cos, sin = _tables(8, 64)
    pos = torch.tensor([0, 8, 7, 2 ** 31 - 1], dtype=torch.int32, device=dev())
    out, _ = attn.attn_rope(q, None, cos, sin, positions=pos)
    assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
    assert torch.equal(out[[1, 3]], q[[1, 3]])
    _check(out[[0, 2]], q[[0, 2]], np.array([0, 7])[:, None], cos, sin, False, False)
    assert attn.attn_get_device_status() == 0


def test_gradient_by_differences(attn):
    """<R x, y> is linear in x: its slope along w, from the kernel's own outputs, is
    <w, inverse y>.  Values are multiples of 1/8 below 8, so x + w is exact."""
    N, H, d, rot = 50, 2, 64, 32
    cos, sin = _tables(N, rot)
    g = torch.Generator().manual_seed(3)
    x, w, y = ((torch.rand(N, H, d, generator=g) * 64 - 32).round().div(8).to(dev(), torch.float16) for _ in range(3))
    fwd = lambda t: attn.attn_rope(t, None, cos, sin)[0].double()
    slope = ((fwd((x + w)) - fwd(x)) * y.double()).sum()
    back = attn.attn_rope(y, None, cos, sin, inverse=True)[0].double()
    check_status(attn)
    mine = (w.double() * back).sum()
    # roundings of R(x + w), R x and R' y: 2^-11 of at most 12, 6 and 6 (|pair| <= sqrt 2 |value|)
    bound = 2.0 ** -11 * 1.1 * ((12 + 6) * y.double().abs().sum() + 6 * w.double().abs().sum())
    assert abs((slope - mine).item()) <= bound.item()


def test_host_tensors_and_graph(attn):
    q, k = (torch.from_numpy(workloads.normal(7 + i, (1, 2, 9, 64))).to(torch.bfloat16) for i in range(2))
    cos, sin = _tables(9, 64)
    qo, ko = attn.attn_rope(q, k, cos.cpu(), sin.cpu())
    assert qo.device.type == "cpu" and ko.device.type == "cpu"
    gq, gk = q.to(dev()), k.to(dev())
    oq, ok = torch.empty_like(gq), torch.empty_like(gk)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.attn_rope(gq, gk, cos, sin, q_out=oq, k_out=ok)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(oq.cpu(), qo) and torch.equal(ok.cpu(), ko)
    check_status(attn)


def test_explicit_stream(attn):
    q = torch.from_numpy(workloads.normal(8, (700, 32, 128))).to(dev(), torch.bfloat16)
    side = torch.cuda.Stream()
    cos, sin = attn.attn_rope_table(700, 128, stream=side)
    side.synchronize()
    want, _ = attn.attn_rope(q, None, cos, sin)
    torch.cuda.synchronize()
    for _ in range(10):
        c, s = attn.attn_rope_table(700, 128, stream=side)
        got, _ = attn.attn_rope(q, None, c, s, stream=side)
        del c, s
        torch.empty(700 * 64, device=dev()).fill_(9.0)
        side.synchronize()
        assert torch.equal(got, want)
    check_status(attn)


@pytest.mark.parametrize("captured", [False, True])
def test_rows_and_tables_written_by_the_kernel_before(attn, captured):
    """The kernels start before the stream's previous one has ended: tables, positions and rows
    of other contents in the same memory right before each call, in place and not, give the
    bits of calls with pauses between."""
    B, H, N, d = 2, 6, 700, 128
    sets, want = [], []
    for i in range(3):
        q, k = (torch.from_numpy(workloads.normal(60 + 2 * i + j, (B, H, N, d))).to(dev(), torch.bfloat16) for j in range(2))
        pos = torch.randint(0, 900, (B, N), dtype=torch.int32, device=dev(), generator=torch.Generator(dev()).manual_seed(i))
        cos, sin = attn.attn_rope_table(900, d, base=10000.0 + i, first=7 * i)
        torch.cuda.synchronize()
        sets.append((q, k, pos))
        want.append((*attn.attn_rope(q, k, cos, sin, pos), cos, sin))
        torch.cuda.synchronize()
    q, k, pos = now = [torch.zeros_like(t) for t in sets[0]]
    cos, sin = (torch.zeros(900, d // 2, device=dev()) for _ in range(2))
    outs = [t.expand(6, *t.shape).contiguous() for t in want[0]]

    def run():
        for i in range(6):
            for to, source in zip(now, sets[i % 3]):
                torch.mul(source, 1, out=to)
            attn.attn_rope_table(900, d, base=10000.0 + i % 3, first=7 * (i % 3), rope_cos=cos, rope_sin=sin)
            attn.attn_rope(q, k, cos, sin, pos, q_out=q, k_out=k)
            for to, source in zip(outs, (q, k, cos, sin)):
                torch.mul(source, 1, out=to[i])
            attn.attn_rope(q, k, cos, sin, pos, q_out=q, k_out=k, inverse=True)

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
        for got, ref in zip(outs, want[i % 3]):
            assert torch.equal(got[i], ref), i


def test_outputs_larger_than_the_device(attn):
    """PyTorch's own error, which its users catch, as from the other calls' allocations."""
    with pytest.raises(torch.OutOfMemoryError):
        attn.attn_rope_table(2 ** 31 - 1, 256)
    check_status(attn)
