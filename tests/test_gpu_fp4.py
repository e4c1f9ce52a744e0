"""The 4-bit paged cache (append, decode, read back), reading the other caches back, and joining
partial attentions, against the float64 oracle.

Tolerances.  Codes, descales and everything that is only moved or rounded once: exact (the
oracle's key rows repeat the float32 steps).  Rows read back through the transform: eight
float32 steps (2^-20 of the row's length) and the rounding (half a step: bf16 2^-8, fp16
2^-11 of the value, and half the smallest fp16, 2^-25).

Decode.  With A_i = scale sum_j |q_i||k_j| over the components of the largest score: a score is
off by at most e = 2^-16 max_j A_ij (128 float32 sums of exact products, the transform's steps
and the last e4m3 term of q, each below 2^-18 of the products' sizes; the exponent's
sums add 2^-22 of a score of at most A).  LSE: e + 2^-20 (1 + |LSE|) (ex2, lg2 and sums).
O: with V_i = sum_j P_ij |v_j|, probabilities off by 2 e and held to w, float32 sums and factors
(2^-16), then the output's rounding u: (w + 2 e + 2^-16) V + u |O| + 2^-24.  fp16: u = w = 2^-11
(a float16, which three e4m3 terms of four bits and a sign hold exactly).  bf16: u = 2^-8, and two
terms leave 2^-9 of the float16: w = 2^-9 + 2^-11.  P_ij s_j (s_j the value descale) is
2^5 at a reference no larger than the largest of them and its last term's step is 2^-9 2^-5 (bf16) or 2^-9 2^-10
(fp16), so where it is small it is off by half of that over 2^5, 2^-20 or 2^-25 of the largest, whatever
its own size: that times max_j(P_ij s_j) sum_j |code_j| more."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from gpu_util import check_status, dev, guarded, lib

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
PROB = {torch.bfloat16: 2.0 ** -9 + 2.0 ** -11, torch.float16: 2.0 ** -11}
LAST = {torch.bfloat16: 2.0 ** -20, torch.float16: 2.0 ** -25}


@pytest.fixture(scope="module")
def attn():
    return lib()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev())


def _np(t):
    return t.double().cpu().numpy()


def _table(rng, lens, page, spare=3):
    """Shuffled pages for sequences of these lengths; unused entries point nowhere."""
    need = [-(-int(n) // page) for n in lens]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(1, max(need))), -5)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, len(order)


class Cache:
    """A 4-bit cache of random rows; unowned slots hold any codes and NaN descales."""

    def __init__(self, seed, lens, page, H_kv, d):
        rng = np.random.default_rng(seed)
        self.lens, self.page, self.H_kv, self.d = np.asarray(lens), page, H_kv, d
        self.table, num = _table(rng, lens, page)
        shape = (num, H_kv, page)
        self.codes = [rng.integers(0, 256, (*shape, d // 2)).astype(np.uint8) for _ in range(2)]
        owned = np.zeros((num, page), bool)
        for b, n in enumerate(lens):
            for t in range(int(n)):
                owned[self.table[b, t // page], t % page] = True
        self.owned = owned[:, None] & np.ones(shape, bool)
        self.descale = []
        for _ in range(2):
            s = torch.from_numpy(rng.uniform(0.05, 0.4, shape)).bfloat16().float().numpy()
            self.descale.append(np.where(self.owned, s, np.nan).astype(np.float32))

    def values(self):
        return [np.nan_to_num(oracle.dequantize_cache_fp4(c, s)) for c, s in zip(self.codes, self.descale)]

    def args(self):
        """k_cache, v_cache, k_descale, v_descale, block_table, seq_lens on the GPU."""
        return (*(torch.from_numpy(c).to(dev()) for c in self.codes),
                *(torch.from_numpy(s).bfloat16().to(dev()) for s in self.descale), _i32(self.table), _i32(self.lens))


def _signs(d, seed=7):
    return torch.from_numpy(np.where(np.random.default_rng(seed).random(d) < 0.5, -1.0, 1.0)).float().to(dev())


# -------------------------------------------------------------------- append ----
def _append_case(attn, seed, total, H, H_kv, d, page, dtype, rot=None, interleaved=False, signs=False, slots=None,
                 scale=None):
    rng = np.random.default_rng(seed)
    num = -(-total // page) + 3
    if slots is None:
        slots = rng.permutation(num * page)[:total]
        slots[total // 2:total // 2 + 1] = -1
    rows = torch.from_numpy(rng.standard_normal((total, H + 2 * H_kv, d)).astype(np.float32)).to(dev(), dtype)
    if scale is not None:
        rows = (rows.float() * scale).to(dtype)
    q, k, v = rows[:, :H], rows[:, H:H + H_kv], rows[:, H + H_kv:]
    pos = rng.integers(0, 60, total)
    state = []
    for _ in range(2):
        c, check_c = guarded((num, H_kv, page, d // 2), torch.uint8, 0x5A)
        s, check_s = guarded((num, H_kv, page), torch.bfloat16, -7.0)
        c.copy_(torch.from_numpy(rng.integers(0, 256, c.shape).astype(np.uint8)))
        state.append((c, s, c.cpu().numpy(), s.float().cpu().numpy(), check_c, check_s))
    kw = {}
    cos = sin = None
    if rot:
        cos, sin = (torch.from_numpy(x).float().to(dev()) for x in oracle.rope_table(60, rot))
        kw = dict(rope_cos=cos, rope_sin=sin, positions=_i32(pos), q=q, interleaved=interleaved)
    sg = _signs(d) if signs else None
    (kc, kd, *_), (vc, vd, *_) = state
    qo = attn.attn_cache_append_fp4(k, v, kc, vc, kd, vd, torch.from_numpy(slots).to(dev()), hadamard_signs=sg, **kw)
    check_status(attn)
    host = lambda x: None if x is None else x.cpu().numpy()
    kf = oracle.key_rows_f32(k.float().cpu().numpy(), pos, host(cos), host(sin), interleaved, host(sg))
    for (c, s, c0, s0, *checks), x in zip(state, (kf, v.float().cpu().numpy())):
        want_c, want_s = oracle.append_fp4(x, c0, s0, slots)
        assert np.array_equal(s.float().cpu().numpy(), want_s, equal_nan=True)
        assert np.array_equal(oracle.e2m1_decode(c.cpu().numpy()), oracle.e2m1_decode(want_c))
        for check in checks:
            check()
    if rot:
        want, _ = attn.attn_rope(q.contiguous(), None, cos, sin, positions=_i32(pos), interleaved=interleaved)
        assert torch.equal(qo, want)
    else:
        assert qo is None


@pytest.mark.parametrize("d,rot,interleaved", [(64, 64, False), (64, 16, False), (64, 48, True), (128, 128, False),
                                               (128, 48, False), (128, 112, False), (128, 128, True), (128, None, False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("signs", [False, True])
def test_append(attn, d, rot, interleaved, dtype, signs):
    _append_case(attn, 1, 37, 4, 2, d, 16, dtype, rot, interleaved, signs)


@pytest.mark.parametrize("total,H,H_kv,page", [(1, 8, 1, 16), (3, 6, 3, 64), (2, 32, 8, 256), (700, 4, 4, 32)])
def test_append_shapes(attn, total, H, H_kv, page):
    _append_case(attn, 2, total, H, H_kv, 128, page, torch.bfloat16, 64, False, True)


@pytest.mark.parametrize("d,rot,interleaved,signs", [(64, 32, False, True), (128, 128, False, True), (128, 128, True, False)])
def test_append_of_many_rows_is_that_of_few(attn, d, rot, interleaved, signs):
    """A block of a long append walks over several heads, one of a short append over a single one: the same bits."""
    total, H, H_kv, page, pages = 12000, 4, 5, 64, 200
    k, v = (torch.randn(total, H_kv, d, device=dev()).bfloat16() for _ in range(2))
    q = torch.randn(total, H, d, device=dev()).bfloat16()
    slots = torch.randperm(pages * page, device=dev())[:total]
    slots[5::97] = -1
    pos = torch.randint(0, 500, (total,), device=dev(), dtype=torch.int32)
    cos, sin = attn.attn_rope_table(500, rot)
    kw = dict(hadamard_signs=_signs(d) if signs else None, interleaved=interleaved)
    got = []
    for step in (total, 100):
        cache = [torch.full((pages, H_kv, page, d // 2), 0x55, dtype=torch.uint8, device=dev()) for _ in range(2)]
        des = [torch.ones(pages, H_kv, page, device=dev()).bfloat16() for _ in range(2)]
        qs = []
        for a in range(0, total, step):
            at = slice(a, a + step)
            qs.append(attn.attn_cache_append_fp4(k[at], v[at], *cache, *des, slots[at], cos, sin, pos[at], q=q[at], **kw))
        got.append((*cache, *des, torch.cat(qs)))
    check_status(attn)
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("d,rot", [(64, None), (64, 48), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_transforms_large_keys(attn, d, rot, interleaved):
    """Keys of up to 2^126: the transform's sums stay in range.  The codes of rows a power of two smaller, and
    that power in the descales."""
    k = torch.from_numpy(workloads.normal(43, (20, 2, d))).to(dev(), torch.bfloat16)
    kw = {}
    if rot:
        cos, sin = attn.attn_rope_table(32, rot)
        kw = dict(rope_cos=cos, rope_sin=sin, positions=torch.arange(20, device=dev(), dtype=torch.int32), interleaved=interleaved)
    got = []
    for x in (k, k * 2.0 ** 124):
        c = [torch.zeros(2, 2, 16, d // 2, dtype=torch.uint8, device=dev()) for _ in range(2)]
        s = [torch.zeros(2, 2, 16, device=dev()).bfloat16() for _ in range(2)]
        attn.attn_cache_append_fp4(x, x, *c, *s, torch.arange(20, device=dev()), hadamard_signs=_signs(d), **kw)
        got.append((c, s))
    check_status(attn)
    (c0, s0), (c1, s1) = got
    assert torch.any(s0[0] != 0) and all(torch.equal(a, b) for a, b in zip(c0, c1))
    assert all(torch.equal(a * 2.0 ** 124, b) for a, b in zip(s0, s1))


def test_append_of_rows_that_have_no_scale(attn):
    """Zeros, the smallest and the largest values, infinities and NaN: each row by itself."""
    d, H_kv, page = 128, 2, 16
    x = torch.randn(8, H_kv, d, device=dev())
    x[0] = 0
    x[1, 0, 5:] = 0
    x[2] *= 1e-38
    x[3] *= 1e36
    x[4, 1, 77] = float("inf")
    x[5, 0, 3] = float("nan")
    x[6] = 2.0 ** -133          # a bfloat16 subnormal
    x = x.bfloat16()
    kc, vc = (torch.full((1, H_kv, page, d // 2), 0x33, dtype=torch.uint8, device=dev()) for _ in range(2))
    kd, vd = (torch.ones(1, H_kv, page, device=dev()).bfloat16() for _ in range(2))
    slots = torch.arange(8, device=dev())
    attn.attn_cache_append_fp4(x, x, kc, vc, kd, vd, slots)
    check_status(attn)
    want_c, want_s = oracle.append_fp4(x.float().cpu().numpy(), np.full(kc.shape, 0x33, np.uint8), np.ones(kd.shape), np.arange(8))
    for c, s in ((kc, kd), (vc, vd)):
        assert np.array_equal(s.float().cpu().numpy(), want_s, equal_nan=True)
        assert np.array_equal(oracle.e2m1_decode(c.cpu().numpy()), oracle.e2m1_decode(want_c))
    k, v = attn.attn_cache_read_fp4(kc, vc, kd, vd, _i32([[0]]), _i32([8]), 8)
    bad = torch.zeros(H_kv, 8, dtype=torch.bool)
    bad[1, 4] = bad[0, 5] = True
    assert torch.equal(torch.isnan(k[0]).all(-1).cpu(), bad) and torch.equal(torch.isnan(v[0]).any(-1).cpu(), bad)
    assert torch.all(k[0, :, 0] == 0)


def test_append_reports_slots_and_positions(attn):
    d, H_kv, page = 64, 2, 16
    x = torch.randn(4, H_kv, d, device=dev()).half()
    kc, vc = (torch.full((2, H_kv, page, d // 2), 0x33, dtype=torch.uint8, device=dev()) for _ in range(2))
    kd, vd = (torch.ones(2, H_kv, page, device=dev()).bfloat16() for _ in range(2))
    attn.attn_cache_append_fp4(x, x, kc, vc, kd, vd, torch.tensor([32, -2, -1, 5], device=dev()))
    assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
    assert torch.all(kc[1] == 0x33) and (kc[0] != 0x33).any(-1).any(0).nonzero().ravel().tolist() == [5]
    cos, sin = (torch.from_numpy(t).float().to(dev()) for t in oracle.rope_table(8, d))
    slots = torch.arange(4, device=dev())
    for last, code in ((-1, 0), (8, attn.ATTN_ERR_INVALID_ARG)):
        attn.attn_cache_append_fp4(x, x, kc, vc, kd, vd, slots, cos, sin, _i32([0, 3, 7, last]))
        assert attn.attn_get_device_status() == code
        # unrotated: as the values of the same row
        assert torch.equal(kc[0, :, 3], vc[0, :, 3]) and torch.equal(kd[0, :, 3], vd[0, :, 3])
        assert not torch.equal(kc[0, :, 2], vc[0, :, 2])
    empty = x[:0]
    assert attn.attn_cache_append_fp4(empty, empty, kc, vc, kd, vd, slots[:0]) is None
    check_status(attn)


# -------------------------------------------------------------------- decode ----
def _decode_ref(q, cache, causal, signs, scale):
    kv, vv = cache.values()
    qq = _np(q)
    if signs is not None:
        qq = oracle.incoherent_transform(qq, signs.cpu().numpy())
    o, lse = oracle.attention_decode_paged(qq, kv, vv, cache.table, cache.lens, scale, causal)
    va, _ = oracle.attention_decode_paged(qq, kv, np.abs(vv), cache.table, cache.lens, scale, causal)
    G = q.shape[1] // cache.H_kv
    e = np.zeros(lse.shape)
    low = np.zeros(o.shape)
    sv = np.nan_to_num(np.float64(cache.descale[1]))
    code = np.swapaxes(np.abs(oracle.e2m1_decode(cache.codes[1])), 1, 2)
    for b, n in enumerate(cache.lens):
        if n == 0:
            continue
        at = np.arange(n)
        pages, rows = cache.table[b][at // cache.page], at % cache.page
        k = kv[pages, rows]                                                        # [n, H_kv, d]
        total = code[pages, rows].sum(0)
        for h in range(q.shape[1]):
            e[b, h] = scale * (np.abs(qq[b, h]) @ np.abs(k[:, h // G]).T).max(1) * 2.0 ** -16
            x = qq[b, h] @ k[:, h // G].T * scale
            p = np.exp(np.minimum(x - np.where(np.isfinite(lse[b, h]), lse[b, h], np.inf)[:, None], 0.0))
            low[b, h] = LAST[q.dtype] * (p * sv[pages, h // G, rows]).max(1)[:, None] * total[h // G]
    return o, lse, va, e, low


def _check_decode(q, o, lse, ref, what=""):
    ref_o, ref_l, va, e, low = ref
    got_l, got_o = _np(lse), _np(o)
    seen = np.isfinite(ref_l)
    assert np.array_equal(np.isfinite(got_l), seen) and np.all(got_l[~seen] == -np.inf) and np.all(got_o[~seen] == 0)
    off = np.abs(got_l[seen] - ref_l[seen])
    assert np.all(off <= e[seen] + 2.0 ** -20 * (1 + np.abs(ref_l[seen]))), (what, off.max())
    tol = (PROB[q.dtype] + 2.0 ** -16 + 2 * e[..., None]) * va + HALF[q.dtype] * np.abs(ref_o) + low + 2.0 ** -24
    assert np.all(np.abs(got_o - ref_o)[seen] <= tol[seen]), (what, np.abs(got_o - ref_o).max())


def _decode_case(attn, lens, page, H, H_kv, n_q, d, causal=True, dtype=torch.bfloat16, signs=False, seed=11, most=None,
                 cache=None, q=None):
    cache = cache or Cache(seed, lens, page, H_kv, d)
    if q is None:
        q = torch.from_numpy(workloads.normal(seed + 1, (len(lens), H, n_q, d))).to(dev(), dtype)
    sg = _signs(d) if signs else None
    o, co = guarded(q.shape, q.dtype, -7.0)
    lse, cl = guarded(q.shape[:3], torch.float32, -7.0)
    scale = 1 / np.sqrt(d)
    attn.attn_decode_paged_fp4(q, *cache.args(), max(1, most or max(lens)), causal=causal, softmax_scale=scale,
                               hadamard_signs=sg, o=o, lse=lse)
    check_status(attn)
    co()
    cl()
    _check_decode(q, o, lse, _decode_ref(q, cache, causal, sg, scale))
    return cache, q, o, lse


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_decode_page_sizes(attn, page, d, causal):
    _decode_case(attn, [1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 700], page, 8, 2, 2, d, causal)


@pytest.mark.parametrize("H,H_kv,n_q", [(32, 8, 1), (8, 1, 1), (4, 4, 1), (9, 1, 1), (8, 1, 2), (6, 2, 3), (17, 1, 1), (8, 1, 4),
                                        (16, 2, 16), (25, 5, 7)])
@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_heads_and_query_tokens(attn, H, H_kv, n_q, signs, d):
    _decode_case(attn, [300, 1025, 64, 0, 3], 32, H, H_kv, n_q, d, True, torch.float16, signs)


@pytest.mark.parametrize("G", [1, 5, 8, 11, 16, 40])
@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_every_kernel_in_bfloat16(attn, G, signs, d):
    """4, 8 and 16 rows, by clusters and (many sequences) by shares that segments cross."""
    _decode_case(attn, [700, 0, 129], 64, 2 * G, 2, 1, d, True, torch.bfloat16, signs)
    lens = np.random.default_rng(G).integers(0, 900, 90).tolist()
    _decode_case(attn, lens, 16, 4 * G, 4, 1, d, False, torch.bfloat16, signs)


@pytest.mark.parametrize("signs", [False, True])
def test_decode_long_sequences_are_shared(attn, signs):
    _decode_case(attn, [9000, 20000, 1], 64, 8, 2, 1, 128, True, torch.bfloat16, signs)


def test_decode_many_short_sequences(attn):
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, 400)
    lens[:130] = 0
    _decode_case(attn, lens.tolist(), 16, 4, 4, 1, 64, True, torch.float16)


def test_decode_rows_that_see_nothing_and_a_larger_bound(attn):
    _decode_case(attn, [2, 300, 0, 1], 16, 4, 4, 4, 64, True, torch.float16, most=5000)
    # a bound too small for the lengths costs time, not results
    _decode_case(attn, [700, 300, 0, 1000], 16, 4, 2, 1, 128, True, most=1)


@pytest.mark.parametrize("factor", [1e-20, 1e-3, 30.0, 3e4])
@pytest.mark.parametrize("signs", [False, True])
def test_decode_scales_of_queries(attn, factor, signs):
    """Queries far from 1: peaked rows and flat ones."""
    q = (torch.randn(3, 4, 1, 128, device=dev()) * factor).bfloat16()
    _decode_case(attn, [40, 333, 1000], 16, 4, 2, 1, 128, q=q, signs=signs)


@pytest.mark.parametrize("exponent", [-118, -121, -125])
@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_tiny_queries_and_large_keys(attn, exponent, signs, d):
    """Queries near the smallest normal number and keys as much above 1: ordinary scores."""
    lens = [40, 333, 1000]
    c = Cache(57, lens, 16, 2, d)
    c.descale[0] = c.descale[0] * np.float32(2.0 ** -exponent)
    q = torch.from_numpy(workloads.normal(58, (3, 4, 1, d)) * 2.0 ** exponent).to(dev(), torch.bfloat16)
    _decode_case(attn, lens, 16, 4, 2, 1, d, cache=c, q=q, signs=signs)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_transforms_large_queries(attn, d):
    """Queries of up to 2^127: the transform's sums stay in range.  All else is a power of two away: the same bits."""
    lens = [40, 333, 1000]
    c = Cache(59, lens, 16, 2, d)
    q = torch.from_numpy(workloads.normal(60, (3, 4, 2, d))).to(dev(), torch.bfloat16)
    got = []
    for up, down in ((1.0, 1.0), (2.0 ** 125, 2.0 ** -100)):
        kc, vc, kd, vd, bt, n = c.args()
        got.append(attn.attn_decode_paged_fp4(q * up, kc, vc, kd * down, vd, bt, n, 1000, hadamard_signs=_signs(d),
                                              softmax_scale=1 / np.sqrt(d) / (up * down)))
    check_status(attn)
    assert torch.isfinite(got[0][0].float()).all()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_decode_value_descales_that_differ(attn):
    """Rows of values of 0, of 2^-90 and of 2^60 beside ordinary ones, wherever they stand."""
    lens = [5, 200, 900]
    c = Cache(21, lens, 16, 2, 128)
    rng = np.random.default_rng(1)
    pick = rng.random(c.descale[1].shape)
    c.descale[1] = np.where(pick < 0.3, np.float32(0), np.where(pick < 0.4, np.float32(2.0 ** -90), c.descale[1])).astype(np.float32)
    c.descale[1][c.table[0, 0], 0, :5] = 0                     # all of a sequence's head
    c.descale[1][c.table[1, 3], 1, 7] = 2.0 ** 60
    c.descale[0][c.table[1, 2], 0, 3] = 0
    c.descale[0][c.table[2, 2], 1, 3] = 2.0 ** -100
    _decode_case(attn, lens, 16, 4, 2, 1, 128, cache=c)


def _one_hot(c, lens, d, n_heads, dtype, size, n_q=1, signs=None):
    """Makes one key of each request and head the only one with a component of 6 in column 0, the others have
    none there, and returns queries of `size` in that column (transformed ones where signs are given) and that
    key's position: every other key's score is `size` x 6 x its descale lower."""
    c.codes[0][..., 0] &= 0xF0
    at = [n // 2 for n in lens]
    for b, t in enumerate(at):
        if lens[b]:
            c.codes[0][c.table[b, t // c.page], :, t % c.page, 0] |= 7
            c.descale[0][c.table[b, t // c.page], :, t % c.page] = 1
    q = torch.zeros(len(lens), n_heads, n_q, d, device=dev())
    if signs is None:
        q[..., 0] = size
    else:
        q[:] = size / np.sqrt(d) * signs
    return q.to(dtype), at


SHAPES = [([300, 40, 1000, 1], 2), (list(range(3, 550, 6)), 4)]        # by clusters; by shares (92 sequences, 4 heads)
TYPES = [(64, torch.bfloat16), (128, torch.bfloat16), (128, torch.float16)]


@pytest.mark.parametrize("lens,H_kv", SHAPES, ids=["clusters", "shares"])
@pytest.mark.parametrize("G", [1, 8, 16])
@pytest.mark.parametrize("d,dtype", TYPES)
def test_decode_large_values_of_far_lower_scores(attn, lens, H_kv, G, d, dtype):
    """The key with the largest score has values of zero, the others (196 or more below in powers of two) large
    ones: their weights are 0, whatever the values are."""
    c = Cache(51, lens, 16, H_kv, d)
    c.descale[1] = np.where(c.owned, np.float32(1024), c.descale[1])
    q, at = _one_hot(c, lens, d, G * H_kv, dtype, 256.0)
    for b, t in enumerate(at):
        c.descale[1][c.table[b, t // 16], :, t % 16] = 0
    _decode_case(attn, lens, 16, G * H_kv, H_kv, 1, d, cache=c, q=q)


@pytest.mark.parametrize("lens,H_kv", SHAPES, ids=["clusters", "shares"])
@pytest.mark.parametrize("G", [1, 8, 16])
@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("d,dtype", TYPES)
def test_decode_of_one_key_with_all_the_weight(attn, lens, H_kv, G, signs, d, dtype):
    """Queries of 2^14 against keys of which one has a component there: the others' weights are below
    2^-10000.  O is that key's value row but for its own weight (1: the terms of 1 x descale), factors and
    rounding; a row of zeros, half of the row or another key's fail."""
    c = Cache(61, lens, 16, H_kv, d)
    c.codes[1] |= 0x22                   # magnitudes 1, 1.5, 4 and 6: no zeros
    sg = _signs(d) if signs else None
    q, at = _one_hot(c, lens, d, G * H_kv, dtype, 2.0 ** 14, signs=sg)
    o, lse = attn.attn_decode_paged_fp4(q, *c.args(), max(lens), hadamard_signs=sg)
    check_status(attn)
    v = c.values()[1]
    want = np.stack([np.repeat(v[c.table[b, t // 16], t % 16], G, 0) for b, t in enumerate(at)])[:, :, None]
    assert np.abs(want).min() > 0
    assert np.all(np.abs(_np(o) - want) <= (PROB[dtype] + 2.0 ** -16 + HALF[dtype]) * np.abs(want))
    # the score as the queries are rounded; the transform's float32 steps are each off by 2^-24
    x = _np(q)
    x = (x if sg is None else oracle.incoherent_transform(x, sg.cpu().numpy()))[..., 0] * 6 / np.sqrt(d)
    assert np.all(np.abs(_np(lse) - x) <= 2.0 ** -18 * x)


@pytest.mark.parametrize("lens,H_kv", SHAPES, ids=["clusters", "shares"])
@pytest.mark.parametrize("G", [1, 2, 4])
@pytest.mark.parametrize("d,dtype", TYPES)
def test_decode_large_values_of_unseen_tokens(attn, lens, H_kv, G, d, dtype):
    """The first query tokens see values of zero only, the last ones large values too."""
    c = Cache(52, lens, 16, H_kv, d)
    for b, n in enumerate(lens):
        at = np.arange(n)
        c.descale[1][c.table[b][at // 16], :, at % 16] = np.where(at < n - 2, 0, np.where(at < n - 1, 0.25, 1024))[:, None]
    q = torch.from_numpy(workloads.normal(53, (len(lens), G * H_kv, 4, d))).to(dev(), dtype)
    _, _, o, _ = _decode_case(attn, lens, 16, G * H_kv, H_kv, 4, d, cache=c, q=q)
    assert torch.all(o[:, :, :2] == 0)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_value_descales_130_powers_of_two_apart(attn, d):
    """The key that has all the weight has the smallest descale: O is its row, exact but for the last e4m3
    term, the factors' and the output's rounding."""
    lens, dtype = [300, 40, 1000, 1], torch.bfloat16
    c = Cache(54, lens, 16, 2, d)
    c.descale[1] = np.where(c.owned, np.float32(2.0 ** 30), c.descale[1])
    q, at = _one_hot(c, lens, d, 4, dtype, 256.0)
    for b, t in enumerate(at):
        c.descale[1][c.table[b, t // 16], :, t % 16] = 2.0 ** -100
    o, lse = attn.attn_decode_paged_fp4(q, *c.args(), 1000)
    check_status(attn)
    v = c.values()[1]
    want = np.stack([np.repeat(v[c.table[b, t // 16], t % 16], 2, 0) for b, t in enumerate(at)])[:, :, None]
    assert np.all(np.abs(_np(o) - want) <= (PROB[dtype] + 2.0 ** -16 + HALF[dtype]) * np.abs(want))


@pytest.mark.parametrize("lens,H_kv", SHAPES, ids=["clusters", "shares"])
@pytest.mark.parametrize("G", [1, 2, 4])
@pytest.mark.parametrize("d,dtype", TYPES)
def test_decode_nan_values_of_unseen_tokens(attn, lens, H_kv, G, d, dtype):
    """The last token's value rows are NaN: only the last query token, which sees it, shows that."""
    lens = [*lens, 2]                    # (the first two of four query tokens see nothing)
    c = Cache(55, lens, 16, H_kv, d)
    q = torch.from_numpy(workloads.normal(56, (len(lens), G * H_kv, 4, d))).to(dev(), dtype)
    got = []
    for last in (0.0, np.nan):
        for b, n in enumerate(lens):
            c.descale[1][c.table[b, (n - 1) // 16], :, (n - 1) % 16] = last
        got.append(attn.attn_decode_paged_fp4(q, *c.args(), max(lens)))
        if last == 0:
            ref = _decode_ref(q, c, True, None, 1 / np.sqrt(d))
    check_status(attn)
    _check_decode(q, *got[0], ref)
    assert torch.isnan(got[1][0][:, :, 3].float()).all()
    got[1][0][:, :, 3] = got[0][0][:, :, 3]
    _check_decode(q, *got[1], ref)


def test_decode_nan_rows_show(attn):
    lens = [300, 40]
    for which in (0, 1):
        c = Cache(22, lens, 32, 2, 64)
        c.descale[which][c.table[0, 2], 1, 9] = np.nan
        q = torch.randn(2, 4, 1, 64, device=dev()).half()
        o, lse = attn.attn_decode_paged_fp4(q, *c.args(), 300)
        check_status(attn)
        assert torch.isnan(o[0, 2:].float()).all() and torch.isfinite(o[0, :2].float()).all() and torch.isfinite(o[1].float()).all()
        assert torch.isnan(lse[0, 2:]).all() == (which == 0) and torch.isfinite(lse[0, :2]).all()


def test_decode_reports_bad_pages_and_lengths(attn):
    c = Cache(23, [200, 90], 32, 2, 128)
    q = torch.randn(2, 4, 1, 128, device=dev()).bfloat16()
    args = list(c.args())
    for bad in (-1, c.codes[0].shape[0], 2 ** 31 - 1):
        table = c.table.copy()
        table[0, 2] = bad
        args[4] = _i32(table)
        o, lse = attn.attn_decode_paged_fp4(q, *args, 200)
        assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
        # the page's tokens are not seen
        keep = [t for t in range(200) if t // 32 != 2]
        kv, vv = c.values()
        k, v = (x[c.table[0][np.array(keep) // 32], np.array(keep) % 32] for x in (kv, vv))
        for h in range(4):
            s = k[:, h // 2] @ _np(q[0, h, 0]) / np.sqrt(128)
            p = np.exp(s - s.max())
            want = p @ v[:, h // 2] / p.sum()
            assert np.abs(_np(o[0, h, 0]) - want).max() < 2.0 ** -7 * np.abs(v).max()
    args[4] = _i32(c.table)
    for bad in (-3, c.table.shape[1] * 32 + 1):
        args[5] = _i32([bad, 90])
        o, lse = attn.attn_decode_paged_fp4(q, *args, 200)
        assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
        assert torch.all(o[0] == 0) and torch.all(lse[0] == -np.inf) and torch.isfinite(lse[1]).all()
    check_status(attn)


def test_decode_offsets_beyond_32_bits(attn):
    """A cache of over 2^32 bytes, the sequences on its last pages."""
    H_kv, page, d, lens = 8, 64, 128, [150, 70]
    c = Cache(24, lens, page, H_kv, d)
    num = 2 ** 32 // (H_kv * page * d // 2) + 40
    used = c.codes[0].shape[0]
    big = [torch.empty(num, H_kv, page, d // 2, dtype=torch.uint8, device=dev()) for _ in range(2)]
    des = [torch.empty(num, H_kv, page, dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    args = c.args()
    for x, y in zip(big + des, args[:4]):
        x[num - used:] = y
    table = _i32(np.where(c.table >= 0, c.table + num - used, -5))
    q = torch.randn(2, 16, 1, d, device=dev()).bfloat16()
    got = attn.attn_decode_paged_fp4(q, *big, *des, table, args[5], 150)
    want = attn.attn_decode_paged_fp4(q, *args, 150)
    k1, v1 = attn.attn_cache_read_fp4(*big, *des, table, args[5], 150)
    k0, v0 = attn.attn_cache_read_fp4(*args, 150)
    x = torch.randn(2, H_kv, d, device=dev()).bfloat16()
    attn.attn_cache_append_fp4(x, x, *big, *des, torch.tensor([num * page - 1, num * page - 70], device=dev()))
    check_status(attn)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(k0, k1) and torch.equal(v0, v1)
    assert torch.equal(big[0][-1, :, -1], big[1][-1, :, -1]) and torch.isfinite(des[0][-1, :, -1].float()).all()


@pytest.mark.parametrize("lens", [[3000, 17, 0, 900], [3000, 0, *range(5, 3000, 31)]], ids=["clusters", "shares"])
def test_decode_runs_alike_in_graphs_on_other_streams_and_again(attn, lens):
    """The same bits from a second call, from another stream and from two captured graphs that
    replay at the same time, each with its own workspace."""
    c = Cache(25, lens, 32, 2, 128)
    q = torch.randn(len(lens), 8, 1, 128, device=dev()).bfloat16()
    args, sg = c.args(), _signs(128)
    ref = attn.attn_decode_paged_fp4(q, *args, 3000, hadamard_signs=sg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = [attn.attn_decode_paged_fp4(q, *args, 3000, hadamard_signs=sg),
            attn.attn_decode_paged_fp4(q, *args, 3000, hadamard_signs=sg, stream=side)]
    torch.cuda.synchronize()
    graphs = []
    for s in (side, torch.cuda.Stream()):
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = attn.attn_decode_paged_fp4(q, *args, 3000, hadamard_signs=sg)
        graphs.append((g, out, s))
    for _ in range(5):
        for g, out, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    check_status(attn)
    for o, lse in runs + [out for _, out, _ in graphs]:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


# ----------------------------------------------------------------- reading back ----
def _rows(c, which, first, counts, signs=None):
    v = c.values()[which]
    rows = oracle.read_cache(v, c.table, c.lens, first, counts)
    if signs is not None:       # x M^T: the transform of the transformed, signs last
        one = np.ones(c.d)
        rows = [oracle.incoherent_transform(r, one) * signs.cpu().numpy() if len(r) else r for r in rows]
    return rows


def _close_rows(got, want, dtype, exact):
    got, want = _np(got), np.asarray(want)
    if exact:
        rounded = torch.from_numpy(want).float().to(dtype).double().numpy()
        assert np.array_equal(got, rounded)
        return
    tol = HALF[dtype] * np.abs(want) + 2.0 ** -20 * np.linalg.norm(want, axis=-1, keepdims=True) + 2.0 ** -25
    assert np.all(np.abs(got - want) <= tol * (1 + 2.0 ** -8))


@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (128, 256)])
@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_read_fp4(attn, d, page, signs, dtype):
    lens, first = [300, 0, 1, 129, 64], [17, 0, 0, 128, 64]
    c = Cache(31, lens, page, 3, d)
    sg = _signs(d) if signs else None
    n = 200
    k, ck = guarded((5, 3, n, d), dtype, -7.0)
    v, cv = guarded((5, 3, n, d), dtype, -7.0)
    attn.attn_cache_read_fp4(*c.args(), n, first=_i32(first), hadamard_signs=sg, dtype=dtype, k=k, v=v)
    check_status(attn)
    ck()
    cv()
    for got, which in ((k, 0), (v, 1)):
        s = sg if which == 0 else None
        want = np.stack(_rows(c, which, first, [n] * 5, s)).transpose(0, 2, 1, 3)
        _close_rows(got, want, dtype, s is None)
    # packed, with room behind the last request
    counts = [283, 0, 1, 1, 0]
    cu = np.concatenate([[0], np.cumsum(counts)])
    room = int(cu[-1]) + 40
    k, ck = guarded((room, 3, d), dtype, -7.0)
    v, cv = guarded((room, 3, d), dtype, -7.0)
    attn.attn_cache_read_fp4(*c.args(), room, first=_i32(first), cu_seqlens=_i32(cu), hadamard_signs=sg, dtype=dtype, k=k, v=v)
    check_status(attn)
    ck()
    cv()
    for got, which in ((k, 0), (v, 1)):
        s = sg if which == 0 else None
        _close_rows(got[:cu[-1]], np.concatenate(_rows(c, which, first, counts, s)), dtype, s is None)
        assert torch.all(got[cu[-1]:] == -7.0)


@pytest.mark.parametrize("bits,d", [(4, 64), (4, 128), (8, 128)])
def test_read_restores_large_keys(attn, bits, d):
    """Keys of up to 2^127: the transform's sums stay in range.  All is a power of two larger, the same bits."""
    lens, page = [70, 1, 33], 16
    if bits == 4:
        c = Cache(44, lens, page, 2, d)
        c.descale = [np.nan_to_num(s) for s in c.descale]
        kc, vc, kd, vd, bt, n = c.args()
        read = attn.attn_cache_read_fp4
    else:
        rng = np.random.default_rng(45)
        table, num = _table(rng, lens, page)
        (kc, kd), (vc, vd) = (oracle.quantize_paged_cache(rng.standard_normal((num, page, 2, d)).astype(np.float32)) for _ in range(2))
        kc, kd, vc, vd = (torch.from_numpy(np.ascontiguousarray(x)).to(dev()) for x in (kc, kd, vc, vd))
        bt, n, read = _i32(table), _i32(lens), attn.attn_cache_read_fp8
    k, v = read(kc, vc, kd, vd, bt, n, 70, hadamard_signs=_signs(d))
    up = 2.0 ** 125
    big_k, big_v = read(kc, vc, kd * up, vd * up, bt, n, 70, hadamard_signs=_signs(d))
    check_status(attn)
    assert torch.isfinite((k * up).float()).all() and torch.any(k != 0)
    assert torch.equal(k * up, big_k) and torch.equal(v * up, big_v)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_read_other_caches(attn, bits, d):
    if bits == 8 and d != 128:
        pytest.skip("the e4m3 cache has d = 128")
    lens, page, H_kv, n = [70, 1, 0, 33], 16, 2, 71
    rng = np.random.default_rng(6)
    table, num = _table(rng, lens, page)
    sg = _signs(d) if bits == 8 else None
    shape = (num, page, H_kv, d)
    if bits == 16:
        kc, vc = (torch.from_numpy(rng.standard_normal(shape)).half().to(dev()) for _ in range(2))
        read = lambda **kw: attn.attn_cache_read(kc, vc, _i32(table), _i32(lens), kw.pop("n", n), **kw)
        values, dtype = [_np(kc), _np(vc)], torch.float16
    else:
        (kc, ks), (vc, vs) = (oracle.quantize_paged_cache(rng.standard_normal(shape).astype(np.float32)) for _ in range(2))
        up = [torch.from_numpy(np.ascontiguousarray(x)).to(dev()) for x in (kc, vc, ks, vs)]
        read = lambda **kw: attn.attn_cache_read_fp8(*up, _i32(table), _i32(lens), kw.pop("n", n), hadamard_signs=sg, **kw)
        # code x descale as a float32 product
        values = [np.float64(np.float32(oracle.dequantize_paged_cache(c, s))) for c, s in ((kc, ks), (vc, vs))]
        dtype = torch.bfloat16
    k, v = read()
    pk, pv = read(n=75, first=_i32([40, 0, 0, 0]), cu_seqlens=_i32([0, 30, 31, 31, 64]))
    check_status(attn)
    for got, packed, val, s in ((k, pk, values[0], sg), (v, pv, values[1], None)):
        def undo(r):
            return r if s is None else oracle.incoherent_transform(r, np.ones(d)) * s.cpu().numpy()
        want = undo(np.stack(oracle.read_cache(val, table, lens, [0] * 4, [n] * 4))).transpose(0, 2, 1, 3)
        _close_rows(got, want, dtype, s is None)
        want = undo(np.concatenate(oracle.read_cache(val, table, lens, [40, 0, 0, 0], [30, 1, 0, 33])))
        _close_rows(packed[:64], want, dtype, s is None)


@pytest.mark.parametrize("bits,d", [(16, 64), (16, 256), (8, 128), (4, 64), (4, 128)])
def test_read_of_many_rows_is_that_of_few(attn, bits, d):
    """A block of a long range takes several planes (keys and values of 5 heads: not a multiple of them), one
    of a short range a single one: the same bits, padded and packed."""
    lens, page, H_kv, n = [9000, 0, 7001], 32, 5, 9000
    if bits == 4:
        c = Cache(35, lens, page, H_kv, d)
        args, kw, call = c.args(), dict(hadamard_signs=_signs(d)), attn.attn_cache_read_fp4
    else:
        rng = np.random.default_rng(36)
        table, pages = _table(rng, lens, page)
        shape = (pages, page, H_kv, d)
        kc, vc = (torch.randn(shape, device=dev()).bfloat16() if bits == 16 else
                  torch.randint(0, 120, shape, device=dev(), dtype=torch.uint8) for _ in range(2))
        scales = [torch.rand(pages, H_kv, device=dev()) + 0.5 for _ in range(2)] if bits == 8 else []
        args = (kc, vc, *scales, _i32(table), _i32(lens))
        kw, call = (dict(hadamard_signs=_signs(d)), attn.attn_cache_read_fp8) if bits == 8 else ({}, attn.attn_cache_read)
    k, v = call(*args, n, **kw)
    for at in (0, 4000, 7000, 8970):
        few = call(*args, 30, first=_i32([at] * 3), **kw)
        assert torch.equal(k[:, :, at:at + 30], few[0]) and torch.equal(v[:, :, at:at + 30], few[1])
    assert torch.all(k[1] == 0) and torch.all(v[2, :, 7001:] == 0) and torch.any(v[0, :, 8999] != 0)
    cu = _i32(np.concatenate([[0], np.cumsum(lens)]))
    kp, vp = call(*args, sum(lens), cu_seqlens=cu, **kw)
    check_status(attn)
    for packed, padded in ((kp, k), (vp, v)):
        assert torch.equal(packed[:9000], padded[0].transpose(0, 1)) and torch.equal(packed[9000:], padded[2, :, :7001].transpose(0, 1))


def test_read_of_very_many_requests(attn):
    """Packed outputs take any number of requests, padded ones up to 65,535 (a dimension of the grid)."""
    B, page, H_kv, d = 70000, 16, 1, 64
    rng = np.random.default_rng(37)
    lens = rng.integers(0, 3, B)
    lens[30000:30500] = 0                         # more empty ones than a block keeps at hand
    cu = np.concatenate([[0], np.cumsum(lens)])
    kc, vc = (torch.randn(50, page, H_kv, d, device=dev()).bfloat16() for _ in range(2))
    table = rng.integers(0, 50, (B, 1))
    k, v = attn.attn_cache_read(kc, vc, _i32(table), _i32(lens), int(cu[-1]), cu_seqlens=_i32(cu))
    check_status(attn)
    b = np.repeat(np.arange(B), lens)
    at = torch.from_numpy(table[b, 0]).to(dev()), torch.from_numpy(np.arange(cu[-1]) - cu[b]).to(dev())
    assert torch.equal(k, kc[at]) and torch.equal(v, vc[at])
    with pytest.raises(attn.AttnError, match="65535"):
        attn.attn_cache_read(kc, vc, _i32(table), _i32(lens), 1)


def test_read_reports_what_does_not_fit(attn):
    c = Cache(33, [40, 40], 16, 2, 64)
    kc, vc, kd, vd, bt, lens = c.args()
    good, _ = attn.attn_cache_read_fp4(kc, vc, kd, vd, bt, lens, 40)
    bad = bt.clone()
    bad[0, 1] = kc.shape[0]
    cases = [(bad, lens, None), (bt, _i32([-1, 40]), None), (bt, _i32([2 ** 31 - 1, 40]), None), (bt, lens, _i32([-1, 0]))]
    for table, n, first in cases:
        k, v = attn.attn_cache_read_fp4(kc, vc, kd, vd, table, n, 40, first=first)
        assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
        assert torch.equal(k[1], good[1])
        if table is bad:
            assert torch.equal(k[0, :, :16], good[0, :, :16]) and torch.all(k[0, :, 16:32] == 0)
            assert torch.equal(k[0, :, 32:], good[0, :, 32:])
        else:
            assert torch.all(k[0] == 0) and torch.all(v[0] == 0)
    # a first position behind the sequence: nothing, padded; packed rows there are reported
    k, _ = attn.attn_cache_read_fp4(kc, vc, kd, vd, bt, lens, 40, first=_i32([2 ** 31 - 1, 40]))
    check_status(attn)
    assert torch.all(k == 0)
    packed = good.transpose(1, 2).reshape(80, 2, 64)
    for cu, first in (([0, 41, 80], None), ([0, 40, 79], [1, 1])):
        k, _ = attn.attn_cache_read_fp4(kc, vc, kd, vd, bt, lens, 80, cu_seqlens=_i32(cu), first=None if first is None else _i32(first))
        assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
    assert torch.equal(k[:39], packed[1:40]) and torch.all(k[39] == 0)
    for cu in ([0, 50, 40], [-1, 40, 80], [0, 40, 81], [1, 40, 80]):
        k, ck = guarded((80, 2, 64), torch.bfloat16, -7.0)
        v, cv = guarded((80, 2, 64), torch.bfloat16, -7.0)
        attn.attn_cache_read_fp4(kc, vc, kd, vd, bt, lens, 80, cu_seqlens=_i32(cu), k=k, v=v)
        assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG, cu
        ck()
        cv()
    k, v = attn.attn_cache_read_fp4(kc, vc, kd, vd, bt, lens, 0)
    check_status(attn)
    assert k.shape == (2, 2, 0, 64)


# ------------------------------------------------------------------------ merge ----
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 3, 33), (3, 8, 130)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("packed", [False, True])
def test_merge(attn, shape, d, packed):
    B, H, N = shape
    dtype = torch.float16 if d == 64 else torch.bfloat16
    rng = np.random.default_rng(B * N)
    full, rows = ((N, H, d), (H, N)) if packed else ((B, H, N, d), (B, H, N))
    oa, ob = (torch.from_numpy(rng.standard_normal(full)).to(dev(), dtype) for _ in range(2))
    la, lb = (torch.from_numpy(5 * rng.standard_normal(rows)).float().to(dev()) for _ in range(2))
    if N > 8:
        la[..., 2], lb[..., 3], la[..., 4], lb[..., 4] = [-float("inf")] * 4
        for o, n in ((oa, 2), (ob, 3), (oa, 4)):
            (o[n] if packed else o[:, :, n]).fill_(float("nan"))
        la[..., 5] = 200.0
    host = lambda o: _np(o).swapaxes(0, 1) if packed else _np(o)
    ref_o, ref_l = oracle.merge_attention(host(oa), _np(la), host(ob), _np(lb))
    o, lse = attn.attn_merge(oa, la, ob, lb)
    check_status(attn)
    tol = HALF[dtype] * np.abs(ref_o) + 2.0 ** -20 * (np.abs(np.nan_to_num(host(oa))) + np.abs(np.nan_to_num(host(ob))))
    assert np.all(np.abs(host(o) - ref_o) <= tol + 2.0 ** -25)
    fin = np.isfinite(ref_l)
    assert np.array_equal(_np(lse)[~fin], ref_l[~fin])
    assert np.all(np.abs(_np(lse) - ref_l)[fin] <= 2.0 ** -21 * (2 + np.abs(ref_l[fin])))
    # in place over either input
    for x, y in (((oa, la), (ob, lb)), ((ob, lb), (oa, la))):
        xo, xl = x[0].clone(), x[1].clone()
        got = attn.attn_merge(xo, xl, *y, o=xo, lse=xl)
        assert got[0].data_ptr() == xo.data_ptr()
        swapped = attn.attn_merge(*x, *y)
        assert torch.equal(xo, swapped[0]) and torch.equal(xl, swapped[1])
    check_status(attn)


def test_merge_of_unusual_log_sum_exps(attn):
    """+inf beats every finite one; NaN shows."""
    inf = float("inf")
    o = torch.ones(1, 1, 3, 64, device=dev()).half()
    la = torch.tensor([[[float("nan"), 1e30, -1e30]]], device=dev())
    lb = torch.tensor([[[1.0, 1.0, -inf]]], device=dev())
    got, lse = attn.attn_merge(o, la, 2 * o, lb)
    check_status(attn)
    assert torch.isnan(got[0, 0, 0]).all() and torch.isnan(lse[0, 0, 0])
    assert torch.all(got[0, 0, 1:] == 1) and lse[0, 0, 1] == 1e30 and lse[0, 0, 2] == -1e30


@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 8, 130)])
@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.float16), (256, torch.float16)])
@pytest.mark.parametrize("packed", [False, True])
def test_merge_of_the_other_types(attn, shape, d, dtype, packed):
    """The kernels that test_merge does not run, in place too."""
    B, H, N = shape
    rng = np.random.default_rng(71 + B * N)
    full, rows = ((N, H, d), (H, N)) if packed else ((B, H, N, d), (B, H, N))
    oa, ob = (torch.from_numpy(rng.standard_normal(full)).to(dev(), dtype) for _ in range(2))
    la, lb = (torch.from_numpy(5 * rng.standard_normal(rows)).float().to(dev()) for _ in range(2))
    la[..., ::7], lb[..., ::5] = -float("inf"), -float("inf")
    host = lambda o: _np(o).swapaxes(0, 1) if packed else _np(o)
    ref_o, ref_l = oracle.merge_attention(host(oa), _np(la), host(ob), _np(lb))
    o, lse = attn.attn_merge(oa, la, ob, lb)
    check_status(attn)
    tol = HALF[dtype] * np.abs(ref_o) + 2.0 ** -20 * (np.abs(host(oa)) + np.abs(host(ob))) + 2.0 ** -25
    assert np.all(np.abs(host(o) - ref_o) <= tol)
    fin = np.isfinite(ref_l)
    assert np.array_equal(_np(lse)[~fin], ref_l[~fin])
    assert np.all(np.abs(_np(lse)[fin] - ref_l[fin]) <= 2.0 ** -21 * (2 + np.abs(ref_l[fin])))
    for xo, xl, a, b in ((oa.clone(), la.clone(), None, (ob, lb)), (ob.clone(), lb.clone(), (oa, la), None)):
        attn.attn_merge(*(a or (xo, xl)), *(b or (xo, xl)), o=xo, lse=xl)
        assert torch.equal(xo, o) and torch.equal(xl, lse)
    check_status(attn)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_merge_of_infinities_and_nan(attn, d, packed, dtype):
    """They show unless their part is empty, also where its weight is 0 in float32; an lse of +inf is NaN."""
    inf, nan = float("inf"), float("nan")
    la = torch.tensor([0.0, 0.0, 0.0, 0.0, -inf, inf, inf, 0.0], device=dev())
    lb = torch.tensor([-5.0, -150.0, -900.0, -150.0, 0.0, 0.0, inf, 0.0], device=dev())
    oa, ob = (torch.ones(8, 1, d, device=dev()).to(dtype) for _ in range(2))
    ob[0:3, :, 7] = inf
    ob[3, :, 7] = nan
    oa[4] = nan
    shape = (lambda x: x) if packed else (lambda x: x.transpose(0, 1)[None])
    rows = (lambda x: x[None]) if packed else (lambda x: x[None, None])
    want_bad = torch.zeros(8, d, dtype=torch.bool)
    want_bad[0:4, 7] = True
    want_bad[5:7] = True
    for first, second in (((oa, la), (ob, lb)), ((ob, lb), (oa, la))):
        o, lse = attn.attn_merge(shape(first[0]), rows(first[1]), shape(second[0]), rows(second[1]))
        check_status(attn)
        o, lse = o.reshape(8, d).float().cpu(), lse.ravel().cpu()
        assert torch.equal(~torch.isfinite(o), want_bad) and torch.all(o[~want_bad] == 1)
        assert torch.equal(torch.isnan(lse), want_bad[:, 0]) and lse[4] == 0


# ---------------------------------------------------------------------- together ----
@pytest.mark.parametrize("d,signs", [(128, True), (64, False)])
def test_prompts_in_chunks_then_tokens(attn, d, signs):
    """As a server uses it: block tables -> append -> [prefix read back -> cross attention over it,
    causal attention over the chunk, joined] for two chunks of each prompt, then decode steps from
    a captured graph, against attention over the values that the cache holds."""
    B, H, H_kv, page, chunk, dtype = 2, 4, 2, 16, 40, torch.bfloat16
    G, scale, sg = H // H_kv, 1 / np.sqrt(d), _signs(d) if signs else None
    cos, sin = attn.attn_rope_table(128, d)
    num = 20
    kc, vc = (torch.zeros(num, H_kv, page, d // 2, dtype=torch.uint8, device=dev()) for _ in range(2))
    kd, vd = (torch.full((num, H_kv, page), float("nan"), device=dev()).bfloat16() for _ in range(2))
    table = torch.full((B, 8), -1, dtype=torch.int32, device=dev())
    free = torch.randperm(num, device=dev()).int()
    old, taken = _i32([0] * B), 0

    def stored(lens):
        c = [oracle.dequantize_cache_fp4(x.cpu().numpy(), s.float().cpu().numpy()) for x, s in ((kc, kd), (vc, vd))]
        at = lambda x, b, n: np.stack([x[int(table[b, t // page]), t % page] for t in range(n)])
        k, v = ([at(x, b, int(n)) for b, n in enumerate(lens)] for x in c)
        if sg is not None:
            k = [oracle.incoherent_transform(x, np.ones(d)) * sg.cpu().numpy() for x in k]
        return k, v

    for step in range(2):
        new = _i32([chunk] * B)
        rows = torch.randn(B * chunk, H + 2 * H_kv, d, device=dev()).to(dtype)
        lens, cu, slots, pos, used = attn.attn_block_tables(table, old, new, free[taken:], page, B * chunk)
        taken += int(used)
        q = attn.attn_cache_append_fp4(rows[:, H:H + H_kv], rows[:, H + H_kv:], kc, vc, kd, vd, slots, cos, sin, pos,
                                       hadamard_signs=sg, q=rows[:, :H])
        q4 = q.view(B, chunk, H, d).transpose(1, 2).contiguous()
        # the chunk itself attends over what was stored, as the decode will
        ck, cv = attn.attn_cache_read_fp4(kc, vc, kd, vd, table, lens, chunk, first=old, hadamard_signs=sg)
        o, lse = attn.attn_fwd_gqa(q4, ck, cv, causal=True)
        n = max(1, int(old.max()))
        pk, pv = attn.attn_cache_read_fp4(kc, vc, kd, vd, table, old, n, hadamard_signs=sg)
        po, pl = attn.attn_cross_fwd(q4, pk, pv, kv_lens=old)
        attn.attn_merge(o, lse, po, pl, o=o, lse=lse)
        check_status(attn)
        k, v = stored(lens.cpu())
        n0 = int(old[0])
        for b in range(B):
            for h in range(H):
                s = _np(q4[b, h]) @ k[b][:, h // G].T * scale
                s[np.arange(chunk)[:, None] + n0 < np.arange(n0 + chunk)[None, :]] = -np.inf
                p = np.exp(s - s.max(1, keepdims=True))
                want = p @ v[b][:, h // G] / p.sum(1, keepdims=True)
                # three roundings of O, of stored rows and of P: 2^-8 each of sizes of at most max |v|
                assert np.abs(_np(o[b, h]) - want).max() < 6 * 2.0 ** -8 * np.abs(v[b]).max()
                assert np.abs(_np(lse[b, h]) - (s.max(1) + np.log(p.sum(1)))).max() < 2.0 ** -8 * 8
        old = lens
    # decode steps: one graph, its inputs replaced
    rows = torch.randn(B, H + 2 * H_kv, d, device=dev()).to(dtype)
    one, lens_in, pages = _i32([1] * B), old.clone(), free.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def decode():
        lens, cu, slots, pos, used = attn.attn_block_tables(table, lens_in, one, pages, page, B)
        q = attn.attn_cache_append_fp4(rows[:, H:H + H_kv], rows[:, H + H_kv:], kc, vc, kd, vd, slots, cos, sin, pos,
                                       hadamard_signs=sg, q=rows[:, :H])
        o, lse = attn.attn_decode_paged_fp4(q[:, :, None].contiguous(), kc, vc, kd, vd, table, lens, 128, hadamard_signs=sg)
        return lens, q, o, lse, used

    pages[:num - taken] = free[taken:]
    saved = table.clone()
    with torch.cuda.stream(side):
        decode()
    torch.cuda.synchronize()
    table.copy_(saved)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lens, q, o, lse, used = decode()
    for _ in range(3):
        pages[:num - taken] = free[taken:]
        rows.copy_(torch.randn(rows.shape, device=dev()))
        g.replay()
        torch.cuda.synchronize()
        check_status(attn)
        taken += int(used)
        k, v = stored(lens.cpu())
        for b in range(B):
            for h in range(H):
                s = _np(q[b, h]) @ k[b][:, h // G].T * scale
                p = np.exp(s - s.max())
                want = p @ v[b][:, h // G] / p.sum()
                assert np.abs(_np(o[b, h, 0]) - want).max() < 2 * 2.0 ** -8 * np.abs(v[b]).max()
                assert abs(float(lse[b, h, 0]) - s.max() - np.log(p.sum())) < 2.0 ** -12
        lens_in.copy_(lens)


def test_host_tensors(attn):
    """CPU tensors are copied to the device and the results back."""
    c = Cache(41, [50, 7], 16, 2, 64)
    args = [x.cpu() for x in c.args()]
    q = torch.randn(2, 4, 1, 64).half()
    o, lse = attn.attn_decode_paged_fp4(q, *args, 50)
    go, gl = attn.attn_decode_paged_fp4(q.to(dev()), *c.args(), 50)
    assert o.device.type == "cpu" and torch.equal(o, go.cpu()) and torch.equal(lse, gl.cpu())
    k, v = attn.attn_cache_read_fp4(*args, 50, first=torch.tensor([1, 0], dtype=torch.int32))
    gk, gv = attn.attn_cache_read_fp4(*c.args(), 50, first=_i32([1, 0]))
    assert torch.equal(k, gk.cpu()) and torch.equal(v, gv.cpu())
    m = attn.attn_merge(o, lse, o, lse)
    assert m[0].device.type == "cpu" and torch.allclose(m[1], lse + np.log(2), atol=1e-5)


def test_calls_on_another_stream_than_the_current(attn):
    """Inputs and outputs belong to the call's stream; the current one is not waited for."""
    side = torch.cuda.Stream()
    c = Cache(42, [333, 1], 64, 2, 128)
    args = c.args()
    q = torch.randn(2, 4, 1, 128, device=dev()).bfloat16()
    ref = attn.attn_decode_paged_fp4(q, *args, 333)
    rk = attn.attn_cache_read_fp4(*args, 333)
    torch.cuda.synchronize()
    for _ in range(10):
        o, lse = attn.attn_decode_paged_fp4(q, *args, 333, stream=side)
        k, _ = attn.attn_cache_read_fp4(*args, 333, stream=side)
        side.synchronize()
        assert torch.equal(o, ref[0]) and torch.equal(k, rk[0])
    check_status(attn)
