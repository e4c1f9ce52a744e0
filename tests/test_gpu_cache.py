"""Block tables, slot maps and cache appends against the oracle, and a decoder layer's
attention run through them.

Tolerances.  Tables, slots, copied values and everything of an append that only
moves or requantises are exact.  Rotated 16-bit values: as for the rotation
(2^-22 of the two products, then one rounding).  e4m3 codes of rotated or
transformed keys: the float32 row is off by at most e = 2^-20 |row| (the rotation's
products, seven butterfly stages and two scalings), so the value is within half an
e4m3 step (2^-4 of it, or 2^-10 descales) plus e."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from gpu_util import LSE_ABS, check_status, dev, guarded, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    return lib()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev())


def _state(seed, old, new, page, spare=5):
    """Block table of the old tokens, free list and page count from one shuffled pool."""
    rng = np.random.default_rng(seed)
    old, new = np.asarray(old), np.asarray(new)
    have, need = -(-old // page), -(-(old + new) // page)
    num = int(need.sum()) + spare
    order = rng.permutation(num)
    width = max(1, int(need.max()))
    table = np.full((len(old), width), -1)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order[at:], num


def _tables_match(attn, old, new, page, seed=1, extra=0):
    table, free, _ = _state(seed, old, new, page)
    total = int(np.sum(new))
    cap = total + extra
    bt, check = guarded(table.shape, torch.int32, -77)
    bt.copy_(_i32(table))
    got = attn.attn_block_tables(bt, _i32(old), _i32(new), _i32(free), page, cap)
    check_status(attn)
    check()
    ref = oracle.block_tables(table, old, new, free, page, cap)
    for x, y, what in zip((bt, *got), ref, ("table", "seq_lens", "cu", "slots", "positions", "used")):
        assert np.array_equal(x.cpu().numpy().ravel(), np.ravel(y)), what
    return bt, got


@pytest.mark.parametrize("page", [8, 16, 256])
@pytest.mark.parametrize("B", [1, 3, 33, 700])
def test_tables_of_decode_steps(attn, page, B):
    rng = np.random.default_rng(B)
    _tables_match(attn, rng.integers(0, 600, B), rng.integers(0, 3, B), page, extra=B % 5)


@pytest.mark.parametrize("B,most", [(1, 5000), (40, 900), (1100, 60)])
def test_tables_of_prompts(attn, B, most):
    rng = np.random.default_rng(most)
    _tables_match(attn, rng.integers(0, 300, B) * (rng.random(B) < 0.5), rng.integers(0, most, B), 16)


def test_tables_of_nothing_and_of_page_borders(attn):
    _tables_match(attn, [0, 16, 5], [0, 0, 0], 16)
    _tables_match(attn, [0, 15, 16, 17, 31, 32], [16, 1, 1, 15, 1, 33], 16, extra=3)
    _tables_match(attn, np.arange(16384) % 40, np.arange(16384) % 2, 8)


def test_tables_report_what_does_not_fit(attn):
    table = np.full((4, 4), -1)
    table[1, :1] = 3
    bt = _i32(table)
    # request 0: negative, 2: too long for its row, 3: the free list ends in it
    got = attn.attn_block_tables(bt, _i32([-4, 5, 60, 0]), _i32([3, 4, 9, 40]), _i32([8, 9]), 16, 44)
    assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
    assert got[0].tolist() == [0, 9, 60, 40] and got[1].tolist() == [0, 0, 4, 4, 44] and got[4].item() == 2
    assert bt.tolist() == [[-1] * 4, [3, -1, -1, -1], [-1] * 4, [8, 9, -1, -1]]
    assert got[2][:4].tolist() == [3 * 16 + i for i in range(5, 9)]
    assert got[2][4:36].tolist() == list(range(128, 160)) and got[2][36:].tolist() == [-1] * 8
    # room for fewer tokens than there are
    got = attn.attn_block_tables(_i32(table), _i32([0] * 4), _i32([2] * 4), _i32(range(9)), 16, 5)
    assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
    assert got[2].tolist() == [0, 1, 16, 17, 32] and got[1].tolist() == [0, 2, 4, 6, 8]
    with pytest.raises(attn.AttnError, match="16384"):
        attn.attn_block_tables(_i32(np.zeros((16385, 1))), *(_i32(np.zeros(16385)),) * 2, _i32([1]), 16, 4)
    assert attn.attn_get_device_status() == 0


def _rope(n, rot):
    c, s = oracle.rope_table(n, rot)
    return torch.from_numpy(c).float().to(dev()), torch.from_numpy(s).float().to(dev())


def _step(attn, seed, old, new, page, H, H_kv, d, dtype):
    """Tables of a step and strided views of its fused projection rows."""
    table, free, num = _state(seed, old, new, page)
    bt = _i32(table)
    got = attn.attn_block_tables(bt, _i32(old), _i32(new), _i32(free), page, int(np.sum(new)))
    total = int(np.sum(new))
    rows = torch.from_numpy(workloads.normal(seed, (total, H + 2 * H_kv, d))).to(dev(), dtype)
    return bt, got, num, rows[:, :H], rows[:, H:H + H_kv], rows[:, H + H_kv:]


@pytest.mark.parametrize("d,rot,interleaved", [(64, 64, False), (128, 48, False), (128, 128, True), (256, 64, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append(attn, d, rot, interleaved, dtype):
    H, H_kv, page = 4, 2, 16
    bt, (lens, cu, slots, pos, _), num, q, k, v = _step(attn, 3, [0, 15, 16, 40], [20, 2, 0, 1], page, H, H_kv, d, dtype)
    cos, sin = _rope(64, rot)
    kc, c1 = guarded((num, page, H_kv, d), dtype, -7.0)
    vc, c2 = guarded((num, page, H_kv, d), dtype, -7.0)
    kc.copy_(torch.randn_like(kc.float()))
    vc.copy_(torch.randn_like(vc.float()))
    k0, v0 = kc.clone(), vc.clone()
    qo = attn.attn_cache_append(k, v, kc, vc, slots, cos, sin, pos, q=q, interleaved=interleaved)
    check_status(attn)
    c1()
    c2()
    want_q, want_k = attn.attn_rope(q, k, cos, sin, positions=pos, interleaved=interleaved)
    assert torch.equal(qo, want_q)
    k0.view(-1, H_kv, d)[slots] = want_k
    v0.view(-1, H_kv, d)[slots] = v
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    # without rotation, and without q
    assert attn.attn_cache_append(k, v, kc, vc, slots) is None
    k0.view(-1, H_kv, d)[slots] = k
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    check_status(attn)


def test_append_padding_bad_slots_and_nothing(attn):
    H_kv, d, page = 2, 64, 8
    k = torch.randn(5, H_kv, d, device=dev()).bfloat16()
    kc, c1 = guarded((3, page, H_kv, d), torch.bfloat16, -7.0)
    vc, c2 = guarded((3, page, H_kv, d), torch.bfloat16, -7.0)
    kc.zero_()
    vc.zero_()
    slots = torch.tensor([3, -1, 23, -1, 0], device=dev())
    attn.attn_cache_append(k, -k, kc, vc, slots)
    check_status(attn)
    want = torch.zeros(24, H_kv, d, device=dev()).bfloat16()
    want[[3, 23, 0]] = k[[0, 2, 4]]
    assert torch.equal(kc.view(24, H_kv, d), want) and torch.equal(vc.view(24, H_kv, d), -want)
    attn.attn_cache_append(k, -k, kc, vc, torch.tensor([24, -2, 2 ** 62, -1, -1], device=dev()))
    assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
    assert torch.equal(kc.view(24, H_kv, d), want)
    attn.attn_cache_append(k[:0], k[:0], kc, vc, slots[:0])
    check_status(attn)
    c1()
    c2()


def test_append_past_32_bit_offsets(attn):
    """A cache of more than 2^32 elements: its last and first rows."""
    H_kv, d, page = 8, 256, 256
    num = (1 << 32) // (page * H_kv * d) + 2
    kc = torch.empty(num, page, H_kv, d, dtype=torch.bfloat16, device=dev())
    vc = torch.empty_like(kc)
    kc[-1].zero_(), vc[-1].zero_(), kc[0].zero_(), vc[0].zero_()
    k, v = (torch.randn(2, H_kv, d, device=dev()).bfloat16() for _ in range(2))
    attn.attn_cache_append(k, v, kc, vc, torch.tensor([num * page - 1, 3], device=dev()))
    check_status(attn)
    assert torch.equal(kc[-1, -1], k[0]) and torch.equal(vc[-1, -1], v[0]) and torch.equal(kc[0, 3], k[1])
    assert not kc[-1, :-1].any() and not kc[0, 4:].any() and not kc[0, :3].any()


def _signs(d=128):
    return torch.from_numpy(workloads.random_signs(9, d)).to(dev())


def _random_cache(seed, num, page, H_kv):
    rng = np.random.default_rng(seed)
    codes = oracle.e4m3_encode(np.clip(rng.standard_normal((num, page, H_kv, 128)) * 100, -448, 448).astype(np.float32))
    return codes, rng.uniform(0.004, 0.01, (num, H_kv)).astype(np.float32)


@pytest.mark.parametrize("page", [16, 64, 256, 512])
@pytest.mark.parametrize("old,new", [([0], [1]), ([5, 0, 64, 130], [1, 1, 1, 1]), ([0, 15, 16, 250], [300, 2, 0, 700])])
@pytest.mark.parametrize("rot,signs", [(0, False), (128, False), (48, True), (0, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append_fp8(attn, page, old, new, rot, signs, dtype):
    H, H_kv, d = 4, 2, 128
    interleaved = rot == 48
    bt, (lens, cu, slots, pos, _), num, q, k, v = _step(attn, 5, old, new, page, H, H_kv, d, dtype)
    cos, sin = _rope(1000, rot) if rot else (None, None)
    sg = _signs() if signs else None
    caches = []
    for i in range(2):
        codes, desc = _random_cache(6 + i, num, page, H_kv)
        c, cc = guarded(codes.shape, torch.uint8, 0x5A)
        s, cs = guarded(desc.shape, torch.float32, -7.0)
        c.copy_(torch.from_numpy(codes))
        s.copy_(torch.from_numpy(desc))
        caches.append((c, s, cc, cs, codes, desc))
    (kc, ks, *_), (vc, vs, *_) = caches
    qo = attn.attn_cache_append_fp8(k, v, kc, vc, ks, vs, bt, lens, cu, rope_cos=cos, rope_sin=sin, hadamard_signs=sg,
                                    q=q if rot else None, interleaved=interleaved)
    check_status(attn)
    if rot:
        assert torch.equal(qo, attn.attn_rope(q, None, cos, sin, positions=pos, interleaved=interleaved)[0])
    at = slots.cpu().numpy()
    table = [None if t is None else t.cpu().numpy() for t in (cos, sin, sg)]
    rows = (oracle.key_rows(k.double().cpu().numpy(), pos.cpu().numpy(), *table[:2], interleaved, table[2]),
            v.double().cpu().numpy())
    for (c, s, cc, cs, codes, desc), x, plain in zip(caches, rows, (not rot and not signs, True)):
        cc()
        cs()
        got_c, got_s = c.cpu().numpy(), s.cpu().numpy()
        ref_c, ref_s = oracle.append_fp8(x, codes, desc, at)
        if plain:
            assert np.array_equal(got_c, ref_c) and np.array_equal(got_s, ref_s)
            continue
        assert np.all(np.abs(got_s - ref_s) <= 2.0 ** -19 * ref_s)
        untouched = np.setdiff1d(np.arange(num), at // page)
        assert np.array_equal(got_c[untouched], codes[untouched]) and np.array_equal(got_s[untouched], desc[untouched])
        # the new rows' values
        val = oracle.e4m3_decode(got_c.reshape(-1, H_kv, d)[at]) * got_s[at // page][:, :, None].astype(np.float64)
        size = np.linalg.norm(x, axis=2, keepdims=True)
        tol = np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * got_s[at // page][:, :, None]) * (1 + 2.0 ** -10) + 2.0 ** -19 * size
        assert np.all(np.abs(val - x) <= tol)
        # earlier rows: requantised by the ratio of the descales, exactly; cleared rests
        for p in np.unique(at // page):
            off = at[at // page == p] % page
            first, end = off.min(), off.max() + 1
            rest = codes[p].copy() if first else np.zeros_like(codes[p])
            for h in range(H_kv):
                if first and got_s[p, h] > desc[p, h]:
                    ratio = np.float32(desc[p, h] / got_s[p, h])
                    old_rows = oracle.e4m3_decode(codes[p, :first, h]).astype(np.float32)
                    rest[:first, h] = oracle.e4m3_encode((old_rows * ratio).astype(np.float32))
            assert np.array_equal(got_c[p, :first], rest[:first]) and np.array_equal(got_c[p, end:], rest[end:])


@pytest.mark.parametrize("signs", [False, True])
def test_append_fp8_of_whole_pages_is_the_prepass(attn, signs):
    """Pages of 128 tokens filled from their first row hold the pre-pass's codes and
    descales of the packed batch, bit for bit (rotation and transform included)."""
    H_kv, d, page, new = 2, 128, 128, [300, 128, 77]
    bt, (lens, cu, slots, pos, _), num, q, k, v = _step(attn, 8, [0, 0, 0], new, page, H_kv, H_kv, d, torch.bfloat16)
    cos, sin = _rope(300, d)
    sg = _signs() if signs else None
    kc, vc = (torch.empty(num, page, H_kv, d, dtype=torch.uint8, device=dev()) for _ in range(2))
    ks, vs = (torch.empty(num, H_kv, device=dev()) for _ in range(2))
    attn.attn_cache_append_fp8(k, v, kc, vc, ks, vs, bt, lens, cu, cos, sin, sg)
    (q8, k8, v8), (dq, dk, dv) = attn.attn_fp8_quantize_ex(q.contiguous(), k.contiguous(), v.contiguous(), cos, sin, sg,
                                                          cu_seqlens=cu, max_seqlen=300)
    check_status(attn)
    assert torch.equal(kc.view(-1, H_kv, d)[slots], k8) and torch.equal(vc.view(-1, H_kv, d)[slots], v8)
    for b, n in enumerate(new):
        for lp in range(-(-n // page)):
            assert torch.equal(ks[bt[b, lp]], dk[b, :, lp]) and torch.equal(vs[bt[b, lp]], dv[b, :, lp])


def test_append_fp8_zero_rows_and_bad_requests(attn):
    H_kv, d, page = 2, 128, 16
    kc, vc = (torch.full((4, page, H_kv, d), 0x33, dtype=torch.uint8, device=dev()) for _ in range(2))
    ks, vs = (torch.full((4, H_kv), 0.5, device=dev()) for _ in range(2))
    rows = torch.zeros(3, H_kv, d, device=dev()).half()
    call = lambda bt, lens, cu, r=rows: attn.attn_cache_append_fp8(r, r, kc, vc, ks, vs, _i32(bt), _i32(lens), _i32(cu))
    call([[2]], [3], [0, 3])
    check_status(attn)
    assert not kc[2].any() and torch.all(ks[2] == 1) and torch.all(ks[[0, 1, 3]] == 0.5)
    k0, s0 = kc.clone(), ks.clone()
    # a page outside the cache, more new tokens than the length, a length past the table's
    # row, offsets that decrease or pass the rows
    for bt, lens, cu in (([[4]], [3], [0, 3]), ([[-1]], [3], [0, 3]), ([[1]], [2], [0, 3]), ([[1]], [17], [0, 3]),
                         ([[1], [0]], [3, 3], [0, 5, 3]), ([[1]], [5], [0, 5]), ([[1]], [3], [-3, 0])):
        call(bt, lens, cu)
        assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG, (bt, lens, cu)
        assert torch.equal(kc, k0) and torch.equal(ks, s0)
    call([[1]], [3], [0, 0], rows[:0])
    check_status(attn)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("top", [1, 3, 60])
def test_append_fp8_of_a_batch_is_its_requests_one_by_one(attn, page, top):
    """Hundreds of requests, most with a token or none, some with up to `top` (8, 9 and 10 of one
    page, across a border, a whole page), whichever way the call takes them: the bytes of one
    call per request."""
    H_kv, d, B = 8, 128, 300
    rng = np.random.default_rng(80 + top)
    new = rng.integers(0, 2, B)
    for i in range(0, B, 7):
        new[i] = rng.integers(1, top + 1)
    if top > 8:
        new[1:6] = [8, 9, 10, page, page + 9]
    old = rng.integers(0, 3 * page, B)
    old[1:6] = [2 * page, page - 8, page - 9, 0, page - 9]
    bt, (lens, cu, slots, pos, _), num, _, k, v = _step(attn, 81, old.tolist(), new.tolist(), page, 1, H_kv, d, torch.bfloat16)
    cos, sin = _rope(1200, d)
    sg = _signs()
    state = (torch.randint(0, 0x7E, (num, page, H_kv, d), dtype=torch.uint8, device=dev()),
             torch.randint(0, 0x7E, (num, page, H_kv, d), dtype=torch.uint8, device=dev()),
             torch.rand(num, H_kv, device=dev()) * 0.02, torch.rand(num, H_kv, device=dev()) * 0.02)
    one = [t.clone() for t in state]
    all_ = [t.clone() for t in state]
    attn.attn_cache_append_fp8(k, v, *all_, bt, lens, cu, cos, sin, sg)
    check_status(attn)
    first = np.concatenate([[0], np.cumsum(new)])
    for b in range(B):
        n = int(new[b])
        if n:
            at = slice(first[b], first[b] + n)
            attn.attn_cache_append_fp8(k[at], v[at], *one, bt[b:b + 1], lens[b:b + 1], _i32([0, n]), cos, sin, sg)
    check_status(attn)
    for x, y, was in zip(all_, one, state):
        assert torch.equal(x, y) and not torch.equal(x, was)


@pytest.mark.parametrize("new", [[1, 0, 1], [40, 0, 9]])
def test_append_fp8_rows_behind_the_last_request(attn, new):
    """Padding behind cu_seqlens[B] (NaN): nothing of it is stored, its query rows are copied."""
    H, H_kv, d, page, pad = 4, 2, 128, 16, 7
    bt, (lens, cu, _, _, _), num, q, k, v = _step(attn, 12, [0, 5, 15], new, page, H, H_kv, d, torch.bfloat16)
    cos, sin = _rope(64, d)
    caches = []
    for rows in (0, pad):
        more = lambda t: torch.cat([t, torch.full((rows, *t.shape[1:]), float("nan"), device=dev(), dtype=t.dtype)])
        kc, vc = (torch.full((num, page, H_kv, d), 0x33, dtype=torch.uint8, device=dev()) for _ in range(2))
        ks, vs = (torch.full((num, H_kv), 0.5, device=dev()) for _ in range(2))
        qo = attn.attn_cache_append_fp8(more(k), more(v), kc, vc, ks, vs, bt, lens, cu, cos, sin, _signs(), q=more(q))
        check_status(attn)
        assert qo.shape[0] == sum(new) + rows and qo[sum(new):].isnan().all()
        caches.append((kc, vc, ks, vs, qo[:sum(new)]))
    assert all(torch.equal(a, b) for a, b in zip(*caches))


@pytest.mark.parametrize("fp8", [False, True])
def test_decoder_layer_steps(attn, fp8):
    """A prompt and decode steps of an encoder-decoder layer: tables, append with
    rotation, paged decode, cross attention, against the oracle's attention over the
    values the caches hold; the steps run from one captured graph."""
    H, H_kv, d, page, steps = 8, 2, 128, 16, 5
    prompt, enc = np.array([30, 1, 47]), [60, 0, 129]
    B, num, width = 3, 16, 6
    cos, sin = attn.attn_rope_table(64, d)
    sg = _signs() if fp8 else None
    free = np.random.default_rng(1).permutation(num).astype(np.int32)
    if fp8:
        kc, vc = (torch.full((num, page, H_kv, d), 0x7F, dtype=torch.uint8, device=dev()) for _ in range(2))
        ks, vs = (torch.full((num, H_kv), float("nan"), device=dev()) for _ in range(2))
    else:
        kc, vc = (torch.zeros(num, page, H_kv, d, device=dev()).bfloat16() for _ in range(2))
    ek, ev = (torch.from_numpy(workloads.normal(20 + i, (B, H_kv, 130, d))).to(dev(), torch.bfloat16) for i in range(2))
    elens = _i32(enc)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev())

    def append(q, k, v, lens, cu, slots, pos, q_out=None):
        if fp8:
            return attn.attn_cache_append_fp8(k, v, kc, vc, ks, vs, table, lens, cu, cos, sin, sg, q=q, q_out=q_out)
        return attn.attn_cache_append(k, v, kc, vc, slots, cos, sin, pos, q=q, q_out=q_out)

    def rows(seed, n):
        r = torch.from_numpy(workloads.normal(seed, (n, H + 2 * H_kv, d))).to(dev(), torch.bfloat16)
        return r[:, :H], r[:, H:H + H_kv], r[:, H + H_kv:]

    all_k, all_v = [[] for _ in range(B)], [[] for _ in range(B)]

    def remember(k, v, new):
        at = 0
        for b, n in enumerate(new):
            all_k[b].append(k[at:at + n].clone())
            all_v[b].append(v[at:at + n].clone())
            at += n

    total = int(prompt.sum())
    q, k, v = rows(30, total)
    zero = torch.zeros(B, dtype=torch.int32, device=dev())
    lens, cu, slots, pos, used = attn.attn_block_tables(table, zero, _i32(prompt), _i32(free), page, total)
    append(q, k, v, lens, cu, slots, pos)
    remember(k, v, prompt)
    taken = used.item()
    # one decode step, captured: static inputs, a padded slot map
    one = torch.ones(B, dtype=torch.int32, device=dev())
    old, free_now = lens.clone(), torch.zeros(num, dtype=torch.int32, device=dev())
    buf = torch.zeros(B, H + 2 * H_kv, d, device=dev()).bfloat16()
    q1, k1, v1 = buf[:, :H], buf[:, H:H + H_kv], buf[:, H + H_kv:]
    out = dict(lens=torch.empty_like(old), cu=torch.empty(B + 1, dtype=torch.int32, device=dev()),
               slots=torch.empty(B, dtype=torch.int64, device=dev()), pos=torch.empty_like(old), used=torch.empty_like(used))
    qr, o, co = (torch.empty(B, H, 1, d, device=dev()).bfloat16() for _ in range(3))
    lse, cl = (torch.empty(B, H, 1, device=dev()) for _ in range(2))
    ws = torch.empty(attn.attn_decode_workspace_size(B, H, H_kv, 1, d, width * page), dtype=torch.uint8, device=dev())
    cws = torch.empty(max(1, attn.attn_cross_workspace_size(B, H, H_kv, 1, 130, d)), dtype=torch.uint8, device=dev())

    def step():
        attn.attn_block_tables(table, old, one, free_now, page, B, seq_lens=out["lens"], cu_seqlens=out["cu"],
                               slots=out["slots"], positions=out["pos"], used=out["used"])
        append(q1, k1, v1, out["lens"], out["cu"], out["slots"], out["pos"], q_out=qr.view(B, H, d))
        if fp8:
            attn.attn_decode_paged_fp8(qr, kc, vc, ks, vs, table, out["lens"], width * page, hadamard_signs=sg, o=o, lse=lse,
                                       workspace=ws)
        else:
            attn.attn_decode_paged(qr, kc, vc, table, out["lens"], width * page, o=o, lse=lse, workspace=ws)
        attn.attn_cross_fwd(o, ek, ev, elens, o=co, lse=cl, workspace=cws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        a, b_, c = rows(40 + i, B)
        buf.copy_(torch.cat([a, b_, c], 1))
        free_now[:num - taken].copy_(torch.from_numpy(free[taken:]))
        graph.replay()
        check_status(attn)
        remember(b_, c, [1] * B)
        taken += out["used"].item()
        old.copy_(out["lens"])
        assert out["lens"].tolist() == (prompt + i + 1).tolist()
        assert sorted(x for x in table.flatten().tolist() if x >= 0) == sorted(free[:taken].tolist())
        # what the oracle makes of the same layer
        n = out["lens"].cpu().numpy()
        cs = cos.double().cpu().numpy(), sin.double().cpu().numpy()
        want_q = oracle.rope_rotate(a.double().cpu().numpy(), cs[0][n - 1][:, None], cs[1][n - 1][:, None])
        assert np.all(np.abs(qr.view(B, H, d).double().cpu().numpy() - want_q) <= 2.0 ** -8 * np.abs(want_q) + 1e-5)
        qq = qr.double().cpu().numpy()
        if fp8:
            # the caches' own values: half an e4m3 step for each time a page's descale grew
            ref, rl = oracle.attention_decode_paged_fp8(qq, kc.cpu().numpy(), vc.cpu().numpy(),
                                                        np.nan_to_num(ks.cpu().numpy(), nan=1.0),
                                                        np.nan_to_num(vs.cpu().numpy(), nan=1.0), table.cpu().numpy(), n,
                                                        d ** -0.5, True, signs=sg.cpu().numpy())
            rms = np.sqrt(np.mean((o.double().cpu().numpy() - ref) ** 2))
            assert rms <= 3e-2, rms
            for b in range(B):
                x = torch.cat(all_v[b]).double().cpu().numpy()
                p = table[b].cpu().numpy()
                val = np.concatenate([oracle.e4m3_decode(vc[j].cpu().numpy()) * vs[j].double().cpu().numpy()[None, :, None]
                                      for j in p[:-(-n[b] // page)]])[:n[b]]
                # at most one requantisation for each decode step after the prompt
                assert np.all(np.abs(val - x) <= (i + 2) * np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * 0.02) * 1.2)
        else:
            for b in range(B):
                kk = oracle.rope_rotate(torch.cat(all_k[b]).double().cpu().numpy(), cs[0][:n[b]][:, None], cs[1][:n[b]][:, None])
                kk = torch.from_numpy(kk).to(torch.bfloat16).double().numpy()
                vv = torch.cat(all_v[b]).double().cpu().numpy()
                r, rl = oracle.attention_cross_forward(qq[b:b + 1], kk.transpose(1, 0, 2)[None], vv.transpose(1, 0, 2)[None],
                                                       d ** -0.5)
                av, _ = oracle.attention_cross_forward(qq[b:b + 1], kk.transpose(1, 0, 2)[None],
                                                       np.abs(vv).transpose(1, 0, 2)[None], d ** -0.5)
                # P rounded to bfloat16, O rounded; keys that round the other way after the
                # rotation: one bfloat16 step of a key moves a score by 2^-8 |q k| <= 0.1 at most
                got = o[b].double().cpu().numpy()
                assert np.all(np.abs(got - r[0]) <= 2.0 ** -8 * 1.1 * (av[0] + np.abs(r[0])) + 0.02 * av[0])
                assert np.abs(lse[b].double().cpu().numpy() - rl[0]).max() <= LSE_ABS + 0.02
        cr, clr = oracle.attention_cross_forward(o.double().cpu().numpy(), ek.double().cpu().numpy(),
                                                 ev.double().cpu().numpy(), d ** -0.5, enc)
        ca, _ = oracle.attention_cross_forward(o.double().cpu().numpy(), ek.double().cpu().numpy(),
                                               np.abs(ev.double().cpu().numpy()), d ** -0.5, enc)
        assert np.all(np.abs(co.double().cpu().numpy() - cr) <= 2.0 ** -8 * 1.1 * (ca + np.abs(cr)) + 1e-6)
        assert torch.isneginf(cl[1]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_paged_decode_over_pages_never_cleared(attn, d, dtype):
    """Slots behind a sequence (rest of its last page, free pages) hold NaN and infinities:
    the decode's result is the one over clean pages, bit for bit."""
    lens, page = [1, 63, 64, 65, 129, 300], 64
    kc, vc, table = workloads.paged_cache(80, lens, page, 2, d)
    q = workloads.round_to(workloads.normal(81, (len(lens), 8, 1, d)), dtype).to(dev())
    outs = []
    for dirty in (False, True):
        k, v = (workloads.round_to(x, dtype).to(dev()) for x in (kc, vc))
        if dirty:
            used = torch.zeros(k.shape[:2], dtype=torch.bool)
            for b, n in enumerate(lens):
                for t in range(n):
                    used[table[b, t // page], t % page] = True
            k[~used.to(dev())] = float("nan")
            v[~used.to(dev())] = float("nan")
            v[~used.to(dev())][::2] = float("inf")
        outs.append(attn.attn_decode_paged(q, k, v, torch.from_numpy(table).to(dev()), _i32(lens), max(lens)))
        check_status(attn)
    assert torch.isfinite(outs[1][0].float()).all()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_training_layer(attn):
    """Rotation, causal attention and cross attention forward and backward, chained, against
    the oracle's chain (gradient tolerance of the attention tests)."""
    from gpu_util import GRAD_REL_RMSE, rel_rmse
    B, H, N, N_k, d = 1, 2, 150, 90, 64
    q, k, v, do = (workloads.round_to(x, "bf16") for x in workloads.normal(70, (B, H, N, d), 4))
    ek, ev = (workloads.round_to(x, "bf16") for x in workloads.normal(71, (B, H, N_k, d), 2))
    g = [t.to(dev()) for t in (q, k, v, do, ek, ev)]
    cos, sin = attn.attn_rope_table(N, d)
    lens = _i32([80])
    qr, kr = attn.attn_rope(g[0], g[1], cos, sin)
    o1, l1 = attn.attn_fwd(qr, kr, g[2], causal=True)
    o2, l2 = attn.attn_cross_fwd(o1, g[4], g[5], lens)
    do1, dek, dev_ = attn.attn_cross_bwd(o1, g[4], g[5], o2, g[3], l2, lens)
    dqr, dkr, dv = attn.attn_bwd(qr, kr, g[2], o1, do1, l1, causal=True)
    dq, dk = attn.attn_rope(dqr, dkr, cos, sin, inverse=True)
    check_status(attn)
    c, s = cos.double().cpu().numpy(), sin.double().cpu().numpy()
    f = [workloads.as_f64(t) for t in (q, k, v, do, ek, ev)]
    scale = d ** -0.5
    rq, rk = oracle.rope_rotate(f[0], c, s), oracle.rope_rotate(f[1], c, s)
    ro1, _ = oracle.attention_forward(rq, rk, f[2], scale, True)
    e1, e2, e3 = oracle.attention_cross_backward(ro1, f[4], f[5], f[3], scale, [80])
    a1, a2, a3 = oracle.attention_backward(rq, rk, f[2], e1, scale, True)
    refs = (oracle.rope_rotate(a1, c, s, inverse=True), oracle.rope_rotate(a2, c, s, inverse=True), a3, e2, e3)
    # each link rounds its inputs to bfloat16 once more: four roundings' worth
    for x, r in zip((dq, dk, dv, dek, dev_), refs):
        assert rel_rmse(x, r) <= 4 * GRAD_REL_RMSE


def test_dimensions_past_32_bits_are_refused(attn):
    """Found only when the call's arguments are narrowed: a ValueError, and the interpreter goes on."""
    k = torch.zeros(1, 2, 128, device=dev()).bfloat16()
    kc = torch.empty(2 ** 31, 0, 2, 128, dtype=torch.bfloat16, device=dev())
    slots = torch.zeros(1, dtype=torch.int64, device=dev())
    with pytest.raises(ValueError, match="dimension"):
        attn.attn_cache_append(k, k, kc, kc, slots)
    desc = torch.empty(1, 0, device=dev())
    kc8 = torch.empty(1, 2 ** 31, 0, 128, dtype=torch.uint8, device=dev())
    none = torch.empty(1, 0, 128, device=dev()).bfloat16()
    with pytest.raises(ValueError, match="dimension"):
        attn.attn_cache_append_fp8(none, none, kc8, kc8, desc, desc, _i32([[0]]), _i32([1]), _i32([0, 1]))
    check_status(attn)


@pytest.mark.parametrize("size", [1e-24, 1e-30, 1e-37, 2e-40])
@pytest.mark.parametrize("new", [[1, 3, 0, 2], [300, 5, 70, 16]])
@pytest.mark.parametrize("signs", [False, True])
def test_append_fp8_tiny_values(attn, size, new, signs):
    """bfloat16 rows down to subnormal ones, zeros among them, on fresh pages and behind old
    tokens: codes and descales of the rule (2^-90 at least), exact without the transform up to the
    sign of zeros, and a decode over them that stays finite."""
    H, H_kv, d, page = 4, 2, 128, 64
    old = [0, 0, 30, 64]
    bt, (lens, cu, slots, _, _), num, q, k, v = _step(attn, 90, old, new, page, H, H_kv, d, torch.bfloat16)
    k, v = ((t.double() * size).bfloat16() for t in (k, v))
    k[::2, :, 5], v[1::3] = 0, 0
    assert k.any() and v.any()
    at, sg = slots.cpu().numpy(), _signs() if signs else None
    rows = (oracle.key_rows(k.double().cpu().numpy(), None, None, None, False, sg.cpu().numpy() if signs else None),
            v.double().cpu().numpy())
    # old tokens of one request as tiny, of the other of ordinary size
    tiny = np.float32(size)
    state = []
    for i, x in enumerate(rows):
        codes, desc = _random_cache(91 + i, num, page, H_kv)
        if new[2]:
            desc[bt[2, 0].item()] = tiny
        c, s = torch.from_numpy(codes).to(dev()), torch.from_numpy(desc).to(dev())
        state.append((c, s, *oracle.append_fp8(x, codes, desc, at), x, codes))
    (kc, ks, *_), (vc, vs, *_) = state
    attn.attn_cache_append_fp8(k, v, kc, vc, ks, vs, bt, lens, cu, hadamard_signs=sg)
    check_status(attn)
    for (c, s, ref_c, ref_s, x, codes), plain in zip(state, (not signs, True)):
        got_c, got_s = c.cpu().numpy(), s.cpu().numpy()
        if plain:
            assert np.array_equal(oracle.e4m3_decode(got_c), oracle.e4m3_decode(ref_c)) and np.array_equal(got_s, ref_s)
            continue
        # as in test_append_fp8: float32 rows off by 2^-20 of their length, and 2^-140 where subnormal
        assert np.all(np.abs(got_s - ref_s) <= 2.0 ** -19 * ref_s)
        val = oracle.e4m3_decode(got_c.reshape(-1, H_kv, d)[at]) * got_s[at // page][:, :, None].astype(np.float64)
        length = np.linalg.norm(x, axis=2, keepdims=True)
        tol = np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * got_s[at // page][:, :, None]) * (1 + 2.0 ** -10)
        assert np.all(np.abs(val - x) <= tol + 2.0 ** -19 * length + 2.0 ** -140)
    o, lse = attn.attn_decode_paged_fp8(q[:4].reshape(4, H, 1, d).contiguous(), kc, vc, ks, vs, bt, lens, int(lens.max()),
                                        hadamard_signs=sg)
    check_status(attn)
    seen = lens.cpu().numpy() > 0
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse[torch.from_numpy(seen).to(dev())]).all()
    for p in np.unique(at // page):
        assert not np.isnan(oracle.e4m3_decode(kc[p].cpu().numpy())).any()


def test_tables_report_tokens_on_missing_pages(attn):
    """After a step that ran out of pages: its seq_lens fed back with new pages at hand put the next
    tokens on the page that was never given; a negative free page does so too.  Slots -1, reported;
    with the placed lengths fed back everything fits."""
    bt = _i32([[3, -1, -1, -1], [-1, -1, -1, -1]])
    lens, *_ = attn.attn_block_tables(bt, _i32([10, 0]), _i32([10, 20]), _i32([5]), 16, 30)
    assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
    assert bt.tolist() == [[3, 5, -1, -1], [-1, -1, -1, -1]] and lens.tolist() == [20, 20]
    again = bt.clone()
    _, _, slots, pos, used = attn.attn_block_tables(again, lens, _i32([1, 1]), _i32([7, 8]), 16, 2)
    assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
    assert slots.tolist() == [5 * 16 + 4, -1] and pos.tolist() == [20, 20] and used.item() == 0
    _, _, slots, _, used = attn.attn_block_tables(bt, _i32([20, 0]), _i32([1, 20]), _i32([7, 8]), 16, 21)
    check_status(attn)
    assert slots.tolist() == [84] + list(range(7 * 16, 8 * 16)) + list(range(8 * 16, 8 * 16 + 4)) and used.item() == 2
    _, _, slots, _, used = attn.attn_block_tables(_i32([[-1, -1]]), _i32([0]), _i32([17]), _i32([4, -6]), 16, 17)
    assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
    assert slots.tolist() == list(range(64, 80)) + [-1] and used.item() == 2
    # a missing page that no new token stands on is the reader's to report
    attn.attn_block_tables(_i32([[-1, 6, -1]]), _i32([20]), _i32([1]), _i32([1]), 16, 1)
    check_status(attn)


@pytest.mark.parametrize("B,top", [(3, 200), (64, 64), (64, 640), (300, 300), (9, 2000)])
def test_append_fp8_decreasing_offsets_are_reported(attn, B, top):
    """Offsets that rise to `top` and start again from 0, far enough that no unit of the launch
    falls to the request between: reported, and nothing outside the requests' pages is written."""
    H_kv, d, page = 2, 128, 16
    rows = torch.randn(top, H_kv, d, device=dev()).half()
    cu = [0, top] + [min(i, top) for i in range(B - 1)]
    lens = [top] + [0] + [1] * (B - 2)
    width = -(-top // page)
    bt = torch.arange(B * width, dtype=torch.int32, device=dev()).view(B, width)
    kc, ck = guarded((B * width, page, H_kv, d), torch.uint8, 0x5A)
    vc, cv = guarded((B * width, page, H_kv, d), torch.uint8, 0x5A)
    ks, vs = (torch.ones(B * width, H_kv, device=dev()) for _ in range(2))
    attn.attn_cache_append_fp8(rows, rows, kc, vc, ks, vs, bt, _i32(lens), _i32(cu))
    assert attn.attn_get_device_status() == attn.ATTN_ERR_INVALID_ARG
    ck()
    cv()


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_of_positions_past_the_tables(attn, interleaved):
    """Reported; the rows are written unrotated, as is padding of a negative position, which is not."""
    H, H_kv, d, page = 2, 2, 64, 8
    cos, sin = _rope(8, d)
    rows = torch.randn(4, H + 2 * H_kv, d, device=dev()).bfloat16()
    q, k, v = rows[:, :H], rows[:, H:H + H_kv], rows[:, H + H_kv:]
    slots = torch.tensor([5, 0, 9, 15], device=dev())
    for last, code in ((-1, 0), (8, attn.ATTN_ERR_INVALID_ARG), (2 ** 31 - 1, attn.ATTN_ERR_INVALID_ARG)):
        kc, vc = (torch.zeros(2, page, H_kv, d, device=dev()).bfloat16() for _ in range(2))
        qo = attn.attn_cache_append(k, v, kc, vc, slots, cos, sin, _i32([0, 7, 3, last]), q=q, interleaved=interleaved)
        assert attn.attn_get_device_status() == code
        if code:
            assert "unrotated" in attn.attn_last_error()
        wq, wk = attn.attn_rope(q[:3], k[:3], cos, sin, positions=_i32([0, 7, 3]), interleaved=interleaved)
        want, val = torch.zeros_like(kc), torch.zeros_like(vc)
        want.view(-1, H_kv, d)[slots] = torch.cat([wk, k[3:]])
        val.view(-1, H_kv, d)[slots] = v
        assert torch.equal(kc, want) and torch.equal(vc, val) and torch.equal(qo, torch.cat([wq, q[3:]]))
    check_status(attn)


@pytest.mark.parametrize("rot,interleaved", [(128, False), (48, False), (128, True)])
@pytest.mark.parametrize("new", [4, 60])
def test_append_fp8_of_positions_past_the_tables(attn, new, rot, interleaved):
    """The codes, descales and queries of tables whose missing rows turn nothing; reported."""
    H, H_kv, d, page, old = 4, 2, 128, 64, 6
    bt, (lens, cu, *_), num, q, k, v = _step(attn, 95, [old], [new], page, H, H_kv, d, torch.bfloat16)
    rows = old + new - 2                              # the last two positions have none
    cos, sin = _rope(rows, rot)
    one, zero = torch.ones(2, rot // 2, device=dev()), torch.zeros(2, rot // 2, device=dev())
    got = []
    for c, s, code in ((cos, sin, attn.ATTN_ERR_INVALID_ARG), (torch.cat([cos, one]), torch.cat([sin, zero]), 0)):
        kc, vc = (torch.full((num, page, H_kv, d), 0x35, dtype=torch.uint8, device=dev()) for _ in range(2))
        ks, vs = (torch.full((num, H_kv), 0.004, device=dev()) for _ in range(2))
        qo = attn.attn_cache_append_fp8(k, v, kc, vc, ks, vs, bt, lens, cu, c, s, _signs(), q=q, interleaved=interleaved)
        assert attn.attn_get_device_status() == code
        got.append((kc, vc, ks, vs, qo))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dirt", [float("inf"), float("-inf")])
def test_paged_decode_over_pages_of_infinities(attn, d, dtype, dirt):
    """Infinities in every slot behind a sequence, in keys and values: the bits of clean pages."""
    lens, page = [1, 63, 64, 65, 129, 300], 64
    kc, vc, table = workloads.paged_cache(82, lens, page, 2, d)
    q = workloads.round_to(workloads.normal(83, (len(lens), 8, 1, d)), dtype).to(dev())
    unused = torch.ones(kc.shape[:2], dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            unused[table[b, t // page], t % page] = False
    outs = []
    for fill in (0.0, dirt):
        k, v = (workloads.round_to(x, dtype).to(dev()) for x in (kc, vc))
        k[unused.to(dev())] = fill
        v[unused.to(dev())] = fill
        assert fill == 0.0 or (torch.isinf(v).any() and torch.isinf(k).any())
        outs.append(attn.attn_decode_paged(q, k, v, torch.from_numpy(table).to(dev()), _i32(lens), max(lens)))
        check_status(attn)
    assert torch.isfinite(outs[1][0].float()).all()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
