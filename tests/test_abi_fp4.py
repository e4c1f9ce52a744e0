"""Host-side refusals of the 4-bit cache's entry points, of reading a cache back and of merging:
every bad argument is turned away before anything is launched."""
import ctypes

import pytest

S2 = ctypes.c_longlong * 2


@pytest.fixture(scope="module")
def lib():
    from exact_tiled_attention_25_gb300 import build, _lib
    build.build()
    return _lib.load()


def _append(lib, q=16, qo=16, k=16, v=16, kc=16, vc=16, kd=16, vd=16, slots=16, c=16, s=16, pos=16, sg=16, total=4, H=2,
            Hkv=1, d=128, rot=64, mp=8, pages=4, ps=16, qs=None, ks=None, vs=None, il=0, dt=0):
    return lib.attn_cache_append_fp4(q, qo, k, v, kc, vc, kd, vd, slots, c, s, pos, sg, total, H, Hkv, d, rot, mp, pages, ps,
                                     qs, ks, vs, il, dt, None)


@pytest.mark.parametrize("kwargs,why", [
    (dict(ps=8), "page_size"), (dict(ps=48), "page_size"), (dict(ps=1 << 17), "page_size"), (dict(total=-1), "total"),
    (dict(pages=0), "num_pages"), (dict(d=96), "d must"), (dict(rot=40), "rot_dim"), (dict(rot=144), "rot_dim"),
    (dict(s=0), "both"), (dict(c=0, s=0), "needs rope_cos"), (dict(k=0), "null"), (dict(kc=8), "aligned"), (dict(vd=0), "null"),
    (dict(kd=8), "aligned"), (dict(qo=0), "null"), (dict(ks=S2(64, 4)), "strides"), (dict(vs=S2(-64, 64)), "strides"),
    (dict(il=3), "interleaved"), (dict(dt=5), "dtype"), (dict(total=1 << 28), "2^31"), (dict(slots=4), "slots"),
    (dict(slots=0), "slots"), (dict(pos=0), "integer"), (dict(sg=4), "hadamard"), (dict(Hkv=0), "H_kv"), (dict(mp=0), "max_pos"),
])
def test_append_refusals(lib, kwargs, why):
    assert _append(lib, **kwargs) == 1
    assert why in lib.attn_last_error().decode()


def test_unsupported_head_sizes(lib):
    assert _append(lib, d=256) == 2 and _decode(lib, d=256) == 2 and _decode(lib, d=96) == 2
    assert _read(lib, 4, d=256) == 2 and _read(lib, 8, d=64) == 2


def _decode(lib, q=16, kc=32, vc=64, kd=16, vd=16, sg=16, bt=16, sl=16, o=16, l=16, ws=256, wsb=1 << 40, B=2, H=8, Hkv=2, nq=1,
            d=128, pages=9, ps=16, maxp=4, ms=64, causal=1, scale=0.1, dt=0):
    return lib.attn_decode_paged_fp4(q, kc, vc, kd, vd, sg, bt, sl, o, l, ws, wsb, B, H, Hkv, nq, d, pages, ps, maxp, ms, causal,
                                     scale, dt, None)


@pytest.mark.parametrize("kwargs,why", [
    (dict(B=0), "B"), (dict(H=0), "H"), (dict(nq=0), "n_q"), (dict(ms=0), "max_seqlen"), (dict(Hkv=3), "H_kv"), (dict(Hkv=0), "H_kv"),
    (dict(ps=8), "page_size"), (dict(ps=24), "page_size"), (dict(maxp=0), "max_pages"), (dict(maxp=1 << 28), "max_pages"),
    (dict(pages=2 ** 31 - 1, ps=65536, maxp=4, Hkv=8), "too large"), (dict(causal=2), "causal"), (dict(scale=0.0), "scale"),
    (dict(scale=float("inf")), "scale"), (dict(dt=2), "dtype"), (dict(q=0), "null"), (dict(kc=8), "aligned"), (dict(vc=48), "32-byte"), (dict(kd=0), "null"),
    (dict(sg=8), "hadamard"), (dict(bt=0), "integer"), (dict(sl=2), "integer"), (dict(ws=16), "256-byte"), (dict(ws=0), "null"),
    (dict(wsb=16), "workspace"), (dict(B=1 << 28), "2^31"),
])
def test_decode_refusals(lib, kwargs, why):
    assert _decode(lib, **kwargs) == 1
    assert why in lib.attn_last_error().decode()


def test_decode_row_limit_and_workspace(lib):
    assert _decode(lib, H=64, Hkv=1, nq=3) == 2 and b"128" in lib.attn_last_error()
    assert _decode(lib, H=2, Hkv=1, nq=2 ** 31 - 1) == 2
    assert _decode(lib, B=1 << 15, H=8, Hkv=8, maxp=1 << 17, ps=16) == 2 and b"2^31" in lib.attn_last_error()
    size = lib.attn_decode_fp4_workspace_size
    assert size(1, 8, 3, 1, 128, 100) == 0 and size(0, 8, 2, 1, 128, 100) == 0 and size(1, 8, 2, 33, 128, 100) == 0
    need = size(2, 8, 2, 1, 128, 64)
    assert need > 0 and _decode(lib, wsb=need - 1) == 1 and b"workspace" in lib.attn_last_error()
    # bounded by the machine, not by the batch or the context
    assert size(4000, 64, 8, 2, 128, 1 << 20) <= 152 * 4 * (2 * 16 * 129 * 4 + 16) + 3 * 256


def _read(lib, bits, kc=16, vc=16, kd=16, vd=16, sg=16, bt=16, sl=16, first=16, cu=16, ko=16, vo=16, B=2, n=10, Hkv=2, d=128,
          pages=9, ps=16, maxp=4, dt=0):
    tail = (bt, sl, first, cu, ko, vo, B, n, Hkv, d, pages, ps, maxp, dt, None)
    if bits == 16:
        return lib.attn_cache_read(kc, vc, *tail)
    call = lib.attn_cache_read_fp8 if bits == 8 else lib.attn_cache_read_fp4
    return call(kc, vc, kd, vd, sg, *tail)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("kwargs,why", [
    (dict(B=0), "B"), (dict(n=-1), "n must"), (dict(Hkv=0), "H_kv"), (dict(d=80), "d must"), (dict(ps=4), "page_size"),
    (dict(pages=0), "num_pages"), (dict(maxp=1 << 28), "max_pages"), (dict(kc=0), "null"), (dict(vo=8), "aligned"), (dict(ko=0), "null"),
    (dict(bt=0), "integer"), (dict(sl=0), "integer"), (dict(first=2), "integer"), (dict(cu=2), "integer"), (dict(dt=7), "dtype"),
])
def test_read_refusals(lib, bits, kwargs, why):
    assert _read(lib, bits, **kwargs) == 1
    assert why in lib.attn_last_error().decode()


def test_read_refusals_of_quantised_caches(lib):
    for bits in (8, 4):
        assert _read(lib, bits, kd=0) == 1 and _read(lib, bits, vd=8) == 1 and _read(lib, bits, sg=8) == 1
        assert b"hadamard" in lib.attn_last_error()
        assert _read(lib, bits, ps=8) == 1 and b"page_size" in lib.attn_last_error()


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_read_refuses_outputs_that_overlap(lib, bits):
    """Each other or an input, in part too: blocks read while others write.  (Sizes: caches of 9 x 16 x 2
    rows, outputs of 2 x 2 x 10 rows of 256 bytes, 10 x 2 rows packed.)"""
    far = dict(kc=1 << 20, vc=2 << 20, kd=3 << 20, vd=4 << 20, sg=5 << 20, bt=6 << 20, sl=7 << 20, first=8 << 20, cu=0,
               ko=10 << 20, vo=11 << 20)
    cache = 9 * 16 * 2 * 128 * bits // 8
    out = 2 * 2 * 10 * 256
    cases = [dict(ko=far["vo"]), dict(ko=far["vo"] - out + 16), dict(vo=far["ko"] + out - 16), dict(ko=far["kc"]),
             dict(vo=far["kc"] + cache - 16), dict(ko=far["vc"] - out + 16), dict(vo=far["vc"] + 4096), dict(ko=far["bt"] + 16),
             dict(vo=far["bt"] - out + 16), dict(ko=far["sl"]), dict(vo=far["first"] - 16),
             dict(cu=9 << 20, ko=9 << 20), dict(cu=9 << 20, vo=(9 << 20) - out // 2 + 16)]
    if bits < 16:
        scales = 9 * 2 * 4 if bits == 8 else 9 * 16 * 2 * 2
        cases += [dict(ko=far["kd"] + (scales - 1) // 16 * 16), dict(vo=far["vd"] - 16), dict(ko=far["sg"] + 496)]
    for case in cases:
        assert _read(lib, bits, **{**far, **case}) == 1, case
        assert "overlap" in lib.attn_last_error().decode(), case


def _merge(lib, oa=0x10000, la=0x20000, ob=0x30000, lb=0x40000, o=0x50000, l=0x60000, B=1, H=2, N=8, d=128, packed=0, dt=0):
    return lib.attn_merge(oa, la, ob, lb, o, l, B, H, N, d, packed, dt, None)


@pytest.mark.parametrize("kwargs,why", [
    (dict(B=0), "B"), (dict(N=0), "N"), (dict(d=96), "d must"), (dict(packed=2), "packed"), (dict(packed=1, B=2), "packed"),
    (dict(dt=3), "dtype"), (dict(oa=0), "null"), (dict(lb=8), "aligned"), (dict(N=1 << 24), "2^31"),
    (dict(o=0x10010), "overlap"), (dict(o=0x20000), "overlap"), (dict(l=0x10000), "overlap"), (dict(l=0x40010), "overlap"),
    (dict(l=0x50010), "overlap"), (dict(o=0x30000 - 0x800), "overlap"),
])
def test_merge_refusals(lib, kwargs, why):
    assert _merge(lib, **kwargs) == 1
    assert why in lib.attn_last_error().decode()


def test_python_refusals():
    """Shapes and types that the binding turns away by itself, before it looks for a device."""
    import torch
    import exact_tiled_attention_25_gb300 as attn
    nat = attn._binding()
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    rows = torch.zeros(4, 2, 64, **bf)
    kc, kd = torch.zeros(3, 2, 16, 32, dtype=torch.uint8), torch.zeros(3, 2, 16, **bf)
    slots, tab = torch.zeros(4, dtype=torch.int64), torch.zeros(8, 32)

    def append(k=rows, v=rows, kc=kc, vc=kc, kd=kd, vd=kd, slots=slots, cos=None, sin=None, pos=None, sg=None, q=None, qo=None):
        nat.cache_append_fp4(k, v, kc, vc, kd, vd, slots, cos, sin, pos, sg, q, False, qo, None)

    for kw, why in ((dict(kc=kc[:, :1]), "caches"), (dict(kc=kc.transpose(1, 2)), "caches"), (dict(kc=kd), "caches"),
                    (dict(vc=kc.view(torch.int8)), "v_cache"), (dict(kd=kd.float()), "k_descale"), (dict(vd=kd[:, :, :8]), "v_descale"),
                    (dict(v=rows[:, :1]), "k and v"), (dict(k=rows.float(), v=rows.float()), "k and v"), (dict(slots=slots.int()), "slots"),
                    (dict(cos=tab, sin=tab), "positions"), (dict(cos=tab), "both"), (dict(sg=torch.ones(128)), "hadamard_signs"),
                    (dict(qo=rows), "q_out"), (dict(q=rows[:3]), "q must be"), (dict(), "current CUDA device")):
        with pytest.raises(ValueError, match=why):
            append(**kw)
    q, bt, lens = torch.zeros(2, 4, 1, 64, **bf), torch.zeros(2, 3, **i32), torch.zeros(2, **i32)

    def decode(q=q, kc=kc, vc=kc, kd=kd, vd=kd, bt=bt, lens=lens, sg=None, most=16):
        nat.decode_paged_fp4(q, kc, vc, kd, vd, bt, lens, sg, most, True, None, None, None, None, None)

    for kw, why in ((dict(q=q.float()), "q must be"), (dict(q=q[0]), "q must be"), (dict(q=torch.zeros(2, 4, 3, 64, **bf).transpose(1, 2)), "contiguous"),
                    (dict(q=torch.zeros(2, 4, 1, 128, **bf)), "share d"), (dict(bt=bt[:1]), "block_table"), (dict(lens=lens.long()), "seq_lens"),
                    (dict(sg=torch.ones(32)), "hadamard"), (dict(most=2 ** 40), "max_seqlen"), (dict(kd=None), "k_descale is missing"),
                    (dict(), "current CUDA device")):
        with pytest.raises(ValueError, match=why):
            decode(**kw)
    wide = torch.zeros(3, 16, 2, 64, **bf)

    def read(bits=4, kc=kc, vc=kc, kd=kd, vd=kd, sg=None, bt=bt, lens=lens, n=4, first=None, cu=None, k=None, v=None):
        nat.cache_read(bits, kc, vc, kd, vd, sg, bt, lens, n, first, cu, k, v, False, None)

    for kw, why in ((dict(kd=None), "k_descale"), (dict(bits=16, kc=kc, vc=kc), "caches must be"), (dict(bits=16, kc=wide, vc=wide.half()), "v_cache"),
                    (dict(bits=8, kc=wide.byte(), vc=wide.byte()), "k_descale"), (dict(n=-1), "n must"), (dict(bt=bt[0]), "block_table"),
                    (dict(lens=lens[:1]), "seq_lens"), (dict(first=lens.long()), "first"), (dict(cu=lens), "cu_seqlens"),
                    (dict(sg=torch.ones(32)), "hadamard"), (dict(), "current CUDA device")):
        with pytest.raises(ValueError, match=why):
            read(**kw)
    with pytest.raises(ValueError, match="dtype"):
        attn.attn_cache_read_fp4(kc, kc, kd, kd, bt, lens, 4, dtype=torch.float32)
    o, lse = torch.zeros(1, 2, 3, 64, **bf), torch.zeros(1, 2, 3)
    for args, why in (((o.float(), lse, o.float(), lse), "float16"), ((o[0, 0], lse, o, lse), "packed"), ((o, lse, o.half(), lse), "o_b"),
                      ((o, lse[0], o, lse), "lse_a"), ((o[0], lse[0], o[0], lse[0]), "lse_a"), ((o, lse, o, lse.double()), "lse_b"),
                      ((o.transpose(1, 2), lse, o, lse), "o_a"), ((o, lse, o, lse), "current CUDA device")):
        with pytest.raises(ValueError, match=why):
            nat.merge(*args, None, None, None)
    with pytest.raises(TypeError, match="expected 7 arguments"):
        nat.merge(o)
