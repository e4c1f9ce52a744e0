"""Host-side refusals of the cross-attention, rotary and cache entry points: every
bad argument is turned away before anything is launched."""
import ctypes

import pytest

S3, S2 = ctypes.c_longlong * 3, ctypes.c_longlong * 2


@pytest.fixture(scope="module")
def lib():
    from exact_tiled_attention_25_gb300 import build, _lib
    build.build()
    return _lib.load()


def _cross_fwd(lib, q=16, k=16, v=16, lens=None, o=16, l=16, ws=256, wsb=1 << 40, B=1, H=4, Hkv=2, Nq=300, Nk=200,
               d=128, scale=0.1, dt=0):
    return lib.attn_cross_fwd(q, k, v, lens, o, l, ws, wsb, B, H, Hkv, Nq, Nk, d, scale, dt, None)


def _cross_bwd(lib, q=16, k=16, v=16, o=16, do=16, l=16, lens=None, dq=16, dk=16, dv=16, ws=256, wsb=1 << 40, B=1, H=4,
               Hkv=2, Nq=300, Nk=200, d=128, scale=0.1, dt=0):
    return lib.attn_cross_bwd(q, k, v, o, do, l, lens, dq, dk, dv, ws, wsb, B, H, Hkv, Nq, Nk, d, scale, dt, None)


CROSS = [(dict(Nk=0), "N_k"), (dict(Nq=0), "N"), (dict(d=96), "d must"), (dict(Hkv=3), "H_kv"),
         (dict(scale=0.0), "scale"), (dict(scale=float("nan")), "scale"), (dict(dt=2), "dtype"), (dict(k=0), "null"),
         (dict(q=8), "aligned"), (dict(lens=2), "kv_lens"), (dict(Nk=1 << 24), "2^31")]


@pytest.mark.parametrize("call", [_cross_fwd, _cross_bwd])
@pytest.mark.parametrize("kwargs,why", CROSS)
def test_cross_refusals(lib, call, kwargs, why):
    assert call(lib, **kwargs) == 1
    assert why in lib.attn_last_error().decode()


def test_cross_workspaces(lib):
    assert lib.attn_cross_workspace_size(1, 3, 2, 1, 10, 64) == 0          # H_kv does not divide H
    need = lib.attn_cross_workspace_size(1, 4, 2, 1, 8192, 128)
    assert need > 0
    few = dict(Nq=1, Nk=8192)
    assert _cross_fwd(lib, wsb=need - 1, **few) == 1 and b"workspace" in lib.attn_last_error()
    assert _cross_fwd(lib, ws=None, **few) == 1 and b"workspace" in lib.attn_last_error()
    assert _cross_fwd(lib, ws=16, **few) == 1 and b"256-byte" in lib.attn_last_error()
    need = lib.attn_cross_bwd_workspace_size(1, 4, 300, 200, 128)
    assert need > lib.attn_bwd_workspace_size(1, 4, 300, 128)
    assert lib.attn_cross_bwd_workspace_size(1, 4, 0, 200, 128) == 0
    assert _cross_bwd(lib, wsb=need - 1) == 1 and b"workspace" in lib.attn_last_error()
    assert _cross_bwd(lib, ws=16) == 1 and b"256-byte" in lib.attn_last_error()
    assert _cross_bwd(lib, d=256) == 2
    assert _cross_fwd(lib, B=65536, H=1, Hkv=1, Nq=1, Nk=1, d=64) == 2


def _rope(lib, q=16, qo=16, k=16, ko=16, c=16, s=16, pos=None, B=1, N=4, H=2, Hkv=1, d=64, rot=64, mp=8, st=None,
          ot=None, il=0, inv=0, dt=0):
    return lib.attn_rope(q, qo, k, ko, c, s, pos, B, N, H, Hkv, d, rot, mp, st, ot, None, None, il, inv, dt, None)


@pytest.mark.parametrize("kwargs,why", [
    (dict(rot=24), "rot_dim"), (dict(rot=80), "rot_dim"), (dict(rot=0), "rot_dim"), (dict(mp=0), "max_pos"),
    (dict(il=2), "interleaved"), (dict(inv=2), "inverse"), (dict(dt=3), "dtype"), (dict(q=0), "null"),
    (dict(c=0), "null"), (dict(ko=0), "null"), (dict(k=4), "aligned"), (dict(pos=2), "positions"),
    (dict(N=0), "N"), (dict(d=80), "d must"), (dict(Hkv=-1), "H_kv"),
    (dict(st=S3(64, 64, 60)), "strides"), (dict(st=S3(64, -64, 64)), "strides"), (dict(ot=S3(64, 64, 0)), "strides"),
])
def test_rope_refusals(lib, kwargs, why):
    assert _rope(lib, **kwargs) == 1
    assert why in lib.attn_last_error().decode()


def _table(lib, c=16, s=16, n=8, rot=64, base=1e4, f=1.0, ol=0, lo=1.0, hi=32.0, af=1.0, first=0):
    return lib.attn_rope_table(c, s, n, rot, base, f, ol, lo, hi, af, first, None)


@pytest.mark.parametrize("kwargs,why", [
    (dict(n=0), "positions"), (dict(first=-1), "positions"), (dict(first=2 ** 31 - 4, n=8), "positions"),
    (dict(rot=8), "rot_dim"), (dict(rot=272), "rot_dim"), (dict(base=1.0), "base"), (dict(base=float("inf")), "base"),
    (dict(f=0.5), "factor"), (dict(f=float("nan")), "factor"), (dict(ol=-1), "orig_len"),
    (dict(ol=10, lo=2.0, hi=2.0), "low"), (dict(ol=10, lo=-1.0), "low"), (dict(af=0.0), "attn_factor"),
    (dict(c=0), "null"),
])
def test_rope_table_refusals(lib, kwargs, why):
    assert _table(lib, **kwargs) == 1
    assert why in lib.attn_last_error().decode()


def _tables(lib, bt=16, old=16, new=32, free=16, sl=64, cu=16, slots=16, pos=16, used=16, B=2, mp=4, nf=4, ps=16, cap=8):
    return lib.attn_block_tables(bt, old, new, free, sl, cu, slots, pos, used, B, mp, nf, ps, cap, None)


@pytest.mark.parametrize("kwargs,why", [
    (dict(ps=24), "page_size"), (dict(ps=4), "page_size"), (dict(B=0), "B"), (dict(nf=-1), "n_free"),
    (dict(cap=-1), "capacity"), (dict(mp=1 << 28), "max_pages"), (dict(bt=0), "integer"), (dict(free=0), "integer"),
    (dict(pos=0), "integer"), (dict(slots=4), "slots"), (dict(sl=16), "seq_lens"), (dict(sl=32), "seq_lens"),
])
def test_block_table_refusals(lib, kwargs, why):
    assert _tables(lib, **kwargs) == 1
    assert why in lib.attn_last_error().decode()


@pytest.mark.parametrize("kwargs", [dict(sl=0x1004), dict(sl=0xFFC), dict(cu=0x2004), dict(used=0x300C), dict(slots=0xFC8),
                                    dict(pos=0x2000), dict(bt=0xFE4)])
def test_block_table_outputs_over_inputs(lib, kwargs):
    """Partial overlaps too: the other blocks of the kernel still read what one writes."""
    apart = dict(bt=0x10000, old=0x1000, new=0x2000, free=0x3000, sl=0x4000, cu=0x5000, slots=0x6000, pos=0x7000, used=0x8000)
    assert _tables(lib, **{**apart, **kwargs}) == 1
    assert "overlap" in lib.attn_last_error().decode()


def _append(lib, q=16, qo=16, k=16, v=16, kc=16, vc=16, slots=16, c=16, s=16, pos=16, total=4, H=2, Hkv=1, d=64,
            rot=64, mp=8, pages=4, ps=16, qs=None, ks=None, vs=None, il=0, dt=0):
    return lib.attn_cache_append(q, qo, k, v, kc, vc, slots, c, s, pos, total, H, Hkv, d, rot, mp, pages, ps, qs, ks,
                                 vs, il, dt, None)


def _append8(lib, q=16, qo=16, k=16, v=16, kc=16, vc=16, kd=16, vd=16, bt=16, sl=16, cu=16, c=16, s=16, sg=16, B=1,
             total=4, H=2, Hkv=1, d=128, rot=64, mp=8, pages=4, ps=16, maxp=2, qs=None, ks=None, vs=None, il=0, dt=0):
    return lib.attn_cache_append_fp8(q, qo, k, v, kc, vc, kd, vd, bt, sl, cu, c, s, sg, B, total, H, Hkv, d, rot, mp,
                                     pages, ps, maxp, qs, ks, vs, il, dt, None)


@pytest.mark.parametrize("call", [_append, _append8])
@pytest.mark.parametrize("kwargs,why", [
    (dict(ps=12), "page_size"), (dict(total=-1), "total"), (dict(pages=0), "num_pages"), (dict(d=96), "d must"),
    (dict(rot=40), "rot_dim"), (dict(s=0), "both"), (dict(c=0, s=0), "needs rope_cos"), (dict(k=0), "null"),
    (dict(kc=8), "aligned"), (dict(qo=0), "null"), (dict(ks=S2(64, 4)), "strides"), (dict(vs=S2(-64, 64)), "strides"),
    (dict(il=3), "interleaved"), (dict(dt=5), "dtype"), (dict(total=1 << 28), "2^31"),
])
def test_append_refusals(lib, call, kwargs, why):
    assert call(lib, **kwargs) == 1
    assert why in lib.attn_last_error().decode()


def test_append_own_refusals(lib):
    assert _append(lib, slots=4) == 1 and b"slots" in lib.attn_last_error()
    assert _append(lib, pos=0) == 1 and b"integer" in lib.attn_last_error()
    assert _append8(lib, ps=8) == 1 and b"page_size" in lib.attn_last_error()
    assert _append8(lib, d=64) == 2
    assert _append8(lib, sg=4) == 1 and b"hadamard" in lib.attn_last_error()
    assert _append8(lib, kd=0) == 1 and _append8(lib, bt=0) == 1 and _append8(lib, B=0) == 1


def test_python_refusals():
    """Shapes and types that the binding turns away by itself, before it looks for a device."""
    import torch
    import exact_tiled_attention_25_gb300 as attn
    nat = attn._binding()
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)

    def cross(q, k, v, lens=None, o=None):
        nat.cross_fwd(q, k, v, lens, None, o, None, None, None)

    x = torch.zeros(1, 2, 3, 64, **bf)
    for args, why in (((x, x.expand(2, 2, 3, 64).contiguous(), x), "q's B and d"),
                      ((x.float(), x.float(), x.float()), "bfloat16"), ((x, x, x.half()), "bfloat16"),
                      ((x.transpose(1, 2), x, x), "contiguous"), ((x[0], x, x), r"\[B, H, N, d\]"),
                      ((x, x, x, torch.zeros(1)), "kv_lens"), ((x, x, x, torch.zeros(2, **i32)), "kv_lens"),
                      ((x, None, x), "k is missing"), ((x, x, x), "current CUDA device")):
        with pytest.raises(ValueError, match=why):
            cross(*args)
    with pytest.raises(TypeError, match="v must be a tensor"):
        cross(x, x, 3)
    with pytest.raises(TypeError, match="expected 9 arguments"):
        nat.cross_fwd(x)
    with pytest.raises(ValueError, match="lse must be"):
        nat.cross_bwd(x, x, x, x, x, torch.zeros(1, 2, 4), *[None] * 7)
    c = torch.zeros(8, 32)
    rope = lambda q, k=None, cos=c, sin=c, pos=None, qo=None, ko=None: nat.rope(q, k, cos, sin, pos, False, False, qo, ko, None)
    for args, why in (((x, None, c, torch.zeros(8, 16)), "rope_sin"), ((x, None, c[0], c[0]), "rope_cos"),
                      ((x, None, None), "rope_cos is missing"), ((x[0, 0],), "packed"), ((x.float(),), "float16"), ((x[:, :0],), "empty"),
                      ((x, x[:, :, :2]), "k must match"), ((x, x[0]), "k must match"), ((x, None, c, c, torch.zeros(3, **i32)), "positions"),
                      ((x, None, c, c, None, x.half()), "q_out"), ((x, None, c, c, None, None, x), "k_out"),
                      ((x,), "current CUDA device")):
        with pytest.raises(ValueError, match=why):
            rope(*args)
    rows, cache, slots = torch.zeros(4, 6, 64, **bf), torch.zeros(3, 16, 6, 64, **bf), torch.zeros(4, dtype=torch.int64)

    def append(k=rows, v=rows, kc=cache, vc=cache, slots=slots, cos=None, sin=None, pos=None, q=None, qo=None):
        nat.cache_append(k, v, kc, vc, slots, cos, sin, pos, q, False, qo, None)

    for kw, why in ((dict(kc=cache[:, :, :2]), "caches"), (dict(v=rows[:, :2]), "k and v"), (dict(qo=rows), "q_out"),
                    (dict(k=torch.zeros(4, 64, 6, **bf).transpose(1, 2)), "rows"), (dict(slots=slots.int()), "slots"),
                    (dict(cos=c, sin=c), "positions"), (dict(cos=c), "both"), (dict(q=rows[:3]), "q must be"),
                    (dict(vc=cache.half()), "v_cache"), (dict(), "current CUDA device")):
        with pytest.raises(ValueError, match=why):
            append(**kw)
    v8 = torch.zeros(3, 16, 6, 64, dtype=torch.uint8)
    d8, bt, lens = torch.zeros(3, 6), torch.zeros(2, 2, **i32), torch.zeros(2, **i32)
    for i, (bad, why) in enumerate(((cache, "k_cache"), (v8, "v_descale"), (v8, "block_table"), (v8, "cu_seqlens"),
                                    (v8, "current CUDA device"))):
        with pytest.raises(ValueError, match=why):
            nat.cache_append_fp8(rows, rows, bad, v8, d8, d8[:2] if i == 1 else d8, bt[0] if i == 2 else bt, lens,
                                 lens if i == 3 else torch.zeros(3, **i32), None, None, None, None, False, None, None)
    for args, why in (((bt, lens, lens, lens, 16, -1), "capacity"), ((bt[0], lens, lens, lens, 16, 4), "max_pages"),
                      ((bt, lens.long(), lens, lens, 16, 4), "old_lens"), ((bt, lens, lens, lens, 2 ** 40, 4), "page_size"),
                      ((bt, lens, lens, lens, 16, 4), "current CUDA device")):
        with pytest.raises(ValueError, match=why):
            nat.block_tables(*args, *[None] * 6)
    with pytest.raises(ValueError, match="positive"):
        nat.rope_table(0, 64, 1e4, 1.0, 0, 1.0, 32.0, 1.0, 0, None, None, None)
    with pytest.raises(TypeError):
        nat.rope_table(4, 64, "x", 1.0, 0, 1.0, 32.0, 1.0, 0, None, None, None)
