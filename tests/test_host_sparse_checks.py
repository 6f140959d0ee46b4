"""Refusals of the block-sparse entry points, on the host: each call below is refused with
KVP_ERR_INVALID before any CUDA call. The pointers are fake and never dereferenced."""

import ctypes as C

import pytest

from paged_kv_cache_319_b200 import _lib

F16, BF16, FP8 = _lib.KVP_F16, _lib.KVP_BF16, _lib.KVP_FP8_E4M3
INVALID, OK = _lib.KVP_ERR_INVALID, _lib.KVP_OK
MB = 1 << 20


def p(i, off=0):
    return C.c_void_p(i * 64 * MB + off)


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


ROPE = dict(q=p(1), k=p(2), v=p(3), qo=p(4), qs=1024, ks=256, vs=256, qos=1024, cs=p(5), pos=p(6),
            maxp=4096, rot=128, il=0, kc=p(7), vc=p(8), sl=p(9), kscale=None, vscale=None, T=4,
            Hq=8, Hkv=2, D=128, bs=16, NB=8, dt=F16, cdt=F16, st=None)
BOUNDS = dict(k=p(1), b=p(2), t=p(3), l=p(4), new=p(5), S=2, Hkv=2, D=128, bs=16, NB=8, mb=4,
              mcl=64, mnew=3, cdt=F16, st=None)
SELECT = dict(q=p(1), b=p(2), t=p(3), l=p(4), out=p(5), S=2, Hq=8, Hkv=2, D=128, bs=16, NB=8, mb=4,
              mcl=64, keep=4, sink=1, recent=1, dt=F16, cdt=F16, st=None)
DECODE = dict(q=p(1), k=p(2), v=p(3), kscale=None, vscale=None, t=p(4), l=p(5), sel=p(6), S=2, Hq=8,
              Hkv=2, D=128, bs=16, NB=8, mb=4, mcl=64, keep=4, scale=0.1, out=p(7), dt=F16, cdt=F16,
              st=None)


def call(fn, base, **kw):
    assert set(kw) <= set(base)
    return fn(*{**base, **kw}.values())


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(NB=0), dict(bs=0), dict(bs=24), dict(maxp=0),
    dict(D=96), dict(D=8), dict(D=2048), dict(rot=0), dict(rot=8), dict(rot=144), dict(dt=FP8),
    dict(dt=BF16), dict(cdt=BF16), dict(cdt=FP8), dict(cdt=FP8, kscale=p(10)), dict(q=None),
    dict(k=None), dict(v=None), dict(qo=None), dict(cs=None), dict(pos=None), dict(kc=None),
    dict(vc=None), dict(sl=None), dict(q=p(1, 8)), dict(kc=p(7, 8)), dict(sl=p(9, 4)),
    dict(cs=p(5, 4)), dict(qs=1028), dict(ks=-8), dict(qos=1016), dict(qo=p(1, 16)),
    dict(qo=p(2)), dict(qo=p(3, 512)), dict(qo=p(1), qs=1040), dict(Hq=1 << 21)])
def test_append_refuses(lib, bad):
    assert call(lib.rope_reshape_and_cache, ROPE, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(S=-1), dict(Hkv=0), dict(NB=0), dict(mb=0), dict(mcl=-1), dict(mcl=65), dict(bs=4),
    dict(bs=64), dict(D=96), dict(D=64, cdt=FP8), dict(cdt=3), dict(mnew=-1), dict(k=None),
    dict(b=None), dict(t=None), dict(l=None), dict(k=p(1, 8)), dict(b=p(2, 2)), dict(new=p(5, 2)),
    dict(S=1 << 30, new=None)])
def test_bounds_refuse(lib, bad):
    assert call(lib.update_key_bounds, BOUNDS, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(S=-1), dict(Hq=7), dict(Hkv=0), dict(NB=0), dict(mb=0), dict(mcl=65), dict(mcl=-1),
    dict(bs=4), dict(D=96), dict(D=64, cdt=FP8), dict(cdt=BF16), dict(dt=FP8), dict(keep=0),
    dict(keep=-4), dict(sink=-1), dict(recent=-1), dict(sink=3, recent=2),
    dict(sink=(1 << 31) - 1, recent=(1 << 31) - 1), dict(q=None), dict(b=None), dict(t=None),
    dict(l=None), dict(out=None), dict(q=p(1, 8)), dict(out=p(5, 2)),
    dict(mb=1 << 27, mcl=(1 << 31) - 1)])
def test_selection_refuses(lib, bad):
    assert call(lib.select_blocks, SELECT, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(S=-1), dict(Hq=7), dict(Hkv=0), dict(NB=0), dict(mb=0), dict(mcl=65), dict(bs=4),
    dict(D=96), dict(D=64, cdt=FP8, kscale=p(8), vscale=p(9)), dict(cdt=BF16), dict(cdt=FP8),
    dict(dt=FP8), dict(keep=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None),
    dict(k=None), dict(v=None), dict(t=None), dict(l=None), dict(sel=None), dict(out=None),
    dict(k=p(2, 8)), dict(sel=p(6, 2)), dict(NB=1 << 26), dict(cdt=FP8, kscale=p(8, 2), vscale=p(9)),
    dict(S=1 << 30)])
def test_decode_refuses(lib, bad):
    assert call(lib.paged_attention_decode_sparse, DECODE, **bad) == INVALID


def test_empty_calls_are_no_ops(lib):
    assert call(lib.rope_reshape_and_cache, ROPE, T=0, q=None, k=None, v=None, qo=None) == OK
    assert call(lib.update_key_bounds, BOUNDS, S=0, t=None, l=None) == OK
    assert call(lib.update_key_bounds, BOUNDS, mcl=0) == OK
    assert call(lib.update_key_bounds, BOUNDS, mnew=0) == OK
    assert call(lib.select_blocks, SELECT, S=0, q=None, out=None) == OK
    assert call(lib.paged_attention_decode_sparse, DECODE, S=0, q=None, out=None) == OK


def test_the_torch_binding_refuses_without_a_gpu():
    import torch
    import paged_kv_cache_319_b200 as kvp

    x = torch.zeros((2, 2, 64), dtype=torch.float16)
    pool = torch.zeros((4, 2, 16, 64), dtype=torch.float16)
    t, l = torch.zeros((2, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    idx = torch.zeros(2, dtype=torch.int64)
    for call in (lambda: kvp.rope_reshape_and_cache(x, x, x, torch.zeros(8, 64), idx, pool, pool, idx),
                 lambda: kvp.update_key_bounds(pool, pool[:, :, :2], t, l),
                 lambda: kvp.select_blocks(x, pool[:, :, :2], t, l, block_size=16, num_selected=2),
                 lambda: kvp.paged_attention_decode_sparse(x, pool, pool, t, l, t[:, None], 1.0)):
        with pytest.raises(ValueError, match="same CUDA device"):
            call()
    with pytest.raises(TypeError, match="torch tensor"):
        kvp.update_key_bounds([1], pool, t, l)
