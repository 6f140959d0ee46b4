"""Block-sparse decoding on the GPU against the fp64 oracle (oracle/sparse.py).

rope_reshape_and_cache: the bits of the fp32 formula, and within its rounding of the exact
rotation. update_key_bounds and select_blocks: equal to the oracle's (no rounding is
involved in bounds; scores of equal blocks are equal sums). paged_attention_decode_sparse:
within half a step of the output's type of the exact result, plus the bound that
oracle.sparse.decode_error derives for fp32 logits, weights and sums.
"""



import numpy as np
import pytest

from oracle import attention, fp8, sparse
from oracle.numerics import half_ulp, to_f64
from parity import from_bits, random_e4m3_codes, to_bits
import workloads

pytestmark = pytest.mark.gpu

SCALE = 1 / np.sqrt(128.0)


def _torch():
    import torch

    return torch


def _kvp():
    import paged_kv_cache_319_b200 as kvp

    return kvp


def _dev(x):
    return _torch().from_numpy(np.ascontiguousarray(x)).cuda()


def _tdt(dtype):
    return _torch().float16 if dtype == "f16" else _torch().bfloat16


def _tables(rng, lens, bs, extra=5):
    need = [-(-int(n) // bs) for n in lens]
    nb = sum(need) + extra
    perm = rng.permutation(nb).astype(np.int32)
    t = np.full((len(lens), max(need + [1])), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        t[s, :n] = perm[at:at + n]
        at += n
    return t, nb


def _raises(kind):
    kvp = _kvp()
    with pytest.raises(kvp.KvpError) as e:
        kvp.check_device_error()
    assert e.value.kind == kind
    return str(e.value)


# ---- rope_reshape_and_cache -----------------------------------------------------------
def _append_case(seed, T, Hq, Hkv, D, rot, bs, NB, dtype, far=5000):
    rng = np.random.default_rng(seed)
    bits = workloads.normal_bits([seed, 7], (T, Hq + 2 * Hkv, D), dtype)
    half = rot // 2
    ang = np.arange(far)[:, None] * 10000.0 ** (-np.arange(half) / half)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pos = rng.integers(0, far, T)
    slots = rng.permutation(NB * bs)[:T].astype(np.int64)
    return bits, cs, pos, slots


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,bs,dtype,cache,paired", [
    (1, 4, 4, 64, 64, 16, "f16", "f16", False),
    (3, 1, 1, 16, 16, 1, "bf16", "bf16", True),
    (37, 8, 2, 128, 128, 16, "bf16", "bf16", False),
    (37, 8, 2, 128, 64, 32, "f16", "f16", True),
    (5, 40, 40, 128, 32, 8, "f16", "e4m3", False),
    (130, 6, 2, 128, 112, 16, "bf16", "e4m3", True),
    (2, 3, 1, 256, 256, 16, "bf16", "e4m3", False),
    (1500, 16, 4, 64, 48, 16, "bf16", "bf16", False),
    (5003, 8, 1, 128, 64, 16, "bf16", "bf16", False),
    (4999, 3, 1, 64, 16, 8, "f16", "f16", True),
    (4801, 1, 1, 128, 128, 16, "f16", "e4m3", False),
])
def test_append_rotates_and_stores(T, Hq, Hkv, D, rot, bs, dtype, cache, paired):
    torch, kvp = _torch(), _kvp()
    NB = -(-T // bs) + 4
    bits, cs, pos, slots = _append_case(11, T, Hq, Hkv, D, rot, bs, NB, dtype)
    rows = from_bits(bits, dtype).view(T, -1)
    q, k, v = (x.unflatten(1, (-1, D)) for x in rows.split([Hq * D, Hkv * D, Hkv * D], 1))
    ks = vs = None
    if cache == "e4m3":
        before = [random_e4m3_codes(5 + i, (NB, Hkv, bs, D)) for i in range(2)]
        pools = [_dev(x) for x in before]
        ks, vs = (np.random.default_rng(i).uniform(0.003, 0.02, Hkv).astype(np.float32) for i in (1, 2))
        kw = dict(k_scale=_dev(ks), v_scale=_dev(vs))
    else:
        before = [workloads.normal_bits([9, i], (NB, Hkv, bs, D), dtype) for i in range(2)]
        pools, kw = [from_bits(x, dtype) for x in before], {}
    out = kvp.rope_reshape_and_cache(q, k, v, _dev(cs), _dev(pos), *pools, _dev(slots),
                                     interleaved=paired, **kw)
    kvp.check_device_error()
    x = to_f64(bits, dtype)
    qx, kx, vx = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]

    def rounded(y32):  # fp32 -> bits
        t = torch.from_numpy(y32).to(_tdt(dtype))
        return t.view(torch.int16).numpy().view(np.uint16)

    def check(bits_got, src, turn):
        y32 = sparse.rotate(src, cs[pos], paired, np.float32) if turn else src.astype(np.float32)
        assert np.array_equal(bits_got, rounded(y32))
        exact = sparse.rotate(src, cs[pos].astype(np.float64), paired) if turn else src
        err = sparse.rotation_error(src, cs[pos], paired) if turn else 0.0
        assert (np.abs(to_f64(bits_got, dtype) - exact)
                <= half_ulp(np.abs(exact) + err, dtype) + err).all()

    check(to_bits(out), qx, True)
    blk, off = slots // bs, slots % bs
    for pool, old, src, turn, scale in ((pools[0], before[0], kx, True, ks),
                                        (pools[1], before[1], vx, False, vs)):
        if cache == "e4m3":
            got = pool.cpu().numpy()
            y32 = sparse.rotate(src, cs[pos], paired, np.float32) if turn else src
            assert np.array_equal(got[blk, :, off], fp8.quantize(y32, scale[:, None]))
        else:
            got = to_bits(pool)
            check(got[blk, :, off], src, turn)
        rest = np.ones((NB, bs), bool)
        rest[blk, off] = False
        assert np.array_equal(got.transpose(0, 2, 1, 3)[rest], old.transpose(0, 2, 1, 3)[rest])


def test_append_in_place_padding_and_bad_indexes():
    torch, kvp = _torch(), _kvp()
    T, Hq, Hkv, D, bs, NB = 9, 4, 2, 64, 16, 3
    bits, cs, pos, slots = _append_case(13, T, Hq, Hkv, D, 64, bs, NB, "f16", far=100)
    slots[1] = -1                    # padding that keeps its rotation
    slots[2], pos[2] = -1, -1        # padding that leaves its row
    rows = from_bits(bits, "f16").view(T, -1)
    first = rows.clone()
    q, k, v = (x.unflatten(1, (-1, D)) for x in rows.split([Hq * D, Hkv * D, Hkv * D], 1))
    pools = [torch.zeros((NB, Hkv, bs, D), dtype=torch.float16, device="cuda") for _ in range(2)]
    out = kvp.rope_reshape_and_cache(q, k, v, _dev(cs), _dev(pos), *pools, _dev(slots), q)
    kvp.check_device_error()
    assert out.data_ptr() == q.data_ptr()
    want = sparse.rotate(to_f64(bits[:, :Hq], "f16"), cs[np.maximum(pos, 0)], False, np.float32)
    want[2] = to_f64(bits[2, :Hq], "f16")
    got = to_bits(rows).reshape(T, -1, D)
    assert np.array_equal(got[:, :Hq], want.astype(np.float16).view(np.uint16))
    assert np.array_equal(got[:, Hq:], to_bits(first).reshape(T, -1, D)[:, Hq:])
    held = np.zeros((NB, bs), bool)
    held[slots[slots >= 0] // bs, slots[slots >= 0] % bs] = True
    filled = (pools[1] != 0).any(3).any(1).cpu().numpy()
    assert np.array_equal(filled, held)

    for slot, at, text in ((NB * bs, 5, "slot"), (0, 100, "position"), (0, -1, "position")):
        s2, p2 = np.array([slot, 17]), np.array([at, 3])
        pools = [torch.zeros((NB, Hkv, bs, D), dtype=torch.float16, device="cuda") for _ in range(2)]
        kvp.rope_reshape_and_cache(q[:2], k[:2], v[:2], _dev(cs), _dev(p2), *pools, _dev(s2))
        assert text in _raises("bounds")
        filled = (pools[1] != 0).any(3).any(1).cpu().numpy()
        assert filled.sum() == 1 and filled[17 // bs, 17 % bs]


def test_append_python_refusals():
    torch, kvp = _torch(), _kvp()
    z = dict(dtype=torch.float16, device="cuda")
    q, k, pool = torch.zeros((2, 4, 64), **z), torch.zeros((2, 2, 64), **z), torch.zeros((2, 2, 16, 64), **z)
    cs, idx = torch.zeros((8, 64), device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    good = [q, k, k.clone(), cs, idx, pool, pool.clone(), idx]
    kvp.rope_reshape_and_cache(*good)
    for i, bad, err in ((0, q.bfloat16(), TypeError), (0, q.transpose(0, 1).contiguous().transpose(0, 1), ValueError),
                        (1, k[:1], ValueError), (3, cs.half(), TypeError), (4, idx.int(), TypeError),
                        (5, pool[..., :32].contiguous(), ValueError), (5, pool.bfloat16(), TypeError),
                        (3, cs[:, :24].contiguous(), kvp.KvpError), (0, q.cpu(), ValueError),
                        (7, idx[:1], ValueError)):
        with pytest.raises(err):
            kvp.rope_reshape_and_cache(*good[:i], bad, *good[i + 1:])
    with pytest.raises(ValueError):
        kvp.rope_reshape_and_cache(*good, k_scale=torch.ones(2, device="cuda"),
                                   v_scale=torch.ones(2, device="cuda"))
    codes = pool.to(torch.uint8)
    with pytest.raises(ValueError):
        kvp.rope_reshape_and_cache(*good[:5], codes, codes.clone(), idx)
    with pytest.raises(kvp.KvpError):
        kvp.rope_reshape_and_cache(*good, k.repeat(1, 2, 1).as_strided((2, 4, 64), (0, 64, 1)))
    kvp.check_device_error()


# ---- update_key_bounds ------------------------------------------------------------------
def _key_pool(seed, shape, cache):
    """(device pool, fp64 values)"""
    if cache == "e4m3":
        codes = random_e4m3_codes(seed, shape)
        return _dev(codes), fp8.decode(codes)
    bits = workloads.normal_bits([seed, 3], shape, cache)
    return from_bits(bits, cache), to_f64(bits, cache)


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("cache,D,Hkv", [("f16", 64, 3), ("f16", 128, 2), ("bf16", 64, 1),
                                         ("bf16", 128, 5), ("e4m3", 128, 2)])
@pytest.mark.parametrize("new", [None, [0, 1, 1, 40, 2, 17, 3]])
def test_bounds_of_touched_blocks(bs, cache, D, Hkv, new):
    torch, kvp = _torch(), _kvp()
    lens = [70, 1, 65, 33, bs, 2 * bs + 1, 0]
    t, nb = _tables(np.random.default_rng(21), lens, bs)
    pool, vals = _key_pool(22, (nb, Hkv, bs, D), cache)
    # NaN behind every context: never read
    for s, n in enumerate(lens):
        if n % bs:
            pool[int(t[s, n // bs]), :, n % bs:] = 0x7F if cache == "e4m3" else float("nan")
    small = "f16" if cache == "e4m3" else cache
    bounds = torch.full((nb, Hkv, 2, D), 7.5, dtype=_tdt(small), device="cuda")
    kvp.update_key_bounds(pool, bounds, _dev(t), _dev(np.int32(lens)),
                          new_tokens=None if new is None else _dev(np.int32(new)),
                          max_new_tokens=None if new is None else 40)
    kvp.check_device_error()
    want = sparse.key_bounds(np.full((nb, Hkv, 2, D), 7.5), vals, t, lens, new)
    assert np.array_equal(to_f64(to_bits(bounds), small), want)


def test_bounds_hold_infinities_and_nan():
    torch, kvp = _torch(), _kvp()
    pool = torch.zeros((2, 1, 8, 64), dtype=torch.bfloat16, device="cuda")
    pool[1, 0, 2, 5], pool[1, 0, 3, 6], pool[1, 0, 4, 7] = float("nan"), float("inf"), -float("inf")
    bounds = torch.zeros((2, 1, 2, 64), dtype=torch.bfloat16, device="cuda")
    kvp.update_key_bounds(pool, bounds, _dev(np.int32([[1]])), _dev(np.int32([8])))
    kvp.check_device_error()
    b = bounds[1, 0].float().cpu()
    assert b[:, 5].isnan().all() and b[0, 6] == float("inf") and b[1, 7] == -float("inf")
    assert b[1, 6] == 0 and b[0, 7] == 0 and not b[:, :5].any()


def test_bounds_report_bad_metadata():
    torch, kvp = _torch(), _kvp()
    pool, vals = _key_pool(23, (4, 1, 16, 64), "f16")

    def run(table, lens, new=None, most=None, mcl=None):
        b = torch.zeros((4, 1, 2, 64), dtype=torch.float16, device="cuda")
        kvp.update_key_bounds(pool, b, _dev(np.int32(table)), _dev(np.int32(lens)),
                              new_tokens=None if new is None else _dev(np.int32(new)),
                              max_new_tokens=most, max_context_len=mcl)
        return to_f64(to_bits(b), "f16")

    zero = np.zeros((4, 1, 2, 64))
    good = sparse.key_bounds(zero, vals, [[0, 1]], [32])
    assert np.array_equal(run([[0, 1]], [40], mcl=32), good) and "length" in _raises("bounds")
    assert np.array_equal(run([[0, 1]], [-1]), zero) and "length" in _raises("bounds")
    assert np.array_equal(run([[0, 4]], [32]), sparse.key_bounds(zero, vals, [[0, 1]], [16]))
    assert "block table" in _raises("bounds")
    assert np.array_equal(run([[0, 1]], [32], [9], 3), sparse.key_bounds(zero, vals, [[0, 1]], [32], [3]))
    _raises("bounds")
    # more new tokens than the context holds is all of them
    assert np.array_equal(run([[0, 1]], [32], [50], 64), good)
    _kvp().check_device_error()


# ---- select_blocks ------------------------------------------------------------------------
@pytest.mark.parametrize("Hq,Hkv,D,bs,dtype,cache,keep,sink,recent,lens", [
    (4, 4, 64, 16, "f16", "f16", 4, 1, 1, [0, 1, 16, 64, 65, 80, 700]),
    (8, 1, 128, 8, "bf16", "bf16", 9, 0, 0, [71, 72, 73, 1001]),
    (8, 2, 128, 32, "bf16", "e4m3", 7, 2, 3, [1, 224, 225, 3000]),
    (3, 3, 128, 16, "f16", "e4m3", 5, 0, 5, [500, 80, 81]),
    (16, 1, 64, 8, "bf16", "bf16", 130, 4, 4, [9000, 1040, 1041]),
    (2, 1, 128, 16, "f16", "f16", 1, 1, 0, [100, 16, 17]),
    (1, 1, 64, 8, "f16", "f16", 33, 1, 2, [25001]),
])
def test_selection_equals_the_oracle(Hq, Hkv, D, bs, dtype, cache, keep, sink, recent, lens):
    kvp = _kvp()
    rng = np.random.default_rng(31)
    t, nb = _tables(rng, lens, bs)
    small = "f16" if cache == "e4m3" else cache
    _, keys = _key_pool(32, (nb, Hkv, 4, D), cache)
    bounds64 = np.stack([keys.max(2), keys.min(2)], 2)
    qb = workloads.normal_bits([33, 1], (len(lens), Hq, D), dtype)
    got = kvp.select_blocks(from_bits(qb, dtype), _dev(bounds64).to(_tdt(small)), _dev(t),
                            _dev(np.int32(lens)), block_size=bs, num_selected=keep,
                            num_sink=sink, num_recent=recent)
    kvp.check_device_error()
    want = sparse.select_blocks(to_f64(qb, dtype), bounds64, t, lens, bs, keep, sink, recent)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["ties", "few values", "nan", "inf", "all nan", "zero query"])
@pytest.mark.parametrize("n", [150, 2500])
def test_selection_of_equal_and_nonfinite_scores(kind, n):
    kvp = _kvp()
    rng = np.random.default_rng(41)
    D, bs, keep = 64, 8, 40
    bounds = np.ones((n, 1, 2, D))
    q = np.full((1, 2, D), 0.5)
    if kind == "few values":
        bounds[:] = rng.integers(-2, 3, (n, 1, 1, 1))
    elif kind == "nan":
        bounds[rng.permutation(n)[:5], 0, 0, 3] = np.nan
        bounds[:, 0, 1, 7] = -rng.integers(0, 9, n)
    elif kind == "inf":
        bounds[rng.permutation(n)[:60], 0, 0, 3] = np.inf
        bounds[rng.permutation(n)[:5], 0, 0, 9] = -np.inf
    elif kind == "all nan":
        q[0, 0, 0] = np.nan
    elif kind == "zero query":
        q[:] = 0
    table = rng.permutation(n).astype(np.int32)[None]
    got = kvp.select_blocks(_dev(q).half(), _dev(bounds).half(), _dev(table),
                            _dev(np.int32([n * bs])), block_size=bs, num_selected=keep,
                            num_sink=1, num_recent=2)
    kvp.check_device_error()
    with np.errstate(invalid="ignore"):
        want = sparse.select_blocks(q, bounds, table, [n * bs], bs, keep, 1, 2)
    assert np.array_equal(got.cpu().numpy(), want)


def test_selection_over_many_blocks_in_one_cluster():
    # more scores than one CTA's shared memory holds, after a small launch of the same kernel
    kvp = _kvp()
    rng = np.random.default_rng(43)
    for n in (7000, 40, 60001):
        vals = rng.permutation(n).astype(np.float32)  # block b's score is vals[b]
        bounds = np.zeros((n, 1, 2, 64), np.float32)
        bounds[:, 0, :, 0] = (vals % 256)[:, None]
        bounds[:, 0, :, 1] = (vals // 256)[:, None]
        q = np.zeros((1, 1, 64), np.float32)
        q[0, 0, 0], q[0, 0, 1] = 1.0, 256.0
        table = np.arange(n, dtype=np.int32)[None]
        got = kvp.select_blocks(_dev(q).half(), _dev(bounds).half(), _dev(table),
                                _dev(np.int32([n * 8])), block_size=8, num_selected=30,
                                num_sink=0, num_recent=0).cpu().numpy()[0, 0]
        kvp.check_device_error()
        assert np.array_equal(got, np.sort(np.argsort(-vals, kind="stable")[:30]))


@pytest.mark.parametrize("n,close", [(500, 500), (500, 20), (30000, 40), (30000, 30000), (3000, 65)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_selection_of_scores_closer_than_fp32_tells(n, close, dtype):
    # every block scores 1024 + 2^-12 v, v one of 0..127 for `close` blocks (ties among
    # them), 1104 for 10 blocks and 1000 for the rest; the cut falls among the close ones
    kvp = _kvp()
    rng = np.random.default_rng(44)
    keep = 10 + close // 3
    hi = np.zeros((n, 128))
    hi[:, 0] = 1000
    order = rng.permutation(n)
    hi[order[:close], 0] = 1024
    hi[order[:close], 1] = rng.integers(0, 128, close)
    if close < n:
        hi[order[close:close + 10], 0] = 1104
    bounds = np.stack([hi, hi - 0.0], 1)[:, None]
    q = np.zeros((1, 1, 128))
    q[0, 0, 0], q[0, 0, 1] = 1.0, 2.0**-12
    table = rng.permutation(n).astype(np.int32)[None]
    got = kvp.select_blocks(_dev(q).to(_tdt(dtype)), _dev(bounds).to(_tdt(dtype)), _dev(table),
                            _dev(np.int32([n * 16])), block_size=16, num_selected=keep,
                            num_sink=0, num_recent=0)
    kvp.check_device_error()
    score = hi[table[0], 0] + 2.0**-12 * hi[table[0], 1]
    assert np.array_equal(got.cpu().numpy()[0, 0], np.sort(np.argsort(-score, kind="stable")[:keep]))


@pytest.mark.parametrize("dtype,quantum", [("f16", 2.0**-24), ("bf16", 2.0**-133), ("bf16", 2.0**110)])
@pytest.mark.parametrize("n", [50, 900])
def test_selection_of_tiny_and_huge_bounds(dtype, quantum, n):
    # bounds of 1 to 127 quanta: below the type's normal range, or with sums past fp32's
    kvp = _kvp()
    rng = np.random.default_rng(45)
    hi = rng.integers(1, 128, (n, 1, 64)) * quantum
    bounds = np.stack([hi, -hi], 2)
    qb = workloads.normal_bits([46, n], (1, 2, 64), dtype)
    table = rng.permutation(n).astype(np.int32)[None]
    bd = _dev(bounds).to(_tdt(dtype))
    assert np.array_equal(to_f64(to_bits(bd), dtype), bounds)
    got = kvp.select_blocks(from_bits(qb, dtype), bd, _dev(table), _dev(np.int32([n * 8])),
                            block_size=8, num_selected=20)
    kvp.check_device_error()
    want = sparse.select_blocks(to_f64(qb, dtype), bounds, table, [n * 8], 8, 20, 1, 1)
    assert np.array_equal(got.cpu().numpy(), want)


def test_selection_reports_bad_metadata():
    torch, kvp = _torch(), _kvp()
    bounds = torch.rand((20, 1, 2, 64), device="cuda").half()
    q = torch.ones((1, 1, 64), device="cuda").half()
    table = np.arange(20, dtype=np.int32)[None]

    def run(t, n, **kw):
        return kvp.select_blocks(q, bounds, _dev(t), _dev(np.int32([n])), block_size=8,
                                 num_selected=4, num_sink=1, num_recent=1, **kw).cpu().numpy()

    good = run(table, 160)
    assert np.array_equal(run(table, 161), good) and "length" in _raises("bounds")
    assert (run(table, -5) == -1).all() and "length" in _raises("bounds")
    bad = table.copy()
    bad[0, good[0, 0, 1]] = 20
    assert good[0, 0, 1] not in run(bad, 160) and "block table" in _raises("bounds")
    for kw in (dict(num_selected=2, num_sink=2, num_recent=1), dict(num_selected=0)):
        with pytest.raises(kvp.KvpError):
            kvp.select_blocks(q, bounds, _dev(table), _dev(np.int32([9])), block_size=8, **kw)
    with pytest.raises(TypeError):
        kvp.select_blocks(q, bounds.bfloat16(), _dev(table), _dev(np.int32([9])), block_size=8,
                          num_selected=4)


# ---- paged_attention_decode_sparse --------------------------------------------------------
def _decode_case(seed, lens, Hq, Hkv, D, bs, dtype, cache):
    t, nb = _tables(np.random.default_rng(seed), lens, bs)
    qb = workloads.normal_bits([seed, 1], (len(lens), Hq, D), dtype)
    pools, vals, kw = [], [], {}
    for i in range(2):
        pool, val = _key_pool(seed + 1 + i, (nb, Hkv, bs, D), cache)
        if cache == "e4m3":  # uniform codes reach 448: scales that keep logits moderate
            sc = np.random.default_rng(seed + i).uniform(0.005, 0.02, Hkv).astype(np.float32)
            kw["k_scale" if i == 0 else "v_scale"] = _dev(sc)
            val = val * sc.astype(np.float64)[:, None, None]
        for s, n in enumerate(lens):  # NaN behind every context: never read
            if n % bs:
                pool[int(t[s, n // bs]), :, n % bs:] = 0x7F if cache == "e4m3" else float("nan")
        pools.append(pool)
        vals.append(val)
    return qb, t, pools, vals, kw


def _check_decode(got_bits, qb, vals, t, lens, sel, dtype, scale):
    q = to_f64(qb, dtype)
    ref = sparse.decode_sparse(q, *vals, t, lens, sel, scale)
    err = sparse.decode_error(q, *vals, t, lens, sel, scale, 2.0**-11)
    got = to_f64(got_bits, dtype)
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > err + half_ulp(np.abs(ref) + err, dtype)
    assert not bad.any(), (np.abs(got - ref).max(), np.argwhere(bad)[:5].tolist())
    return ref


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("Hq,Hkv,D,dtype,cache", [
    (4, 4, 64, "f16", "f16"), (5, 5, 128, "bf16", "bf16"), (8, 2, 128, "f16", "f16"),
    (8, 1, 128, "bf16", "e4m3"), (6, 2, 128, "f16", "e4m3"), (16, 1, 64, "bf16", "bf16"),
    (9, 1, 128, "f16", "f16"), (35, 1, 128, "bf16", "bf16"), (24, 2, 128, "bf16", "e4m3")])
def test_decode_over_listed_blocks(Hq, Hkv, D, dtype, cache, bs):
    kvp = _kvp()
    lens = [0, 1, bs, bs + 1, 333, 700]
    qb, t, pools, vals, kw = _decode_case(51, lens, Hq, Hkv, D, bs, dtype, cache)
    rng = np.random.default_rng(52)
    keep = 13
    sel = np.full((len(lens), Hkv, keep), -1, np.int32)
    for s, n in enumerate(lens):
        blocks = -(-n // bs)
        for h in range(Hkv):
            take = rng.permutation(blocks)[:rng.integers(0, min(keep, blocks) + 1)]
            if s == 4:  # with the partial last block, and holes in the list
                take = np.unique(np.append(take[:keep - 1], blocks - 1))[::-1]
            sel[s, h, np.sort(rng.permutation(keep)[:len(take)])] = take
    got = kvp.paged_attention_decode_sparse(from_bits(qb, dtype), *pools, _dev(t),
                                            _dev(np.int32(lens)), _dev(sel), SCALE, **kw)
    kvp.check_device_error()
    _check_decode(to_bits(got), qb, vals, t, lens, sel, dtype, SCALE)


@pytest.mark.parametrize("Hq,Hkv,bs,dtype,cache,lens,keep", [
    (32, 8, 16, "bf16", "bf16", [9000, 4096], 256),     # clusters of CTAs
    (16, 2, 32, "bf16", "e4m3", [20001], 400),
    (2, 2, 8, "f16", "f16", [5, 9000, 0, 3000], 700),   # a list longer than some contexts
    (4, 4, 16, "f16", "f16", [300] * 130, 12)])
def test_decode_over_long_lists(Hq, Hkv, bs, dtype, cache, lens, keep):
    kvp = _kvp()
    qb, t, pools, vals, kw = _decode_case(55, lens, Hq, Hkv, 128, bs, dtype, cache)
    rng = np.random.default_rng(56)
    sel = np.full((len(lens), Hkv, keep), -1, np.int32)
    for s, n in enumerate(lens):
        blocks = -(-n // bs)
        for h in range(Hkv):
            take = np.sort(rng.permutation(blocks)[:keep])
            sel[s, h, :len(take)] = take
    got = kvp.paged_attention_decode_sparse(from_bits(qb, dtype), *pools, _dev(t),
                                            _dev(np.int32(lens)), _dev(sel), SCALE, **kw)
    kvp.check_device_error()
    _check_decode(to_bits(got), qb, vals, t, lens, sel, dtype, SCALE)


@pytest.mark.parametrize("S,Hq,Hkv,D,bs,dtype,cache", [
    (77, 41, 41, 128, 16, "f16", "f16"), (77, 41, 41, 64, 8, "bf16", "bf16"),
    (97, 62, 31, 128, 8, "bf16", "bf16"), (97, 33, 33, 128, 32, "bf16", "e4m3"),
    (600, 48, 4, 128, 16, "f16", "f16"), (601, 45, 5, 128, 8, "bf16", "e4m3"),
    (600, 40, 4, 64, 32, "f16", "f16")])
def test_decode_of_many_rows_over_short_lists(S, Hq, Hkv, D, bs, dtype, cache):
    kvp = _kvp()
    rng = np.random.default_rng(67)
    lens = rng.integers(0, 5 * bs + 1, S).tolist()
    qb, t, pools, vals, kw = _decode_case(68, lens, Hq, Hkv, D, bs, dtype, cache)
    sel = np.full((S, Hkv, 5), -1, np.int32)
    for s, n in enumerate(lens):
        blocks = -(-n // bs)
        for h in range(Hkv):
            take = rng.permutation(blocks)[:rng.integers(0, blocks + 1)]
            sel[s, h, rng.permutation(5)[:len(take)]] = take
    got = kvp.paged_attention_decode_sparse(from_bits(qb, dtype), *pools, _dev(t),
                                            _dev(np.int32(lens)), _dev(sel), SCALE, **kw)
    kvp.check_device_error()
    _check_decode(to_bits(got), qb, vals, t, lens, sel, dtype, SCALE)


@pytest.mark.parametrize("Hq,Hkv,D,bs,dtype,cache", [
    (16, 1, 64, 16, "f16", "f16"), (4, 1, 64, 8, "bf16", "bf16"), (2, 1, 64, 32, "f16", "f16"),
    (12, 1, 128, 16, "bf16", "e4m3"), (10, 1, 128, 8, "f16", "e4m3"), (5, 1, 128, 8, "bf16", "e4m3"),
    (16, 1, 128, 32, "bf16", "bf16"), (11, 1, 128, 8, "f16", "f16"), (1, 1, 128, 16, "bf16", "bf16")])
@pytest.mark.parametrize("seqs", [1, 21])
def test_decode_of_few_rows_over_long_lists(Hq, Hkv, D, bs, dtype, cache, seqs):
    kvp = _kvp()
    lens = [6000 - 3 * s for s in range(seqs)]
    qb, t, pools, vals, kw = _decode_case(63, lens, Hq, Hkv, D, bs, dtype, cache)
    rng = np.random.default_rng(64)
    keep = 4808 // bs
    sel = np.stack([[np.sort(rng.permutation(-(-n // bs))[:keep]) for _ in range(Hkv)] for n in lens])
    sel = sel.astype(np.int32)
    got = kvp.paged_attention_decode_sparse(from_bits(qb, dtype), *pools, _dev(t),
                                            _dev(np.int32(lens)), _dev(sel), 1 / np.sqrt(D), **kw)
    kvp.check_device_error()
    _check_decode(to_bits(got), qb, vals, t, lens, sel, dtype, 1 / np.sqrt(D))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_of_large_and_tiny_queries_over_e4m3(dtype):
    # bf16 queries far outside fp16's range, one head of zeros
    torch, kvp = _torch(), _kvp()
    lens = [200, 37]
    qb, t, pools, vals, kw = _decode_case(65, lens, 4, 1, 128, 16, dtype, "e4m3")
    factors = [1.0, 2.0**12, 2.0**-9, 0.0] if dtype == "f16" else [2.0**90, 2.0**-100, 1.0, 0.0]
    q = from_bits(qb, dtype) * torch.tensor(factors, device="cuda", dtype=_tdt(dtype))[:, None]
    sel = np.tile(np.arange(13, dtype=np.int32), (2, 1, 1))
    sel[1, 0, 3:] = -1
    # a scale per head cannot be given, so each factor's call uses its own
    for h, f in enumerate(factors):
        scale = SCALE / f if f else SCALE
        got = kvp.paged_attention_decode_sparse(q[:, h:h + 1].contiguous(), *pools, _dev(t),
                                                _dev(np.int32(lens)), _dev(sel), scale, **kw)
        _check_decode(to_bits(got), to_bits(q[:, h:h + 1]), vals, t, lens, sel, dtype, scale)
    both = kvp.paged_attention_decode_sparse(q, *pools, _dev(t), _dev(np.int32(lens)), _dev(sel),
                                             SCALE, **kw)
    kvp.check_device_error()
    assert torch.isfinite(both[:, 2:]).all()


@pytest.mark.parametrize("dtype,Hq,Hkv", [("f16", 4, 4), ("bf16", 8, 2)])
def test_decode_over_every_block_is_the_paged_decode(dtype, Hq, Hkv):
    kvp = _kvp()
    lens = [1, 200, 1025]
    qb, t, pools, vals, _ = _decode_case(57, lens, Hq, Hkv, 128, 16, dtype, dtype)
    sel = np.full((3, Hkv, 65), -1, np.int32)
    for s, n in enumerate(lens):
        sel[s, :, :-(-n // 16)] = np.arange(-(-n // 16))
    got = kvp.paged_attention_decode_sparse(from_bits(qb, dtype), *pools, _dev(t),
                                            _dev(np.int32(lens)), _dev(sel), SCALE)
    ref = _check_decode(to_bits(got), qb, vals, t, lens, sel, dtype, SCALE)
    assert np.allclose(ref, attention.paged_decode(to_f64(qb, dtype), *vals, t, lens, SCALE, 16))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_with_far_apart_logits_and_a_repeated_block(dtype):
    kvp = _kvp()
    lens = [400]
    qb, t, pools, vals, _ = _decode_case(59, lens, 4, 1, 64, 16, dtype, dtype)
    sel = np.int32([[[3, 24, 3, 0, 3]]])
    for scale in (8.0, -8.0, 0.0):  # logits of several hundred, and none
        got = kvp.paged_attention_decode_sparse(from_bits(qb, dtype), *pools, _dev(t),
                                                _dev(np.int32(lens)), _dev(sel), scale)
        _check_decode(to_bits(got), qb, vals, t, lens, sel, dtype, scale)
    kvp.check_device_error()


def test_decode_reports_bad_metadata():
    torch, kvp = _torch(), _kvp()
    lens = [100, 40]
    qb, t, pools, vals, _ = _decode_case(61, lens, 2, 1, 64, 16, "f16", "f16")
    q = from_bits(qb, "f16")
    good = np.int32([[[0, 2, -1, -1]], [[0, 1, 2, -1]]])

    def run(table, ln, sel, **kw):
        return kvp.paged_attention_decode_sparse(q, *pools, _dev(table), _dev(np.int32(ln)),
                                                 _dev(np.int32(sel)), SCALE, **kw)

    ref = run(t, lens, good)
    kvp.check_device_error()
    past = good.copy()
    past[0, 0, 2] = 7          # the context has blocks 0..6
    assert torch.equal(run(t, lens, past), ref) and "selected" in _raises("bounds")
    past[0, 0, 2] = 2**31 - 1
    assert torch.equal(run(t, lens, past), ref) and "selected" in _raises("bounds")
    bad = t.copy()
    bad[0, 4] = pools[0].shape[0]
    with_bad = good.copy()
    with_bad[0, 0, 3] = 4
    assert torch.equal(run(bad, lens, with_bad), ref) and "block table" in _raises("bounds")
    # a token of NaN within the context: the bound on the lengths changes nothing
    torch.testing.assert_close(run(t, [100, 41], good, max_context_len=100),
                               run(t, [100, 41], good), rtol=0, atol=0, equal_nan=True)
    kvp.check_device_error()
    run(t, [101, 40], good, max_context_len=100)
    assert "length" in _raises("bounds")
    none = run(t, [100, -3], good)
    assert "length" in _raises("bounds")
    assert torch.equal(none[0], ref[0]) and not none[1].any()
    with pytest.raises(ValueError):
        run(t, lens, good[:1])
    with pytest.raises(ValueError):
        run(t, lens, good, k_scale=torch.ones(1, device="cuda"))


# ---- together -------------------------------------------------------------------------------
def test_pools_past_32_bit_offsets():
    # 9 GiB of keys: the few blocks in use lie at both ends
    torch, kvp = _torch(), _kvp()
    NB, Hkv, bs, D = 294919, 8, 16, 128
    assert NB * Hkv * bs * D > 2**32
    kc, vc = (torch.empty((NB, Hkv, bs, D), dtype=torch.float16, device="cuda") for _ in range(2))
    bounds = torch.empty((NB, Hkv, 2, D), dtype=torch.float16, device="cuda")
    table = np.int32([[NB - 1, 0, NB - 2, 3]])
    T, cs = 50, np.concatenate([np.ones((64, 64)), np.zeros((64, 64))], 1).astype(np.float32)
    bits = workloads.normal_bits([71, 1], (T, 3 * Hkv, D), "f16")
    x = from_bits(bits, "f16")
    slots = np.array([int(table[0, i // bs]) * bs + i % bs for i in range(T)], np.int64)
    kvp.rope_reshape_and_cache(x[:, :Hkv], x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:], _dev(cs),
                               _dev(np.arange(T)), kc, vc, _dev(slots))
    lens = _dev(np.int32([T]))
    kvp.update_key_bounds(kc, bounds, _dev(table), lens)
    q = x[-1:, :Hkv].contiguous()
    sel = kvp.select_blocks(q, bounds, _dev(table), lens, block_size=bs, num_selected=3)
    out = kvp.paged_attention_decode_sparse(q, kc, vc, _dev(table), lens, sel, SCALE)
    kvp.check_device_error()
    ids = table[0].astype(np.int64)
    small = np.stack([to_f64(to_bits(kc[i]), "f16") for i in ids])
    smallv = np.stack([to_f64(to_bits(vc[i]), "f16") for i in ids])
    t2 = np.int32([[0, 1, 2, 3]])
    y = to_f64(bits, "f16")
    for i in range(T):
        assert np.array_equal(small[i // bs, :, i % bs], y[i, Hkv:2 * Hkv])
    b64 = sparse.key_bounds(np.zeros((4, Hkv, 2, D)), small, t2, [T])
    want = sparse.select_blocks(y[-1:, :Hkv], b64, t2, [T], bs, 3, 1, 1)
    assert np.array_equal(sel.cpu().numpy(), want)
    _check_decode(to_bits(out), bits[-1:, :Hkv], (small, smallv), t2, [T], want, "f16", SCALE)


@pytest.mark.parametrize("Hq,Hkv,dtype,cache,bs", [(4, 4, "f16", "f16", 16), (8, 2, "bf16", "bf16", 8),
                                                   (8, 2, "bf16", "e4m3", 32)])
def test_decode_steps_with_forks_over_a_block_pool(Hq, Hkv, dtype, cache, bs):
    """Prompts, forks and decode steps through the allocator: after each step every
    operator's result is the oracle's, on the oracle's own pools and bounds."""
    torch, kvp = _torch(), _kvp()
    D, NB, keep, rot, far = 128, 90, 6, 64, 600
    small = "f16" if cache == "e4m3" else dtype
    rng = np.random.default_rng(81)
    pool = kvp.BlockPool(NB, bs, Hkv, D, "fp8_e4m3" if cache == "e4m3" else dtype)
    shape = (NB, Hkv, bs, D)
    scales = [np.float32([0.02, 0.013][:Hkv] * 1)[:Hkv] for _ in range(2)] if cache == "e4m3" else None
    kw = dict(k_scale=_dev(scales[0]), v_scale=_dev(scales[1])) if scales else {}
    ct = torch.uint8 if cache == "e4m3" else _tdt(dtype)
    kc, vc = (torch.zeros(shape, dtype=ct, device="cuda") for _ in range(2))
    bounds = torch.zeros((NB, Hkv, 2, D), dtype=_tdt(small), device="cuda")
    ang = np.arange(far)[:, None] * 10000.0 ** (-np.arange(rot // 2) * 2 / rot)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    cs_d, step = _dev(cs), 0

    def values(p):
        if cache == "e4m3":
            return fp8.decode(p.cpu().numpy())
        return to_f64(to_bits(p), dtype)

    def forward(seqs, counts):
        """One step of new tokens for each sequence; checks all four operators."""
        nonlocal step
        step += 1
        slots, pos = [], []
        for s, n in zip(seqs, counts):
            at = pool.seq_len(s)
            slots += pool.append(s, n)
            pos += range(at, at + n)
        pairs = pool.take_copies()
        if pairs:
            kvp.copy_blocks(kc, vc, _dev(np.int32(pairs)))
        kv0, vv0 = values(kc), values(vc)
        T = len(slots)
        bits = workloads.normal_bits([82, step], (T, Hq + 2 * Hkv, D), dtype)
        x = from_bits(bits, dtype)
        q = kvp.rope_reshape_and_cache(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cs_d,
                                       _dev(np.int64(pos)), kc, vc, _dev(np.int64(slots)), **kw)
        y = to_f64(bits, dtype)
        kx = sparse.rotate(y[:, Hq:Hq + Hkv], cs[pos], False, np.float32)
        vx = y[:, Hq + Hkv:].astype(np.float32)
        for j, slot in enumerate(slots):
            for i, (ref, src) in enumerate(((kv0, kx), (vv0, vx))):
                if cache == "e4m3":
                    ref[slot // bs, :, slot % bs] = fp8.decode(fp8.quantize(src[j], scales[i][:, None]))
                else:
                    t = torch.from_numpy(src[j].copy()).to(_tdt(dtype))
                    ref[slot // bs, :, slot % bs] = t.double().numpy()
        assert np.array_equal(values(kc), kv0) and np.array_equal(values(vc), vv0)
        most = max(len(pool.block_table(s)) for s in seqs) + 1
        tables, lens = pool.build_batch(seqs, most)
        b0 = to_f64(to_bits(bounds), small)
        t_d, l_d = _dev(tables), _dev(lens)
        kvp.update_key_bounds(kc, bounds, t_d, l_d, new_tokens=_dev(np.int32(counts)),
                              max_new_tokens=max(counts))
        b0 = sparse.key_bounds(b0, kv0, tables, lens, counts)
        assert np.array_equal(to_f64(to_bits(bounds), small), b0)
        last = np.cumsum(counts) - 1
        ql = q[torch.from_numpy(last).cuda()].contiguous()
        qb = to_bits(ql)
        sel = kvp.select_blocks(ql, bounds, t_d, l_d, block_size=bs, num_selected=keep, num_recent=2)
        want = sparse.select_blocks(to_f64(qb, dtype), b0, tables, lens, bs, keep, 1, 2)
        assert np.array_equal(sel.cpu().numpy(), want)
        out = kvp.paged_attention_decode_sparse(ql, kc, vc, t_d, l_d, sel, SCALE, **kw)
        kvp.check_device_error()
        if scales:
            kv0, vv0 = (v * s.astype(np.float64)[:, None, None] for v, s in zip((kv0, vv0), scales))
        _check_decode(to_bits(out), qb, (kv0, vv0), tables, lens, want, dtype, SCALE)

    seqs = [pool.create() for _ in range(3)]
    forward(seqs, [1, 10 * bs + 3, 15 * bs - 1])
    seqs += [pool.fork(seqs[1]), pool.fork(seqs[2])]
    for _ in range(3):
        forward(seqs, [1] * 5)
    pool.release(seqs.pop(1))
    forward(seqs + [pool.create()], [2, 1, 1, bs + 1, 5])


def test_captured_and_replayed_on_another_stream():
    torch, kvp = _torch(), _kvp()
    lens = [700, 90, 1]
    qb, t, pools, vals, _ = _decode_case(91, lens, 8, 2, 128, 16, "f16", "f16")
    nb, bs, keep = pools[0].shape[0], 16, 9
    for p in pools:
        p.nan_to_num_(0.0)
    q, t_d, l_d = from_bits(qb, "f16"), _dev(t), _dev(np.int32(lens))
    new = torch.ones(3, dtype=torch.int32, device="cuda")
    rows = torch.randn((3, 12, 128), device="cuda").half()
    cs = torch.rand((1024, 128), device="cuda")
    pos = _dev(np.int64([n - 1 for n in lens]))
    slots = _dev(np.int64([int(t[s, (n - 1) // bs]) * bs + (n - 1) % bs for s, n in enumerate(lens)]))
    bounds = torch.zeros((nb, 2, 2, 128), dtype=torch.float16, device="cuda")
    q_out, sel = torch.empty_like(q), torch.empty((3, 2, keep), dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    kvp.update_key_bounds(pools[0], bounds, t_d, l_d)

    def step():
        kvp.rope_reshape_and_cache(rows[:, :8], rows[:, 8:10], rows[:, 10:], cs, pos, *pools, slots,
                                   q_out)
        kvp.update_key_bounds(pools[0], bounds, t_d, l_d, new_tokens=new, max_new_tokens=1)
        kvp.select_blocks(q_out, bounds, t_d, l_d, sel, block_size=bs, num_selected=keep)
        kvp.paged_attention_decode_sparse(q_out, *pools, t_d, l_d, sel, SCALE, out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(3):
        rows.copy_(torch.randn((3, 12, 128), generator=torch.Generator(device="cuda").manual_seed(i),
                               device="cuda").half())
        saved = [x.clone() for x in (*pools, bounds)]
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (*pools, bounds, q_out, sel, out)]
        for x, y in zip((*pools, bounds), saved):
            x.copy_(y)
        for x in (q_out, sel, out):
            x.zero_()
        step()
        torch.cuda.synchronize()
        for x, y in zip((*pools, bounds, q_out, sel, out), got):
            assert torch.equal(x, y)
    kvp.check_device_error()


def test_two_streams_at_once():
    torch, kvp = _torch(), _kvp()
    work = []
    for i in range(2):
        lens = [3000 + 100 * i, 17]
        qb, t, pools, vals, _ = _decode_case(95 + i, lens, 4, 1, 128, 16, "bf16", "bf16")
        sel = np.full((2, 1, 64), -1, np.int32)
        sel[0, 0] = np.sort(np.random.default_rng(i).permutation(187)[:64])
        sel[1, 0, 0] = 1
        work.append((from_bits(qb, "bf16"), pools, _dev(t), _dev(np.int32(lens)), _dev(sel)))
    alone = [kvp.paged_attention_decode_sparse(q, *p, t, l, s, SCALE) for q, p, t, l, s in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    outs = [[], []]
    for _ in range(20):
        for i, (q, p, t, l, s) in enumerate(work):
            with torch.cuda.stream(streams[i]):
                outs[i].append(kvp.paged_attention_decode_sparse(q, *p, t, l, s, SCALE))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in outs[i])
    kvp.check_device_error()
