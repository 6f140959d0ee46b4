"""Block-sparse decoding on the GPU where 16- and 32-bit numbers run out of range or of bits:
huge bounds and queries in the selection, large logits and far-apart or barely
representable weights in the attention. References are the fp64 oracle's."""

import numpy as np
import pytest

from oracle import sparse
from oracle.numerics import half_ulp
import workloads

pytestmark = pytest.mark.gpu


def _torch():
    import torch

    return torch


def _kvp():
    import paged_kv_cache_319_b200 as kvp

    return kvp


def _dev(x):
    return _torch().from_numpy(np.ascontiguousarray(x)).cuda()


def _tdt(dtype):
    torch = _torch()
    return {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[dtype]


def _put(x, dtype):
    """(device tensor of the rounded values, those values in fp64)."""
    t = _dev(np.asarray(x, np.float64)).to(_tdt(dtype))
    return t, t.double().cpu().numpy()


def _check_selection(q, q_dtype, bounds, bounds_dtype, bs, keep, sink=1, recent=1):
    kvp = _kvp()
    n = bounds.shape[0]
    table = np.random.default_rng(n).permutation(n).astype(np.int32)[None]
    qd, q = _put(q, q_dtype)
    bd, bounds = _put(bounds, bounds_dtype)
    assert np.isfinite(q).all() and np.isfinite(bounds).all()
    want = None
    for k in keep:
        got = kvp.select_blocks(qd, bd, _dev(table), _dev(np.int32([n * bs])), block_size=bs,
                                num_selected=k, num_sink=sink, num_recent=recent)
        kvp.check_device_error()
        want = sparse.select_blocks(q, bounds, table, [n * bs], bs, k, sink, recent)
        bad = np.setdiff1d(got.cpu().numpy(), want)
        assert np.array_equal(got.cpu().numpy(), want), (k, bad.size)


# ---- select_blocks: scores past fp32's range ------------------------------------------------
@pytest.mark.parametrize("exponent", [107, 109, 110, 112, 114, 120])
@pytest.mark.parametrize("n,D,Hq,keep", [(1000, 128, 1, (130, 600, 990)), (700, 64, 4, (20, 350)),
                                         (27000, 64, 1, (200,))])
def test_selection_of_huge_bounds_of_one_sign(exponent, n, D, Hq, keep):
    # a block's largest and smallest key are one value per channel, so that terms of both
    # signs cancel; sums of 2 D products reach 2^(exponent + 22) of the scaled weights
    rng = np.random.default_rng([exponent, n])
    v = rng.uniform(1, 2, (n, 1, D)) * 2.0**exponent * 2.0**rng.uniform(-3, 1, (n, 1, 1))
    _check_selection(rng.standard_normal((1, Hq, D)), "bf16", np.stack([v, v], 2), "bf16", 16, keep)


@pytest.mark.parametrize("n,huge,keep", [(500, 12, (8, 40, 300)), (500, 200, (100, 250)),
                                         (3000, 70, (20, 200))])
def test_selection_with_some_blocks_past_fp32(n, huge, keep):
    # +2^115 and -2^115 in two channels cancel in fp64; in fp32 they are inf - inf. What the
    # other channels add is lost or not by the order of the fp64 sum, so these blocks may be
    # kept or dropped: each of the 2 D additions is off by at most 2^-53 of the sum of the
    # terms' sizes, and no kept block may lie further than both errors below a dropped one.
    kvp = _kvp()
    rng = np.random.default_rng([n, huge])
    v = rng.standard_normal((n, 1, 64))
    at = rng.permutation(n)[:huge]
    v[at, 0, 0], v[at, 0, 4] = 2.0**115, -2.0**115
    qd, q = _put(np.ones((1, 1, 64)), "bf16")
    bd, bounds = _put(np.stack([v, v], 2), "bf16")
    table = np.random.default_rng(n).permutation(n).astype(np.int32)[None]
    score = sparse.block_scores(q[0], bounds, table[0], n)[0]
    err = 128 * 2.0**-53 * np.abs(bounds[table[0], 0, 0]).sum(1)
    for k in keep:
        got = kvp.select_blocks(qd, bd, _dev(table), _dev(np.int32([n * 8])), block_size=8,
                                num_selected=k, num_sink=1, num_recent=1).cpu().numpy()[0, 0]
        kvp.check_device_error()
        assert got[0] == 0 and got[-1] == n - 1 and (np.diff(got) > 0).all()
        kept = got[1:-1]
        dropped = np.setdiff1d(np.arange(n), got)
        assert (score + err)[kept].min() >= (score - err)[dropped].max()


@pytest.mark.parametrize("n,huge,keep", [(500, 12, (8, 40, 300)), (500, 200, (100, 250)),
                                         (3000, 70, (20, 200))])
def test_selection_with_exact_sums_past_fp32(n, huge, keep):
    # the same with the other channels multiples of 2^80: every fp64 sum is exact
    rng = np.random.default_rng([n, huge])
    v = rng.integers(-127, 128, (n, 1, 64)) * 2.0**80
    at = rng.permutation(n)[:huge]
    v[at, 0, 0], v[at, 0, 4] = 2.0**115, -2.0**115
    _check_selection(np.ones((1, 1, 64)), "bf16", np.stack([v, v], 2), "bf16", 8, keep)


@pytest.mark.parametrize("bounds_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("Hq,keep", [(4, (90, 300)), (16, (30,))])
def test_selection_of_query_groups_past_fp32(Hq, keep, bounds_dtype):
    # the group's sum of a channel passes fp32's largest number though every query is finite
    rng = np.random.default_rng([Hq, 71])
    q = rng.uniform(1, 1.9, (1, Hq, 128)) * 2.0**127 * rng.choice([-1, 1], (1, 1, 128))
    hi = rng.integers(-60, 127, (700, 1, 128)).astype(np.float64)
    lo = hi - rng.integers(0, 60, hi.shape)
    _check_selection(q, "bf16", np.stack([hi, lo], 2), bounds_dtype, 16, keep)


@pytest.mark.parametrize("bounds_dtype", ["f16", "bf16"])
def test_selection_of_query_groups_past_fp32_among_bad_block_ids(bounds_dtype):
    # 60 of 100 table entries lie outside the pool and are scored last
    kvp = _kvp()
    rng = np.random.default_rng(76)
    qd, q = _put(rng.uniform(1, 1.9, (1, 16, 128)) * 2.0**127, "bf16")
    hi = rng.integers(1, 127, (100, 1, 128)).astype(np.float64)
    bd, bounds = _put(np.stack([hi, hi], 2), bounds_dtype)
    table = np.arange(100, dtype=np.int32)[None]
    bad = rng.permutation(100)[:60]
    table[0, bad] += 100
    got = kvp.select_blocks(qd, bd, _dev(table), _dev(np.int32([1600])), block_size=16,
                            num_selected=20, num_sink=0, num_recent=0).cpu().numpy()[0, 0]
    with pytest.raises(kvp.KvpError):
        kvp.check_device_error()
    score = sparse.block_scores(q[0], bounds, np.arange(100), 100)[0]
    score[bad] = -np.inf
    assert np.array_equal(got, np.sort(np.argsort(-score, kind="stable")[:20]))


# ---- paged_attention_decode_sparse --------------------------------------------------------
# Rows that take the kernel's three forms: a cluster of wide CTAs, a CTA, and a warp per row.
FORMS = [(1, 384), (200, 384), (3000, 6)]  # (sequences, 16-token tiles in the list)


def _attend(q, q_dtype, k, v, cache, scale, seqs, **kw):
    """Every sequence lists all blocks of the same context; keys and values [Hkv, tokens, D] in
    blocks of 16. Returns row 0 and the values that the kernel read."""
    torch, kvp = _torch(), _kvp()
    Hkv, tokens, D = k.shape
    NB = tokens // 16
    kd, k = _put(np.ascontiguousarray(k.reshape(Hkv, NB, 16, D).transpose(1, 0, 2, 3)), cache)
    vd, v = _put(np.ascontiguousarray(v.reshape(Hkv, NB, 16, D).transpose(1, 0, 2, 3)), cache)
    qd, q = _put(q, q_dtype)
    if cache == "e4m3":
        for name in ("k_scale", "v_scale"):
            kw[name] = _dev(np.float32(kw.get(name, np.ones(Hkv))))
        k = k * kw["k_scale"].double().cpu().numpy()[:, None, None]
        v = v * kw["v_scale"].double().cpu().numpy()[:, None, None]
    table = torch.arange(NB, dtype=torch.int32, device="cuda").repeat(seqs, 1)
    sel = table[:, None].repeat(1, Hkv, 1)
    lens = torch.full((seqs,), tokens, dtype=torch.int32, device="cuda")
    got = kvp.paged_attention_decode_sparse(qd[None].repeat(seqs, 1, 1), kd, vd, table, lens, sel,
                                            float(scale), **kw)
    kvp.check_device_error()
    assert torch.equal(got, got[:1].expand_as(got))
    return got[0].double().cpu().numpy(), (q[None], k, v, table[:1].cpu().numpy(), [tokens],
                                           sel[:1].cpu().numpy(), float(scale))


TYPES = [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")]


@pytest.mark.parametrize("seqs,tiles", FORMS)
@pytest.mark.parametrize("dtype,cache", TYPES)
def test_decode_of_logits_with_few_bits_below_one(dtype, cache, seqs, tiles):
    # logits of 2^27, 2^27 + 16 and 2^27 + 32 in units of ln 2, neighbours in fp32: a reference
    # that lags by 8 cannot be added to. The last third of the tokens has all the weight but
    # 2^-16; what is left are the values' mean and its roundings.
    rng = np.random.default_rng(72)
    tokens = tiles * 16
    third = np.arange(tokens) // (tokens // 3)
    q, k = np.zeros((1, 128)), np.zeros((1, tokens, 128))
    v = rng.integers(-8, 9, (1, tokens, 128)) / 8
    kw = {}
    if cache == "e4m3":
        q[0, :2], k[0, :, 0], k[0, :, 1], kw["k_scale"] = [2.0**15, 1], 256, third, [16.0]
    else:
        q[0, :2], k[0, :, 0], k[0, :, 1] = [2.0**14, 16], 2.0**13, third
    scale = np.float32(np.log(2.0))  # times log2(e) it is 1 in fp32
    got, case = _attend(q, dtype, k, v, cache, scale, seqs, **kw)
    ref = sparse.decode_sparse(*case)[0]
    assert (np.abs(got - ref) <= half_ulp(ref, dtype) + 2.0**-15).all(), got


def _weight_step(dtype, cache):
    """Half a step of the weights in the second product: two 16-bit parts, of bf16 where the
    cache is bf16, else of fp16; each is off by at most 2^-8 or 2^-11 of what it stands for."""
    return 2.0**-16 if cache == "bf16" else 2.0**-22


def _check_attend(got, case, dtype, cache, **kw):
    ref = sparse.decode_sparse(*case)[0]
    err = sparse.decode_error(*case, _weight_step(dtype, cache), **kw)[0]
    bad = np.abs(got - ref) > err + half_ulp(np.abs(ref) + err, dtype)
    assert not bad.any(), (bad.sum(), (np.abs(got - ref) / err).max())


@pytest.mark.parametrize("seqs,tiles", FORMS)
@pytest.mark.parametrize("dtype,cache", TYPES)
def test_decode_of_weights_beside_a_half_step(dtype, cache, seqs, tiles):
    # of 16 tokens one has weight 1 and the others 0.5 (1 + 0.98 h), h the half step of one
    # 16-bit number: rounded to one, all of them lose 0.98 h
    rng = np.random.default_rng(73)
    tokens, Hkv = tiles * 16, 8
    h = 2.0**-8 if cache == "bf16" else 2.0**-11
    k = np.zeros((Hkv, tokens, 128))
    k[:, np.arange(tokens) % 16 != 5, 0] = 1
    q = np.zeros((2 * Hkv, 128))
    q[:, 0] = 1
    v = np.zeros((Hkv, tokens, 128)) + rng.uniform(1, 2, (Hkv, 1, 128))
    v[:, np.arange(tokens) % 16 == 5] = 0
    kw = {} if cache != "e4m3" else dict(v_scale=rng.uniform(1, 2, Hkv))
    got, case = _attend(q, dtype, k, v, cache, np.log(0.5 * (1 + 0.98 * h)), seqs, **kw)
    _check_attend(got, case, dtype, cache)


@pytest.mark.parametrize("seqs,tiles", FORMS)
@pytest.mark.parametrize("G", [1, 3, 12])
@pytest.mark.parametrize("dtype,cache", TYPES)
def test_decode_within_the_error_of_two_part_weights(dtype, cache, G, seqs, tiles):
    rng = np.random.default_rng([74, G])
    k, v = rng.standard_normal((2, 2, tiles * 16, 128))
    kw = {} if cache != "e4m3" else dict(k_scale=[1.5, 0.7], v_scale=[0.8, 1.3])
    got, case = _attend(rng.standard_normal((2 * G, 128)), dtype, k, v, cache, 128**-0.5, seqs, **kw)
    _check_attend(got, case, dtype, cache)


@pytest.mark.parametrize("seqs,tiles", FORMS + [(1, 30)])
@pytest.mark.parametrize("nats", [17.4, 18.5, 20.0])
@pytest.mark.parametrize("dtype,cache", TYPES)
def test_decode_of_one_strong_token_over_a_weak_tail(dtype, cache, nats, seqs, tiles):
    # each of the others has a weight of 2^-25 to 2^-29 of the strong token's; in the even
    # channels they are all there is
    rng = np.random.default_rng(75)
    tokens, strong = tiles * 16, tiles * 8 + 3
    k = np.zeros((1, tokens, 128))
    k[0, :, 0] = np.arange(tokens) != strong
    q = np.zeros((1, 128))
    q[0, 0] = 1
    v = rng.integers(8, 16, (1, tokens, 128)) / 8
    v[0, strong, ::2] = 0
    got, case = _attend(q, dtype, k, v, cache, -nats, seqs)
    # a part is off by at most 2^-25, half of fp16's smallest number, and the strongest
    # weight is 2^7 or more; bf16 has fp32's range
    _check_attend(got, case, dtype, cache, p_floor=0.0 if cache == "bf16" else 2.0**-32)
