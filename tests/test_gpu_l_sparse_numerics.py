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
    # +2^115 and -2^115 in two channels cancel in fp64; in fp32 they are inf - inf
    rng = np.random.default_rng([n, huge])
    v = rng.standard_normal((n, 1, 64))
    at = rng.permutation(n)[:huge]
    v[at, 0, 0], v[at, 0, 4] = 2.0**115, -2.0**115
    q = np.ones((1, 1, 64))
    _check_selection(q, "bf16", np.stack([v, v], 2), "bf16", 8, keep)
