"""Decode over bf16 caches, dense and paged, at scales of any sign: negative, zero, and large
enough that the scores of a row spread over more than fp32's exponentials reach."""
import math

import numpy as np
import pytest

import oracle
import paged
from helpers import ETA, U_BF16, bf16_ulp, bits_of, f64, fp32_gamma
from test_gpu_paged import decode_inputs, dev, ok_status, poison, to_torch

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# lens, Hq, Hkv, D, page size: whole and ragged tiles, one token, none, several splits
SHAPES = [([200, 37, 128, 1, 0], 8, 2, 64, 32), ([1300, 130], 28, 4, 128, 16), ([90, 2], 64, 1, 128, 128)]


def check(o, lse, q, dense, lens, scale, partial):
    """Every element against the fp64 oracle: the weights' rounding to bf16 (2^-8 of the row's
    dispersion, at most P|V| + |O|), twice the scores' error e_s, half a step of the result, fp32
    sums, and `partial` of P|V| for partial results that are rounded to bf16.  e_s: 16 tensor-core
    and scale steps in fp32 (2^-23 each) on |scale| max_j sum |q k|, and the exponential's 2^-22.
    lse: e_s, fp32 sums, and the logarithm's and the last roundings, 2^-20 and 2^-22 of itself."""
    cl = np.array(lens, dtype=np.int32)
    o_r, l_r = oracle.decode(q, *dense, cl, scale)
    oa_r, _ = oracle.decode(q, dense[0], np.abs(dense[1]), cl, scale)
    og, lg = f64(bits_of(o)).reshape(q.shape), lse.double().cpu().numpy()
    G = q.shape[1] // dense.shape[3]
    for b, L in enumerate(lens):
        if L == 0:
            assert (og[b] == 0).all() and np.isneginf(lg[b]).all()
            continue
        for h in range(q.shape[1]):
            A = abs(scale) * (np.abs(dense[0, b, :L, h // G]) @ np.abs(q[b, h])).max()
            e_s = A * 16 * 2.0 ** -23 + 2.0 ** -22
            tol = 0.5 * bf16_ulp(np.maximum(np.abs(og[b, h]), np.abs(o_r[b, h]))) \
                + (U_BF16 + ETA + 2 * e_s) * (oa_r[b, h] + np.abs(o_r[b, h])) + (fp32_gamma(L) + partial) * oa_r[b, h]
            err = np.abs(og[b, h] - o_r[b, h])
            assert (err <= tol).all(), (b, h, err.max(), og[b, h][:4], o_r[b, h][:4])
            assert abs(lg[b, h] - l_r[b, h]) <= e_s + fp32_gamma(L) + 2.0 ** -20 + 2.0 ** -22 * abs(l_r[b, h]), (b, h, lg[b, h], l_r[b, h])


@pytest.mark.parametrize("scale", [-0.3, 0.0, -0.0, -3.0, 3.0, -1e-30])
@pytest.mark.parametrize("case", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_decode_at_any_scale(case, scale):
    from long_context_attention_fwd_b200 import ops
    lens, Hq, Hkv, D, ps = case
    rng, q, kv = decode_inputs(lens, Hq, Hkv, D, 51)
    table, P = paged.table_for(rng, lens, ps, width=-(-max(lens) // ps) + 1)
    B, cap = len(lens), max(lens) + 70
    kp, vp = poison((P, ps, Hkv, D), torch.bfloat16), poison((P, ps, Hkv, D), torch.bfloat16)
    kd, vd = poison((B, cap, Hkv, D), torch.bfloat16), poison((B, cap, Hkv, D), torch.bfloat16)
    dense = np.zeros((2, B, cap, Hkv, D))
    for b, L in enumerate(lens):
        if L == 0:
            continue
        k, v = to_torch(kv[b][0]), to_torch(kv[b][1])
        pos = torch.arange(L, device="cuda")
        pg = dev(table[b])[pos // ps].long()
        kp[pg, pos % ps], vp[pg, pos % ps] = k, v
        kd[b, :L], vd[b, :L] = k, v
        dense[:, b, :L] = kv[b]
    cl = dev(np.array(lens, dtype=np.int32))
    scale = float(np.float32(scale))
    got = ops.attn_decode_paged(to_torch(q), kp, vp, dev(table), cl, scale=scale)
    ok_status()
    check(*got, q, dense, lens, scale, 0.0)
    got = ops.attn_decode(to_torch(q), kd, vd, cl, scale=scale)
    ok_status()
    check(*got, q, dense, lens, scale, 2.0 ** -8)
