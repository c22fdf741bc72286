"""The forward in bf16 and e4m3, and the gradients, at scales of any sign: masked scores stay masked
and the softmax's reference stays the row's largest scaled score."""
import numpy as np
import pytest

import oracle
from helpers import ETA, TOL_GRAD, TOL_LSE, U_BF16, DeviceRun, bf16_ulp, fp32_gamma, make_case, oracle_args, rel_l2
from test_gpu_fp8 import _check_rows, _fp8_inputs, _run
from long_context_attention_fwd_b200 import inputs as I

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SHAPES = [dict(B=1, Hq=4, Hkv=2, S=300, D=128, causal=True), dict(B=2, Hq=2, Hkv=2, S=200, D=64, causal=True),
          dict(B=1, Hq=2, Hkv=1, S=129, D=128, causal=False), dict(B=0, Hq=3, Hkv=1, S=0, D=64, causal=True, lens=[1, 130, 257])]


@pytest.mark.parametrize("scale", [-0.2, 0.0, -2.5, -1e-30])
@pytest.mark.parametrize("shape", SHAPES, ids=["causal_D128", "causal_D64", "full_ragged", "packed"])
def test_forward_and_gradients_at_any_scale(shape, scale):
    """O: the weights' rounding (2^-8 of the dispersion, at most P|V| + |O|), twice the scores'
    error, half a step, fp32 sums.  The scores' error: 16 fp32 steps (2^-23 each) on |scale| max
    sum |q k|, and the exponential's 2^-22; it adds to the log-sum's bar."""
    w = make_case(**shape, scale=float(np.float32(scale)), seed=97)
    r = DeviceRun(w)
    g = r.np_out()
    q, k, v, do, kw = oracle_args(w, r.x)
    o_r, l_r = oracle.fwd(q, k, v, w.causal, w.softmax_scale, **kw)
    oa_r, _ = oracle.fwd(q, k, np.abs(v), w.causal, w.softmax_scale, **kw)
    qk = np.abs(q).sum(-1).max() * np.abs(k).max()
    e_s = abs(scale) * qk * 16 * 2.0 ** -23 + 2.0 ** -22
    tol = 0.5 * bf16_ulp(np.maximum(np.abs(o_r), np.abs(g["o"]))) + (U_BF16 + ETA + 2 * e_s) * (oa_r + np.abs(o_r)) \
        + fp32_gamma(512) * oa_r
    assert (np.abs(g["o"] - o_r) <= tol).all()
    assert np.abs(g["lse"] - l_r).max() <= TOL_LSE + e_s
    for n, x in zip(("dq", "dk", "dv"), oracle.bwd(q, k, v, do, w.causal, w.softmax_scale, **kw)):
        assert rel_l2(g[n], x) <= TOL_GRAD + 2 * e_s, n


@pytest.mark.parametrize("scale,sign", [(-0.2, 1), (0.0, 1), (0.1, -1)])
@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[2]], ids=["causal", "full_ragged"])
def test_fp8_forward_at_any_scale(shape, scale, sign):
    """A negative or zero scale, and a negative factor of q."""
    w = make_case(**shape, scale=float(np.float32(scale)), seed=98)
    x, out = _fp8_inputs(w)
    b, d, val = out["q"]
    out["q"] = (b, sign * d, sign * val)
    o_g, lse_g = _run(w, out)
    q, k, v = (out[n][2].reshape(w.tokens, -1, w.D) for n in ("q", "k", "v"))
    o_r, l_r = oracle.fwd(q, k, v, w.causal, w.softmax_scale, B=w.B, S=w.S)
    rows = [(b, h, i) for b in range(w.B) for h in range(w.Hq) for i in range(w.S)]
    _check_rows(w, out, o_g, lse_g, rows, [o_r[b * w.S + i, h] for b, h, i in rows], [l_r[b, h, i] for b, h, i in rows])
