"""Paged caches on the GPU at the edges of what their documentation allows."""
import math

import numpy as np
import pytest

import paged
from helpers import bits_of, f64
from test_gpu_paged import (check_decode4, decode_inputs, dev, ok_status, pages4_of, poison, rope_table,
                            status, to_torch, values_of)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("lens", [[20, 33, 7], [1 << 30, 31], [33], [20] * 40 + [1000]])
def test_decode_records_a_length_past_the_table(four, lens):
    """A length that the table has no pages for is recorded, once and with the call's site; the
    sequence attends to the tokens that its table holds, the others are as always."""
    from long_context_attention_fwd_b200 import capi, ops
    ps, width, Hkv, D = 16, 2, 2, 64
    B, P = len(lens), 2 * len(lens)
    gen = torch.Generator(device="cuda").manual_seed(5)
    table = torch.randperm(P, generator=gen, device="cuda").to(torch.int32).view(B, width).contiguous()
    kv = [torch.randn(P, ps, Hkv, D, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    q = torch.randn(B, 4, D, generator=gen, device="cuda").bfloat16()
    if four:
        pages = ops.kv4_pages(P, ps, Hkv, D)
        ops.attn_append_kv4(kv[0].view(-1, Hkv, D), kv[1].view(-1, Hkv, D), pages,
                            dev(np.arange(P, dtype=np.int32)[:, None]),
                            torch.full((P,), ps, dtype=torch.int32, device="cuda"),
                            cu_seqlens=dev(np.arange(0, P * ps + 1, ps, dtype=np.int32)))
        run = lambda n: ops.attn_decode_kv4(q, pages, table, n)      # noqa: E731
    else:
        run = lambda n: ops.attn_decode_paged(q, *kv, table, n)      # noqa: E731
    lens = np.array(lens, dtype=np.int32)
    want = run(dev(np.minimum(lens, ps * width)))
    ok_status()
    got = run(dev(lens))
    st, site = status()
    assert st == capi.ATTN_ERR_INVALID_ARG and site == (0x503 if four else 0x502)
    ok_status()
    assert same(got, want)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("B", [1, 3, 32, 33, 100])
@pytest.mark.parametrize("length", [0, -5])
def test_decode_of_empty_sequences_only(four, B, length):
    """A batch without a token: outputs 0, log-sums minus infinity, nothing else touched; also in a
    captured step whose sequences grow between replays."""
    from long_context_attention_fwd_b200 import ops
    Hq, Hkv, D, ps, n = 8, 2, 128, 16, 5
    gen = torch.Generator(device="cuda").manual_seed(7)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    q = torch.randn(B, Hq, D, generator=gen, device="cuda").bfloat16()
    k, v = (torch.randn(B * n, Hkv, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    full = torch.full((B,), n, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    if four:
        pool = (poison((B, Hkv, 1, 18 * D), torch.uint8),)
    else:
        pool = (poison((B, ps, Hkv, D), torch.bfloat16), poison((B, ps, Hkv, D), torch.bfloat16))
    append, decode = (ops.attn_append_kv4, ops.attn_decode_kv4) if four else (ops.attn_append_kv, ops.attn_decode_paged)
    append(k, v, *pool, table, full, cu_seqlens=cu)
    want = decode(q, *pool, table, full)
    lens = torch.full((B,), length, dtype=torch.int32, device="cuda")
    o, lse = poison((B, Hq, D), torch.bfloat16), poison((B, Hq), torch.float32)
    decode(q, *pool, table, lens, out=o, lse=lse)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        decode(q, *pool, table, lens, out=o, lse=lse)
    for m in (length, n, 0):
        lens.fill_(m)
        o.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        if m == n:
            assert same((o, lse), want)
        else:
            assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    ok_status()
    del g


@pytest.mark.parametrize("qe,ke,scale,positive", [
    (119, -116, None, False), (122, -119, None, True), (126, -110, 2.0 ** -14, True), (100, -97, None, True),
    (-100, 100, None, False)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_4bit_large_queries(qe, ke, scale, positive, D):
    """Queries up to 2^127 over keys so small that the scores are ordinary; all of one sign, so that
    their sums leave fp32."""
    from long_context_attention_fwd_b200 import ops
    lens, Hq, Hkv, ps = [200, 37], 12, 2, 32
    rng, q, kv = decode_inputs(lens, Hq, Hkv, D, 63)
    if positive:
        q = np.minimum(np.abs(q), 1.9)
    q = paged.bf16(q * 2.0 ** qe)
    for k, _ in kv:
        k[:] = paged.bf16(k * 2.0 ** ke)
    table, P = paged.table_for(rng, lens, ps)
    pages, vals = pages4_of(kv, lens, table, P, ps, Hkv, D)
    o, lse = ops.attn_decode_kv4(to_torch(q), dev(pages), dev(table), dev(np.array(lens, dtype=np.int32)), scale=scale)
    ok_status()
    check_decode4(o, lse, q, vals, lens, Hkv, D, 1 / math.sqrt(D) if scale is None else scale)


@pytest.mark.parametrize("heads", [(7, 1), (20, 1)], ids=["7", "20"])
@pytest.mark.parametrize("e0,e1,by_token", [(0, -22, False), (0, 24, False), (-15, 15, False), (20, -20, False),
                                            (-40, 40, False), (0, -30, True), (15, -15, True), (30, -30, True)])
def test_decode_4bit_groups_of_very_different_steps(heads, e0, e1, by_token):
    """The two groups of 64 elements of V differ in size by 2^22 to 2^80, all over or, by token, in
    turn: each group's outputs are held to its own size, with scores that rise and fall along the
    sequence and differ from head to head."""
    from long_context_attention_fwd_b200 import ops
    (Hq, Hkv), D, ps, lens = heads, 128, 32, [900, 64, 3]
    rng, q, kv = decode_inputs(lens, Hq, Hkv, D, 61)
    for b, L in enumerate(lens):
        k, v = kv[b]
        k[:] = paged.bf16(k * (1 + 15 * np.abs(np.sin(np.arange(L) / 90))[:, None, None]))
        size = np.empty((L, 1, D))
        size[:, :, :64], size[:, :, 64:] = 2.0 ** e0, 2.0 ** e1
        if by_token:
            size[1::3] = size[1::3, :, ::-1]
        v[:] = paged.bf16(v * size)
    table, P = paged.table_for(rng, lens, ps)
    pages, vals = pages4_of(kv, lens, table, P, ps, Hkv, D)
    o, lse = ops.attn_decode_kv4(to_torch(q), dev(pages), dev(table), dev(np.array(lens, dtype=np.int32)))
    ok_status()
    check_decode4(o, lse, q, vals, lens, Hkv, D, 1 / math.sqrt(D))


@pytest.mark.parametrize("heads", [(7, 1), (20, 1)], ids=["7", "20"])
@pytest.mark.parametrize("e0,e1", [(0, -5), (6, 0), (0, -8), (-10, 0), (0, -16), (60, -50), (-70, 40)])
def test_decode_4bit_groups_of_different_steps_all_along(heads, e0, e1):
    """From alike to far apart, with few and many tokens of the same weight and one of all."""
    from long_context_attention_fwd_b200 import ops
    (Hq, Hkv), D, ps, lens = heads, 128, 64, [1500, 130, 65]
    rng, q, kv = decode_inputs(lens, Hq, Hkv, D, 62)
    for b, mult in enumerate((1, 0, 40)):
        k, v = kv[b]
        k[:] = paged.bf16(k * mult)
        v[..., :64], v[..., 64:] = paged.bf16(v[..., :64] * 2.0 ** e0), paged.bf16(v[..., 64:] * 2.0 ** e1)
    table, P = paged.table_for(rng, lens, ps)
    pages, vals = pages4_of(kv, lens, table, P, ps, Hkv, D)
    o, lse = ops.attn_decode_kv4(to_torch(q), dev(pages), dev(table), dev(np.array(lens, dtype=np.int32)))
    ok_status()
    check_decode4(o, lse, q, vals, lens, Hkv, D, 1 / math.sqrt(D))


@pytest.mark.parametrize("heads", [(7, 1), (12, 1)], ids=["7", "12"])
@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("kind", ["small", "zero", "equal"])
def test_decode_4bit_one_token_takes_a_head(heads, first, kind):
    """One head sees one token only, whose steps in one group are 2^-30 of the others' or 0 (elements
    all zero or all equal), while the other heads see all tokens; then the token is the last one."""
    from long_context_attention_fwd_b200 import ops
    (Hq, Hkv), D, ps, lens = heads, 128, 16, [400, 400]
    rng, q, kv = decode_inputs(lens, Hq, Hkv, D, 64)
    group = slice(64 * first, 64 * first + 64)
    for b, at in enumerate((5, 399)):
        k, v = kv[b]
        k[at, 0] = paged.bf16(q[b, 0] * 6)
        x = v[at, 0, group]
        v[at, 0, group] = {"small": paged.bf16(x * 2.0 ** -30), "zero": 0 * x, "equal": 0 * x + 0.75}[kind]
    table, P = paged.table_for(rng, lens, ps)
    pages, vals = pages4_of(kv, lens, table, P, ps, Hkv, D)
    o, lse = ops.attn_decode_kv4(to_torch(q), dev(pages), dev(table), dev(np.array(lens, dtype=np.int32)))
    ok_status()
    check_decode4(o, lse, q, vals, lens, Hkv, D, 1 / math.sqrt(D))


@pytest.mark.parametrize("first", [0, 1])
def test_decode_4bit_a_group_without_steps(first):
    """A group of V that is constant in every token: its outputs are the weighted minima."""
    from long_context_attention_fwd_b200 import ops
    Hq, Hkv, D, ps, lens = 8, 2, 128, 32, [700, 31]
    rng, q, kv = decode_inputs(lens, Hq, Hkv, D, 65)
    for _, v in kv:
        v[..., 64 * first:64 * first + 64] = paged.bf16(rng.normal(size=v.shape[:2] + (1,)))
    table, P = paged.table_for(rng, lens, ps)
    pages, vals = pages4_of(kv, lens, table, P, ps, Hkv, D)
    o, lse = ops.attn_decode_kv4(to_torch(q), dev(pages), dev(table), dev(np.array(lens, dtype=np.int32)))
    ok_status()
    check_decode4(o, lse, q, vals, lens, Hkv, D, 1 / math.sqrt(D))


def test_decode_4bit_step_by_step_against_64_bits():
    """Tokens appended one by one with the rotation, after prompts of two lengths: every decode is
    the softmax in 64 bits over the values that the pages then hold, key by key and to fp16's
    rounding of the weights."""
    from long_context_attention_fwd_b200 import ops
    lens, Hq, Hkv, D, ps, steps = [70, 33, 0], 8, 2, 128, 32, 4
    B, total = len(lens), [n + steps for n in lens]
    rng = np.random.default_rng(71)
    table, P = paged.table_for(rng, total, ps)
    rope = tuple(dev(t) for t in rope_table(128, D // 2, 72))
    pages = poison((P, Hkv, ps // 16, 18 * D), torch.uint8)
    done = np.zeros(B, dtype=np.int32)
    for new in [lens] + [[1] * B] * steps:
        x = to_torch(paged.bf16(2 * rng.normal(size=(sum(new), Hq + 2 * Hkv, D))))
        done = done + np.array(new, dtype=np.int32)
        cu = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
        q = ops.attn_append_kv4(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pages, dev(table), dev(done), q=x[:, :Hq],
                                rope=rope, cu_seqlens=cu)
        if new != [1] * B:
            continue
        o, lse = ops.attn_decode_kv4(q, pages, dev(table), dev(done))
        ok_status()
        qf = f64(bits_of(q)).reshape(B, Hq, D)
        check_decode4(o, lse, qf, values_of(table, pages.cpu().numpy(), ps, done.tolist(), D), done.tolist(), Hkv, D,
                      1 / math.sqrt(D))


def test_append_4bit_differences_are_rounded_to_fp32():
    """Elements next to the middle between two codes by less than fp32 keeps of x - m: the code is
    that of the rounded difference, ties to even."""
    from long_context_attention_fwd_b200 import ops
    x = np.zeros((6, 1, 64))
    tiny = 2.0 ** -30
    for t, lo in enumerate([-7.5, -8.5, -0.5, -14.5, tiny, -tiny]):    # steps of 1
        x[t, 0, :5] = lo, (lo + 15 if t < 4 else 15), tiny, -tiny if t != 4 else tiny, 0.0 if t != 4 else tiny
        x[t, 0, 5:] = 7.5 if t >= 4 else lo
        x[t, 0, 6:] = 6.5 if t >= 4 else lo
    assert np.array_equal(paged.bf16(x), x)
    pages = poison((1, 1, 1, 18 * 64), torch.uint8)
    k = to_torch(x)
    cl, cu = dev(np.array([6], dtype=np.int32)), dev(np.array([0, 6], dtype=np.int32))
    ops.attn_append_kv4(k, k, pages, dev(np.zeros((1, 1), dtype=np.int32)), cl, cu_seqlens=cu)
    ok_status()
    got = paged.load4(pages.cpu().numpy(), [0], 16, 6, 64)
    x32 = x.astype(np.float32)
    lo = x32.min(-1, keepdims=True)
    step = ((x32.max(-1, keepdims=True) - lo) / np.float32(15)).astype(np.float64)
    assert (paged.bf16(step) == 1).all()
    want = np.rint((x32 - lo).astype(np.float64)).astype(np.uint8)
    for w in "kv":
        assert np.array_equal(got[w][0], want) and (got[w][1] == 1).all()


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_attention_over_what_the_4bit_cache_keeps(D):
    """Whole prompts: appended, read back and attended to as one packed batch, rotated q and all."""
    import oracle
    from helpers import TOL_LSE, o_error_report
    from long_context_attention_fwd_b200 import ops
    lens, Hq, Hkv, ps = [70, 1, 33, 130], 8, 2, 16
    rng = np.random.default_rng(81)
    table, P = paged.table_for(rng, lens, ps)
    cu_h = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T, cu, cl, tb = int(cu_h[-1]), dev(cu_h), dev(np.array(lens, dtype=np.int32)), dev(table)
    x = to_torch(paged.bf16(0.5 * rng.normal(size=(T, Hq + 2 * Hkv, D))))
    pages = poison((P, Hkv, ps // 16, 18 * D), torch.uint8)
    rope = tuple(dev(t) for t in rope_table(128 + 16, D // 2, 82))
    q = ops.attn_append_kv4(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pages, tb, cl, q=x[:, :Hq], rope=rope, cu_seqlens=cu)
    k, v = ops.attn_gather_kv4(pages, tb, cl, cu, T)
    o, lse = ops.attn_fwd(q, k, v, causal=True, cu_seqlens=cu)
    ok_status()
    qf, kf, vf = (f64(bits_of(t)).reshape(t.shape) for t in (q, k, v))
    o_r, l_r = oracle.fwd(qf, kf, vf, True, 1 / math.sqrt(D), cu_seqlens=cu_h)
    oa_r, _ = oracle.fwd(qf, kf, np.abs(vf), True, 1 / math.sqrt(D), cu_seqlens=cu_h)
    rep = o_error_report(f64(bits_of(o)).reshape(o.shape), o_r, oa_r, nkeys=max(lens))
    assert rep["n_over_model"] == 0, rep
    assert np.abs(lse.double().cpu().numpy() - l_r).max() <= TOL_LSE


@pytest.mark.parametrize("heads", [(7, 1), (12, 1)], ids=["7", "12"])
@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 60, 2.0 ** 90])
def test_decode_4bit_a_token_of_large_equal_elements(heads, first, size):
    """One token's groups are constant, and so large in one group that its minima set the softmax's
    reference: the other group's outputs keep what the other tokens give them."""
    from long_context_attention_fwd_b200 import ops
    (Hq, Hkv), D, ps, lens = heads, 128, 16, [300, 40]
    rng, q, kv = decode_inputs(lens, Hq, Hkv, D, 66)
    for (_, v), at in zip(kv, (7, 39)):
        v[at, 0, :] = 0.5
        v[at, 0, 64 * first:64 * first + 64] = size
    table, P = paged.table_for(rng, lens, ps)
    pages, vals = pages4_of(kv, lens, table, P, ps, Hkv, D)
    o, lse = ops.attn_decode_kv4(to_torch(q), dev(pages), dev(table), dev(np.array(lens, dtype=np.int32)))
    ok_status()
    check_decode4(o, lse, q, vals, lens, Hkv, D, 1 / math.sqrt(D))
