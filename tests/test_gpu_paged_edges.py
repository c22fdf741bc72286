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
