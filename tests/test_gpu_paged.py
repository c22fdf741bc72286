"""Paged key/value caches on the GPU: append, gather, decode over bf16 and over 4-bit pages,
against plain models in 64 bits (tests/paged.py, the fp64 oracle).

Pools start as 0xFF bytes (NaN as bf16 and as scales), and tables hold pages that do not exist
past each sequence's length, so that a read or a write out of place shows."""
import math

import numpy as np
import pytest

import oracle
import paged
from helpers import TOL_LSE, bits_of, bf16_ulp, f64, fp32_gamma, o_error_report, torch_bf16
from long_context_attention_fwd_b200 import inputs as I

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def status():
    from long_context_attention_fwd_b200 import capi
    torch.cuda.synchronize()
    return capi.attn_device_status(None)


def ok_status():
    st, site = status()
    assert st == 0, (st, hex(site))


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def to_torch(x):
    """fp64 values that bf16 holds, as a CUDA bf16 tensor."""
    return torch_bf16(paged.bits16(x)).view(x.shape)


def poison(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.view(torch.uint8).fill_(255)
    return t


def rope_table(n, r, seed):
    """Angles of any size; cos and sin as fp32."""
    ang = np.random.default_rng(seed).uniform(-math.pi, math.pi, (n, r))
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


# ---------------------------------------------------------------- append and gather
# (lens with the new tokens, new tokens, Hq, Hkv, D, page size, rotated elements, interleaved, rows behind)
APPENDS = [
    ([1], [1], 28, 4, 128, 64, 128, False, 0),
    ([17, 0, 16, 40, 7], [17, 0, 1, 33, 7], 28, 4, 128, 16, 128, False, 5),
    ([100, 33, 64], [5, 33, 64], 8, 2, 64, 32, 64, False, 0),
    ([100, 33, 64], [5, 33, 1], 8, 2, 64, 32, 32, True, 3),
    ([300, 1, 129], [299, 1, 128], 5, 1, 128, 256, 128, True, 0),
    ([65, 2], [65, 2], 40, 40, 128, 64, 48, False, 0),       # more rows than a pass, odd rotation
    ([9, 31], [9, 30], 32, 32, 64, 16, 0, False, 0),         # no rotation, no queries
    ([20] * 70, [3] * 70, 3, 3, 64, 16, 16, True, 0),
]


def make_append(case, seed=0):
    lens, new, Hq, Hkv, D, ps, rot, inter, behind = case
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1]) + behind
    table, P = paged.table_for(rng, lens, ps, width=-(-max(lens) // ps) + 1)
    nq = Hq if rot else 0
    x = paged.bf16(rng.normal(size=(T, nq + 2 * Hkv, D)) * np.exp(0.5 * rng.normal(size=(1, nq + 2 * Hkv, D))))
    qkv = to_torch(x).view(T, -1)
    q = qkv[:, :nq * D].view(T, nq, D) if rot else None
    k = qkv[:, nq * D:(nq + Hkv) * D].view(T, Hkv, D)
    v = qkv[:, (nq + Hkv) * D:].view(T, Hkv, D)
    tab = rope_table(max(lens) + 1, rot // 2, seed) if rot else None
    args = dict(q=q, rope=None if tab is None else tuple(dev(t) for t in tab), interleaved=inter,
                cu_seqlens=dev(cu))
    return dict(x=x, k=k, v=v, table=table, P=P, cu=cu, T=T, tab=tab, args=args, nq=nq, lens=lens,
                Hkv=Hkv, D=D, ps=ps, inter=inter,
                cache_len=dev(np.array(lens, dtype=np.int32)), block_table=dev(table))


def rotated(c, t, pos, heads):
    x = c["x"][t, heads]
    if c["tab"] is None:
        return x, np.zeros_like(x)
    return paged.rotate(x, c["tab"][0][pos].astype(np.float64), c["tab"][1][pos].astype(np.float64), c["inter"])


def assert_rounded(got, want, mag):
    """|got - want| at most half a bf16 step of the result and three fp32 roundings: two
    products (2^-24 of each) and their sum (2^-24 of at most both), so 2^-23 of |a c| + |b s|;
    an error there can also move the result across a step's end, hence of got too."""
    tol = 0.5 * bf16_ulp(np.maximum(np.abs(want), np.abs(got))) + 2.0 ** -23 * mag
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("case", APPENDS, ids=[str(i) for i in range(len(APPENDS))])
def test_append_bf16(case):
    from long_context_attention_fwd_b200 import ops
    c = make_append(case)
    shape = (c["P"], c["ps"], c["Hkv"], c["D"])
    kp, vp = poison(shape, torch.bfloat16), poison(shape, torch.bfloat16)
    q_out = poison((c["T"], c["nq"], c["D"]), torch.bfloat16) if c["nq"] else None
    got = ops.attn_append_kv(c["k"], c["v"], kp, vp, c["block_table"], c["cache_len"], q_out=q_out, **c["args"])
    ok_status()
    assert got is q_out
    kb, vb = bits_of(kp).reshape(shape).copy(), bits_of(vp).reshape(shape).copy()
    qb = bits_of(q_out).reshape(c["T"], c["nq"], c["D"]).copy() if c["nq"] else None
    nq, H = c["nq"], c["Hkv"]
    for t, b, pos in paged.places(c["lens"], c["cu"], c["T"]):
        pg, slot = c["table"][b, pos // c["ps"]], pos % c["ps"]
        y, mag = rotated(c, t, pos, slice(nq, nq + H))
        assert_rounded(f64(kb[pg, slot]), y, mag)
        assert np.array_equal(vb[pg, slot], paged.bits16(c["x"][t, nq + H:]))
        kb[pg, slot] = vb[pg, slot] = 0xFFFF
        if nq:
            y, mag = rotated(c, t, pos, slice(0, nq))
            assert_rounded(f64(qb[t]), y, mag)
            qb[t] = 0xFFFF
    # nothing else was written: other slots, other pages, rows behind the last sequence
    assert (kb == 0xFFFF).all() and (vb == 0xFFFF).all() and (qb is None or (qb == 0xFFFF).all())


@pytest.mark.parametrize("case", APPENDS, ids=[str(i) for i in range(len(APPENDS))])
def test_append_4bit_and_gather(case):
    """The bytes are those of the model on the bf16 rows that bf16 pages hold, every one of them;
    gather returns each value rounded once, and leaves rows behind the last sequence alone."""
    from long_context_attention_fwd_b200 import ops
    c = make_append(case, seed=1)
    D, ps, H, nq = c["D"], c["ps"], c["Hkv"], c["nq"]
    shape = (c["P"], ps, H, D)
    kp, vp = poison(shape, torch.bfloat16), poison(shape, torch.bfloat16)
    q1 = ops.attn_append_kv(c["k"], c["v"], kp, vp, c["block_table"], c["cache_len"], **c["args"])
    pages = poison((c["P"], H, ps // 16, 18 * D), torch.uint8)
    q2 = ops.attn_append_kv4(c["k"], c["v"], pages, c["block_table"], c["cache_len"], **c["args"])
    kg, vg = poison((c["T"], H, D), torch.bfloat16), poison((c["T"], H, D), torch.bfloat16)
    ops.attn_gather_kv4(pages, c["block_table"], c["cache_len"], c["args"]["cu_seqlens"], c["T"], k=kg, v=vg)
    ok_status()
    n = int(c["cu"][-1])
    if nq:
        assert torch.equal(q1[:n].view(torch.int16), q2[:n].view(torch.int16))
    want = np.full(tuple(pages.shape), 255, dtype=np.uint8)
    kb, vb = f64(bits_of(kp)).reshape(shape), f64(bits_of(vp)).reshape(shape)
    back = {w: np.full((c["T"], H, D), 0xFFFF, dtype=np.uint16) for w in "kv"}
    for t, b, pos in paged.places(c["lens"], c["cu"], c["T"]):
        pg, slot = c["table"][b, pos // ps], pos % ps
        for w, src in (("k", kb), ("v", vb)):
            code, step, lo = paged.quantise(src[pg, slot])
            paged.store4(want, pg, slot, D, w, paged.row_bytes(code, step, lo))
            val = np.float32(np.float32(code.reshape(H, -1, 64) * step[..., None]) + np.float32(lo[..., None]))
            back[w][t] = paged.bits16(paged.bf16(val.reshape(H, D)))
    assert np.array_equal(pages.cpu().numpy(), want)
    for w, g in (("k", kg), ("v", vg)):
        assert np.array_equal(f64(bits_of(g)[:].reshape(c["T"], H, D)[:n]), f64(back[w][:n]))
        assert (bits_of(g).reshape(c["T"], H, D)[n:] == 0xFFFF).all()


def test_append_without_offsets_in_place_and_unused_entries():
    """Without cu_seqlens there is one token per sequence; entries of length 0 are left out; q may
    be rotated in place; contiguous and strided inputs give the same."""
    from long_context_attention_fwd_b200 import ops
    rng = np.random.default_rng(3)
    lens = np.array([5, 0, 33, 16, 0, 17], dtype=np.int32)
    table, P = paged.table_for(rng, lens, 16, width=4)
    x = paged.bf16(rng.normal(size=(6, 3 + 4, 128)))
    qkv = to_torch(x)
    q, k, v = qkv[:, :3], qkv[:, 3:5], qkv[:, 5:]
    rope = tuple(dev(t) for t in rope_table(64, 64, 4))
    outs = []
    for contiguous in (False, True):
        kp, vp = poison((P, 16, 2, 128), torch.bfloat16), poison((P, 16, 2, 128), torch.bfloat16)
        qq, kk, vv = (t.contiguous() if contiguous else t for t in (q, k, v))
        out = qq.clone() if contiguous else poison((6, 3, 128), torch.bfloat16)
        ops.attn_append_kv(kk, vv, kp, vp, dev(table), dev(lens), q=out if contiguous else qq, rope=rope, q_out=out)
        ok_status()
        outs.append((out, kp, vp))
    live = torch.from_numpy(lens > 0).cuda()
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    assert same(outs[0][0][live], outs[1][0][live]) and same(outs[0][1], outs[1][1]) and same(outs[0][2], outs[1][2])
    assert (outs[0][0][~live].view(torch.int16) == -1).all()           # not written
    assert same(outs[1][0][~live], q[~live])                           # in place: as it was
    touched = (outs[0][2].view(torch.int16) != -1).any(-1).any(-1)
    assert int(touched.sum()) == int(live.sum())


def test_append_overwrites_and_other_dtypes_of_values():
    """Appending again to the same positions replaces what was there; infinities and NaN pass
    through bf16 pages and make their group of 64 read back as NaN from 4-bit pages; equal
    elements come back exactly."""
    from long_context_attention_fwd_b200 import ops
    x = np.zeros((4, 2, 128))
    x[0] = paged.bf16(np.random.default_rng(1).normal(size=(2, 128)))
    x[1, 0, 70], x[1, 1, 3] = np.inf, -np.inf
    x[2, 0, 0], x[2, 1, :64] = np.nan, -2.5
    x[3, 0, 0], x[3, 0, 1], x[3, 1] = 3e38, -3e38, 1e-38
    x = paged.bf16(x)
    t = to_torch(np.nan_to_num(x, nan=0.0, posinf=0, neginf=0))
    t[1, 0, 70], t[1, 1, 3], t[2, 0, 0] = math.inf, -math.inf, math.nan
    cl, table = dev(np.array([4], dtype=np.int32)), dev(np.array([[1]], dtype=np.int32))
    cu = dev(np.array([0, 4], dtype=np.int32))
    kp, vp = poison((2, 16, 2, 128), torch.bfloat16), poison((2, 16, 2, 128), torch.bfloat16)
    pages = poison((2, 2, 1, 18 * 128), torch.uint8)
    for src in (torch.randn_like(t), t):
        ops.attn_append_kv(src, src, kp, vp, table, cl, cu_seqlens=cu)
        ops.attn_append_kv4(src, src, pages, table, cl, cu_seqlens=cu)
    k, v = ops.attn_gather_kv4(pages, table, cl, cu, 4)
    ok_status()
    assert torch.equal(kp[1, :4].nan_to_num(9.0), t.nan_to_num(9.0)) and torch.equal(vp[1, :4].nan_to_num(9.0), t.nan_to_num(9.0))
    code, step, lo = paged.quantise(f64(bits_of(t)).reshape(4, 2, 128))
    val = paged.value(code, step, lo)
    for g in (k, v):
        got = f64(bits_of(g)).reshape(4, 2, 128)
        assert np.array_equal(np.isnan(got), np.isnan(val))
        fine = ~np.isnan(val)
        assert (np.abs(got - val)[fine] <= 0.5 * bf16_ulp(val[fine])).all()
    assert torch.equal(k[2, 1, :64], t[2, 1, :64])


@pytest.mark.parametrize("four", [False, True])
def test_append_records_tokens_without_a_place(four):
    """A page outside the pool, a position past the table and one past the rotation's rows:
    those tokens are left out, the others are written, and the status tells of it once."""
    from long_context_attention_fwd_b200 import capi, ops
    rng = np.random.default_rng(6)
    x = to_torch(paged.bf16(rng.normal(size=(5, 3, 64))))
    q, k, v = x[:, :1], x[:, 1:2], x[:, 2:]
    rope = tuple(dev(t) for t in rope_table(40, 32, 4))
    table = np.array([[7, 0], [1, -1], [2, 3], [99, 4], [5, 6]], dtype=np.int32)
    lens = np.array([3, 17, 33, 4, 20], dtype=np.int32)       # b = 1: page -1; 2: past the table; 3: page 99
    good = {0: (7, 2), 4: (6, 3)}
    run = dict(q=q, rope=rope, q_out=poison((5, 1, 64), torch.bfloat16))
    if four:
        pool = poison((8, 1, 1, 18 * 64), torch.uint8)
        ops.attn_append_kv4(k, v, pool, dev(table), dev(lens), **run)
        row = pool.cpu().numpy()
        touched = {(int(p), s) for p in range(8) for s in range(16) if (row[p, 0, 0, s * 32:(s + 1) * 32] != 255).any()}
    else:
        pool, vp = poison((8, 16, 1, 64), torch.bfloat16), poison((8, 16, 1, 64), torch.bfloat16)
        ops.attn_append_kv(k, v, pool, vp, dev(table), dev(lens), **run)
        touched = {tuple(map(int, i[:2])) for i in (pool.view(torch.int16) != -1).nonzero().cpu()}
    st, site = status()
    assert st == capi.ATTN_ERR_INVALID_ARG and site == 0x500
    assert touched == set(good.values())
    wrote = (run["q_out"].view(torch.int16) != -1).any(-1).any(-1).cpu().numpy()
    assert set(np.flatnonzero(wrote)) == set(good)
    ok_status()                                                # reported once
    # a rotation with fewer rows than the positions
    short = tuple(t[:19].contiguous() for t in rope)
    if four:
        ops.attn_append_kv4(k[4:], v[4:], pool, dev(table[4:]), dev(lens[4:]), rope=short)
    else:
        ops.attn_append_kv(k[4:], v[4:], pool, vp, dev(table[4:]), dev(lens[4:]), rope=short)
    assert status()[0] == capi.ATTN_ERR_INVALID_ARG


def test_gather_reads_zeros_without_a_place():
    from long_context_attention_fwd_b200 import capi, ops
    pages = torch.zeros((2, 1, 1, 18 * 64), dtype=torch.uint8, device="cuda")
    pages[..., 16 * 64:] = 63                                   # scales of about 0.7
    table, cl = dev(np.array([[1], [5]], dtype=np.int32)), dev(np.array([2, 1], dtype=np.int32))
    k, v = ops.attn_gather_kv4(pages, table, cl, dev(np.array([0, 4, 5], dtype=np.int32)), 5)
    assert status()[0] == capi.ATTN_ERR_INVALID_ARG            # sequence 1's page
    for t in (k, v):                                           # two positions before the start, two tokens, no page
        assert [bool((t[i] != 0).all()) for i in range(5)] == [False, False, True, True, False]
        assert (t[[0, 1, 4]] == 0).all()


# ---------------------------------------------------------------- decode
def decode_inputs(lens, Hq, Hkv, D, seed, mult=0.5):
    rng = np.random.default_rng(seed)
    q = paged.bf16(rng.normal(size=(len(lens), Hq, D)))
    kv = [paged.bf16(rng.normal(size=(2, L, Hkv, D)) * mult * np.exp(0.5 * rng.normal(size=(1, 1, Hkv, D)))) for L in lens]
    return rng, q, kv


DECODES = [
    # lens, Hq, Hkv, D, page size
    ([1], 28, 4, 128, 16),
    ([0, 1, 15, 16, 17, 127, 128, 129, 700, 0], 8, 2, 64, 16),
    ([1000, 385, 129, 2], 28, 4, 128, 64),
    ([513, 31, 32, 33, 63, 64, 65], 32, 32, 64, 32),
    ([520, 1, 255], 64, 1, 128, 128),
    ([300, 777], 12, 1, 64, 256),
    ([260, 47], 40, 2, 128, 32),
    ([1300], 9, 1, 128, 16),
]


@pytest.mark.parametrize("case", DECODES, ids=[str(i) for i in range(len(DECODES))])
def test_decode_paged(case):
    """Against the fp64 oracle, and next to what attn_decode gives on the dense cache of the same
    capacity: the same products and statistics, with partial results that are not rounded to bf16
    and splits by the lengths in place of the capacity (bit for bit where a sequence is not split:
    up to four tiles of 128)."""
    from long_context_attention_fwd_b200 import ops
    lens, Hq, Hkv, D, ps = case
    rng, q, kv = decode_inputs(lens, Hq, Hkv, D, 21)
    table, P = paged.table_for(rng, lens, ps, width=-(-max(lens) // ps) + 2)
    cap = table.shape[1] * ps
    B = len(lens)
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
    cl = np.array(lens, dtype=np.int32)
    qt = to_torch(q)
    scale = 1 / math.sqrt(D)
    o, lse = poison((B, Hq, D), torch.bfloat16), poison((B, Hq), torch.float32)
    ops.attn_decode_paged(qt, kp, vp, dev(table), dev(cl), out=o, lse=lse)
    o2, lse2 = ops.attn_decode(qt, kd, vd, dev(cl))
    vmax = float(np.abs(dense[1]).max())
    ok_status()
    short = dev(cl) <= 4 * 128
    assert torch.equal(lse[short], lse2[short])
    assert torch.equal(o[short].view(torch.int16), o2[short].view(torch.int16))
    # A weight is rounded to bf16 relative to its own split's maximum, 2^-9 of it either way: sums
    # with other splits are within 2^-8 of each other, and so are their logarithms.
    live = dev(cl) > 0
    assert float((lse - lse2)[live].abs().max()) <= 2.0 ** -8
    # two roundings of the result (half a step each), one of the partials' and two of the weights'
    # (2^-9 of P|V| each)
    near = (o.float() - o2.float()).abs() <= 2.0 ** -7 * o2.float().abs() + 2.0 ** -7 * vmax
    assert bool(near.all())
    o_r, l_r = oracle.decode(q, dense[0], dense[1], cl, scale)
    oa_r, _ = oracle.decode(q, dense[0], np.abs(dense[1]), cl, scale)
    og, lg = f64(bits_of(o)).reshape(B, Hq, D), lse.double().cpu().numpy()
    full = cl > 0
    assert (og[~full] == 0).all() and np.isneginf(lg[~full]).all()
    rep = o_error_report(og[full], o_r[full], oa_r[full])
    assert rep["n_over_model"] == 0, rep
    assert np.abs(lg[full] - l_r[full]).max() <= TOL_LSE


@pytest.mark.parametrize("lens,Hq,Hkv,D,ps,width", [
    ([int(n) for n in np.random.default_rng(5).integers(0, 600, 40)], 8, 2, 64, 16, 4096),
    ([20000], 28, 4, 128, 64, 131072), ([9000, 1, 0, 300, 9000], 8, 1, 128, 32, 32768), ([3, 2500], 4, 4, 64, 256, 1 << 20)],
    ids=["many_short", "one_long", "uneven", "wide"])
def test_decode_paged_tables_wider_than_the_lengths(lens, Hq, Hkv, D, ps, width):
    """The splits go by the lengths, whatever the table could hold; the last sequence of an uneven
    batch has the first one's pages.  Pages behind the lengths do not exist."""
    from long_context_attention_fwd_b200 import ops
    shared = len(lens) == 5
    rng, q, kv = decode_inputs(lens, Hq, Hkv, D, 41)
    table, P = paged.table_for(rng, lens, ps, width=width // ps)
    if shared:
        table[4], kv[4] = table[0], kv[0]
    kp, vp = poison((P, ps, Hkv, D), torch.bfloat16), poison((P, ps, Hkv, D), torch.bfloat16)
    dense = np.zeros((2, len(lens), max(lens), Hkv, D))
    for b, L in enumerate(lens):
        if L == 0:
            continue
        pos = torch.arange(L, device="cuda")
        pg = dev(table[b])[pos // ps].long()
        kp[pg, pos % ps], vp[pg, pos % ps] = to_torch(kv[b][0]), to_torch(kv[b][1])
        dense[:, b, :L] = kv[b]
    cl = np.array(lens, dtype=np.int32)
    run = lambda: ops.attn_decode_paged(to_torch(q), kp, vp, dev(table), dev(cl))    # noqa: E731
    (o, lse), (o2, lse2) = run(), run()
    ok_status()
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
    o_r, l_r = oracle.decode(q, dense[0], dense[1], cl, 1 / math.sqrt(D))
    oa_r, _ = oracle.decode(q, dense[0], np.abs(dense[1]), cl, 1 / math.sqrt(D))
    og, lg = f64(bits_of(o)).reshape(o.shape), lse.double().cpu().numpy()
    full = cl > 0
    assert (og[~full] == 0).all() and np.isneginf(lg[~full]).all()
    rep = o_error_report(og[full], o_r[full], oa_r[full])
    assert rep["n_over_model"] == 0, rep
    assert np.abs(lg[full] - l_r[full]).max() <= TOL_LSE


def pages4_of(kv, lens, table, P, ps, Hkv, D, fill=255):
    """A pool of 4-bit pages holding the model's rows of kv, the rest `fill`, and the values."""
    pages = np.full((P, Hkv, ps // 16, 18 * D), fill, dtype=np.uint8)
    vals = []
    for b, L in enumerate(lens):
        both = []
        for i, w in enumerate("kv"):
            code, step, lo = paged.quantise(kv[b][i])
            cb, sb = paged.row_bytes(code, step, lo)
            for pos in range(L):
                paged.store4(pages, table[b, pos // ps], pos % ps, D, w, (cb[pos], sb[pos]))
            both.append((paged.value(code, step, lo), step, lo))
        vals.append(both)
    return pages, vals


def check_decode4(o, lse, q, vals, lens, Hkv, D, scale):
    """Every element against softmax in 64 bits over the pages' values, within bounds from the
    kernel's arithmetic.  Per weight: its rounding to fp16 (2^-11 of p s code, the part of the
    value above the minimum; below 2^-14 at most 2^-25, where the largest weight so far is 2^6
    or more, hence 15 2^-31 of the largest p s) and the score's error, e_s; the output's
    rounding, half a bf16 step.  e_s: 16 tensor-core and scale steps in fp32 (2^-23 each, truncation allowed) on
    A = scale max_j sum |q| (s code + |m|), q's 2^-25, the exponential's 2^-22.  fp32 sums over
    the keys: fp32_gamma.  lse: e_s and four fp32 roundings of itself."""
    og, lg = f64(bits_of(o)).reshape(q.shape), lse.double().cpu().numpy()
    G = q.shape[1] // Hkv
    for b, L in enumerate(lens):
        if L == 0:
            assert (og[b] == 0).all() and np.isneginf(lg[b]).all()
            continue
        (K, ks, km), (V, vs, vm) = vals[b]
        low = np.repeat(vm, 64, -1)
        Kabs = (K - np.repeat(km, 64, -1)) + np.abs(np.repeat(km, 64, -1))
        for h in range(q.shape[1]):
            g = h // G
            s = scale * (K[:, g] @ q[b, h])
            p = np.exp(s - s.max())
            l_ref = s.max() + np.log(p.sum())
            p /= p.sum()
            o_ref = p @ V[:, g]
            A = abs(scale) * (Kabs[:, g] @ np.abs(q[b, h])).max()
            e_s = A * (16 * 2.0 ** -23 + 2.0 ** -25) + 2.0 ** -22
            mag = p @ (np.abs(V[:, g] - low[:, g]) + np.abs(low[:, g]))
            tol = 0.5 * bf16_ulp(np.maximum(np.abs(o_ref), np.abs(og[b, h]))) \
                + (1 + 2.0 ** -11) * 2.0 ** -11 * (p @ (V[:, g] - low[:, g])) + (2 * e_s + fp32_gamma(L)) * mag \
                + L * 15 * 2.0 ** -31 * np.repeat((p[:, None] * vs[:, g]).max(0), 64)
            assert (np.abs(og[b, h] - o_ref) <= tol).all(), (b, h, np.abs(og[b, h] - o_ref).max())
            assert abs(lg[b, h] - l_ref) <= e_s + 2.0 ** -22 * abs(l_ref) + fp32_gamma(L), (b, h, lg[b, h], l_ref)


@pytest.mark.parametrize("case", DECODES, ids=[str(i) for i in range(len(DECODES))])
def test_decode_4bit(case):
    from long_context_attention_fwd_b200 import ops
    lens, Hq, Hkv, D, ps = case
    rng, q, kv = decode_inputs(lens, Hq, Hkv, D, 22, mult=1.0)
    table, P = paged.table_for(rng, lens, ps, width=-(-max(lens) // ps) + 2)
    pages, vals = pages4_of(kv, lens, table, P, ps, Hkv, D)
    B = len(lens)
    o, lse = poison((B, Hq, D), torch.bfloat16), poison((B, Hq), torch.float32)
    ops.attn_decode_kv4(to_torch(q), dev(pages), dev(table), dev(np.array(lens, dtype=np.int32)), out=o, lse=lse)
    ok_status()
    check_decode4(o, lse, q, vals, lens, Hkv, D, 1 / math.sqrt(D))


@pytest.mark.parametrize("scale,qmult", [(-0.3, 1.0), (0.0, 1.0), (2.0, 30.0), (0.05, 2.0 ** -120), (1e-4, 2.0 ** 100)])
def test_decode_4bit_scales_and_query_sizes(scale, qmult):
    """Negative and zero scales, scores in the hundreds (one key takes all), queries far from 1."""
    from long_context_attention_fwd_b200 import ops
    lens, Hq, Hkv, D, ps = [200, 37], 10, 2, 128, 32
    rng, q, kv = decode_inputs(lens, Hq, Hkv, D, 23)
    qt = to_torch(q * qmult)
    q = f64(bits_of(qt)).reshape(q.shape)      # what the kernel is given: 30 times a bf16 is cut to one
    scale = scale if qmult < 2.0 ** 50 else scale * 2.0 ** -90
    table, P = paged.table_for(rng, lens, ps)
    pages, vals = pages4_of(kv, lens, table, P, ps, Hkv, D)
    o, lse = ops.attn_decode_kv4(qt, dev(pages), dev(table), dev(np.array(lens, dtype=np.int32)), scale=scale)
    ok_status()
    check_decode4(o, lse, q, vals, lens, Hkv, D, float(np.float32(scale)))


@pytest.mark.parametrize("kind", ["constant", "huge", "tiny", "mixed", "zero"])
def test_decode_4bit_values_of_any_size(kind):
    """V whose groups are constant (steps of 0), near 1e30, near 1e-25, of sizes 2^60 apart from
    token to token, or all 0, with scores that rise by hundreds after the first tokens."""
    from long_context_attention_fwd_b200 import ops
    lens, Hq, Hkv, D, ps = [700, 90], 7, 1, 128, 16
    rng, q, kv = decode_inputs(lens, Hq, Hkv, D, 29)
    for b, L in enumerate(lens):
        k, v = kv[b]
        ramp = np.linspace(0, 1, L)[:, None, None]
        k[:] = paged.bf16(k * (1 + 40 * ramp))               # later keys score far higher
        if kind == "constant":
            v[:] = paged.bf16(rng.normal(size=(L, Hkv, 1)))
        elif kind == "zero":
            v[:] = 0
        else:
            size = {"huge": 2.0 ** 100, "tiny": 2.0 ** -80, "mixed": 2.0 ** rng.integers(-30, 31, (L, 1, 1))}[kind]
            v[:] = paged.bf16(v * size)
    table, P = paged.table_for(rng, lens, ps)
    pages, vals = pages4_of(kv, lens, table, P, ps, Hkv, D)
    o, lse = ops.attn_decode_kv4(to_torch(q), dev(pages), dev(table), dev(np.array(lens, dtype=np.int32)))
    ok_status()
    check_decode4(o, lse, q, vals, lens, Hkv, D, 1 / math.sqrt(D))


@pytest.mark.parametrize("lens,Hq,Hkv,D,ps", [
    ([int(n) for n in np.random.default_rng(6).integers(0, 600, 64)], 8, 2, 64, 16),
    ([1] * 70, 4, 4, 64, 32), ([852, 1], 40, 40, 128, 32), ([1, 500, 200], 32, 4, 128, 64),
    ([64 * i for i in range(33)], 4, 1, 64, 64), ([3000, 0, 1, 1, 0, 65, 1100] * 6, 20, 1, 128, 128)],
    ids=["ragged", "ones", "many_heads", "few", "full_tiles", "long_and_short"])
def test_decode_4bit_many_short(lens, Hq, Hkv, D, ps):
    """Several sequences and heads in a block, cut anywhere; tables also wider than the lengths."""
    from long_context_attention_fwd_b200 import ops
    rng, q, kv = decode_inputs(lens, Hq, Hkv, D, 33)
    for width in (None, 8192 // ps):
        table, P = paged.table_for(rng, lens, ps, width=width)
        pages, vals = pages4_of(kv, lens, table, P, ps, Hkv, D)
        o, lse = ops.attn_decode_kv4(to_torch(q), dev(pages), dev(table), dev(np.array(lens, dtype=np.int32)))
        ok_status()
        check_decode4(o, lse, q, vals, lens, Hkv, D, 1 / math.sqrt(D))


def values_of(table, pages, ps, lens, D):
    out = []
    for b, L in enumerate(lens):
        got = paged.load4(pages, table[b], ps, L, D)
        out.append([(paged.value(*got[w]), got[w][1], got[w][2]) for w in "kv"])
    return out


@pytest.mark.parametrize("lens,Hq,Hkv,D,ps", [([32768], 28, 4, 128, 64), ([20000, 3, 9001, 16384], 8, 8, 64, 16),
                                              ([5000] * 40, 7, 1, 128, 32)],
                         ids=["one_32K", "ragged_mha", "many_5K"])
def test_decode_4bit_long(lens, Hq, Hkv, D, ps):
    """Long caches, split over many blocks; the pages are filled by attn_append_kv4."""
    from long_context_attention_fwd_b200 import ops
    rng = np.random.default_rng(31)
    table, P = paged.table_for(rng, lens, ps)
    T = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(4)
    k = torch.randn(T, Hkv, D, generator=gen, device="cuda").bfloat16()
    v = torch.randn(T, Hkv, D, generator=gen, device="cuda").bfloat16()
    cu = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    cl = dev(np.array(lens, dtype=np.int32))
    pages = poison((P, Hkv, ps // 16, 18 * D), torch.uint8)
    ops.attn_append_kv4(k, v, pages, dev(table), cl, cu_seqlens=cu)
    q = paged.bf16(rng.normal(size=(len(lens), Hq, D)) * 2)
    o, lse = ops.attn_decode_kv4(to_torch(q), pages, dev(table), cl)
    ok_status()
    some = [0, len(lens) - 1] if len(lens) > 4 else range(len(lens))
    vals = values_of(table[some], pages.cpu().numpy(), ps, [lens[b] for b in some], D)
    check_decode4(o[list(some)], lse[list(some)], q[list(some)], vals, [lens[b] for b in some], Hkv, D, 1 / math.sqrt(D))


@pytest.mark.parametrize("four", [False, True])
def test_decode_workspace_graphs_and_repeats(four):
    """Whatever the workspace holds, twice on it, on another stream, and from two captured graphs
    that share it, replayed in turn: the same bits."""
    from long_context_attention_fwd_b200 import ops
    lens, Hq, Hkv, D, ps = [3000, 1, 777, 0, 64], 28, 4, 128, 64
    rng, q, _ = decode_inputs([0] * 5, Hq, Hkv, D, 24)
    table, P = paged.table_for(rng, lens, ps)
    gen = torch.Generator(device="cuda").manual_seed(8)
    kv = [torch.randn(P, ps, Hkv, D, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    q2 = to_torch(paged.bf16(rng.normal(size=q.shape)))
    q, cl, tb = to_torch(q), dev(np.array(lens, dtype=np.int32)), dev(table)
    if four:
        pages = ops.kv4_pages(P, ps, Hkv, D)
        one = dev(np.arange(P, dtype=np.int32)[:, None])
        ops.attn_append_kv4(kv[0].view(-1, Hkv, D), kv[1].view(-1, Hkv, D), pages, one,
                            torch.full((P,), ps, dtype=torch.int32, device="cuda"),
                            cu_seqlens=dev(np.arange(0, P * ps + 1, ps, dtype=np.int32)))
        need = ops.attn_decode_kv4_workspace_size(q, pages, tb)
        run = lambda x, **a: ops.attn_decode_kv4(x, pages, tb, cl, **a)          # noqa: E731
    else:
        need = ops.attn_decode_paged_workspace_size(q, kv[0], tb)
        run = lambda x, **a: ops.attn_decode_paged(x, *kv, tb, cl, **a)          # noqa: E731
    want, want2 = run(q), run(q2)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    same = lambda a, b: torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])  # noqa: E731
    for fill in (0, 255, None, None):
        if fill is not None:
            ws.fill_(fill)
        assert same(run(q, workspace=ws), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = run(q2, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    assert same(other, want2)
    graphs = []
    for x in (q, q2):
        out = dict(out=torch.empty_like(q), lse=torch.empty(5, Hq, device="cuda"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="relaxed"):
            run(x, workspace=ws, **out)
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), w in zip(graphs, (want, want2)):
            out["out"].fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert same((out["out"], out["lse"]), w)
    del graphs, g
    ok_status()


@pytest.mark.parametrize("four", [False, True])
def test_decode_records_a_page_outside_the_pool(four):
    """The bad sequence is reported and touches no other; the next call is clean."""
    from long_context_attention_fwd_b200 import capi, ops
    lens, ps = np.array([40, 40, 40], dtype=np.int32), 16
    table = np.array([[0, 1, 2], [3, 77, 4], [5, 6, 7]], dtype=np.int32)
    fixed = table.copy()
    fixed[1, 1] = 8
    kv = [torch.randn(9, ps, 2, 64, device="cuda").bfloat16() for _ in range(2)]
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    if four:
        pages = ops.kv4_pages(9, ps, 2, 64)
        ops.attn_append_kv4(kv[0].view(-1, 2, 64), kv[1].view(-1, 2, 64), pages, dev(np.arange(9, dtype=np.int32)[:, None]),
                            torch.full((9,), ps, dtype=torch.int32, device="cuda"),
                            cu_seqlens=dev(np.arange(0, 145, 16, dtype=np.int32)))
        run = lambda t: ops.attn_decode_kv4(q, pages, dev(t), dev(lens))      # noqa: E731
    else:
        run = lambda t: ops.attn_decode_paged(q, *kv, dev(t), dev(lens))      # noqa: E731
    good, _ = run(fixed)
    ok_status()
    bad, _ = run(table)
    st, site = status()
    assert st == capi.ATTN_ERR_INVALID_ARG and site == (0x503 if four else 0x502)
    assert torch.equal(good[[0, 2]], bad[[0, 2]])
    again, _ = run(fixed)
    ok_status()
    assert torch.equal(good, again)


def test_pools_past_32_bits():
    """Pages whose offsets pass 2^32 bytes (and 2^31 elements): the same tokens as in a small pool
    are appended to the last pages of large ones, decoded and gathered, to the same bits."""
    from long_context_attention_fwd_b200 import ops
    Hq, Hkv, D, ps, n = 8, 4, 128, 64, 300
    gen = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(n, Hkv, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(1, Hq, D, generator=gen, device="cuda").bfloat16()
    cl, cu = dev(np.array([n], dtype=np.int32)), dev(np.array([0, n], dtype=np.int32))
    outs = []
    for P in (5, 130000):                                     # 4.8 GB of 4-bit pages, 8.5 GB of K
        tb = torch.arange(P - 1, P - 6, -1, dtype=torch.int32, device="cuda")[None].contiguous()
        pages = ops.kv4_pages(P, ps, Hkv, D)
        ops.attn_append_kv4(k, v, pages, tb, cl, cu_seqlens=cu)
        got = [*ops.attn_decode_kv4(q, pages, tb, cl), *ops.attn_gather_kv4(pages, tb, cl, cu, n)]
        del pages
        kp, vp = (torch.empty(P, ps, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ops.attn_append_kv(k, v, kp, vp, tb, cl, cu_seqlens=cu)
        got += [*ops.attn_decode_paged(q, kp, vp, tb, cl), kp[P - 5:].flip(0), vp[P - 5:].flip(0)]
        got[-2:] = [t.reshape(-1, Hkv, D)[:n].clone() for t in got[-2:]]
        outs.append(got)
        del kp, vp
        torch.cuda.empty_cache()
    ok_status()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_two_decodes_at_once():
    """Two streams, each with its own workspace, overlapping: the bits of one at a time."""
    from long_context_attention_fwd_b200 import ops
    Hq, Hkv, D, ps, L, B = 28, 4, 128, 16, 2000, 6
    gen = torch.Generator(device="cuda").manual_seed(3)
    P = B * L // ps
    table = torch.randperm(P, generator=gen, device="cuda").to(torch.int32).view(B, -1).contiguous()
    k, v = (torch.randn(B * L, Hkv, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    cl = torch.full((B,), L, dtype=torch.int32, device="cuda")
    pages = ops.kv4_pages(P, ps, Hkv, D)
    ops.attn_append_kv4(k, v, pages, table, cl, cu_seqlens=torch.arange(0, B * L + 1, L, dtype=torch.int32, device="cuda"))
    qs = [torch.randn(B, Hq, D, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    want = [ops.attn_decode_kv4(q, pages, table, cl) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(ops.attn_decode_kv4(qs[i], pages, table, cl))
    torch.cuda.synchronize()
    ok_status()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_serving_steps_together():
    """A prompt appended in two chunks, then token after token: at each step the decode over the
    paged caches is attn_fwd's last row over all tokens so far (bf16 pages), and the same over
    the gathered values of the 4-bit pages."""
    from long_context_attention_fwd_b200 import ops
    lens, Hq, Hkv, D, ps, steps = [70, 33], 8, 2, 128, 32, 3
    B, total = len(lens), [n + 3 for n in lens]
    rng = np.random.default_rng(12)
    table, P = paged.table_for(rng, total, ps)
    tb = dev(table)
    rope = tuple(dev(t) for t in rope_table(128, D // 2, 7))
    x = [to_torch(paged.bf16(rng.normal(size=(n, Hq + 2 * Hkv, D)))) for n in total]
    kp, vp = poison((P, ps, Hkv, D), torch.bfloat16), poison((P, ps, Hkv, D), torch.bfloat16)
    pages = poison((P, Hkv, ps // 16, 18 * D), torch.uint8)
    done = np.zeros(B, dtype=np.int32)
    for new in ([40, 0], [30, 33], [1, 1], [1, 1], [1, 1]):
        part = torch.cat([x[b][done[b]:done[b] + n] for b, n in enumerate(new)])
        done = done + np.array(new, dtype=np.int32)
        cl, cu = dev(done), dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
        q, k, v = part[:, :Hq], part[:, Hq:Hq + Hkv], part[:, Hq + Hkv:]
        qr = ops.attn_append_kv(k, v, kp, vp, tb, cl, q=q, rope=rope, cu_seqlens=cu)
        q4 = ops.attn_append_kv4(k, v, pages, tb, cl, q=q, rope=rope, cu_seqlens=cu)
        assert torch.equal(qr, q4)
        if new != [1, 1]:
            continue
        o, lse = ops.attn_decode_paged(qr, kp, vp, tb, cl)
        o4, lse4 = ops.attn_decode_kv4(qr, pages, tb, cl)
        cuk = dev(np.concatenate([[0], np.cumsum(done)]).astype(np.int32))
        kg, vg = ops.attn_gather_kv4(pages, tb, cl, cuk, int(done.sum()))
        at = 0
        for b in range(B):
            n = int(done[b])
            pos = torch.arange(n, device="cuda")
            pg = tb[b].long()[pos // ps]
            for kk, vv, oo, ll in ((kp[pg, pos % ps], vp[pg, pos % ps], o, lse), (kg[at:at + n], vg[at:at + n], o4, lse4)):
                qq = torch.zeros(1, n, Hq, D, dtype=torch.bfloat16, device="cuda")
                qq[0, -1] = qr[b]
                of, lf = ops.attn_fwd(qq, kk[None].contiguous(), vv[None].contiguous(), causal=True)
                # two kernels' roundings: 2^-8 of the weights and of the output each; gather's
                # values are rounded to bf16 (2^-8 of V; of K, 2^-8 sum |q k| scale in the score)
                e = 2.0 ** -8 * float((qr[b].float().abs().amax() * kk.float().abs().sum(-1).amax()) / math.sqrt(D)) if oo is o4 else 0
                assert float((oo[b].float() - of[0, -1].float()).abs().max()) <= (4 * 2.0 ** -8 + 2 * e) * float(vv.float().abs().max())
                assert float((ll[b] - lf[0, :, -1]).abs().max()) <= 1e-4 + e
            at += n
    ok_status()


@pytest.mark.parametrize("four", [False, True])
def test_captured_step_replayed(four):
    """One token per sequence appended and attended to, captured once: replays that advance the
    lengths on the GPU give the bits of the same steps called one by one.  One entry is unused."""
    from long_context_attention_fwd_b200 import ops
    start, Hq, Hkv, D, ps, steps = [30, 126, 5], 8, 2, 128, 16, 6
    B = len(start) + 1
    rng = np.random.default_rng(17)
    table, P = paged.table_for(rng, [n + steps for n in start] + [0], ps)
    tb, rope = dev(table), tuple(dev(t) for t in rope_table(256, D // 2, 9))
    x = to_torch(paged.bf16(rng.normal(size=(steps, B, Hq + 2 * Hkv, D))))
    gen = torch.Generator(device="cuda").manual_seed(6)
    T = sum(start)
    k0, v0 = (torch.randn(T, Hkv, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    one = dev(np.array([1, 1, 1, 0], dtype=np.int32))

    def pools():
        p = (torch.zeros(P, Hkv, ps // 16, 18 * D, dtype=torch.uint8, device="cuda"),) if four else tuple(
            torch.zeros(P, ps, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        cl = dev(np.array(start + [0], dtype=np.int32))
        cu = dev(np.concatenate([[0], np.cumsum(start + [0])]).astype(np.int32))
        (ops.attn_append_kv4 if four else ops.attn_append_kv)(k0, v0, *p, tb, cl, rope=rope, cu_seqlens=cu)
        return p, cl

    def step(p, cl, cur, q_out):
        cl.add_(one)
        q, k, v = cur[:, :Hq], cur[:, Hq:Hq + Hkv], cur[:, Hq + Hkv:]
        q = (ops.attn_append_kv4 if four else ops.attn_append_kv)(k, v, *p, tb, cl, q=q, rope=rope, q_out=q_out)
        return (ops.attn_decode_kv4 if four else ops.attn_decode_paged)(q, *p, tb, cl)

    zeros = lambda: torch.zeros(B, Hq, D, dtype=torch.bfloat16, device="cuda")    # noqa: E731
    p, cl = pools()
    want = [step(p, cl, x[i], zeros()) for i in range(steps)]
    pools_want = p
    p, cl = pools()
    cur, q_out = x[0].clone(), zeros()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        out = step(p, cl, cur, q_out)
    for i in range(steps):
        cur.copy_(x[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0].view(torch.int16), want[i][0].view(torch.int16)) and torch.equal(out[1], want[i][1])
        assert bool((out[0][3] == 0).all())
    assert all(torch.equal(a, b) for a, b in zip(p, pools_want))
    assert cl.tolist() == [n + steps for n in start] + [0]
    ok_status()
    del g
