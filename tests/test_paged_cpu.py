"""Paged caches without a GPU: the refusals of the entry points and of their Python forms,
the 4-bit rows of the plain model, and workspace sizes."""
import numpy as np
import pytest

import paged
from long_context_attention_fwd_b200 import capi

A = 0x10000  # fake, aligned addresses: validation fails before any CUDA call
BAD, UNSUP, MIS = capi.ATTN_ERR_INVALID_ARG, capi.ATTN_ERR_UNSUPPORTED, capi.ATTN_ERR_MISALIGNED

APPEND = dict(q=A, k=A, v=A, q_stride=4608, k_stride=4608, v_stride=4608, rope_cos=A, rope_sin=A,
              rope_len=100, rope_dim=128, interleaved=0, cu_seqlens=A, cache_len=A, block_table=A,
              q_out=A, k_pages=A, v_pages=A, B=2, T=9, Hq=28, Hkv=4, D=128, max_pages=4,
              num_pages=8, page_size=16, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(B=0), BAD), (dict(T=-1), BAD), (dict(Hkv=0), BAD), (dict(Hkv=5000), BAD), (dict(Hq=0), BAD),
    (dict(D=96), UNSUP), (dict(max_pages=0), BAD), (dict(num_pages=0), BAD), (dict(page_size=8), BAD),
    (dict(page_size=48), BAD), (dict(page_size=512), BAD), (dict(page_size=0), BAD),
    (dict(num_pages=1 << 27), BAD), (dict(max_pages=1 << 27), BAD),
    (dict(rope_dim=8), BAD), (dict(rope_dim=144), BAD), (dict(rope_dim=24), BAD), (dict(rope_len=0), BAD),
    (dict(rope_cos=None), BAD), (dict(rope_cos=None, rope_sin=None), BAD),   # q without a rotation
    (dict(q=None), BAD), (dict(q_out=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD),
    (dict(cache_len=None), BAD), (dict(block_table=None), BAD), (dict(cu_seqlens=None), BAD),  # T != B
    (dict(k_stride=4604), MIS), (dict(q_stride=1), MIS), (dict(v_stride=12), MIS), (dict(k=A + 8), MIS),
    (dict(rope_sin=A + 4), MIS), (dict(q_out=A + 2), MIS), (dict(cache_len=A + 2), MIS),
    (dict(cu_seqlens=A + 1), MIS), (dict(block_table=A + 2), MIS),
])
def test_append_refusals(change, want):
    a = dict(APPEND, **change)
    assert capi.attn_append_kv(**a) == want
    a = {n: x for n, x in a.items() if n not in ("k_pages", "v_pages")}
    assert capi.attn_append_kv4(pages=A, **a) == want


def test_append_refuses_its_pages_and_takes_no_tokens():
    assert capi.attn_append_kv(**dict(APPEND, k_pages=None)) == BAD
    assert capi.attn_append_kv(**dict(APPEND, v_pages=A + 8)) == MIS
    assert capi.attn_append_kv(**dict(APPEND, T=0)) == capi.ATTN_OK
    a = {n: x for n, x in APPEND.items() if n not in ("k_pages", "v_pages")}
    assert capi.attn_append_kv4(pages=None, **a) == BAD
    assert capi.attn_append_kv4(pages=A + 8, **a) == MIS
    assert capi.attn_append_kv4(pages=A, **dict(a, T=0)) == capi.ATTN_OK


def test_gather_refusals():
    ok = dict(pages=A, block_table=A, cache_len=A, cu_seqlens=A, k=A, v=A, B=2, T=9, Hkv=4, D=128,
              max_pages=4, num_pages=8, page_size=16, stream=None)
    for change, want in [(dict(B=0), BAD), (dict(T=-1), BAD), (dict(D=32), UNSUP), (dict(Hkv=0), BAD),
                         (dict(page_size=20), BAD), (dict(pages=None), BAD), (dict(k=None), BAD),
                         (dict(v=A + 8), MIS), (dict(cu_seqlens=None), BAD), (dict(block_table=None), BAD),
                         (dict(T=0), capi.ATTN_OK)]:
        assert capi.attn_gather_kv4(**dict(ok, **change)) == want, change


@pytest.mark.parametrize("four", [False, True])
def test_decode_refusals_and_workspace(four):
    size = capi.attn_decode_kv4_workspace_size if four else capi.attn_decode_paged_workspace_size
    run = capi.attn_decode_kv4 if four else capi.attn_decode_paged
    assert size(16, 28, 4, 128, 512, 64) > 0
    for bad in [(0, 28, 4, 128, 512, 64), (1, 28, 3, 128, 512, 64), (1, 256, 1, 128, 512, 64),
                (1, 28, 4, 96, 512, 64), (1, 8192, 8192, 128, 4, 64), (1, 28, 4, 128, 0, 64), (1, 28, 4, 128, 512, 65),
                (1, 28, 4, 128, 1 << 26, 64)]:
        assert size(*bad) == 0, bad
    need = size(2, 8, 2, 64, 4, 16)
    ok = dict(q=A, block_table=A, cache_len=A, o=A, lse=A, B=2, Hq=8, Hkv=2, D=64, max_pages=4,
              num_pages=9, page_size=16, scale=0.125, workspace=A, workspace_bytes=need, stream=None)
    ok.update(dict(pages=A) if four else dict(k_pages=A, v_pages=A))
    pool = "pages" if four else "k_pages"
    for change, want in [(dict(B=0), BAD), (dict(Hq=7), BAD), (dict(Hq=8192, Hkv=8192), BAD), (dict(D=80), UNSUP), (dict(page_size=1), BAD),
                         (dict(num_pages=0), BAD), (dict(num_pages=1 << 28), BAD),
                         (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD),
                         (dict(workspace=None), BAD), (dict(workspace_bytes=need - 1), BAD),
                         (dict(workspace=A + 16), MIS), (dict(q=None), BAD), (dict(q=A + 8), MIS),
                         ({pool: None}, BAD), ({pool: A + 8}, MIS), (dict(block_table=None), BAD),
                         (dict(block_table=A + 2), MIS), (dict(cache_len=A + 2), MIS), (dict(lse=A + 2), MIS)]:
        assert run(**dict(ok, **change)) == want, change


def test_workspace_of_4bit_decode_does_not_grow_with_the_context():
    size = capi.attn_decode_kv4_workspace_size
    assert size(64, 28, 4, 128, 2048, 64) == size(64, 28, 4, 128, 512, 64)
    assert size(1, 28, 4, 128, 1, 16) < size(64, 28, 4, 128, 512, 64)


def test_python_forms_refuse_cpu_tensors_and_wrong_shapes():
    torch = pytest.importorskip("torch")
    from long_context_attention_fwd_b200 import ops
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)          # noqa: E731
    b16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)       # noqa: E731
    pages = ops.kv4_pages(3, 32, 2, 64, device="cpu")
    assert pages.shape == (3, 2, 2, 18 * 64) and pages.dtype == torch.uint8
    for ps, D in [(24, 64), (8, 64), (32, 96), (512, 128)]:
        with pytest.raises(ValueError):
            ops.kv4_pages(3, ps, 2, D, device="cpu")
    with pytest.raises(ValueError):
        ops.attn_append_kv(b16(2, 2, 64), b16(2, 2, 64), b16(3, 16, 2, 64), b16(3, 16, 2, 64), i32(2, 1), i32(2))
    with pytest.raises(ValueError):
        ops.attn_append_kv4(b16(2, 2, 64), b16(2, 2, 64), pages, i32(2, 1), i32(2))
    with pytest.raises(ValueError):
        ops.attn_gather_kv4(pages, i32(2, 1), i32(2), i32(3), 2)
    with pytest.raises(ValueError):
        ops.attn_decode_paged(b16(2, 4, 64), b16(3, 16, 2, 64), b16(3, 16, 2, 64), i32(2, 1), i32(2))
    with pytest.raises(ValueError):
        ops.attn_decode_kv4(b16(2, 4, 64), pages, i32(2, 1), i32(2))


def test_plain_model_round_trip():
    """The model's own pieces: a row's bytes read back give its codes, and every value is
    within half a step (and the step's own rounding, 2^-8 of 15 steps) of what was stored."""
    rng = np.random.default_rng(5)
    for D in (64, 128):
        ps, L, H = 32, 45, 3
        table, P = paged.table_for(rng, [L], ps)
        pages = rng.integers(0, 256, (P, H, ps // 16, 18 * D), dtype=np.uint8)
        x = {w: paged.bf16(rng.normal(size=(L, H, D)) * np.exp(rng.normal(size=(1, H, D)))) for w in "kv"}
        want = {w: paged.quantise(x[w]) for w in "kv"}
        for j in range(L):
            for w in "kv":
                rows = paged.row_bytes(*(a[j] for a in want[w]))
                paged.store4(pages, table[0, j // ps], j % ps, D, w, rows)
        got = paged.load4(pages, table[0], ps, L, D)
        for w in "kv":
            for a, b in zip(got[w], want[w]):
                assert np.array_equal(a, b)
            err = np.abs(paged.value(*got[w]) - x[w]).reshape(L, H, -1, 64)
            assert (err <= (0.5 + 15 * 2.0 ** -8) * got[w][1][..., None]).all()


def test_plain_quantiser_at_its_edges():
    x = np.zeros((5, 64))
    x[1] = 3.0                      # equal elements: the step is 0
    x[2, 0], x[3, 5] = np.nan, np.inf
    x[4, 0], x[4, 1] = 3e38, -3e38  # the range leaves fp32
    code, step, lo = paged.quantise(x)
    assert (code == 0).all() and (step[:2] == 0).all() and lo[1] == 3 and np.isnan(step[2:]).all() and np.isnan(lo[2:]).all()


def search(cu, B, t):
    """The kernels' 32-way search for the last i in 0..B with cu[i] <= t, lane by lane; every
    index it reads is checked against the array."""
    lo, n = 0, B + 1
    while True:
        step = (n + 31) // 32
        hits = []
        for lane in range(32):
            off = lane * step
            if off < n:
                assert 0 <= lo + off <= B
                if cu[lo + off] <= t:
                    hits.append(lane)
        if not hits:
            return None
        c = hits[-1] * step
        lo, n = lo + c, min(step, n - c)
        if n <= 1:
            return lo


def test_sequence_search_finds_the_token_and_stays_inside():
    rng = np.random.default_rng(9)
    for B in (1, 2, 31, 32, 33, 500, 1023, 1024, 1500):
        lens = rng.integers(0, 4, B)
        cu = np.concatenate([[0], np.cumsum(lens)])
        for t in {0, int(cu[-1]) - 1, int(cu[-1]), int(cu[-1]) + 5, *rng.integers(0, cu[-1] + 1, 40).tolist()}:
            got = search(cu, B, t)
            if t >= cu[-1] or t < 0:
                assert t < 0 or got == B
            else:
                assert cu[got] <= t < cu[got + 1]
        junk = rng.integers(-2 ** 31, 2 ** 31 - 1, B + 1)
        for t in rng.integers(0, 100, 20):
            search(junk, B, int(t))      # malformed offsets: only the reads are checked


@pytest.mark.parametrize("with_q", [False, True])
def test_a_rotation_table_without_rows_is_refused(with_q):
    """An empty tensor's address is null, which the C entry reads as "no rotation"."""
    torch = pytest.importorskip("torch")
    from long_context_attention_fwd_b200 import ops
    b16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)          # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)             # noqa: E731
    rope = (torch.ones(3, 32)[:0], torch.ones(3, 32)[:0])
    args = lambda r: (b16(2, 2, 64), b16(2, 2, 64), i32(2, 1), i32(2), b16(2, 4, 64) if with_q else None,  # noqa: E731
                      r, False, None, None, 2, 64, torch.device("cpu"))
    with pytest.raises(ValueError, match="rows"):
        ops._append_args(*args(rope))
    ops._append_args(*args((torch.ones(3, 32), torch.ones(3, 32))))
