"""The cases the key/value-cache operators are measured on, with their plain forms.

Five operators of serving with a paged cache, as `ops` offers them:

  append        ops.attn_append_kv     new tokens' K (rotated by position) and V into bf16 pages,
                                       the rotated queries on the way
  append_kv4    ops.attn_append_kv4    the same into 4-bit pages
  gather_kv4    ops.attn_gather_kv4    cached tokens of 4-bit pages back as bf16 K and V
  decode        ops.attn_decode_paged  one new query token per sequence over bf16 pages
  decode_kv4    ops.attn_decode_kv4    the same over 4-bit pages

`cache_len[b]` counts the tokens of sequence b including those being appended, so the same
array serves the append and the attention that follows.

4-bit pages: uint8 [num_pages][Hkv][page_size / 16][18 D].  A unit of 16 tokens of one head is
contiguous: K codes [16][D / 2], V codes [16][D / 2], K scales [16][D / 64][2] bf16, V scales
likewise.  Each group of 64 elements has (scale, minimum) and a value is scale * code + minimum;
of a token's 4-byte words, number (D / 64) * i + g holds the codes of elements
64 g + 8 i ... 64 g + 8 i + 7, lowest bits first.
"""
import math

import numpy as np
import torch

own = False

UNIT = 16     # tokens of a unit of 4-bit pages
GROUP = 64    # elements that share a scale and a minimum


# ---------------------------------------------------------------- cases
def listed():
    gqa = {"Hq": 28, "Hkv": 4, "D": 128}       # the grouped heads of this repository's workloads
    mha = {"Hq": 32, "Hkv": 32, "D": 64}       # its workload with one kv head per query head
    return [
        # one user's next token late in a 32K context: latency is all there is
        dict(gqa, name="append_b1_32k", op="append", B=1, ctx_lo=32767, ctx_hi=32767, new_lo=1,
             new_hi=1, ps=64, rot=128, interleaved=False, shape_seed=1),
        # a decode step of a full server, small pages, rotation of half of each head in adjacent pairs
        dict(gqa, name="append_b256", op="append", B=256, ctx_lo=0, ctx_hi=8192, new_lo=1, new_hi=1,
             ps=16, rot=64, interleaved=True, shape_seed=2),
        # the prompt of this repository's packed workload: ragged sequences, 32K tokens or so
        dict(gqa, name="append_prompts_32k", op="append", B=8, ctx_lo=0, ctx_hi=0, new_lo=512,
             new_hi=8192, ps=64, rot=128, interleaved=False, shape_seed=3),
        # a decode step into 4-bit pages, one kv head per query head
        dict(mha, name="append4_b64_mha", op="append_kv4", B=64, ctx_lo=1, ctx_hi=4095, new_lo=1,
             new_hi=1, ps=32, rot=64, interleaved=False, shape_seed=4),
        # chunks of long prompts on top of what is cached, into 4-bit pages
        dict(gqa, name="append4_chunks_32k", op="append_kv4", B=16, ctx_lo=0, ctx_hi=30000, new_lo=1,
             new_hi=4096, ps=64, rot=128, interleaved=False, shape_seed=5),
        # a few short sequences leave the cache
        dict(gqa, name="gather4_short", op="gather_kv4", B=5, ctx_lo=1, ctx_hi=999, ps=16,
             shape_seed=6),
        # long sequences leave the cache, as K and V of the training kernels
        dict(gqa, name="gather4_8x32k", op="gather_kv4", B=8, ctx_lo=16384, ctx_hi=32768, ps=128,
             shape_seed=7),
        # this repository's decode workloads, paged
        dict(gqa, name="decode_b1_32k", op="decode", B=1, ctx_lo=32768, ctx_hi=32768, ps=64,
             shape_seed=8),
        dict(gqa, name="decode_b16_32k", op="decode", B=16, ctx_lo=16384, ctx_hi=32768, ps=16,
             shape_seed=9),
        # the same over 4 bits: the first tokens of a chat, one long context, a mixed batch
        dict(gqa, name="decode4_b1_513", op="decode_kv4", B=1, ctx_lo=513, ctx_hi=513, ps=64,
             shape_seed=10),
        dict(gqa, name="decode4_b1_32k", op="decode_kv4", B=1, ctx_lo=32768, ctx_hi=32768, ps=64,
             shape_seed=11),
        dict(gqa, name="decode4_b48_mixed", op="decode_kv4", B=48, ctx_lo=1, ctx_hi=32768, ps=16,
             shape_seed=12),
    ]


def draw(rng):
    """One more case: any operator, batch and lengths over their logarithm, odd lengths."""
    logu = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["append", "append_kv4", "gather_kv4", "decode", "decode", "decode_kv4", "decode_kv4"])
    Hq, Hkv, D = rng.choice([(28, 4, 128), (28, 4, 128), (32, 32, 64), (8, 2, 64), (14, 2, 64),
                             (32, 8, 128), (16, 1, 128), (40, 40, 128), (64, 4, 128)])
    ps = rng.choice([16, 32, 64, 128])
    # no more cached values than the largest listed case of the operator has, and a table to match
    most = {"append": 1 << 24, "append_kv4": 1 << 24, "gather_kv4": 1 << 26, "decode": 3 << 26,
            "decode_kv4": 3 << 27}[op] // (Hkv * D)
    hi = logu(1, min(32768, most))
    lo = rng.choice([1, hi, max(1, hi // 2)])
    B = max(1, min(logu(1, 64), most // hi))
    case = {"op": op, "Hq": Hq, "Hkv": Hkv, "D": D, "ps": ps, "B": B, "ctx_lo": lo, "ctx_hi": hi,
            "shape_seed": rng.randrange(1 << 30)}
    if op.startswith("append"):
        new = 1 if rng.random() < 0.4 else max(1, min(logu(1, 8192), (1 << 24) // (B * (Hq + 2 * Hkv) * D)))
        case.update(new_lo=min(new, rng.choice([1, new])), new_hi=new, rot=rng.choice([D, D, D // 2]),
                    interleaved=rng.random() < 0.3)
    return case


def _shape(case):
    """Context lengths and new tokens of the case's sequences (numpy, from the case alone)."""
    r = np.random.RandomState(case["shape_seed"])
    ctx = r.randint(case["ctx_lo"], case["ctx_hi"] + 1, case["B"])
    new = r.randint(case["new_lo"], case["new_hi"] + 1, case["B"]) if "new_lo" in case else 0 * ctx
    return ctx.astype(np.int64), new.astype(np.int64)


def work(case):
    """What one pass cannot do without: every input read and every output written once."""
    ctx, new = _shape(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    row16, row4 = 2 * D, D // 2 + 4 * (D // GROUP)     # bytes of a head's vector in bf16, in 4 bits
    n, L = int(new.sum()), int(ctx.sum())
    table = 4 * sum(-(-int(x) // case["ps"]) for x in ctx + new)
    if case["op"].startswith("append"):
        stored = 2 * Hkv * (row16 if case["op"] == "append" else row4)
        # q, k, v and a row of cosines and sines in; the rotated q and the cache rows out; for the
        # 4-bit cache the rows are also read back as values
        moved = n * ((2 * Hq + 2 * Hkv) * row16 + 4 * case["rot"] + stored)
        if case["op"] == "append_kv4":
            moved += n * (stored + 2 * Hkv * row16)
        return {"bytes": moved + table, "flops": n * (3 * case["rot"] * (Hq + Hkv) + (0 if case["op"] == "append" else 8 * Hkv * D))}
    if case["op"] == "gather_kv4":
        return {"bytes": L * 2 * Hkv * (row4 + row16) + table, "flops": L * 2 * Hkv * D * 2}
    row = row16 if case["op"] == "decode" else row4
    return {"bytes": L * 2 * Hkv * row + table + case["B"] * Hq * (2 * row16 + 4), "flops": 4 * L * Hq * D}


# ---------------------------------------------------------------- inputs
def _tokens(gen, T, Hkv, D):
    """K and V of T tokens: bf16 normals; channels of K differ in size, a few by a lot."""
    size = torch.exp(0.4 * torch.randn(Hkv, D, generator=gen, device="cuda"))
    size *= 1 + 5 * (torch.rand(Hkv, D, generator=gen, device="cuda") < 0.02)
    k = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen).mul_(size.bfloat16())
    v = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    return k, v


def _quantise(x):
    """Codes (uint8), scales and minima (bf16) of x [..., D], per group of 64 elements."""
    g = x.float().unflatten(-1, (-1, GROUP))
    low = g.amin(-1, keepdim=True)
    scale = ((g.amax(-1, keepdim=True) - low) / 15).bfloat16().float()
    code = torch.where(scale > 0, ((g - low) / scale).round(), torch.zeros_like(g)).clamp(0, 15)
    return code.to(torch.uint8).flatten(-2), torch.cat([scale, low], -1).bfloat16()


def _pack(x):
    """x [T, H, D] as the bytes of a 4-bit row: codes [T, H, D / 2] and scales [T, H, D / 16]."""
    code, scale = _quantise(x)
    T, H, D = x.shape
    byte = code[..., 0::2] | (code[..., 1::2] << 4)
    word = byte.view(T, H, D // GROUP, 8, 4).transpose(2, 3).reshape(T, H, D // 2)
    return word, scale.reshape(T, H, -1).view(torch.uint8)


def _rows(pages, D):
    """The four parts of every unit of 4-bit pages, as views [P, Hkv, units, 16, bytes]."""
    a, s = D // 2, D // 16
    cut = [0, UNIT * a, 2 * UNIT * a, UNIT * (2 * a + s), UNIT * (2 * a + 2 * s)]
    return [pages[..., i:j].unflatten(-1, (UNIT, -1)) for i, j in zip(cut[:-1], cut[1:])]


def _value(words, scales):
    """fp32 values of 4-bit rows: words [..., D / 2] uint8, scales [..., D / 16] uint8."""
    ng = scales.shape[-1] // 4
    byte = words.unflatten(-1, (8, ng, 4)).transpose(-3, -2)
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(-4).unflatten(-1, (ng, GROUP)).float()
    sm = scales.contiguous().view(torch.bfloat16).float().unflatten(-1, (ng, 2))
    return (code * sm[..., :1] + sm[..., 1:]).flatten(-2)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ctx, new = _shape(case)
    B, Hq, Hkv, D, ps, op = (case[n] for n in ("B", "Hq", "Hkv", "D", "ps", "op"))
    total = ctx + new
    width = -(-int(case["ctx_hi"] + case.get("new_hi", 0)) // ps)
    used = -(-total // ps)
    P = int(used.sum()) + 7
    s = {"op": op, "D": D, "ps": ps, "Lmax": width * ps, "scale": 1 / math.sqrt(D)}
    # the pages of a sequence lie anywhere in the pool; table entries past its length hold 0
    order = torch.randperm(P, generator=gen, device="cuda").to(torch.int32)
    first = torch.from_numpy(np.cumsum(used) - used).cuda()
    col = torch.arange(width, device="cuda")
    taken = col < torch.from_numpy(used).cuda()[:, None]
    s["table"] = torch.where(taken, order[(first[:, None] + col).clamp(max=P - 1)], 0).to(torch.int32).contiguous()
    s["cache_len"] = torch.from_numpy(total.astype(np.int32)).cuda()
    k, v = _tokens(gen, P * ps, Hkv, D)
    if op in ("append", "decode"):
        s["k_pages"], s["v_pages"] = k.view(P, ps, Hkv, D), v.view(P, ps, Hkv, D)
    else:
        s["pages"] = torch.empty(P, Hkv, ps // UNIT, 18 * D, dtype=torch.uint8, device="cuda")
        kc, vc, ks, vs = _rows(s["pages"], D)
        step = max(1, (1 << 27) // (ps * Hkv * D))
        for a in range(0, P, step):     # a part of the pool at a time
            for src, codes, scales in ((k, kc, ks), (v, vc, vs)):
                part = src[a * ps:(a + step) * ps]
                w, c = _pack(part)
                lay = lambda t: t.view(-1, ps // UNIT, UNIT, Hkv, t.shape[-1]).permute(0, 3, 1, 2, 4)  # noqa: E731
                codes[a:a + step].copy_(lay(w))
                scales[a:a + step].copy_(lay(c))
    del k, v
    if op.startswith("append"):
        cu = np.concatenate([[0], np.cumsum(new)])
        T = int(cu[-1])
        s["cu"] = torch.from_numpy(cu.astype(np.int32)).cuda()
        # one projection's output holds q, k and v of a token side by side
        qkv = torch.empty(T, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        half = case["rot"] // 2
        angle = torch.arange(s["Lmax"], device="cuda", dtype=torch.float64)[:, None] * \
            1e6 ** -(torch.arange(half, device="cuda", dtype=torch.float64) / half)
        s["rope"] = (angle.cos().float(), angle.sin().float())
        s["interleaved"] = case["interleaved"]
    elif op == "gather_kv4":
        cu = np.concatenate([[0], np.cumsum(ctx)])
        s["cu"], s["T"] = torch.from_numpy(cu.astype(np.int32)).cuda(), int(cu[-1])
    else:
        s["q"] = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    return s


# ---------------------------------------------------------------- plain forms
def _place(s, T):
    """Position, page and slot of each of the T packed tokens."""
    t = torch.arange(T, device="cuda")
    cu = s["cu"].long()
    b = torch.bucketize(t, cu[1:], right=True)
    pos = s["cache_len"].long()[b] - cu[b + 1] + t
    return pos, s["table"].long()[b, pos // s["ps"]], pos % s["ps"]


def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] with its first elements turned by the angles of cos, sin [T, rot / 2]."""
    x, r = x.float(), cos.shape[-1]
    c, n = cos[:, None], sin[:, None]
    a, b = (x[..., 0:2 * r:2], x[..., 1:2 * r:2]) if interleaved else (x[..., :r], x[..., r:2 * r])
    a, b = a * c - b * n, b * c + a * n
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * r:]], -1).bfloat16()


def _attend(q, k, v, cache_len, scale):
    """q [B, Hq, D] over k, v [B, L, Hkv, D] in fp32; rows past cache_len are not used."""
    B, Hq, D = q.shape
    L, Hkv = k.shape[1:3]
    seen = torch.arange(L, device=q.device) < cache_len[:, None]
    qg = q.float().view(B, Hkv, Hq // Hkv, D)
    v = torch.where(seen[:, :, None, None], v, 0.0)
    score = torch.einsum("bhgd,blhd->bhgl", qg, k) * scale
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgl,blhd->bhgd", p, v) / torch.where(total == 0, 1.0, total)
    return o.reshape(B, Hq, D).bfloat16(), (top + total.log()).reshape(B, Hq)


def _every(s):
    """Page and slot of every position of every sequence, [B, Lmax]."""
    at = torch.arange(s["Lmax"], device="cuda")
    return s["table"].long()[:, at // s["ps"]], (at % s["ps"]).expand(s["table"].shape[0], -1)


def _plain(s):
    op, D = s["op"], s["D"]
    if op.startswith("append"):
        pos, page, slot = _place(s, s["k"].shape[0])
        cos, sin = (t[pos] for t in s["rope"])
        q = _rotate(s["q"], cos, sin, s["interleaved"])
        k = _rotate(s["k"], cos, sin, s["interleaved"])
        if op == "append":
            s["k_pages"][page, slot], s["v_pages"][page, slot] = k, s["v"]
            return q, s["k_pages"], s["v_pages"]
        kc, vc, ks, vs = _rows(s["pages"], D)
        where = (page, slice(None), slot // UNIT, slot % UNIT)
        kc[where], ks[where] = _pack(k)
        vc[where], vs[where] = _pack(s["v"])
        return q, _value(kc[where], ks[where]).bfloat16(), _value(vc[where], vs[where]).bfloat16()
    if op == "gather_kv4":
        _, page, slot = _place(s, s["T"])
        kc, vc, ks, vs = (t[page, :, slot // UNIT, slot % UNIT] for t in _rows(s["pages"], D))
        return _value(kc, ks).bfloat16(), _value(vc, vs).bfloat16()
    page, slot = _every(s)
    if op == "decode":
        k, v = (s[n][page, slot].float() for n in ("k_pages", "v_pages"))
    else:
        kc, vc, ks, vs = (t[page, :, slot // UNIT, slot % UNIT] for t in _rows(s["pages"], D))
        k, v = _value(kc, ks), _value(vc, vs)
    return _attend(s["q"], k, v, s["cache_len"], s["scale"])


def run(s):
    if not own:
        return _plain(s)
    from long_context_attention_fwd_b200 import ops
    op = s["op"]
    if op == "append":
        q = ops.attn_append_kv(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["cache_len"],
                               q=s["q"], rope=s["rope"], interleaved=s["interleaved"], cu_seqlens=s["cu"])
        return q, s["k_pages"], s["v_pages"]
    if op == "append_kv4":
        q = ops.attn_append_kv4(s["k"], s["v"], s["pages"], s["table"], s["cache_len"], q=s["q"],
                                rope=s["rope"], interleaved=s["interleaved"], cu_seqlens=s["cu"])
        k, v = ops.attn_gather_kv4(s["pages"], s["table"], s["cache_len"], s["cu"], s["k"].shape[0])
        return q, k, v
    if op == "gather_kv4":
        return ops.attn_gather_kv4(s["pages"], s["table"], s["cache_len"], s["cu"], s["T"])
    if op == "decode":
        return ops.attn_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cache_len"], scale=s["scale"])
    return ops.attn_decode_kv4(s["q"], s["pages"], s["table"], s["cache_len"], scale=s["scale"])


# ---------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    """run()'s outputs from the definitions, sequence by sequence, in 64 bits."""
    s = prepare(case, seed)
    ctx, new = _shape(case)
    D, ps, op = case["D"], case["ps"], case["op"]
    B, Hkv, G = case["B"], case["Hkv"], case["Hq"] // case["Hkv"]
    table = s["table"].long()

    def unpacked(b, lo, hi, which):
        """Values of positions lo..hi-1 of sequence b from its 4-bit pages, fp64 [n, Hkv, D]."""
        pos = torch.arange(lo, hi, device="cuda")
        unit = s["pages"][table[b, pos // ps], :, (pos % ps) // 16]        # [n, Hkv, 18 D]
        j = (pos % 16)[:, None, None]
        d = torch.arange(D, device="cuda")
        g, i, n = d // 64, d % 64 // 8, d % 8
        at = which * 8 * D + j * (D // 2) + 4 * ((D // 64) * i + g) + n // 2
        code = torch.gather(unit, 2, at.expand(-1, Hkv, -1)) >> (4 * (n % 2)).to(torch.uint8) & 15
        at = 16 * D + which * D + j * (D // 16) + 4 * g
        half = lambda k: (torch.gather(unit, 2, (at + k).expand(-1, Hkv, -1)).int()  # noqa: E731
                          + 256 * torch.gather(unit, 2, (at + k + 1).expand(-1, Hkv, -1)).int())
        f = lambda bits: (bits << 16).view(torch.float32).double()  # noqa: E731
        return code.double() * f(half(0)) + f(half(2))

    if op.startswith("decode"):
        outs, lses = [], []
        for b in range(B):
            L = int(ctx[b])
            if op == "decode":
                pos = torch.arange(L, device="cuda")
                k, v = (s[n][table[b, pos // ps], pos % ps].double() for n in ("k_pages", "v_pages"))
            else:
                k, v = unpacked(b, 0, L, 0), unpacked(b, 0, L, 1)
            q = s["q"][b].double().view(Hkv, G, D)
            sc = (q @ k.permute(1, 2, 0)) * s["scale"]
            lses.append(torch.logsumexp(sc, -1).flatten())
            outs.append((torch.softmax(sc, -1) @ v.permute(1, 0, 2)).reshape(-1, D))
        return torch.stack(outs), torch.stack(lses)
    if op == "gather_kv4":
        return tuple(torch.cat([unpacked(b, 0, int(ctx[b]), w) for b in range(B)]) for w in (0, 1))

    def turn(x, pos):
        r = case["rot"] // 2
        c, n = (t[pos].double()[:, None] for t in s["rope"])
        y = x.double().clone()
        ia = torch.arange(r, device="cuda") * 2 if case["interleaved"] else torch.arange(r, device="cuda")
        ib = ia + 1 if case["interleaved"] else ia + r
        y[..., ia] = x[..., ia].double() * c - x[..., ib].double() * n
        y[..., ib] = x[..., ib].double() * c + x[..., ia].double() * n
        return y

    def kept(x):
        """What a 4-bit cache keeps of x [n, Hkv, D]: the nearest of 16 steps from the minimum."""
        y = x.bfloat16().double().unflatten(-1, (D // 64, 64))
        low = y.min(-1, keepdim=True).values
        step = ((y.max(-1, keepdim=True).values - low) / 15).bfloat16().double()
        code = torch.nan_to_num((y - low) / step).round().clamp(0, 15)
        return (code * step + low).flatten(-2)

    pos = torch.cat([torch.arange(int(c), int(c + n), device="cuda") for c, n in zip(ctx, new)])
    seq = torch.cat([torch.full((int(n),), b, device="cuda") for b, n in enumerate(new)])
    q, k, v = turn(s["q"], pos), turn(s["k"], pos), s["v"].double()
    if op == "append_kv4":
        return q, kept(k), kept(v)
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    kp[table[seq, pos // ps], pos % ps] = k
    vp[table[seq, pos // ps], pos % ps] = v
    return q, kp, vp
