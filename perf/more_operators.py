"""Cases for the 4-bit cache and for the append that rotates on its way: new tokens' rows normed, rotated and written
into bf16, FP8 or INT4 pages together with the rotation of their queries, the decode of single and of speculative tokens over INT4
pages, and the attention of ragged chunks over them.

Each case is run in one of two ways, on the same inputs: in plain torch operations in float32
(``own`` false), or through the package's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

PAGE, D_C, D_R, D_N = 64, 512, 64, 128
ROW = {"bf16": 2 * (D_C + D_R), "fp8": D_C + 16 + 2 * D_R, "int4": D_C // 2 + 32 + 2 * D_R}   # bytes of one cached token
SCALE = 1.0 / math.sqrt(192.0)
THETA, EPS = 10000.0, 1e-6


# ------------------------------------------------------------------------------------ the cases
def listed():
    rot = dict(op="rotate", pairs="adjacent", norm=True, pad=0)
    dec = dict(op="decode", s_q=1)
    chunk = dict(op="chunk", pad=0)
    return [
        # a decode step's new tokens on 16 heads of a sharded model: launches are all there is
        dict(rot, name="rotate_step_bf16_h16", batch=64, heads=16, new_lo=1, new_hi=1, past_lo=256, past_hi=2048, kv="bf16", norm=False, lens=1),
        # the same at 128 heads into 4-bit pages, speculative tokens of some streams beside single ones
        dict(rot, name="rotate_step_int4_h128", batch=64, heads=128, new_lo=1, new_hi=3, past_lo=64, past_hi=300, kv="int4", lens=2, pad=11),
        # prompt pieces on 16 heads, quantised on their way, halves rotated against each other
        dict(rot, name="rotate_prompts_fp8_h16", batch=16, heads=16, new_lo=256, new_hi=1024, past_lo=1, past_hi=4096, kv="fp8", pairs="halves", lens=3),
        # a step full of prompt pieces at 128 heads
        dict(rot, name="rotate_prompts_int4_h128", batch=12, heads=128, new_lo=300, new_hi=1500, past_lo=1, past_hi=500, kv="int4", lens=4),
        # few short streams: latency
        dict(dec, name="decode_few_h16", batch=4, heads=16, past_lo=90, past_hi=500, lens=5),
        # many streams on 16 heads of a sharded model: the pages' bytes
        dict(dec, name="decode_streams_h16", batch=64, heads=16, past_lo=2048, past_hi=16384, lens=6),
        # four speculative tokens of each stream, 20 heads
        dict(dec, name="decode_spec_h20", batch=24, heads=20, s_q=4, past_lo=500, past_hi=9000, lens=7),
        # the ragged decode benchmark's lengths at 128 heads
        dict(dec, name="decode_ragged_h128", batch=64, heads=128, past_lo=256, past_hi=32768, lens=8),
        # few very long streams, split over the GPU
        dict(dec, name="decode_long_h128", batch=4, heads=128, past_lo=8192, past_hi=131072, lens=9),
        # a prompt's pieces on 16 heads
        dict(chunk, name="chunk_prompts_h16", batch=4, heads=16, new_lo=384, new_hi=512, past_lo=2048, past_hi=4096, lens=10),
        # a serving step at 128 heads: short pieces beside single tokens, padded rows behind them
        dict(chunk, name="chunk_mixed_h128", batch=16, heads=128, new_lo=1, new_hi=16, past_lo=256, past_hi=8192, lens=11, pad=5),
        # one append after a long prefix
        dict(chunk, name="chunk_long_h128", batch=1, heads=128, new_lo=256, new_hi=256, past_lo=16384, past_hi=16384, lens=12),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    op = rng.choice(["rotate", "rotate", "decode", "decode", "decode", "chunk"])
    lens = rng.randrange(1000, 1 << 30)
    heads = rng.choice([1, 8, 16, 20, 32, 40, 64, 96, 128])
    if op == "rotate":
        new_hi = log(1, 1500)
        return dict(op=op, pairs=rng.choice(["adjacent", "halves"]), norm=rng.random() < 0.6, pad=rng.choice([0, 0, 7]), heads=heads,
                    batch=log(1, 64) if new_hi < 100 else log(1, 10), new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi, past_lo=1, past_hi=log(16, 1000),
                    kv=rng.choice(["bf16", "fp8", "int4", "int4"]), lens=lens)
    if op == "decode":
        batch, s_q, past_hi = log(1, 64), rng.choice([1, 1, 1, 2, 3, 4, 6, 8]), log(16, 100000)
        while batch * s_q * heads * float(past_hi) > 2.5e8 or batch * past_hi > 2000000:   # no more work than the largest listed cases
            batch, past_hi = max(1, batch * 3 // 4), max(16, past_hi * 3 // 4)
        return dict(op=op, batch=batch, heads=heads, s_q=s_q, past_lo=rng.choice([1, max(1, past_hi // 8), past_hi]), past_hi=past_hi, lens=lens)
    batch, new_hi, past_hi = log(1, 24), log(1, 300), log(16, 16000)
    while batch * new_hi * heads * float(past_hi + new_hi) > 4.5e8:
        new_hi, past_hi = max(1, new_hi * 3 // 4), max(16, past_hi * 3 // 4)
    return dict(op=op, batch=batch, heads=heads, new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi, past_lo=rng.choice([16, max(16, past_hi // 4), past_hi]),
                past_hi=past_hi, lens=lens, pad=rng.choice([0, 0, 13]))


def _lengths(case):
    """Per sequence: (new tokens, length with them). Fixed by the case, so that its work is."""
    r = np.random.default_rng(case["lens"])
    B = case["batch"]
    n = np.full(B, case["s_q"]) if case["op"] == "decode" else r.integers(case["new_lo"], case["new_hi"] + 1, B)
    if not n.any():
        n[-1] = 1
    past = np.round(np.exp(r.uniform(math.log(case["past_lo"]), math.log(case["past_hi"]), B))).astype(np.int64)
    return n.astype(np.int64), past + n


def _pages_of(lens):
    return -(-lens // PAGE)


def work(case):
    n, L = _lengths(case)
    T, H = float(n.sum()), case["heads"]
    if case["op"] == "rotate":
        return {"bytes": T * (ROW["bf16"] + ROW[case["kv"]] + 4 * D_R + 4 * H * D_R) + (2 * D_C if case["norm"] else 0) + 8.0 * case["batch"],
                "flops": T * ((H + 1) * 3 * D_R + (4 * D_C if case["norm"] else 0))}
    pairs = float(sum(int(k) * int(m) - int(k) * (int(k) - 1) // 2 for k, m in zip(n, L)))
    by = float(L[n > 0].sum()) * ROW["int4"] + T * H * (2 * (D_C + D_R) + 2 * D_C + 4) + 4.0 * float(_pages_of(L).sum() + 2 * case["batch"] + 1)
    return {"bytes": by, "flops": pairs * H * 2.0 * (2 * D_C + D_R)}


# ------------------------------------------------------------------------------------ cache rows
def _int4(lat):
    """Latent values [..., 512] -> 256 bytes of codes and 16 scales as bytes: scale = max / 7 of 32 values, rounded up to four
    significant bits; the 32-bit word of dims 8w .. 8w + 7 has dim 8w + 2i in bits 4i and dim 8w + 2i + 1 in bits 16 + 4i.
    (Divided by a tensor: by a number torch multiplies with its reciprocal, which rounds up quotients that have four bits.)"""
    g = lat.float().unflatten(-1, (16, 32))
    top = g.abs().amax(-1)
    s = ((top / torch.full_like(top, 7.0)).view(torch.int32) + 0xFFFFF & ~0xFFFFF).view(torch.float32)
    s = torch.where(top > 0, s, 1.0)
    n = ((g / s[..., None]).round().clamp(-7.0, 7.0) + 8.0).to(torch.uint8).flatten(-2).unflatten(-1, (64, 2, 2, 2))   # word, half, nibble, parity
    n = n.movedim(-1, -3)
    return torch.cat([(n[..., 0] | n[..., 1] << 4).flatten(-3), s.to(torch.bfloat16).view(torch.uint8)], -1)


def _from_int4(rows, dtype):
    """The values that rows of bytes [..., 416] stand for: [..., 576]."""
    b = rows[..., : D_C // 2].unflatten(-1, (64, 2, 2))                          # word, parity, half
    n = torch.stack([b & 15, b >> 4], -1).movedim(-3, -1).flatten(-4)            # half, nibble, parity: the dims in order
    s = rows[..., D_C // 2: D_C // 2 + 32].contiguous().view(torch.bfloat16)
    lat = ((n.to(dtype) - 8.0).unflatten(-1, (16, 32)) * s.to(dtype)[..., None]).flatten(-2)
    return torch.cat([lat, rows[..., D_C // 2 + 32:].contiguous().view(torch.bfloat16).to(dtype)], -1)


def _fp8(lat):
    """Latent values [..., 512] -> 512 E4M3 codes and 4 float32 scales as bytes."""
    t = lat.float().unflatten(-1, (4, 128))
    top = t.abs().amax(-1)
    s = torch.where(top > 0, top / torch.full_like(top, 448.0), 1.0)
    codes = (t / s[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).flatten(-2)
    return torch.cat([codes.view(torch.uint8), s.view(torch.uint8)], -1)


def _rows(lat, rope, kv):
    """Cache rows of these latents and RoPE keys (bf16): bf16 [..., 576], or bytes."""
    if kv == "bf16":
        return torch.cat([lat, rope], -1)
    return torch.cat([_int4(lat) if kv == "int4" else _fp8(lat), rope.contiguous().view(torch.uint8)], -1)


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    r = np.random.default_rng(seed)
    op, B, H, kv = case["op"], case["batch"], case["heads"], case.get("kv", "int4")
    ints = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    bf16 = lambda *shape: torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    n, L = _lengths(case)
    need = _pages_of(L)
    P = int(need.sum()) + 3
    perm, bt, o = r.permutation(P), np.full((B, int(need.max())), -1, np.int32), 0
    for b, k in enumerate(need):
        bt[b, :k] = perm[o:o + k]
        o += k
    T = int(n.sum()) + case.get("pad", 0)
    x = bf16(P, PAGE, D_C + D_R)
    s = {"case": case, "n": n, "L": L, "T": int(n.sum()), "cu": ints(np.concatenate([[0], np.cumsum(n)])), "lens": ints(L), "table": ints(bt),
         "pool": _rows(x[..., :D_C], x[..., D_C:], kv)}
    if op == "rotate":
        x = bf16(T, D_C + D_R)
        s["latent"], s["rope"] = x[:, :D_C], x[:, D_C:]                          # the two parts of a projection's output
        s["q"] = bf16(T, H, D_N + D_R)[..., D_N:]                                # the heads' parts that carry positions
        s["q_out"] = torch.zeros(T, H, D_R, dtype=torch.bfloat16, device="cuda")
        s["weight"] = bf16(D_C) * 0.1 + 1.0 if case["norm"] else None
        angle = torch.arange(int(need.max()) * PAGE, dtype=torch.float64, device="cuda")[:, None] * _frequencies()
        s["table_cs"] = torch.cat([angle.cos(), angle.sin()], -1).float()        # 32 cosines, 32 sines a position
    elif op == "decode":
        s["q"], s["qr"] = bf16(B, case["s_q"], H, D_C), bf16(B, case["s_q"], H, D_R)
        s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros(B, case["s_q"], H, device="cuda")
    else:
        s["q"], s["qr"] = bf16(T, H, D_C), bf16(T, H, D_R)
        s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros(T, H, device="cuda")
    if own:
        _handles(case, s)
    return s


def _frequencies():
    return THETA ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32.0)


def _handles(case, s):
    """What a program keeps between calls: params, the plan of a step's lengths."""
    import mla_absorbed_decode_02_gb300 as mla
    B, pages, width = case["batch"], s["pool"].shape[0], s["table"].shape[1]
    kv = {"bf16": mla.MLA_KV_BF16, "fp8": mla.MLA_KV_FP8_E4M3, "int4": mla.MLA_KV_INT4}[case.get("kv", "int4")]
    if case["op"] == "rotate":
        s["params"] = mla.MlaPoolParams.make(batch=B, num_pages=pages, max_pages_per_seq=width, kv_dtype=kv)
        s["values"] = torch.zeros(pages * PAGE, D_C + D_R, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "decode":
        s["decoder"] = mla.Decoder(mla.MlaDecodeParams.make(batch=B, s_q=case["s_q"], num_heads=case["heads"], num_pages=pages, max_pages_per_seq=width, kv_dtype=kv))
        s["decoder"].plan(s["lens"])
    else:
        s["attn"] = mla.ChunkAttention(mla.MlaChunkParams.make(batch=B, max_tokens=s["q"].shape[0], num_heads=case["heads"], num_pages=pages, max_pages_per_seq=width,
                                                               kv_dtype=kv, max_kv_tokens=int((_pages_of(s["L"]) * PAGE).sum())))
        s["attn"].plan(s["cu"], s["lens"])


# ------------------------------------------------------------------------------------ one pass
def _tokens(s):
    """(sequence, position) of each new token."""
    n, L = s["cu"].diff().long(), s["lens"].long()
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=s["T"])
    return seq, torch.arange(s["T"], device="cuda") - s["cu"].long()[seq] + (L - n)[seq]


def _rotated(x, cos, sin, pairs):
    """x [..., 64] turned by its angles [..., 32], in their precision."""
    a, b = (x[..., :32], x[..., 32:]) if pairs == "halves" else (x[..., 0::2], x[..., 1::2])
    a, b = a.to(cos.dtype), b.to(cos.dtype)
    y = a * cos - b * sin, b * cos + a * sin
    return torch.cat(y, -1) if pairs == "halves" else torch.stack(y, -1).flatten(-2)


def _rotate_plain(s):
    case, T = s["case"], s["T"]
    seq, pos = _tokens(s)
    cos, sin = s["table_cs"][pos].split(32, -1)
    lat = s["latent"][:T]
    if case["norm"]:
        x = lat.float()
        lat = (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()).to(torch.bfloat16)   # a norm's output: bf16, as the cache's rows
    k = _rotated(s["rope"][:T], cos, sin, case["pairs"]).to(torch.bfloat16)
    s["q_out"][:T] = _rotated(s["q"][:T], cos[:, None], sin[:, None], case["pairs"]).to(torch.bfloat16)
    at = s["table"][seq, pos // PAGE].long() * PAGE + pos % PAGE
    s["pool"].view(-1, s["pool"].shape[-1])[at] = _rows(lat, k, case["kv"])


def _held(s, dtype):
    """Every sequence's rows, dequantised and padded to the longest: [B, longest, 576], the padding zero."""
    rows = _from_int4(s["pool"][s["table"].clamp_min(0).long()], dtype).flatten(1, 2)
    return rows * (torch.arange(rows.shape[1], device="cuda")[None, :] < s["lens"][:, None])[..., None]


def _softmax(q, rows, seen):
    """q [B, n, H, 576] over rows [B, K, 576], of which token i of sequence b sees seen[b, i]: (out, lse)."""
    B, n, H = q.shape[:3]
    x = (q.flatten(1, 2) @ rows.mT).mul_(SCALE).unflatten(1, (n, H))
    x.masked_fill_(torch.arange(rows.shape[1], device="cuda") >= seen[:, :, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    return (x.flatten(1, 2) @ rows[..., :D_C]).unflatten(1, (n, H)) / total, (top + total.log())[..., 0]


def _padded(s, dtype):
    """Ragged chunk tokens as [B, most, H, 576], where each lies, and how many keys it sees (one at least: padding is not read)."""
    seq, pos = _tokens(s)
    i = torch.arange(s["T"], device="cuda") - s["cu"].long()[seq]
    q = torch.zeros(s["case"]["batch"], int(s["n"].max()), s["case"]["heads"], D_C + D_R, dtype=dtype, device="cuda")
    q[seq, i] = torch.cat([s["q"][: s["T"]], s["qr"][: s["T"]]], -1).to(dtype)
    seen = torch.ones(q.shape[:2], dtype=torch.long, device="cuda")
    seen[seq, i] = pos + 1
    return q, seq, i, seen


def run(s):
    op, case, T = s["case"]["op"], s["case"], s["T"]
    if own:
        import mla_absorbed_decode_02_gb300 as mla
    if op == "rotate":
        if own:
            mla.mla_append_rotated_kv(s["params"], s["latent"], s["rope"], s["table_cs"], s["cu"], s["lens"], s["table"], s["pool"], q_rope=s["q"], q_out=s["q_out"],
                                      norm_weight=s["weight"], norm_eps=EPS, interleaved=case["pairs"] == "adjacent")
        else:
            _rotate_plain(s)
        pool = s["pool"]
        if case["kv"] == "bf16":
            return {"rows": pool, "q": s["q_out"]}
        if case["kv"] == "fp8":
            return {"codes": pool[..., :D_C].view(torch.float8_e4m3fn), "scales": pool[..., D_C:D_C + 16].view(torch.float32),
                    "rope": pool[..., D_C + 16:].view(torch.bfloat16), "q": s["q_out"]}
        if own:
            mla.mla_dequantize_kv(mla.MLA_KV_INT4, pool, s["values"], pool.shape[0] * PAGE)
            return {"values": s["values"], "q": s["q_out"]}
        return {"values": _from_int4(pool.flatten(0, 1), torch.float32).to(torch.bfloat16), "q": s["q_out"]}
    if op == "decode":
        if own:
            s["decoder"].decode(s["q"], s["qr"], s["pool"], s["table"], s["lens"], SCALE, out=s["out"], lse=s["lse"])
        else:
            seen = s["lens"].long()[:, None] - torch.arange(case["s_q"] - 1, -1, -1, device="cuda")
            out, s["lse"] = _softmax(torch.cat([s["q"], s["qr"]], -1).float(), _held(s, torch.float32), seen)
            s["out"] = out.to(torch.bfloat16)
        return {"out": s["out"], "lse": s["lse"]}
    if own:
        s["attn"].attend(s["q"], s["qr"], s["pool"], s["table"], SCALE, out=s["out"], lse=s["lse"])
    else:
        q, seq, i, seen = _padded(s, torch.float32)
        out, lse = _softmax(q, _held(s, torch.float32), seen)
        s["out"][:T], s["lse"][:T] = out[seq, i].to(torch.bfloat16), lse[seq, i]
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------ 64 bits
def _two_to(e):
    """2 ** e for whole e, to the bit (pow is not, on the GPU)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _exact_values(pool):
    """What each 4-bit row stands for, word by word: float64 [..., 576]."""
    words = pool[..., : D_C // 2].contiguous().view(torch.int32).long() & 0xFFFFFFFF
    scales = pool[..., D_C // 2: D_C // 2 + 32].contiguous().view(torch.int16).long() & 0xFFFF
    sign, e, m = 1 - 2 * (scales >> 15), scales >> 7 & 255, scales & 127
    sc = sign.double() * torch.where(e > 0, 128 + m, 2 * m).double() * _two_to(e - 134)
    out = torch.empty(*pool.shape[:-1], D_C + D_R, dtype=torch.float64, device="cuda")
    for k in range(8):                                                           # dim 8 w + k of every word
        code = words >> 4 * (k // 2) + 16 * (k % 2) & 15
        out[..., k:D_C:8] = (code - 8).double() * sc.repeat_interleave(4, -1)
    out[..., D_C:] = pool[..., D_C // 2 + 32:].contiguous().view(torch.bfloat16).double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    n, L, cu = s["n"].tolist(), s["L"].tolist(), s["cu"].tolist()
    if case["op"] == "rotate":
        T, pool, table = s["T"], s["pool"], s["table"].cpu().numpy()
        pos = np.concatenate([np.arange(l - k, l) for k, l in zip(n, L)])
        seq = np.repeat(np.arange(case["batch"]), n)
        at = torch.from_numpy(table[seq, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE).cuda()
        z = torch.polar(torch.ones(T, 32, dtype=torch.float64, device="cuda"), torch.from_numpy(pos).cuda().double()[:, None] * _frequencies())

        def turned(x):
            x = x.double()
            c = torch.complex(*((x[..., :32], x[..., 32:]) if case["pairs"] == "halves" else (x[..., ::2], x[..., 1::2])))
            c = c * (z if x.dim() == 2 else z[:, None])
            return torch.cat([c.real, c.imag], -1) if case["pairs"] == "halves" else torch.view_as_real(c).flatten(-2)

        lat = s["latent"][:T].double()
        if case["norm"]:
            lat = lat / torch.sqrt((lat * lat).sum(-1, keepdim=True) / D_C + EPS) * s["weight"].double()
            lat = lat.to(torch.bfloat16).double()                                # what the cache's rows are made of
        k, q = turned(s["rope"][:T]), s["q_out"].double()
        q[:T] = turned(s["q"][:T])
        if case["kv"] == "fp8":
            codes, scales, rope = pool[..., :D_C].view(torch.float8_e4m3fn).double(), pool[..., D_C:D_C + 16].view(torch.float32).double(), pool[..., D_C + 16:].view(torch.bfloat16).double()
            top = lat.view(-1, 4, 128).abs().max(-1).values / 448.0
            codes.view(-1, D_C)[at], scales.view(-1, 4)[at], rope.view(-1, D_R)[at] = lat / top.repeat_interleave(128, 1), top, k
            return {"codes": codes, "scales": scales, "rope": rope, "q": q}
        rows = pool.double() if case["kv"] == "bf16" else _exact_values(pool).flatten(0, 1)
        if case["kv"] == "int4":
            top = lat.view(-1, 16, 32).abs().max(-1).values
            unit = _two_to(torch.frexp(top.clamp_min(1e-30) / 7.0 * (1.0 + 1e-12)).exponent - 4)
            steps = torch.ceil(top / (7.0 * unit))                               # (7 times a power of two: the quotient is exact where it is whole)
            sc = torch.where(top > 0, steps * unit, 1.0).repeat_interleave(32, 1)
            lat = torch.round(lat / sc) * sc
        rows.view(-1, D_C + D_R)[at] = torch.cat([lat, k], -1)
        return {"rows" if case["kv"] == "bf16" else "values": rows, "q": q}
    H = case["heads"]
    out, lse = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda"), torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    o, z, q, qr = out.view(-1, H, D_C), lse.view(-1, H), s["q"].view(-1, H, D_C), s["qr"].view(-1, H, D_R)
    for b in range(case["batch"]):
        if n[b] == 0:
            continue
        rows = _exact_values(s["pool"][s["table"][b, : -(-L[b] // PAGE)].long()]).flatten(0, 1)[: L[b]]
        step = max(1, (1 << 27) // (H * L[b]))
        for t in range(0, n[b], step):
            m = min(step, n[b] - t)
            a, e = cu[b] + t, cu[b] + t + m
            keys = L[b] - n[b] + t + m                                           # the last of these tokens sees so many
            x = (torch.tensordot(q[a:e].double(), rows[:keys, :D_C], ([2], [1])) + torch.tensordot(qr[a:e].double(), rows[:keys, D_C:], ([2], [1]))) * SCALE
            late = torch.ones(m, keys, dtype=torch.bool, device="cuda").tril_(keys - m)
            x = x.masked_fill(~late[:, None], -math.inf)
            z[a:e] = torch.logsumexp(x, -1)
            o[a:e] = torch.tensordot(torch.exp(x - z[a:e, :, None]), rows[:keys, :D_C], ([2], [0]))
    return {"out": out, "lse": lse}
