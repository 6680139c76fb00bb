"""Cases for the paged-cache operators around the absorbed decode: the attention of ragged chunks of
new tokens over the cache, the rows that the new tokens add to it, and the upkeep of its pages.

Each case is run in one of two ways, on the same inputs: in plain torch operations in float32
(``own`` false), or through the package's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

PAGE, D_C, D_R = 64, 512, 64
ROW = {"bf16": 2 * (D_C + D_R), "fp8": D_C + 16 + 2 * D_R}   # bytes of one cached token
SCALE = 1.0 / math.sqrt(192.0)


# ------------------------------------------------------------------------------------ the cases
def listed():
    chunk = dict(op="chunk", pad=0)
    return [
        # a few streams, each with the tokens that a speculative step proposes, on 16 heads of a sharded model
        dict(chunk, name="chunk_few_h16", batch=8, heads=16, new_lo=1, new_hi=8, past_lo=64, past_hi=512, kv="bf16", lens=1),
        # a prompt's pieces on 16 heads: eight tokens share a tile of 128 rows
        dict(chunk, name="chunk_prompts_h16", batch=4, heads=16, new_lo=384, new_hi=512, past_lo=2048, past_hi=4096, kv="bf16", lens=2),
        # a serving step at 128 heads: streams with one new token beside streams with a short piece of prompt, padded rows behind them
        dict(chunk, name="chunk_mixed_h128", batch=32, heads=128, new_lo=1, new_hi=24, past_lo=256, past_hi=8192, kv="bf16", lens=3, pad=37),
        # the same on the FP8 cache, with the lengths of the FP8 decode benchmark
        dict(chunk, name="chunk_fp8_h128", batch=8, heads=128, new_lo=48, new_hi=80, past_lo=2048, past_hi=16384, kv="fp8", lens=4),
        # one long append: 512 new tokens after 32,768 cached rows
        dict(chunk, name="chunk_long_h128", batch=1, heads=128, new_lo=512, new_hi=512, past_lo=32768, past_hi=32768, kv="bf16", lens=5),
        # the rows of a decode step's new tokens
        dict(op="append", name="append_step_bf16", batch=64, new_lo=1, new_hi=1, past_lo=256, past_hi=4096, kv="bf16", lens=6, pad=0),
        # the rows of a step full of prompt pieces, quantised on their way into the cache
        dict(op="append", name="append_prompts_fp8", batch=16, new_lo=512, new_hi=2048, past_lo=1, past_hi=4096, kv="fp8", lens=7, pad=0),
        # beam search or parallel samples: streams that go on from a shared prefix
        dict(op="fork", name="fork_few", batch=32, live=8, forks=8, layers=4, pages=512, len_lo=64, len_hi=1000, kv="fp8", lens=8),
        dict(op="fork", name="fork_many", batch=256, live=64, forks=192, layers=16, pages=1100, len_lo=200, len_hi=1000, kv="bf16", lens=9),
        # a fragmented pool drawn together
        dict(op="compact", name="compact_half", batch=64, live=40, layers=16, pages=1000, len_lo=100, len_hi=1300, kv="bf16", lens=10),
        # copies between pages (a copy on write, a swap area inside the pool)
        dict(op="copy", name="copy_pages_fp8", n=300, layers=8, pages=1000, kv="fp8", lens=11),
        # streams end and others take their pages: no cached byte moves, latency is all there is
        dict(op="turnover", name="turnover_128", batch=128, live=128, ended=32, pages=8192, len_lo=64, len_hi=4000, new_lo=1, new_hi=300, lens=12),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    op = rng.choice(["chunk", "chunk", "chunk", "append", "fork", "compact", "copy", "turnover"])
    lens = rng.randrange(1000, 1 << 30)
    kv = rng.choice(["bf16", "fp8"])
    if op == "chunk":
        heads = rng.choice([8, 16, 20, 32, 40, 64, 96, 128])
        batch = log(1, 48)
        new_hi = log(1, 400)
        past_hi = log(16, 24000)
        # no more work than the largest listed case
        while 2176.0 * heads * batch * new_hi * (past_hi + new_hi) > 4.5e12:
            new_hi, past_hi = max(1, new_hi // 2), max(16, past_hi // 2)
        return dict(op=op, batch=batch, heads=heads, new_lo=rng.choice([0, 1, (new_hi + 1) // 2, new_hi]), new_hi=new_hi,
                    past_lo=rng.choice([16, max(16, past_hi // 4), past_hi]), past_hi=past_hi, kv=kv, lens=lens,
                    pad=rng.choice([0, 0, 1, 19]))
    if op == "append":
        new_hi = log(1, 1024)
        return dict(op=op, batch=log(1, 64) if new_hi < 256 else log(1, 12), new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi,
                    past_lo=1, past_hi=log(16, 4000), kv=kv, lens=lens, pad=rng.choice([0, 5]))
    if op == "fork":
        live, forks = log(1, 48), log(1, 150)
        return dict(op=op, batch=live + forks + rng.randrange(4), live=live, forks=forks, layers=log(1, 12), pages=live * 16 + forks + rng.randrange(50),
                    len_lo=1, len_hi=log(64, 1000), kv=kv, lens=lens)
    if op == "compact":
        live = log(1, 40)
        return dict(op=op, batch=live + rng.randrange(8), live=live, layers=log(1, 12), pages=live * 16 + rng.randrange(1, 300), len_lo=1,
                    len_hi=log(64, 1000), kv=kv, lens=lens)
    if op == "copy":
        n = log(1, 300)
        return dict(op=op, n=n, layers=log(1, 8), pages=2 * n + rng.randrange(1, 200), kv=kv, lens=lens)
    live = log(1, 250)
    return dict(op=op, batch=live + rng.randrange(9), live=live, ended=max(1, int(live * rng.random())), pages=live * 70 + 64 + rng.randrange(500), len_lo=1,
                len_hi=log(64, 4000), new_lo=0, new_hi=log(1, 300), lens=lens)


def _lengths(case):
    """Per sequence: (new tokens, length with them). Fixed by the case, so that its work is."""
    r = np.random.default_rng(case["lens"])
    n = r.integers(case["new_lo"], case["new_hi"] + 1, case["batch"])
    if not n.any():
        n[-1] = 1
    past = np.round(np.exp(r.uniform(math.log(case["past_lo"]), math.log(case["past_hi"]), case["batch"]))).astype(np.int64)
    return n.astype(np.int64), past + n


def _held(case):
    """Lengths of the sequences that hold pages, in rows 0 .. live - 1 of the table."""
    r = np.random.default_rng(case["lens"])
    return np.round(np.exp(r.uniform(math.log(case["len_lo"]), math.log(case["len_hi"]), case["live"]))).astype(np.int64)


def _pages_of(lens):
    return -(-lens // PAGE)


def _fork_plan(case):
    r = np.random.default_rng(case["lens"] + 1)
    return r.integers(0, case["live"], case["forks"])


def work(case):
    op = case["op"]
    if op == "chunk":
        n, L = _lengths(case)
        pairs = float(sum(int(k) * int(m) - int(k) * (int(k) - 1) // 2 for k, m in zip(n, L)))
        rows = float(n.sum()) * case["heads"]
        by = float(L[n > 0].sum()) * ROW[case["kv"]] + rows * (2 * (D_C + D_R) + 2 * D_C + 4) + 4.0 * float(_pages_of(L).sum() + 2 * case["batch"] + 1)
        return {"bytes": by, "flops": pairs * case["heads"] * 2.0 * (2 * D_C + D_R)}
    if op == "append":
        n, L = _lengths(case)
        return {"bytes": float(n.sum()) * (ROW["bf16"] + ROW[case["kv"]] + 4), "flops": 0.0}
    row = ROW[case.get("kv", "fp8")]
    if op == "copy":
        return {"bytes": 2.0 * case["n"] * case["layers"] * PAGE * row + 8.0 * case["n"], "flops": 0.0}
    held = _held(case)
    if op == "fork":
        L = held[_fork_plan(case)]
        shared = float(_pages_of(L).sum())
        return {"bytes": 2.0 * float((L % PAGE).sum()) * row * case["layers"] + 4.0 * (2 * shared + case["pages"]) + 16.0 * case["forks"], "flops": 0.0}
    if op == "compact":
        r = np.random.default_rng(case["lens"] + 2)
        at = r.permutation(case["pages"])[: int(_pages_of(held).sum())]
        moved = float((at >= len(at)).sum())
        return {"bytes": 2.0 * moved * PAGE * row * case["layers"] + 4.0 * (2 * len(at) + case["pages"]), "flops": 0.0}
    n = np.random.default_rng(case["lens"] + 3).integers(case["new_lo"], case["new_hi"] + 1, case["batch"])
    return {"bytes": 4.0 * (2 * float(_pages_of(held[: case["ended"]]).sum()) + case["pages"] + 3 * case["batch"] + float(_pages_of(n).sum())), "flops": 0.0}


# ------------------------------------------------------------------------------------ inputs
def _rows(g, shape, kv):
    """Cache rows with N(0, 1) latents and RoPE keys: bf16 [..., 576], or FP8 rows as bytes [..., 656]."""
    x = torch.randn(*shape, D_C + D_R, device="cuda", generator=g)
    if kv == "bf16":
        return x.to(torch.bfloat16)
    tiles = x[..., :D_C].reshape(*shape, 4, 128)
    s = tiles.abs().amax(-1) / 448.0
    codes = (tiles / s[..., None]).to(torch.float8_e4m3fn).reshape(*shape, D_C)
    return torch.cat([codes.view(torch.uint8), s.contiguous().view(torch.uint8), x[..., D_C:].to(torch.bfloat16).contiguous().view(torch.uint8)], -1)


def _pool(g, layers, pages, kv):
    """Pools of random bits: the upkeep moves bytes and never looks at them."""
    return torch.randint(-(1 << 31), (1 << 31) - 1, (layers, pages, PAGE, ROW[kv] // 4), device="cuda", generator=g, dtype=torch.int32)


def _split(case, tables):
    """The page pool's tables in one buffer: reference counts, lengths, block table."""
    a, b = -(-case["pages"] // 4) * 4, -(-case["batch"] // 4) * 4
    return tables[: case["pages"]], tables[a: a + case["batch"]], tables[a + b:].view(case["batch"], -1)


def _tables(case, seed):
    held, P, B = _held(case), case["pages"], case["batch"]
    lens = np.zeros(B, np.int32)
    lens[: case["live"]] = held
    used = _pages_of(held)
    # which pages are held is fixed by the case (so that its work is), whose they are by the seed
    at = np.random.default_rng(case["lens"] + 2).permutation(P)[: int(used.sum())].astype(np.int32)
    np.random.default_rng(seed).shuffle(at)
    width = max(int(used.max()) + 8, 16)
    bt = np.full((B, width), -1, np.int32)
    ref = np.zeros(P, np.int32)
    ref[at] = 1
    o = 0
    for b, k in enumerate(used):
        bt[b, :k] = at[o:o + k]
        o += k
    pad = lambda x: np.concatenate([x, np.zeros(-len(x) % 4, np.int32)])  # noqa: E731
    return torch.from_numpy(np.concatenate([pad(ref), pad(lens), bt.reshape(-1)])).cuda(), width


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    r = np.random.default_rng(seed)
    op = case["op"]
    ints = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    s = {"case": case}
    if op in ("chunk", "append"):
        n, L = _lengths(case)
        need = _pages_of(L)
        P = int(need.sum()) + 3
        perm, bt, o = r.permutation(P), np.full((case["batch"], int(need.max())), -1, np.int32), 0
        for b, k in enumerate(need):
            bt[b, :k] = perm[o:o + k]
            o += k
        s["n"], s["L"] = n, L
        s["cu"], s["lens"], s["table"] = ints(np.concatenate([[0], np.cumsum(n)])), ints(L), ints(bt)
        T = int(n.sum()) + case["pad"]
        s["pool"] = _rows(g, (P, PAGE), case["kv"])
        if op == "append":
            x = torch.randn(T, D_C + D_R, device="cuda", generator=g).to(torch.bfloat16)
            s["latent"], s["rope"] = x[:, :D_C], x[:, D_C:]      # the two parts of a projection's output
        else:
            H = case["heads"]
            s["q"] = torch.randn(T, H, D_C, device="cuda", generator=g).to(torch.bfloat16)
            s["qr"] = torch.randn(T, H, D_R, device="cuda", generator=g).to(torch.bfloat16)
            s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros(T, H, device="cuda")
    else:
        if op == "turnover":
            s["ended"] = ints(r.permutation(case["live"])[: case["ended"]])
            s["new"] = ints(np.random.default_rng(case["lens"] + 3).integers(case["new_lo"], case["new_hi"] + 1, case["batch"]))
        else:
            s["pool"] = _pool(g, case["layers"], case["pages"], case["kv"])
        if op == "copy":
            perm = r.permutation(case["pages"])
            s["src"], s["dst"] = ints(perm[: case["n"]]), ints(perm[case["n"]: 2 * case["n"]])
        else:
            s["tables"], s["width"] = _tables(case, seed)
        if op == "fork":
            s["parents"], s["children"] = ints(_fork_plan(case)), ints(case["live"] + np.arange(case["forks"]))
    if own:
        _handles(case, s)
    return s


def _handles(case, s):
    """What a program keeps between calls: the plan of a step's lengths, the buffers of the pool's upkeep."""
    import mla_absorbed_decode_02_gb300 as mla
    kv = {"bf16": mla.MLA_KV_BF16, "fp8": mla.MLA_KV_FP8_E4M3}[case.get("kv", "bf16")]
    if case["op"] == "chunk":
        p = mla.MlaChunkParams.make(batch=case["batch"], max_tokens=s["q"].shape[0], num_heads=case["heads"], num_pages=s["pool"].shape[0],
                                    max_pages_per_seq=s["table"].shape[1], kv_dtype=kv, max_kv_tokens=int((_pages_of(s["L"]) * PAGE).sum()))
        s["attn"] = mla.ChunkAttention(p)
        s["attn"].plan(s["cu"], s["lens"])
    elif case["op"] == "append":
        s["params"] = mla.MlaPoolParams.make(batch=case["batch"], num_pages=s["pool"].shape[0], max_pages_per_seq=s["table"].shape[1], kv_dtype=kv)
    else:
        s["upkeep"] = mla.PagePool(mla.MlaPoolParams.make(batch=case.get("batch", 1), num_pages=case["pages"], max_pages_per_seq=s.get("width", 1), kv_dtype=kv,
                                                          num_layers=case.get("layers", 1)))


# ------------------------------------------------------------------------------------ one pass
def _dequantised(pool, kv):
    """Pool rows as bf16 [pages, 64, 576]: an FP8 row stands for code x scale in bf16, the attention's own type."""
    if kv == "bf16":
        return pool
    codes = pool[..., :D_C].view(torch.float8_e4m3fn).float().view(*pool.shape[:-1], 4, 128)
    lat = (codes * pool[..., D_C:D_C + 16].view(torch.float32)[..., None]).flatten(-2).to(torch.bfloat16)
    return torch.cat([lat, pool[..., D_C + 16:].view(torch.bfloat16)], -1)


def _chunk_plain(s):
    kv, H, at = s["case"]["kv"], s["case"]["heads"], 0
    for b, (n, L) in enumerate(zip(s["n"].tolist(), s["L"].tolist())):
        if n == 0:
            continue
        rows = _dequantised(s["pool"][s["table"][b, : -(-L // PAGE)].long()], kv).reshape(-1, D_C + D_R)[:L].float()
        step = max(1, (1 << 29) // (H * L))
        for t in range(0, n, step):
            m = min(step, n - t)
            q = torch.cat([s["q"][at + t: at + t + m], s["qr"][at + t: at + t + m]], -1).float().view(m * H, -1)
            x = (q @ rows.T * SCALE).view(m, H, L)
            hidden = torch.arange(L, device="cuda")[None, :] > L - n + t + torch.arange(m, device="cuda")[:, None]
            x.masked_fill_(hidden[:, None, :], -math.inf)
            top = x.amax(-1, keepdim=True)
            x = (x - top).exp_()
            total = x.sum(-1, keepdim=True)
            s["out"][at + t: at + t + m] = ((x.view(m * H, L) @ rows[:, :D_C]).view(m, H, D_C) / total).to(torch.bfloat16)
            s["lse"][at + t: at + t + m] = (top + total.log())[..., 0]
        at += n
    return {"out": s["out"], "lse": s["lse"]}


def _places(s):
    """Row of the pool for each new token."""
    n, L = s["cu"].diff().long(), s["lens"].long()
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=int(s["n"].sum()))
    pos = torch.arange(len(seq), device="cuda") - s["cu"].long()[seq] + (L - n)[seq]
    return s["table"][seq, pos // PAGE].long() * PAGE + pos % PAGE


def _append_plain(s):
    at = _places(s)
    lat, rope = s["latent"][: len(at)], s["rope"][: len(at)]
    flat = s["pool"].view(-1, s["pool"].shape[-1])
    if s["case"]["kv"] == "bf16":
        flat[at] = torch.cat([lat, rope], -1)
    else:
        tiles = lat.float().view(-1, 4, 128)
        top = tiles.abs().amax(-1)
        scale = torch.where(top > 0, top / 448.0, 1.0)
        codes = (tiles / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        flat[at] = torch.cat([codes.view(torch.uint8).flatten(1), scale.view(torch.uint8), rope.contiguous().view(torch.uint8)], -1)


def _append_answer(s):
    pool = s["pool"]
    if s["case"]["kv"] == "bf16":
        return {"rows": pool}
    return {"codes": pool[..., :D_C].view(torch.float8_e4m3fn), "scales": pool[..., D_C:D_C + 16].view(torch.float32),
            "rope": pool[..., D_C + 16:].view(torch.bfloat16)}


def _free_list(ref):
    return torch.argsort((ref != 0).to(torch.int32), stable=True)


def _held_mask(bt, lens):
    return torch.arange(bt.shape[1], device="cuda")[None, :] < ((lens.long() + PAGE - 1) // PAGE)[:, None]


def _fork_plain(s, ref, lens, bt):
    par, chi = s["parents"].long(), s["children"].long()
    L = lens[par].long()
    tail = L % PAGE
    k = torch.nonzero(tail)[:, 0]
    fresh = _free_list(ref)[: len(k)]
    rows, mask = bt[par], _held_mask(bt[par], L)
    src = rows[k, L[k] // PAGE].long()
    shared = mask & (torch.arange(bt.shape[1], device="cuda")[None, :] < (L // PAGE)[:, None])
    ref.index_add_(0, rows.long().clamp_min(0).flatten(), shared.to(torch.int32).flatten())
    ref[fresh] = 1
    rows[k, L[k] // PAGE] = fresh.to(torch.int32)
    bt[chi] = torch.where(mask, rows, -1)
    lens[chi] = L.to(torch.int32)
    took = torch.full_like(s["parents"], -1)
    took[k] = fresh.to(torch.int32)
    pool = s["pool"]
    keep = torch.arange(PAGE, device="cuda")[None, :] < tail[k][:, None]
    pool[:, fresh] = torch.where(keep[None, :, :, None], pool[:, src], pool[:, fresh])
    return took


def _compact_plain(s, ref, lens, bt):
    used = ref != 0
    total = used.sum()
    index = torch.arange(len(ref), device="cuda")
    src, dst = torch.nonzero(used & (index >= total))[:, 0], torch.nonzero(~used & (index < total))[:, 0]
    to = index.to(torch.int32)
    to[src] = dst.to(torch.int32)
    s["pool"][:, dst] = s["pool"][:, src]
    ref[dst] = ref[src]
    ref[src] = 0
    mask = _held_mask(bt, lens)
    bt.copy_(torch.where(mask, to[bt.clamp_min(0).long()], bt))
    return total.to(torch.int32)


def _turnover_plain(s, ref, lens, bt):
    e = s["ended"].long()
    mask = _held_mask(bt[e], lens[e])
    ref.index_add_(0, bt[e].long().clamp_min(0).flatten(), -mask.to(torch.int32).flatten())
    bt[e] = torch.where(mask, -1, bt[e])
    lens[e] = 0
    old, new = (lens.long() + PAGE - 1) // PAGE, (lens.long() + s["new"] + PAGE - 1) // PAGE
    first = torch.cumsum(new - old, 0) - (new - old)
    col = torch.arange(bt.shape[1], device="cuda")[None, :]
    fills = (col >= old[:, None]) & (col < new[:, None])
    page = _free_list(ref)[torch.where(fills, first[:, None] + col - old[:, None], 0)].to(torch.int32)
    bt.copy_(torch.where(fills, page, bt))
    ref.index_add_(0, page.long().flatten(), fills.to(torch.int32).flatten())
    lens.add_(s["new"])
    return torch.ones_like(lens)


def run(s):
    op = s["case"]["op"]
    if op == "chunk":
        if own:
            s["attn"].attend(s["q"], s["qr"], s["pool"], s["table"], SCALE, out=s["out"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        return _chunk_plain(s)
    if op == "append":
        if own:
            import mla_absorbed_decode_02_gb300 as mla
            mla.mla_append_kv(s["params"], s["latent"], s["rope"], s["cu"], s["lens"], s["table"], s["pool"])
        else:
            _append_plain(s)
        return _append_answer(s)
    if op == "copy":
        if own:
            s["upkeep"].copy(s["pool"], s["src"], s["dst"])
        else:
            s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
        return {"pool": s["pool"]}
    tables = s["tables"].clone()      # the tables are updated in place: each pass starts from the same ones
    ref, lens, bt = _split(s["case"], tables)
    if op == "fork":
        got = s["upkeep"].fork(s["pool"], s["parents"], s["children"], bt, lens, ref) if own else _fork_plain(s, ref, lens, bt)
        return {"tables": tables, "fresh": got, "pool": s["pool"]}
    if op == "compact":
        got = s["upkeep"].compact(s["pool"], bt, lens, ref) if own else _compact_plain(s, ref, lens, bt)
        return {"tables": tables, "used": got.reshape(()), "pool": s["pool"]}
    if own:
        s["upkeep"].free(s["ended"], bt, lens, ref)
        got = s["upkeep"].reserve(s["new"], bt, lens, ref)
    else:
        got = _turnover_plain(s, ref, lens, bt)
    return {"tables": tables, "served": got}


# ------------------------------------------------------------------------------------ 64 bits
def _value64(pool, kv):
    """(latent, RoPE) of pool rows in float64, by the format's definition."""
    if kv == "bf16":
        return pool[..., :D_C].double(), pool[..., D_C:].double()
    bits = pool[..., :D_C].long()
    sign, e, m = 1.0 - 2.0 * (bits >> 7).double(), (bits >> 3) & 15, (bits & 7).double()
    v = sign * torch.where(e > 0, (8.0 + m) * torch.pow(2.0, (e - 10).double()), m * 2.0 ** -9)
    sc = pool[..., D_C:D_C + 16].contiguous().view(torch.float32).double()
    lat = v * sc.repeat_interleave(128, -1)
    return lat.to(torch.bfloat16).double(), pool[..., D_C + 16:].contiguous().view(torch.bfloat16).double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "chunk":
        if work(case)["flops"] > 6e12:
            return None
        out, lse = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda"), torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
        start = s["cu"].tolist()
        for b, L in enumerate(s["L"].tolist()):
            first, n = start[b], start[b + 1] - start[b]
            if n == 0:
                continue
            c, k = _value64(s["pool"][s["table"][b, : (L + PAGE - 1) // PAGE].long()], case["kv"])
            c, k = c.reshape(-1, D_C)[:L], k.reshape(-1, D_R)[:L]
            group = max(1, min(n, (1 << 27) // (case["heads"] * L)))
            for t0 in range(0, n, group):
                t1 = min(n, t0 + group)
                seen = L - n + t1                     # keys that the group's last token sees
                q, qr = s["q"][first + t0: first + t1].double(), s["qr"][first + t0: first + t1].double()
                a = (torch.tensordot(q, c[:seen], ([2], [1])) + torch.tensordot(qr, k[:seen], ([2], [1]))) * SCALE
                late = torch.tril(torch.ones(t1 - t0, seen, dtype=torch.bool, device="cuda"), diagonal=L - n + t0)
                a = torch.where(late[:, None], a, torch.full_like(a, -math.inf))
                z = torch.logsumexp(a, -1)
                out[first + t0: first + t1] = torch.tensordot(torch.exp(a - z[..., None]), c[:seen], ([2], [0]))
                lse[first + t0: first + t1] = z
        return {"out": out, "lse": lse}
    if case["op"] == "append":
        pool, kv = s["pool"], case["kv"]
        cu, L, table = s["cu"].tolist(), s["L"].tolist(), s["table"].cpu().numpy()
        at = np.array([int(table[b, p // PAGE]) * PAGE + p % PAGE for b in range(case["batch"]) for p in range(L[b] - cu[b + 1] + cu[b], L[b])], np.int64)
        at = torch.from_numpy(at).cuda()
        lat, rope = s["latent"][: len(at)].double(), s["rope"][: len(at)].double()
        if kv == "bf16":
            rows = pool.double().view(-1, D_C + D_R)
            rows[at, :D_C], rows[at, D_C:] = lat, rope
            return {"rows": rows.view(pool.shape)}
        old = _append_answer(s)
        codes, scales, r = (old[x].double().reshape(-1, w) for x, w in (("codes", D_C), ("scales", 4), ("rope", D_R)))
        sc = lat.view(-1, 4, 128).abs().max(-1).values / 448.0
        sc = torch.where(sc == 0, torch.ones_like(sc), sc)
        codes[at], scales[at], r[at] = lat / sc.repeat_interleave(128, 1), sc, rope
        shape = pool.shape[:-1]
        return {"codes": codes.view(*shape, D_C), "scales": scales.view(*shape, 4), "rope": r.view(*shape, D_R)}
    return None
