"""The operators of one serving step over the paged cache, as cases that can be measured.

A step takes the new tokens of a batch of requests through the cache: slots are reserved for them
(kvc_reserve_slots), queries and keys are normalised and rotated and written (kvc_norm_rope_write), the pages'
key bounds are brought up to date (kvc_block_bounds), the best pages for each query are chosen
(kvc_select_blocks) and the query attends to them, or to its whole row (kvc_block_attention).

Every case names its operator ("op") and its sizes.  A row is one (sequence, layer, KV head) stream with its own
length (rows differ after evictions), pages lie permuted in the pool, and outputs are returned whole.  Where
``own`` is false ``run`` computes the operator with elementary torch operations; where it is true it calls the
framework.
"""
import math

import torch

own = False

INT_MAX = 2**31 - 1
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token for each of 16 requests of 8K to 33K tokens: the slots of a decode step, where latency counts
        dict(name="reserve_decode_16", op="reserve", seqs=16, layers=1, kv_heads=8, page=16, len_lo=8192, len_hi=33792,
             new_lo=1, new_hi=1),
        # ragged prompts (0 to 1,700 tokens) of 33 requests enter caches of four layers at once
        dict(name="reserve_prompts_33", op="reserve", seqs=33, layers=4, kv_heads=8, page=16, len_lo=0, len_hi=700,
             new_lo=0, new_hi=1700),
        # the queries, keys and values of one decode step of 16 requests (32 query heads, 8 KV heads)
        dict(name="write_decode_16", op="write", tokens=16, per_seq=1, layers=1, q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", page=16, rope=128, interleaved=False, norm=True, pos_hi=33792),
        # a packed prefill of 32,768 tokens through one layer
        dict(name="write_prefill_32k", op="write", tokens=32768, per_seq=8192, layers=1, q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", page=16, rope=128, interleaved=False, norm=True, pos_hi=32768),
        # fp32, small heads, part of the head rotated, neighbouring pairs, far positions, an odd number of tokens
        dict(name="write_f32_1003", op="write", tokens=1003, per_seq=59, layers=2, q_heads=28, kv_heads=4, dim=64,
             dtype="f32", page=16, rope=32, interleaved=True, norm=True, pos_hi=4000000),
        # bounds of a whole layer of 32K tokens (after a prefill or a compaction)
        dict(name="bounds_layer_32k", op="bounds", seqs=1, layers=1, kv_heads=8, dim=128, dtype="bf16", page=16,
             len_lo=32768, len_hi=32768, fresh=0),
        # bounds of the pages that a decode step of 16 requests and 8 layers touched
        dict(name="bounds_decode_16x8", op="bounds", seqs=16, layers=8, kv_heads=8, dim=128, dtype="bf16", page=16,
             len_lo=500, len_hi=4000, fresh=1),
        # the choice of 128 pages of 2,048 for one request of 32K tokens
        dict(name="select_32k_of_128", op="select", seqs=1, layers=1, q_heads=32, kv_heads=8, dim=128, dtype="bf16",
             page=16, len_lo=32768, len_hi=32768, top_k=128, sink=1, recent=4, hidden=False),
        # 16 requests of 8K to 33K tokens, four layers, 64 pages each
        dict(name="select_batch16x4", op="select", seqs=16, layers=4, q_heads=32, kv_heads=8, dim=128, dtype="bf16",
             page=16, len_lo=8192, len_hi=33792, top_k=64, sink=1, recent=2, hidden=False),
        # attention to 128 chosen pages of each row, 16 requests
        dict(name="attend_chosen_16", op="attend", seqs=16, layers=1, q_heads=32, kv_heads=8, dim=128, dtype="bf16",
             page=16, len_lo=8192, len_hi=33792, blocks=128, hidden=False),
        # one request of 131,072 tokens, whole rows: few rows, split over their length
        dict(name="attend_whole_1x131072", op="attend", seqs=1, layers=1, q_heads=32, kv_heads=8, dim=128, dtype="bf16",
             page=16, len_lo=131072, len_hi=131072, blocks=0, hidden=False),
        # the layer of the batch of 16, whole rows of 8K to 33K tokens (many rows of unlike lengths)
        dict(name="attend_whole_16", op="attend", seqs=16, layers=1, q_heads=32, kv_heads=8, dim=128, dtype="bf16",
             page=16, len_lo=8192, len_hi=33792, blocks=0, hidden=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _heads(rng):
    kv = rng.choice((1, 2, 3, 4, 5, 8))
    return kv, kv * rng.choice((1, 2, 4, 5, 7, 8))


def draw(rng):
    op = rng.choice(("reserve", "write", "bounds", "select", "attend", "attend"))
    kv, hq = _heads(rng)
    dtype, dim = rng.choice(("bf16", "bf16", "f32")), rng.choice((64, 128, 128))
    page = rng.choice((16, 16, 16, 32, 8, 12))
    seqs, layers = _log(rng, 1, 48), rng.choice((1, 1, 2, 3))
    hi = _log(rng, 40, 131072)
    lo = rng.randrange(0, hi + 1)
    if op == "reserve":
        new = _log(rng, 1, 1700)
        hi = min(hi, 4000)
        return dict(op=op, seqs=seqs, layers=layers, kv_heads=kv, page=page, len_lo=min(lo, hi), len_hi=hi,
                    new_lo=rng.randrange(0, new + 1), new_hi=new)
    if op == "write":
        return dict(op=op, tokens=_log(rng, 1, 10000), per_seq=_log(rng, 1, 2000), layers=layers, q_heads=hq, kv_heads=kv,
                    dim=dim, dtype=dtype, page=page, rope=rng.choice((dim, dim, dim // 2, 48, 0)),
                    interleaved=rng.random() < 0.3, norm=rng.random() < 0.8, pos_hi=_log(rng, 1, 8000000))
    rows = seqs * layers * kv
    # entries times bytes of a vector stay below those of the layer of the batch of 16
    hi = max(1, min(hi, 2600000 * 256 // (rows * dim * ESIZE[dtype])))
    lo = min(lo, hi)
    case = dict(op=op, seqs=seqs, layers=layers, kv_heads=kv, dim=dim, dtype=dtype, page=page, len_lo=lo, len_hi=hi)
    if op == "bounds":
        return dict(case, fresh=rng.choice((0, 0, 1, _log(rng, 1, 64))))
    case.update(q_heads=hq, hidden=rng.random() < 0.4)
    pages = -(-hi // page)
    if op == "select":
        k = _log(rng, 1, max(1, min(512, pages + 3)))
        sink = rng.randrange(0, min(k, 3) + 1)
        return dict(case, top_k=k, sink=sink, recent=rng.randrange(0, min(k - sink, 5) + 1))
    return dict(case, blocks=rng.choice((0, _log(rng, 1, max(1, min(512, pages))))))


def work(case):
    c = case
    if c["op"] == "write":
        vec = c["layers"] * c["dim"]
        n = c["tokens"] * vec * (c["q_heads"] + 2 * c["kv_heads"])
        b = 2 * n * ESIZE[c["dtype"]] + c["tokens"] * (4 + 8 * c["layers"] * c["kv_heads"])
        return {"bytes": b, "flops": 7 * c["tokens"] * vec * (c["q_heads"] + c["kv_heads"])}
    rows = c["seqs"] * c["layers"] * c["kv_heads"]
    if c["op"] == "reserve":
        new = sum(_spread(c["seqs"], c["new_lo"], c["new_hi"]))
        cells = new * c["layers"] * c["kv_heads"]
        return {"bytes": cells * (8 + 4 + 1 + 4) + 8 * cells / c["page"] + 8 * rows + 4 * new + 12 * c["seqs"], "flops": 0}
    es, d, page = ESIZE[c["dtype"]], c["dim"], c["page"]
    lens = _spread(rows, c["len_lo"], c["len_hi"])
    if c["op"] == "bounds":
        old = [max(0, n - c["fresh"]) if c["fresh"] else 0 for n in lens]
        pages = sum(-(-n // page) - o // page for n, o in zip(lens, old))
        slots = sum(n - o // page * page for n, o in zip(lens, old))
        return {"bytes": slots * (d * es + 4) + pages * (2 * d * es + 4 + 4) + 8 * rows, "flops": 2 * slots * d}
    q = c["seqs"] * c["layers"] * c["q_heads"] * d
    if c["op"] == "select":
        pages = sum(-(-n // page) for n in lens)
        return {"bytes": pages * (2 * d * es + 4) + q * es + rows * 4 * (c["top_k"] + 2), "flops": 4 * pages * d}
    slots = sum(min(n, c["blocks"] * page) if c["blocks"] else n for n in lens)
    pages = sum(min(-(-n // page), c["blocks"]) if c["blocks"] else -(-n // page) for n in lens)
    group = c["q_heads"] // c["kv_heads"]
    return {"bytes": slots * (2 * d * es + 4) + pages * (8 if c["blocks"] else 4) + q * (es + 4) + 4 * q // d,
            "flops": 4 * slots * d * group}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def _spread(n, lo, hi):
    """n whole numbers spread evenly over [lo, hi]."""
    return [lo + (hi - lo) * (2 * i + 1) // (2 * n) for i in range(n)]


def _shuffled(n, lo, hi, gen):
    v = torch.tensor(_spread(n, lo, hi), dtype=torch.int32)
    return v[torch.randperm(n, generator=gen)]


def _layout(rows, lens, page, max_pages, spare, gen, num_pages=None):
    """A block table over a permuted pool: (table [rows][max_pages], unused page ids)."""
    need = (lens.to(torch.int64) + page - 1) // page
    used = int(need.sum())
    num_pages = used + spare if num_pages is None else num_pages
    perm = torch.randperm(num_pages, generator=gen).to(torch.int32)
    at = torch.arange(max_pages)[None, :] + (torch.cumsum(need, 0) - need)[:, None]
    held = torch.arange(max_pages)[None, :] < need[:, None]
    table = torch.where(held, perm[at.clamp(max=num_pages - 1)], torch.tensor(-1, dtype=torch.int32))
    return table.contiguous(), perm[used:].clone(), num_pages


def prepare(case, seed):
    c = case
    cpu = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device=DEV).manual_seed(seed + 1)
    s = {"case": dict(c), "op": c["op"]}
    if c["op"] == "write":
        return _prepare_write(c, s, cpu, gpu)
    S, L, H, P = c["seqs"], c["layers"], c["kv_heads"], c["page"]
    rows = S * L * H
    if c["op"] == "reserve":
        new = _shuffled(S, c["new_lo"], c["new_hi"], cpu)
        lens = _shuffled(rows, c["len_lo"], c["len_hi"], cpu)
        mp = -(-(c["len_hi"] + c["new_hi"]) // P) + 2
        row_new = new.repeat_interleave(L * H)
        spare = int((((lens + row_new + P - 1) // P) - ((lens + P - 1) // P)).sum()) + 5
        table, free, num_pages = _layout(rows, lens, P, mp, spare, cpu)
        T = int(new.sum()) + 3
        s.update(table=table, row_len=lens, new_count=new, free=free, free_count=torch.tensor([free.numel()]),
                 next_pos=(lens.view(S, -1).amax(1) + 7).to(torch.int32))
        s = {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in s.items()}
        s.update(slot_pos=torch.randint(0, 1 << 20, (rows, mp * P), dtype=torch.int32, device=DEV, generator=gpu),
                 label=torch.randint(0, 3, (rows, mp * P), dtype=torch.uint8, device=DEV, generator=gpu),
                 crf=torch.rand((rows, mp * P), device=DEV, generator=gpu), T=T, num_pages=num_pages)
        s["out"] = dict(row_len=torch.zeros_like(s["row_len"]), free_count=torch.zeros_like(s["free_count"]),
                        token_start=torch.zeros(S + 1, dtype=torch.int32, device=DEV),
                        token_pos=torch.zeros(T, dtype=torch.int32, device=DEV),
                        slot_map=torch.zeros((T, L, H), dtype=torch.int64, device=DEV))
        if own:
            from agent_kv_cache_lse_b200 import kvc
            pool = torch.zeros((num_pages, P, 64), dtype=torch.bfloat16, device=DEV)
            s["cache"] = kvc.Cache(pool, pool, s["table"], s["row_len"], s["slot_pos"], s["label"], S, L, H)
            s["workspace"] = torch.zeros(kvc.kvc_reserve_workspace_bytes(rows) // 8, dtype=torch.int64, device=DEV)
        return s
    dt, D = DTYPES[c["dtype"]], c["dim"]
    lens = _shuffled(rows, c["len_lo"], c["len_hi"], cpu)
    mp = max(1, -(-c["len_hi"] // P)) + 1
    table, _, num_pages = _layout(rows, lens, P, mp, 1, cpu)
    s.update(table=table.to(DEV), row_len=lens.to(DEV))
    # positions: a slot's own index, one slot in seven (filled later, from the end of the trace) past the row's length
    slot = torch.arange(mp * P, dtype=torch.int32, device=DEV).expand(rows, -1)
    late = torch.rand((rows, mp * P), device=DEV, generator=gpu) < 1 / 7
    s["slot_pos"] = torch.where(late, slot + c["len_hi"], slot).contiguous()
    if c["op"] != "select":
        s["k"] = torch.randn((num_pages, P, D), device=DEV, generator=gpu, dtype=dt)
    if c["op"] == "attend":
        s["v"] = torch.randn((num_pages, P, D), device=DEV, generator=gpu, dtype=dt)
    if c["op"] == "bounds":
        s["from_len"] = (s["row_len"] - c["fresh"]).clamp(min=0) if c["fresh"] else None
        s["out"] = dict(bounds=torch.zeros((rows, mp, 2, D), dtype=dt, device=DEV),
                        pos=torch.zeros((rows, mp), dtype=torch.int32, device=DEV))
    else:
        s["q"] = torch.randn((S, L, c["q_heads"], D), device=DEV, generator=gpu, dtype=dt)
        s["q_pos"] = torch.full((S,), c["len_hi"] - 1 if c["hidden"] else INT_MAX, dtype=torch.int32, device=DEV)
    if c["op"] == "select":
        # bounds of 16 unit-normal keys lie near -1.77 and 1.77; a page's keys have something in common
        mid = torch.randn((rows, mp, D), device=DEV, generator=gpu) * 0.5
        s["bounds"] = torch.empty((rows, mp, 2, D), dtype=dt, device=DEV)
        s["bounds"][:, :, 0] = mid - torch.rand((rows, mp, D), device=DEV, generator=gpu) - 1.3
        s["bounds"][:, :, 1] = mid + torch.rand((rows, mp, D), device=DEV, generator=gpu) + 1.3
        s["pos"] = s["slot_pos"].view(rows, mp, P).amin(2)
        s["out"] = dict(list=torch.zeros((rows, c["top_k"]), dtype=torch.int32, device=DEV),
                        count=torch.zeros(rows, dtype=torch.int32, device=DEV))
    if c["op"] == "attend":
        if c["blocks"]:
            held = (s["row_len"] + P - 1) // P
            rank = torch.rand((rows, mp), device=DEV, generator=gpu)
            rank = rank.masked_fill(torch.arange(mp, device=DEV)[None] >= held[:, None], 2.0)
            rank.scatter_(1, (held - 1).clamp(min=0).long()[:, None], -1.0)  # the newest page is always read
            k = min(c["blocks"], mp)
            some = torch.sort(rank, 1)[1][:, :k]
            s["count"] = held.clamp(max=k).to(torch.int32)
            some = some.masked_fill(torch.arange(k, device=DEV)[None] >= s["count"][:, None], mp)
            some = torch.sort(some, 1)[0].to(torch.int32)
            s["list"] = some.masked_fill(some == mp, -1).contiguous()
        s["out"] = dict(out=torch.zeros((S, L, c["q_heads"], D), device=DEV),
                        lse=torch.zeros((S, L, c["q_heads"]), device=DEV))
    if own:
        from agent_kv_cache_lse_b200 import kvc
        k = s.get("k")
        if k is None:
            k = torch.zeros((1, P, D), dtype=dt, device=DEV)
        s["cache"] = kvc.Cache(k, s.get("v", k), s["table"], s["row_len"], s["slot_pos"], None, S, L, H)
        need = 0
        if c["op"] == "select":
            need = kvc.kvc_select_blocks_workspace_bytes(rows, mp)
        elif c["op"] == "attend":
            need = kvc.kvc_block_attention_workspace_bytes(rows, c["q_heads"] // H, D)
        s["workspace"] = torch.zeros(-(-need // 8), dtype=torch.int64, device=DEV)
    return s


def _prepare_write(c, s, cpu, gpu):
    T, L, Hq, H, D, P = c["tokens"], c["layers"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    dt, cap = DTYPES[c["dtype"]], T + 3
    seqs = -(-T // c["per_seq"])
    start = torch.arange(T) // c["per_seq"]
    i = torch.arange(T) % c["per_seq"]
    # each (sequence, layer, head) fills pages of its own from a random first slot on
    first = torch.randint(0, P, (seqs, L, H), generator=cpu)
    pages = -(-(P + c["per_seq"]) // P)
    num_pages = seqs * L * H * pages
    table = torch.randperm(num_pages, generator=cpu).view(seqs, L, H, pages)
    slot = first[start] + i[:, None, None]
    page = torch.gather(table[start], 3, (slot // P)[..., None])[..., 0]
    smap = torch.full((cap, L, H), -1, dtype=torch.int64)
    smap[:T] = page * P + slot % P
    pos0 = torch.randint(0, max(1, c["pos_hi"] - c["per_seq"]), (seqs,), generator=cpu)
    pos = torch.full((cap,), -1, dtype=torch.int32)
    pos[:T] = (pos0[start] + i).to(torch.int32)
    s.update(slot_map=smap.to(DEV), pos=pos.to(DEV), count=torch.tensor([T], dtype=torch.int32, device=DEV),
             qkv=torch.randn((cap, L, Hq + 2 * H, D), device=DEV, generator=gpu, dtype=dt),
             k=torch.randn((num_pages, P, D), device=DEV, generator=gpu, dtype=dt),
             v=torch.randn((num_pages, P, D), device=DEV, generator=gpu, dtype=dt),
             q_out=torch.zeros((cap, L, Hq, D), device=DEV, dtype=dt), eps=1e-6, qw=None, kw=None, inv_freq=None)
    if c["norm"]:
        s["qw"] = (1 + 0.2 * torch.randn((L, D), device=DEV, generator=gpu)).to(dt)
        s["kw"] = (1 + 0.2 * torch.randn((L, D), device=DEV, generator=gpu)).to(dt)
    if c["rope"]:
        s["inv_freq"] = (500000.0 ** (-torch.arange(0, c["rope"], 2, dtype=torch.float64) / c["rope"])).float().to(DEV)
    if own:
        from agent_kv_cache_lse_b200 import kvc
        one = torch.zeros((seqs * L * H, 1), dtype=torch.int32, device=DEV)
        s["cache"] = kvc.Cache(s["k"], s["v"], one, one[:, 0].contiguous(),
                               torch.zeros((seqs * L * H, P), dtype=torch.int32, device=DEV), None, seqs, L, H)
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    return {"reserve": _plain_reserve, "write": _plain_write, "bounds": _plain_bounds, "select": _plain_select,
            "attend": _plain_attend}[s["op"]](s, c)


def _run_own(s, c):
    from agent_kv_cache_lse_b200 import kvc
    if s["op"] == "reserve":
        o = s["out"]
        kvc.kvc_reserve_slots(s["cache"], s["new_count"], s["next_pos"], 1, s["crf"], s["free"], s["free_count"],
                              o["row_len"], o["free_count"], o["token_start"], o["token_pos"], o["slot_map"],
                              s["workspace"])
        return dict(o, table=s["table"], slot_pos=s["slot_pos"], label=s["label"], crf=s["crf"])
    if s["op"] == "write":
        kvc.kvc_norm_rope_write(s["cache"], s["qkv"], s["pos"], s["slot_map"], s["q_out"], s["qw"], s["kw"], s["eps"],
                                s["inv_freq"], interleaved=c["interleaved"], token_count=s["count"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if s["op"] == "bounds":
        kvc.kvc_block_bounds(s["cache"], s["out"]["bounds"], s["out"]["pos"], s["from_len"])
    elif s["op"] == "select":
        kvc.kvc_select_blocks(s["cache"], s["bounds"], s["pos"], s["q"], s["q_pos"], s["out"]["list"],
                              s["out"]["count"], s["workspace"], sink_blocks=c["sink"], recent_blocks=c["recent"])
    else:
        kvc.kvc_block_attention(s["cache"], s["q"], s["q_pos"], s["out"]["out"], s["out"]["lse"], s["workspace"],
                                s.get("list"), s.get("count"))
    return s["out"]


def _plain_reserve(s, c):
    P, per = c["page"], c["layers"] * c["kv_heads"]
    n, T, o = s["row_len"].long(), s["T"], s["out"]
    rows, mp = s["table"].shape
    start = torch.zeros(c["seqs"] + 1, dtype=torch.int64, device=DEV)
    start[1:] = torch.cumsum(s["new_count"], 0)
    new = s["new_count"].long().repeat_interleave(per, output_size=rows)
    first, end = (n + P - 1) // P, (n + new + P - 1) // P
    need = end - first
    base = s["free_count"] - need.sum()
    take = base + torch.cumsum(need, 0) - need  # the row's first new page on the stack
    lp = torch.arange(mp, device=DEV)[None]
    fresh = (lp >= first[:, None]) & (lp < end[:, None])
    at = (take[:, None] + lp - first[:, None]).clamp(0, s["free"].numel() - 1)
    s["table"].copy_(torch.where(fresh, s["free"][at], s["table"]))
    slot = torch.arange(mp * P, device=DEV)[None]
    mine = (slot >= n[:, None]) & (slot < (n + new)[:, None])
    pos = s["next_pos"].long().repeat_interleave(per, output_size=rows)[:, None] + slot - n[:, None]
    s["slot_pos"].copy_(torch.where(mine, pos, s["slot_pos"].long()))
    s["label"].masked_fill_(mine, 1)
    s["crf"].masked_fill_(mine, 0.0)
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(start, t, right=True) - 1
    real = t < start[-1]
    seq = seq.clamp(max=c["seqs"] - 1)
    i = t - start[seq]
    row = seq[:, None] * per + torch.arange(per, device=DEV)[None]
    sl = n[row] + i[:, None]
    page = s["table"][row, (sl // P).clamp(max=mp - 1)].long()
    o["slot_map"].copy_(torch.where(real[:, None], page * P + sl % P, -1).view_as(o["slot_map"]))
    o["token_pos"].copy_(torch.where(real, s["next_pos"][seq] + i, -1))
    o["token_start"].copy_(start)
    o["row_len"].copy_(n + new)
    o["free_count"].copy_(base)
    return dict(o, table=s["table"], slot_pos=s["slot_pos"], label=s["label"], crf=s["crf"])


def _plain_write(s, c):
    T, Hq, H, R = c["tokens"], c["q_heads"], c["kv_heads"], c["rope"]
    x = s["qkv"][:T].float()

    def turned(x, w):
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()[:, None]
        if not R:
            return x
        angle = s["pos"][:T].double()[:, None] * s["inv_freq"].double()
        cos, sin = (f(angle).float()[:, None, None] for f in (torch.cos, torch.sin))
        r = x[..., :R]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., : R // 2], r[..., R // 2:])
        pair = (a * cos - b * sin, a * sin + b * cos)
        r = torch.stack(pair, -1).flatten(-2) if c["interleaved"] else torch.cat(pair, -1)
        return torch.cat((r, x[..., R:]), -1)

    slots = s["slot_map"][:T].reshape(-1)
    D = c["dim"]
    s["q_out"][:T] = turned(x[:, :, :Hq], s["qw"]).to(s["q_out"].dtype)
    s["k"].view(-1, D)[slots] = turned(x[:, :, Hq:Hq + H], s["kw"]).to(s["k"].dtype).reshape(-1, D)
    s["v"].view(-1, D)[slots] = s["qkv"][:T, :, Hq + H:].reshape(-1, D)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _plain_bounds(s, c):
    P, o = c["page"], s["out"]
    rows, mp = s["table"].shape
    n = s["row_len"].long()
    first = torch.zeros_like(n) if s["from_len"] is None else s["from_len"].long() // P
    b = torch.arange(mp, device=DEV)[None]
    todo = (b >= first[:, None]) & (b * P < n[:, None])
    row, b = torch.nonzero(todo, as_tuple=True)
    inside = b[:, None] * P + torch.arange(P, device=DEV) < n[row][:, None]
    k = s["k"][s["table"][row, b].long()].float()
    lo = k.masked_fill(~inside[..., None], math.inf).amin(1)
    hi = k.masked_fill(~inside[..., None], -math.inf).amax(1)
    o["bounds"][row, b] = torch.stack((lo, hi), 1).to(o["bounds"].dtype)
    o["pos"][row, b] = s["slot_pos"].view(rows, mp, P)[row, b].masked_fill(~inside, INT_MAX).amin(1)
    return o


def _plain_select(s, c):
    P, o, k = c["page"], s["out"], c["top_k"]
    rows, mp = s["table"].shape
    q = s["q"].double().view(rows, -1, c["dim"])
    up, down = q.clamp(min=0).sum(1), q.clamp(max=0).sum(1)
    score = (s["bounds"][:, :, 1].double() * up[:, None]).sum(-1) + (s["bounds"][:, :, 0].double() * down[:, None]).sum(-1)
    score = score.masked_fill(score.isnan(), math.inf)
    held = (s["row_len"].long() + P - 1) // P
    b = torch.arange(mp, device=DEV)[None]
    q_pos = s["q_pos"].repeat_interleave(rows // c["seqs"], output_size=rows)
    seen = (b < held[:, None]) & (s["pos"] <= q_pos[:, None])
    always = seen & ((b < c["sink"]) | (b >= held[:, None] - c["recent"]))
    order = torch.sort(score, dim=1, descending=True, stable=True)[1]
    kind = torch.where(always, 0, torch.where(seen, 1, 2)).gather(1, order)
    order = order.gather(1, torch.sort(kind, dim=1, stable=True)[1])[:, :k]
    count = seen.sum(1).clamp(max=k)
    chosen = order.masked_fill(torch.arange(order.shape[1], device=DEV)[None] >= count[:, None], INT_MAX)
    chosen = torch.sort(chosen, 1)[0]
    o["list"].fill_(-1)
    o["list"][:, : order.shape[1]] = chosen.masked_fill(chosen == INT_MAX, -1)
    o["count"].copy_(count)
    return o


def _plain_attend(s, c):
    P, D, o = c["page"], c["dim"], s["out"]
    rows, mp = s["table"].shape
    q = s["q"].float().view(rows, -1, D)
    q_pos = s["q_pos"].repeat_interleave(rows // c["seqs"], output_size=rows)
    slot = torch.arange(mp * P, device=DEV)[None]
    seen = (slot < s["row_len"][:, None]) & (s["slot_pos"] <= q_pos[:, None])
    pages, seen = s["table"], seen.view(rows, mp, P)
    if c["blocks"]:
        b = s["list"].long().clamp(min=0)
        pages = pages.gather(1, b)
        seen = seen.gather(1, b[..., None].expand(-1, -1, P)) & (s["list"] >= 0)[..., None]
    pages, seen = pages.long().clamp(min=0), seen.reshape(rows, 1, -1)
    k = s["k"][pages].view(rows, -1, D).float()
    logit = (q @ k.transpose(1, 2)) / math.sqrt(D)
    logit = logit.masked_fill(~seen, -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    v = s["v"][pages].view(rows, -1, D).float()
    out = (p @ v) / total.clamp(min=1e-30)
    o["out"].copy_(out.view_as(o["out"]))
    o["lse"].copy_((top + torch.log(total)).view_as(o["lse"]))
    return o


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    """Outputs that are whole numbers (slots, choices, positions) have no entry here; the others in 64 bits."""
    c = case
    if c["op"] == "select":
        return None
    s = prepare(case, seed)
    if c["op"] == "reserve":
        crf, per = s["crf"].double(), c["layers"] * c["kv_heads"]
        for r, n in enumerate(s["row_len"].tolist()):
            crf[r, n:n + int(s["new_count"][r // per])] = 0
        return {"crf": crf}
    if c["op"] == "write":
        return _exact_write(c, s)
    P, D = c["page"], c["dim"]
    rows = c["seqs"] * c["layers"] * c["kv_heads"]
    lens, table = s["row_len"].tolist(), s["table"].long()
    if c["op"] == "bounds":
        bounds = s["out"]["bounds"].double()
        for r in range(rows):
            n, old = lens[r], max(0, lens[r] - c["fresh"]) if c["fresh"] else 0
            b0, whole = old // P, n // P
            keys = s["k"][table[r, b0:-(-n // P)]].double()
            if whole > b0:
                bounds[r, b0:whole, 0], bounds[r, b0:whole, 1] = keys[: whole - b0].amin(1), keys[: whole - b0].amax(1)
            if n % P:
                bounds[r, whole, 0], bounds[r, whole, 1] = keys[-1, : n % P].amin(0), keys[-1, : n % P].amax(0)
        return {"bounds": bounds, "pos": None}
    G, H = c["q_heads"] // c["kv_heads"], c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=DEV)
    for r in range(rows):
        i, l, h = r // (c["layers"] * H), r // H % c["layers"], r % H
        blocks = torch.arange(-(-lens[r] // P), device=DEV)
        if c["blocks"]:
            blocks = s["list"][r, : int(s["count"][r])].long()
        slots = (blocks[:, None] * P + torch.arange(P, device=DEV)).flatten()
        keep = (slots < lens[r]) & (s["slot_pos"][r, slots] <= s["q_pos"][i])
        slots = slots[keep]
        if slots.numel() == 0:
            continue
        where = table[r, slots // P] * P + slots % P
        k, v = (s[x].view(-1, D)[where].double() for x in ("k", "v"))
        logit = torch.einsum("gd,nd->gn", s["q"][i, l, h * G:(h + 1) * G].double(), k) * D ** -0.5
        out[i, l, h * G:(h + 1) * G] = torch.einsum("gn,nd->gd", torch.softmax(logit, -1), v)
        lse[i, l, h * G:(h + 1) * G] = torch.logsumexp(logit, -1)
    return {"out": out, "lse": lse}


def _exact_write(c, s):
    T, Hq, H, D, R = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"], c["rope"]
    q, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
    step = max(1, (1 << 26) // (c["layers"] * (Hq + 2 * H) * D))
    for t0 in range(0, T, step):
        t = torch.arange(t0, min(T, t0 + step), device=DEV)
        x = s["qkv"][t].double()
        for lo, hi, w in ((0, Hq, s["qw"]), (Hq, Hq + H, s["kw"])):
            y = x[:, :, lo:hi]
            if w is not None:
                y = y / (y.square().sum(-1, keepdim=True) / D + s["eps"]).sqrt() * w.double().view(1, -1, 1, D)
            if R:
                even = torch.arange(0, R, 2, device=DEV) if c["interleaved"] else torch.arange(R // 2, device=DEV)
                odd = even + 1 if c["interleaved"] else even + R // 2
                z = torch.complex(y[..., even], y[..., odd])
                turn = s["pos"][t].double().view(-1, 1, 1, 1) * s["inv_freq"].double()
                z = z * torch.polar(torch.ones_like(turn), turn)
                y = y.clone()
                y[..., even], y[..., odd] = z.real, z.imag
            x[:, :, lo:hi] = y
        q[t] = x[:, :, :Hq]
        where = s["slot_map"][t].flatten()
        k.view(-1, D)[where] = x[:, :, Hq:Hq + H].reshape(-1, D)
        v.view(-1, D)[where] = x[:, :, Hq + H:].reshape(-1, D)
    return {"q": q, "k": k, "v": v}
