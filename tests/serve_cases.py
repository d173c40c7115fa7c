"""Small seeded paged caches for the tests of one model step over the cache."""
import numpy as np
import torch

from agent_kv_cache_lse_b200 import kvc

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def cache_of(lengths, P, D, dtype, S, L, H, seed, spare=0, extra_pages=1, device="cpu", late=True):
    """Rows of the given lengths on permuted pages: (cache, unused page ids).  Positions are a slot's index, one in
    seven of them past every length (entries filled from the end of a trace)."""
    g = torch.Generator().manual_seed(seed)
    rows = S * L * H
    assert len(lengths) == rows
    held = [-(-n // P) for n in lengths]
    mp = max(1, max(held) + extra_pages)
    num = sum(held) + spare + 1
    perm = torch.randperm(num, generator=g).to(torch.int32)
    bt = torch.full((rows, mp), -1, dtype=torch.int32)
    used = 0
    for r, k in enumerate(held):
        bt[r, :k] = perm[used:used + k]
        used += k
    k = torch.randn((num, P, D), generator=g).to(DT[dtype])
    v = torch.randn((num, P, D), generator=g).to(DT[dtype])
    pos = torch.arange(mp * P, dtype=torch.int32).repeat(rows, 1)
    if late:
        pos[torch.rand((rows, mp * P), generator=g) < 1 / 7] += 1 << 20
    lab = torch.randint(0, 3, (rows, mp * P), dtype=torch.uint8, generator=g)
    c = kvc.Cache(*(t.to(device) for t in (k, v, bt, torch.tensor(lengths, dtype=torch.int32), pos, lab)), S, L, H)
    return c, perm[used:].clone()


def row_kv(cache, r):
    """(keys [n, D], values [n, D], positions [n]) of row r in slot order, 64 bits."""
    n, P = int(cache.row_len[r]), cache.page_size
    pages = cache.block_table[r, : -(-n // P)].long()
    k, v = (np64(t[pages]).reshape(-1, t.shape[-1])[:n] for t in (cache.k_pool, cache.v_pool))
    return k, v, cache.slot_pos[r, :n].cpu().numpy()


def coords(cache, r):
    return r // (cache.num_layers * cache.num_kv_heads), r // cache.num_kv_heads % cache.num_layers, r % cache.num_kv_heads


def step(t):
    """Half a step of the type, relative to the value."""
    return torch.finfo(t).eps / 2
