"""What the entry points of one model step over the cache refuse before anything reaches a device."""
import ctypes

import pytest
import torch

from agent_kv_cache_lse_b200 import kvc

BAD, UNSUPPORTED = kvc.KVC_ERR_INVALID_ARGUMENT, kvc.KVC_ERR_UNSUPPORTED
F = ctypes.c_void_p(256)  # never dereferenced


def fake_cache(**kw):
    c = kvc.KvcCache()
    c.num_seqs, c.num_layers, c.num_kv_heads = 1, 1, 2
    c.page_size, c.max_pages_per_row, c.head_dim, c.dtype = 16, 4, 128, kvc.KVC_BF16
    c.block_table = c.row_len = c.slot_pos = c.k_pool = c.v_pool = 256
    c.num_pages = 8
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_reserve_refusals():
    L = kvc.lib()

    def call(cache=None, cnt=F, nxt=F, fp=F, cap=9, fc=F, T=4, rl=F, fo=F, ts=F, tp=F, sm=F, ws=F, nb=1 << 20):
        return L.kvc_reserve_slots(ctypes.byref(cache or fake_cache()), cnt, nxt, 1, None, fp, cap, fc, T, rl, fo, ts, tp, sm,
                                   ws, nb, None, None)
    for name in ("cnt", "nxt", "fp", "fc", "rl", "fo", "ts", "tp", "sm", "ws"):
        assert call(**{name: None}) == BAD, name
    assert call(T=-1) == BAD and call(cap=-1) == BAD and call(nb=8) == BAD and call(ws=ctypes.c_void_p(260)) == BAD
    assert call(cache=fake_cache(page_size=0)) == BAD and call(cache=fake_cache(num_seqs=40000)) == UNSUPPORTED
    assert call(cache=fake_cache(head_dim=96)) == UNSUPPORTED
    assert kvc.kvc_reserve_workspace_bytes(7) == 64 and kvc.kvc_reserve_workspace_bytes(-1) == 0


def test_norm_rope_refusals():
    L = kvc.lib()

    def call(cache=None, qkv=F, stride=6 * 128, T=3, hq=2, qw=None, kw=None, eps=1e-6, inv=F, R=128, flags=0, pos=F, sm=F,
             out=F):
        return L.kvc_norm_rope_write(ctypes.byref(cache or fake_cache()), qkv, stride, T, None, hq, qw, kw,
                                     ctypes.c_float(eps), inv, R, flags, pos, sm, out, None, None)
    for name in ("qkv", "inv", "pos", "sm", "out"):
        assert call(**{name: None}) == BAD, name
    assert call(T=-1) == BAD and call(hq=3) == BAD and call(hq=0) == BAD and call(hq=258, stride=1 << 20) == UNSUPPORTED
    assert call(flags=2) == BAD and call(R=-16) == BAD and call(R=144) == BAD and call(R=40) == UNSUPPORTED
    assert call(stride=6 * 128 - 8) == BAD and call(stride=6 * 128 + 4) == BAD
    assert call(qw=F, eps=-1.0) == BAD and call(kw=F, eps=float("nan")) == BAD and call(qw=F, eps=float("inf")) == BAD
    assert call(qkv=ctypes.c_void_p(264)) == BAD and call(qw=ctypes.c_void_p(264)) == BAD
    assert call(cache=fake_cache(k_pool=0)) == BAD
    assert call(T=0, qkv=None) == kvc.KVC_OK


def test_bounds_refusals():
    L = kvc.lib()
    call = lambda c=None, b=F, p=F: L.kvc_block_bounds(ctypes.byref(c or fake_cache()), None, b, p, None, None)
    assert call(b=None) == BAD and call(p=None) == BAD and call(b=ctypes.c_void_p(264)) == BAD
    assert call(fake_cache(v_pool=0)) == BAD and call(fake_cache(dtype=2)) == UNSUPPORTED


def test_select_refusals():
    L = kvc.lib()

    def call(cache=None, b=F, p=F, q=F, qp=F, hq=8, k=4, sink=0, recent=0, li=F, n=F, ws=F, nb=1 << 20):
        return L.kvc_select_blocks(ctypes.byref(cache or fake_cache()), b, p, q, qp, hq, k, sink, recent, li, n, ws, nb,
                                   None, None)
    for name in ("b", "p", "q", "qp", "li", "n", "ws"):
        assert call(**{name: None}) == BAD, name
    assert call(hq=7) == BAD and call(hq=258) == UNSUPPORTED and call(k=0) == BAD and call(k=(1 << 24) + 1) == BAD
    assert call(sink=-1) == BAD and call(recent=-1) == BAD and call(sink=3, recent=2) == BAD
    assert call(sink=2**31 - 1, recent=2**31 - 1) == BAD
    assert call(nb=63) == BAD and call(ws=ctypes.c_void_p(260)) == BAD and call(b=ctypes.c_void_p(264)) == BAD
    assert call(nb=kvc.kvc_select_blocks_workspace_bytes(2, 4) - 1) == BAD


def test_attention_refusals():
    L = kvc.lib()

    def call(cache=None, q=F, qp=F, hq=8, li=None, stride=0, n=None, out=F, lse=F, ws=F, nb=1 << 30):
        return L.kvc_block_attention(ctypes.byref(cache or fake_cache()), q, qp, hq, li, stride, n, out, lse, ws, nb, None,
                                     None)
    for name in ("q", "qp", "out", "lse", "ws"):
        assert call(**{name: None}) == BAD, name
    assert call(hq=9) == BAD and call(hq=18) == UNSUPPORTED and call(hq=0) == BAD
    assert call(li=F, stride=4) == BAD and call(li=F, n=F) == BAD
    assert call(nb=kvc.kvc_block_attention_workspace_bytes(2, 4, 128) - 1) == BAD
    assert call(ws=ctypes.c_void_p(260)) == BAD and call(cache=fake_cache(k_pool=8)) == BAD


def test_binding_checks():
    """Shapes, types and devices are checked before the C call (CPU tensors: nothing reaches a device)."""
    S, L, H, P, D, mp = 2, 1, 2, 16, 64, 4
    rows, i32 = S * L * H, torch.int32
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)
    bf = torch.bfloat16
    cache = kvc.Cache(z(8, P, D, dt=bf), z(8, P, D, dt=bf), z(rows, mp, dt=i32), z(rows, dt=i32), z(rows, mp * P, dt=i32),
                      None, S, L, H)
    cnt, ws = z(S, dt=i32), z(4096)

    def reserve(cnt=cnt, crf=None, label=1, rl=z(rows, dt=i32), sm=z(5, L, H, dt=torch.int64)):
        kvc.kvc_reserve_slots(cache, cnt, z(S, dt=i32), label, crf, z(9, dt=i32), z(1, dt=torch.int64), rl,
                              z(1, dt=torch.int64), z(S + 1, dt=i32), z(5, dt=i32), sm, ws)
    for kw, text in ((dict(cnt=cnt[:1]), "new_count: shape"), (dict(cnt=cnt.long()), "new_count: dtype"),
                     (dict(crf=z(rows, 3)), "crf: shape"), (dict(label=256), "label"), (dict(rl=z(3, dt=i32)), "row_len_out"),
                     (dict(sm=z(5, H, L, dt=torch.int64)), "slot_map: shape"), ({}, "CUDA")):
        with pytest.raises(kvc.KvcError, match=text):
            reserve(**kw)

    def write(qkv=z(3, L, 8, D, dt=bf), out=z(3, L, 4, D, dt=bf), qw=None, inv=z(16)):
        kvc.kvc_norm_rope_write(cache, qkv, z(3, dt=i32), z(3, L, H, dt=torch.int64), out, qw, None, 1e-6, inv)
    for kw, text in ((dict(qkv=z(3, L, 4, D, dt=bf)), "qkv: shape"), (dict(qkv=z(3, L, 8, D)), "qkv: dtype"),
                     (dict(qkv=z(3, L, 8, 2 * D, dt=bf)[..., ::2]), "contiguous within"),
                     (dict(qkv=z(1, L, 8, D, dt=bf).expand(3, -1, -1, -1)), "overlap"),
                     (dict(out=z(3, L, 3, D, dt=bf)), "q_out: shape"), (dict(qw=z(L, D)), "q_weight: dtype"),
                     (dict(inv=z(16).double()), "inv_freq: dtype"), ({}, "CUDA")):
        with pytest.raises(kvc.KvcError, match=text):
            write(**kw)
    bounds, bp = z(rows, mp, 2, D, dt=bf), z(rows, mp, dt=i32)
    with pytest.raises(kvc.KvcError, match="bounds: shape"):
        kvc.kvc_block_bounds(cache, bounds[:, :2], bp)
    with pytest.raises(kvc.KvcError, match="from_len"):
        kvc.kvc_block_bounds(cache, bounds, bp, z(2, dt=i32))
    with pytest.raises(kvc.KvcError, match="CUDA"):
        kvc.kvc_block_bounds(cache, bounds, bp)
    q, qp, li, n = z(S, L, 4, D, dt=bf), z(S, dt=i32), z(rows, 3, dt=i32), z(rows, dt=i32)
    with pytest.raises(kvc.KvcError, match="q: dtype"):
        kvc.kvc_select_blocks(cache, bounds, bp, q.float(), qp, li, n, ws)
    with pytest.raises(kvc.KvcError, match="block_count: shape"):
        kvc.kvc_select_blocks(cache, bounds, bp, q, qp, li, n[:1], ws)
    out, lse = z(S, L, 4, D), z(S, L, 4)
    with pytest.raises(kvc.KvcError, match="go together"):
        kvc.kvc_block_attention(cache, q, qp, out, lse, ws, li)
    with pytest.raises(kvc.KvcError, match="out: dtype"):
        kvc.kvc_block_attention(cache, q, qp, out.to(bf), lse, ws)
    with pytest.raises(kvc.KvcError, match="CUDA"):
        kvc.kvc_block_attention(cache, q, qp, out, lse, ws, li, n)


def test_push_refusals():
    L = kvc.lib()
    G = ctypes.c_void_p(4096)

    def call(fp=F, cap=9, fc=F, fr=G, n=5, nf=G):
        return L.kvc_push_pages(fp, cap, fc, fr, n, nf, None, None)
    for name in ("fp", "fc", "fr", "nf"):
        assert call(**{name: None}) == BAD, name
    assert call(cap=-1) == BAD and call(n=-1) == BAD and call(nf=F) == BAD
    assert call(fr=F) == BAD and call(fr=ctypes.c_void_p(256 + 32)) == BAD and call(fp=ctypes.c_void_p(4096 + 16)) == BAD
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)
    one = z(1, dt=torch.int64)
    for a, text in (((z(9), z(1), z(5), one), "free_count: dtype"), ((z(9), one, z(5).long(), one), "freed: dtype"),
                    ((z(9), one, z(5, 2)[:, 0], one), "contiguous"), ((z(9), one, z(5), z(2, dt=torch.int64)), "num_freed: shape"),
                    ((z(9), one, z(5), one.clone()), "CUDA")):
        with pytest.raises(kvc.KvcError, match=text):
            kvc.kvc_push_pages(*a)


def test_reserve_asks_for_no_pools():
    """Slots are reserved in the tables alone: the checks after the cache's are reached without pools (num_pages still counts)."""
    L = kvc.lib()

    def call(**kw):
        return L.kvc_reserve_slots(ctypes.byref(fake_cache(k_pool=None, v_pool=None, **kw)), F, F, 1, None, F, 9, F, 4, F, F, F, F,
                                   F, F, 8, None, None)
    assert call() == BAD and b"workspace" in L.kvc_last_error()
    assert call(num_pages=0) == BAD and b"num_pages" in L.kvc_last_error()


def test_reserve_takes_a_stack_without_room():
    """A stack of no entries (a torch tensor of size 0 has no address) serves steps that need no page."""
    L = kvc.lib()

    def call(fp, cap):
        return L.kvc_reserve_slots(ctypes.byref(fake_cache()), F, F, 1, None, fp, cap, F, 4, F, F, F, F, F, F, 8, None, None)
    assert call(None, 1) == BAD and b"free_pages" in L.kvc_last_error()
    assert call(None, 0) == BAD and b"workspace" in L.kvc_last_error()
