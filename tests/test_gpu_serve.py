"""One model step over the paged cache on the GPU, each entry point against oracle.serve.

Whole numbers (slots, tables, choices) and page bounds are compared exactly.  Rounding bounds, in units of u = 2^-24
(half a step of fp32, relative):
* norm and rotation: the sum of D <= 128 squares carries at most (8 + 5) u, the mean, eps and rsqrtf 2 u + 4 u, halved or
  not at most 13 u for the factor with the two products; cos and sin are off by at most 2 pi 2^-26 (the turn rounded to
  fp32) + 2 ulp of sincospif = 7 u + 4 u; the rotation's two products and sum add 3 u.  In all below 32 u = 2^-19 of the
  magnitudes an element is made of, and half a step of the output's type on top.
* attention: a logit's error is at most e = 8 * 2^-22 of the largest sum |q_d k_d| / sqrt(D) (eight tensor-core steps of 16
  products, or twelve fp32 additions), plus 4 u of the logit itself (scale, difference, ex2.approx); probabilities enter
  numerator and denominator, so out is off by 2 e, plus u for each of the sums' terms: at most 3 n / 8 additions for n slots
  (three parts a chunk of 16, or one a step of at least 2 keys in a chunk of 8), relative to sum p |v|; lse by e and half that.
"""
import numpy as np
import pytest
import torch

from agent_kv_cache_lse_b200 import kvc
from oracle import serve
from tests.serve_cases import DT, cache_of, coords, np64, row_kv, step

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
I32 = torch.int32


def status():
    return torch.zeros(2, dtype=I32, device=DEV)


def code(st):
    torch.cuda.synchronize()
    return kvc.device_status(st)[0]


def words(nbytes):
    return torch.full((nbytes // 8 + 1,), -1, dtype=torch.int64, device=DEV)


# -- slots -----------------------------------------------------------------------------------------------------------

def reserve_case(lengths, counts, P, S, L, H, seed, spare=None, max_tokens=None, nxt=None, spoil=None, optional=True,
                 in_place=False, extra_pages=None, deeper=0):
    c, free = cache_of(lengths, P, 64, "bf16", S, L, H, seed, spare=0, extra_pages=extra_pages or -(-max(counts + [1]) // P) + 1)
    per = L * H
    need = sum(max(0, -(-(n + max(0, counts[r // per])) // P) - -(-n // P)) for r, n in enumerate(lengths))
    spare = need + 3 if spare is None else need + spare
    num = c.k_pool.shape[0]
    g = torch.Generator().manual_seed(seed)
    free = torch.randperm(max(spare, 1), generator=g).to(I32) + num
    c.k_pool = c.v_pool = torch.zeros((num + max(spare, 1), P, 64), dtype=torch.bfloat16)
    if spoil:
        spoil(c, free)
    crf = torch.rand((c.rows, c.max_slots), generator=g) if optional else None
    if not optional:
        c.slot_label = None
    cnt = torch.tensor(counts, dtype=I32)
    nxt = torch.tensor(nxt if nxt is not None else [100 * (s + 1) for s in range(S)], dtype=I32)
    total = sum(max(0, x) for x in counts)
    T = total + 2 if max_tokens is None else max_tokens
    depth = spare + deeper
    h = lambda t: None if t is None else t.numpy()
    want = serve.reserve_slots(h(c.block_table), h(c.row_len), h(c.slot_pos), h(c.slot_label), h(crf), h(cnt), h(nxt), 2,
                               h(free), depth, T, L, H, P, c.k_pool.shape[0])
    d = lambda t: None if t is None else t.to(DEV)
    c = kvc.Cache(*(d(t) for t in (c.k_pool, c.v_pool, c.block_table, c.row_len, c.slot_pos, c.slot_label)), S, L, H)
    crf, st = d(crf), status()
    fc = torch.tensor([depth], device=DEV)
    rl = c.row_len if in_place else torch.full_like(c.row_len, 77)
    fo = fc if in_place else torch.full_like(fc, 77)
    ts = torch.full((S + 1,), 77, dtype=I32, device=DEV)
    tp, sm = torch.full((T,), 77, dtype=I32, device=DEV), torch.full((T, L, H), 77, dtype=torch.int64, device=DEV)
    old = c.row_len.clone()
    kvc.kvc_reserve_slots(c, d(cnt), d(nxt), 2, crf, d(free), fc, rl, fo, ts, tp, sm,
                          words(kvc.kvc_reserve_workspace_bytes(c.rows)), st)
    got = code(st)
    same = lambda t, w: np.testing.assert_array_equal(t.cpu().numpy(), w)
    same(rl, want["row_len"])
    same(c.block_table, want["bt"])
    same(c.slot_pos, want["slot_pos"])
    same(sm, want["slot_map"])
    same(tp, want["token_pos"])
    same(ts, want["token_start"])
    assert int(fo[0]) == want["depth"]
    if optional:
        same(c.slot_label, want["slot_label"])
        same(crf, want["crf"])
    if not in_place:
        assert torch.equal(c.row_len, old) and int(fc[0]) == depth
    return got, want


@pytest.mark.parametrize("P", [16, 12, 1])
@pytest.mark.parametrize("counts", [[1, 1, 1], [0, 17, 100], [0, 0, 0], [33, 0, 1]])
def test_reserve(P, counts):
    lengths = [0, 1, P - 1, P, P + 1, 5 * P, 100, 7, 64, 31, 32, 33]
    got, want = reserve_case(lengths, counts, P, 3, 2, 2, seed=P + sum(counts))
    assert got == 0 and not want["refused"]


def test_reserve_in_place_many_rows_without_optional_arrays():
    rng = np.random.default_rng(5)
    lengths = rng.integers(0, 90, 1100 * 2).tolist()
    counts = rng.integers(0, 4, 1100).tolist()
    assert reserve_case(lengths, counts, 16, 1100, 1, 2, 6, optional=False, in_place=True)[0] == 0
    assert reserve_case(lengths[:8], [700, 0, 1, 2000], 16, 4, 1, 2, 7, in_place=True)[0] == 0
    lengths = rng.integers(0, 40, 2500 * 2).tolist()  # more than four rows a planning thread
    got, want = reserve_case(lengths, rng.integers(0, 4, 2500).tolist(), 16, 2500, 1, 2, 9, in_place=True)
    assert got == 0 and not want["refused"]


def test_reserve_exact_stack_and_tokens():
    lengths, counts = [0, 16, 5, 40], [20, 3]
    assert reserve_case(lengths, counts, 16, 2, 1, 2, 8, spare=0, max_tokens=23)[0] == 0
    got, want = reserve_case(lengths, counts, 16, 2, 1, 2, 8, deeper=1)  # a depth past the end of the stack's array
    assert got == 5 and -1 in want["refused"]
    got, want = reserve_case([5, 6], [1], 16, 1, 1, 2, 8, spare=0, deeper=-1)  # below none, though no page is needed
    assert got == 5 and -1 in want["refused"]
    got, want = reserve_case(lengths, counts, 16, 2, 1, 2, 8, spare=-1)
    assert got == 5 and -1 in want["refused"]
    got, want = reserve_case(lengths, counts, 16, 2, 1, 2, 8, max_tokens=22)
    assert got == 2 and -1 in want["refused"]
    assert reserve_case([3, 4], [0, 0], 16, 2, 1, 1, 8, max_tokens=0)[0] == 0


def test_reserve_refused_rows_leave_the_others():
    def bad_page(c, free):
        c.block_table[1, 0] = c.k_pool.shape[0] + 9

    def bad_length(c, free):
        c.row_len[2] = -4

    def bad_free(c, free):
        free[:] = c.k_pool.shape[0] + 1000
    lengths = [5, 5, 30, 16]
    got, want = reserve_case(lengths, [3, 2], 16, 2, 1, 2, 9, spoil=bad_page)
    assert got == 1 and want["refused"] == {1: "page"}
    got, want = reserve_case(lengths, [3, 2], 16, 2, 1, 2, 9, spoil=bad_length)
    assert got == 2 and want["refused"] == {2: "length"}
    got, want = reserve_case([5, 60, 30, 16], [3, 20], 16, 2, 1, 2, 9, extra_pages=1)
    assert got == 0
    got, want = reserve_case([5, 5, 79, 16], [3, 20], 16, 2, 1, 2, 9, extra_pages=1)
    assert got == 5 and want["refused"] == {2: "full"}
    got, want = reserve_case(lengths, [3, 2], 16, 2, 1, 2, 9, nxt=[-1, 4])
    assert got == 2 and set(want["refused"]) == {0, 1}
    got, want = reserve_case(lengths, [3, 2], 16, 2, 1, 2, 9, nxt=[2**31 - 4, 2**31 - 2])
    assert got == 2 and set(want["refused"]) == {2, 3}
    assert reserve_case(lengths, [-3, 2], 16, 2, 1, 2, 9)[0] == 2
    assert reserve_case(lengths, [14, 2], 16, 2, 1, 2, 9, spoil=bad_free)[0] == 1


# -- norms and rotation -----------------------------------------------------------------------------------------------

def write_case(T, L, Hq, H, D, dtype, P=16, R=None, interleaved=False, norm=(True, True), present=None, pad=0, skip=(),
               far=None, spoil=None, seed=1, eps=1e-6, check_code=0):
    g = torch.Generator().manual_seed(seed)
    dt, R = DT[dtype], D if R is None else R
    num = -(-(T * L * H + 3) // P) + 1
    k, v = (torch.randn((num, P, D), generator=g).to(dt) for _ in range(2))
    wide = torch.randn((T, L * (Hq + 2 * H) * D + pad), generator=g).to(dt)
    if spoil:
        spoil(wide)
    qkv = lambda w: w[:, : L * (Hq + 2 * H) * D].view(T, L, Hq + 2 * H, D)
    sm = torch.randperm(num * P, generator=g)[: T * L * H].view(T, L, H).contiguous()
    for t, l, h, value in skip:
        sm[t, l, h] = value
    pos = torch.randint(0, far or 40000, (T,), generator=g).to(I32)
    ws = [(1 + 0.3 * torch.randn((L, D), generator=g)).to(dt) if n else None for n in norm]
    inv = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float() if R else None
    d = lambda t: None if t is None else t.to(DEV)
    cache = kvc.Cache(d(k), d(v), torch.zeros((L * H, 1), dtype=I32, device=DEV), torch.zeros(L * H, dtype=I32, device=DEV),
                      torch.zeros((L * H, P), dtype=I32, device=DEV), None, 1, L, H)
    q0 = torch.randn((T, L, Hq, D), generator=g).to(dt)
    out, st = d(q0), status()
    count = None if present is None else torch.tensor([present], dtype=I32, device=DEV)
    kvc.kvc_norm_rope_write(cache, qkv(d(wide)), d(pos), d(sm), out, *(d(w) for w in ws), eps, d(inv), interleaved, count, st)
    assert code(st) == check_code
    n = T if present is None else max(0, min(present, T))
    x, freq = np64(qkv(wide)), [] if inv is None else np64(inv)
    want_k, tol_k = np64(k).reshape(-1, D), np.zeros((num * P, D))
    want_q, tol_q = np64(q0), np.zeros((T, L, Hq, D))
    half = step(dt)

    def put(want, tol, at, y, reach):
        want[at], tol[at] = y, reach * 32 * U + np.abs(y) * half
    w64 = [None if w is None else np64(w) for w in ws]
    yq, rq = serve.norm_rope(x[:n, :, :Hq], w64[0], eps, pos[:n].numpy(), freq, interleaved)
    put(want_q, tol_q, slice(0, n), yq, rq)
    yk, rk = serve.norm_rope(x[:n, :, Hq:Hq + H], w64[1], eps, pos[:n].numpy(), freq, interleaved)
    want_v = np64(v).reshape(-1, D)
    for t in range(n):
        for l in range(L):
            for h in range(H):
                s = int(sm[t, l, h])
                if 0 <= s < num * P:
                    put(want_k, tol_k, s, yk[t, l, h], rk[t, l, h])
                    want_v[s] = x[t, l, Hq + H + h]
    assert (np.abs(np64(out) - want_q) <= tol_q).all()
    assert (np.abs(np64(cache.k_pool).reshape(-1, D) - want_k) <= tol_k).all()
    assert np.array_equal(np64(cache.v_pool).reshape(-1, D), want_v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope(dtype, D, interleaved):
    write_case(37, 2, 6, 2, D, dtype, interleaved=interleaved)
    write_case(1, 1, 1, 1, D, dtype, interleaved=interleaved, seed=2)
    write_case(5, 1, 7, 1, D, dtype, R=D // 2, interleaved=interleaved, seed=3, P=12)
    write_case(5, 3, 4, 4, D, dtype, R=48, interleaved=interleaved, norm=(True, False), seed=4, P=1)
    write_case(5, 1, 8, 2, D, dtype, R=16, interleaved=interleaved, norm=(False, False), seed=5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_rope_edges(dtype):
    write_case(9, 1, 4, 2, 128, dtype, R=0)
    write_case(300, 1, 4, 1, 64, dtype, far=1 << 24, seed=6)           # far positions keep their angles
    write_case(9, 1, 4, 2, 64, dtype, pad=64, seed=7)                   # tokens inside a wider array
    write_case(9, 1, 4, 2, 64, dtype, present=5, seed=8)                # rows behind the last token stay
    write_case(9, 1, 4, 2, 64, dtype, present=0, seed=8)
    write_case(9, 1, 4, 2, 64, dtype, present=-2, seed=8)
    write_case(9, 1, 4, 2, 64, dtype, present=50, seed=8)
    write_case(9, 1, 4, 2, 64, dtype, skip=[(0, 0, 0, -1), (8, 0, 1, -1)], seed=9)
    write_case(9, 1, 4, 2, 64, dtype, skip=[(3, 0, 1, 1 << 40)], seed=9, check_code=1)
    write_case(9, 1, 4, 2, 64, dtype, skip=[(3, 0, 1, -7)], seed=9, check_code=1)
    write_case(4, 1, 4, 2, 64, dtype, spoil=lambda w: w[1].zero_(), seed=10)             # a zero vector
    write_case(4, 1, 4, 2, 64, dtype, spoil=lambda w: w.mul_(1e-12), eps=0.0, seed=11)
    write_case(4, 1, 4, 2, 64, dtype, spoil=lambda w: w.mul_(1e15), seed=12)
    write_case(2500, 1, 4, 1, 64, dtype, seed=13)                       # more tokens than CTAs


# -- page bounds ------------------------------------------------------------------------------------------------------

LENGTHS = [0, 1, 15, 16, 17, 100, 255, 256]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 12, 1, 40])
def test_bounds(dtype, D, P):
    c, _ = cache_of(LENGTHS, P, D, dtype, 2, 2, 2, seed=P, device=DEV)
    rows, mp = c.block_table.shape
    for from_len in (None, [0, 0, 14, 16, 3, 77, 250, 400]):
        bounds = torch.full((rows, mp, 2, D), 7.0, dtype=DT[dtype], device=DEV)
        pos, st = torch.full((rows, mp), -7, dtype=I32, device=DEV), status()
        fl = None if from_len is None else torch.tensor(from_len, dtype=I32, device=DEV)
        kvc.kvc_block_bounds(c, bounds, pos, fl, st)
        assert code(st) == 0
        want, want_pos = np.full(bounds.shape, 7.0), np.full(pos.shape, -7)
        for r in range(rows):
            k, _, sp = row_kv(c, r)
            for b, (lo, hi, first) in enumerate(serve.block_bounds(k, sp, P)):
                if from_len is None or b >= from_len[r] // P:
                    want[r, b, 0], want[r, b, 1], want_pos[r, b] = lo, hi, first
        np.testing.assert_array_equal(np64(bounds), want)
        np.testing.assert_array_equal(pos.cpu().numpy(), want_pos)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bounds_of_keys_that_are_not_finite_and_bad_pages(dtype):
    c, _ = cache_of([40, 40, 40], 16, 64, dtype, 3, 1, 1, seed=3, device=DEV)
    rows, mp = c.block_table.shape
    c.k_pool[c.block_table[0, 1], 5, 3] = float("nan")
    c.k_pool[c.block_table[0, 2], 9, 3] = float("nan")  # past the row's length: not read
    c.k_pool[c.block_table[0, 0], 2, 4] = float("-inf")
    c.block_table[1, 1], c.row_len[2] = c.k_pool.shape[0], mp * 16 + 1
    bounds = torch.full((rows, mp, 2, 64), 7.0, dtype=DT[dtype], device=DEV)
    pos, st = torch.full((rows, mp), -7, dtype=I32, device=DEV), status()
    kvc.kvc_block_bounds(c, bounds, pos, None, st)
    assert code(st) in (1, 2)
    b = np64(bounds)
    assert np.isnan(b[0, 1, :, 3]).all() and not np.isnan(b[0, 2]).any() and b[0, 0, 0, 4] == -np.inf
    assert (b[1, 1] == 7).all() and int(pos[1, 1]) == 2**31 - 1 and (b[2] == 7).all() and (pos[2] == -7).all()


# -- the choice of pages ----------------------------------------------------------------------------------------------

def select(c, bounds, pos, q, q_pos, k, sink=0, recent=0):
    rows, mp = c.block_table.shape
    li, n, st = torch.full((rows, k), 77, dtype=I32, device=DEV), torch.full((rows,), 77, dtype=I32, device=DEV), status()
    kvc.kvc_select_blocks(c, bounds, pos, q, q_pos, li, n, words(kvc.kvc_select_blocks_workspace_bytes(rows, mp)), sink,
                          recent, st)
    return li, n, code(st)


def check_select(c, bounds, pos, q, q_pos, k, sink=0, recent=0):
    li, n, got = select(c, bounds, pos, q, q_pos, k, sink, recent)
    assert got == 0
    G, b64, P = q.shape[2] // c.num_kv_heads, np64(bounds), c.page_size
    for r in range(c.rows):
        s, l, h = coords(c, r)
        held = -(-int(c.row_len[r]) // P)
        rated = [(b64[r, b, 0], b64[r, b, 1], int(pos[r, b])) for b in range(held)]
        want = serve.select_blocks(rated, np64(q[s, l, h * G:(h + 1) * G]), int(q_pos[s]), k, sink, recent)
        assert li[r].tolist() == want + [-1] * (k - len(want)) and int(n[r]) == len(want), r


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P,G", [(16, 4), (12, 1), (1, 7), (16, 20)])
def test_select(dtype, D, P, G):
    lengths = [0, 1, P, 5 * P - 1, 100, 33 * P, 200, 64]
    c, _ = cache_of(lengths, P, D, dtype, 2, 2, 2, seed=P + D, device=DEV)
    rows, mp = c.block_table.shape
    g = torch.Generator().manual_seed(G)
    q = torch.randn((2, 2, 2 * G, D), generator=g).to(DT[dtype]).to(DEV)
    bounds = torch.full((rows, mp, 2, D), float("nan"), dtype=DT[dtype], device=DEV)
    pos = torch.zeros((rows, mp), dtype=I32, device=DEV)
    kvc.kvc_block_bounds(c, bounds, pos)
    for q_pos in ([2**31 - 1] * 2, [40, 0], [-1, 3 * P]):
        qp = torch.tensor(q_pos, dtype=I32, device=DEV)
        for k, sink, recent in ((1, 0, 0), (4, 1, 1), (9, 0, 9), (300, 2, 1)):
            check_select(c, bounds, pos, q, qp, k, sink, recent)


def test_select_long_rows_and_ties():
    """Rows of thousands of pages; scores that repeat, that are all the same, and neighbours one step apart."""
    D, P = 64, 16
    c, _ = cache_of([5000 * P + 3, 700 * P, 2600 * P], P, D, "f32", 3, 1, 1, seed=5, device=DEV, late=False)
    rows, mp = c.block_table.shape
    g = torch.Generator(device=DEV).manual_seed(6)
    q = torch.randn((3, 1, 1, D), device=DEV, generator=g)
    qp = torch.full((3,), 2**31 - 1, dtype=I32, device=DEV)
    pos = torch.zeros((rows, mp), dtype=I32, device=DEV)
    few = torch.randn((9, D), device=DEV, generator=g)[torch.randint(0, 9, (rows, mp), device=DEV, generator=g)]
    for lo in (few, torch.zeros_like(few), torch.randn(few.shape, device=DEV, generator=g),
               torch.randint(0, 2, few.shape, device=DEV, generator=g) * 2.0**-23 + 1):
        bounds = torch.stack((lo, lo + 1), 2).contiguous()
        for k in (3, 64, 1000, 6000):
            check_select(c, bounds, pos, q, qp, k, 1, 2)
    check_select(c, bounds, pos, torch.zeros_like(q), qp, 100)


def test_select_values_that_are_not_finite():
    c, _ = cache_of([20 * 16, 20 * 16], 16, 64, "f32", 2, 1, 1, seed=7, device=DEV, late=False)
    mp = c.block_table.shape[1]
    b = torch.randn((2, mp, 2, 64), device=DEV).sort(2)[0].contiguous()
    b[0, 3, 0, 5], b[0, 7, 1, 1], b[0, 9, 0, 2] = float("nan"), float("inf"), float("-inf")
    q = torch.randn((2, 1, 2, 64), device=DEV).abs()
    q[1, 0, 1, 3] = float("nan")
    pos, qp = torch.zeros((2, mp), dtype=I32, device=DEV), torch.zeros(2, dtype=I32, device=DEV)
    for k in (1, 2, 3, 19):
        check_select(c, b, pos, q, qp, k)


def test_select_bad_length():
    c, _ = cache_of([40, 40], 16, 64, "f32", 2, 1, 1, seed=7, device=DEV)
    c.row_len[0] = -1
    mp = c.block_table.shape[1]
    b, q = torch.randn((2, mp, 2, 64), device=DEV), torch.randn((2, 1, 2, 64), device=DEV)
    li, n, got = select(c, b, torch.zeros((2, mp), dtype=I32, device=DEV), q, torch.full((2,), 9, dtype=I32, device=DEV), 2)
    assert got == 2 and n.tolist() == [0, 2] and li[0].tolist() == [-1, -1]


# -- attention --------------------------------------------------------------------------------------------------------

def attend(c, q, q_pos, li=None, n=None, st=None):
    S, L, Hq, D = q.shape
    out, lse = torch.full((S, L, Hq, D), 77.0, device=DEV), torch.full((S, L, Hq), 77.0, device=DEV)
    st = status() if st is None else st
    ws = words(kvc.kvc_block_attention_workspace_bytes(c.rows, Hq // c.num_kv_heads, D))
    kvc.kvc_block_attention(c, q, q_pos, out, lse, ws, li, n, st)
    return out, lse, st


def check_attention(c, q, q_pos, li=None, n=None, rows=None, want_code=0):
    out, lse, st = attend(c, q, q_pos, li, n)
    assert code(st) == want_code
    G, P = q.shape[2] // c.num_kv_heads, c.page_size
    for r in range(c.rows) if rows is None else rows:
        s, l, h = coords(c, r)
        hs = slice(h * G, (h + 1) * G)
        k, v, pos = row_kv(c, r)
        slots = None
        if li is not None:
            b = li[r, : int(n[r])].cpu().numpy().astype(np.int64)
            slots = (b[:, None] * P + np.arange(P)).ravel()
            slots = slots[slots < len(k)]
        wo, wl, reach, big = serve.attention(np64(q[s, l, hs]), k, v, pos, int(q_pos[s]), slots)
        count = len(k) if slots is None else len(slots)
        top = np.abs(wl[np.isfinite(wl)]).max(initial=0)
        e = 8 * 2.0 ** -22 * big + 4 * U * (big + top + np.log(count + 1) + 10)
        sums = (3 * count / 8 + 20) * U
        go, gl = np64(out[s, l, hs]), np64(lse[s, l, hs])
        assert (np.abs(go - wo) <= (2 * e + 2 * sums) * reach + 1e-38).all(), (r, np.abs(go - wo).max())
        if np.isfinite(wl).all():
            assert (np.abs(gl - wl) <= e + sums + 2 * U * np.abs(wl)).all(), (r, np.abs(gl - wl).max())
        else:
            assert np.array_equal(gl, wl) and (go == 0).all()
    return out, lse


def a_list(c, take, seed):
    """Random ascending pages of each row: (list, count)."""
    rng = np.random.default_rng(seed)
    li = np.full((c.rows, take), -1, dtype=np.int32)
    n = np.zeros(c.rows, dtype=np.int32)
    for r in range(c.rows):
        held = -(-int(c.row_len[r]) // c.page_size)
        n[r] = min(held, rng.integers(0, take + 1) if r % 3 else take)
        li[r, : n[r]] = np.sort(rng.choice(held, n[r], replace=False))
    return torch.from_numpy(li).to(DEV), torch.from_numpy(n).to(DEV)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 8, 12, 32, 5])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 7, 8])
def test_attention(dtype, D, P, G):
    lengths = [0, 1, P, 5 * P - 1, 100, 33 * P + 1, 1000, 64]
    c, _ = cache_of(lengths, P, D, dtype, 2, 2, 2, seed=P + G, device=DEV)
    q = torch.randn((2, 2, 2 * G, D), generator=torch.Generator().manual_seed(G)).to(DT[dtype]).to(DEV)
    li, n = a_list(c, 9, P * G)
    for q_pos in ([2**31 - 1] * 2, [70, -1]):
        qp = torch.tensor(q_pos, dtype=I32, device=DEV)
        check_attention(c, q, qp)
        check_attention(c, q, qp, li, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_one_long_row(dtype):
    c, _ = cache_of([20011], 16, 128, dtype, 1, 1, 1, seed=3, device=DEV)
    q = torch.randn((1, 1, 4, 128), generator=torch.Generator().manual_seed(2)).to(DT[dtype]).to(DEV)
    qp = torch.full((1,), 2**31 - 1, dtype=I32, device=DEV)
    check_attention(c, 3 * q, qp)
    check_attention(c, q, qp - 2**30)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_many_rows(dtype):
    """More rows than runs, empty ones among them: runs that cover several rows and rows that cover several runs."""
    rng = np.random.default_rng(8)
    lengths = (rng.integers(0, 60, 2000) * rng.integers(0, 2, 2000)).tolist()
    lengths[7] = 9000
    c, _ = cache_of(lengths, 16, 64, dtype, 2000, 1, 1, seed=4, device=DEV)
    q = torch.randn((2000, 1, 2, 64), generator=torch.Generator().manual_seed(2)).to(DT[dtype]).to(DEV)
    qp = torch.full((2000,), 2**31 - 1, dtype=I32, device=DEV)
    check_attention(c, q, qp, rows=list(range(0, 2000, 7)) + [7, 1999])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P", [16, 12])
def test_attention_hidden_slots_may_hold_anything(dtype, P):
    c, _ = cache_of([50, 50, 50, 50], P, 64, dtype, 2, 1, 2, seed=5, device=DEV, late=False)
    q = torch.randn((2, 1, 6, 64), generator=torch.Generator().manual_seed(2)).to(DT[dtype]).to(DEV)
    qp = torch.tensor([20, 49], dtype=I32, device=DEV)
    clean = check_attention(c, q, qp)
    for r in range(4):
        first = 21 if r < 2 else 50
        for slot in range(first, -(-50 // P) * P):
            for pool, x in ((c.k_pool, float("nan")), (c.v_pool, float("inf") if slot % 2 else float("nan"))):
                pool[c.block_table[r, slot // P], slot % P] = x
    out, lse, st = attend(c, q, qp)
    assert code(st) == 0 and torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


def test_attention_extreme_logits():
    """Logits hundreds apart, in rising and falling order, and a row whose logits are all hugely negative."""
    c, _ = cache_of([300, 300, 40], 16, 64, "bf16", 3, 1, 1, seed=6, device=DEV, late=False)
    q = torch.full((3, 1, 2, 64), 1.0, dtype=torch.bfloat16, device=DEV)
    rise = torch.arange(304, device=DEV).view(19, 16, 1) / 16.0
    for r, x in ((0, rise), (1, -rise)):
        c.k_pool[c.block_table[r, :19].long()] = x.expand(-1, -1, 64).to(torch.bfloat16)
    c.k_pool[c.block_table[2, :3].long()] -= 3000
    check_attention(c, q, torch.full((3,), 2**31 - 1, dtype=I32, device=DEV))


def test_attention_repeats_bit_for_bit_and_leaves_no_state():
    c, _ = cache_of([3000, 17, 900, 0], 16, 128, "bf16", 2, 1, 2, seed=9, device=DEV)
    q = torch.randn((2, 1, 8, 128), device=DEV).to(torch.bfloat16)
    qp = torch.full((2,), 2**31 - 1, dtype=I32, device=DEV)
    first = attend(c, q, qp)
    for _ in range(5):
        again = attend(c, q, qp)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attention_device_faults():
    c, _ = cache_of([40, 40, 40, 40], 16, 64, "bf16", 4, 1, 1, seed=5, device=DEV, late=False)
    q = torch.randn((4, 1, 2, 64), device=DEV).to(torch.bfloat16)
    qp = torch.full((4,), 2**31 - 1, dtype=I32, device=DEV)
    li = torch.tensor([[0, 2, -1]] * 4, dtype=I32, device=DEV)
    n = torch.full((4,), 2, dtype=I32, device=DEV)
    clean = check_attention(c, q, qp, li, n)

    def spoiled(row, values, count, empty):
        bad, m = li.clone(), n.clone()
        bad[row], m[row] = torch.tensor(values, dtype=I32, device=DEV), count
        out, lse, st = attend(c, q, qp, bad, m)
        assert code(st) == 9 and int(st[1]) == row
        others = [r for r in range(4) if r != row]
        assert torch.equal(out[others], clean[0][others]) and torch.equal(lse[others], clean[1][others])
        if empty:
            assert (out[row] == 0).all() and (lse[row] == -float("inf")).all()
    spoiled(1, [0, 3, -1], 2, False)       # an entry past the row
    spoiled(1, [0, 1, 2], 4, True)         # more entries than the list has
    spoiled(1, [0, 1, 2], -1, True)
    spoiled(1, [2, 2, 0], 2, False)        # the same page twice
    spoiled(1, [2, 1, 0], 3, False)        # falling
    spoiled(1, [-5, 1, 0], 2, False)
    spoiled(1, [1 << 30, 1, 0], 2, False)
    bt = c.block_table.clone()
    c.block_table[2, 0] = 1 << 30
    out, lse, st = attend(c, q, qp, li, n)
    assert code(st) == 1 and int(st[1]) == 2 and torch.equal(out[0], clean[0][0])
    only = serve.attention(np64(q[2, 0]), *row_kv(kvc.Cache(c.k_pool, c.v_pool, bt, c.row_len, c.slot_pos, None, 4, 1, 1), 2),
                           2**31 - 1, np.arange(32, 40))
    assert np.abs(np64(out[2, 0]) - only[0]).max() < 1e-4
    c.block_table.copy_(bt)
    c.row_len[3] = 10**6
    out, lse, st = attend(c, q, qp)
    assert code(st) == 2 and (out[3] == 0).all() and (lse[3] == -float("inf")).all()


def test_pools_past_32_bit_offsets():
    """Pages above element 2^31 of the pool: every entry point gives what it gives on a small pool."""
    lengths, P, D = [300, 77, 0, 1000], 16, 128
    c, _ = cache_of(lengths, P, D, "bf16", 2, 1, 2, seed=11, device=DEV)
    n = c.k_pool.shape[0]
    shift = (1 << 31) // (P * D) + 5
    big = torch.empty((shift + n, P, D), dtype=torch.bfloat16, device=DEV)  # keys and values share it: 4.3 GB
    big[shift:] = c.k_pool
    far = kvc.Cache(big, big, torch.where(c.block_table >= 0, c.block_table + shift, -1), c.row_len, c.slot_pos, None, 2, 1, 2)
    near = kvc.Cache(c.k_pool, c.k_pool, c.block_table, c.row_len, c.slot_pos, None, 2, 1, 2)
    q = torch.randn((2, 1, 8, D), device=DEV).to(torch.bfloat16)
    qp = torch.full((2,), 2**31 - 1, dtype=I32, device=DEV)
    li, m = a_list(c, 9, 1)
    got = []
    for x in (near, far):
        st = status()
        b = torch.zeros((4, c.block_table.shape[1], 2, D), dtype=torch.bfloat16, device=DEV)
        pos = torch.zeros(c.block_table.shape, dtype=I32, device=DEV)
        kvc.kvc_block_bounds(x, b, pos, None, st)
        assert code(st) == 0
        out = attend(x, q, qp)
        some = attend(x, q, qp, li, m)
        assert code(out[2]) == 0 and code(some[2]) == 0
        got.append([b, pos, *out[:2], *some[:2]])
    assert all(torch.equal(x, y) for x, y in zip(*got))
    qkv = torch.randn((3, 1, 6, D), device=DEV).to(torch.bfloat16)
    slots = torch.tensor([5, 17, 40, 41, 100, 200], device=DEV).view(3, 1, 2)
    where = torch.arange(3, dtype=I32, device=DEV)
    for x, at in ((near, slots), (far, slots + shift * P)):
        kvc.kvc_norm_rope_write(x, qkv, where, at, torch.zeros((3, 1, 2, D), dtype=torch.bfloat16, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(big[shift:], c.k_pool)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_queries_and_outputs_at_odd_addresses(dtype):
    """Contiguous arrays that begin anywhere in an allocation."""
    c, _ = cache_of([300, 77, 9, 1000], 16, 64, dtype, 2, 1, 2, seed=12, device=DEV)
    q = torch.randn((2, 1, 6, 64), device=DEV).to(DT[dtype])
    odd = torch.zeros(q.numel() + 1, dtype=DT[dtype], device=DEV)[1:].view(q.shape)
    odd.copy_(q)
    qp = torch.full((2,), 2**31 - 1, dtype=I32, device=DEV)
    want = check_attention(c, q, qp)
    pos = torch.zeros(c.slot_pos.numel() + 1, dtype=I32, device=DEV)[1:].view(c.slot_pos.shape)
    pos.copy_(c.slot_pos)
    moved = kvc.Cache(c.k_pool, c.v_pool, c.block_table, c.row_len, pos, None, 2, 1, 2)
    out = torch.zeros(q.numel() + 1, device=DEV)[1:].view(q.shape)
    lse = torch.zeros(13, device=DEV)[1:].view(2, 1, 6)
    st = status()
    kvc.kvc_block_attention(moved, odd, qp, out, lse, words(kvc.kvc_block_attention_workspace_bytes(4, 3, 64)), None, None, st)
    assert code(st) == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    mp = c.block_table.shape[1]
    b, bp = torch.randn((4, mp, 2, 64), device=DEV).to(DT[dtype]).sort(2)[0].contiguous(), torch.zeros((4, mp), dtype=I32, device=DEV)
    one, other = select(c, b, bp, q, qp, 7), select(moved, b, bp, odd, qp, 7)
    assert torch.equal(one[0], other[0]) and torch.equal(one[1], other[1])


def test_select_scores_that_32_bits_cannot_tell_apart():
    """Pages whose scores differ by less than fp32 resolves, in every order: the choice is that of 64 bits."""
    D, P, n = 128, 16, 600
    c, _ = cache_of([n * P], P, D, "f32", 1, 1, 1, seed=13, device=DEV, late=False)
    mp = c.block_table.shape[1]
    g = torch.Generator(device=DEV).manual_seed(3)
    base = torch.randn((D,), device=DEV, generator=g)
    lo = base.repeat(1, mp, 1).clone()
    where = torch.randint(0, D, (mp,), device=DEV, generator=g)
    ulps = torch.randint(-3, 4, (mp,), device=DEV, generator=g)
    for b in range(mp):
        lo[0, b, where[b]] *= 1 + int(ulps[b]) * 2.0**-23
    bounds = torch.stack((lo, lo + 1), 2).contiguous()
    q = torch.randn((1, 1, 3, D), device=DEV, generator=g)
    pos, qp = torch.zeros((1, mp), dtype=I32, device=DEV), torch.zeros(1, dtype=I32, device=DEV)
    for k in (1, 17, 300, 599):
        check_select(c, bounds, pos, q, qp, k)
    big = bounds * 1e37  # sums past fp32's range: nothing is known in 32 bits
    for k in (1, 17, 300):
        check_select(c, big, pos, 1e3 * q, qp, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("reach", [1e36, 1e38, 1e39, 1e40, 1e42, 1e44])
def test_select_sums_that_leave_fp32(dtype, D, reach):
    """Unlike pages whose sums of magnitudes come to `reach`: single sums past fp32's range of either sign, and sums in range
    of terms that are not.  The choice is that of 64 bits all the same."""
    n = 400
    c, _ = cache_of([n * 16, n * 16], 16, D, dtype, 2, 1, 1, seed=14, device=DEV, late=False)
    mp = c.block_table.shape[1]
    g = torch.Generator(device=DEV).manual_seed(D)
    size = 10 ** (4 * torch.rand((2, mp, 1, 1), device=DEV, generator=g, dtype=torch.float64) - 4)
    b = torch.randn((2, mp, 2, D), device=DEV, generator=g, dtype=torch.float64).clamp(-3, 3).sort(2)[0]
    q = torch.randn((2, 1, 2, D), device=DEV, generator=g, dtype=torch.float64)
    unit = reach ** 0.5 / D ** 0.5  # sums of 2 D terms of about unit * unit
    b, q = (b * size * unit / 3).to(DT[dtype]), (q * unit).to(DT[dtype])
    pos, qp = torch.zeros((2, mp), dtype=I32, device=DEV), torch.zeros(2, dtype=I32, device=DEV)
    for k in (2, 5, 100, 200, 300, 399):
        check_select(c, b.contiguous(), pos, q, qp, k, 1, 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_one_page_past_fp32_among_ordinary_ones(dtype):
    """Lanes of one page overflow with both signs; its score is far below the others'."""
    c, _ = cache_of([40 * 16], 16, 64, dtype, 1, 1, 1, seed=15, device=DEV, late=False)
    mp = c.block_table.shape[1]
    b = torch.ones((1, mp, 2, 64), device=DEV)
    b[:, :, 0] = -1
    b[0, 17, 1, 0:4], b[0, 17, 1, 4:8], b[0, 17, 0] = 3e37, -3.1e37, -3.2e37
    q = torch.full((1, 1, 1, 64), 1e3, device=DEV)
    pos, qp = torch.zeros((1, mp), dtype=I32, device=DEV), torch.zeros(1, dtype=I32, device=DEV)
    for k in (1, 7, 39):
        check_select(c, b.to(DT[dtype]), pos, q.to(DT[dtype]), qp, k)


def test_reserve_with_a_stack_of_no_entries():
    """Tokens that fit the pages a row holds need none; a row that needs one refuses the call."""
    c, _ = cache_of([5, 17], 16, 64, "bf16", 1, 1, 2, seed=3, device=DEV)
    before = c.block_table.clone()
    for new, want in ((3, 0), (12, 5)):
        st, z = status(), lambda *s, dt=I32: torch.zeros(s, dtype=dt, device=DEV)
        sm, old = z(new, 1, 2, dt=torch.int64), c.row_len.tolist()
        kvc.kvc_reserve_slots(c, torch.tensor([new], dtype=I32, device=DEV), z(1), 0, None, z(0), z(1, dt=torch.int64), c.row_len,
                              z(1, dt=torch.int64), z(2), z(new), sm, words(kvc.kvc_reserve_workspace_bytes(2)), st)
        assert code(st) == want
        if want:
            assert c.row_len.tolist() == old and (sm == -1).all()
        else:
            assert c.row_len.tolist() == [n + new for n in old]
            assert sm[:, 0].tolist() == [[int(before[r, n // 16]) * 16 + n % 16 + i for r, n in enumerate(old)] for i in range(new)]
    assert torch.equal(c.block_table, before)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_select_rows_of_more_pages_than_a_cta_keeps(dtype, D):
    """Rows of 20,000 and 16,385 pages (their keys do not fit a CTA's shared memory) beside one that just fits and a short one."""
    c, _ = cache_of([20000, 16385, 16384, 70], 1, D, dtype, 4, 1, 1, seed=16, device=DEV, late=False)
    rows, mp = c.block_table.shape
    g = torch.Generator(device=DEV).manual_seed(D)
    b = torch.randn((rows, mp, 2, D), device=DEV, generator=g).sort(2)[0].to(DT[dtype]).contiguous()
    b[1, 5000:9000] = b[1, 5000]  # many ties
    q = torch.randn((4, 1, 2, D), device=DEV, generator=g).to(DT[dtype])
    pos = torch.randint(0, 10, (rows, mp), device=DEV, generator=g, dtype=I32)
    for q_pos, k, sink, recent in ((9, 1, 0, 0), (9, 300, 1, 2), (4, 7000, 3, 100), (9, 25000, 0, 1)):
        check_select(c, b, pos, q, torch.full((4,), q_pos, dtype=I32, device=DEV), k, sink, recent)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_select_bounds_that_are_not_finite(dtype, D):
    """NaN and both infinities in every place of a word and lane, negative factors among the query's, and a query with a NaN."""
    n = 200
    c, _ = cache_of([n * 16, n * 16], 16, D, dtype, 2, 1, 1, seed=17, device=DEV, late=False)
    mp = c.block_table.shape[1]
    g = torch.Generator(device=DEV).manual_seed(D + 1)
    b = torch.randn((2, mp, 2, D), device=DEV, generator=g).sort(2)[0].to(DT[dtype]).contiguous()
    bad = [float("nan"), float("inf"), float("-inf")]
    for i in range(40):
        b[0, 3 + 4 * i, i % 2, (7 * i) % D] = bad[i % 3]
    q = torch.randn((2, 1, 2, D), device=DEV, generator=g).to(DT[dtype])
    q[1, 0, 1, 3] = float("nan")
    pos, qp = torch.zeros((2, mp), dtype=I32, device=DEV), torch.zeros(2, dtype=I32, device=DEV)
    for k in (1, 17, 40, 41, 120):
        check_select(c, b, pos, q, qp, k)


@pytest.mark.parametrize("D", [64, 128])
def test_select_bf16_scores_that_32_bits_cannot_tell_apart(D):
    """Pages that differ in one element with a tiny factor: by far less than fp32 resolves of the score."""
    n = 600
    c, _ = cache_of([n * 16], 16, D, "bf16", 1, 1, 1, seed=18, device=DEV, late=False)
    mp = c.block_table.shape[1]
    g = torch.Generator(device=DEV).manual_seed(D)
    lo = torch.randn((D,), device=DEV, generator=g).repeat(1, mp, 1).to(torch.bfloat16)
    lo[0, :, D // 2] = torch.randint(-100, 100, (mp,), device=DEV, generator=g).to(torch.bfloat16) / 64
    b = torch.stack((lo, lo + 1), 2).contiguous()
    q = torch.randn((1, 1, 3, D), device=DEV, generator=g)
    q[..., D // 2] = torch.tensor([1e-9, -2e-9, 3e-10], device=DEV)
    pos, qp = torch.zeros((1, mp), dtype=I32, device=DEV), torch.zeros(1, dtype=I32, device=DEV)
    for k in (1, 17, 300, 599):
        check_select(c, b, pos, q.to(torch.bfloat16), qp, k)
