"""The entry points of one model step run together (agent_kv_cache_lse_b200.step.ServingStep): after an eviction round, over
many tokens, ragged prompts, on another stream, captured and replayed; everything against oracle.serve."""
import numpy as np
import pytest
import torch

from agent_kv_cache_lse_b200 import kvc, step, synth
from agent_kv_cache_lse_b200.round import EvictionRound
from oracle import serve
from tests import helpers
from tests.serve_cases import DT, cache_of, coords, np64, row_kv, step as half_step
from tests.test_gpu_serve import U, check_attention, check_select

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = torch.int32


def inv_freq(R):
    return (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().to(DEV)


def written(c, rows, qkv, start, counts, next_pos, old_len, w, R):
    """The newest entries of the rows hold the normalised, rotated keys and the values of their tokens."""
    S, L, H = c.num_seqs, c.num_layers, c.num_kv_heads
    Hq = qkv.shape[2] - 2 * H
    x = np64(qkv)
    for r in rows:
        s, l, h = coords(c, r)
        k, v, pos = row_kv(c, r)
        n, new = old_len[r], counts[s]
        assert len(k) == n + new
        at = np.arange(new) + next_pos[s]
        np.testing.assert_array_equal(pos[n:], at)
        t = slice(start[s], start[s] + new)
        want, reach = serve.norm_rope(x[t, l:l + 1, Hq + h:Hq + h + 1], None if w is None else np64(w)[l:l + 1], 1e-6, at,
                                      np64(inv_freq(R)), False)
        tol = reach * 32 * U + np.abs(want) * half_step(c.k_pool.dtype)
        assert (np.abs(k[n:] - want[:, 0, 0]) <= tol[:, 0, 0]).all()
        np.testing.assert_array_equal(v[n:], x[t, l, Hq + H + h])


def test_steps_after_an_eviction_round():
    """A compacted cache (rows of unlike lengths), its freed pages as the stack, 40 decode steps and a ragged extension."""
    spec = synth.batch16(num_seqs=3, num_layers=2, lo=300, hi=700)
    w = helpers.build(spec, DEV)
    rnd = EvictionRound(w.cache)
    budget = torch.tensor([64, 113, 160], dtype=I32, device=DEV)
    rnd.budget.copy_(budget)
    rnd.run(w.queries, None, score_flags=kvc.KVC_SCORE_COMPUTE_LSE)
    torch.cuda.synchronize()
    assert rnd.device_status()[0] == 0
    c, G, D = w.cache, spec.group, spec.head_dim
    assert int(rnd.num_freed[0]) > 0
    ones = (1 + 0.1 * torch.randn((2, D), device=DEV)).to(torch.bfloat16)
    st = step.ServingStep(c, spec.num_q_heads, 64, rnd.freed, rnd.num_freed, top_k=5, q_weight=ones, k_weight=ones,
                          inv_freq=inv_freq(D), crf=rnd.crf)
    next_pos = torch.tensor(spec.ctx, dtype=I32, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(3)
    rows = [0, 7, 8, 23, 31, 47]
    depth = int(rnd.num_freed[0])
    for i in range(40):
        qkv = torch.randn((3, 2, spec.num_q_heads + 16, D), device=DEV, generator=gen).to(torch.bfloat16)
        old = c.row_len.tolist()
        out, lse = st.decode(qkv, next_pos, label=2)
        torch.cuda.synchronize()
        assert st.device_status()[0] == 0, st.device_status()
        if i in (0, 1, 17, 39):
            written(c, rows, qkv, [0, 1, 2], [1, 1, 1], next_pos.tolist(), old, ones, D)
            q = st.q[:3]
            fresh = torch.zeros_like(st.bounds), torch.zeros_like(st.block_pos)
            kvc.kvc_block_bounds(c, *fresh)
            held = (torch.arange(c.block_table.shape[1], device=DEV)[None] * 16 < c.row_len[:, None])
            assert torch.equal(st.bounds[held], fresh[0][held]) and torch.equal(st.block_pos[held], fresh[1][held])
            check_select(c, st.bounds, st.block_pos, q, next_pos, 5, 1, 2)
            again = check_attention(c, q, next_pos, st.block_list, st.block_count, rows=rows)
            assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
        next_pos += 1
    assert (rnd.crf[0, 64:104] == 0).all() and (c.slot_label[0, 64:104] == 2).all()
    taken = sum(-(-(int(n)) // 16) - -(-(int(n) - 40) // 16) for n in c.row_len.tolist())
    assert int(rnd.num_freed[0]) == depth - taken
    used = c.block_table[c.block_table >= 0]
    assert len(torch.unique(used)) == len(used)  # no page in two places
    counts = torch.tensor([30, 0, 17], dtype=I32, device=DEV)
    qkv = torch.randn((50, 2, spec.num_q_heads + 16, D), device=DEV, generator=gen).to(torch.bfloat16)
    old = c.row_len.tolist()
    kept = st.q[47:].clone()
    st.extend(qkv, counts, next_pos)
    torch.cuda.synchronize()
    assert st.device_status()[0] == 0 and torch.equal(st.q[47:], kept)
    written(c, rows, qkv, [0, 30, 30], [30, 0, 17], next_pos.tolist(), old, ones, D)


@pytest.mark.parametrize("top_k", [0, 4])
def test_captured_step_replays_with_new_inputs(top_k):
    c, free = cache_of([100, 31, 64, 7], 16, 64, "bf16", 2, 1, 2, seed=1, spare=40, extra_pages=6, device=DEV)
    stack = free.to(DEV)
    count = torch.tensor([len(free)], device=DEV)
    next_pos = torch.tensor([100, 64], dtype=I32, device=DEV)
    qkv = torch.zeros((2, 1, 8, 64), dtype=torch.bfloat16, device=DEV)
    twin = kvc.Cache(*(t.clone() for t in (c.k_pool, c.v_pool, c.block_table, c.row_len, c.slot_pos, c.slot_label)), 2, 1, 2)
    kw = dict(top_k=top_k, inv_freq=inv_freq(64))
    a = step.ServingStep(c, 4, 2, stack, count, **kw)
    b = step.ServingStep(twin, 4, 2, stack.clone(), count.clone(), **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        a.decode(qkv, next_pos)
        next_pos += 1
    torch.cuda.synchronize()
    assert c.row_len.tolist() == [100, 31, 64, 7]  # capture runs nothing
    for i in range(20):
        x = torch.randn(qkv.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(i)).to(torch.bfloat16)
        qkv.copy_(x)
        here = next_pos.clone()
        g.replay()
        out, lse = b.decode(x, here)
        torch.cuda.synchronize()
        assert a.device_status()[0] == 0 and b.device_status()[0] == 0
        assert torch.equal(a.out, out) and torch.equal(a.lse, lse)
    for x, y in ((c.k_pool, twin.k_pool), (c.v_pool, twin.v_pool), (c.block_table, twin.block_table),
                 (c.row_len, twin.row_len), (c.slot_pos, twin.slot_pos), (c.slot_label, twin.slot_label)):
        assert torch.equal(x, y)
    assert c.row_len.tolist() == [120, 51, 84, 27]
    check_attention(c, a.q, next_pos - 1, *((a.block_list, a.block_count) if top_k else ()))


def test_two_steps_at_once_on_two_streams():
    """Two caches with buffers of their own, their steps interleaved on two streams: the same results as alone."""
    def make(seed):
        c, free = cache_of([900, 31, 640, 70], 16, 128, "bf16", 2, 1, 2, seed=seed, spare=40, extra_pages=6, device=DEV)
        s = step.ServingStep(c, 8, 2, free.to(DEV), torch.tensor([len(free)], device=DEV), top_k=9, inv_freq=inv_freq(128))
        x = torch.randn((30, 2, 1, 12, 128), device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)).to(torch.bfloat16)
        return c, s, x, torch.tensor([900, 640], dtype=I32, device=DEV)

    def run(case, stream):
        c, s, x, pos = case
        with torch.cuda.stream(stream):
            for i in range(30):
                s.decode(x[i], pos)
                pos.add_(1)
                yield s.out.clone()
    alone = []
    for seed in (5, 6):
        stream = torch.cuda.Stream()
        case = make(seed)
        torch.cuda.synchronize()
        alone.append(list(run(case, stream)))
        torch.cuda.synchronize()
    cases, streams = [make(5), make(6)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    both = list(zip(run(cases[0], streams[0]), run(cases[1], streams[1])))
    torch.cuda.synchronize()
    for i in range(30):
        assert torch.equal(both[i][0], alone[0][i]) and torch.equal(both[i][1], alone[1][i])
    assert cases[0][1].device_status()[0] == 0 and cases[1][1].device_status()[0] == 0


def test_binding_without_the_native_module_makes_the_same_calls(monkeypatch):
    def go():
        c, free = cache_of([90, 31, 64, 70], 16, 64, "f32", 2, 1, 2, seed=8, spare=9, extra_pages=3, device=DEV)
        s = step.ServingStep(c, 4, 2, free.to(DEV), torch.tensor([len(free)], device=DEV), top_k=3, inv_freq=inv_freq(32))
        x = torch.randn((2, 1, 8, 64), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
        s.decode(x, torch.tensor([90, 70], dtype=I32, device=DEV))
        torch.cuda.synchronize()
        assert s.device_status()[0] == 0
        return s.out, s.lse, c.k_pool, c.block_table, s.block_list, s.q
    assert kvc._bind is not None
    native = go()
    monkeypatch.setattr(kvc, "_bind", None)
    for x, y in zip(native, go()):
        assert torch.equal(x, y)


def test_calls_the_native_module_hands_back():
    """Refusals have their words, and tokens inside a wider array are taken, with the native module present."""
    c, _ = cache_of([40], 16, 64, "f32", 1, 1, 1, seed=8, device=DEV)
    q, qp = torch.randn((1, 1, 2, 64), device=DEV), torch.zeros(1, dtype=I32, device=DEV)
    out, lse, ws = torch.zeros((1, 1, 2, 64), device=DEV), torch.zeros((1, 1, 2), device=DEV), torch.zeros(1 << 20, device=DEV)
    with pytest.raises(kvc.KvcError, match="q: dtype"):
        kvc.kvc_block_attention(c, q.double(), qp, out, lse, ws)
    with pytest.raises(kvc.KvcError, match="lse: shape"):
        kvc.kvc_block_attention(c, q, qp, out, lse[..., :1], ws)
    with pytest.raises(kvc.KvcError, match="on cpu"):
        kvc.kvc_block_attention(c, q, qp.cpu(), out, lse, ws)
    with pytest.raises(kvc.KvcError, match="workspace"):
        kvc.kvc_block_attention(c, q, qp, out, lse, ws[:4])
    with pytest.raises(kvc.KvcError, match="block_table: shape|slot_pos: shape"):
        kvc.kvc_block_attention(kvc.Cache(c.k_pool, c.v_pool, c.block_table, c.row_len, c.slot_pos[:, :-1].contiguous(), None, 1, 1, 1),
                                q, qp, out, lse, ws)
    with pytest.raises(kvc.KvcError, match="at most 8"):
        big = torch.zeros((1, 1, 9, 64), device=DEV)
        kvc.kvc_block_attention(c, big, qp, torch.zeros_like(big), torch.zeros((1, 1, 9), device=DEV), ws)
    kvc.kvc_block_attention(c, q, qp, out, lse, ws, stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()


def test_a_refused_call_changes_nothing():
    """The step refuses before it reserves: lengths, tables and the stack stay, and the call made right gives what it would have."""
    c, free = cache_of([100, 31, 64, 7], 16, 64, "bf16", 2, 1, 2, seed=2, spare=40, extra_pages=6, device=DEV)
    count, next_pos = torch.tensor([len(free)], device=DEV), torch.tensor([100, 64], dtype=I32, device=DEV)
    st = step.ServingStep(c, 4, 4, free.to(DEV), count, top_k=4, inv_freq=inv_freq(64))
    x = torch.randn((4, 1, 8, 64), device=DEV).to(torch.bfloat16)
    ones = torch.ones(2, dtype=I32, device=DEV)
    before = [t.clone() for t in (c.row_len, c.block_table, c.slot_pos, c.k_pool, c.v_pool, count)]
    big = torch.randn((5, 1, 8, 64), device=DEV).to(torch.bfloat16)
    for bad in (big, x.float(), x[:, :, :7], x[..., ::2], x.cpu()):
        with pytest.raises(kvc.KvcError):
            st.extend(bad, ones, next_pos)
        with pytest.raises(kvc.KvcError):
            st.decode(bad, next_pos)
    with pytest.raises(kvc.KvcError):
        st.decode(x[:1], next_pos)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (c.row_len, c.block_table, c.slot_pos, c.k_pool, c.v_pool, count)))
    assert st.device_status()[0] == 0
    st.decode(x, next_pos)
    torch.cuda.synchronize()
    assert st.device_status()[0] == 0 and c.row_len.tolist() == [101, 32, 65, 8]


@pytest.mark.parametrize("n", [0, 1, 300, 100_003])
def test_push(n):
    """A list on top of a stack, counts moved over; a second push finds nothing; what does not fit stays where it is."""
    cap, depth = n + 20, 20
    stack = torch.arange(cap, dtype=I32, device=DEV)
    freed = torch.arange(n + 7, dtype=I32, device=DEV) + 5_000_000
    fc, nf, st = (torch.tensor(x, device=DEV) for x in ([depth], [n], [0, 0]))
    st = st.to(I32)
    for _ in range(2):
        kvc.kvc_push_pages(stack, fc, freed, nf, st)
        torch.cuda.synchronize()
        assert int(fc[0]) == depth + n and int(nf[0]) == 0 and int(st[0]) == 0
        assert stack.tolist() == list(range(depth)) + list(range(5_000_000, 5_000_000 + n))
    kept = stack.clone()
    for d, m in ((cap - 2, 3), (-1, 1), (cap + 1, 0), (0, -1), (0, n + 8)):
        st.zero_()
        fc.fill_(d)
        nf.fill_(m)
        kvc.kvc_push_pages(stack, fc, freed, nf, st)
        torch.cuda.synchronize()
        assert st.tolist() == [5, -1] and int(fc[0]) == d and int(nf[0]) == m and torch.equal(stack, kept)


@pytest.mark.parametrize("top_k", [0, 4])
def test_pages_go_round_over_several_evictions(top_k):
    """Evict, decode, evict, decode, ...: every page is in one row or once on the stack, whatever was left on it."""
    spec = synth.batch16(num_seqs=3, num_layers=2, lo=300, hi=700)
    w = helpers.build(spec, DEV)
    c, G, D, P = w.cache, spec.group, spec.head_dim, 16
    rnd = EvictionRound(c)
    rnd.budget.copy_(torch.tensor([64, 113, 160], dtype=I32, device=DEV))
    num = c.k_pool.shape[0]
    held = lambda: [p for r in range(c.rows) for p in c.block_table[r, : -(-int(c.row_len[r]) // P)].tolist()]
    free = sorted(set(range(num)) - set(held()))
    stack = torch.full((num,), -7, dtype=I32, device=DEV)
    stack[: len(free)] = torch.tensor(free, dtype=I32, device=DEV)
    count = torch.tensor([len(free)], device=DEV)
    st = step.ServingStep(c, spec.num_q_heads, 3, stack, count, top_k=top_k, inv_freq=inv_freq(D), crf=rnd.crf)
    next_pos = torch.tensor(spec.ctx, dtype=I32, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(9)
    for cycle in range(4):
        rnd.run(w.queries, None, score_flags=kvc.KVC_SCORE_COMPUTE_LSE)
        st.reclaim(rnd.freed, rnd.num_freed)
        for i in range(5 + 20 * cycle):
            qkv = torch.randn((3, 2, spec.num_q_heads + 16, D), device=DEV, generator=gen).to(torch.bfloat16)
            st.decode(qkv, next_pos)
            next_pos += 1
        torch.cuda.synchronize()
        assert rnd.device_status()[0] == 0 and st.device_status()[0] == 0
        pages = held() + stack[: int(count[0])].tolist()
        assert len(pages) == num and sorted(pages) == list(range(num))
    if top_k:
        check_select(c, st.bounds, st.block_pos, st.q[:3], next_pos - 1, 4, 1, 2)
    check_attention(c, st.q[:3], next_pos - 1, *((st.block_list, st.block_count) if top_k else ()), rows=[0, 11, 23, 47])


@pytest.mark.parametrize("native", [True, False])
def test_a_number_that_is_no_stream_is_refused(monkeypatch, native):
    c, _ = cache_of([40], 16, 64, "f32", 1, 1, 1, seed=8, device=DEV)
    mp = c.block_table.shape[1]
    b, pos = torch.zeros((1, mp, 2, 64), device=DEV), torch.full((1, mp), 7, dtype=I32, device=DEV)
    if not native:
        monkeypatch.setattr(kvc, "_bind", None)
    for bad in (1 << 70, -(1 << 70), -1):
        with pytest.raises(kvc.KvcError, match="no stream"):
            kvc.kvc_block_bounds(c, b, pos, stream=bad)
    torch.cuda.synchronize()
    assert (pos == 7).all()
    kvc.kvc_block_bounds(c, b, pos, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert (pos[0, :3] < 7).any()


@pytest.mark.parametrize("top_k", [0, 3])
def test_a_step_on_a_stream_given_by_its_handle(top_k):
    """As the entry points, the step takes a stream object or its address; a step on each of them gives the same."""
    def go(stream):
        c, free = cache_of([90, 31, 64, 70], 16, 64, "bf16", 2, 1, 2, seed=8, spare=9, extra_pages=3, device=DEV)
        s = step.ServingStep(c, 4, 2, free.to(DEV), torch.tensor([len(free)], device=DEV), top_k=top_k, inv_freq=inv_freq(32))
        x = torch.randn((2, 1, 8, 64), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(torch.bfloat16)
        pos, freed = torch.tensor([90, 70], dtype=I32, device=DEV), torch.zeros((0,), dtype=I32, device=DEV)
        none = torch.zeros(1, dtype=torch.int64, device=DEV)
        torch.cuda.synchronize()
        s.decode(x, pos, stream=stream)
        s.reclaim(freed, none, stream=stream)
        torch.cuda.synchronize()
        assert s.device_status()[0] == 0
        return s.out, s.lse, c.k_pool, c.row_len
    side = torch.cuda.Stream()
    want = go(None)
    for stream in (side, side.cuda_stream, 0):
        assert all(torch.equal(x, y) for x, y in zip(want, go(stream)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top_k", [0, 3])
@pytest.mark.parametrize("weights", [True, False])
def test_native_and_python_packing_make_the_same_calls(monkeypatch, dtype, top_k, weights):
    """Every argument a step passes, optional ones among them, arrives the same either way, and a refusal says the same."""
    w = (1 + 0.1 * torch.randn((2, 64), device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))).to(DT[dtype]) if weights else None

    def go():
        c, free = cache_of([90, 31, 64, 70, 1, 0, 16, 33], 16, 64, dtype, 2, 2, 2, seed=8, spare=20, extra_pages=4, device=DEV)
        crf = torch.ones((8, c.max_slots), device=DEV)
        s = step.ServingStep(c, 4, 40, free.to(DEV), torch.tensor([len(free)], device=DEV), top_k=top_k, q_weight=w, k_weight=w,
                             eps=1e-5, inv_freq=inv_freq(48) if weights else None, interleaved=weights, crf=crf if weights else None)
        if not weights:
            c.slot_label = None
        x = torch.randn((37, 2, 8, 64), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(DT[dtype])
        pos = torch.tensor([90, 70], dtype=I32, device=DEV)
        s.extend(x, torch.tensor([30, 5], dtype=I32, device=DEV), pos, label=2)
        s.decode(x[35:], pos + 40, label=1)
        torch.cuda.synchronize()
        assert s.device_status()[0] == 0
        words = []
        for bad in (dict(block_list=torch.zeros((8, 2), dtype=I32, device=DEV)), dict(out=s.out.to(torch.bfloat16)),
                    dict(workspace=s.attend_ws[:1]), dict(q_pos=pos[:1])):
            a = {**dict(q=s.q[:2], q_pos=pos, out=s.out, lse=s.lse, workspace=s.attend_ws), **bad}
            with pytest.raises(kvc.KvcError) as e:
                kvc.kvc_block_attention(c, **a)
            words.append(str(e.value))
        return [s.out, s.lse, s.q, s.slot_map, s.token_pos, s.token_start, s.free_count, crf, c.k_pool, c.v_pool, c.block_table,
                c.row_len, c.slot_pos] + ([s.block_list, s.bounds, s.block_pos] if top_k else []), words
    native = go()
    monkeypatch.setattr(kvc, "_bind", None)
    python = go()
    assert native[1] == python[1] and all(torch.equal(x, y) for x, y in zip(native[0], python[0]))
