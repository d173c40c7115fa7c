"""What ServingStep refuses, and that it does so before any entry point is called (CPU tensors: nothing reaches a device)."""
import pytest
import torch

from agent_kv_cache_lse_b200 import kvc, step

I32 = torch.int32


def cache_on_cpu(H=2, D=64, dtype=torch.bfloat16, S=3, L=1):
    rows, P, mp = S * L * H, 16, 4
    z = lambda *s, dt=I32: torch.zeros(s, dtype=dt)
    return kvc.Cache(z(8, P, D, dt=dtype), z(8, P, D, dt=dtype), z(rows, mp), z(rows), z(rows, mp * P), None, S, L, H)


def make(Hq=4, max_tokens=5, H=2, **kw):
    return step.ServingStep(cache_on_cpu(H), Hq, max_tokens, torch.zeros(9, dtype=I32), torch.zeros(1, dtype=torch.int64), **kw)


@pytest.mark.parametrize("kw,text", [
    (dict(Hq=3), "num_q_heads"), (dict(Hq=0), "num_q_heads"), (dict(Hq=258), "num_q_heads"), (dict(max_tokens=-1), "max_tokens"),
    (dict(top_k=-1), "top_k"), (dict(top_k=2), "together"), (dict(top_k=9, sink_blocks=-1), "sink_blocks"),
    (dict(top_k=9, sink_blocks=5, recent_blocks=5), "together"),
    (dict(q_weight=torch.zeros(1, 64)), "q_weight: dtype"), (dict(k_weight=torch.zeros(64).bfloat16()), "k_weight: shape"),
    (dict(q_weight=torch.zeros(1, 64).bfloat16(), eps=float("nan")), "eps"),
    (dict(k_weight=torch.zeros(1, 64).bfloat16(), eps=-1e-6), "eps"),
    (dict(inv_freq=torch.zeros(16).double()), "inv_freq: dtype"), (dict(inv_freq=torch.zeros(20)), "multiple of 8"),
    (dict(inv_freq=torch.zeros(40)), "multiple of 8"),
    (dict(k_weight=torch.zeros(65).bfloat16()[1:].view(1, 64)), "16-byte")])
def test_constructor_refusals(kw, text):
    with pytest.raises(kvc.KvcError, match=text):
        make(**kw)


def test_calls_are_refused_before_anything_is_enqueued(monkeypatch):
    called = []
    for name in kvc.EXPORTS:
        if hasattr(kvc, name) and not name.endswith("_bytes"):
            monkeypatch.setattr(kvc, name, lambda *a, _n=name, **k: called.append(_n))
    bf = torch.bfloat16
    x = lambda T=3, heads=8, L=1, D=64, dt=bf: torch.zeros((T, L, heads, D), dtype=dt)
    pos, cnt = torch.zeros(3, dtype=I32), torch.ones(3, dtype=I32)
    st = make(max_tokens=5)
    odd = torch.zeros(3 * 8 * 64 + 1, dtype=bf)[1:].view(3, 1, 8, 64)
    apart = torch.zeros(3 * (8 * 64 + 4), dtype=bf).view(3, -1)[:, :8 * 64].view(3, 1, 8, 64)
    for qkv, text in ((x(6), "at most max_tokens"), (x(heads=9), "query heads"), (x(heads=4), "qkv: shape"), (x(L=2), "qkv: shape"),
                      (x(D=128), "qkv: shape"), (x(dt=torch.float32), "qkv: dtype"), (x()[0], "qkv: shape"), (odd, "aligned"),
                      (apart, "aligned"), (x().expand(3, 1, 8, 64)[:, :, ::2], "qkv: shape|query heads|contiguous"),
                      (x(1).expand(3, -1, -1, -1), "overlap")):
        with pytest.raises(kvc.KvcError, match=text):
            st.extend(qkv, cnt, pos)
        with pytest.raises(kvc.KvcError, match=text):
            st.decode(qkv, pos)
    for kw, text in ((dict(new_count=cnt.long()), "new_count: dtype"), (dict(new_count=cnt[:2]), "new_count: shape"),
                     (dict(next_pos=pos[:1]), "next_pos: shape"), (dict(next_pos=pos.long()), "next_pos: dtype"),
                     (dict(label=256), "label"), (dict(label=-1), "label")):
        with pytest.raises(kvc.KvcError, match=text):
            st.extend(**{**dict(qkv=x(), new_count=cnt, next_pos=pos), **kw})
    with pytest.raises(kvc.KvcError, match="one for each"):
        st.decode(x(2), pos)
    with pytest.raises(kvc.KvcError, match="at most 8"):
        make(Hq=18).decode(x(heads=22), pos)
    late = make()
    late.top_k = 2
    with pytest.raises(kvc.KvcError, match="together"):
        late.decode(x(), pos)
    assert called == []


def test_a_number_that_is_no_stream():
    for bad in (-1, 1 << 64, 1 << 70):
        with pytest.raises(kvc.KvcError, match="no stream"):
            make()._stream(bad)
    assert make()._stream(None) is None
