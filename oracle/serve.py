"""One model step over the paged cache, in numpy: slots for new tokens, head norms with rotation, page bounds, the
choice of pages and one-token attention over them.  64-bit floating point and plain loops over rows; shares no
code with the CUDA side.  Rows are numbered (seq * num_layers + layer) * num_kv_heads + head.
"""
import numpy as np


def reserve_slots(bt, row_len, slot_pos, slot_label, crf, new_count, next_pos, label, free_pages, depth, max_tokens,
                  layers, heads, P, num_pages):
    """Returns a dict of every array after the call (copies) and the refused rows {row: code}."""
    bt, slot_pos, row_len = bt.copy(), slot_pos.copy(), row_len.copy()
    slot_label = None if slot_label is None else slot_label.copy()
    crf = None if crf is None else crf.copy()
    S, per, max_slots = len(new_count), layers * heads, bt.shape[1] * P
    counts = [max(0, int(c)) for c in new_count]
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    slot_map = np.full((max_tokens, layers, heads), -1, dtype=np.int64)
    token_pos = np.full(max_tokens, -1, dtype=np.int32)
    refused = {}
    out = dict(bt=bt, row_len=row_len, slot_pos=slot_pos, slot_label=slot_label, crf=crf, slot_map=slot_map,
               token_pos=token_pos, depth=depth, refused=refused, token_start=np.minimum(start, max_tokens))
    takes = {}
    for r in range(len(row_len)):
        s, n = r // per, int(row_len[r])
        c = counts[s]
        if c == 0:
            continue
        if n < 0 or n > max_slots or next_pos[s] < 0 or int(next_pos[s]) + c > 2**31 - 1:
            refused[r] = "length"
        elif n + c > max_slots:
            refused[r] = "full"
        elif n % P and not 0 <= bt[r, n // P] < num_pages:
            refused[r] = "page"
        else:
            takes[r] = -(-(n + c) // P) - -(-n // P)
    total = sum(takes.values())
    if start[-1] > max_tokens or not 0 <= depth <= len(free_pages) or total > depth:
        refused[-1] = "call"
        return out
    for s in range(S):
        for i in range(counts[s]):
            if next_pos[s] >= 0 and int(next_pos[s]) + counts[s] <= 2**31 - 1:
                token_pos[start[s] + i] = next_pos[s] + i
    top = depth - total
    out["depth"] = top
    for r, need in takes.items():
        s, n = r // per, int(row_len[r])
        for k in range(need):
            bt[r, -(-n // P) + k] = free_pages[top + k]
        top += need
        for i in range(counts[s]):
            slot = n + i
            page = int(bt[r, slot // P])
            if 0 <= page < num_pages:
                slot_map[start[s] + i, r % per // heads, r % heads] = page * P + slot % P
            slot_pos[r, slot] = next_pos[s] + i
            if slot_label is not None:
                slot_label[r, slot] = label
            if crf is not None:
                crf[r, slot] = 0
        row_len[r] = n + counts[s]
    return out


def norm_rope(x, weight, eps, pos, inv_freq, interleaved):
    """x [T, L, H, D], weight [L, D] or None -> (y, reach): reach is the sum of the magnitudes that each output
    element is made of, which is what its rounding errors are relative to."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)[None, :, None, :]
    y, reach = x.copy(), np.abs(x)
    for j, f in enumerate(np.asarray(inv_freq, dtype=np.float64)):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + len(inv_freq))
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos.astype(np.float64) * f)[:, None, None]
        y[..., a], y[..., b] = z.real, z.imag
        reach[..., a] = reach[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, reach


def block_bounds(keys, pos, P):
    """keys [n, D] in slot order, pos [n] -> list over pages of (lo [D], hi [D], lowest position)."""
    return [(keys[a:a + P].min(0), keys[a:a + P].max(0), int(pos[a:a + P].min())) for a in range(0, len(keys), P)]


def select_blocks(bounds, q, q_pos, top_k, sink, recent):
    """bounds as block_bounds gives them, q [G, D] -> ascending page indexes."""
    q = q.astype(np.float64)
    rated = []
    for b, (lo, hi, first) in enumerate(bounds):
        if first > q_pos:
            continue
        with np.errstate(invalid="ignore"):
            score = np.maximum(q * lo.astype(np.float64), q * hi.astype(np.float64)).sum()
        if np.isnan(score) or not (np.isfinite(lo).all() and np.isfinite(hi).all()):
            score = np.inf  # keys that are not finite are not passed over
        always = b < sink or b >= len(bounds) - recent
        rated.append((not always, 0.0 if always else -score, b))
    return sorted(b for _, _, b in sorted(rated)[:top_k])


def attention(q, keys, values, pos, q_pos, slots=None):
    """q [G, D] over the given slots of a row (all when None) -> (out [G, D], lse [G], reach [G, D], largest sum of
    |q_d k_d| / sqrt(D) over the visible keys).  reach = sum_i p_i |v_i|."""
    G, D = q.shape
    slots = np.arange(len(keys)) if slots is None else np.asarray(slots, dtype=np.int64)
    seen = slots[pos[slots] <= q_pos] if len(slots) else slots
    if len(seen) == 0:
        return np.zeros((G, D)), np.full(G, -np.inf), np.zeros((G, D)), 0.0
    k, v, q = keys[seen].astype(np.float64), values[seen].astype(np.float64), q.astype(np.float64)
    logit = q @ k.T / np.sqrt(D)
    top = logit.max(1, keepdims=True)
    p = np.exp(logit - top)
    total = p.sum(1, keepdims=True)
    p /= total
    return p @ v, (top + np.log(total))[:, 0], p @ np.abs(v), float((np.abs(q) @ np.abs(k).T).max() / np.sqrt(D))
