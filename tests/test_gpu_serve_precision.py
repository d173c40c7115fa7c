"""The precision the attention states: probabilities with all of fp32's bits, and sums over long runs that do not drift."""
import numpy as np
import pytest
import torch

from agent_kv_cache_lse_b200 import kvc
from tests.serve_cases import DT, cache_of, np64
from tests.serve_precision import CHUNK, JOINS, RUN, TWO_SLOTS, drift
from tests.test_gpu_serve import attend, code

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = torch.int32


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 12])
def test_probabilities_keep_fp32s_bits(dtype, D, P):
    S, H, G = 64, 2, 8
    c, _ = cache_of([2] * S * H, P, D, dtype, S, 1, H, seed=1, device=DEV, late=False)
    g = torch.Generator().manual_seed(D)
    x = (0.5 + 3.5 * torch.rand((S * H,), generator=g)).to(DT[dtype])
    y = (-4 * torch.rand((S, 1, H * G), generator=g)).to(DT[dtype])
    pages = c.block_table[:, 0].long()
    c.k_pool.zero_()
    c.v_pool.zero_()
    c.k_pool[pages, 1, 0] = x.to(DEV)
    c.v_pool[pages, 1] = 1
    q = torch.zeros((S, 1, H * G, D), dtype=DT[dtype])
    q[..., 0] = y
    out, lse, st = attend(c, q.to(DEV), torch.full((S,), 9, dtype=I32, device=DEV))
    assert code(st) == 0
    logit = np64(y).reshape(S * H, G) * np64(x)[:, None] / np.sqrt(D)
    assert -4 < logit.min() / np.log(2) and logit.max() <= 0
    want = 1 / (1 + np.exp(-logit)).reshape(S, 1, H * G)
    assert (np.abs(np64(out) / want[..., None] - 1) <= TWO_SLOTS).all()
    assert (np.abs(np64(lse) - np.log1p(np.exp(logit)).reshape(S, 1, H * G)) <= TWO_SLOTS).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 12])
def test_sums_over_long_runs_do_not_drift(D, P):
    """One row of about 9.5 million slots (its pages repeat), so that each warp adds RUN chunks."""
    warps = torch.cuda.get_device_properties(0).multi_processor_count * 8
    assert warps <= 8 * 160  # the joins' bound
    n = RUN * warps * 16 // 48 * 48
    unit = 48 // P if P == 12 else 1
    values = torch.from_numpy(np.tile(CHUNK, 3)[: unit * P]).to(torch.bfloat16).to(DEV)
    pool = values.view(unit, P, 1).repeat(1, 1, D).contiguous()
    mp = n // P
    c = kvc.Cache(torch.ones_like(pool), pool, (torch.arange(mp, dtype=I32, device=DEV) % unit).view(1, mp),
                  torch.tensor([n], dtype=I32, device=DEV), torch.zeros((1, n), dtype=I32, device=DEV), None, 1, 1, 1)
    q = torch.zeros((1, 1, 2, D), dtype=torch.bfloat16, device=DEV)
    out, lse, st = attend(c, q, torch.zeros(1, dtype=I32, device=DEV))
    assert code(st) == 0
    tol = max(abs(drift(r)) for r in (RUN - 1, RUN, RUN + 1)) + JOINS
    assert (np.abs(np64(out) / CHUNK.mean() - 1) <= tol).all()
    assert np.abs(np64(lse) - np.log(n)).max() <= 4 * 2.0**-24 * np.log(n)
