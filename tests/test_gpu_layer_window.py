"""Attention with a sliding window over a cache whose old pages are gone: the
block table holds -1 for every page that lies before all windows, and the pool's
first page, which a clamped -1 would read, holds NaN."""
import math

import pytest

import layer_util as U
from test_gpu_layer import _cache, _cuda, _layer, _near, _rand, _starts  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("heads, kv_heads, d, page, block, window, new, kv", [
    (2, 2, 64, 16, 1, 40, [40], [300]),               # tiles: keys from 221, the chunk begins at 128
    (2, 2, 64, 16, 1, 40, [3], [300]),                # the kernel for few rows
    (2, 2, 128, 16, 1, 30, [40, 1, 20], [300, 500, 255]),
    (5, 1, 128, 32, 8, 70, [60, 33], [400, 1000]),
    (4, 2, 64, 64, 0, 50, [20, 20], [700, 310]),      # no causal limit
    (3, 3, 64, 16, 1, 1, [130], [700]),               # every token sees itself alone
    (2, 2, 128, 128, 1, 100, [300], [2000]),          # pages as high as a chunk
    (1, 1, 64, 1024, 1, 600, [20], [5000]),           # and higher
    (1, 1, 128, 16, 1, 3000, [20], [9000]),           # cut along the keys
    (40, 40, 64, 16, 1, 2100, [200, 180], [3000, 2500]),  # more units than SMs
])
def test_released_pages(heads, kv_heads, d, page, block, window, new, kv):
    lay = _layer(heads=heads, kv_heads=kv_heads, d=d, page_size=page, causal_block=block, window=window)
    kp, vp, bt = _cache(lay, kv)
    kp, vp = (torch.cat([torch.full_like(p[:1], math.nan), p]) for p in (kp, vp))
    bt = torch.where(bt < 10 ** 9, bt + 1, bt)
    whole = bt.clone()
    gone = 0
    for s, (m, n) in enumerate(zip(new, kv)):
        first = max(0, n - m - window + 1) // page  # the page of the first new token's lowest key
        bt[s, :first] = -1
        gone += first
    assert gone
    q = _rand(sum(new), heads, d, seed=7)
    lens = torch.tensor(kv, dtype=torch.int32).cuda()
    got, lse = lay.ac_cache_attn(q, kp, vp, bt, _starts(new), lens, max_q=max(new), max_kv=max(kv), lse=True)
    assert lay.get_status() == 0
    kd, vd = (p.double().cpu() for p in (kp, vp))
    ref, rl, absv, big, _ = U.attend(lay.cfg, q.double().cpu(), kd, vd, whole.cpu(), _starts(new).cpu(), kv)
    _near(got, ref, U.attend_tol(ref, absv, big), "out")
    # the bound of the log-sum-exp as for whole tables: the sum's 1.1e-4 by weight, the
    # score's error, log2's and the product's roundings
    assert ((lse.double().cpu() - rl).abs() <= 1.2e-4 + 136 * U.EPS32 * big + 8 * U.EPS32 * rl.abs()).all()
    # bit for bit what the whole table gives, on pages that were never there
    kp[0], vp[0] = 0, 0
    again = lay.ac_cache_attn(q, kp, vp, whole, _starts(new), lens, max_q=max(new), max_kv=max(kv))
    assert torch.equal(got, again)
