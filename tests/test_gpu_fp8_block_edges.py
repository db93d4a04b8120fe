"""GPU: pools of e4m3 codes with block scales where their records, scales and sums are unusual."""
import numpy as np
import pytest
import torch

import fp8_block_model as M
from gpu_util import la
from test_gpu_fp8_block import documents, filled_pools, params, rows, same_records, scatter

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    la().device_status(clear=True)
    yield
    assert la().device_status(clear=True) == 0, "device status word set"


# scales that no call wrote, as uninitialised pools hold them: a block that its first call writes behind row 0 begins anew.
# One token a warp, and windows of a block's length
@pytest.mark.parametrize("hkv,d,docs", [(3, 128, 24), (2, 64, 24), (8, 64, 400)])
def test_writes_behind_row_0_of_blocks_that_nothing_wrote(hkv, d, docs):
    L = la()
    rng = np.random.default_rng(d + docs)
    p = params(hkv, d, 2 * docs)
    (kp, vp), (k0, v0) = filled_pools(p, 11)
    odd = np.array([3.14, -0.5, np.nan, np.inf, 2.0 ** -120, 2.0 ** 125, 0.0, 1e-40, 1.5, -np.inf], "<f4")
    n = 16 * d
    for x, y in ((kp, k0), (vp, v0)):
        pick = rng.integers(0, 2 * len(odd), y.shape[:2])  # half of the records keep a proper scale
        bad = pick < len(odd)
        y[..., n:n + 4][bad] = odd[pick[bad]][:, None].view(np.uint8)
        x.copy_(torch.from_numpy(y))
        begun = y.copy()
        begun[bad] = 0
        begun[..., n:n + 4][bad] = np.frombuffer(np.float32(2.0 ** -100).tobytes(), np.uint8)
        y[...] = begun  # what the model continues
    lens, first = rng.integers(1, 9, docs), rng.integers(1, 8, docs)
    slots = documents(rng, 2 * docs, lens, first)
    if docs > 100:
        assert len(slots) * 2 * hkv > 152 * 128
    untouched = np.setdiff1d(np.arange(2 * docs), slots // 16)
    k, v = rows("normal", len(slots), hkv, d, rng), rows("outliers", len(slots), hkv, d, rng)
    before = [x.cpu().numpy() for x in (kp, vp)]
    L.cache_write(p, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), kp, vp)
    for x, y, src, old, is_v in ((kp, k0, k, before[0], False), (vp, v0, v, before[1], True)):
        scatter(slots, y, src, is_v)
        y[untouched] = old[untouched]
        same_records(x, y, d)
