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


# Weights times V scales are rounded once: a block of weight 1 whose scale is 2^-25 of the part's largest (the least step of
# f16 is 2^-24) keeps its values. All scores are 0, so that every weight is 1; the header's bound on a product that is rounded to
# f16 is 2^-11 of it, or 2^-29 of the largest scale. Codes are whole powers of two: with weights and scales they are exact, and so are
# the sums. A warp's part has the blocks of both scales (one warp: one split of at most 4 blocks a warp).
@pytest.mark.parametrize("hq", [4, 8, 16, 32])
@pytest.mark.parametrize("down", [14, 20, 24, 25, 27])
@pytest.mark.parametrize("shared", [False, True])
def test_small_v_scales_beside_large_ones(hq, down, shared):
    L = la()
    d, nb = 128, 8
    p = L.make_params(num_seqs=1, num_q_heads=hq, num_kv_heads=1, head_dim=d, num_pool_blocks=nb, max_blocks_per_seq=nb, kv_dtype="fp8_e4m3_block",
                      num_splits=1)
    kp, vp = L.empty_pools(p)
    k = torch.zeros(16 * nb, 1, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    big = torch.arange(16 * nb, device="cuda") // 16 % 2 == 0
    v[big, 0, 0] = 256.0                   # scale 1, in the first dim
    v[~big, 0, 1:] = 256.0 * 2.0 ** -down  # scale 2^-down, in the others
    L.cache_write(p, k, v, torch.arange(16 * nb, dtype=torch.int32, device="cuda"), kp, vp)
    q = torch.zeros(1, hq, d, dtype=torch.bfloat16, device="cuda")
    words = torch.arange(nb, dtype=torch.int32, device="cuda")[None].contiguous()
    lens = torch.tensor([16 * nb], dtype=torch.int32, device="cuda")
    rope = L.rope_table_init(p)
    if shared:
        one = np.array([0, 1], np.int32)
        items, slots = L.plan_shared_host(p, 1, one, [0], [16 * nb], [0, nb], np.arange(nb, dtype=np.int32), chunk_blocks=nb)
        out = L.decode_shared(p, q, kp, vp, words, lens, rope, L.SharedPlan(items, slots))
    else:
        out = L.decode(p, q, kp, vp, words, lens, lens, rope)
    out = out.double()[0]
    assert (out[:, 0] == 128).all()
    want = 128 * 2.0 ** -down
    # half of the keys have a weight of 1 and a product that is off by 2^-29 at most (f16's least step: 2^-25 with weights of 2^4), times 256
    assert ((out[:, 1:] - want).abs() <= 128 * 2.0 ** -29 + 2.0 ** -8 * want).all(), out[0, 1].item() / want
