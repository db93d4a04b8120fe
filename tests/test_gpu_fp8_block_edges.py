"""GPU: pools of e4m3 codes with block scales where their records, scales and sums are unusual."""
import numpy as np
import pytest
import torch

import fp8_block_model as M
from gpu_util import la
from paged_kv_cache_57_gb300 import workloads as W
from test_gpu_fp8_block import check, decode, documents, filled_pools, on_device, params, rows, same_records, scatter

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


# Long sums. The products truncate: 16384 blocks of a warp, a quarter of a sequence, would lose 2^-12 or so of what they add
# up. Here a warp's values rise to a sum of thousands of blocks and fall back to 0: scores are 0, weights a power of two, and products
# and the 64-bit sum exact, so that what is left over is what the sums lost. Within 512 blocks each addition is off by at most a unit of
# the last place, 2^-23 of the run's sum: 2^-14 of the mean size in all; the additions of the 32 runs' sums round, 2^-24 each.
@pytest.mark.parametrize("hq,d", [(4, 64), (8, 64), (16, 128), (32, 64), (32, 128)])
def test_long_sums_are_not_truncated(hq, d):
    L = la()
    nb, run = 65536, 16384
    rng = np.random.default_rng(hq + d)
    p = L.make_params(num_seqs=1, num_q_heads=hq, num_kv_heads=1, head_dim=d, num_pool_blocks=128, max_blocks_per_seq=nb, kv_dtype="fp8_e4m3_block",
                      num_splits=1, id_bits=8)
    assert L.decode_workspace_bytes(p) == 0  # one part
    kp, vp = L.empty_pools(p)
    x = np.abs(rng.standard_normal((64, 16, 1, d))) * 2.0 ** rng.integers(-6, 1, (64, 1, 1, 1))
    x = torch.from_numpy(np.concatenate((x, -x)).reshape(2048, 1, d)).to(torch.bfloat16).cuda()
    L.cache_write(p, torch.zeros_like(x), x, torch.arange(2048, dtype=torch.int32, device="cuda"), kp, vp)
    order = rng.integers(0, 64, run // 2)
    ids = np.tile(np.concatenate((order, 64 + rng.permutation(order))), nb // run)
    words = torch.from_numpy((16 * np.arange(nb) << 8 | ids).astype(np.int32)[None]).cuda()
    size = np.abs(M.values(vp.cpu().numpy(), d, True))[ids[:run]].mean((0, 1, 2))
    q = torch.zeros(1, hq, d, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([16 * nb], dtype=torch.int32, device="cuda")
    out = L.decode(p, q, kp, vp, words, lens, lens, L.rope_table_init(p))
    worst = (out.double()[0].abs().cpu().numpy() / size).max()
    assert worst <= 2.0 ** -14 + 2.0 ** -18, np.log2(worst)


# References that move between and within the runs of sums that were put aside: maxima and V scales that grow and fall
@pytest.mark.parametrize("hq,d", [(3, 128), (8, 64), (16, 64), (32, 64), (32, 128)])
@pytest.mark.parametrize("how", ["growing", "falling", "mixed"])
def test_sums_put_aside_follow_their_references(hq, d, how):
    L = la()
    w = W.decode_zipf("f8aside", batch=1, hq=hq, hkv=1, d=d, docs_per_seq=2, doc_tokens=70000, pool_docs=2, zipf_s=0.5, share=False, seed=1901)
    w.k_pool[:], w.v_pool[:] = torch.nan_to_num(w.k_pool), torch.nan_to_num(w.v_pool)
    nb = w.num_pool_blocks
    at = torch.empty(nb, dtype=torch.float64)
    at[torch.from_numpy(w.doc_blocks.astype(np.int64))] = torch.arange(nb, dtype=torch.float64)
    if how == "falling":
        at = nb - 1 - at
    elif how == "mixed":
        at = torch.randperm(nb, generator=torch.Generator().manual_seed(9)).double()
    at = at.view(-1, 1, 1, 1)
    w.k_pool = (w.k_pool.double() * (0.25 + 1.5 * at / nb)).to(torch.bfloat16)
    w.v_pool = ((1 + w.v_pool.double() / 4) * 2.0 ** (at // 700)).to(torch.bfloat16)
    dv, kp, vp, kv, vv = on_device(w, num_splits=1, id_bits=14)
    check(decode(dv, kp, vp), M.attention(w, kv, vv), how)
    w.q[0, hq - 1, 3] = float("nan")  # a row without a finite score stays one
    dv.q.copy_(w.q)
    assert torch.isnan(decode(dv, kp, vp)[0, hq - 1]).all()
