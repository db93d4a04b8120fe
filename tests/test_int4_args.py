"""The decodes refuse int4 pools that hold fewer records than the params say, before anything else."""
import numpy as np
import pytest
import torch


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", ["decode", "decode_noalloc", "decode_shared", "decode_shared_partials"])
def test_short_int4_pools_are_refused(which, d):
    from paged_kv_cache_57_gb300 import lazy_attn as L
    p = L.make_params(num_seqs=1, num_q_heads=4, num_kv_heads=2, head_dim=d, num_pool_blocks=10, max_blocks_per_seq=4, kv_dtype="int4")
    q, words, i32 = torch.zeros(1, 4, d, dtype=torch.bfloat16), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    rope, ws = torch.zeros(L.rope_table_bytes(p), dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8)
    plan = L.SharedPlan(np.zeros((1, L.PLAN_ITEM_INTS), np.int32), np.array([0, 1], np.int32), device="cpu")
    args = {"decode": (words, i32, i32, rope), "decode_noalloc": (words, i32, i32, rope, torch.empty_like(q)),
            "decode_shared": (words, i32, rope, plan), "decode_shared_partials": (words, i32, rope, plan, ws)}[which]
    whole = L.empty_pools(p, device="cpu")
    for k, v in ((whole[0].flatten()[:-1], whole[1]), (whole[0], whole[1][:9]), (torch.zeros(0, dtype=torch.uint8),) * 2):
        with pytest.raises(ValueError, match="num_pool_blocks"):
            getattr(L, which)(p, q, k, v, *args)
    with pytest.raises(ValueError, match="k_pool must be a CUDA tensor"):  # whole ones go on to the next check
        getattr(L, which)(p, q, *whole, *args)
