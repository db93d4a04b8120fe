"""GPU: the decodes over int4 pools where a softmax's or a sum's range ends: scores far below
0, NaN, long sums, blocks that are left out, weights and scales far apart. Against 64-bit
attention over the same codes, with the error bound of tests/int4_model.py unless a test
derives its own."""
import numpy as np
import pytest
import torch

import int4_model as M
from gpu_util import la, shared_plan
from paged_kv_cache_57_gb300 import workloads as W
from test_gpu_int4 import check, decode, on_device

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    la().device_status(clear=True)
    yield
    assert la().device_status(clear=True) == 0, "device status word set"


def opposed(w, c=8.0):
    """The workload with every key's slowest dims (the last quarter of each half) near c and every query's near -c: all
    scores lie near -d c^2 / 4 / sqrt(d), far below 2^-126 of a weight of 1. V lies near 1, so that an output of 0 is
    outside every bound."""
    d = w.head_dim
    slow = torch.zeros(d)
    slow[3 * d // 8:d // 2] = slow[7 * d // 8:] = c
    w.k_pool = (w.k_pool.float() + slow).to(torch.bfloat16)
    w.q = (w.q.float() - slow).to(torch.bfloat16)
    w.v_pool = (1 + w.v_pool.float() / 8).to(torch.bfloat16)
    return w


# parts without keys: a ragged batch cut for its longest sequence, and more splits than most sequences have blocks
@pytest.mark.parametrize("hq,hkv,d,c", [(8, 2, 128, 8.0), (16, 2, 64, 10.0), (32, 1, 128, 10.0)])
def test_low_scores_beside_parts_without_keys(hq, hkv, d, c):
    dw, _ = W.mixed_mqa(n_decode=9, n_prefill=1, chunk=16, hq=hq, hkv=hkv, d=d, pool_docs=60, ctx_lo=1, ctx_hi=5000,
                        doc_lo=1, doc_hi=300, seed=810)
    dv, k4, v4, kv, vv = on_device(opposed(dw, c))
    ref = M.attention(dw, kv, vv)
    for splits in (0, 1, 7, 300):
        dv.p.num_splits = splits
        check(decode(dv, k4, v4), ref, f"ragged, splits {splits}")
    for chunk in (0, 4):
        check(la().decode_shared(dv.p, dv.q, k4, v4, dv.words, dv.q_pos, dv.rope, shared_plan(dv, chunk)), ref, f"shared, chunk {chunk}")


# a query with a NaN, and a sequence whose keys are all NaN for one KV head: their rows are NaN, on both decodes, the others
# as without them
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (2, 2, 64), (48, 2, 128)])
def test_rows_without_a_finite_score_are_nan(hq, hkv, d):
    w = W.decode_zipf("i4n", batch=3, hq=hq, hkv=hkv, d=d, docs_per_seq=2, doc_tokens=90, pool_docs=3, zipf_s=0.5, share=False,
                      suffix_tokens=7, seed=820)
    G = hq // hkv
    for doc, _ in w.seq_segments(2):  # KV head 0 of sequence 2
        w.k_pool[w.doc_blocks[int(w.doc_block_indptr[doc]):int(w.doc_block_indptr[doc + 1])].astype(np.int64), 0] = float("nan")
    w.q[1, hq - 1, 5] = float("nan")
    dv, k4, v4, kv, vv = on_device(w)
    want, bound = M.attention(w, kv, vv)
    nan = torch.zeros(3, hq, dtype=torch.bool, device="cuda")
    nan[1, hq - 1] = nan[2, :G] = True
    outs = {}
    for splits in (0, 1, 3):
        dv.p.num_splits = splits
        outs[f"splits {splits}"] = decode(dv, k4, v4)
    for chunk in (0, 2):
        outs[f"chunk {chunk}"] = la().decode_shared(dv.p, dv.q, k4, v4, dv.words, dv.q_pos, dv.rope, shared_plan(dv, chunk))
    for what, out in outs.items():
        assert torch.isnan(out[nan]).all(), what
        check(out[~nan], (want[~nan], bound[~nan]), what)
