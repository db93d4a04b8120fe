"""GPU: the decodes over int4 pools, against 64-bit attention over the same codes, with
the error bound of tests/int4_model.py; and the way the calls are used together."""
import numpy as np
import pytest
import torch

import int4_model as M
from gpu_util import la, shared_plan, to_device
from paged_kv_cache_57_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    la().device_status(clear=True)
    yield
    assert la().device_status(clear=True) == 0, "device status word set"


def on_device(w, **kw):
    """(Dev with int4 params, k_pool, v_pool on the GPU, their values in fp64)."""
    L = la()
    dv = to_device(w, **kw)
    dv.p.kv_dtype = L.LAZY_INT4
    k4, v4 = M.int4_pools(w)
    kv = torch.from_numpy(np.nan_to_num(M.int4_values(k4.numpy(), w.head_dim, False)))
    vv = torch.from_numpy(np.nan_to_num(M.int4_values(v4.numpy(), w.head_dim, True)))
    return dv, k4.cuda(), v4.cuda(), kv.cuda(), vv.cuda()


def check(out, ref, what):
    want, bound = ref
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all(), what
    worst = (err / bound).max().item() if bound.numel() else 0.0
    assert worst <= 1.0, f"{what}: off by {worst:.2f} of the bound at {np.unravel_index((err / bound).argmax().item(), err.shape)}"


def decode(dv, k4, v4, **kw):
    return la().decode(dv.p, dv.q, k4, v4, dv.words, dv.seq_lens, dv.q_pos, dv.rope, **kw)


# 1, 2, 4, 7, 8, 9, 16, 32 and 64 query heads per KV head (tiles of 8 and 16 rows, several
# tiles), both head sizes; documents whose last block is partial, slots behind them NaN
@pytest.mark.parametrize("hq,hkv,d,splits", [(8, 8, 128, 0), (4, 2, 64, 1), (32, 8, 128, 3), (28, 4, 128, 0), (64, 8, 128, 2),
                                             (18, 2, 128, 0), (32, 2, 64, 5), (32, 1, 128, 0), (64, 1, 128, 2), (64, 1, 64, 0)])
def test_decode_matches_64_bits(hq, hkv, d, splits):
    w = W.decode_zipf(f"i4{hq}", batch=6, hq=hq, hkv=hkv, d=d, docs_per_seq=4, doc_tokens=150, pool_docs=5, zipf_s=1.0,
                      suffix_tokens=21, seed=620 + hq + splits)
    dv, k4, v4, kv, vv = on_device(w, num_splits=splits)
    check(decode(dv, k4, v4), M.attention(w, kv, vv), f"int4 decode {hq}/{hkv} d{d} splits {splits}")


# contexts of 1, 2, 15 .. 33 tokens, documents of one token, one block and parts of one
@pytest.mark.parametrize("doc,docs", [(1, 1), (1, 2), (1, 33), (15, 1), (16, 1), (17, 1), (16, 2), (3, 11), (32, 1), (33, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_short_contexts(doc, docs, d):
    w = W.decode_zipf("i4s", batch=3, hq=8, hkv=2, d=d, docs_per_seq=docs, doc_tokens=doc, pool_docs=3, zipf_s=0.5,
                      share=False, seed=700 + doc + docs)
    dv, k4, v4, kv, vv = on_device(w)
    check(decode(dv, k4, v4), M.attention(w, kv, vv), f"int4 decode, {docs} documents of {doc}")


def test_decode_ragged_batch_with_empty_sequences():
    dw, _ = W.mixed_mqa(n_decode=9, n_prefill=1, chunk=16, hq=8, hkv=2, d=128, pool_docs=60, ctx_lo=1, ctx_hi=5000,
                        doc_lo=1, doc_hi=300, seed=710)
    dv, k4, v4, kv, vv = on_device(dw)
    want, bound = M.attention(dw, kv, vv)
    for splits in (0, 1, 7):
        dv.p.num_splits = splits
        check(decode(dv, k4, v4), (want, bound), f"ragged, splits {splits}")
        lens = dv.seq_lens.clone()
        lens[[2, 8]] = 0
        out = la().decode(dv.p, dv.q, k4, v4, dv.words, lens, dv.q_pos, dv.rope)
        assert torch.count_nonzero(out[[2, 8]]) == 0
        keep = [0, 1, 3, 4, 5, 6, 7]
        check(out[keep], (want[keep], bound[keep]), "beside empty sequences")


# (sequences, query heads) on both sides of 456 pairs, where a join's CTA takes eight pairs; batches of more than 32
# sequences (several scans of the lengths), runs of empty ones before, between and behind the others, parts of one
# sequence in more than eight ranges, and a workspace that held NaN
@pytest.mark.parametrize("batch,hq", [(33, 8), (57, 8), (58, 8), (90, 14)])
def test_decode_many_sequences(batch, hq):
    L = la()
    dw, _ = W.mixed_mqa(n_decode=batch, n_prefill=1, chunk=16, hq=hq, hkv=2, d=64, pool_docs=60, ctx_lo=1, ctx_hi=6000,
                        doc_lo=1, doc_hi=300, seed=712 + batch)
    dv, k4, v4, kv, vv = on_device(dw)
    want, bound = M.attention(dw, kv, vv)
    ws = torch.full((L.decode_workspace_bytes(dv.p),), 255, dtype=torch.uint8, device="cuda")
    first = decode(dv, k4, v4, workspace=ws)
    check(first, (want, bound), "all")
    assert torch.equal(decode(dv, k4, v4, workspace=ws), first)
    for keep in ([batch - 1], [0], [3, batch // 2], list(range(32, batch)), []):
        lens = torch.zeros_like(dv.seq_lens)
        lens[keep] = dv.seq_lens[keep]
        ws.fill_(255)
        out = L.decode(dv.p, dv.q, k4, v4, dv.words, lens, dv.q_pos, dv.rope, workspace=ws)
        check(out[keep], (want[keep], bound[keep]), f"only {keep[:3]}")
        assert torch.count_nonzero(out).item() == torch.count_nonzero(out[keep]).item()


# more units than a device has resident CTAs and sequences of more than 512 blocks among short ones: ranges of the units'
# blocks laid end to end, several units or parts of one in a CTA's range
@pytest.mark.parametrize("batch,hq,hkv,d", [(330, 8, 2, 64), (330, 12, 2, 128), (160, 32, 1, 128)])
def test_decode_ranges_of_ragged_batches(batch, hq, hkv, d):
    L = la()
    dw, _ = W.mixed_mqa(n_decode=batch, n_prefill=1, chunk=16, hq=hq, hkv=hkv, d=d, pool_docs=60, ctx_lo=1, ctx_hi=9500,
                        doc_lo=1, doc_hi=700, seed=713 + hq)
    dv, k4, v4, kv, vv = on_device(dw)
    assert dw.max_blocks_per_seq > 512 and 0 < L.decode_workspace_bytes(dv.p)
    want, bound = M.attention(dw, kv, vv)
    ws = torch.full((L.decode_workspace_bytes(dv.p),), 255, dtype=torch.uint8, device="cuda")
    first = decode(dv, k4, v4, workspace=ws)
    check(first, (want, bound), "all")
    assert torch.equal(decode(dv, k4, v4, workspace=ws), first)
    long = int(dv.seq_lens.argmax())
    for keep in ([batch - 1], [0], [long], [3, batch // 2, long], list(range(40, batch)), []):
        lens = torch.zeros_like(dv.seq_lens)
        lens[keep] = dv.seq_lens[keep]
        ws.fill_(255)
        out = L.decode(dv.p, dv.q, k4, v4, dv.words, lens, dv.q_pos, dv.rope, workspace=ws)
        check(out[keep], (want[keep], bound[keep]), f"only {keep[:3]}")
        assert torch.count_nonzero(out).item() == torch.count_nonzero(out[keep]).item()


def test_two_decodes_at_once():
    # each call with its own workspace, on its own stream, several in flight
    L = la()
    dw, _ = W.mixed_mqa(n_decode=20, n_prefill=1, chunk=16, hq=16, hkv=2, d=128, pool_docs=40, ctx_lo=1, ctx_hi=4000,
                        doc_lo=1, doc_hi=300, seed=716)
    dv, k4, v4, kv, vv = on_device(dw)
    alone = decode(dv, k4, v4)
    check(alone, M.attention(dw, kv, vv), "alone")
    n = L.decode_workspace_bytes(dv.p)
    runs = [(torch.cuda.Stream(), torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(dv.q)) for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, ws, out in runs:
            decode(dv, k4, v4, out=out, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for _, _, out in runs:
        assert torch.equal(out, alone)


def test_decode_more_splits_than_blocks_and_small_workspace():
    L = la()
    w = W.decode_zipf("i4sp", batch=2, hq=8, hkv=2, d=128, docs_per_seq=2, doc_tokens=60, pool_docs=4, zipf_s=0.5, seed=717)
    dv, k4, v4, kv, vv = on_device(w, num_splits=1000)
    check(decode(dv, k4, v4), M.attention(w, kv, vv), "1000 splits")
    need = L.decode_workspace_bytes(dv.p)
    with pytest.raises(L.LazyAttnError, match="WORKSPACE"):
        decode(dv, k4, v4, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(L.LazyAttnError, match="WORKSPACE"):
        decode(dv, k4, v4, workspace=torch.empty(need + 16, dtype=torch.uint8, device="cuda")[8:])


def test_decode_far_positions_and_control():
    w = W.decode_zipf("i4far", batch=2, hq=16, hkv=4, d=128, docs_per_seq=3, doc_tokens=70, pool_docs=4, zipf_s=1.0,
                      suffix_tokens=9, seed=720, shift=100000)
    dv, k4, v4, kv, vv = on_device(w, id_bits=8)
    check(decode(dv, k4, v4), M.attention(w, kv, vv), "far positions")
    # lazy = 0: the pool holds absolute-position keys; with zero rates every rotation is the identity
    L = la()
    w = W.decode_zipf("i4ctl", batch=5, hq=32, hkv=8, d=128, docs_per_seq=3, doc_tokens=90, pool_docs=4, zipf_s=1.0,
                      suffix_tokens=11, share=False, seed=721)
    dv, k4, v4, kv, vv = on_device(w, lazy=False)
    zero = np.zeros(64)
    rope = L.rope_table_init(dv.p, freqs=zero)
    ref = M.attention(w, kv, vv, freqs=zero)
    check(L.decode(dv.p, dv.q, k4, v4, dv.words, dv.seq_lens, dv.q_pos, rope), ref, "lazy=0")
    check(L.decode_shared(dv.p, dv.q, k4, v4, dv.words, dv.q_pos, rope, shared_plan(dv)), ref, "shared, lazy=0")


def test_decode_long_context():
    # one sequence of 40000 tokens: many splits of one row of heads
    w = W.decode_zipf("i4long", batch=1, hq=4, hkv=1, d=128, docs_per_seq=40, doc_tokens=1000, pool_docs=44, zipf_s=0.1,
                      seed=722)
    dv, k4, v4, kv, vv = on_device(w)
    check(decode(dv, k4, v4), M.attention(w, kv, vv), "40000 tokens")


@pytest.mark.parametrize("hq", [1, 8, 16])
def test_long_sums_stay_exact(hq):
    # 131072 keys of nearly equal weight in one part, 2048 blocks a warp: outputs of about 1/200 of a value, from sums of
    # codes that cancel against the zeros'. In the 2-norm the output's rounding to bf16 is at most 2^-8 (a half step of a
    # power of two's least value) and the rounding of weights and of weight times scale to f16 (2^-11 each, independent)
    # at most 2^-10 of s c, 1.7 standard deviations of a value for normal values: 2^-8 + 1.7 * 2^-10 < 2^-7.
    # Truncated sums would be off by 2048 * 2^-25 of 1.35 ranges' middle, 2 % of the output.
    w = W.decode_zipf("i4sum", batch=1, hq=hq, hkv=1, d=128, docs_per_seq=32, doc_tokens=4096, pool_docs=1, zipf_s=1.0,
                      share=False, seed=723)
    dv, k4, v4, kv, vv = on_device(w, num_splits=1)
    want, _ = M.attention(w, kv, vv)
    out = decode(dv, k4, v4).double()
    assert ((out - want).norm() / want.norm()).item() < 2.0 ** -7


def _rescaled(w, k_mul, v_mul):
    """The workload with each token's stored rows multiplied (per block and slot)."""
    w.k_pool = (w.k_pool.double() * k_mul).to(torch.bfloat16)
    w.v_pool = (w.v_pool.double() * v_mul).to(torch.bfloat16)
    return w


# scales that differ from token to token by powers of two, and values far from 1
@pytest.mark.parametrize("case", ["v_growing", "v_falling", "v_mixed", "v_tiny", "v_huge", "k_sharp", "k_flat", "v_constant"])
@pytest.mark.parametrize("shared", [False, True])
def test_decode_scales(case, shared):
    w = W.decode_zipf("i4sc", batch=2, hq=8, hkv=2, d=128, docs_per_seq=2, doc_tokens=130, pool_docs=4, zipf_s=0.5,
                      suffix_tokens=5, seed=730)
    nb = w.num_pool_blocks
    rng = np.random.default_rng(731)
    one = torch.ones(nb, 1, 16, 1, dtype=torch.float64)
    inv = np.empty(nb, np.int64)  # position of a block in its document
    for doc in range(len(w.doc_len)):
        a, b = int(w.doc_block_indptr[doc]), int(w.doc_block_indptr[doc + 1])
        inv[w.doc_blocks[a:b]] = np.arange(b - a)
    step = torch.from_numpy(inv).double().view(-1, 1, 1, 1)
    kmul, vmul = one, one
    if case == "v_growing":
        vmul = 2.0 ** (3 * step)
    elif case == "v_falling":
        vmul = 2.0 ** (-3 * step)
    elif case == "v_mixed":
        vmul = torch.from_numpy(2.0 ** rng.integers(-6, 7, (nb, 1, 16, 1)).astype(np.float64))
    elif case == "v_tiny":
        vmul = one * 2.0 ** -60
    elif case == "v_huge":
        vmul = one * 2.0 ** 100
    elif case == "k_sharp":
        kmul = one * 8
    elif case == "k_flat":
        kmul = one * 2.0 ** -20
    elif case == "v_constant":
        w.v_pool[:] = torch.where(torch.isnan(w.v_pool), w.v_pool, torch.full_like(w.v_pool, 1.5))
    w = _rescaled(w, kmul, vmul)
    dv, k4, v4, kv, vv = on_device(w)
    if shared:
        out = la().decode_shared(dv.p, dv.q, k4, v4, dv.words, dv.q_pos, dv.rope, shared_plan(dv))
    else:
        out = decode(dv, k4, v4)
    check(out, M.attention(w, kv, vv), case)


@pytest.mark.parametrize("qscale", [2.0 ** -30, 2.0 ** 4])
def test_decode_query_sizes(qscale):
    w = W.decode_zipf("i4q", batch=2, hq=8, hkv=2, d=64, docs_per_seq=2, doc_tokens=50, pool_docs=3, zipf_s=0.5, seed=740)
    w.q = (w.q.float() * qscale).to(torch.bfloat16)
    dv, k4, v4, kv, vv = on_device(w)
    check(decode(dv, k4, v4), M.attention(w, kv, vv), f"queries x {qscale}")


def test_nan_of_a_visible_key_shows():
    w = W.decode_zipf("i4nan", batch=2, hq=4, hkv=2, d=128, docs_per_seq=2, doc_tokens=50, pool_docs=3, zipf_s=0.5,
                      share=False, seed=741)
    blk = int(w.doc_blocks[int(w.doc_block_indptr[w.seq_segments(1)[0][0]])])
    w.v_pool[blk, 1, 3, 5] = float("nan")  # sequence 1, KV head 1: query heads 2 and 3
    dv, k4, v4, kv, vv = on_device(w)
    for splits in (1, 2):
        dv.p.num_splits = splits
        out = decode(dv, k4, v4).float()
        assert torch.isnan(out[1, 2:, :64]).all()
        assert torch.isfinite(out[0]).all() and torch.isfinite(out[1, :2]).all() and torch.isfinite(out[1, 2:, 64:]).all()


def test_device_errors_are_reported():
    L = la()
    w = W.decode_zipf("i4err", batch=3, hq=8, hkv=2, d=128, docs_per_seq=2, doc_tokens=50, pool_docs=3, zipf_s=0.5, seed=742)
    dv, k4, v4, kv, vv = on_device(w)
    lens = dv.seq_lens.clone()
    lens[1] = 16 * dv.p.max_blocks_per_seq + 1
    L.decode(dv.p, dv.q, k4, v4, dv.words, lens, dv.q_pos, dv.rope)
    assert L.device_status(clear=True) & L.LAZY_DEV_BAD_LEN
    lens[1] = -5
    out = L.decode(dv.p, dv.q, k4, v4, dv.words, lens, dv.q_pos, dv.rope)
    assert L.device_status(clear=True) == L.LAZY_DEV_BAD_LEN and torch.count_nonzero(out[1]) == 0
    words = dv.words.clone()
    words[2, 1] = (words[2, 1] & ~0x3FFFF) | 0x3FFFE
    L.decode(dv.p, dv.q, k4, v4, words, dv.seq_lens, dv.q_pos, dv.rope)
    assert L.device_status(clear=True) == L.LAZY_DEV_BAD_BLOCK_ID
    plan = shared_plan(dv)
    plan.items.view(-1, L.PLAN_ITEM_INTS)[0, 0] = 99
    L.decode_shared(dv.p, dv.q, k4, v4, dv.words, dv.q_pos, dv.rope, plan)
    assert L.device_status(clear=True) == L.LAZY_DEV_LAYOUT


def test_noalloc_gives_the_same_bits():
    L = la()
    w = W.decode_zipf("i4na", batch=16, hq=32, hkv=8, d=128, docs_per_seq=6, doc_tokens=272, pool_docs=40, zipf_s=1.0,
                      suffix_tokens=33, seed=743)
    dv, k4, v4, kv, vv = on_device(w)
    assert 0 < L.decode_workspace_bytes(dv.p) <= L.NOALLOC_SCRATCH_BYTES
    out = L.decode_noalloc(dv.p, dv.q, k4, v4, dv.words, dv.seq_lens, dv.q_pos, dv.rope, torch.empty_like(dv.q))
    assert torch.equal(out.view(torch.int16), decode(dv, k4, v4).view(torch.int16))
    check(out, M.attention(w, kv, vv), "decode_noalloc")


# ---------------------------------------------------------------- shared runs

@pytest.mark.parametrize("hq,hkv,d,chunk", [(8, 8, 128, 0), (4, 2, 64, 0), (32, 8, 128, 3), (28, 4, 128, 5), (16, 2, 64, 1),
                                            (32, 1, 128, 0), (64, 1, 128, 5), (64, 8, 128, 0)])
def test_shared_decode_matches_64_bits(hq, hkv, d, chunk):
    w = W.decode_zipf(f"i4sh{hq}", batch=10, hq=hq, hkv=hkv, d=d, docs_per_seq=4, doc_tokens=150, pool_docs=4, zipf_s=1.0,
                      suffix_tokens=21, seed=760 + hq + chunk)
    dv, k4, v4, kv, vv = on_device(w)
    plan = shared_plan(dv, chunk)
    assert (plan.items_host[:, 4] * (hq // hkv) <= 64).all()
    ref = M.attention(w, kv, vv)
    out = la().decode_shared(dv.p, dv.q, k4, v4, dv.words, dv.q_pos, dv.rope, plan)
    check(out, ref, f"int4 shared-run decode {hq}/{hkv} chunk {chunk}")
    ws = torch.empty(la().decode_shared_workspace_bytes(dv.p, plan.num_slots), dtype=torch.uint8, device="cuda")
    la().decode_shared_partials(dv.p, dv.q, k4, v4, dv.words, dv.q_pos, dv.rope, plan, ws)
    two = la().decode_shared_combine(dv.p, plan, ws, torch.empty_like(dv.q))
    assert torch.equal(two.view(torch.int16), out.view(torch.int16))


def test_shared_decode_holes_and_long_items():
    dw, _ = W.mixed_mqa(n_decode=8, n_prefill=1, chunk=16, hq=32, hkv=1, d=128, pool_docs=40, ctx_lo=1, ctx_hi=3000,
                        doc_lo=1, doc_hi=700, seed=765)
    dv, k4, v4, kv, vv = on_device(dw)
    ref = M.attention(dw, kv, vv)
    for chunk in (0, 4, 64):
        check(la().decode_shared(dv.p, dv.q, k4, v4, dv.words, dv.q_pos, dv.rope, shared_plan(dv, chunk)), ref, f"chunk {chunk}")


# ---------------------------------------------------------------- the calls together

def _model(batch, hq, hkv, d, seed):
    """Documents of a small model layer: bf16 rows per document, as K rotated at local positions and V."""
    w = W.decode_zipf("i4run", batch=batch, hq=hq, hkv=hkv, d=d, docs_per_seq=3, doc_tokens=83, pool_docs=5, zipf_s=1.0,
                      suffix_tokens=13, seed=seed)
    return w


def test_ingest_decode_append_and_stage_for_prefill():
    """Documents are written as they are ingested, a batch decodes over them, every sequence appends the decoded
    token's row to its tail, decodes again, and the same blocks are staged for a prefill in bf16."""
    L = la()
    w = _model(4, 8, 2, 128, 780)
    dv = to_device(w)
    dv.p.kv_dtype = L.LAZY_INT4
    kp, vp = L.empty_pools(dv.p)
    kp.fill_(255), vp.fill_(255)  # NaN scales wherever nothing is written
    for doc in range(len(w.doc_len)):
        n = int(w.doc_len[doc])
        blocks = w.doc_blocks[int(w.doc_block_indptr[doc]):int(w.doc_block_indptr[doc + 1])]
        if n == 0 or len(blocks) == 0:
            continue
        slots = torch.from_numpy(L.token_slots(blocks, 0, n)).cuda()
        at = slots.long().cpu()
        k, v = (x[at // 16, :, at % 16].cuda() for x in (w.k_pool, w.v_pool))
        for a in range(0, n, 50):  # in pieces
            L.cache_write(dv.p, k[a:a + 50], v[a:a + 50], slots[a:a + 50], kp, vp)
    k4, v4 = M.int4_pools(w)
    kv = torch.from_numpy(np.nan_to_num(M.int4_values(k4.numpy(), 128, False))).cuda()
    vv = torch.from_numpy(np.nan_to_num(M.int4_values(v4.numpy(), 128, True))).cuda()
    ref = M.attention(w, kv, vv)
    check(decode(dv, kp, vp), ref, "decode after ingestion")
    check(L.decode_shared(dv.p, dv.q, kp, vp, dv.words, dv.q_pos, dv.rope, shared_plan(dv)), ref, "shared after ingestion")
    # the tail document of 13 tokens grows by one
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(4, 2, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    slots = []
    for s in range(4):
        doc, n = w.seq_segments(s)[-1]
        slots.append(int(w.doc_blocks[int(w.doc_block_indptr[doc])]) * 16 + n)
        w.seg_len[int(w.seg_indptr[s + 1]) - 1] = n + 1
        w.doc_len[doc] = n + 1
    slots = torch.tensor(slots, dtype=torch.int32)
    L.cache_write(dv.p, k.cuda(), v.cuda(), slots.cuda(), kp, vp)
    w.k_pool[slots.long() // 16, :, slots.long() % 16] = k
    w.v_pool[slots.long() // 16, :, slots.long() % 16] = v
    w.q_pos = w.q_pos + 1
    k4, v4 = M.int4_pools(w)
    kv = torch.from_numpy(np.nan_to_num(M.int4_values(k4.numpy(), 128, False))).cuda()
    vv = torch.from_numpy(np.nan_to_num(M.int4_values(v4.numpy(), 128, True))).cuda()
    ref = M.attention(w, kv, vv)
    d2 = to_device(w)
    d2.p.kv_dtype = L.LAZY_INT4
    check(decode(d2, kp, vp), ref, "decode after the append")
    # staged in bf16 for the calls that take no quantised pool: decode and prefill over the staged blocks
    ids = torch.arange(w.num_pool_blocks, dtype=torch.int32, device="cuda")
    ks, vs = L.cache_read(d2.p, kp, vp, ids)
    d2.p.kv_dtype = 0
    staged = L.decode(d2.p, d2.q, ks, vs, d2.words, d2.seq_lens, d2.q_pos, d2.rope)
    assert (staged.double() - ref[0]).abs().max() < 2e-2  # bf16 keys, values and weights
    cu = torch.arange(5, dtype=torch.int32, device="cuda") * 14  # the tail as a chunk: its last row sees what the decode saw
    q = torch.zeros(56, 8, 128, dtype=torch.bfloat16, device="cuda")
    q[13::14] = d2.q
    out = L.prefill(d2.p, q, cu, d2.q_pos - 14, 14, ks, vs, d2.words, d2.seq_lens, d2.rope)
    # (a decode's query sits one past its last key, a chunk's on it: compare with a decode there)
    near = L.decode(d2.p, d2.q, ks, vs, d2.words, d2.seq_lens, d2.q_pos - 1, d2.rope)
    assert (out[13::14].float() - near.float()).abs().max() < 2e-2


def test_captured_steps_replay():
    """A decode step (write the new token, then attend) captured once and replayed on new inputs, with its own
    workspace; a second captured step beside it."""
    L = la()
    w = _model(4, 8, 2, 128, 790)
    dv, k4, v4, kv, vv = on_device(w)
    steps = []
    for i in range(2):
        st = dict(q=dv.q.clone(), k=torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda"), out=torch.empty_like(dv.q),
                  kp=k4.clone(), vp=v4.clone(), ws=torch.empty(max(256, L.decode_workspace_bytes(dv.p)), dtype=torch.uint8, device="cuda"),
                  slots=torch.full((4,), -1, dtype=torch.int32, device="cuda"))

        def step(st=st):
            L.cache_write(dv.p, st["k"], st["k"], st["slots"], st["kp"], st["vp"])
            L.decode(dv.p, st["q"], st["kp"], st["vp"], dv.words, dv.seq_lens, dv.q_pos, dv.rope, out=st["out"], workspace=st["ws"])

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        steps.append((g, st))
    for i, (g, st) in enumerate(steps):
        st["q"].copy_(dv.q * (i + 2))
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for (g, st), s in zip(steps, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for i, (g, st) in enumerate(steps):
        w2 = _model(4, 8, 2, 128, 790)
        w2.q = (w2.q.float() * (i + 2)).to(torch.bfloat16)
        check(st["out"], M.attention(w2, kv, vv), f"replay {i}")
        assert torch.equal(st["kp"], k4)


def test_captured_behind_copies_and_joined_streams():
    # In a captured step every call follows what a launch may not overlap: a copy, a fill, two streams that join; and its
    # inputs come from right before it. Replayed on new inputs, twice in a row.
    L = la()
    w = _model(3, 8, 2, 128, 792)
    dv, k4, v4, kv, vv = on_device(w)
    ids = torch.arange(w.num_pool_blocks, dtype=torch.int32, device="cuda")
    plan = shared_plan(dv)
    src = [k4.clone(), v4.clone(), dv.q.clone()]
    kp, vp, q = torch.zeros_like(k4), torch.zeros_like(v4), torch.zeros_like(dv.q)
    out, outs = torch.empty_like(dv.q), torch.empty_like(dv.q)
    rows = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(256, L.decode_workspace_bytes(dv.p)), dtype=torch.uint8, device="cuda")
    wss = torch.empty(L.decode_shared_workspace_bytes(dv.p, plan.num_slots), dtype=torch.uint8, device="cuda")
    ko = torch.empty(w.num_pool_blocks, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        kp.copy_(src[0])  # a copy, then the join of two streams
        side.wait_stream(here)
        with torch.cuda.stream(side):
            vp.copy_(src[1])
        q.copy_(src[2]).mul_(1)
        here.wait_stream(side)
        L.decode(dv.p, q, kp, vp, dv.words, dv.seq_lens, dv.q_pos, dv.rope, out=out, workspace=ws)
        side.wait_stream(here)
        with torch.cuda.stream(side):
            L.cache_read(dv.p, kp, vp, ids, ko, vo)
        rows.zero_()
        L.cache_write(dv.p, rows, rows, slots, kp, vp)
        here.wait_stream(side)
        L.decode_shared(dv.p, q, kp, vp, dv.words, dv.q_pos, dv.rope, plan, out=outs, workspace=wss)
        ws.fill_(255)

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for scale in (1, 2):
        src[2].copy_(dv.q * scale)
        for x in (kp, vp, out, outs, ko, vo):
            x.zero_()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        w2 = _model(3, 8, 2, 128, 792)
        w2.q = (w2.q.float() * scale).to(torch.bfloat16)
        ref = M.attention(w2, kv, vv)
        check(out, ref, f"replay, queries times {scale}")
        check(outs, ref, f"shared replay, queries times {scale}")
        assert torch.equal(torch.nan_to_num(ko.float()), torch.nan_to_num(kv.float().to(torch.bfloat16).float()))
        assert torch.equal(torch.nan_to_num(vo.float()), torch.nan_to_num(vv.float().to(torch.bfloat16).float()))


def test_side_stream():
    L = la()
    w = _model(3, 8, 2, 64, 791)
    dv, k4, v4, kv, vv = on_device(w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = L.decode(dv.p, dv.q, k4, v4, dv.words, dv.seq_lens, dv.q_pos, dv.rope, stream=s)
    back = L.cache_read(dv.p, k4, v4, torch.arange(w.num_pool_blocks, dtype=torch.int32, device="cuda"), stream=s)
    s.synchronize()
    check(out, M.attention(w, kv, vv), "side stream")
    assert torch.equal(torch.nan_to_num(back[0].float()), torch.nan_to_num(kv.float().to(torch.bfloat16).float()))
