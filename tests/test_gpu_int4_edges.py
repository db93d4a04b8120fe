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


def attend(w, s, kv, vv, keep=None, freqs=None, scale=None):
    """M.attention of sequence s alone over the keys that `keep` (one truth value per token) names: output, bound, and
    weights [hkv, G, t]."""
    hkv, d = w.num_kv_heads, w.head_dim
    scale = d ** -0.5 if scale is None else scale
    f = torch.as_tensor(w.rope_theta ** (-2.0 * np.arange(d // 2) / d) if freqs is None else freqs, dtype=torch.float64, device="cuda")

    def rotate(x, n):
        c, r = torch.cos(n[:, None, None] * f), torch.sin(n[:, None, None] * f)
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat((a * c - b * r, a * r + b * c), -1)

    ks, vs, pos, p = [], [], [], int(w.seq_pos0[s])
    for doc, n in w.seq_segments(s):
        blk = torch.as_tensor(w.doc_blocks[int(w.doc_block_indptr[doc]):][:(n + 15) // 16].astype(np.int64), device="cuda")
        ks.append(kv[blk].transpose(1, 2).reshape(-1, hkv, d)[:n])
        vs.append(vv[blk].transpose(1, 2).reshape(-1, hkv, d)[:n])
        pos.append(torch.full((n,), float(p), dtype=torch.float64, device="cuda"))
        p += n
    k, v = rotate(torch.cat(ks), torch.cat(pos)), torch.cat(vs)
    if keep is not None:
        k, v = k[keep], v[keep]
    q = rotate(w.q[s].double().cuda()[None], torch.tensor([float(w.q_pos[s])], dtype=torch.float64, device="cuda"))[0].reshape(hkv, -1, d)
    wgt = torch.softmax(torch.einsum("hgd,thd->hgt", q, k) * scale, -1)
    o = torch.einsum("hgt,thd->hgd", wgt, v)
    e = scale * 2.0 ** -11 * 9 / 8 * q.norm(dim=-1) * k.norm(dim=-1).amax(0)[:, None]
    big = 2 * v.abs().reshape(-1, hkv, d // 64, 64).amax(-1)
    spread = torch.einsum("hgt,thj->hgj", wgt, big).repeat_interleave(64, -1)
    dev = torch.stack([torch.einsum("gt,tgd->gd", wgt[h], (v[:, h, None] - o[h][None]).abs()) for h in range(hkv)])
    bound = 2.0 ** -8 * o.abs() + e[..., None] * dev + 2.0 ** -10 * spread + 2.0 ** -18 * torch.einsum("hgt,thd->hgd", wgt, v.abs())
    return o.reshape(-1, d), bound.reshape(-1, d), wgt


def partials_out(dv, k4, v4, plan, rope=None):
    """The shared-run decode's fp32 partials merged in 64 bits: [B, Hq, d], without the output's rounding to bf16."""
    L = la()
    hq, d, n = dv.p.num_q_heads, dv.p.head_dim, plan.num_slots
    ws = torch.full((L.decode_shared_workspace_bytes(dv.p, n) // 4,), float("nan"), device="cuda")
    L.decode_shared_partials(dv.p, dv.q, k4, v4, dv.words, dv.q_pos, dv.rope if rope is None else rope, plan, ws)
    acc = ws[:n * hq * d].view(n, hq, d).double()
    m, l = ws[n * hq * d:n * hq * (d + 2)].view(n, hq, 2).double().unbind(-1)
    out = []
    for a, b in zip(plan.slot_indptr_host, plan.slot_indptr_host[1:]):
        f = torch.exp2(m[a:b] - m[a:b].amax(0))
        out.append((f[..., None] * acc[a:b]).sum(0) / (f * l[a:b]).sum(0)[..., None])
    return torch.stack(out)


def spans(v4, w):
    """Per key and dim s c, the part of a V value above its group's zero, of a pool [blocks, heads, 16, d]."""
    z = M.int4_values(np.concatenate((np.zeros_like(v4[..., :16 * w.head_dim // 2]), v4[..., 16 * w.head_dim // 2:]), -1), w.head_dim, True)
    return torch.from_numpy(np.nan_to_num(M.int4_values(v4, w.head_dim, True) - z)).cuda()


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


# one long document: its blocks' words take id_bits = 14 (18 bits of offset from its start)
def one_document(tokens, hq, seed, d=128):
    return W.decode_zipf("i4one", batch=1, hq=hq, hkv=1, d=d, docs_per_seq=1, doc_tokens=tokens, pool_docs=1, zipf_s=1.0, seed=seed)


# 131072 keys of nearly equal weight as one item: 8192, 4096 or 2048 blocks a team of warps for more than 16, up to 16 and up
# to 8 rows (4 rows: another tile), and two CTAs' rows. In the 2-norm the output's rounding to bf16 is at most 2^-8 and that
# of the weights' f16 products 1.7 * 2^-10 (see test_long_sums_stay_exact); sums that the products truncate would be off by
# 2048 * 2^-25 of 1.35 ranges' middle and more, 2 to 8 % of the output.
@pytest.mark.parametrize("hq", [3, 8, 16, 32, 48])
def test_shared_long_items_stay_exact(hq):
    w = one_document(131072, hq, 830)
    dv, k4, v4, kv, vv = on_device(w, id_bits=14)
    want, _ = M.attention(w, kv, vv)
    plan = shared_plan(dv, 8192)
    assert plan.num_items == 1
    out = la().decode_shared(dv.p, dv.q, k4, v4, dv.words, dv.q_pos, dv.rope, plan).double()
    assert ((out - want).norm() / want.norm()).item() < 2.0 ** -7


# The same keys in items of 256 blocks, the automatic plan's longest, for more than 16 rows, from the fp32 partials (no
# rounding to bf16). A term w s c is off by two roundings of 2^-11 at most, each of standard deviation 2^-11 / sqrt(3) or
# less, and s c has 2.6 standard deviations of a value in the root mean square (codes from 0, 7.5 steps their middle): like
# the output itself these errors add up as independent ones, 2.6 sqrt(2 / 3) 2^-11 = 2.1 * 2^-11 of it; the queries' rounding
# to f16 moves the weights by less than 2^-11 of each. sqrt(2.1^2 + 1) * 2^-11 = 2.3 * 2^-11 < 2^-9. Truncated over 256
# blocks the sums would be off by 1.5 times that bound.
@pytest.mark.parametrize("hq", [32, 48])
def test_shared_partials_of_256_blocks_stay_exact(hq):
    w = one_document(131072, hq, 831)
    dv, k4, v4, kv, vv = on_device(w, id_bits=14)
    want, _ = M.attention(w, kv, vv)
    plan = shared_plan(dv, 256)
    assert plan.num_items == 32
    out = partials_out(dv, k4, v4, plan)[0]
    assert ((out - want[0]).norm() / want.norm()).item() < 2.0 ** -9


# maxima and V scales that keep growing behind the first 64 blocks of a warp: sums that were set aside follow them
@pytest.mark.parametrize("hq,d", [(3, 128), (8, 128), (16, 64), (32, 128)])
def test_set_aside_sums_follow_new_maxima_and_scales(hq, d):
    w = one_document(16000, hq, 832, d)
    nb = w.num_pool_blocks
    at = torch.empty(nb, dtype=torch.float64)
    at[torch.from_numpy(w.doc_blocks.astype(np.int64))] = torch.arange(nb, dtype=torch.float64)
    at = at.view(-1, 1, 1, 1)
    w.k_pool = (w.k_pool.double() * (0.25 + 2 * at / nb)).to(torch.bfloat16)
    w.v_pool = (w.v_pool.double() * 2.0 ** (at // 64)).to(torch.bfloat16)
    dv, k4, v4, kv, vv = on_device(w, num_splits=1, id_bits=14)
    ref = M.attention(w, kv, vv)
    check(decode(dv, k4, v4), ref, "per sequence")
    for chunk in (1000, 130):
        check(la().decode_shared(dv.p, dv.q, k4, v4, dv.words, dv.q_pos, dv.rope, shared_plan(dv, chunk)), ref, f"chunk {chunk}")


# a document whose first block, the second of a pair, is not in the pool: that block is left out, and the document's others
# are attended at their own positions
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 1, 64), (32, 1, 128)])
@pytest.mark.parametrize("bad", [3, 4, 10])
def test_blocks_behind_a_bad_one_keep_their_positions(hq, hkv, d, bad):
    L = la()
    w = W.decode_zipf("i4bad", batch=2, hq=hq, hkv=hkv, d=d, docs_per_seq=1, doc_tokens=48, pool_docs=2, zipf_s=0.5, share=False,
                      suffix_tokens=900, seed=840, shift=5000)
    dv, k4, v4, kv, vv = on_device(w, num_splits=1)
    words = dv.words.clone()
    words[1, bad] |= (1 << 18) - 1
    out = L.decode(dv.p, dv.q, k4, v4, words, dv.seq_lens, dv.q_pos, dv.rope)
    assert L.device_status(clear=True) == L.LAZY_DEV_BAD_BLOCK_ID
    for s in range(2):
        keep = torch.ones(948, dtype=torch.bool, device="cuda")
        if s == 1:
            keep[16 * bad:16 * bad + 16] = False
        want, bound, _ = attend(w, s, kv, vv, keep)
        check(out[s], (want, bound), f"sequence {s}")


# A weight times a V scale is rounded to f16 once. Every row has one key that outweighs the others by 2^4 to 2^7.9, in a tile
# behind the first (so its weight is no power of two); no rotation, queries and keys of a single dim. Elementwise the fp32
# partials are off by 2^-11 of sum_j w_j s c, by fp32's 2^-18 of sum_j w_j |v_j|, and by the rounding of the query times the
# softmax scale to f16: 2^-11 of that key's score x in its exponent, which moves the output by 2^-11 x sum_j w_j |v_j - out|
# at most. With a softmax scale of ln 2 / 8 the products are the queries times a power of two: nothing is rounded there.
@pytest.mark.parametrize("hq,hkv,d", [(64, 1, 128), (32, 8, 128), (32, 2, 64)])
@pytest.mark.parametrize("exact_scores", [False, True])
def test_weight_times_scale_is_rounded_once(hq, hkv, d, exact_scores):
    w = W.decode_zipf("i4w", batch=12, hq=hq, hkv=hkv, d=d, docs_per_seq=1, doc_tokens=41, pool_docs=1, zipf_s=1.0, share=False, seed=850)
    last = w.doc_blocks[w.doc_block_indptr[1:][np.diff(w.doc_block_indptr) > 0] - 1].astype(np.int64)
    w.k_pool = torch.where(torch.isnan(w.k_pool), w.k_pool, torch.zeros_like(w.k_pool))
    w.k_pool[last, :, 8, 0] = 15.0  # token 40: code 15 of scale 1
    w.q.zero_()
    g = torch.Generator().manual_seed(851)
    score = 4 + 3.9 * torch.rand(12, hq, generator=g, dtype=torch.float64)  # in log2 units
    scale = float(np.float32(np.log(2.0) / 8)) if exact_scores else d ** -0.5
    w.q[..., 0] = (score / scale / 15 / np.log2(np.e)).to(torch.bfloat16)
    dv, k4, v4, kv, vv = on_device(w)
    if exact_scores:
        dv.p.sm_scale = scale
    zero = np.zeros(d // 2)
    out = partials_out(dv, k4, v4, shared_plan(dv), la().rope_table_init(dv.p, freqs=zero))
    sc = spans(v4.cpu().numpy(), w)
    worst = 0.0
    for s in range(12):
        want, _, wgt = attend(w, s, kv, vv, freqs=zero, scale=scale)
        part = attend(w, s, kv, sc, freqs=zero, scale=scale)[0]
        mean = attend(w, s, kv, vv.abs(), freqs=zero, scale=scale)[0]
        bound = 2.0 ** -11 * part + 2.0 ** -18 * mean
        if not exact_scores:
            blk = torch.as_tensor(w.doc_blocks[int(w.doc_block_indptr[w.seq_segments(s)[0][0]]):][:3].astype(np.int64), device="cuda")
            v = vv[blk].transpose(1, 2).reshape(-1, hkv, d)[:41]
            x = w.q[s, :, 0].double().cuda() * 15 * scale
            dev = torch.einsum("hgt,thgd->hgd", wgt, (v[:, :, None] - want.view(1, hkv, -1, d)).abs()).reshape(hq, d)
            bound = bound + 2.0 ** -11 * x[:, None] * dev
        worst = max(worst, ((out[s] - want).abs() / bound).max().item())
    assert worst <= 1.0, f"off by {worst:.2f} of the bound"


def product_bound(w, s, v4, wgt):
    """The bound on sequence s's fp32 partials that lazy_attn.h states for the weights' products, elementwise [hq, d]: with W
    the weights over the row's largest, sum_j max(2^-11 W_j s_j, 2^-29 max s) c_j / sum_j W_j. wgt: softmax weights [hkv, G, t]."""
    d, hkv = w.head_dim, w.num_kv_heads
    pool = v4.cpu().numpy()
    one = pool.copy()  # scales of 1, zeros of 0: the values are the codes; and codes of 1: the values are scales
    meta = one[..., 8 * d:].reshape(*one.shape[:-1], -1, 4)
    meta[...] = np.array([0x80, 0x3F, 0, 0], np.uint8)
    codes = M.int4_values(one, d, True)
    sc = pool.copy()
    sc[..., :8 * d] = 0x11
    sc[..., 8 * d:].reshape(*sc.shape[:-1], -1, 4)[..., 2:] = 0
    scales = np.nan_to_num(M.int4_values(sc, d, True))

    def tokens(x):
        x, got = torch.from_numpy(x), []
        for doc, n in w.seq_segments(s):
            blk = torch.as_tensor(w.doc_blocks[int(w.doc_block_indptr[doc]):][:(n + 15) // 16].astype(np.int64))
            got.append(x[blk].transpose(1, 2).reshape(-1, hkv, d)[:n])
        return torch.cat(got).cuda()

    c, sc = tokens(codes), tokens(scales)
    top = sc.amax(0)
    W = wgt / wgt.amax(-1, keepdim=True)
    out = torch.empty(hkv, W.shape[1], d, dtype=torch.float64, device="cuda")
    for h in range(hkv):
        for g in range(W.shape[1]):
            x = torch.maximum(2.0 ** -11 * W[h, g, :, None] * sc[:, h], 2.0 ** -29 * top[h]) * c[:, h]
            out[h, g] = x.sum(0) / W[h, g].sum()
    return out.reshape(-1, d)


# One key far above a long flat tail, whose weights of 2^-20 to 2^-28 add up to between 2^-11 and 2^-3 of it: one team of warps
# attends all of them (32 rows in one item). Scores without a rounding, as above. A lane adds the weights, and the weights times
# zeros, of an eighth of the 131072 keys one by one in fp32, each sum off by 2^-24 of itself at most: 2^14 * 2^-24 of the sums
# in all, which is 2^-10 (|out| + max |z|) of the output. (Tails below 2^-25 of the first key are lost there in its own lane.)
def test_long_tail_of_small_weights():
    w = one_document(131072, 32, 860)
    w.k_pool.zero_()
    w.k_pool[int(w.doc_blocks[0]), :, 0, 0] = 15.0  # the first key: code 15 of scale 1
    scale = float(np.float32(np.log(2.0) / 8))
    w.q.zero_()
    w.q[0, :, 0] = (torch.linspace(20, 28, 32, dtype=torch.float64) * 8 / 15).to(torch.bfloat16)
    dv, k4, v4, kv, vv = on_device(w, id_bits=14)
    dv.p.sm_scale = scale
    zero = np.zeros(64)
    plan = shared_plan(dv, 8192)
    out = partials_out(dv, k4, v4, plan, la().rope_table_init(dv.p, freqs=zero))[0]
    want, _, wgt = attend(w, 0, kv, vv, freqs=zero, scale=scale)
    bound = product_bound(w, 0, v4, wgt) + 2.0 ** -18 * attend(w, 0, kv, vv.abs(), freqs=zero, scale=scale)[0]
    least = (vv - spans(v4.cpu().numpy(), w)).abs().max()
    bound = bound + 2.0 ** -10 * (want.abs() + least)
    worst = ((out - want).abs() / bound).max().item()
    assert worst <= 1.0, f"off by {worst:.2f} of the bound"


# A key that no query attends to (weight 2^-120) has V values of 2^10, 2^17 and 2^24 times the others', all of weight 1: what
# it leaves of their products. Scores without a rounding, as above.
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (32, 2, 128), (16, 2, 64)])
@pytest.mark.parametrize("big", [10, 17, 24])
def test_large_v_scale_without_weight(hq, hkv, d, big):
    w = W.decode_zipf("i4big", batch=2, hq=hq, hkv=hkv, d=d, docs_per_seq=1, doc_tokens=20, pool_docs=1, zipf_s=1.0, share=False, seed=861)
    w.k_pool = torch.where(torch.isnan(w.k_pool), w.k_pool, torch.zeros_like(w.k_pool))
    for s in range(2):
        blk = int(w.doc_blocks[int(w.doc_block_indptr[w.seq_segments(s)[0][0]])])
        w.k_pool[blk, :, 5, 0] = -60.0  # exact: the group's least value
        w.v_pool[blk, :, 5] = (w.v_pool[blk, :, 5].double() * 2.0 ** big).to(torch.bfloat16)
    w.q.zero_()
    w.q[..., 0] = 16.0
    dv, k4, v4, kv, vv = on_device(w)
    dv.p.sm_scale = scale = float(np.float32(np.log(2.0) / 8))
    zero = np.zeros(d // 2)
    out = partials_out(dv, k4, v4, shared_plan(dv), la().rope_table_init(dv.p, freqs=zero))
    for s in range(2):
        want, _, wgt = attend(w, s, kv, vv, freqs=zero, scale=scale)
        assert (wgt[:, :, 5] < 2.0 ** -119).all()
        bound = product_bound(w, s, v4, wgt) + 2.0 ** -18 * attend(w, s, kv, vv.abs(), freqs=zero, scale=scale)[0]
        worst = ((out[s] - want).abs() / bound).max().item()
        assert worst <= 1.0, f"off by {worst:.2f} of the bound"


# A captured step's block table is as wide as its longest sequence may become: pieces and ranges go by the sequences' own
# lengths, so the same bits come out at every width. 4, 3 and 96 sequences: several pieces a unit, one piece a unit, and ranges
# (a sequence of more than 512 blocks a piece); entries behind a sequence are never read.
@pytest.mark.parametrize("batch,hq,hkv,d,hi", [(4, 32, 8, 128, 4200), (3, 8, 1, 64, 9000), (96, 16, 8, 64, 3000), (96, 16, 8, 64, 12000),
                                               (20, 32, 1, 128, 60000)])
def test_width_of_the_table_changes_nothing(batch, hq, hkv, d, hi):
    L = la()
    dw, _ = W.mixed_mqa(n_decode=batch, n_prefill=1, chunk=16, hq=hq, hkv=hkv, d=d, pool_docs=40, ctx_lo=1, ctx_hi=hi, doc_lo=1,
                        doc_hi=700, seed=870 + batch)
    dv, k4, v4, kv, vv = on_device(dw)
    tight, ref = decode(dv, k4, v4), M.attention(dw, kv, vv)
    check(tight, ref, "tight")
    mb, words = dv.p.max_blocks_per_seq, dv.words
    for wide in (mb + 1, 2048, 8192, 30000):
        if wide <= mb:
            continue
        dv.p.max_blocks_per_seq = wide
        dv.words = torch.full((batch, wide), -1, dtype=torch.int32, device="cuda")
        dv.words[:, :mb] = words
        ws = torch.full((L.decode_workspace_bytes(dv.p),), 255, dtype=torch.uint8, device="cuda")
        out = decode(dv, k4, v4, workspace=ws)
        check(out, ref, f"{wide} blocks wide")
        assert torch.equal(out.view(torch.int16), tight.view(torch.int16)), f"{wide} blocks wide"


def test_captured_step_follows_its_lengths():
    # one capture, a wide table, lengths that pass from ranges to whole units, to pieces, to nothing and back; the workspace is
    # another captured call's too
    L = la()
    dw, _ = W.mixed_mqa(n_decode=96, n_prefill=1, chunk=16, hq=16, hkv=8, d=64, pool_docs=40, ctx_lo=1, ctx_hi=12000, doc_lo=1,
                        doc_hi=700, seed=880)
    dv, k4, v4, _, _ = on_device(dw)
    mb, full = dv.p.max_blocks_per_seq, dv.seq_lens.clone()
    assert mb > 512
    words = torch.full((96, 4096), -1, dtype=torch.int32, device="cuda")
    words[:, :mb] = dv.words
    dv.words, dv.p.max_blocks_per_seq = words, 4096
    ws = torch.empty(L.decode_workspace_bytes(dv.p), dtype=torch.uint8, device="cuda")
    small = L.Params.from_buffer_copy(dv.p)
    small.num_seqs = 2  # many pieces a unit
    lens, out, out2 = full.clone(), torch.empty_like(dv.q), torch.empty_like(dv.q[:2])

    def step():
        L.decode(dv.p, dv.q, k4, v4, dv.words, lens, dv.q_pos, dv.rope, out=out, workspace=ws)
        L.decode(small, dv.q[:2], k4, v4, dv.words[:2], lens[:2], dv.q_pos[:2], dv.rope, out=out2, workspace=ws)

    assert L.decode_workspace_bytes(small) <= ws.numel()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for what, new in (("ranges", full), ("whole units", full.clamp(max=16 * 500)), ("nothing", full * 0), ("ranges again", full),
                      ("one long", torch.where(full == full.max(), full, 0)), ("tokens", full.clamp(max=1))):
        lens.copy_(new)
        want, want2 = (L.decode(p, dv.q[:n], k4, v4, dv.words[:n], lens[:n], dv.q_pos[:n], dv.rope) for p, n in ((dv.p, 96), (small, 2)))
        out.fill_(7), out2.fill_(7), ws.fill_(255)
        g.replay()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(out2.view(torch.int16), want2.view(torch.int16)), what
        # (a length cut at 500 blocks may name a document's unwritten slots as keys: NaN, the same on both sides)
        assert torch.count_nonzero(out[new == 0]) == 0 and not (out == 7).flatten(1).all(1).any(), what


# V values of 2^118 over 20 keys: the sums of codes times scales reach 20 * 5 * 2^118 < 2^125, inside fp32 (a weight of 1 may
# not be held as more). And of 2^124 on a single key, whose scale is among the largest that a group of bf16 values has.
@pytest.mark.parametrize("hq,hkv,d", [(3, 1, 128), (8, 1, 64), (32, 2, 128)])
@pytest.mark.parametrize("tokens,power", [(20, 118), (1, 124)])
def test_v_values_near_the_end_of_fp32(hq, hkv, d, tokens, power):
    w = W.decode_zipf("i4top", batch=2, hq=hq, hkv=hkv, d=d, docs_per_seq=1, doc_tokens=tokens, pool_docs=1, zipf_s=1.0, share=False,
                      seed=890)
    w.v_pool = (w.v_pool.double() * 2.0 ** power).to(torch.bfloat16)
    dv, k4, v4, kv, vv = on_device(w)
    ref = M.attention(w, kv, vv)
    check(decode(dv, k4, v4), ref, "per sequence")
    check(la().decode_shared(dv.p, dv.q, k4, v4, dv.words, dv.q_pos, dv.rope, shared_plan(dv)), ref, "shared")


def test_wide_table_of_many_sequences():
    # more sequences than every CTA looks through: ranges, whatever the lengths
    L = la()
    dw, _ = W.mixed_mqa(n_decode=2100, n_prefill=1, chunk=16, hq=2, hkv=1, d=64, pool_docs=20, ctx_lo=1, ctx_hi=90, doc_lo=1, doc_hi=40,
                        seed=871)
    dv, k4, v4, kv, vv = on_device(dw)
    ref = M.attention(dw, kv, vv)
    check(decode(dv, k4, v4), ref, "tight")
    words = torch.full((2100, 600), -1, dtype=torch.int32, device="cuda")
    words[:, :dv.p.max_blocks_per_seq] = dv.words
    dv.words, dv.p.max_blocks_per_seq = words, 600
    ws = torch.full((L.decode_workspace_bytes(dv.p),), 255, dtype=torch.uint8, device="cuda")
    check(decode(dv, k4, v4, workspace=ws), ref, "600 blocks wide")
