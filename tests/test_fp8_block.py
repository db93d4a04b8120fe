"""CPU: pools of e4m3 codes with block scales and the tables of new tokens -- sizes, refusals, planner,
and the 64-bit models that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import append_model as A
import fp8_block_model as M
from paged_kv_cache_57_gb300 import workloads as W

FAKE = 1 << 20
KIND = "fp8_e4m3_block"


def _L():
    from paged_kv_cache_57_gb300 import build
    build.build()
    from paged_kv_cache_57_gb300 import lazy_attn
    return lazy_attn


def _params(**kw):
    base = dict(num_seqs=2, num_q_heads=4, num_kv_heads=2, head_dim=128, num_pool_blocks=10, max_blocks_per_seq=4, kv_dtype=KIND)
    return _L().make_params(**{**base, **kw})


@pytest.mark.parametrize("d,want", [(128, 2080), (64, 1056)])
def test_record_bytes(d, want):
    L = _L()
    p = _params(head_dim=d)
    assert L.pool_record_bytes(p) == want == M.record_bytes(d)
    k, v = L.empty_pools(p, device="cpu")
    assert k.shape == v.shape == (10, 2, want) and k.dtype == torch.uint8


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", ["decode", "decode_noalloc", "decode_shared", "decode_shared_partials"])
def test_short_pools_are_refused(which, d):
    L = _L()
    p = _params(num_seqs=1, head_dim=d)
    q, words, i32 = torch.zeros(1, 4, d, dtype=torch.bfloat16), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    rope, ws = torch.zeros(L.rope_table_bytes(p), dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8)
    plan = L.SharedPlan(np.zeros((1, L.PLAN_ITEM_INTS), np.int32), np.array([0, 1], np.int32), device="cpu")
    args = {"decode": (words, i32, i32, rope), "decode_noalloc": (words, i32, i32, rope, torch.empty_like(q)),
            "decode_shared": (words, i32, rope, plan), "decode_shared_partials": (words, i32, rope, plan, ws)}[which]
    whole = L.empty_pools(p, device="cpu")
    for k, v in ((whole[0].flatten()[:-1], whole[1]), (whole[0], whole[1][:9])):
        with pytest.raises(ValueError, match="num_pool_blocks"):
            getattr(L, which)(p, q, k, v, *args)
    with pytest.raises(ValueError, match="k_pool must be a CUDA tensor"):  # whole ones go on to the next check
        getattr(L, which)(p, q, *whole, *args)


def test_refusals_come_before_cuda():
    L = _L()
    fake = ctypes.c_void_p(FAKE)
    bad, un = L.LAZY_ERR_INVALID_ARG, L.LAZY_ERR_UNSUPPORTED

    def write(p, k=FAKE, slots=FAKE, kp=FAKE, vp=FAKE, n=3, ks=(256, 128)):
        return L._lib.lazy_attn_cache_write(ctypes.byref(p), k, *ks, FAKE, 256, 128, n, slots, kp, vp, None)

    def read(p, kp=FAKE, n=3, ids=FAKE, ko=FAKE):
        return L._lib.lazy_attn_cache_read(ctypes.byref(p), kp, FAKE, n, ids, ko, FAKE, None)

    def decode(p, pool=FAKE):
        return L._lib.lazy_attn_decode(ctypes.byref(p), fake, ctypes.c_void_p(pool), *([fake] * 6), fake, 1 << 20, None)

    def shared(p):
        return L._lib.lazy_attn_decode_shared(ctypes.byref(p), *([fake] * 6), 1, fake, 1, fake, fake, fake, 1 << 20, None)

    p = _params()
    assert write(p, n=0) == 0 and read(p, n=0) == 0 and write(p, n=-1) == bad and read(p, n=-1) == bad
    assert write(p, ks=(-1, 128)) == bad and write(p, kp=FAKE + 8) == bad and write(p, k=FAKE + 1) == bad
    assert write(p, slots=FAKE + 2) == bad and read(p, kp=FAKE + 8) == bad and read(p, ids=FAKE + 1) == bad
    assert write(p, n=2 ** 30) == un and read(p, n=2 ** 30) == un
    for q in (_params(dtype="f32"),):
        assert write(q) == un and read(q) == un and decode(q) == un and shared(q) == un
    for kw in (dict(k_scale=0.5), dict(v_scale=2.0)):  # the records carry the scales
        assert decode(_params(**kw)) == bad and shared(_params(**kw)) == bad and write(_params(**kw)) == bad
    q = _params(key_positions=True)
    assert L._lib.lazy_attn_decode_alibi(ctypes.byref(q), *([fake] * 7), fake, fake, fake, 1 << 20, None) == un
    assert L._lib.lazy_attn_decode_shared_alibi(ctypes.byref(q), *([fake] * 6), 1, fake, 1, fake, fake, fake, fake, 1 << 20, None) == un
    assert L._lib.lazy_attn_prefill(ctypes.byref(p), fake, fake, fake, 1, 1, *([fake] * 7), 1 << 20, None) == un
    assert L._lib.lazy_attn_materialize(ctypes.byref(p), *([fake] * 8), None) == un
    assert L._lib.lazy_attn_debug_gather(ctypes.byref(p), *([fake] * 7), None) == un
    q = _params(num_q_heads=32)
    assert L._lib.lazy_attn_mixed(ctypes.byref(q), *([fake] * 3), 1, fake, 1, fake, fake, ctypes.byref(q), *([fake] * 3), 1, 1,
                                  *([fake] * 6), 1 << 30, None) == un
    assert decode(_params(num_seqs=2 ** 30)) == un and decode(p, FAKE + 8) == bad
    many = _params(num_q_heads=65536, num_kv_heads=65536)
    assert decode(many) == un and shared(many) == un
    assert decode(_params(num_q_heads=130)) == un and shared(_params(num_q_heads=130)) == un
    for other in (6, 7, -1):
        q = _params()
        q.kv_dtype = other
        assert decode(q) == un and write(q) == un


def test_plan_keeps_items_of_at_most_64_rows():
    L = _L()
    w = W.decode_zipf("plan8", batch=16, hq=64, hkv=4, d=128, docs_per_seq=4, doc_tokens=64, pool_docs=3, zipf_s=1.0, seed=77)
    p = _params(num_seqs=16, num_q_heads=64, num_kv_heads=4, num_pool_blocks=w.num_pool_blocks, max_blocks_per_seq=w.max_blocks_per_seq)
    items, _ = L.plan_shared_host(p, len(w.doc_len), w.seg_indptr, w.seg_doc, w.seg_len, w.doc_block_indptr, w.doc_blocks)
    assert (items[:, 4] * 16 <= 64).all() and (items[:, 4] > 1).any()


def test_plan_takes_long_items_from_both_ends():
    L = _L()
    w = W.decode_zipf("order8", batch=16, hq=16, hkv=2, d=128, docs_per_seq=4, doc_tokens=640, pool_docs=9, zipf_s=1.0, suffix_tokens=50, seed=78)
    p = _params(num_seqs=16, num_q_heads=16, num_kv_heads=2, num_pool_blocks=w.num_pool_blocks, max_blocks_per_seq=w.max_blocks_per_seq)
    for chunk in (0, 3, 40):
        items, slots = L.plan_shared_host(p, len(w.doc_len), w.seg_indptr, w.seg_doc, w.seg_len, w.doc_block_indptr, w.doc_blocks, chunk_blocks=chunk)
        nb, rows = items[:, 2], items[:, 4] * 8
        cost = nb * np.array([1, 2, 4])[np.searchsorted([8, 16], rows)]
        long = 2 * nb > nb.max()
        n = int(long.sum())
        assert 0 < n and long[:n].all() and (np.diff(cost[n:]) <= 0).all()
        assert (np.diff(cost[:n:2]) <= 0).all() and (np.diff(cost[1:n:2]) >= 0).all() and cost[:n:2].min() >= cost[1:n:2].max(initial=0)
        # every member's slots once, in the order of its partials
        taken = [(int(m[0]), int(m[2])) for it in items for m in it[8:8 + 4 * it[4]].reshape(-1, 4)]
        assert sorted(x for _, x in taken) == list(range(int(slots[-1]))) and all(slots[s] <= x < slots[s + 1] for s, x in taken)


def test_long_sequences_and_items_are_cut():
    # a warp adds up 16384 blocks at most, and a CTA has four
    L = _L()
    for hq in (4, 32, 33, 64):
        for wide in (65536, 65537):
            p = _params(num_seqs=1, num_q_heads=hq, num_kv_heads=1, num_pool_blocks=8, max_blocks_per_seq=wide, num_splits=1)
            assert (L.decode_workspace_bytes(p) > 0) == (wide > 65536), (hq, wide)
    n = 40000
    p = _params(num_seqs=1, num_q_heads=4, num_kv_heads=1, num_pool_blocks=n, max_blocks_per_seq=n)
    i32 = lambda *x: np.array(x, dtype=np.int32)
    items, _ = L.plan_shared_host(p, 1, i32(0, 1), i32(0), i32(16 * n), i32(0, n), np.arange(n, dtype=np.int32), chunk_blocks=n)
    assert items[:, 2].max() == 16384 and items[:, 2].sum() == n


# ---------------------------------------------------------------- the models

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("is_v", [False, True])
def test_model_rows_round_trip(d, is_v):
    rng = np.random.default_rng(d)
    rec = rng.integers(0, 256, M.record_bytes(d)).astype(np.uint8)
    x = rng.standard_normal((16, d))
    M.put(rec, {t: x[t] for t in range(5)}, is_v)
    got = M.values(rec, d, is_v)
    s = M.scale_of(rec, d)
    assert 224 * s < np.abs(x[:5]).max() <= 448 * s and not got[5:].any()
    assert (np.abs(got[:5] - x[:5]) <= np.maximum(2.0 ** -4 * np.abs(x[:5]), 2.0 ** -10 * s)).all()
    before = got[:5].copy()
    M.put(rec, {5: 100 * x[5], 7: x[7]}, is_v)  # the scale grows; row 6 stays 0
    got, s2 = M.values(rec, d, is_v), M.scale_of(rec, d)
    assert s2 > 8 * s and not got[6].any() and np.abs(got[5] - 100 * x[5]).max() <= 2.0 ** -4 * np.abs(100 * x[5]).max()
    big = np.abs(before) >= 2.0 ** -6 * s2  # codes that stay normal keep their values
    assert big.any() and np.array_equal(got[:5][big], before[big])
    M.put(rec, {9: 1e-3 * x[9]}, is_v)  # and does not shrink
    assert M.scale_of(rec, d) == s2 and np.array_equal(M.values(rec, d, is_v)[:9], got[:9])


def test_model_exponents_and_not_finite():
    assert M.exponent([448.0]) == 0 and M.exponent([448.5]) == 1 and M.exponent([224.0]) == -1
    assert M.exponent([0.0]) == M.exponent([np.nan, np.inf]) == M.exponent([1e-38]) == -100 and M.exponent([3.3e38]) == 119
    rec = np.zeros(M.record_bytes(64), np.uint8)
    M.put(rec, {0: np.r_[np.nan, np.inf, -np.inf, np.ones(61)]}, False)
    got = M.values(rec, 64, False)[0]
    assert np.isnan(got[:3]).all() and (got[3:] == 1).all()


def test_model_codes_agree_with_torch():
    codes = np.arange(256).astype(np.uint8)
    assert np.array_equal(M.E4M3, torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)


def test_model_pools_agree_with_rows():
    w = W.decode_zipf("m8", batch=2, hq=4, hkv=2, d=64, docs_per_seq=2, doc_tokens=37, pool_docs=3, zipf_s=1.0, seed=5)
    for pool, src, is_v in zip(M.pools(w), (w.k_pool, w.v_pool), (False, True)):
        x = src.double().numpy()
        for b, h in ((0, 0), (1, 1), (w.num_pool_blocks - 1, 0)):
            rec = np.zeros(M.record_bytes(64), np.uint8)
            rows = {t: x[b, h, t] for t in range(16)}
            if np.isnan(x[b, h]).all():
                continue
            M.put(rec, rows, is_v)
            assert np.array_equal(rec, pool[b, h].numpy())


def test_model_attention_agrees_with_the_oracle():
    import oracle
    w = W.decode_zipf("mo8", batch=3, hq=4, hkv=2, d=64, docs_per_seq=2, doc_tokens=37, pool_docs=3, zipf_s=1.0, suffix_tokens=5, seed=6)
    out, _ = M.attention(w, torch.nan_to_num(w.k_pool.double()), torch.nan_to_num(w.v_pool.double()))
    assert np.abs(out.numpy() - oracle.attention(w)).max() < 1e-12


# ---------------------------------------------------------------- tables of new tokens

def test_append_refusals_come_before_cuda():
    L = _L()
    bad = L.LAZY_ERR_INVALID_ARG
    names = ("new_lens", "seq_lens", "pos", "tail_start", "free", "words", "len_out", "pos_out", "q_start", "cu", "indptr", "slots")

    def call(p, num_free=4, doc=16, rows=8, **kw):
        a = {**{n: FAKE for n in names}, **kw}
        return L._lib.lazy_attn_append_tokens(ctypes.byref(p), a["new_lens"], a["seq_lens"], a["pos"], a["tail_start"], a["free"], num_free,
                                              None, doc, rows, a["words"], a["len_out"], a["pos_out"], a["q_start"], a["cu"], a["indptr"],
                                              a["slots"], None, None)

    p = _params(kv_dtype=None)
    for n in names:
        assert call(p, **{n: None}) == bad, n
    assert call(p, num_free=-1) == bad and call(p, rows=-1) == bad and call(p, doc=-16) == bad and call(p, doc=24) == bad
    assert call(_params(head_dim=96)) == L.LAZY_ERR_UNSUPPORTED
    assert call(_params(num_seqs=-1)) == bad


def test_append_binding_checks_shapes():
    L = _L()
    p = _params(kv_dtype=None)
    z = lambda n: torch.zeros(n, dtype=torch.int32)
    ok = dict(new_lens=z(2), seq_lens=z(2), pos=z(2), tail_start=z(2), free_blocks=z(9), block_words=z(8), out=L.AppendTables.empty(p, 5, "cpu"))
    for name, x in (("new_lens", z(1)), ("seq_lens", z(1)), ("pos", z(1)), ("tail_start", z(0)), ("block_words", z(7)), ("first_free", z(2)),
                    ("num_rows", 4), ("out", ok["out"].replace(cu_rows=z(2))), ("out", ok["out"].replace(block_indptr=z(2))),
                    ("out", ok["out"].replace(q_start=z(1)))):
        with pytest.raises(ValueError):
            L.append_tokens(p, **{**ok, name: x})
    for name, x in (("local_pos", z(4)), ("slots", z(5).long()), ("pos", z(4)[::2])):
        with pytest.raises(ValueError):
            ok["out"].replace(**{name: x})
    with pytest.raises(ValueError, match="num_rows or out"):
        L.append_tokens(p, **{**ok, "out": None})
    with pytest.raises(ValueError, match="CUDA"):
        L.append_tokens(p, **ok)


def test_append_tables_are_fixed():
    # a call writes where the tables were when they were made
    L = _L()
    t = L.AppendTables.empty(_params(kv_dtype=None), 5, "cpu")
    for name in ("slots", "pos", "rows", "_ptrs"):
        with pytest.raises(AttributeError):
            setattr(t, name, getattr(t, name))
    other = t.replace(pos=torch.zeros(2, dtype=torch.int32))
    assert other.slots is t.slots and other.pos is not t.pos


@pytest.mark.parametrize("key_positions", [False, True])
def test_model_appends_what_the_packer_packs(key_positions):
    # requests from nothing, one document each: the words and lengths of the packer, whose documents are the blocks given
    L = _L()
    lens = [1, 16, 17, 100, 5]
    n = [-(-x // 16) for x in lens]
    free = np.random.default_rng(3).permutation(40)[:sum(n) + 2].astype(np.int32)
    p = L.make_params(num_seqs=5, num_q_heads=4, num_kv_heads=2, head_dim=64, num_pool_blocks=40, max_blocks_per_seq=7,
                      key_positions=key_positions)
    indptr = np.cumsum([0] + n)
    words, used = L.pack_block_words_host(p, 5, np.arange(6), np.arange(5), lens, None, indptr, free)
    z = np.zeros(5, np.int32)
    got = A.append(lens, z, z, z, free, np.zeros((5, 7), np.uint32), 140, max_blocks=7, id_bits=18, pool=40, doc=0,
                   key_positions=key_positions)
    assert np.array_equal(got[0], words) and np.array_equal(got[1], used) and got[2].tolist() == lens and got[-1] == 0
    assert got[4].tolist() == np.cumsum([0] + lens).tolist() and got[5].tolist() == indptr.tolist()
    slots = np.concatenate([L.token_slots(free[indptr[i]:indptr[i + 1]], 0, lens[i]) for i in range(5)])
    assert np.array_equal(got[6][:139], slots) and got[6][139] == -1
