"""Pool writes and reads, and int4 pools, on the CPU: argument rules, slots, the format's
restatement against itself."""
import ctypes

import numpy as np
import pytest
import torch

import int4_model as M
import oracle
from paged_kv_cache_57_gb300 import workloads as W


def _L():
    from paged_kv_cache_57_gb300 import lazy_attn
    return lazy_attn


def _params(**kw):
    base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, num_pool_blocks=10, max_blocks_per_seq=4,
                dtype="bf16", kv_dtype="int4")
    base.update(kw)
    return _L().make_params(**base)


FAKE = 4096  # never dereferenced: the arguments are rejected first


def _write(p, k=FAKE, ks=(256, 128), v=FAKE, vs=(256, 128), n=3, slots=FAKE, kp=FAKE, vp=FAKE):
    return _L()._lib.lazy_attn_cache_write(ctypes.byref(p), k, *ks, v, *vs, n, slots, kp, vp, None)


def _read(p, kp=FAKE, vp=FAKE, n=3, ids=FAKE, ko=FAKE, vo=FAKE):
    return _L()._lib.lazy_attn_cache_read(ctypes.byref(p), kp, vp, n, ids, ko, vo, None)


@pytest.mark.parametrize("kv,dtype,d,want", [("int4", "bf16", 128, 1152), ("int4", "bf16", 64, 576),
                                             ("fp8_e4m3", "bf16", 128, 2048), (None, "bf16", 128, 4096),
                                             (None, "bf16", 64, 2048), (None, "f32", 64, 4096)])
def test_record_bytes(kv, dtype, d, want):
    L = _L()
    p = _params(kv_dtype=kv, dtype=dtype, head_dim=d)
    assert L.pool_record_bytes(p) == want
    k, v = L.empty_pools(p, device="cpu")
    assert k.numel() * k.element_size() == v.numel() * v.element_size() == 10 * 2 * want
    if kv == "int4":
        assert M.record_bytes(d) == want


def test_bad_params_have_no_record():
    L = _L()
    assert L.pool_record_bytes(_params(head_dim=80)) == 0
    assert L._lib.lazy_attn_pool_record_bytes(None) == 0


def test_write_and_read_refusals_come_before_cuda():
    L = _L()
    bad, un = L.LAZY_ERR_INVALID_ARG, L.LAZY_ERR_UNSUPPORTED
    p = _params()
    assert _write(p, n=0) == 0 and _read(p, n=0) == 0
    assert _write(p, n=-1) == bad and _read(p, n=-1) == bad
    for name in ("k", "v", "slots", "kp", "vp"):
        assert _write(p, **{name: None}) == bad, name
    for name in ("kp", "vp", "ids", "ko", "vo"):
        assert _read(p, **{name: None}) == bad, name
    assert _write(p, ks=(-256, 128)) == bad and _write(p, vs=(256, -128)) == bad
    assert _write(p, kp=FAKE + 8) == bad and _write(p, vp=FAKE + 4) == bad
    assert _write(p, k=FAKE + 1) == bad and _write(p, v=FAKE + 1) == bad and _write(p, slots=FAKE + 2) == bad
    for name in ("kp", "vp", "ko", "vo"):
        assert _read(p, **{name: FAKE + 8}) == bad, name
    assert _read(p, ids=FAKE + 1) == bad
    assert _write(_params(num_pool_blocks=0)) == bad and _read(_params(num_pool_blocks=0)) == bad
    assert _write(p, n=2 ** 30) == un and _read(p, n=2 ** 30) == un
    for q in (_params(dtype="f32"), _params(dtype="f32", kv_dtype="fp8_e4m3")):
        assert _write(q) == un and _read(q) == un
    for scale in (1e-31, 1e31):
        q = _params(kv_dtype="fp8_e4m3", v_scale=scale)
        assert _write(q) == bad and _read(q) == bad
    q = _params(kv_dtype="fp8_e4m3", dtype="bf16")
    q.kv_dtype = 4
    assert _write(q) == un and _read(q) == un
    assert _write(_params(head_dim=96)) == un


def test_int4_argument_rules():
    L = _L()
    fake = ctypes.c_void_p(FAKE)
    bad, un = L.LAZY_ERR_INVALID_ARG, L.LAZY_ERR_UNSUPPORTED

    def decode(p):
        return L._lib.lazy_attn_decode(ctypes.byref(p), *([fake] * 8), fake, 1 << 20, None)

    def shared(p):
        return L._lib.lazy_attn_decode_shared(ctypes.byref(p), *([fake] * 6), 1, fake, 1, fake, fake, fake, 1 << 20,
                                              None)

    assert decode(_params(dtype="f32")) == un and shared(_params(dtype="f32")) == un
    # the records carry the scales
    for kw in (dict(k_scale=0.5), dict(v_scale=2.0)):
        assert decode(_params(**kw)) == bad and shared(_params(**kw)) == bad and _write(_params(**kw)) == bad
    p = _params(key_positions=True)
    assert L._lib.lazy_attn_decode_alibi(ctypes.byref(p), *([fake] * 7), fake, fake, fake, 1 << 20, None) == un
    assert L._lib.lazy_attn_decode_shared_alibi(ctypes.byref(p), *([fake] * 6), 1, fake, 1, fake, fake, fake, fake,
                                                1 << 20, None) == un
    p = _params()
    assert L._lib.lazy_attn_prefill(ctypes.byref(p), fake, fake, fake, 1, 1, *([fake] * 7), 1 << 20, None) == un
    assert L._lib.lazy_attn_materialize(ctypes.byref(p), *([fake] * 8), None) == un
    assert L._lib.lazy_attn_debug_gather(ctypes.byref(p), *([fake] * 7), None) == un
    p = _params(num_q_heads=32, num_kv_heads=2)
    assert L._lib.lazy_attn_mixed(ctypes.byref(p), *([fake] * 3), 1, fake, 1, fake, fake, ctypes.byref(p),
                                  *([fake] * 3), 1, 1, *([fake] * 6), 1 << 30, None) == un
    # more work units than a grid has CTAs (each needs a row of q: none is launched)
    assert decode(_params(num_seqs=2 ** 30, max_blocks_per_seq=4)) == un
    for many in (_params(num_q_heads=65536, num_kv_heads=65536), _params(num_q_heads=131072, num_kv_heads=65536)):
        assert decode(many) == un and shared(many) == un
    # an unaligned pool, workspace too small
    p = _params()
    assert L._lib.lazy_attn_decode(ctypes.byref(p), fake, ctypes.c_void_p(FAKE + 8), *([fake] * 6), fake, 1 << 20,
                                   None) == bad


def test_int4_plan_keeps_items_of_at_most_64_rows():
    L = _L()
    w = W.decode_zipf("plan4", batch=16, hq=64, hkv=4, d=128, docs_per_seq=4, doc_tokens=64, pool_docs=3, zipf_s=1.0,
                      seed=77)
    p = _params(num_seqs=16, num_q_heads=64, num_kv_heads=4, num_pool_blocks=w.num_pool_blocks,
                max_blocks_per_seq=w.max_blocks_per_seq)
    items, _ = L.plan_shared_host(p, len(w.doc_len), w.seg_indptr, w.seg_doc, w.seg_len, w.doc_block_indptr,
                                  w.doc_blocks)
    assert (items[:, 4] * 16 <= 64).all() and (items[:, 4] > 1).any()
    # the widest and longest first
    cost = items[:, 2] * np.array([1, 2, 4])[np.searchsorted([8, 16], items[:, 4] * 16)]
    assert (np.diff(cost) <= 0).all()


def test_token_slots():
    L = _L()
    blocks = [7, 3, 11]
    assert L.token_slots(blocks, 0, 48).tolist() == [16 * b + r for b in blocks for r in range(16)]
    assert L.token_slots(blocks, 15, 2).tolist() == [7 * 16 + 15, 3 * 16]
    assert L.token_slots(blocks, 48, 0).tolist() == []
    assert L.token_slots([], 0, 0).tolist() == []
    for first, count in ((-1, 2), (0, 49), (47, 2), (5, -1)):
        with pytest.raises(ValueError):
            L.token_slots(blocks, first, count)


def test_binding_checks_shapes():
    L = _L()
    p = _params()
    k = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        L.cache_write(p, k, k, torch.zeros(3, dtype=torch.int32), *L.empty_pools(p, device="cpu"))
    small = torch.zeros((9, 2, 1152), dtype=torch.uint8)
    with pytest.raises(ValueError, match="records"):
        L.cache_read(p, small, small, torch.zeros(3, dtype=torch.int32))


# ---------------------------------------------------------------- the restatement itself

def test_model_rows_round_trip():
    rng = np.random.default_rng(1)
    for d in (64, 128):
        pool = rng.integers(0, 256, (2, 1, M.record_bytes(d)), dtype=np.uint8)
        x = M.bf16_round(rng.standard_normal((16, d)) * 3)
        for is_v in (False, True):
            for t in range(16):
                M.int4_put(pool, 1, 0, t, x[t], is_v)
            got = M.int4_values(pool, d, is_v)[1, 0]
            _, s, z = M.int4_quantise(x)
            # half a step, and the scale's rounding (2^-9) over 15 steps for the largest
            assert (np.abs(got - x) <= np.repeat(s, 64, -1) * (0.5 + 15 * 2.0 ** -8)).all()


def test_model_whole_pools_agree_with_rows():
    w = W.decode_zipf("pools4", batch=2, hq=4, hkv=2, d=128, docs_per_seq=2, doc_tokens=20, pool_docs=3, zipf_s=1.0,
                      seed=3)
    k4, v4 = M.int4_pools(w)
    for pool, src, is_v in ((k4, w.k_pool, False), (v4, w.v_pool, True)):
        one = np.zeros_like(pool.numpy())
        x = src.double().numpy()
        for b in range(x.shape[0]):
            for h in range(2):
                for t in range(16):
                    M.int4_put(one, b, h, t, x[b, h, t], is_v)
        assert np.array_equal(one, pool.numpy())


def test_model_e4m3_agrees_with_torch():
    x = np.concatenate([np.linspace(-448, 448, 20001), np.linspace(-0.1, 0.1, 5001)]).astype(np.float32)
    lib = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(M.e4m3_codes(x.astype(np.float64)), lib)


def test_model_attention_agrees_with_the_oracle():
    w = W.decode_zipf("att4", batch=3, hq=6, hkv=2, d=64, docs_per_seq=3, doc_tokens=21, pool_docs=4, zipf_s=1.0,
                      suffix_tokens=5, seed=4)
    out, bound = M.attention(w, torch.nan_to_num(w.k_pool.double()), torch.nan_to_num(w.v_pool.double()))
    assert np.abs(out.numpy() - oracle.attention(w)).max() < 1e-12
    assert (bound > 0).all() and bound.max() < 0.05
