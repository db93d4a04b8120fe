"""CPU: arguments of append_tokens that are refused."""
import ctypes



def _L():
    from paged_kv_cache_57_gb300 import build
    build.build()
    from paged_kv_cache_57_gb300 import lazy_attn
    return lazy_attn


def _params(**kw):
    base = dict(num_seqs=2, num_q_heads=4, num_kv_heads=2, head_dim=128, num_pool_blocks=10, max_blocks_per_seq=4)
    return _L().make_params(**{**base, **kw})


def test_pos_out_in_the_place_of_another_tail_start():
    L = _L()
    new, lens, pos, start, free, words, len_out, q_start, cu, indptr, slots = (ctypes.c_void_p(1 << 20 | i << 12) for i in range(11))
    rc = L._lib.lazy_attn_append_tokens(ctypes.byref(_params()), new, lens, pos, start, free, 4, None, 16, 8, words, len_out, start, q_start, cu,
                                        indptr, slots, None, None)
    assert rc == L.LAZY_ERR_INVALID_ARG
