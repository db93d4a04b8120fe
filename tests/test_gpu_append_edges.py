"""GPU: tables of new tokens where the arrays of a call are one another's, or end beside one another."""
import numpy as np
import pytest
import torch

import append_model as A
from gpu_util import la
from test_gpu_append import i32, params, u32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    la().device_status(clear=True)
    yield
    assert la().device_status(clear=True) == 0, "device status word set"


# one CTA's rows, a thread a row (few sequences, many), a warp 256 rows
@pytest.mark.parametrize("batch,new_hi", [(5, 9), (5, 40), (20, 900), (1100, 5), (3, 200000)])
def test_chunks_that_begin_at_pos_in_place(batch, new_hi):
    # every sequence's tokens begin a document: tail_start is pos, and both lengths are updated where they are
    L = la()
    rng = np.random.default_rng(batch + new_hi)
    new = rng.integers(0, new_hi + 1, batch)
    new[:2] = new_hi
    used = rng.integers(0, 300, batch)
    pos = used - np.minimum(used, rng.integers(0, 16, batch))  # documents that ended inside blocks
    need = int(sum(-(-n // 16) for n in new))
    wide = int(max(-(-u // 16) + -(-n // 16) for u, n in zip(used, new)))
    p = params(batch, wide, need + 20)
    words = rng.integers(0, 1 << 30, (batch, wide)).astype(np.uint32)
    free, rows = rng.permutation(need + 20)[:need], int(new.sum()) + 3
    doc = 1024 if new_hi > 8000 else 0
    want = A.append(new, used, pos, pos, free, words, rows, max_blocks=wide, id_bits=18, pool=need + 20, doc=doc)
    assert want[-1] == 0
    w, seq_lens, at = u32(words), i32(used), i32(pos)
    out = L.AppendTables.empty(p, rows).replace(seq_lens=seq_lens, pos=at)
    L.append_tokens(p, i32(new), seq_lens, at, at, i32(free), w, doc_tokens=doc, out=out)
    got = (w, out.seq_lens, out.pos, out.q_start, out.cu_rows, out.block_indptr, out.slots, out.local_pos)
    for name, g, x in zip(("words", "seq_lens", "pos", "q_start", "cu_rows", "block_indptr", "slots", "local_pos"), got, want):
        assert np.array_equal(g.cpu().numpy(), np.ascontiguousarray(x).view(np.int32)), name
