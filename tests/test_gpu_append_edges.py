"""GPU: tables of new tokens where the arrays of a call are one another's, end beside one another or hold bad ids, and a server's
steps against what its pools hold."""
import numpy as np
import pytest
import torch

import append_model as A
import fp8_block_model as M
from gpu_util import la
from test_gpu_append import THETA, Server, i32, params, u32
from test_gpu_fp8_block import check, same_records, scatter

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


# ids outside the pool where every id of the words' field is a block: no word can say that a block is none. One CTA's rows,
# a thread a row; a document of more ids than a warp looks at at once
@pytest.mark.parametrize("batch,new_hi,room", [(6, 60, 0), (6, 60, 2000), (300, 1, 0), (3, 1200, 0)])
@pytest.mark.parametrize("key_positions", [False, True])
def test_bad_ids_of_a_full_field_add_nothing(batch, new_hi, room, key_positions):
    L = la()
    rng = np.random.default_rng(batch + new_hi)
    p = params(batch, 80, 256, bits=8, key_positions=key_positions)
    new = np.where(np.arange(batch) % 3 == 2, 0, rng.integers(1, new_hi + 1, batch))
    zero = np.zeros(batch, np.int64)
    new[np.cumsum(-(-new // 16)) > 250] = 0
    need = -(-new // 16)
    at = np.cumsum(need) - need
    free = rng.permutation(256)[:int(need.sum()) + 4]
    bad = [0, int(np.argmax(np.where(np.arange(batch) > 0, need, 0)))]  # the first and the longest other
    broken = free.copy()
    broken[at[bad[0]]], broken[at[bad[1]] + need[bad[1]] - 1] = 256, -3
    words = rng.integers(0, 1 << 31, (batch, 80)).astype(np.uint32)
    rows = int(new.sum()) + room
    want = list(A.append(new, zero, zero, zero, free, words, rows, max_blocks=80, id_bits=8, pool=256, doc=1024, key_positions=key_positions))
    assert want[-1] == 0
    for s in bad:  # as it was, but for its place in the list and among the rows
        want[0][s], want[1][s], want[2][s] = words[s], 0, 0
        want[6][want[4][s]:want[4][s + 1]], want[7][want[4][s]:want[4][s + 1]] = -1, 0
    w, lens, pos, start = u32(words), i32(zero), i32(zero), i32(zero)
    out = L.AppendTables.empty(p, rows).replace(seq_lens=lens, pos=pos)

    def call(n, first):
        L.append_tokens(p, i32(n), lens, pos, start, i32(broken), w, first_free=first, doc_tokens=1024, out=out)

    call(new, None)
    assert L.device_status(clear=True) == L.LAZY_DEV_BAD_BLOCK_ID
    got = (w, out.seq_lens, out.pos, out.q_start, out.cu_rows, out.block_indptr, out.slots, out.local_pos)
    for name, g, x in zip(("words", "seq_lens", "pos", "q_start", "cu_rows", "block_indptr", "slots", "local_pos"), got, want):
        assert np.array_equal(g.cpu().numpy(), np.ascontiguousarray(x).view(np.int32)), name
    # the next call's tokens go into a block of the list's, not into the pool's last one
    again = np.zeros(batch, np.int64)
    again[bad[0]] = 2
    call(again, out.block_indptr[-1:])
    block = int(free[int(need.sum())])
    assert L.device_status(clear=True) == 0 and out.slots[:2].tolist() == [16 * block, 16 * block + 1]


def test_a_smaller_batch_in_slices_of_the_tables_goes_on_in_the_list():
    L = la()
    big, p = params(5, 8, 40), params(2, 8, 40)
    t = L.AppendTables.empty(big, 64)
    z5, z2, free = i32([0] * 5), i32([0] * 2), i32(np.random.default_rng(2).permutation(40))
    L.append_tokens(big, i32([17, 1, 16, 0, 3]), z5, z5, z5, free, u32(np.zeros((5, 8), np.uint32)), out=t)
    taken = set((t.slots[:37] // 16).tolist())
    assert int(t.block_indptr[-1]) == len(taken) == 5
    first = t.block_indptr[-1:].clone()
    t = t.replace(cu_rows=t.cu_rows[:3], block_indptr=t.block_indptr[:3])
    L.append_tokens(p, i32([20, 2]), z2, z2, z2, free, u32(np.zeros((2, 8), np.uint32)), first_free=first, out=t)
    assert int(t.block_indptr[-1]) == 8 and not taken & set((t.slots[:22] // 16).tolist()) and int(t.cu_rows[-1]) == 22


class Held:
    """What fp8_block_model.attention asks of a workload, of a server's sequences: documents of srv.doc tokens behind one another."""

    def __init__(self, srv, words, lens, q):
        self.num_seqs, self.num_q_heads, self.num_kv_heads, self.head_dim, self.rope_theta = srv.batch, srv.hq, srv.hkv, srv.d, THETA
        self.q, self.q_pos, self.seq_pos0 = q, lens, np.zeros(srv.batch, np.int64)
        ids = words & (1 << 18) - 1
        self.segs, self.doc_blocks, self.doc_block_indptr = [], [], [0]
        for s, n in enumerate(lens):
            self.segs.append([])
            for a in range(0, int(n), srv.doc):
                self.segs[s].append((len(self.doc_block_indptr) - 1, min(srv.doc, int(n) - a)))
                self.doc_blocks += ids[s, a // 16:-(-min(int(n), a + srv.doc) // 16)].tolist()
                self.doc_block_indptr.append(len(self.doc_blocks))
        self.doc_blocks = np.array(self.doc_blocks)

    def seq_segments(self, s):
        return self.segs[s]


@pytest.mark.parametrize("d", [64, 128])
def test_captured_steps_against_what_the_pools_hold(d):
    # tables, records and both decodes of every step: tables against the model of them, records byte for byte, outputs within the
    # elementwise bound of 64-bit attention over the records' values
    L = la()
    batch, cap = 5, 300
    srv = Server("fp8_e4m3_block", batch, d, cap, 60)
    g = torch.Generator("cuda").manual_seed(17)
    words, lens, free = np.zeros((batch, 60), np.uint32), np.zeros(batch, np.int64), srv.free.cpu().numpy()
    pools, first, start = [x.cpu().numpy() for x in srv.pools], 0, np.zeros(batch, np.int64)
    q_in = torch.zeros(batch, 8, d, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q_in)
    ws = torch.empty(max(256, L.decode_workspace_bytes(srv.p)), dtype=torch.uint8, device="cuda")

    def step():
        srv.step()
        srv.attend(q_in, out, ws)

    def follow(new, run):
        nonlocal words, lens, first
        srv.new.copy_(i32(new))
        srv.rows(new, g)
        q_in.copy_(torch.randn(batch, 8, d, generator=g, device="cuda").to(torch.bfloat16))
        run()
        want = A.append(new, lens, lens, start, free, words, cap, max_blocks=60, id_bits=18, pool=400, first=first, doc=srv.doc)
        assert want[-1] == 0
        for name, got, x in zip(("words", "seq_lens", "pos", "q_start", "cu_rows", "block_indptr", "slots", "local_pos"), (srv.words, *srv.out), want):
            assert np.array_equal(got.cpu().numpy(), np.ascontiguousarray(x).view(np.int32)), name
        words, lens, first = want[0], want[1].astype(np.int64), int(want[5][-1])
        total = int(sum(new))
        for x, y, rows, is_v in zip(srv.pools, pools, (srv.k, srv.v), (False, True)):
            scatter(want[6][:total], y, rows[:total].cpu(), is_v)
            same_records(x, y, d)

    def attention():
        values = [torch.from_numpy(np.nan_to_num(M.values(y, d, is_v))).cuda() for y, is_v in zip(pools, (False, True))]
        w = Held(srv, words, lens, q_in)
        return w, M.attention(w, *values)

    follow([100, 1, 64, 16, 0], step)
    want, bound = attention()[1]
    check(out[:4], (want[:4], bound[:4]), "prompts")
    assert not out[4].any()  # a sequence without a token
    srv.new.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(24):
        follow([(i + s) % 4 if s < 4 else 1 for s in range(batch)], graph.replay)
        w, ref = attention()
        check(out, ref, f"step {i}")
    docs = [n for s in range(batch) for _, n in w.segs[s]]
    seg = np.cumsum([0] + [len(s) for s in w.segs])
    items, slots = L.plan_shared_host(srv.p, len(docs), seg, np.arange(len(docs)), docs, w.doc_block_indptr, w.doc_blocks)
    two = L.decode_shared(srv.p, q_in, *srv.pools, srv.words, srv.pos, srv.rope, L.SharedPlan(items, slots))
    check(two, ref, "shared")
