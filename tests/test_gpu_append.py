"""GPU: tables of new tokens against the sequence-by-sequence model, and the step that they make with
the pool writes, the decodes and the prefill."""
import numpy as np
import pytest
import torch

import append_model as A
import fp8_block_model as M
from gpu_util import la

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    la().device_status(clear=True)
    yield
    assert la().device_status(clear=True) == 0, "device status word set"


def i32(x):
    return torch.from_numpy(np.asarray(x, np.int64).astype(np.int32)).cuda()


def u32(words):
    return torch.from_numpy(np.ascontiguousarray(words).view(np.int32)).cuda()


def params(batch, wide, pool, bits=18, key_positions=False):
    return la().make_params(num_seqs=batch, num_q_heads=8, num_kv_heads=2, head_dim=128, num_pool_blocks=pool, max_blocks_per_seq=wide,
                            id_bits=bits, key_positions=key_positions)


def requests(rng, batch, new_hi, ctx_hi, tail_hi):
    new = rng.integers(0, new_hi + 1, batch)
    ctx = rng.integers(0, ctx_hi + 1, batch)
    tail = np.where(rng.random(batch) < 0.3, 0, rng.integers(0, tail_hi + 1, batch))
    holes = np.where(ctx > 0, rng.integers(0, 16, batch), 0)
    used = np.where(tail > 0, 16 * (-(-(ctx + holes) // 16)) + tail, ctx + holes)
    return new, used, ctx + tail, ctx


def compare(p, new, used, pos, start, free, words, rows, first=0, doc=4096, local=True, stream=None, inplace=False):
    L = la()
    want = A.append(new, used, pos, start, free, words, rows, max_blocks=p.max_blocks_per_seq, id_bits=p.id_bits or 18,
                    pool=p.num_pool_blocks, first=first, doc=doc, key_positions=bool(p.key_positions))
    w = u32(words)
    out = L.AppendTables.empty(p, rows)
    for x in out:
        x.fill_(-77)
    seq_lens, at = i32(used), i32(pos)
    if inplace:
        out = out.replace(seq_lens=seq_lens, pos=at)
    if not local:
        out = out.replace(local_pos=None)
    got = L.append_tokens(p, i32(new), seq_lens, at, i32(start), i32(free) if len(free) else i32([0])[:0], w,
                          first_free=i32([first]) if first else None, doc_tokens=doc, out=out, stream=stream)
    assert got is out
    assert L.device_status(clear=True) == want[-1]
    got = [w, out.seq_lens, out.pos, out.q_start, out.cu_rows, out.block_indptr, out.slots] + ([out.local_pos] if local else [])
    for name, g, x in zip(("words", "seq_lens", "pos", "q_start", "cu_rows", "block_indptr", "slots", "local_pos"), got, want):
        x = np.ascontiguousarray(x).view(np.int32)
        assert np.array_equal(g.cpu().numpy(), x), (name, np.argwhere(g.cpu().numpy() != x)[:4])
    return want


# one CTA for few rows, two launches for many; batches beside multiples of 32 and 1024; no sequence at all
@pytest.mark.parametrize("batch,new_hi,ctx,tail,room", [(1, 1, 0, 0, 0), (1, 40000, 100, 30, 3), (3, 0, 50, 20, 5), (31, 1, 3000, 64, 1), (64, 1, 4096, 64, 0),
                                                        (33, 200, 300, 100, 17), (700, 8, 2000, 300, 2001), (1024, 3, 100, 10, 0), (1025, 5, 100, 40, 1),
                                                        (3000, 1, 500, 40, 9), (2500, 30, 0, 0, 2), (5, 3000, 5000, 900, 0), (0, 0, 0, 0, 7), (9000, 1, 30, 20, 0)])
@pytest.mark.parametrize("key_positions", [False, True])
def test_tables_match_the_model(batch, new_hi, ctx, tail, room, key_positions):
    rng = np.random.default_rng(batch + new_hi)
    new, used, pos, start = requests(rng, batch, new_hi, ctx, tail)
    need = int(sum(-(-(q - a + n) // 16) - -(-(q - a) // 16) for n, q, a in zip(new, pos, start)))
    pool = need + 50
    wide = int(max([-(-u // 16) + -(-n // 16) + 1 for u, n in zip(used, new)] or [1]))
    p = params(batch, wide, pool, key_positions=key_positions)
    words = (rng.integers(0, 1 << 14, (batch, wide)) << 18 | rng.integers(0, pool, (batch, wide))).astype(np.uint32)
    free = rng.permutation(pool)[:need + 7]
    for i, doc in enumerate((4096, 16, 0, 1008)):
        if doc == 0 and not key_positions and new_hi > 8000:
            continue  # a document whose offsets leave their field: refused, see below
        compare(p, new, used, pos, start, free, words, int(new.sum()) + room, first=[0, 5, 7, 0][i], doc=doc, local=i != 2, inplace=i == 3)


# a few long sequences among many short ones, a warp's and the grid's
@pytest.mark.parametrize("batch,long", [(300, 3000), (300, 900), (2100, 40000), (260, 9), (1500, 1025)])
def test_long_among_short(batch, long):
    rng = np.random.default_rng(batch + long)
    new, used, pos, start = requests(rng, batch, 3, 100, 40)
    new[[1, batch // 2, batch - 1]] = long, long // 2, long - 1
    need = int(sum(-(-(q - a + n) // 16) - -(-(q - a) // 16) for n, q, a in zip(new, pos, start)))
    wide = int(max(-(-u // 16) + -(-n // 16) + 1 for u, n in zip(used, new)))
    p = params(batch, wide, need + 50)
    words = (rng.integers(0, 1 << 14, (batch, wide)) << 18 | rng.integers(0, need + 50, (batch, wide))).astype(np.uint32)
    rows = int(new.sum())
    free = rng.permutation(need + 50)[:need + 3]
    for cut in (rows + 100, rows, rows - 5):
        compare(p, new, used, pos, start, free, words, cut, doc=1024)


def test_sequences_that_do_not_fit():
    L = la()
    rng = np.random.default_rng(9)
    for batch, few in ((12, True), (40, False), (1500, False)):
        new, used, pos, start = requests(rng, batch, 60 if few else 700, 400, 90)
        new[1::5] = 0
        wide = int(max(-(-u // 16) + -(-n // 16) + 1 for u, n in zip(used, new)))
        pool = 100000
        p = params(batch, wide, pool)
        words = rng.integers(0, pool, (batch, wide)).astype(np.uint32)
        free = rng.permutation(pool)[:200000 // 16]
        need = int(sum(-(-(q - a + n) // 16) - -(-(q - a) // 16) for n, q, a in zip(new, pos, start)))
        rows = int(new.sum())
        free = free[:need]
        for cut in (0, 1, need // 2, need - 1):  # the list ends
            want = compare(p, new, used, pos, start, free[:cut], words, rows)
            assert want[-1] == A.NO_BLOCKS
        for cut in (0, 1, rows // 2, rows - 1):  # the rows end
            want = compare(p, new, used, pos, start, free, words, cut)
            # (the largest batch's list is shorter than its need too)
            assert want[-1] & A.BAD_LEN and not want[-1] & ~(A.BAD_LEN | (A.NO_BLOCKS if len(free) < need else 0))
        for first in (-1, need + 1):
            assert compare(p, new, used, pos, start, free, words, rows, first=first)[-1] & A.LAYOUT
        bad = [x.copy() for x in (new, used, pos, start)]  # of everything something: the others go on
        bad[0][2], bad[1][4], bad[1][5], bad[3][7], bad[2][8] = -3, -1, 16 * wide + 1, bad[2][7] + 1, -5
        bad[1][9] = bad[1][9] // 16 * 16 + (bad[2][9] - bad[3][9] + 3) % 16
        assert compare(p, *bad, free, words, rows + 5)[-1] & (A.LAYOUT | A.BAD_LEN) == A.LAYOUT | A.BAD_LEN
        narrow = params(batch, max(1, wide // 2), pool)  # the table ends
        compare(narrow, new, used, pos, start, free, words[:, :max(1, wide // 2)], rows)
    # offsets that leave their field, and the same as documents that do not
    p = params(2, 1000, 2000)
    words = np.zeros((2, 1000), np.uint32)
    free = rng.permutation(2000)[:1100]
    for doc, ok in ((0, False), (8192, True), (8208, False), (4096, True)):
        want = compare(p, [9000, 3], [0, 0], [0, 0], [0, 0], free, words, 9003, doc=doc)
        assert (want[-1] == 0) == ok and want[1][1] == 3
    want = compare(p, [100, 3], [16, 16], [100000, 100000], [100000, 100000], free, words, 103)  # a start far from its block
    assert want[-1] == A.LAYOUT
    # ids outside the pool
    free[[0, 3]] = [2000, -4]
    assert compare(p, [40, 33], [0, 0], [0, 0], [0, 0], free, words, 73)[-1] == A.BAD_ID
    assert L.device_status(clear=True) == 0


@pytest.mark.parametrize("batch,rows", [(6, 20), (6, 2000), (300, 20)])
def test_rows_whose_sum_leaves_32_bits(batch, rows):
    # one CTA's rows, a thread a row, more sequences than one CTA writes the rows of
    L = la()
    top = 2 ** 31 - 1
    new = np.zeros(batch, np.int64)
    new[:6] = [3, top, top, top, 5, 0]
    p = params(batch, 4, 600)
    buf = torch.full((2, rows + 64), -5, dtype=torch.int32, device="cuda")
    out = L.AppendTables.empty(p, rows).replace(slots=buf[0, 32:32 + rows], local_pos=buf[1, 32:32 + rows])
    zero, words = i32([0] * batch), u32(np.zeros((batch, 4), np.uint32))
    L.append_tokens(p, i32(new), zero, zero, zero, i32(np.arange(600)), words, out=out)
    assert L.device_status(clear=True) == L.LAZY_DEV_LAYOUT | L.LAZY_DEV_BAD_LEN
    assert (buf[:, :32] == -5).all() and (buf[:, 32 + rows:] == -5).all()
    assert out.slots[:3].tolist() == [0, 1, 2] and (out.slots[3:] == -1).all()
    assert out.local_pos[:3].tolist() == [0, 1, 2] and not out.local_pos[3:].any()
    cu = np.minimum(np.cumsum([0, *new]), top)
    assert out.cu_rows.tolist() == cu.tolist() and out.seq_lens.tolist() == [3] + [0] * (batch - 1)


def test_unaligned_outputs_and_side_stream():
    L = la()
    rng = np.random.default_rng(4)
    new, used, pos, start = requests(rng, 20, 900, 100, 30)
    wide = 80
    p = params(20, wide, 5000)
    words = rng.integers(0, 5000, (20, wide)).astype(np.uint32)
    free = rng.permutation(5000)[:2000]
    rows = int(new.sum()) + 2
    want = A.append(new, used, pos, start, free, words, rows, max_blocks=wide, id_bits=18, pool=5000)
    w, ins = u32(words), [i32(x) for x in (new, used, pos, start)]
    fr = i32(free)
    big = [torch.full((rows + 8,), -5, dtype=torch.int32, device="cuda") for _ in range(2)]
    out = L.AppendTables.empty(p, rows).replace(slots=big[0][1:rows + 1], local_pos=big[1][3:rows + 3])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    L.append_tokens(p, *ins, fr, w, out=out, stream=s)
    s.synchronize()
    assert np.array_equal(out.slots.cpu().numpy(), want[6]) and np.array_equal(out.local_pos.cpu().numpy(), want[7])
    for x, a, b in ((big[0], 1, rows + 1), (big[1], 3, rows + 3)):  # nothing beside them
        assert (x[:a] == -5).all() and (x[b:] == -5).all()
    assert np.array_equal(w.cpu().numpy(), want[0].view(np.int32))


# ---------------------------------------------------------------- the calls together

THETA = 1e4


def rotate(x, n):
    d = x.shape[-1]
    f = torch.as_tensor(THETA ** (-2.0 * np.arange(d // 2) / d), dtype=torch.float64, device=x.device)
    c, s = torch.cos(n[:, None, None] * f), torch.sin(n[:, None, None] * f)
    a, b = x[..., :d // 2], x[..., d // 2:]
    return torch.cat((a * c - b * s, a * s + b * c), -1)


class Server:
    """A few sequences that share a cached document: prompts of their own, then decoded tokens, in a captured step."""

    def __init__(self, kv, batch, d, cap, wide, doc=64):
        L = self.L = la()
        self.kv, self.batch, self.d, self.doc, self.hq, self.hkv = kv, batch, d, doc, 8, 2
        self.p = L.make_params(num_seqs=batch, num_q_heads=8, num_kv_heads=2, head_dim=d, num_pool_blocks=400, max_blocks_per_seq=wide,
                               kv_dtype=kv, rope_theta=THETA)
        self.pools = L.empty_pools(self.p)
        for x in self.pools:
            x.view(torch.uint8).fill_(0x7F)  # NaN wherever nothing is written
        self.rope = L.rope_table_init(self.p)
        self.words = torch.zeros(batch, wide, dtype=torch.int32, device="cuda")
        self.lens, self.pos, self.start = (torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(3))
        self.free = i32(np.random.default_rng(1).permutation(400)[:350])
        self.out = L.AppendTables.empty(self.p, cap).replace(seq_lens=self.lens, pos=self.pos)
        self.out.block_indptr.zero_()
        self.new = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.k, self.v = (torch.zeros(cap, 2, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.keys = [[] for _ in range(batch)]  # what was written, unrotated K and V, in fp64

    def rows(self, new, g):
        """Rows of K (raw) and V for new tokens, K rotated at its document-local positions as a model would."""
        total = int(sum(new))
        kr, vr = (torch.randn(total, 2, self.d, generator=g, device="cuda", dtype=torch.float64) for _ in range(2))
        at = 0
        local = []
        for s, n in enumerate(new):
            have = sum(len(x[0]) for x in self.keys[s])
            local.append(torch.arange(have, have + n, device="cuda") % self.doc)
            self.keys[s].append((kr[at:at + n], vr[at:at + n]))
            at += n
        self.k[:total] = rotate(kr, torch.cat(local).double()).to(torch.bfloat16)
        self.v[:total] = vr.to(torch.bfloat16)
        return torch.cat(local)

    def step(self):
        L = self.L
        L.append_tokens(self.p, self.new, self.lens, self.pos, self.start, self.free, self.words, first_free=self.out.block_indptr[-1:],
                        doc_tokens=self.doc, out=self.out)
        L.cache_write(self.p, self.k, self.v, self.out.slots, *self.pools)

    def attend(self, q, out=None, ws=None):
        return self.L.decode(self.p, q, *self.pools, self.words, self.lens, self.pos, self.rope, out=out, workspace=ws)

    def reference(self, q):
        """64-bit attention from the raw rows at their absolute positions."""
        want = torch.zeros(self.batch, 8, self.d, dtype=torch.float64, device="cuda")
        for s in range(self.batch):
            if not sum(len(x[0]) for x in self.keys[s]):
                continue
            k, v = (torch.cat([x[i] for x in self.keys[s]]) for i in (0, 1))
            k = rotate(k, torch.arange(len(k), device="cuda").double())
            qs = rotate(q[s].double()[None], torch.tensor([float(len(k))], device="cuda", dtype=torch.float64))[0].view(2, 4, self.d)
            wgt = torch.softmax(torch.einsum("hgd,thd->hgt", qs, k) * self.d ** -0.5, -1)
            want[s] = torch.einsum("hgt,thd->hgd", wgt, v).reshape(8, self.d)
        return want


# Tolerance against raw rows: e4m3 codes are off by 2^-4 of a value (bf16 by 2^-8), K and V alike; over the about 100 keys of
# a context with normal rows the weighted sum of V's errors and the change of weights by K's (a score is off by at most 2^-4 |q| |k|
# / sqrt(d) in the worst case, normal with 2^-4 / sqrt(3) in the mean) stay below a tenth; bounds of 0.35 and 0.05 leave
# three times that, while a wrong slot, position or block gives errors near 1.
@pytest.mark.parametrize("kv,tol", [("fp8_e4m3_block", 0.35), (None, 0.05)])
@pytest.mark.parametrize("d", [64, 128])
def test_prompts_then_captured_decode_steps(kv, tol, d):
    batch, cap = 5, 300
    srv = Server(kv, batch, d, cap, 60)
    g = torch.Generator("cuda").manual_seed(7)
    prompt = [100, 1, 64, 16, 0]
    srv.new.copy_(i32(prompt))
    local = srv.rows(prompt, g)
    srv.step()
    assert torch.equal(srv.out.local_pos[:181].long(), local) and (srv.out.slots[181:] == -1).all()
    q = torch.randn(batch, 8, d, generator=g, device="cuda").to(torch.bfloat16)
    got = srv.attend(q).double()
    err = (got - srv.reference(q)).abs()
    assert err.max() < tol and not got[4].any()
    # the step captured once, replayed with 0 to 3 new tokens a sequence: blocks fill, documents end, tables grow
    q_in, out = q.clone(), torch.empty_like(q)
    ws = torch.empty(max(256, srv.L.decode_workspace_bytes(srv.p)), dtype=torch.uint8, device="cuda")
    srv.new.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        srv.step()
        srv.attend(q_in, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        srv.step()
        srv.attend(q_in, out, ws)
    for i in range(40):
        new = [(i + s) % 4 if s < 4 else 1 for s in range(batch)]
        srv.new.copy_(i32(new))
        srv.rows(new, g)
        q_in.copy_(torch.randn(batch, 8, d, generator=g, device="cuda").to(torch.bfloat16))
        graph.replay()
        err = (out.double() - srv.reference(q_in)).abs()
        assert err.max() < tol, (i, err.max())
    taken = int(srv.out.block_indptr[-1])
    lens = [sum(len(x[0]) for x in k) for k in srv.keys]
    assert taken == sum(-(-n // 16) for n in lens) and srv.pos.tolist() == lens
    # the shared-run decode over the same tables, every sequence's blocks as one run of its documents
    docs = [min(srv.doc, n - a) for n in lens for a in range(0, n, srv.doc)]
    if kv is not None:
        ids = srv.words.cpu().numpy().view(np.uint32) & ((1 << 18) - 1)
        blocks = np.concatenate([ids[s, :-(-n // 16)] for s, n in enumerate(lens)])
        indptr = np.cumsum([0] + [-(-n // 16) for n in docs])
        seg = np.cumsum([0] + [-(-n // srv.doc) for n in lens])
        items, slot_indptr = srv.L.plan_shared_host(srv.p, len(docs), seg, np.arange(len(docs)), docs, indptr, blocks)
        two = srv.L.decode_shared(srv.p, q_in, *srv.pools, srv.words, srv.pos, srv.rope, srv.L.SharedPlan(items, slot_indptr))
        assert (two.double() - srv.reference(q_in)).abs().max() < tol
    # staged in bf16
    if kv is not None and d == 128:
        L = srv.L
        every = torch.arange(400, dtype=torch.int32, device="cuda")
        k16, v16 = L.cache_read(srv.p, *srv.pools, every)
        srv.p.kv_dtype = 0
        staged = L.decode(srv.p, q_in, k16, v16, srv.words, srv.lens, srv.pos, srv.rope)
        assert (staged.double() - srv.reference(q_in)).abs().max() < tol


def test_prefill_chunk_behind_cached_tokens():
    """A chunk as a document of its own: append_tokens gives the prefill its tables, over a staged pool."""
    L = la()
    srv = Server("fp8_e4m3_block", 3, 128, 200, 40, doc=0)
    srv.doc = 10 ** 6
    g = torch.Generator("cuda").manual_seed(8)
    first = [50, 3, 20]
    srv.new.copy_(i32(first))
    srv.rows(first, g)
    L.append_tokens(srv.p, srv.new, srv.lens, srv.pos, srv.start, srv.free, srv.words, first_free=srv.out.block_indptr[-1:], doc_tokens=0,
                    out=srv.out)
    L.cache_write(srv.p, srv.k, srv.v, srv.out.slots, *srv.pools)
    chunk = [17, 40, 1]
    srv.new.copy_(i32(chunk))
    srv.start.copy_(srv.pos)  # the chunk begins a document
    total = sum(chunk)
    kr, vr = (torch.randn(total, 2, 128, generator=g, device="cuda", dtype=torch.float64) for _ in range(2))
    local = torch.cat([torch.arange(n, device="cuda") for n in chunk])
    srv.k[:total], srv.v[:total] = rotate(kr, local.double()).to(torch.bfloat16), vr.to(torch.bfloat16)
    L.append_tokens(srv.p, srv.new, srv.lens, srv.pos, srv.start, srv.free, srv.words, first_free=srv.out.block_indptr[-1:], doc_tokens=0,
                    out=srv.out)
    L.cache_write(srv.p, srv.k, srv.v, srv.out.slots, *srv.pools)
    assert torch.equal(srv.out.local_pos[:total].long(), local) and srv.out.cu_rows.tolist() == np.cumsum([0] + chunk).tolist()
    every = torch.arange(400, dtype=torch.int32, device="cuda")
    k16, v16 = L.cache_read(srv.p, *srv.pools, every)
    q = torch.randn(total, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
    srv.p.kv_dtype = 0
    out = L.prefill(srv.p, q, srv.out.cu_rows, srv.out.q_start, max(chunk), k16, v16, srv.words, srv.lens, srv.rope)
    at = 0
    for s, n in enumerate(chunk):
        k0, v0 = (torch.cat([x[i] for x in srv.keys[s]]) for i in (0, 1))
        k = rotate(torch.cat((k0, kr[at:at + n])), torch.arange(first[s] + n, device="cuda").double())
        v = torch.cat((v0, vr[at:at + n]))
        qs = rotate(q[at:at + n].double(), torch.arange(first[s], first[s] + n, device="cuda").double()).view(n, 2, 4, 128)
        score = torch.einsum("nhgd,thd->nhgt", qs, k) * 128 ** -0.5
        hide = torch.arange(first[s] + n, device="cuda")[None] > torch.arange(first[s], first[s] + n, device="cuda")[:, None]
        wgt = torch.softmax(score.masked_fill(hide[:, None, None], -np.inf), -1)
        want = torch.einsum("nhgt,thd->nhgd", wgt, v).reshape(n, 8, 128)
        assert (out[at:at + n].double() - want).abs().max() < 0.5  # few keys in the first rows: a value's own 2^-4, up to 4.5
        at += n
