"""Cases of a step over a KV cache held in 8 bits with a scale per block of tokens and head: block
tables and slots from request lengths, rows into the pools, and the decodes that attend over them.

Operators
  tables append_tokens makes room for each request's new tokens: block words, lengths, row offsets, cache slots and
         document-local positions, with blocks from a free list. A request's own tokens lie in documents of `doc` tokens
  write  cache_write quantises new K/V rows (a slice of a fused qkv product) into the slots of a paged pool, then
         cache_read returns the blocks that were touched
  decode one query per sequence over its block table
  shared the same attention for a batch whose sequences cite the same documents: each cited block is read once per
         KV head for all of them

Format of a (block, KV head) record of 16 tokens of d dims: 16 d bytes of e4m3 codes, then 32 bytes of which the first
four are the scale 2^e (fp32). A value is code * 2^e.
  K: 16-byte chunk 32 j + 4 g + t holds dims 16 (t + 4 (j // 2)) .. + 15 of token g + 8 (j % 2)
  V: with n = d / 64, chunk 32 j + 4 g + t holds, for the dims 8 (g + 8 (j % n)) .. + 7, the codes of
     tokens 2 (t + 4 (j // n)) and that + 1 side by side
Writing rows into a block: e is the least whole number with max |x| <= 448 * 2^e over the written rows' finite values,
and at least the block's old e unless token 0 is among the rows; -100 <= e <= 119. Codes are x / 2^e to the nearest
(ties to even); what is not finite becomes NaN. The block's other tokens keep their values, rounded to the new scale; where
token 0 was written the block begins anew and they are 0.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
ID_BITS = 18
THETA = 5e5
FP8_MAX = 448.0
E_MIN, E_MAX = -100, 119
KIND = "fp8_e4m3_block"


# --------------------------------------------------------------------------- cases

def listed():
    heads8b = dict(q_heads=32, kv_heads=8, dim=128)
    heads70b = dict(q_heads=64, kv_heads=8, dim=128)
    return [
        # a decode step of 64 running sequences: one token each behind 4096 tokens of documents and a private tail
        dict(name="tables step", op="tables", batch=64, new_lo=1, new_hi=1, ctx_lo=4096, ctx_hi=4096, tail_hi=64, room=0, doc=4096),
        # a step of a large server: decodes, drafts of a few tokens, idle requests, in arrays made for a captured step
        dict(name="tables drafts", op="tables", batch=1021, new_lo=0, new_hi=8, ctx_lo=0, ctx_hi=16384, tail_hi=500, room=2000, doc=1024),
        # whole tables of 48 requests of 256 to 131072 tokens
        dict(name="tables prompts", op="tables", batch=48, new_lo=256, new_hi=131072, ctx_lo=0, ctx_hi=0, tail_hi=0, room=0, doc=4096),
        # a decode step's rows: 64 sequences, one token each, into a block that holds earlier ones
        dict(name="write step", op="write", docs=64, doc_lo=1, doc_hi=1, append=True, padding=0.0, **heads8b),
        # documents of uneven lengths in a padded batch, small heads
        dict(name="write ragged d64", op="write", docs=37, doc_lo=1, doc_hi=211, append=True, padding=0.1, q_heads=4, kv_heads=2, dim=64),
        # ingestion of sixteen 1024-token documents
        dict(name="write documents", op="write", docs=16, doc_lo=1024, doc_hi=1024, append=False, padding=0.0, **heads70b),
        # the smallest decode: one sequence of 96 tokens
        dict(name="decode tiny", op="decode", batch=1, ctx_lo=96, ctx_hi=96, doc_lo=16, doc_hi=48, tail=0, pool_docs=0, zipf=0.0,
             q_heads=4, kv_heads=2, dim=64),
        # a batch of 64 sequences of eight documents and a private tail
        dict(name="decode 8b", op="decode", batch=64, ctx_lo=4096, ctx_hi=4096, doc_lo=512, doc_hi=512, tail=64, pool_docs=0, zipf=0.0, **heads8b),
        # one long sequence alone: the work of few rows is split over its length
        dict(name="decode 70b single", op="decode", batch=1, ctx_lo=16384, ctx_hi=16384, doc_lo=1024, doc_hi=1024, tail=0, pool_docs=0, zipf=0.0, **heads70b),
        # contexts from short to 128 k tokens in one batch, documents of uneven lengths, one KV head for 32 query heads
        dict(name="decode mqa ragged", op="decode", batch=48, ctx_lo=256, ctx_hi=131072, doc_lo=64, doc_hi=4096, tail=0, pool_docs=0, zipf=0.0,
             q_heads=32, kv_heads=1, dim=128),
        # the batch of 64 with documents drawn by Zipf's law from 256
        dict(name="shared 8b", op="shared", batch=64, ctx_lo=4096, ctx_hi=4096, doc_lo=512, doc_hi=512, tail=64, pool_docs=256, zipf=1.0, **heads8b),
        # 32 sequences of sixteen 1024-token documents, drawn from 512, 8 query heads a KV head
        dict(name="shared 70b", op="shared", batch=32, ctx_lo=16384, ctx_hi=16384, doc_lo=1024, doc_hi=1024, tail=0, pool_docs=512, zipf=1.0, **heads70b),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "write", "decode", "decode", "shared"])
    if op == "tables":
        batch = _log(rng, 1, 4096)
        hi = _log(rng, 1, max(2, min(131072, 2500000 // batch)))
        ctx = rng.choice([0, _log(rng, 1, 65536)])
        return dict(op=op, batch=batch, new_lo=rng.choice([0, 1, hi // 3, hi]), new_hi=hi, ctx_lo=ctx // 3, ctx_hi=ctx,
                    tail_hi=rng.choice([0, _log(rng, 1, 1000)]), room=rng.choice([0, _log(rng, 1, 5000)]),
                    doc=rng.choice([16, 512, 1024, 4096]))
    kv_heads, group, dim = rng.choice([(8, 4, 128), (8, 8, 128), (1, 32, 128), (2, 2, 64), (8, 1, 128), (4, 7, 128), (1, 64, 128),
                                       (5, 3, 64), (2, 16, 64)])
    heads = dict(q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim)
    if op == "write":
        hi = _log(rng, 1, 1024)
        docs = max(1, min(256, _log(rng, 1, 16384) // hi))
        return dict(op=op, docs=docs, doc_lo=max(1, hi // rng.choice([1, 3, 10])), doc_hi=hi, append=rng.random() < 0.5,
                    padding=rng.choice([0.0, 0.0, 0.05, 0.2]), **heads)
    batch = _log(rng, 1, 96)
    # keys x heads of the largest listed batch bound the context
    top = min(131072, int(32 * 16384 * 8 * 64 / (batch * max(8, heads["q_heads"]) * kv_heads)))
    hi = _log(rng, 1, max(2, top))
    doc_hi = max(1, _log(rng, max(1, hi // 40), hi))
    case = dict(op=op, batch=batch, ctx_lo=max(1, hi // rng.choice([1, 2, 20])), ctx_hi=hi, doc_lo=max(1, doc_hi // rng.choice([1, 2, 8])),
                doc_hi=doc_hi, tail=rng.choice([0, 1, rng.randrange(2, 200)]), pool_docs=0, zipf=0.0, **heads)
    if op == "shared":
        case.update(pool_docs=_log(rng, 1, 512), zipf=round(rng.uniform(0.5, 1.3), 2))
    return case


# --------------------------------------------------------------------------- layout: the same for every seed

def _rng_of(case):
    return random.Random("layout " + " ".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))


def _blocks(tokens):
    return -(-tokens // BLOCK)


def _requests(case):
    """Per request its new tokens, the slots that its documents fill, its position and where its own last document starts."""
    rng = _rng_of(case)
    out = []
    for _ in range(case["batch"]):
        n, ctx, tail = rng.randint(case["new_lo"], case["new_hi"]), rng.randint(case["ctx_lo"], case["ctx_hi"]), rng.randint(0, case["tail_hi"])
        holes = rng.randrange(BLOCK) if ctx else 0  # documents end inside blocks
        full = BLOCK * _blocks(ctx + holes)
        out.append((n, full + tail if tail else ctx + holes, ctx + tail, ctx))
    return out


def _segments(case):
    """Per sequence its (document, tokens used), and every document's length."""
    rng = _rng_of(case)
    doc_len, seqs = [], []
    n = case["pool_docs"]
    if n:
        doc_len = [rng.randint(case["doc_lo"], case["doc_hi"]) for _ in range(n)]
        weights = [(r + 1) ** -case["zipf"] for r in range(n)]
    for _ in range(case["batch"]):
        left, segs = rng.randint(case["ctx_lo"], case["ctx_hi"]), []
        while left > 0:
            if n:
                doc = rng.choices(range(n), weights)[0]
            else:
                doc = len(doc_len)
                doc_len.append(rng.randint(case["doc_lo"], case["doc_hi"]))
            segs.append((doc, min(left, doc_len[doc])))
            left -= segs[-1][1]
        if case["tail"]:
            segs.append((len(doc_len), case["tail"]))
            doc_len.append(case["tail"])
        seqs.append(segs)
    return seqs, doc_len


def _used_blocks(seqs):
    """(blocks that some sequence reads, block table entries of all of them, tokens of all of them)."""
    used = {}
    for segs in seqs:
        for doc, n in segs:
            used[doc] = max(used.get(doc, 0), _blocks(n))
    return sum(used.values()), sum(_blocks(n) for s in seqs for _, n in s), sum(n for s in seqs for _, n in s)


def _documents(case):
    """Lengths of the written documents, the first slot of each in its first block, and which rows are padding."""
    rng = _rng_of(case)
    lens = [rng.randint(case["doc_lo"], case["doc_hi"]) for _ in range(case["docs"])]
    first = [rng.randrange(BLOCK) if case["append"] else 0 for _ in lens]
    skip = [rng.random() < case["padding"] for _ in range(sum(lens))]
    return lens, first, skip


def _record(dim):
    return BLOCK * dim + 32


def work(case):
    if case["op"] == "tables":
        reqs = _requests(case)
        rows = sum(r[0] for r in reqs) + case["room"]
        new = sum(_blocks(m - a + n) - _blocks(m - a) for n, _, m, a in reqs)
        # in: four numbers a request, an id a block; out: slots and positions of the rows, words, five numbers a request
        return {"bytes": 4 * (4 * len(reqs) + 2 * new + 2 * rows + 5 * len(reqs)), "flops": 4.0 * rows}
    hkv, dim = case["kv_heads"], case["dim"]
    stored = BLOCK * dim + 4
    if case["op"] == "write":
        lens, first, skip = _documents(case)
        blocks = sum(_blocks(f + n) for f, n in zip(first, lens))
        rows = len(skip) - sum(skip)
        return {"bytes": rows * 2 * hkv * 3 * dim + 4 * len(skip) + blocks * (2 * hkv * (4 + stored + 2 * BLOCK * dim) + 4),
                "flops": 3.0 * rows * 2 * hkv * dim + 1.0 * blocks * 2 * hkv * BLOCK * dim}
    unique, table, tokens = _used_blocks(_segments(case)[0])
    io = case["batch"] * case["q_heads"] * dim * 2 * 2
    return {"bytes": unique * 2 * hkv * stored + 4 * table + io + 8 * case["batch"], "flops": 4.0 * tokens * case["q_heads"] * dim}


# --------------------------------------------------------------------------- the format in plain torch

def _order(dim, is_v, device):
    """[16, d]: where a token's dim lies among a record's codes."""
    r, e = torch.arange(BLOCK, device=device)[:, None], torch.arange(dim, device=device)[None]
    if is_v:
        pair, group = r // 2, e // 8
        return 16 * (32 * (group // 8 + dim // 64 * (pair // 4)) + 4 * (group % 8) + pair % 4) + 2 * (e % 8) + r % 2
    chunk = e // 16
    return 16 * (32 * (r // 8 + 2 * (chunk // 4)) + 4 * (r % 8) + chunk % 4) + e % 16


def _parts(pool, dim):
    """Views of a pool [blocks, heads, record]: codes [.., 16 d] and scales [..]."""
    return pool[..., :BLOCK * dim], pool[..., BLOCK * dim:].view(torch.float32)[..., 0]


def _pow2(e):
    """2^e in 32 bits, -126 <= e <= 127."""
    return (e.int() + 127 << 23).view(torch.float32)


def _exponent(most):
    """The least e with most <= 448 * 2^e = 0.875 * 2^(e + 9)."""
    part, e = torch.frexp(most)
    e = torch.where(part <= 0.875, e - 9, e - 8)
    return torch.where(most > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def _codes(x, e):
    """x / 2^e (exact in 32 bits) as e4m3 bytes; not finite: NaN."""
    y = x * _pow2(-e)
    return torch.where(x.isfinite(), y.clamp(-FP8_MAX, FP8_MAX), math.nan).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(pool, dim, is_v):
    """A pool's values [blocks, heads, 16, d] in 32 bits."""
    codes, scale = _parts(pool, dim)
    return codes[..., _order(dim, is_v, pool.device)].view(torch.float8_e4m3fn).float() * scale[..., None, None]


def _random_pool(gen, blocks, hkv, dim, is_v):
    """A pool of normal rows, quantised. A few channels of K are larger, and blocks differ in size, as in real caches."""
    pool = torch.zeros((blocks, hkv, _record(dim)), dtype=torch.uint8, device="cuda")
    gain = torch.ones(dim, device="cuda")
    if not is_v:
        gain[torch.randint(dim, (dim // 32,), generator=gen, device="cuda")] = 5.0
    back = torch.argsort(_order(dim, is_v, "cuda").flatten())  # code byte -> token and dim
    step = max(1, (1 << 26) // (hkv * BLOCK * dim))
    for at in range(0, blocks, step):
        part = pool[at:at + step]
        x = torch.randn((part.shape[0], hkv, BLOCK, dim), generator=gen, device="cuda") * gain
        x *= torch.exp2(torch.rand((part.shape[0], hkv, 1, 1), generator=gen, device="cuda") - 0.5)
        x = x.to(torch.bfloat16).float()
        e = _exponent(x.abs().amax((-1, -2)))
        codes, scale = _parts(part, dim)
        codes[...] = _codes(x, e[..., None, None]).flatten(-2)[..., back]
        scale[...] = _pow2(e)
    return pool


# --------------------------------------------------------------------------- prepare

def _params(case, module, **more):
    return module.make_params(num_q_heads=case["q_heads"], num_kv_heads=case["kv_heads"], head_dim=case["dim"], dtype="bf16", rope_theta=THETA,
                              id_bits=ID_BITS, **more)


def _int32(x):
    return torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()


def _prepare_tables(case, seed):
    shuffle = np.random.default_rng(seed)
    reqs = _requests(case)
    n, used, pos, start = (np.array(x) for x in zip(*reqs))
    need = int(sum(_blocks(m - a + k) - _blocks(m - a) for k, _, m, a in reqs))
    pool = need + need // 4 + 1000
    first = int(shuffle.integers(0, 40))  # blocks of the list that earlier steps took
    free = shuffle.permutation(pool)[:need + first + 17]
    rows = int(n.sum()) + case["room"]
    wide = int(max(_blocks(u) + _blocks(k) + 1 for k, u, _, _ in reqs))
    bits = max(ID_BITS, pool.bit_length())
    words = shuffle.integers(0, 1 << 32 - bits, (len(reqs), wide)) << bits | shuffle.integers(0, pool, (len(reqs), wide))  # of earlier steps
    s = dict(case=case, new_lens=_int32(n), seq_lens=_int32(used), pos=_int32(pos), start=_int32(start), free=_int32(free), first=_int32([first]),
             words=torch.from_numpy(words.astype(np.uint32).view(np.int32)).cuda(), rows=rows, bits=bits, pool=pool)
    if own:
        from paged_kv_cache_57_gb300 import lazy_attn
        p = lazy_attn.make_params(num_seqs=len(reqs), num_q_heads=32, num_kv_heads=8, head_dim=128, num_pool_blocks=pool, max_blocks_per_seq=wide,
                                  id_bits=bits)
        s.update(lib=lazy_attn, p=p, out=lazy_attn.AppendTables.empty(p, rows))
    return s


def _prepare_write(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    shuffle = np.random.default_rng(seed)
    lens, first, skip = _documents(case)
    spans = [_blocks(f + n) for f, n in zip(first, lens)]
    pool = sum(spans) + 16
    ids = shuffle.permutation(pool)[:sum(spans)]
    at = np.concatenate(([0], np.cumsum(spans)))
    place = np.concatenate([BLOCK * at[i] + first[i] + np.arange(n) for i, n in enumerate(lens)])
    slots = np.where(skip, -1, ids[place // BLOCK] * BLOCK + place % BLOCK)
    # K and V are slices of the layer's fused product, as the model leaves them
    qkv = torch.randn((len(slots), hq + 2 * hkv, dim), generator=gen, device="cuda").to(torch.bfloat16)
    qkv[:, hq:hq + hkv, :: max(1, dim // 4)] *= 5
    s = dict(case=case, k_pool=_random_pool(gen, pool, hkv, dim, False), v_pool=_random_pool(gen, pool, hkv, dim, True), ids=_int32(ids),
             k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], slots=_int32(slots))
    if own:
        from paged_kv_cache_57_gb300 import lazy_attn
        s.update(lib=lazy_attn, p=_params(case, lazy_attn, num_seqs=0, num_pool_blocks=pool, max_blocks_per_seq=0, kv_dtype=KIND))
    return s


def _prepare_attention(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    seqs, doc_len = _segments(case)
    cited = sorted({doc for segs in seqs for doc, _ in segs})
    spans = {doc: _blocks(doc_len[doc]) for doc in cited}
    pool = sum(spans.values())
    order = np.random.default_rng(seed).permutation(pool).astype(np.int32)  # blocks lie anywhere in the pool
    at, starts = {}, 0
    for doc in cited:
        at[doc] = starts
        starts += spans[doc]
    max_blocks = max(sum(_blocks(n) for _, n in segs) for segs in seqs)
    words = np.zeros((len(seqs), max_blocks), np.uint32)
    seq_lens, q_pos = np.zeros(len(seqs), np.int32), np.zeros(len(seqs), np.int32)
    for i, segs in enumerate(seqs):
        b = p = 0
        for doc, n in segs:
            nb = _blocks(n)
            off = BLOCK * (b + np.arange(nb)) - p
            words[i, b:b + nb] = ((off.astype(np.int64) << ID_BITS) & 0xFFFFFFFF).astype(np.uint32) | order[at[doc]:at[doc] + nb].astype(np.uint32)
            b, p, last = b + nb, p + n, n - BLOCK * (nb - 1)
        seq_lens[i], q_pos[i] = BLOCK * (b - 1) + last, p
    kp, vp = (_random_pool(gen, pool, hkv, dim, is_v) for is_v in (False, True))
    ends = [(order[at[doc] + spans[doc] - 1], doc_len[doc] % BLOCK) for doc in cited if doc_len[doc] % BLOCK]
    if ends:  # slots behind a document's end hold what nothing wrote: NaN
        blk = torch.tensor([int(b) for b, _ in ends], device="cuda")
        gone = torch.arange(BLOCK, device="cuda")[None] >= torch.tensor([n for _, n in ends], device="cuda")[:, None]
        for x, is_v in ((kp, False), (vp, True)):
            place = _order(dim, is_v, "cuda")
            token = torch.empty(BLOCK * dim, dtype=torch.long, device="cuda")
            token[place.flatten()] = torch.arange(BLOCK, device="cuda").repeat_interleave(dim)
            codes = _parts(x, dim)[0]
            codes[blk] = torch.where(gone[:, token][:, None], 0x7f, codes[blk])
    s = dict(case=case, k_pool=kp, v_pool=vp, q=torch.randn((len(seqs), hq, dim), generator=gen, device="cuda").to(torch.bfloat16),
             words=torch.from_numpy(words.view(np.int32)).cuda(), seq_lens=torch.from_numpy(seq_lens).cuda(), q_pos=torch.from_numpy(q_pos).cuda(),
             freqs=THETA ** (-2.0 * torch.arange(dim // 2, dtype=torch.float64, device="cuda") / dim))
    if own:
        from paged_kv_cache_57_gb300 import lazy_attn
        p = _params(case, lazy_attn, num_seqs=len(seqs), num_pool_blocks=pool, max_blocks_per_seq=max_blocks, kv_dtype=KIND)
        s.update(lib=lazy_attn, p=p, rope=lazy_attn.rope_table_init(p), out=torch.empty_like(s["q"]))
        if case["op"] == "decode":
            need = lazy_attn.decode_workspace_bytes(p)
        else:
            flat = [x for segs in seqs for x in segs]
            indptr = np.cumsum([0] + [spans.get(doc, 0) for doc in range(len(doc_len))])
            items, slots = lazy_attn.plan_shared_host(p, len(doc_len), np.cumsum([0] + [len(segs) for segs in seqs]), [d for d, _ in flat],
                                                      [n for _, n in flat], indptr, order)
            s["plan"] = lazy_attn.SharedPlan(items, slots)
            need = lazy_attn.decode_shared_workspace_bytes(p, s["plan"].num_slots)
        s["workspace"] = torch.empty(max(256, need), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    torch.backends.cuda.matmul.allow_tf32 = False
    return {"tables": _prepare_tables, "write": _prepare_write}.get(case["op"], _prepare_attention)(case, seed)


# --------------------------------------------------------------------------- run

def _tables_plain(s):
    n, used, pos, start = s["new_lens"], s["seq_lens"], s["pos"], s["start"]
    zero = n.new_zeros(1)
    up = lambda x: (x + BLOCK - 1) // BLOCK
    tail = pos - start
    b0 = up(used) - up(tail)
    take = up(tail + n) - up(tail)
    cu = torch.cat((zero, n.cumsum(0).int()))
    indptr = s["first"] + torch.cat((zero, take.cumsum(0).int()))
    row = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    live = row < cu[-1]
    seq = torch.searchsorted(cu[1:], row, right=True).clamp(max=len(n) - 1)
    local = row - cu[seq] + tail[seq]
    block = b0[seq] + local // BLOCK
    fresh = live & (local % BLOCK == 0)
    got = s["free"][(indptr[seq] + local // BLOCK - up(tail)[seq]).clamp(0, len(s["free"]) - 1).long()]
    doc = s["case"]["doc"]
    word = (BLOCK * block - start[seq] - local // doc * doc) << s["bits"] | got
    at = (seq * s["words"].shape[1] + block)[fresh]
    s["words"].view(-1)[at] = word[fresh]
    phys = s["words"][seq, block.clamp(max=s["words"].shape[1] - 1).long()] & ((1 << s["bits"]) - 1)
    slots = torch.where(live, phys * BLOCK + local % BLOCK, -1)
    grown = torch.where(n > 0, BLOCK * b0 + tail + n, used)
    return s["words"], grown, pos + n, pos, cu, indptr, slots, torch.where(live, local % doc, 0)


def _write_plain(s):
    dim = s["case"]["dim"]
    keep = (s["slots"] >= 0).nonzero()[:, 0]
    block, row = s["slots"][keep].long() // BLOCK, s["slots"][keep].long() % BLOCK
    touched, where = torch.unique(block, return_inverse=True)
    written = torch.zeros((len(touched), BLOCK), dtype=torch.bool, device="cuda")
    written[where, row] = True
    anew = written[:, :1, None, None]  # begun with this call
    for x, pool, is_v in ((s["k"], s["k_pool"], False), (s["v"], s["v_pool"], True)):
        part = pool[touched]
        rows = torch.where(anew, 0.0, _values(part, dim, is_v).transpose(1, 2))  # [n, 16, heads, d]
        rows[where, row] = x[keep].float()
        fresh = torch.where(written[..., None, None] & rows.isfinite(), rows.abs(), 0.0)
        e = _exponent(fresh.amax((1, 3)))
        old = torch.where(anew[:, 0, 0], E_MIN, torch.frexp(_parts(part, dim)[1]).exponent - 1)
        e = torch.maximum(e, old)
        codes, scale = _parts(part, dim)
        codes[..., _order(dim, is_v, "cuda")] = _codes(rows, e[:, None, :, None]).transpose(1, 2)
        scale[...] = _pow2(e)
        pool[touched] = part


def _read_plain(s):
    ids = s["ids"].long()
    return tuple(_values(pool[ids], s["case"]["dim"], is_v).to(torch.bfloat16) for pool, is_v in ((s["k_pool"], False), (s["v_pool"], True)))


def _attend_plain(s):
    case, hkv, dim = s["case"], s["case"]["kv_heads"], s["case"]["dim"]
    words, batch = s["words"], s["words"].shape[0]
    nb = words.shape[1]
    b = torch.arange(nb, device="cuda")
    phys = (words & ((1 << ID_BITS) - 1)).long()
    start = BLOCK * b - (words >> ID_BITS)  # position of the block's document
    count = (s["seq_lens"][:, None] + BLOCK - 1) // BLOCK
    after = torch.cat((start[:, 1:], start[:, -1:]), 1)
    valid = torch.where(after != start, ((after - start - 1) & 15) + 1, BLOCK)
    valid = torch.where(b == count - 1, s["seq_lens"][:, None] - BLOCK * (count - 1), valid)
    live = (torch.arange(BLOCK, device="cuda") < valid[..., None]) & (b < count)[..., None]  # [B, n, 16]
    k, v = (torch.where(live[:, :, None, :, None], _values(pool, dim, is_v)[phys], 0.0) for pool, is_v in ((s["k_pool"], False), (s["v_pool"], True)))
    angle = (s["q_pos"][:, None] - start)[..., None].double() * s["freqs"]  # in 64 bits: far positions
    cos, sin = (f(angle).float()[:, :, None] for f in (torch.cos, torch.sin))  # [B, n, 1, d / 2]
    x, y = s["q"].float()[:, None].chunk(2, -1)
    q = torch.cat((x * cos - y * sin, y * cos + x * sin), -1).unflatten(2, (hkv, -1))  # [B, n, h, g, d]
    score = (q @ k.transpose(-1, -2)) * dim ** -0.5  # [B, n, h, g, 16]
    score = score.masked_fill(~live[:, :, None, None], -math.inf).permute(0, 2, 3, 1, 4).flatten(-2)
    p = (score - score.amax(-1, keepdim=True)).exp()
    out = (p / p.sum(-1, keepdim=True)) @ v.permute(0, 2, 1, 3, 4).flatten(2, 3)
    return out.reshape(batch, case["q_heads"], dim).to(torch.bfloat16)


def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "tables":
            return _tables_plain(s)
        if op == "write":
            _write_plain(s)
            return _read_plain(s)
        return _attend_plain(s)
    lib, p = s["lib"], s["p"]
    if op == "tables":
        t = lib.append_tokens(p, s["new_lens"], s["seq_lens"], s["pos"], s["start"], s["free"], s["words"], first_free=s["first"],
                              doc_tokens=s["case"]["doc"], out=s["out"])
        return s["words"], t.seq_lens, t.pos, t.q_start, t.cu_rows, t.block_indptr, t.slots, t.local_pos
    if op == "write":
        lib.cache_write(p, s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"])
        return lib.cache_read(p, s["k_pool"], s["v_pool"], s["ids"])
    if op == "decode":
        return lib.decode(p, s["q"], s["k_pool"], s["v_pool"], s["words"], s["seq_lens"], s["q_pos"], s["rope"], out=s["out"], workspace=s["workspace"])
    return lib.decode_shared(p, s["q"], s["k_pool"], s["v_pool"], s["words"], s["q_pos"], s["rope"], s["plan"], out=s["out"], workspace=s["workspace"])


# --------------------------------------------------------------------------- exact: from the definition, in 64 bits

def _exact_tables(case, seed):
    """Request by request on the host, with the bits as whole numbers."""
    s = _prepare_tables(case, seed)
    host = {k: s[k].cpu().numpy().astype(np.int64) for k in ("free", "first", "words")}
    words, free, at, bits = host["words"], host["free"], int(host["first"][0]), s["bits"]
    rows = s["rows"]
    slots, local = np.full(rows, -1, np.int64), np.zeros(rows, np.int64)
    out = dict(used=[], pos=[], start=[], cu=[0], indptr=[at])
    for i, (n, used, pos, start) in enumerate(_requests(case)):
        tail = pos - start
        blocks = _blocks(used)  # entries of the table in use
        first = blocks - _blocks(tail)
        r = out["cu"][-1]
        token = tail + np.arange(n)
        more = _blocks(tail + n) - _blocks(tail)
        for j in range(more):
            begin = start + (_blocks(tail) + j) * BLOCK // case["doc"] * case["doc"]  # of the document that the block lies in
            word = ((BLOCK * (blocks + j) - begin) * 2 ** bits + int(free[at + j])) % 2 ** 32
            words[i, blocks + j] = word - 2 ** 32 if word >= 2 ** 31 else word
        slots[r:r + n] = words[i, first + token // BLOCK] % 2 ** bits * BLOCK + token % BLOCK
        local[r:r + n] = token % case["doc"]
        at += more
        out["cu"].append(r + n)
        out["indptr"].append(at)
        out["used"].append(BLOCK * first + tail + n if n else used)
        out["pos"].append(pos + n)
        out["start"].append(pos)
    return tuple(_int32(x) for x in (words, out["used"], out["pos"], out["start"], out["cu"], out["indptr"], slots, local))


def _two_to(n):
    """2^n in 64 bits by its bits (a library's power may be off in the last place, which makes ties of what is none)."""
    return (n.long() + 1023 << 52).view(torch.float64)


def _one_value(pool, dim, is_v):
    """Values [.., 16, d] of records in 64 bits, chunk by chunk: the codes' bits by their definition."""
    c = torch.arange(dim, device=pool.device)  # 16-byte chunks of a record
    j, g, t, byte = c // 32, c % 32 // 4, c % 4, torch.arange(16, device=pool.device)
    if is_v:
        token = 2 * (t + 4 * (j // (dim // 64)))[:, None] + byte % 2
        e = 8 * (g + 8 * (j % (dim // 64)))[:, None] + byte // 2
    else:
        token = (g + 8 * (j % 2))[:, None].expand(-1, 16)
        e = 16 * (t + 4 * (j // 2))[:, None] + byte
    code = pool[..., :BLOCK * dim].long()
    power, part = code // 8 % 16, code % 8
    value = torch.where(power > 0, (8 + part).double() * _two_to(power - 10), part.double() / 512)
    value = torch.where(code % 128 == 127, math.nan, torch.where(code > 127, -value, value))
    tail = [pool[..., BLOCK * dim + i].int() << 8 * i for i in range(4)]
    value = value * (tail[0] | tail[1] | tail[2] | tail[3]).view(torch.float32).double()[..., None]
    out = torch.empty_like(value)
    out[..., (token * dim + e).flatten()] = value
    return out.unflatten(-1, (BLOCK, dim))


def _exact_write(case, seed):
    s = _prepare_write(case, seed)
    dim, ids, out = case["dim"], s["ids"].long(), []
    where = torch.full((s["k_pool"].shape[0],), -1, device="cuda")
    where[ids] = torch.arange(len(ids), device="cuda")
    keep = s["slots"] >= 0
    slot = s["slots"][keep].long()
    at, row = where[slot // BLOCK], slot % BLOCK
    for name, is_v in (("k", False), ("v", True)):
        part = s[name + "_pool"][ids]
        got = _one_value(part, dim, is_v)
        bits = sum(part[..., BLOCK * dim + i].double() * 256.0 ** i for i in range(4))
        old = (bits / 2 ** 23).floor().long() - 127  # a power of two
        new = s[name][keep].double()
        begun, touched = torch.zeros(len(ids), device="cuda"), torch.zeros(len(ids), device="cuda")
        touched[at] = 1
        begun[at[row == 0]] = 1
        most = torch.zeros((len(ids), case["kv_heads"]), dtype=torch.float64, device="cuda")
        most.index_reduce_(0, at, new.abs().amax(-1), "amax")
        need = torch.ceil(torch.log2(torch.where(most > 0, most, 1.0) / FP8_MAX)).long()
        need = need - (most <= FP8_MAX * _two_to(need - 1)).long() + (most > FP8_MAX * _two_to(need)).long()  # log2 next to a whole number
        need = torch.where(most > 0, need, E_MIN).clamp(E_MIN, E_MAX)
        e = torch.where(begun[:, None] > 0, need, torch.maximum(need, old))
        e = torch.where(touched[:, None] > 0, e, old)
        got[begun > 0] = 0
        got[at, :, row] = new
        scale = _two_to(e)[..., None, None]
        y = got / scale
        unit = _two_to((torch.frexp(y).exponent - 1).clamp(min=-6) - 3)  # 4 significant bits, steps of 2^-9 at least
        out.append(torch.round(y / unit) * unit * scale)
    return tuple(out)


def _exact_attention(case, seed):
    s = _prepare_attention(case, seed)
    hkv, dim, hq = case["kv_heads"], case["dim"], case["q_heads"]
    seqs, _ = _segments(case)
    ids = (s["words"].cpu().numpy().view(np.uint32) & ((1 << ID_BITS) - 1)).astype(np.int64)
    w = THETA ** (-torch.arange(0, dim, 2, device="cuda").double() / dim)

    def rotate(x, n):  # x [t, .., d] at positions n [t]
        c, r = torch.cos(n[:, None] * w), torch.sin(n[:, None] * w)
        c, r = (z.reshape(len(n), *([1] * (x.dim() - 2)), dim // 2) for z in (c, r))
        a, b = x[..., :dim // 2], x[..., dim // 2:]
        return torch.cat((a * c - b * r, a * r + b * c), -1)

    out = torch.zeros((len(seqs), hq, dim), dtype=torch.float64, device="cuda")
    for i, segs in enumerate(seqs):
        tok, start, b, p = [], [], 0, 0
        for _, n in segs:
            tok.append(BLOCK * b + np.arange(n))
            start.append(np.full(n, p))
            b, p = b + _blocks(n), p + n
        tok, start = torch.from_numpy(np.concatenate(tok)).cuda(), torch.from_numpy(np.concatenate(start)).cuda()
        blk = torch.from_numpy(ids[i, :b]).cuda()
        k, v = (_one_value(pool[blk], dim, is_v).transpose(1, 2).reshape(-1, hkv, dim)[tok] for pool, is_v in ((s["k_pool"], False), (s["v_pool"], True)))
        k = rotate(k, start.double())  # from the document's positions to the sequence's
        q = rotate(s["q"][i].double()[None], s["q_pos"][i:i + 1].double())[0].reshape(hkv, hq // hkv, dim)
        score = torch.einsum("hgd,thd->hgt", q, k) / math.sqrt(dim)
        out[i] = torch.einsum("hgt,thd->hgd", torch.softmax(score, -1), v).reshape(hq, dim)
    return out


def exact(case, seed):
    return {"tables": _exact_tables, "write": _exact_write}.get(case["op"], _exact_attention)(case, seed)
