"""Cases of the quantised KV cache: rows written into a paged pool and read back, and the
decodes that attend over a pool held in 4 bits.

Operators
  write  cache_write quantises new K/V rows (a slice of a fused qkv product) into the slots
         of a paged pool, then cache_read returns the blocks that were touched
  read   cache_read returns cited blocks as a bf16 pool (what the prefill takes)
  decode one query per sequence over its block table, int4 pools
  shared the same attention for a batch whose sequences cite the same documents: each cited
         block is read once per KV head for all of them

int4 format of a (block, KV head) record of 16 tokens of d dims (d / 64 groups of 64 dims)
  16 rows of d / 2 bytes: d / 8 words of 8 codes, low nibble first; word j holds the dims
  64 (j % G) + 8 (j // G) + 0 .. 7, G = d / 64. K row t is token t; V row r holds the token t
  with r = (t & 8) + 4 (t & 1) + ((t & 7) >> 1)
  then 16 x G pairs (scale, zero) in bf16, in token order
  zero = the group's least value, scale = bf16((greatest - least) / 15), code = (x - zero) / scale
  to the nearest whole number (ties to even, at most 15), value = scale * code + zero
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


# --------------------------------------------------------------------------- cases

def listed():
    heads8b = dict(q_heads=32, kv_heads=8, dim=128)
    heads70b = dict(q_heads=64, kv_heads=8, dim=128)
    return [
        # one decode step of 64 running sequences: one new token each, into a block that holds earlier ones
        dict(name="write int4 step", op="write", kv="int4", docs=64, doc_lo=1, doc_hi=1, append=True, padding=0.0, **heads8b),
        # ingestion of sixteen 512-token documents (8B heads)
        dict(name="write int4 documents", op="write", kv="int4", docs=16, doc_lo=512, doc_hi=512, append=False, padding=0.0, **heads8b),
        # documents of uneven lengths in a padded batch, small heads
        dict(name="write int4 ragged d64", op="write", kv="int4", docs=37, doc_lo=1, doc_hi=211, append=True, padding=0.1,
             q_heads=4, kv_heads=2, dim=64),
        # ingestion of sixteen 1024-token documents (70B heads) into an e4m3 pool
        dict(name="write fp8 documents", op="write", kv="fp8_e4m3", docs=16, doc_lo=1024, doc_hi=1024, append=False, padding=0.0, **heads70b),
        # one sequence's cited documents staged for its prefill: 6 x 1024 tokens and a 256-token chunk
        dict(name="read int4 context", op="read", kv="int4", blocks=400, pool=4096, **heads8b),
        # the documents of a whole batch staged at once: the pool of the 70B workload
        dict(name="read int4 pool", op="read", kv="int4", blocks=16384, pool=16384, **heads70b),
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
    op = rng.choice(["write", "read", "decode", "decode", "shared"])
    kv_heads, group, dim = rng.choice([(8, 4, 128), (8, 8, 128), (1, 32, 128), (2, 2, 64), (8, 1, 128), (4, 7, 128), (1, 64, 128),
                                       (5, 3, 64), (2, 16, 64)])
    heads = dict(q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim)
    if op == "write":
        hi = _log(rng, 1, 1024)
        docs = max(1, min(256, _log(rng, 1, 16384) // hi))
        return dict(op=op, kv=rng.choice(["int4", "int4", "fp8_e4m3"]), docs=docs, doc_lo=max(1, hi // rng.choice([1, 3, 10])), doc_hi=hi,
                    append=rng.random() < 0.5, padding=rng.choice([0.0, 0.0, 0.05, 0.2]), **heads)
    if op == "read":
        blocks = _log(rng, 1, 12000)
        return dict(op=op, kv=rng.choice(["int4", "int4", "fp8_e4m3"]), blocks=blocks, pool=blocks + _log(rng, 1, 4096), **heads)
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


def _record(kv, dim):
    return BLOCK * (dim // 2 + dim // 64 * 4) if kv == "int4" else BLOCK * dim


def work(case):
    hkv, dim = case["kv_heads"], case["dim"]
    if case["op"] in ("write", "read"):
        back = 2 * hkv * (_record(case["kv"], dim) + BLOCK * dim * 2)  # a block read back: K and V records, bf16 rows
        if case["op"] == "read":
            return {"bytes": case["blocks"] * (back + 4), "flops": 2.0 * case["blocks"] * 2 * hkv * BLOCK * dim}
        lens, first, skip = _documents(case)
        blocks = sum(_blocks(f + n) for f, n in zip(first, lens))
        rows = len(skip) - sum(skip)
        write = rows * 2 * hkv * (2 * dim + _record(case["kv"], dim) // BLOCK) + 4 * len(skip)
        return {"bytes": write + blocks * (back + 4), "flops": 6.0 * rows * 2 * hkv * dim + 2.0 * blocks * 2 * hkv * BLOCK * dim}
    unique, table, tokens = _used_blocks(_segments(case)[0])
    io = case["batch"] * case["q_heads"] * dim * 2 * 2
    return {"bytes": unique * 2 * hkv * _record("int4", dim) + 4 * table + io + 8 * case["batch"],
            "flops": 4.0 * tokens * case["q_heads"] * dim}


# --------------------------------------------------------------------------- the int4 format in plain torch

def _row_order(device):
    t = torch.arange(BLOCK, device=device)
    return (t & 8) + 4 * (t & 1) + ((t & 7) >> 1)  # V: the row that holds token t


def _quantise(x):
    """Codes (0 .. 15), scales and zeros (bf16) of rows [..., d]. In 64 bits: a value next to a border between two codes."""
    g = x.double().unflatten(-1, (-1, 64))
    least, most = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale, zero = ((most - least) / 15).to(torch.bfloat16), least.to(torch.bfloat16)
    code = torch.where(scale > 0, ((g - zero.double()) / scale.double()).round(), 0.0).clamp(0, 15)
    return code.to(torch.uint8).flatten(-2), scale, zero


def _to_e4m3(x):
    """Values in 64 bits to e4m3: 4 significant bits, steps of 2^-9 at least, saturated. (By way of 32 bits, a value next to a tie would become the tie.)"""
    step = torch.ldexp(torch.ones_like(x), (torch.frexp(x).exponent - 4).clamp(min=-9))
    return ((x / step).round() * step).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def _to_bytes(code):
    """Codes [..., d] as the words' bytes [..., d / 2]."""
    w = code.unflatten(-1, (-1, 8, 8)).transpose(-3, -2).flatten(-3)  # [..., word, nibble]
    return w[..., 0::2] | w[..., 1::2] << 4


def _from_bytes(b):
    w = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    return w.unflatten(-1, (8, -1, 8)).transpose(-3, -2).flatten(-3)


def _parts(pool, dim):
    """Views of an int4 pool [blocks, heads, record]: code rows [.., 16, d / 2], (scale, zero) [.., 16, d / 64, 2]."""
    rows, meta = pool[..., :BLOCK * dim // 2], pool[..., BLOCK * dim // 2:]
    return rows.unflatten(-1, (BLOCK, dim // 2)), meta.view(torch.bfloat16).unflatten(-1, (BLOCK, dim // 64, 2))


def _values(pool, dim, is_v):
    """An int4 pool's values [blocks, heads, 16, d] in 32 bits."""
    rows, meta = _parts(pool, dim)
    code = _from_bytes(rows[..., _row_order(pool.device), :] if is_v else rows).unflatten(-1, (-1, 64))
    return (code.float() * meta[..., :1].float() + meta[..., 1:].float()).flatten(-2)


def _random_int4(gen, blocks, hkv, dim, is_v):
    """A pool of normal rows, quantised. A few channels of K are larger, as in real caches."""
    pool = torch.empty((blocks, hkv, _record("int4", dim)), dtype=torch.uint8, device="cuda")
    gain = torch.ones(dim, device="cuda")
    if not is_v:
        gain[torch.randint(dim, (dim // 32,), generator=gen, device="cuda")] = 5.0
    step = max(1, (1 << 26) // (hkv * BLOCK * dim))
    for at in range(0, blocks, step):
        part = pool[at:at + step]
        x = torch.randn((part.shape[0], hkv, BLOCK, dim), generator=gen, device="cuda") * gain
        code, scale, zero = _quantise(x.to(torch.bfloat16))
        rows, meta = _parts(part, dim)
        rows[..., _row_order("cuda") if is_v else torch.arange(BLOCK, device="cuda"), :] = _to_bytes(code)
        meta[...] = torch.cat((scale, zero), -1)
    return pool


# --------------------------------------------------------------------------- prepare

def _params(case, module, **more):
    return module.make_params(num_q_heads=case["q_heads"], num_kv_heads=case["kv_heads"], head_dim=case["dim"], dtype="bf16", rope_theta=THETA,
                              id_bits=ID_BITS, **more)


def _pools(case, gen, blocks):
    hkv, dim = case["kv_heads"], case["dim"]
    if case["kv"] == "int4":
        return _random_int4(gen, blocks, hkv, dim, False), _random_int4(gen, blocks, hkv, dim, True), 1.0, 1.0
    pools = [torch.randn((blocks, hkv, BLOCK, dim), generator=gen, device="cuda").mul_(64).to(torch.float8_e4m3fn) for _ in range(2)]
    return pools[0], pools[1], float(np.float32(5.5 / FP8_MAX)), float(np.float32(6.5 / FP8_MAX))


def _prepare_cache(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    shuffle = np.random.default_rng(seed)
    if case["op"] == "read":
        pool = case["pool"]
        ids = shuffle.permutation(pool)[:case["blocks"]]
    else:
        lens, first, skip = _documents(case)
        spans = [_blocks(f + n) for f, n in zip(first, lens)]
        pool = sum(spans) + 16
        ids = shuffle.permutation(pool)[:sum(spans)]
        at = np.concatenate(([0], np.cumsum(spans)))
        place = [BLOCK * at[i] + first[i] + np.arange(n) for i, n in enumerate(lens)]
        place = np.concatenate(place)
        slots = np.where(skip, -1, ids[place // BLOCK] * BLOCK + place % BLOCK)
    kp, vp, ks, vs = _pools(case, gen, pool)
    s = dict(case=case, k_pool=kp, v_pool=vp, k_scale=ks, v_scale=vs, ids=torch.from_numpy(ids.astype(np.int32)).cuda())
    if case["op"] == "write":
        # K and V are slices of the layer's fused product, as the model leaves them
        qkv = torch.randn((len(slots), hq + 2 * hkv, dim), generator=gen, device="cuda").to(torch.bfloat16)
        qkv[:, hq:hq + hkv, :: max(1, dim // 4)] *= 5
        s.update(k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], slots=torch.from_numpy(slots.astype(np.int32)).cuda())
    if own:
        from paged_kv_cache_57_gb300 import lazy_attn
        s.update(lib=lazy_attn, p=_params(case, lazy_attn, num_seqs=0, num_pool_blocks=pool, max_blocks_per_seq=0, kv_dtype=case["kv"],
                                          k_scale=ks, v_scale=vs))
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
    kp, vp = (_random_int4(gen, pool, hkv, dim, is_v) for is_v in (False, True))
    ends = [(order[at[doc] + spans[doc] - 1], doc_len[doc] % BLOCK) for doc in cited if doc_len[doc] % BLOCK]
    if ends:  # slots behind a document's end hold what nothing wrote: NaN
        blk = torch.tensor([int(b) for b, _ in ends], device="cuda")
        gone = torch.arange(BLOCK, device="cuda")[None] >= torch.tensor([n for _, n in ends], device="cuda")[:, None]
        for x in (kp, vp):
            meta = _parts(x, dim)[1]
            meta[blk] = torch.where(gone[:, None, :, None, None], math.nan, meta[blk])
    s = dict(case=case, k_pool=kp, v_pool=vp, q=torch.randn((len(seqs), hq, dim), generator=gen, device="cuda").to(torch.bfloat16),
             words=torch.from_numpy(words.view(np.int32)).cuda(), seq_lens=torch.from_numpy(seq_lens).cuda(), q_pos=torch.from_numpy(q_pos).cuda(),
             freqs=THETA ** (-2.0 * torch.arange(dim // 2, dtype=torch.float64, device="cuda") / dim))
    if own:
        from paged_kv_cache_57_gb300 import lazy_attn
        p = _params(case, lazy_attn, num_seqs=len(seqs), num_pool_blocks=pool, max_blocks_per_seq=max_blocks, kv_dtype="int4")
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
    return (_prepare_cache if case["op"] in ("write", "read") else _prepare_attention)(case, seed)


# --------------------------------------------------------------------------- run

def _write_plain(s):
    case, dim = s["case"], s["case"]["dim"]
    at = (s["slots"] >= 0).nonzero()[:, 0]
    block, row = s["slots"][at].long() // BLOCK, s["slots"][at].long() % BLOCK
    for x, pool, scale, is_v in ((s["k"], s["k_pool"], s["k_scale"], False), (s["v"], s["v_pool"], s["v_scale"], True)):
        if case["kv"] == "int4":
            rows, meta = _parts(pool, dim)
            code, sc, zero = _quantise(x[at])
            rows[block, :, _row_order("cuda")[row] if is_v else row] = _to_bytes(code)
            meta[block, :, row] = torch.cat((sc, zero), -1)
        else:
            pool[block, :, row] = _to_e4m3(x[at].double() / scale)


def _read_plain(s):
    case, ids = s["case"], s["ids"].long()
    if case["kv"] == "int4":
        return tuple(_values(pool[ids], case["dim"], is_v).to(torch.bfloat16) for pool, is_v in ((s["k_pool"], False), (s["v_pool"], True)))
    return tuple((pool[ids].float() * scale).to(torch.bfloat16) for pool, scale in ((s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"])))


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
    k, v = (torch.where(live[:, :, None, :, None], _values(pool[phys], dim, is_v), 0.0) for pool, is_v in ((s["k_pool"], False), (s["v_pool"], True)))
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
        if op == "write":
            _write_plain(s)
        return _read_plain(s) if op in ("write", "read") else _attend_plain(s)
    lib, p = s["lib"], s["p"]
    if op == "write":
        lib.cache_write(p, s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"])
    if op in ("write", "read"):
        return lib.cache_read(p, s["k_pool"], s["v_pool"], s["ids"])
    if op == "decode":
        return lib.decode(p, s["q"], s["k_pool"], s["v_pool"], s["words"], s["seq_lens"], s["q_pos"], s["rope"], out=s["out"], workspace=s["workspace"])
    return lib.decode_shared(p, s["q"], s["k_pool"], s["v_pool"], s["words"], s["q_pos"], s["rope"], s["plan"], out=s["out"], workspace=s["workspace"])


# --------------------------------------------------------------------------- exact: from the definition, in 64 bits

def _one_value(pool, dim, is_v):
    """Values [.., 16, d] of records, dimension by dimension: dim e is code e % 8 of word G ((e % 64) // 8) + e // 64."""
    e = torch.arange(dim, device=pool.device)
    byte = 4 * (dim // 64 * (e % 64 // 8) + e // 64) + e % 8 // 2
    t = torch.arange(BLOCK, device=pool.device)
    row = torch.where(t % 8 % 2 == 0, t // 8 * 8 + t % 8 // 2, t // 8 * 8 + 4 + t % 8 // 2) if is_v else t
    got = pool[..., (row[:, None] * (dim // 2) + byte[None]).flatten()].unflatten(-1, (BLOCK, dim)).int()
    code = torch.where(e % 2 == 0, got % 16, got // 16).double()
    at = BLOCK * dim // 2 + 4 * (t[:, None] * (dim // 64) + e[None] // 64)
    halves = [(pool[..., at + o].int() | pool[..., at + o + 1].int() << 8) << 16 for o in (0, 2)]
    scale, zero = (h.view(torch.float32).double() for h in halves)
    return code * scale + zero


def _exact_cache(case, seed):
    s = _prepare_cache(case, seed)
    dim, ids, out = case["dim"], s["ids"].long(), []
    for name, is_v in (("k", False), ("v", True)):
        pool, scale = s[name + "_pool"], s[name + "_scale"]
        got = _one_value(pool[ids], dim, is_v) if case["kv"] == "int4" else pool[ids].double() * scale
        if case["op"] == "write":
            where = torch.full((pool.shape[0],), -1, device="cuda")
            where[ids] = torch.arange(len(ids), device="cuda")
            keep = s["slots"] >= 0
            slot, x = s["slots"][keep].long(), s[name][keep].double()
            if case["kv"] == "int4":
                g = x.reshape(*x.shape[:-1], dim // 64, 64)
                zero = g.min(-1).values[..., None]
                step = ((g.max(-1).values[..., None] - zero) / 15).float().bfloat16().double()
                x = (torch.minimum(torch.round((g - zero) / torch.where(step > 0, step, 1.0)), torch.tensor(15.0, device="cuda")) * step + zero).reshape(x.shape)
            else:  # e4m3: 4 significant bits, at least steps of 2^-9, at most 448
                y = x / scale
                unit = torch.exp2(torch.clamp(torch.floor(torch.log2(y.abs().clamp(min=1e-30))), min=-6) - 3)
                x = (torch.round(y / unit) * unit).clamp(-FP8_MAX, FP8_MAX) * scale
            got[where[slot // BLOCK], :, slot % BLOCK] = x
        out.append(got)
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
    return (_exact_cache if case["op"] in ("write", "read") else _exact_attention)(case, seed)
