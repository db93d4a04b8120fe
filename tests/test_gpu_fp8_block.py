"""GPU: pools of e4m3 codes with block scales -- rows written and read back, byte for byte against the
format's restatement (tests/fp8_block_model.py), and the decodes on them against 64-bit attention over
the same codes, with that file's error bound."""
import numpy as np
import pytest
import torch

import fp8_block_model as M
from gpu_util import la, shared_plan, to_device
from paged_kv_cache_57_gb300 import workloads as W

pytestmark = pytest.mark.gpu
KIND = "fp8_e4m3_block"


@pytest.fixture(autouse=True)
def _clean_status():
    la().device_status(clear=True)
    yield
    assert la().device_status(clear=True) == 0, "device status word set"


# ---------------------------------------------------------------- rows into the pools

def params(hkv, d, blocks, hq=None):
    return la().make_params(num_seqs=0, num_q_heads=hq or hkv, num_kv_heads=hkv, head_dim=d, num_pool_blocks=blocks, max_blocks_per_seq=0,
                            kv_dtype=KIND)


def filled_pools(p, seed):
    """Pools of records with scales 2^-8 .. 2^3 and codes of every kind (NaN too) on the GPU, and their copies."""
    L = la()
    g = np.random.default_rng(seed)
    out = []
    for x in L.empty_pools(p):
        y = g.integers(0, 256, tuple(x.shape)).astype(np.uint8)
        n = 16 * p.head_dim
        y[..., n:n + 4] = np.ascontiguousarray((2.0 ** g.integers(-8, 4, x.shape[:2])).astype("<f4")[..., None]).view(np.uint8)
        x.copy_(torch.from_numpy(y))
        out.append((x, y))
    return [x for x, _ in out], [y for _, y in out]


def rows(kind, t, h, d, rng):
    x = rng.standard_normal((t, h, d))
    if kind == "outliers":
        x[..., ::16] *= 50
    elif kind == "growing":  # every token's greatest value above the last one's
        x *= np.minimum(2.0 ** (np.arange(t) % 150 - 20.0), 2.0 ** 100).reshape(-1, 1, 1)
    elif kind == "ties":  # multiples of halves of e4m3's steps
        x = rng.integers(-511, 512, x.shape) * 2.0 ** rng.integers(-12, 1, x.shape)
        x[..., 0] = 448.0 * 2.0 ** rng.integers(-1, 2, x.shape[:2])
    elif kind == "edges":  # greatest values at and next to 448 * 2^e in bf16
        x = rng.uniform(-1, 1, x.shape)
        x[..., d // 2] = rng.choice([1.75, 1.7578125, 1.7421875], x.shape[:2]) * 2.0 ** rng.integers(-3, 4, x.shape[:2])
    elif kind == "extremes":
        x = x * 10.0 ** rng.integers(-37, 38, (t, h, 1))
    elif kind == "zero":
        x[rng.random((t, h)) < 0.7] = 0
    elif kind == "bad":
        for v in (np.nan, np.inf, -np.inf):
            x[rng.random(x.shape) < 0.01] = v
        x[::5, 0] = np.nan
    return torch.from_numpy(x).to(torch.bfloat16)


def scatter(slots, pool, x, is_v):
    """The expected records: `pool` with x's rows put in their slots by one call."""
    xs = x.double().numpy()
    by_block = {}
    for t, s in enumerate(slots):
        if s >= 0:
            by_block.setdefault(int(s) // 16, {})[int(s) % 16] = t
    for b, toks in by_block.items():
        for h in range(xs.shape[1]):
            M.put(pool[b, h], {r: xs[t, h] for r, t in toks.items()}, is_v)


def same_records(got, want, d):
    got = got.cpu().numpy()
    n = 16 * d
    a, b = got[..., :n], want[..., :n]
    # NaN is one value with two codes
    bad = (a != b) & ~(((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F))
    assert not bad.any(), np.argwhere(bad)[:5]
    assert np.array_equal(got[..., n:n + 4], want[..., n:n + 4])


def documents(rng, blocks, lens, firsts, shuffle=False, skip=0.0):
    """Slots of documents that lie in fresh blocks of a pool from row `first` on."""
    ids, out = list(rng.permutation(blocks)), []
    for n, f in zip(lens, firsts):
        mine = [ids.pop() for _ in range((f + n + 15) // 16)]
        t = f + np.arange(n)
        s = np.asarray(mine)[t // 16] * 16 + t % 16
        if shuffle:  # within a block
            s = np.concatenate([rng.permutation(s[t // 16 == b]) for b in np.unique(t // 16)])
        out.append(s)
    out = np.concatenate(out).astype(np.int32)
    out[rng.random(len(out)) < skip] = -1
    return out


@pytest.mark.parametrize("kind", ["normal", "outliers", "growing", "ties", "edges", "extremes", "zero", "bad"])
@pytest.mark.parametrize("hkv,d", [(8, 128), (3, 64)])
def test_write_bytes(kind, hkv, d):
    # whole blocks, parts of one from row 0 or not, a token alone; rows out of order; padding between them
    L = la()
    rng = np.random.default_rng(70 + d)
    p = params(hkv, d, 24)
    (kp, vp), (k0, v0) = filled_pools(p, 1)
    slots = documents(rng, 24, [16, 40, 1, 1, 7, 5, 23, 16], [0, 0, 0, 9, 0, 6, 12, 3], shuffle=kind in ("normal", "growing"), skip=0.1)
    t = len(slots)
    k, v = rows(kind, t, hkv, d, rng), rows(kind, t, hkv, d, rng)
    L.cache_write(p, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), kp, vp)
    scatter(slots, k0, k, False)
    scatter(slots, v0, v, True)
    same_records(kp, k0, d)
    same_records(vp, v0, d)


@pytest.mark.parametrize("hkv,d", [(2, 128), (2, 64)])
@pytest.mark.parametrize("kind", ["normal", "growing", "bad"])
def test_rows_appended_one_call_at_a_time(hkv, d, kind):
    # 40 decode steps of five sequences: blocks begin, grow their scales and fill up
    L = la()
    rng = np.random.default_rng(90 + d)
    p = params(hkv, d, 30)
    (kp, vp), (k0, v0) = filled_pools(p, 2)
    ids, first = rng.permutation(30).reshape(5, 6), np.array([0, 5, 15, 16, 31])
    for b, f in enumerate(first):  # blocks that go on hold finite values
        for pool in (kp, vp):
            pool[int(ids[b, f // 16])] = 0
            pool[int(ids[b, f // 16]), :, 16 * d + 3] = 63  # a scale of 0.5
            pool[int(ids[b, f // 16]), :, 16 * d + 2] = 0
    k0, v0 = kp.cpu().numpy().copy(), vp.cpu().numpy().copy()
    x = [rows(kind, 40, 5 * hkv, d, rng) for _ in range(2)]
    for step in range(40):
        at = first + step
        slots = (ids[np.arange(5), at // 16] * 16 + at % 16).astype(np.int32)
        k, v = (y[step].view(5, hkv, d) for y in x)
        L.cache_write(p, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), kp, vp)
        scatter(slots, k0, k, False)
        scatter(slots, v0, v, True)
    same_records(kp, k0, d)
    same_records(vp, v0, d)


def test_many_tokens():
    # enough tokens for windows of a block's length: documents that straddle windows, single tokens among them
    L = la()
    rng = np.random.default_rng(5)
    hkv, d = 8, 64
    p = params(hkv, d, 600)
    (kp, vp), (k0, v0) = filled_pools(p, 3)
    lens = [1] * 37 + [300, 16, 5, 700] + [1] * 20 + list(rng.integers(1, 90, 40))
    slots = documents(rng, 600, lens, rng.integers(0, 16, len(lens)), skip=0.05)
    t = len(slots)
    assert t * 2 * hkv > 152 * 128
    k, v = rows("outliers", t, hkv, d, rng), rows("growing", t, hkv, d, rng).clamp(-1e6, 1e6)
    L.cache_write(p, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), kp, vp)
    scatter(slots, k0, k, False)
    scatter(slots, v0, v, True)
    same_records(kp, k0, d)
    same_records(vp, v0, d)


@pytest.mark.parametrize("layout", ["fused", "heads_first", "odd", "odd_start", "broadcast"])
@pytest.mark.parametrize("d", [64, 128])
def test_write_strides(layout, d):
    L = la()
    rng = np.random.default_rng(8)
    t, hkv = 33, 4
    p = params(hkv, d, 8)
    (kp, vp), (k0, v0) = filled_pools(p, 4)
    base = torch.from_numpy(rng.standard_normal((t, 12, d + 8))).to(torch.bfloat16).cuda()
    if layout == "fused":
        qkv = base[..., :d].contiguous()
        k, v = qkv[:, 4:8], qkv[:, 8:]
    elif layout == "heads_first":
        k, v = (base[:, a:a + 4, :d].transpose(0, 1).contiguous().transpose(0, 1) for a in (0, 4))
    elif layout == "odd":
        k, v = base[:, :4, 1:d + 1], base[:, 4:8, 3:d + 3]
    elif layout == "odd_start":
        flat = torch.empty(t * 4 * d + 1, dtype=torch.bfloat16, device="cuda")
        k = flat[1:].view(t, 4, d)
        k.copy_(base[:, :4, :d])
        v = base[:, 4:8, :d]
    else:
        k, v = base[:1, :4, :d].expand(t, 4, d), base[:, :1, :d].expand(t, 4, d)
    slots = documents(rng, 8, [33], [2])
    L.cache_write(p, k, v, torch.from_numpy(slots).cuda(), kp, vp)
    scatter(slots, k0, k.cpu(), False)
    scatter(slots, v0, v.cpu(), True)
    same_records(kp, k0, d)
    same_records(vp, v0, d)


def test_write_skips_and_reports_bad_slots():
    L = la()
    p = params(2, 128, 4)
    (kp, vp), (k0, v0) = filled_pools(p, 6)
    x = torch.ones(5, 2, 128, dtype=torch.bfloat16, device="cuda")
    L.cache_write(p, x, x, torch.tensor([-1, -16, -2 ** 31, -1, -5], dtype=torch.int32, device="cuda"), kp, vp)
    assert L.device_status(clear=True) == 0
    L.cache_write(p, x, x, torch.tensor([64, 2 ** 31 - 1, 17, -1, 4 * 16 + 3], dtype=torch.int32, device="cuda"), kp, vp)
    assert L.device_status(clear=True) == L.LAZY_DEV_BAD_BLOCK_ID
    scatter([-1, -1, 17], k0, x.cpu(), False)
    scatter([-1, -1, 17], v0, x.cpu(), True)
    same_records(kp, k0, 128)
    same_records(vp, v0, 128)


@pytest.mark.parametrize("hkv,d,n", [(8, 128, 33), (1, 64, 7), (5, 64, 1), (3, 128, 900)])
def test_read_values(hkv, d, n):
    L = la()
    rng = np.random.default_rng(n)
    p = params(hkv, d, 50)
    (kp, vp), (k0, v0) = filled_pools(p, 7)
    ids = rng.integers(0, 50, n).astype(np.int32)
    ids[rng.random(n) < 0.2] = -1
    outs = [torch.full((n, hkv, 16, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    L.cache_read(p, kp, vp, torch.from_numpy(ids).cuda(), *outs)
    for got, pool, is_v in zip(outs, (k0, v0), (False, True)):
        want = np.where(ids[:, None, None, None] < 0, 7.0, M.values(pool, d, is_v)[np.maximum(ids, 0)])
        assert np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)  # 4 bits times a power of two: exact in bf16
    ids[0] = 50
    L.cache_read(p, kp, vp, torch.from_numpy(ids).cuda(), *outs)
    assert L.device_status(clear=True) == L.LAZY_DEV_BAD_BLOCK_ID


# ---------------------------------------------------------------- the decodes

def on_device(w, **kw):
    """(Dev with block-scaled params, k_pool, v_pool on the GPU, their values in fp64)."""
    L = la()
    dv = to_device(w, **kw)
    dv.p.kv_dtype = L.LAZY_FP8_E4M3_BLOCK
    kp, vp = M.pools(w)
    kv, vv = (torch.from_numpy(np.nan_to_num(M.values(x.numpy(), w.head_dim, is_v))).cuda() for x, is_v in ((kp, False), (vp, True)))
    return dv, kp.cuda(), vp.cuda(), kv, vv


def check(out, ref, what):
    want, bound = ref
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all(), what
    worst = (err / bound).max().item() if bound.numel() else 0.0
    assert worst <= 1.0, f"{what}: off by {worst:.2f} of the bound at {np.unravel_index((err / bound).argmax().item(), err.shape)}"


def decode(dv, kp, vp, **kw):
    return la().decode(dv.p, dv.q, kp, vp, dv.words, dv.seq_lens, dv.q_pos, dv.rope, **kw)


def shared(dv, kp, vp, chunk=0):
    return la().decode_shared(dv.p, dv.q, kp, vp, dv.words, dv.q_pos, dv.rope, shared_plan(dv, chunk))


# every number of rows that a warp or a team takes, and what fills them in part; both head sizes; documents whose last block
# is partial, slots behind them NaN
@pytest.mark.parametrize("hq,hkv,d,splits", [(8, 8, 128, 0), (4, 2, 64, 1), (32, 8, 128, 3), (28, 4, 128, 0), (64, 8, 128, 2), (18, 2, 128, 0),
                                             (32, 2, 64, 5), (32, 1, 128, 0), (64, 1, 128, 2), (64, 1, 64, 0), (17, 1, 64, 1), (33, 1, 128, 0),
                                             (10, 2, 64, 0), (3, 1, 128, 0)])
def test_decode_matches_64_bits(hq, hkv, d, splits):
    w = W.decode_zipf(f"f8{hq}", batch=6, hq=hq, hkv=hkv, d=d, docs_per_seq=4, doc_tokens=150, pool_docs=5, zipf_s=1.0,
                      suffix_tokens=21, seed=1620 + hq + splits)
    dv, kp, vp, kv, vv = on_device(w, num_splits=splits)
    check(decode(dv, kp, vp), M.attention(w, kv, vv), f"decode {hq}/{hkv} d{d} splits {splits}")


@pytest.mark.parametrize("doc,docs", [(1, 1), (1, 2), (1, 33), (15, 1), (16, 1), (17, 1), (16, 2), (3, 11), (32, 1), (33, 1)])
@pytest.mark.parametrize("d,hq", [(64, 8), (128, 8), (128, 64)])
def test_decode_short_contexts(doc, docs, d, hq):
    w = W.decode_zipf("f8s", batch=3, hq=hq, hkv=2, d=d, docs_per_seq=docs, doc_tokens=doc, pool_docs=3, zipf_s=0.5, share=False,
                      seed=1700 + doc + docs)
    dv, kp, vp, kv, vv = on_device(w)
    ref = M.attention(w, kv, vv)
    check(decode(dv, kp, vp), ref, f"{docs} documents of {doc}")
    check(shared(dv, kp, vp), ref, f"shared, {docs} documents of {doc}")


def test_decode_ragged_batch_with_empty_sequences():
    dw, _ = W.mixed_mqa(n_decode=9, n_prefill=1, chunk=16, hq=8, hkv=2, d=128, pool_docs=60, ctx_lo=1, ctx_hi=5000, doc_lo=1, doc_hi=300,
                        seed=1710)
    dv, kp, vp, kv, vv = on_device(dw)
    want, bound = M.attention(dw, kv, vv)
    for splits in (0, 1, 7, 400):
        dv.p.num_splits = splits
        check(decode(dv, kp, vp), (want, bound), f"ragged, splits {splits}")
        lens = dv.seq_lens.clone()
        lens[[2, 8]] = 0
        out = la().decode(dv.p, dv.q, kp, vp, dv.words, lens, dv.q_pos, dv.rope)
        assert torch.count_nonzero(out[[2, 8]]) == 0
        keep = [0, 1, 3, 4, 5, 6, 7]
        check(out[keep], (want[keep], bound[keep]), "beside empty sequences")


# more units than a device has resident CTAs and sequences of more than 512 blocks among short ones: ranges of the units'
# blocks laid end to end, several units or parts of one in a CTA's range
@pytest.mark.parametrize("batch,hq,hkv,d", [(330, 8, 2, 64), (330, 12, 2, 128), (460, 32, 1, 64), (460, 64, 1, 64)])
def test_decode_ranges_of_ragged_batches(batch, hq, hkv, d):
    L = la()
    dw, _ = W.mixed_mqa(n_decode=batch, n_prefill=1, chunk=16, hq=hq, hkv=hkv, d=d, pool_docs=60, ctx_lo=1, ctx_hi=9500, doc_lo=1, doc_hi=700,
                        seed=1713 + hq)
    dv, kp, vp, kv, vv = on_device(dw)
    assert dw.max_blocks_per_seq > 512 and 0 < L.decode_workspace_bytes(dv.p)
    want, bound = M.attention(dw, kv, vv)
    ws = torch.full((L.decode_workspace_bytes(dv.p),), 255, dtype=torch.uint8, device="cuda")
    first = decode(dv, kp, vp, workspace=ws)
    check(first, (want, bound), "all")
    assert torch.equal(decode(dv, kp, vp, workspace=ws), first)
    long = int(dv.seq_lens.argmax())
    for keep in ([batch - 1], [0], [long], [3, batch // 2, long], list(range(40, batch)), []):
        lens = torch.zeros_like(dv.seq_lens)
        lens[keep] = dv.seq_lens[keep]
        ws.fill_(255)
        out = L.decode(dv.p, dv.q, kp, vp, dv.words, lens, dv.q_pos, dv.rope, workspace=ws)
        check(out[keep], (want[keep], bound[keep]), f"only {keep[:3]}")
        assert torch.count_nonzero(out).item() == torch.count_nonzero(out[keep]).item()


@pytest.mark.parametrize("hq,hkv,d,chunk", [(8, 8, 128, 0), (4, 2, 64, 0), (32, 8, 128, 3), (28, 4, 128, 5), (16, 2, 64, 1), (32, 1, 128, 0),
                                            (64, 1, 128, 5), (64, 8, 128, 0), (33, 1, 64, 7)])
def test_shared_decode_matches_64_bits(hq, hkv, d, chunk):
    L = la()
    w = W.decode_zipf(f"f8sh{hq}", batch=10, hq=hq, hkv=hkv, d=d, docs_per_seq=4, doc_tokens=150, pool_docs=4, zipf_s=1.0,
                      suffix_tokens=21, seed=1760 + hq + chunk)
    dv, kp, vp, kv, vv = on_device(w)
    plan = shared_plan(dv, chunk)
    assert (plan.items_host[:, 4] * (hq // hkv) <= 64).all()
    out = L.decode_shared(dv.p, dv.q, kp, vp, dv.words, dv.q_pos, dv.rope, plan)
    check(out, M.attention(w, kv, vv), f"shared-run decode {hq}/{hkv} chunk {chunk}")
    ws = torch.empty(L.decode_shared_workspace_bytes(dv.p, plan.num_slots), dtype=torch.uint8, device="cuda")
    L.decode_shared_partials(dv.p, dv.q, kp, vp, dv.words, dv.q_pos, dv.rope, plan, ws)
    two = L.decode_shared_combine(dv.p, plan, ws, torch.empty_like(dv.q))
    assert torch.equal(two.view(torch.int16), out.view(torch.int16))


def test_shared_decode_holes_and_long_items():
    dw, _ = W.mixed_mqa(n_decode=8, n_prefill=1, chunk=16, hq=32, hkv=1, d=128, pool_docs=40, ctx_lo=1, ctx_hi=3000, doc_lo=1, doc_hi=700,
                        seed=1765)
    dv, kp, vp, kv, vv = on_device(dw)
    ref = M.attention(dw, kv, vv)
    for chunk in (0, 4, 64):
        check(shared(dv, kp, vp, chunk), ref, f"chunk {chunk}")


def test_far_positions_and_control():
    w = W.decode_zipf("f8far", batch=3, hq=8, hkv=2, d=128, docs_per_seq=3, doc_tokens=70, pool_docs=4, zipf_s=0.5, seed=1720,
                      shift=130000)
    dv, kp, vp, kv, vv = on_device(w, id_bits=14)
    ref = M.attention(w, kv, vv)
    check(decode(dv, kp, vp), ref, "far")
    check(shared(dv, kp, vp), ref, "far, shared")
    # control: keys at their absolute positions, every query rotated once
    L = la()
    dv, kp, vp, kv, vv = on_device(w, lazy=False, id_bits=14)
    dv.rope = L.rope_table_init(dv.p, freqs=np.zeros(64))  # no rotation at all: the stored keys are the keys
    w.rope_theta = 1e300
    w.q_pos = np.zeros_like(w.q_pos)
    ref = M.attention(w, kv, vv, lazy=False)
    check(decode(dv, kp, vp), ref, "control")
    check(shared(dv, kp, vp), ref, "control, shared")


# scales that grow and fall from block to block by up to 2^40, tiny and huge ones, sharp and flat scores
@pytest.mark.parametrize("case", ["v_growing", "v_falling", "v_mixed", "v_tiny", "v_huge", "k_mixed", "k_sharp", "k_flat"])
@pytest.mark.parametrize("hq", [3, 8, 16, 48])
def test_decode_scales(case, hq):
    w = W.decode_zipf("f8sc", batch=2, hq=hq, hkv=1, d=128, docs_per_seq=2, doc_tokens=400, pool_docs=3, zipf_s=0.5, share=False, seed=1730)
    nb = w.num_pool_blocks
    g = torch.Generator().manual_seed(3)
    order = torch.empty(nb, dtype=torch.float64)
    order[torch.from_numpy(w.doc_blocks.astype(np.int64))] = torch.arange(len(w.doc_blocks), dtype=torch.float64)
    order = order.view(-1, 1, 1, 1)
    x, at = ("v_pool", w.v_pool) if case[0] == "v" else ("k_pool", w.k_pool)
    f = {"v_growing": 2.0 ** (order // 2 - 20), "v_falling": 2.0 ** (20 - order // 2),
         "v_mixed": 2.0 ** torch.randint(-20, 21, order.shape, generator=g).double(), "v_tiny": 2.0 ** -95, "v_huge": 2.0 ** 100,
         "k_mixed": 2.0 ** torch.randint(-12, 1, order.shape, generator=g).double(), "k_sharp": 6.0, "k_flat": 2.0 ** -40}[case]
    setattr(w, x, (at.double() * f).to(torch.bfloat16))
    dv, kp, vp, kv, vv = on_device(w, num_splits=1)
    ref = M.attention(w, kv, vv)
    check(decode(dv, kp, vp), ref, case)
    check(shared(dv, kp, vp, 200), ref, f"{case}, shared")


@pytest.mark.parametrize("qscale", [2.0 ** -30, 2.0 ** 4])
def test_decode_query_sizes(qscale):
    w = W.decode_zipf("f8q", batch=2, hq=8, hkv=2, d=128, docs_per_seq=2, doc_tokens=100, pool_docs=3, zipf_s=0.5, seed=1735)
    w.q = (w.q.float() * qscale).to(torch.bfloat16)
    dv, kp, vp, kv, vv = on_device(w)
    check(decode(dv, kp, vp), M.attention(w, kv, vv), f"queries times {qscale}")


# thousands of blocks of a warp, with maxima and V scales that keep growing
@pytest.mark.parametrize("hq,d", [(3, 128), (8, 64), (16, 64), (32, 64), (48, 128)])
def test_long_runs(hq, d):
    docs = 2 if hq <= 16 else 1
    w = W.decode_zipf("f8long", batch=1, hq=hq, hkv=1, d=d, docs_per_seq=docs, doc_tokens=80000, pool_docs=docs, zipf_s=0.5, share=False,
                      seed=1832)
    nb = w.num_pool_blocks
    at = torch.empty(nb, dtype=torch.float64)
    at[torch.from_numpy(w.doc_blocks.astype(np.int64))] = torch.arange(nb, dtype=torch.float64)
    at = at.view(-1, 1, 1, 1)
    w.k_pool = (w.k_pool.double() * (0.25 + 1.5 * at / nb)).to(torch.bfloat16)
    w.v_pool = ((1 + w.v_pool.double() / 4) * 2.0 ** (at // 700)).to(torch.bfloat16)
    dv, kp, vp, kv, vv = on_device(w, num_splits=1, id_bits=14)
    ref = M.attention(w, kv, vv)
    check(decode(dv, kp, vp), ref, "per sequence")
    check(shared(dv, kp, vp, 5000), ref, "shared")
    dv.p.num_splits = 0
    check(decode(dv, kp, vp), ref, "split")


def test_a_million_tokens():
    # more blocks than the warps of a CTA add up: cut, whatever num_splits and chunk_blocks say
    L = la()
    w = W.decode_zipf("f8million", batch=1, hq=3, hkv=1, d=64, docs_per_seq=34, doc_tokens=32000, pool_docs=1, zipf_s=0.0, seed=1834)
    w.v_pool = (1 + w.v_pool.double() / 4).to(torch.bfloat16)
    dv, kp, vp, kv, vv = on_device(w, num_splits=1, id_bits=11)
    assert dv.p.max_blocks_per_seq == 68000 and L.decode_workspace_bytes(dv.p) > 0
    ref = M.attention(w, kv, vv)
    check(decode(dv, kp, vp), ref, "per sequence")
    check(shared(dv, kp, vp, 60000), ref, "shared")
    plan = shared_plan(dv)
    plan.items.view(-1)[2] = 16385  # an item longer than a warp adds up: refused
    L.decode_shared(dv.p, dv.q, kp, vp, dv.words, dv.q_pos, dv.rope, plan)
    assert L.device_status(clear=True) == L.LAZY_DEV_LAYOUT


def test_low_scores_beside_parts_without_keys():
    dw, _ = W.mixed_mqa(n_decode=9, n_prefill=1, chunk=16, hq=8, hkv=2, d=128, pool_docs=60, ctx_lo=1, ctx_hi=5000, doc_lo=1, doc_hi=300,
                        seed=1811)
    slow = torch.zeros(128)
    slow[48:64] = slow[112:] = 8.0
    dw.k_pool = (dw.k_pool.float() + slow).to(torch.bfloat16)
    dw.q = (dw.q.float() - slow).to(torch.bfloat16)
    dw.v_pool = (1 + dw.v_pool.float() / 8).to(torch.bfloat16)
    dv, kp, vp, kv, vv = on_device(dw)
    ref = M.attention(dw, kv, vv)
    for splits in (0, 1, 7, 300):
        dv.p.num_splits = splits
        check(decode(dv, kp, vp), ref, f"splits {splits}")
    check(shared(dv, kp, vp, 4), ref, "shared")


def test_nan_of_a_visible_key_shows_and_of_a_hole_does_not():
    w = W.decode_zipf("f8nan", batch=2, hq=4, hkv=2, d=128, docs_per_seq=2, doc_tokens=50, pool_docs=3, zipf_s=0.5, share=False, seed=1741)
    blk = int(w.doc_blocks[int(w.doc_block_indptr[w.seq_segments(1)[0][0]])])
    w.v_pool[blk, 1, 3, 5] = float("nan")  # sequence 1, KV head 1: query heads 2 and 3
    dv, kp, vp, kv, vv = on_device(w)
    for splits in (1, 2):
        dv.p.num_splits = splits
        out = decode(dv, kp, vp).float()
        bad = torch.isnan(out)
        assert bad[1, 2:, 5].all() and bad.sum() == 2
    w.k_pool[blk, 0] = float("nan")  # all of the first block's keys, KV head 0
    dv, kp, vp, kv, vv = on_device(w)
    for out in (decode(dv, kp, vp), shared(dv, kp, vp)):
        bad = torch.isnan(out.float())
        assert bad[1, :2].all() and not bad[0].any()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (2, 2, 64), (48, 2, 128)])
def test_rows_without_a_finite_score_are_nan(hq, hkv, d):
    w = W.decode_zipf("f8n", batch=3, hq=hq, hkv=hkv, d=d, docs_per_seq=2, doc_tokens=90, pool_docs=3, zipf_s=0.5, share=False,
                      suffix_tokens=7, seed=1820)
    w.q[0, 1, 3] = float("nan")
    dv, kp, vp, kv, vv = on_device(w)
    w.q[0, 1] = 0
    want, bound = M.attention(w, kv, vv)
    rest = torch.ones(3, hq, dtype=torch.bool, device="cuda")
    rest[0, 1] = False
    for out in (decode(dv, kp, vp), shared(dv, kp, vp)):
        assert torch.isnan(out[0, 1]).all()
        check(out[rest], (want[rest], bound[rest]), "the other rows")


def test_device_errors_are_reported():
    L = la()
    w = W.decode_zipf("f8err", batch=3, hq=8, hkv=2, d=128, docs_per_seq=2, doc_tokens=50, pool_docs=3, zipf_s=0.5, seed=1742)
    dv, kp, vp, kv, vv = on_device(w)
    lens = dv.seq_lens.clone()
    lens[1] = 16 * dv.p.max_blocks_per_seq + 1
    L.decode(dv.p, dv.q, kp, vp, dv.words, lens, dv.q_pos, dv.rope)
    assert L.device_status(clear=True) & L.LAZY_DEV_BAD_LEN
    lens[1] = -5
    out = L.decode(dv.p, dv.q, kp, vp, dv.words, lens, dv.q_pos, dv.rope)
    assert L.device_status(clear=True) == L.LAZY_DEV_BAD_LEN and torch.count_nonzero(out[1]) == 0
    words = dv.words.clone()
    words[2, 1] = (words[2, 1] & ~0x3FFFF) | 0x3FFFE
    L.decode(dv.p, dv.q, kp, vp, words, dv.seq_lens, dv.q_pos, dv.rope)
    assert L.device_status(clear=True) == L.LAZY_DEV_BAD_BLOCK_ID
    plan = shared_plan(dv)
    plan.items.view(-1, L.PLAN_ITEM_INTS)[0, 0] = 99
    L.decode_shared(dv.p, dv.q, kp, vp, dv.words, dv.q_pos, dv.rope, plan)
    assert L.device_status(clear=True) == L.LAZY_DEV_LAYOUT


# a block whose word and whose item disagree, or which is not in the pool, is left out of shared runs too
@pytest.mark.parametrize("batch,hq", [(1, 4), (1, 16), (3, 8), (4, 16)])
@pytest.mark.parametrize("at", [0, 1, 4, 9])
def test_shared_items_leave_bad_blocks_out(batch, hq, at):
    L = la()
    w = W.decode_zipf("f8badrec", batch=batch, hq=hq, hkv=1, d=128, docs_per_seq=1, doc_tokens=160, pool_docs=1, zipf_s=0.5, seed=1871)
    blocks = w.doc_blocks[:10].astype(int)
    dv, kp, vp, kv, vv = on_device(w)

    def kept(out, what):  # what the other nine blocks give
        want = torch.zeros((batch, hq, 128), dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(want)
        keep = torch.arange(160, device="cuda") // 16 != at
        f = torch.as_tensor(w.rope_theta ** (-2.0 * np.arange(64) / 128), dtype=torch.float64, device="cuda")
        k = kv[torch.as_tensor(blocks, device="cuda")].reshape(160, 128)[keep]
        v = vv[torch.as_tensor(blocks, device="cuda")].reshape(160, 128)[keep]
        for b in range(batch):
            d = (float(w.q_pos[b]) - float(w.seq_pos0[b])) * f
            q = w.q[b].double().cuda()
            r = torch.cat((q[:, :64] * d.cos() - q[:, 64:] * d.sin(), q[:, :64] * d.sin() + q[:, 64:] * d.cos()), -1)
            wt = torch.softmax(r @ k.T * 128 ** -0.5, -1)
            want[b] = wt @ v
            # the terms of the model's bound: query's rounding (2^-11 of each dim: scores off by e, weights by 2 e and a
            # little), weights' (2^-11), sums (2^-18), f16's least step, the output's (2^-8)
            e = 128 ** -0.5 * (2.0 ** -11 + 2.0 ** -24 * 128 ** 0.5) * q.norm(dim=-1) * k.norm(dim=-1).max()
            spread = torch.einsum("ht,htd->hd", wt, (v[None] - want[b][:, None]).abs())
            bound[b] = (2.0 ** -8 * want[b].abs() + torch.expm1(2 * e)[:, None] * spread + (2.0 ** -11 + 2.0 ** -18) * (wt @ v.abs())
                        + 160 * 2.0 ** -28 * v.abs().max())
        check(out, (want, bound), what)

    plan = shared_plan(dv, 10)
    assert plan.num_items == 1 and plan.items_host[0, 2] == 10
    other = blocks[(at + 1) % 10]
    plan.items.view(-1, L.PLAN_ITEM_INTS)[0, 72 + at] = int(other)
    if at > 0:
        kept(L.decode_shared(dv.p, dv.q, kp, vp, dv.words, dv.q_pos, dv.rope, plan), "record")
        assert L.device_status(clear=True) == L.LAZY_DEV_LAYOUT
    last = dv.p.num_pool_blocks
    plan.items.view(-1, L.PLAN_ITEM_INTS)[0, 72 + at] = last
    words = dv.words.clone()
    words[:, at] = (words[:, at] & ~0x3FFFF) | last
    kept(L.decode_shared(dv.p, dv.q, kp, vp, words, dv.q_pos, dv.rope, plan), "id")
    assert L.device_status(clear=True) == L.LAZY_DEV_BAD_BLOCK_ID


# a block that is not in the pool is left out, and the document's others are attended at their own positions
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 1, 64), (32, 1, 128)])
@pytest.mark.parametrize("bad", [0, 3, 10])
def test_blocks_behind_a_bad_one_keep_their_positions(hq, hkv, d, bad):
    L = la()
    w = W.decode_zipf("f8bad", batch=2, hq=hq, hkv=hkv, d=d, docs_per_seq=1, doc_tokens=48, pool_docs=2, zipf_s=0.5, share=False,
                      suffix_tokens=900, seed=1840, shift=5000)
    dv, kp, vp, kv, vv = on_device(w, num_splits=1)
    words = dv.words.clone()
    words[1, bad] |= (1 << 18) - 1
    out = L.decode(dv.p, dv.q, kp, vp, words, dv.seq_lens, dv.q_pos, dv.rope)
    assert L.device_status(clear=True) == L.LAZY_DEV_BAD_BLOCK_ID
    segs = w.seq_segments(1)
    doc, at = (segs[0][0], bad) if bad < 3 else (segs[1][0], bad - 3)
    rest = M.attention(w, kv, vv)
    check(out[:1], (rest[0][:1], rest[1][:1]), "the other sequence")
    # in 64 bits without the block's tokens
    f = torch.as_tensor(w.rope_theta ** (-2.0 * np.arange(d // 2) / d), dtype=torch.float64, device="cuda")

    def rotate(x, n):
        c, s = torch.cos(n * f), torch.sin(n * f)
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat((a * c - b * s, a * s + b * c), -1)

    ks, vs, p = [], [], int(w.seq_pos0[1])
    for dc, n in segs:
        for b in range((n + 15) // 16):
            ph = int(w.doc_blocks[int(w.doc_block_indptr[dc]) + b])
            m = min(16, n - 16 * b)
            if not (dc == doc and b == at):
                ks.append(rotate(kv[ph, :, :m], float(p)))
                vs.append(vv[ph, :, :m])
        p += n
    k, v = torch.cat(ks, 1), torch.cat(vs, 1)
    q = rotate(w.q[1].double().cuda(), float(w.q_pos[1])).reshape(hkv, hq // hkv, d)
    wgt = torch.softmax(torch.einsum("hgd,htd->hgt", q, k) * d ** -0.5, -1)
    want = torch.einsum("hgt,htd->hgd", wgt, v).reshape(hq, d)
    check(out[1], (want, 1.5 * rest[1][1] + 2.0 ** -8 * want.abs()), "behind the bad block")


def test_noalloc_gives_the_same_bits():
    L = la()
    w = W.decode_zipf("f8na", batch=8, hq=32, hkv=8, d=128, docs_per_seq=6, doc_tokens=272, pool_docs=40, zipf_s=1.0, suffix_tokens=33,
                      seed=1743)
    dv, kp, vp, kv, vv = on_device(w)
    assert 0 < L.decode_workspace_bytes(dv.p) <= L.NOALLOC_SCRATCH_BYTES
    out = L.decode_noalloc(dv.p, dv.q, kp, vp, dv.words, dv.seq_lens, dv.q_pos, dv.rope, torch.empty_like(dv.q))
    assert torch.equal(out.view(torch.int16), decode(dv, kp, vp).view(torch.int16))
    check(out, M.attention(w, kv, vv), "decode_noalloc")


def test_two_decodes_at_once():
    # each call with its own workspace, on its own stream, several in flight
    L = la()
    dw, _ = W.mixed_mqa(n_decode=20, n_prefill=1, chunk=16, hq=16, hkv=2, d=128, pool_docs=40, ctx_lo=1, ctx_hi=4000, doc_lo=1, doc_hi=300,
                        seed=1716)
    dv, kp, vp, kv, vv = on_device(dw)
    alone = decode(dv, kp, vp)
    check(alone, M.attention(dw, kv, vv), "alone")
    n = L.decode_workspace_bytes(dv.p)
    runs = [(torch.cuda.Stream(), torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(dv.q)) for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, ws, out in runs:
            decode(dv, kp, vp, out=out, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for _, _, out in runs:
        assert torch.equal(out, alone)


@pytest.mark.parametrize("batch,hq,hkv,d,hi", [(4, 32, 8, 128, 4200), (3, 8, 1, 64, 9000), (96, 16, 8, 64, 3000), (3, 64, 1, 64, 12000)])
def test_width_of_the_table_changes_nothing(batch, hq, hkv, d, hi):
    # a table as wide as a captured step may need, with words of no meaning behind the sequences
    L = la()
    dw, _ = W.mixed_mqa(n_decode=batch, n_prefill=1, chunk=16, hq=hq, hkv=hkv, d=d, pool_docs=30, ctx_lo=1, ctx_hi=hi, doc_lo=1, doc_hi=700,
                        seed=1850 + batch)
    dv, kp, vp, kv, vv = on_device(dw)
    ref = M.attention(dw, kv, vv)
    check(decode(dv, kp, vp), ref, "as it is")
    for wide in (dv.p.max_blocks_per_seq + 7, 3001, 12000):
        words = torch.full((batch, wide), -1, dtype=torch.int32, device="cuda")
        words[:, :dv.words.shape[1]] = dv.words[:, :min(wide, dv.words.shape[1])]
        if wide < dv.words.shape[1]:
            continue
        for s, nb in enumerate((dv.seq_lens.cpu().numpy() + 15) // 16):
            words[s, nb:] = -1
        p2 = la().make_params(num_seqs=batch, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, num_pool_blocks=dv.p.num_pool_blocks,
                              max_blocks_per_seq=wide, rope_theta=dw.rope_theta, kv_dtype=KIND)
        check(L.decode(p2, dv.q, kp, vp, words, dv.seq_lens, dv.q_pos, dv.rope), ref, f"{wide} words a sequence")


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (64, 4, 128), (64, 1, 64)])
def test_captured_decodes_follow_their_inputs(hq, hkv, d):
    # both decodes in one graph on one workspace; queries, lengths and positions change between replays
    L = la()
    w = W.decode_zipf("f8graph", batch=12, hq=hq, hkv=hkv, d=d, docs_per_seq=4, doc_tokens=320, pool_docs=6, zipf_s=1.0, suffix_tokens=40,
                      seed=1861)
    dv, kp, vp, kv, vv = on_device(w)
    plan = shared_plan(dv)
    n = max(L.decode_workspace_bytes(dv.p), L.decode_shared_workspace_bytes(dv.p, plan.num_slots))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    one, two = torch.empty_like(dv.q), torch.empty_like(dv.q)

    def both():
        L.decode(dv.p, dv.q, kp, vp, dv.words, dv.seq_lens, dv.q_pos, dv.rope, out=one, workspace=ws)
        L.decode_shared(dv.p, dv.q, kp, vp, dv.words, dv.q_pos, dv.rope, plan, out=two, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    g = torch.Generator().manual_seed(5)
    for i in range(3):
        w.q = torch.randn(w.q.shape, generator=g).to(torch.bfloat16)
        w.q_pos = w.q_pos + 17 * i
        dv.q.copy_(w.q)
        dv.q_pos.copy_(torch.from_numpy(np.asarray(w.q_pos, dtype=np.int32)))
        ws.fill_(0xff)  # nothing is left over from a replay
        graph.replay()
        ref = M.attention(w, kv, vv)
        check(one, ref, f"replay {i}")
        check(two, ref, f"replay {i}, shared runs")
    cut = dv.seq_lens.clone()  # shorter sequences: as an eager call of those lengths
    dv.seq_lens.copy_(torch.clamp(cut - 333, min=0))
    dv.seq_lens[3] = 0
    graph.replay()
    assert torch.equal(one.view(torch.int16), decode(dv, kp, vp).view(torch.int16)) and not one[3].any()


def test_records_behind_4_gb():
    # the same records at the end of pools of more than 2^32 bytes: written, read back and attended to, bit for bit
    L = la()
    w = W.decode_zipf("f8far", batch=4, hq=32, hkv=8, d=128, docs_per_seq=3, doc_tokens=200, pool_docs=5, zipf_s=1.0, suffix_tokens=9, seed=1881)
    dv, kp, vp, kv, vv = on_device(w)
    n, n_far = w.num_pool_blocks, 1 << 18
    far = torch.arange(n_far - 1, n_far - 1 - n, -1, device="cuda")  # where block b goes
    p = L.make_params(num_seqs=4, num_q_heads=32, num_kv_heads=8, head_dim=128, num_pool_blocks=n_far,
                      max_blocks_per_seq=dv.p.max_blocks_per_seq, rope_theta=w.rope_theta, kv_dtype=KIND)
    big = L.empty_pools(p)
    assert big[0].numel() > 1 << 32
    for x, small in zip(big, (kp, vp)):
        x.fill_(0x7f)
        x[far] = small
    words = dv.words & ~0x3FFFF | far[(dv.words & 0x3FFFF).long()].int()
    for b in range(4):  # words behind the sequences stay 0
        words[b, (int(dv.seq_lens[b]) + 15) // 16:] = 0
    one = L.decode(p, dv.q, *big, words, dv.seq_lens, dv.q_pos, dv.rope)
    assert torch.equal(one.view(torch.int16), decode(dv, kp, vp).view(torch.int16))
    two = shared(dv, kp, vp)
    check(two, M.attention(w, kv, vv), "shared")
    w.doc_blocks, w.num_pool_blocks = (n_far - 1 - w.doc_blocks).astype(w.doc_blocks.dtype), n_far
    dv.p, dv.words = p, words
    assert torch.equal(shared(dv, *big).view(torch.int16), two.view(torch.int16))
    rng = np.random.default_rng(4)
    k, v = rows("normal", 16 * n, 8, 128, rng).cuda(), rows("outliers", 16 * n, 8, 128, rng).cuda()
    slots = torch.arange(16 * n, dtype=torch.int32, device="cuda")
    L.cache_write(p, k, v, 16 * far[slots.long() // 16].int() + slots % 16, *big)
    q = params(8, 128, n)
    near = L.empty_pools(q)
    L.cache_write(q, k, v, slots, *near)
    for x, y in zip(big, near):
        same_records(x[far], y.cpu().numpy(), 128)
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    for x, y in zip(L.cache_read(p, *big, far.int()), L.cache_read(q, *near, ids)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (8, 1, 64), (16, 1, 128), (64, 1, 128)])
def test_blocks_of_zero_bytes_are_keys_and_values_of_zero(hq, hkv, d):
    # as a pool is that was cleared and not written: codes and scales of 0
    w = W.decode_zipf("f8zero", batch=3, hq=hq, hkv=hkv, d=d, docs_per_seq=3, doc_tokens=140, pool_docs=4, zipf_s=0.7, seed=1891)
    dv, kp, vp, kv, vv = on_device(w)
    for doc in range(4):  # the first blocks of two documents, a later one of the others
        a = int(w.doc_block_indptr[doc])
        for b in ([0, 1, 2] if doc % 2 else [1, 5]):
            blk = int(w.doc_blocks[a + b])
            kp[blk], vp[blk], kv[blk], vv[blk] = 0, 0, 0, 0
    ref = M.attention(w, kv, vv)
    for splits in (0, 1, 3):
        dv.p.num_splits = splits
        check(decode(dv, kp, vp), ref, f"splits {splits}")
    check(shared(dv, kp, vp), ref, "shared")
    check(shared(dv, kp, vp, 2), ref, "shared, short items")
