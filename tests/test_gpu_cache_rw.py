"""GPU: rows written into the pools and blocks read back, bit for bit against the formats'
restatement in 64 bits (tests/int4_model.py)."""
import numpy as np
import pytest
import torch

import int4_model as M
from gpu_util import la

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    la().device_status(clear=True)
    yield
    assert la().device_status(clear=True) == 0, "device status word set"


def params(kv, hkv, d, blocks, dtype="bf16", **kw):
    return la().make_params(num_seqs=0, num_q_heads=hkv, num_kv_heads=hkv, head_dim=d, num_pool_blocks=blocks,
                            max_blocks_per_seq=0, dtype=dtype, kv_dtype=kv, **kw)


def filled_pools(p, seed):
    """Pools of random bytes on the GPU (what was there before) and their copies."""
    L = la()
    g = torch.Generator().manual_seed(seed)
    pools = L.empty_pools(p)
    for x in pools:
        n = x.numel() * x.element_size()
        x.view(torch.uint8).view(-1).copy_(torch.randint(0, 256, (n,), dtype=torch.uint8, generator=g))
    return pools, [x.view(torch.uint8).cpu().clone() for x in pools]


def rows(kind, t, h, d, rng):
    x = rng.standard_normal((t, h, d))
    if kind == "outliers":
        x[..., :: 16] *= 50
    elif kind == "relu":
        x = np.maximum(x, 0) + 1e-9 * (rng.random(x.shape) < 0.1)
    elif kind == "borders":  # halves of a step of 1 around a least value just off zero: ties, and values next to them
        x = rng.integers(0, 31, x.shape) / 2.0
        x[..., 0::64], x[..., 1::64] = rng.choice([0.0, -1e-9, 1e-9, -2.0 ** -20], x[..., 0::64].shape), 15.0
    elif kind == "flat":
        x = np.broadcast_to(x[..., :1], x.shape).copy()
        x[..., 1::64] += np.where(rng.random(x[..., 1::64].shape) < 0.5, 2.0 ** -7, 0)
    elif kind == "extremes":
        x = x * 10.0 ** rng.integers(-37, 38, (t, h, 1))
    elif kind == "bad":  # groups with infinities and NaN next to whole ones
        x[rng.random(x.shape) < 0.004] = np.nan
        x[rng.random(x.shape) < 0.004] = np.inf
        x[rng.random(x.shape) < 0.004] = -np.inf
    return torch.from_numpy(x).to(torch.bfloat16)


def scatter(slots, pool, x, is_v, kv, d, scale=1.0):
    """The expected bytes: `pool` with x's rows put in their slots."""
    xs = x.double().numpy()
    for t, s in enumerate(slots):
        if s < 0:
            continue
        b, r = divmod(int(s), 16)
        for h in range(xs.shape[1]):
            if kv == "int4":
                M.int4_put(pool, b, h, r, xs[t, h], is_v)
            else:
                pool[b, h, r] = M.e4m3_codes(xs[t, h] / scale)


@pytest.mark.parametrize("kind", ["normal", "outliers", "relu", "borders", "flat", "extremes", "bad"])
@pytest.mark.parametrize("hkv,d,t", [(8, 128, 37), (3, 64, 50)])
def test_int4_write_bytes(kind, hkv, d, t):
    L = la()
    rng = np.random.default_rng(7 + d)
    p = params("int4", hkv, d, 9)
    (kp, vp), (k0, v0) = filled_pools(p, 1)
    k, v = rows(kind, t, hkv, d, rng), rows(kind, t, hkv, d, rng)
    slots = rng.permutation(9 * 16)[:t].astype(np.int32)
    slots[rng.random(t) < 0.2] = -1
    L.cache_write(p, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), kp, vp)
    for got, want, x, is_v in ((kp, k0.numpy(), k, False), (vp, v0.numpy(), v, True)):
        scatter(slots, want, x, is_v, "int4", d)
        got = got.cpu().numpy()
        # a NaN's bits are one pattern; a zero's sign is free where a group's least value is 0
        m = M.BLOCK * d // 2
        assert np.array_equal(got[..., :m], want[..., :m])
        a, b = (np.ascontiguousarray(y[..., m:]).view("<u2") for y in (got, want))
        assert (((a == b) | ((a & 0x7FFF) + (b & 0x7FFF) == 0))).all()


def test_int4_codes_beside_ties():
    # groups from -(j + 1/2) s to (14.5 - j) s with s a power of two: 0 is a tie of two codes, and a value 2^-k s off it,
    # k = 0 .. 40, lies on one side however little it moves the difference to the least value; beside them the least
    # value itself off zero by as little, with ties and halves elsewhere
    L = la()
    rng = np.random.default_rng(11)
    t, h, d = 400, 2, 64
    p = params("int4", h, d, t // 16)
    x = rng.choice([-1.0, 1.0], (t, h, d)) * 2.0 ** -rng.integers(0, 41, (t, h, d))
    x[rng.random(x.shape) < 0.1] = 0.0
    j = rng.integers(0, 15, (t, h))
    x[..., 0], x[..., 1] = -(j + 0.5), 14.5 - j
    off = x[::4, :, 2].copy()
    x[::4] = rng.integers(0, 31, x[::4].shape) / 2.0
    x[::4, :, 0], x[::4, :, 1] = off * 2.0 ** -6, 15.0
    x *= 2.0 ** rng.integers(-60, 61, (t, h, 1))
    x = torch.from_numpy(x).to(torch.bfloat16)
    (kp, vp), (k0, v0) = filled_pools(p, 12)
    slots = np.arange(t, dtype=np.int32)
    L.cache_write(p, x.cuda(), x.cuda(), torch.from_numpy(slots).cuda(), kp, vp)
    for got, want, is_v in ((kp, k0.numpy(), False), (vp, v0.numpy(), True)):
        scatter(slots, want, x, is_v, "int4", d)
        m = M.BLOCK * d // 2
        assert np.array_equal(got.cpu().numpy()[..., :m], want[..., :m])


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -6, 5.5 / 448, 3.3e-7, 7.0 / 448, 1.1e20])
def test_e4m3_write_of_every_bf16_value(scale):
    # 65536 patterns: ties, subnormal codes, saturation, infinities and NaN
    L = la()
    scale = float(np.float32(scale))
    p = params("fp8_e4m3", 8, 128, 4, k_scale=scale, v_scale=scale)
    (kp, vp), _ = filled_pools(p, 2)
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(64, 8, 128)
    slots = torch.arange(64, dtype=torch.int32)
    L.cache_write(p, x.cuda(), x.flip(0).cuda(), slots.cuda(), kp, vp)
    for got, y in ((kp, x), (vp, x.flip(0))):
        got = got.view(torch.uint8).cpu().numpy().transpose(0, 2, 1, 3).reshape(64, 8, 128)
        y = y.double().numpy()
        want = M.e4m3_codes(y / scale)  # x has 8 bits and the scale 24: the fp64 quotient is next to a tie only on one
        nan = np.isnan(y)
        assert np.array_equal(got[~nan], want[~nan])
        assert ((got[nan] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("kv,dtype,d", [(None, "bf16", 128), (None, "f32", 64), (None, "f32", 128), (None, "bf16", 64)])
def test_copy_write_and_read(kv, dtype, d):
    L = la()
    p = params(kv, 3, d, 6, dtype)
    (kp, vp), (k0, v0) = filled_pools(p, 3)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    k, v = (torch.randn(41, 3, d, generator=torch.Generator().manual_seed(s)).to(dt) for s in (1, 2))
    slots = torch.randperm(96, generator=torch.Generator().manual_seed(3))[:41].to(torch.int32)
    slots[5] = -3
    L.cache_write(p, k.cuda(), v.cuda(), slots.cuda(), kp, vp)
    ids = torch.tensor([5, 0, 0, 3], dtype=torch.int32).cuda()
    ko, vo = L.cache_read(p, kp, vp, ids)
    for got, was, x, back in ((kp, k0, k, ko), (vp, v0, v, vo)):
        want = was.view(dt).view(6, 3, 16, d)
        keep = slots >= 0
        want[slots[keep].long() // 16, :, slots[keep].long() % 16] = x[keep]
        bits = torch.int16 if dtype == "bf16" else torch.int32
        assert torch.equal(got.cpu().view(bits), want.view(bits))
        assert torch.equal(back.cpu().view(bits), want[ids.cpu().long()].view(bits))


# token and head strides: slices of a fused product, heads first, an odd stride and an odd
# start (no 16-byte loads), one token repeated by a stride of zero
@pytest.mark.parametrize("layout", ["fused", "heads_first", "odd", "odd_start", "broadcast"])
@pytest.mark.parametrize("kv,d", [("int4", 128), ("int4", 64), ("fp8_e4m3", 128), (None, 128)])
def test_write_strides(layout, kv, d):
    L = la()
    h, t = 5, 23
    g = torch.Generator().manual_seed(4)
    if layout == "fused":
        x = torch.randn(t, 3 * h, d, generator=g).to(torch.bfloat16).cuda()
        k, v = x[:, h:2 * h], x[:, 2 * h:]
    elif layout == "heads_first":
        x = torch.randn(2, h, t, d, generator=g).to(torch.bfloat16).cuda()
        k, v = x[0].transpose(0, 1), x[1].transpose(0, 1)
    elif layout == "broadcast":
        x = torch.randn(2, 1, h, d, generator=g).to(torch.bfloat16).cuda()
        k, v = x[0].expand(t, h, d), x[1].expand(t, h, d)
    else:
        x = torch.randn(2, t, h, d + (3 if layout == "odd" else 8), generator=g).to(torch.bfloat16).cuda()
        o = 0 if layout == "odd" else 1
        k, v = x[0, ..., o:o + d], x[1, ..., o:o + d]
    p = params(kv, h, d, 5)
    slots = torch.randperm(80, generator=g)[:t].to(torch.int32).cuda()
    (ka, va), _ = filled_pools(p, 5)
    kb, vb = ka.clone(), va.clone()
    L.cache_write(p, k, v, slots, ka, va)
    L.cache_write(p, k.contiguous(), v.contiguous(), slots, kb, vb)
    assert torch.equal(ka.view(torch.uint8), kb.view(torch.uint8)) and torch.equal(va.view(torch.uint8), vb.view(torch.uint8))
    for pool, src, is_v in ((ka, k, False), (va, v, True)):  # and they are the rows
        xs = src.cpu().double().numpy()
        s = slots.cpu().numpy()
        if kv == "int4":
            got = M.int4_values(pool.cpu().numpy(), d, is_v)
            c, sc, z = M.int4_quantise(xs)
            want = c * np.repeat(sc, 64, -1) + np.repeat(z, 64, -1)
        else:
            got = pool.float().cpu().double().numpy()
            want = xs if kv is None else torch.from_numpy(M.e4m3_codes(xs)).view(torch.float8_e4m3fn).double().numpy()
        assert np.array_equal(got[s // 16, :, s % 16], want)


@pytest.mark.parametrize("kv", ["int4", "fp8_e4m3", None])
def test_write_skips_and_reports_bad_slots(kv):
    L = la()
    p = params(kv, 2, 128, 3)
    (kp, vp), (k0, v0) = filled_pools(p, 6)
    x = torch.randn(4, 2, 128).to(torch.bfloat16).cuda()
    L.cache_write(p, x, x, torch.tensor([-1, -2 ** 31, 48, 2 ** 31 - 1], dtype=torch.int32).cuda(), kp, vp)
    assert L.device_status(clear=True) == L.LAZY_DEV_BAD_BLOCK_ID
    assert torch.equal(kp.view(torch.uint8).cpu(), k0) and torch.equal(vp.view(torch.uint8).cpu(), v0)
    L.cache_write(p, x[:0], x[:0], torch.zeros(0, dtype=torch.int32).cuda(), kp, vp)
    assert torch.equal(kp.view(torch.uint8).cpu(), k0)


@pytest.mark.parametrize("kv,hkv,d,n", [("int4", 8, 128, 33), ("int4", 1, 64, 7), ("int4", 5, 64, 1), ("fp8_e4m3", 3, 128, 9),
                                        ("fp8_e4m3", 2, 64, 20)])
def test_read_values(kv, hkv, d, n):
    L = la()
    kw = dict(k_scale=0.37, v_scale=2.5) if kv == "fp8_e4m3" else {}
    p = params(kv, hkv, d, 40, **kw)
    (kp, vp), _ = filled_pools(p, 7)
    rng = np.random.default_rng(8)
    if kv == "int4":  # scales and zeros of every size, none that is not finite
        for pool in (kp, vp):
            m = np.stack([rng.choice([0.0, 1e-30, 0.25, 3.0, 1e30], (40, hkv, 16 * d // 64)),
                          rng.standard_normal((40, hkv, 16 * d // 64)) * 10], -1)
            pool[..., 16 * d // 2:] = torch.from_numpy(m).to(torch.bfloat16).cuda().view(torch.uint8).flatten(-2)
    ids = rng.integers(0, 40, n).astype(np.int32)
    if n > 8:
        ids[[2, 5]] = -1, ids[4]
    ko = torch.full((n, hkv, 16, d), 77.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    L.cache_read(p, kp, vp, torch.from_numpy(ids).cuda(), ko, vo)
    for pool, got, is_v, scale in ((kp, ko, False, p.k_scale), (vp, vo, True, p.v_scale)):
        got = got.float().cpu().double().numpy()
        if kv == "int4":
            want = M.int4_values(pool.cpu().numpy(), d, is_v)
        else:
            want = pool.float().cpu().double().numpy() * scale
        want = want[np.maximum(ids, 0)]
        want[ids < 0] = 77.0
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(got), nan)
        # the product and sum in fp32 (2^-24 of it), then half a step of bf16
        assert (np.abs(got - want)[~nan] <= np.abs(want[~nan]) * (2.0 ** -8 + 2.0 ** -22)).all()


def test_read_reports_bad_ids():
    L = la()
    p = params("int4", 2, 128, 3)
    (kp, vp), _ = filled_pools(p, 9)
    out = torch.full((3, 2, 16, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    vout = out.clone()
    L.cache_read(p, kp, vp, torch.tensor([3, -1, 2 ** 31 - 1], dtype=torch.int32).cuda(), out, vout)
    assert L.device_status(clear=True) == L.LAZY_DEV_BAD_BLOCK_ID
    assert (out == 5.0).all() and (vout == 5.0).all()


def test_group_that_is_not_finite_reads_back_as_nan():
    L = la()
    p = params("int4", 1, 128, 1)
    (kp, vp), _ = filled_pools(p, 10)
    x = torch.randn(3, 1, 128).to(torch.bfloat16)
    x[0, 0, 3], x[1, 0, 70], x[2, 0, 127] = float("inf"), float("nan"), float("-inf")
    L.cache_write(p, x.cuda(), x.cuda(), torch.tensor([0, 1, 2], dtype=torch.int32).cuda(), kp, vp)
    for out in L.cache_read(p, kp, vp, torch.zeros(1, dtype=torch.int32).cuda()):
        nan = torch.isnan(out[0, 0, :3].float()).cpu()
        assert nan[0, :64].all() and not nan[0, 64:].any()
        assert not nan[1, :64].any() and nan[1, 64:].all() and nan[2, 64:].all()


def test_many_tokens_and_blocks():
    # more rows than one pass of the grid takes, and more records
    L = la()
    t, h, d, blocks = 40000, 8, 64, 2600
    p = params("int4", h, d, blocks)
    kp, vp = (torch.zeros_like(x) for x in L.empty_pools(p))
    x = torch.randn(t, h, d, device="cuda").to(torch.bfloat16)
    slots = torch.randperm(blocks * 16, device="cuda")[:t].to(torch.int32)
    L.cache_write(p, x, -x, slots, kp, vp)
    ko, vo = L.cache_read(p, kp, vp, torch.arange(blocks, dtype=torch.int32, device="cuda"))
    step = (x.float().amax(-1, keepdim=True) - x.float().amin(-1, keepdim=True)) / 15
    at = slots.long()
    for got, want in ((ko, x.float()), (vo, -x.float())):
        err = (got[at // 16, :, at % 16].float() - want).abs()
        # half a step, the scale's rounding over 15 steps, the value's rounding to bf16
        assert (err <= step * (0.5 + 15 * 2.0 ** -8) + want.abs() * 2.0 ** -7).all()
    rest = torch.ones(blocks * 16, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (ko.transpose(1, 2).reshape(-1, h, d)[rest] == 0).all()
