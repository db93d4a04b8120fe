"""Plain 64-bit restatement of the quantised pools' formats and of attention over them,
from their definitions in lazy_attn.h, and the error bounds that the tests use."""
from __future__ import annotations

import numpy as np

BLOCK = 16


def bf16_round(x: np.ndarray) -> np.ndarray:
    """To bf16, nearest even, as fp64. Exact inputs in fp64; NaN and infinities kept."""
    f = np.asarray(x, np.float64).astype(np.float32)
    u = f.view(np.uint32)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(f), r, f).astype(np.float64)


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """Bit patterns (uint16) of values that bf16 holds."""
    return (np.asarray(x, np.float64).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def int4_quantise(x: np.ndarray):
    """Codes [..., d], scales and zeros [..., d / 64] (fp64) of rows [..., d] of bf16 values."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 64)
    finite = np.isfinite(g).all(-1)
    g = np.where(finite[..., None], g, 0.0)
    z, hi = g.min(-1), g.max(-1)
    s = bf16_round((hi - z) / 15.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s[..., None] > 0, np.rint((g - z[..., None]) / s[..., None]), 0.0)
    c = np.clip(c, 0, 15).astype(np.uint8)
    s, z = np.where(finite, s, np.nan), np.where(finite, z, np.nan)
    return c.reshape(x.shape), s, z


def int4_place(d: int):
    """(byte, shift) of every dim's code within a row."""
    G = d // 64
    e = np.arange(d)
    word = G * ((e % 64) // 8) + e // 64
    return 4 * word + (e % 8) // 2, 4 * (e % 2)


def v_row(t):
    return (t & 8) + 4 * (t & 1) + ((t & 7) >> 1)


def record_bytes(d: int) -> int:
    return BLOCK * d // 2 + BLOCK * (d // 64) * 4


def int4_put(pool: np.ndarray, block: int, head: int, tok: int, x: np.ndarray, is_v: bool) -> None:
    """Writes one row of d values into pool [blocks, heads, record] (uint8)."""
    d = x.shape[-1]
    c, s, z = int4_quantise(x)
    byte, shift = int4_place(d)
    row = np.zeros(d // 2, np.uint8)
    np.bitwise_or.at(row, byte, (c << shift).astype(np.uint8))
    r = v_row(tok) if is_v else tok
    rec = pool[block, head]
    rec[r * d // 2:(r + 1) * d // 2] = row
    G = d // 64
    for j in range(G):
        at = BLOCK * d // 2 + 4 * (tok * G + j)
        nan = np.isnan(s[j])
        sb, zb = (0x7FC0, 0x7FC0) if nan else (int(bf16_bits(s[j])), int(bf16_bits(z[j])))
        rec[at:at + 4] = np.array([sb | zb << 16], "<u4").view(np.uint8)


def int4_values(pool: np.ndarray, d: int, is_v: bool) -> np.ndarray:
    """fp64 values [..., 16, d] of records [..., record]."""
    pool = np.asarray(pool)
    byte, shift = int4_place(d)
    G, t = d // 64, np.arange(BLOCK)
    rows = v_row(t) if is_v else t
    code = (pool[..., (rows[:, None] * (d // 2) + byte[None]).ravel()].reshape(*pool.shape[:-1], BLOCK, d) >> shift) & 15
    meta = np.ascontiguousarray(pool[..., BLOCK * d // 2:]).view("<u4").reshape(*pool.shape[:-1], BLOCK, G)
    with np.errstate(invalid="ignore"):
        s = ((meta & 0xFFFF) << 16).astype(np.uint32).view(np.float32).astype(np.float64)
        z = (meta & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)
        return code * np.repeat(s, 64, -1) + np.repeat(z, 64, -1)


def int4_pools(w):
    """int4 pools (uint8 torch tensors) of a workload's bf16 pools, whole blocks at a time. Hole slots and
    unused blocks hold NaN, as in the workload."""
    import torch
    out = []
    for src, is_v in ((w.k_pool, False), (w.v_pool, True)):
        x = src.double().numpy()
        nb, h, _, d = x.shape
        pool = np.zeros((nb, h, record_bytes(d)), np.uint8)
        c, s, z = int4_quantise(x)
        byte, shift = int4_place(d)
        rows = np.zeros((nb, h, BLOCK, d // 2), np.uint8)
        for e in range(d):
            rows[..., byte[e]] |= c[..., e] << np.uint8(shift[e])
        order = np.array([v_row(t) if is_v else t for t in range(BLOCK)])
        placed = np.empty_like(rows)
        placed[:, :, order] = rows
        pool[..., :BLOCK * d // 2] = placed.reshape(nb, h, -1)
        sb = np.where(np.isnan(s), 0x7FC0, bf16_bits(np.nan_to_num(s))).astype(np.uint32)
        zb = np.where(np.isnan(z), 0x7FC0, bf16_bits(np.nan_to_num(z))).astype(np.uint32)
        pool[..., BLOCK * d // 2:] = np.ascontiguousarray((sb | zb << 16).astype("<u4")).view(np.uint8).reshape(nb, h, -1)
        out.append(torch.from_numpy(pool))
    return out


def e4m3_codes(y: np.ndarray) -> np.ndarray:
    """Nearest e4m3 codes (ties to even, saturated) of fp64 values: by search in the table of the 127 finite values."""
    table = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                      for e in range(16) for m in range(8)][:127])
    a = np.minimum(np.abs(y), 448.0)
    nan = np.isnan(a)
    a = np.where(nan, 0.0, a)
    hi = np.clip(np.searchsorted(table, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - table[lo], table[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(table[hi] == a, hi, c)
    return np.where(nan, 0x7F, c | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def attention(w, k_values, v_values, lazy=True, freqs=None, sm_scale=0.0):
    """fp64 decode of workload ``w`` over pools of fp64 values [blocks, heads, 16, d] (torch, any device), and the bound
    on an int4 kernel's error, elementwise:
      2^-8 |out|                 the output's rounding to bf16 (half a step);
      e sum_j w_j |v_j - out|    the query's rounding to f16, as q - q'/16 and q'/16 of neighbouring dims (q, q'): the dims
                                 are off by 2^-11 (|q| + |q'| / 8) and 2^-11 |q'|, every score by at most
                                 e = scale * 2^-11 * 9/8 * |q| max_j |k_j|, a weight by that share;
      2^-10 sum_j w_j |v_j - z_j|  the rounding of the weights and of weight times scale to f16, times what they multiply:
                                 s c <= 15 s = max - min of the key's group, taken as 2 max|v_j| over the group;
      2^-18 sum_j w_j |v_j|      fp32 sums, exponentials and angles (5e-7 rad, 2^-20.9)."""
    import torch
    dev = k_values.device
    hq, hkv, d = w.num_q_heads, w.num_kv_heads, w.head_dim
    f = torch.as_tensor(w.rope_theta ** (-2.0 * np.arange(d // 2) / d) if freqs is None else freqs, dtype=torch.float64,
                        device=dev)
    scale = sm_scale or d ** -0.5

    def rotate(x, n):
        c, s = torch.cos(n[:, None, None] * f), torch.sin(n[:, None, None] * f)
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat((a * c - b * s, a * s + b * c), -1)

    out = torch.zeros((w.num_seqs, hq, d), dtype=torch.float64, device=dev)
    bound = torch.zeros_like(out)
    for i in range(w.num_seqs):
        ks, vs, pos, p = [], [], [], int(w.seq_pos0[i])
        for doc, n in w.seq_segments(i):
            a = int(w.doc_block_indptr[doc])
            blk = torch.as_tensor(w.doc_blocks[a:a + (n + 15) // 16].astype(np.int64), device=dev)
            for src, dst in ((k_values, ks), (v_values, vs)):
                dst.append(src[blk].transpose(1, 2).reshape(-1, hkv, d)[:n])
            pos.append(torch.full((n,), float(p), dtype=torch.float64, device=dev))
            p += n
        if not ks:
            continue
        k, v, pos = torch.cat(ks), torch.cat(vs), torch.cat(pos)
        if lazy:
            k = rotate(k, pos)
        q = rotate(w.q[i].double().to(dev)[None], torch.tensor([float(w.q_pos[i])], dtype=torch.float64, device=dev))[0]
        q = q.reshape(hkv, hq // hkv, d)
        wgt = torch.softmax(torch.einsum("hgd,thd->hgt", q, k) * scale, -1)
        o = torch.einsum("hgt,thd->hgd", wgt, v)
        e = scale * 2.0 ** -11 * 9 / 8 * q.norm(dim=-1) * k.norm(dim=-1).amax(0)[:, None]
        big = v.abs().reshape(-1, hkv, d // 64, 64).amax(-1)
        spread = torch.einsum("hgt,thj->hgj", wgt, 2 * big).repeat_interleave(64, -1)
        mean = torch.einsum("hgt,thd->hgd", wgt, v.abs())
        dev_o = torch.stack([torch.einsum("gt,tgd->gd", wgt[h], (v[:, h, None] - o[h][None]).abs()) for h in range(hkv)])
        out[i] = o.reshape(hq, d)
        bound[i] = (2.0 ** -8 * o.abs() + e[..., None] * dev_o + 2.0 ** -10 * spread + 2.0 ** -18 * mean).reshape(hq, d)
    return out, bound
