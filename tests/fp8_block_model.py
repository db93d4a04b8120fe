"""Plain 64-bit restatement of pools of e4m3 codes with block scales, of attention over them and of
the tables of new tokens, from their definitions in lazy_attn.h, and the bound that the tests use."""
from __future__ import annotations

import numpy as np

from int4_model import e4m3_codes

BLOCK, E_MIN, E_MAX = 16, -100, 119


def record_bytes(d: int) -> int:
    return BLOCK * d + 32


def place(d: int, is_v: bool) -> np.ndarray:
    """[16, d]: byte of a token's dim in a record."""
    out = np.full((BLOCK, d), -1)
    for j in range(d // 32):
        for g in range(8):
            for t in range(4):
                at = 16 * (32 * j + 4 * g + t)
                for i in range(16):
                    if is_v:
                        out[2 * (t + 4 * (j // (d // 64))) + i % 2, 8 * (g + 8 * (j % (d // 64))) + i // 2] = at + i
                    else:
                        out[g + 8 * (j % 2), 16 * (t + 4 * (j // 2)) + i] = at + i
    assert sorted(out.ravel()) == list(range(BLOCK * d))
    return out


def exponent(x) -> int:
    """The least e with 448 * 2^e >= every finite |x|."""
    m = np.abs(np.asarray(x, np.float64))
    m = m[np.isfinite(m)].max(initial=0.0)
    e = E_MIN
    while e < E_MAX and 448.0 * 2.0 ** e < m:
        e += 1
    return e


E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)])
E4M3 = np.concatenate([E4M3, -E4M3])
E4M3[[127, 255]] = np.nan


def scale_of(rec: np.ndarray, d: int) -> float:
    return float(np.frombuffer(np.ascontiguousarray(rec[BLOCK * d:BLOCK * d + 4]).tobytes(), "<f4")[0])


def put(rec: np.ndarray, rows: dict, is_v: bool) -> None:
    """Writes rows {token of the block: d values} of one call into a record (uint8), in place."""
    d = len(next(iter(rows.values())))
    at = place(d, is_v)
    e = exponent(np.concatenate([np.atleast_1d(x) for x in rows.values()]))
    if 0 in rows:
        rec[:BLOCK * d] = 0
    else:
        s = scale_of(rec, d)
        e_old = int(np.log2(s))
        old = E4M3[rec[at]] * s
        e = max(e, e_old)
        if e > e_old:
            rec[at] = e4m3_codes(old / 2.0 ** e)
    for t, x in rows.items():
        y = np.where(np.isfinite(x), np.asarray(x, np.float64), np.nan) / 2.0 ** e
        rec[at[t]] = e4m3_codes(y)
    rec[BLOCK * d:BLOCK * d + 4] = np.frombuffer(np.array([2.0 ** e], "<f4").tobytes(), np.uint8)


def values(pool: np.ndarray, d: int, is_v: bool) -> np.ndarray:
    """fp64 values [..., 16, d] of records [..., record]."""
    pool = np.ascontiguousarray(pool)
    s = np.ascontiguousarray(pool[..., BLOCK * d:BLOCK * d + 4]).view("<f4")[..., 0].astype(np.float64)
    with np.errstate(invalid="ignore"):
        return E4M3[pool[..., place(d, is_v)]] * s[..., None, None]


def pools(w):
    """Pools (uint8 torch tensors) of a workload's bf16 pools, whole blocks at a time. Hole slots and unused blocks hold
    NaN, as in the workload."""
    import torch
    out = []
    for src, is_v in ((w.k_pool, False), (w.v_pool, True)):
        x = src.double().numpy()
        nb, h, _, d = x.shape
        pool = np.zeros((nb, h, record_bytes(d)), np.uint8)
        m = np.nan_to_num(np.abs(x)).max((-1, -2))
        e = np.clip(np.ceil(np.log2(np.where(m > 0, m, 2.0 ** -90) / 448.0)), E_MIN, E_MAX)
        e += 448.0 * 2.0 ** e < m
        pool[..., place(d, is_v)] = e4m3_codes(x / (2.0 ** e)[..., None, None])
        pool[..., BLOCK * d:BLOCK * d + 4] = np.ascontiguousarray((2.0 ** e).astype("<f4")[..., None]).view(np.uint8)
        out.append(torch.from_numpy(pool))
    return out


def attention(w, k_values, v_values, lazy=True, sm_scale=0.0):
    """fp64 decode of workload ``w`` over pools of fp64 values [blocks, heads, 16, d] (torch, any device), and the bound on
    a kernel's error, elementwise:
      2^-8 |out|                 the output's rounding to bf16 (half a step);
      e sum_j w_j |v_j - out|    the query's rounding to f16: dims are off by 2^-11 of themselves (and 2^-25 of the row's
                                 largest, in what f16 has below its normal numbers), a score by at most
                                 scale * (2^-11 + 2^-24 sqrt(d)) |q| max_j |k_j|, a weight by that share;
      2^-11 sum_j w_j |v_j|      the rounding of weight times scale to f16;
      2^-18 sum_j w_j |v_j|      fp32 sums, exponentials and angles (5e-7 rad, 2^-20.9);
      n 2^-28 max_j |v_j|        f16's least step: weight times scale is off by 2^-25 where it is below 2^-14, times a code of
                                 at most 448, over a reference that puts the largest V scale at 2^4 at least; 448 times that
                                 scale is at most twice the head's largest value, and the row's weights sum to 1 at least."""
    import torch
    dev = k_values.device
    hq, hkv, d = w.num_q_heads, w.num_kv_heads, w.head_dim
    f = torch.as_tensor(w.rope_theta ** (-2.0 * np.arange(d // 2) / d), dtype=torch.float64, device=dev)
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
        e = scale * (2.0 ** -11 + 2.0 ** -24 * d ** 0.5) * q.norm(dim=-1) * k.norm(dim=-1).amax(0)[:, None]
        mean = torch.einsum("hgt,thd->hgd", wgt, v.abs())
        off = torch.stack([torch.einsum("gt,tgd->gd", wgt[h], (v[:, h, None] - o[h][None]).abs()) for h in range(hkv)])
        out[i] = o.reshape(hq, d)
        tiny = len(k) * 2.0 ** -28 * v.abs().amax((0, 2))[:, None, None]
        bound[i] = (2.0 ** -8 * o.abs() + e[..., None] * off + (2.0 ** -11 + 2.0 ** -18) * mean + tiny).reshape(hq, d)
    return out, bound
