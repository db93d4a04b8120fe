"""The tables of new tokens, sequence by sequence, from their definition in lazy_attn.h."""
import numpy as np

BLOCK = 16
NO_BLOCKS, BAD_LEN, LAYOUT, BAD_ID = 0x20, 0x10, 0x8, 0x1


def append(new_lens, seq_lens, pos, tail_start, free, words, num_rows, *, max_blocks, id_bits, pool, first=0, doc=4096,
           key_positions=False):
    """(words, seq_lens, pos, q_start, cu_rows, block_indptr, slots, local_pos, status bits); words uint32."""
    words = words.copy()
    status = 0
    if first < 0 or first > len(free):
        first, status = len(free), LAYOUT
    at, row = first, 0  # `wanted`: where the list would stand had every sequence got its blocks
    wanted = first
    out_len, out_pos, cu, indptr = [], [], [0], [first]
    slots, local = np.full(num_rows, -1, np.int64), np.zeros(num_rows, np.int64)
    half = 1 << (31 - id_bits)
    closed = False
    for s, (n, used, p, a) in enumerate(zip(*(map(int, x) for x in (new_lens, seq_lens, pos, tail_start)))):
        if n < 0:
            n, status = 0, status | BAD_LEN
        row += n
        ok, need, tail = n > 0, 0, p - a
        if ok and not 0 <= used <= BLOCK * max_blocks:
            ok, status = False, status | BAD_LEN
        if ok:
            fits = p >= 0 and 0 <= tail <= used and (tail == 0 or (used - tail) % BLOCK == 0) and p + n < 2 ** 31
            if fits:
                b0 = -(-used // BLOCK) - -(-tail // BLOCK)
                have, end = -(-tail // BLOCK), -(-(tail + n) // BLOCK)
                offs = [BLOCK * (b0 + j) - (a + (BLOCK * j if key_positions else (BLOCK * j // doc * doc if doc else 0)))
                        for j in range(have, end)]
                fits = b0 + end <= max_blocks and all(-half <= o < half for o in offs)
            if fits:
                need = end - have
            else:
                ok, status = False, status | LAYOUT
        if ok:
            wanted += need
            if row > num_rows:
                ok, status = False, status | BAD_LEN
            elif need and wanted > len(free):
                ok, status = False, status | NO_BLOCKS
            if not ok and need:
                closed = True
        if ok:
            assert not (closed and need)
            ids = free[at:at + need]
            at += need
            for j, (i, o) in enumerate(zip(ids, offs)):
                good = 0 <= i < pool
                status |= 0 if good else BAD_ID
                words[s, b0 + have + j] = ((o << id_bits) & 0xFFFFFFFF) | (int(i) if good else (1 << id_bits) - 1)
            for i in range(n):
                t = tail + i
                j = t // BLOCK
                phys = int(words[s, b0 + j]) & ((1 << id_bits) - 1) if j < have else int(ids[j - have])
                if 0 <= phys < pool:
                    slots[row - n + i] = phys * BLOCK + t % BLOCK
                else:
                    status |= BAD_ID
                local[row - n + i] = t % doc if doc else t
            used, p = BLOCK * b0 + tail + n, p + n
        out_len.append(used)
        out_pos.append(p)
        cu.append(min(row, 2 ** 31 - 1))
        indptr.append(at)
    i32 = lambda x: np.asarray(x, np.int64).astype(np.int32)
    return words, i32(out_len), i32(out_pos), i32(pos), i32(cu), i32(indptr), i32(slots), i32(local), status
