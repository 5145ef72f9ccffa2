"""fp64 / integer oracle of the operators around the recurrence (kda_norm_quant, kda_fp8_matmul,
kda_batch_maps), written from their definitions with numpy loops; shares no code with the library."""
import numpy as np

E4M3_MAX = 448.0
GROUP = 128
SLOT_PAGES, SLOT_LENGTHS = 8, 16   # the error bits of kda_batch_maps


def e4m3_value(code):
    """The value of an e4m3 bit pattern (0..255)."""
    sign, exp, man = -1.0 if code & 0x80 else 1.0, (code >> 3) & 15, code & 7
    if exp == 15 and man == 7:
        return np.nan
    return sign * (man * 2.0 ** -9 if exp == 0 else (8 + man) * 2.0 ** (exp - 10))


E4M3_TABLE = np.array([e4m3_value(c) for c in range(256)])


def e4m3_values(codes):
    """fp64 values of a uint8 array of bit patterns."""
    return E4M3_TABLE[np.asarray(codes, np.uint8)]


def norm_quant(x, residual, weight, eps):
    """h, y, scales [N, G] and the unrounded y / s, all fp64. x, residual: [N, D]; weight [D] or None."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    y = h
    if weight is not None:
        y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    N, D = y.shape
    scales, v = np.empty((N, -(-D // GROUP))), np.empty_like(y)
    for g in range(scales.shape[1]):
        part = y[:, g * GROUP:(g + 1) * GROUP]
        top = np.max(np.abs(part), axis=1)          # keeps a NaN
        scales[:, g] = np.maximum(top, E4M3_MAX * 2.0 ** -126) / E4M3_MAX
        with np.errstate(invalid="ignore"):
            v[:, g * GROUP:(g + 1) * GROUP] = part / scales[:, g, None]
    return h, y, scales, v


def fp8_matmul(a, a_scales, w, w_scales):
    """(exact product, sum of the magnitudes of its terms); a [M, K], w [N, K] fp64 values of e4m3."""
    a, w = np.asarray(a, np.float64), np.asarray(w, np.float64)
    (M, K), N = a.shape, w.shape[0]
    k, n = np.arange(K) // GROUP, np.arange(N) // GROUP
    fa = a * np.asarray(a_scales, np.float64)[:, k]
    fw = w * np.asarray(w_scales, np.float64)[n][:, k]
    return fa @ fw.T, np.abs(fa) @ np.abs(fw).T


def batch_maps(q_lens, c_lens, state_slots, table, free_pages, free_count, page, num_pages, num_tokens):
    """The maps as a dict of arrays (block_table a new array) and the error bits, request by request."""
    R, width = table.shape
    table = table.copy()
    err = 0
    q, c = [int(v) for v in q_lens], [int(v) for v in c_lens]
    for r in range(R):
        if q[r] < 0 or c[r] < 0 or q[r] + c[r] > 2 ** 31 - 1:
            q[r] = c[r] = 0
            err |= SLOT_LENGTHS
    order = [r for r in range(R) if q[r] == 1] + [r for r in range(R) if q[r] != 1]
    decodes = sum(v == 1 for v in q)
    cu, rows = [0], 0
    for r in order:
        if rows + q[r] > num_tokens:
            err |= SLOT_LENGTHS
            q[r] = num_tokens - rows
        rows += q[r]
        cu.append(rows)
    left = min(max(int(free_count), 0), len(free_pages))
    for r in range(R):
        have, want = -(-c[r] // page), -(-(c[r] + q[r]) // page)
        if q[r] > 0 and want > width:
            err |= SLOT_PAGES
        for j in range(have, min(want, width)):
            table[r, j] = free_pages[left - 1] if left > 0 else -1
            err |= 0 if left > 0 else SLOT_PAGES
            left = max(left - 1, 0)
    positions, slots = np.zeros(num_tokens, np.int64), np.full(num_tokens, -1, np.int64)
    t = 0
    for r in order:
        for i in range(q[r]):
            p = c[r] + i
            positions[t] = p
            entry = int(table[r, p // page]) if p // page < width else -1
            if 0 <= entry < num_pages:
                slots[t] = entry * page + p % page
            else:
                err |= SLOT_PAGES
            t += 1
    return {"order": np.array(order, np.int64), "cu_seqlens": np.array(cu, np.int64),
            "state_indices": np.array([state_slots[r] for r in order], np.int64), "num_decodes": np.array([decodes]),
            "positions": positions, "slot_map": slots, "free_left": np.array([left]), "block_table": table}, err
