"""Definitions of the pieces of an expert layer: the slots' sort by expert,
rows copied for their experts and summed back, and dropout."""
import numpy as np


def sort_slots(idx, num_local, begin=0):
    """(slot_row [T, k], offsets [num_local + 1], row_src [R]) of expert numbers
    idx [T, k]: one expert after the other, its slots in ascending order."""
    flat = np.asarray(idx).reshape(-1)
    slot_row = np.full(flat.size, -1, dtype=np.int64)
    offsets, row_src = [0], []
    for e in range(begin, begin + num_local):
        slots = np.nonzero(flat == e)[0]
        slot_row[slots] = np.arange(slots.size) + offsets[-1]
        row_src.extend(slots.tolist())
        offsets.append(offsets[-1] + slots.size)
    return slot_row.reshape(np.shape(idx)), np.array(offsets), np.array(row_src, dtype=np.int64)


def permute_rows(x, slot_row, rows):
    """rows with rows[slot_row[t, j]] = x[t]."""
    out = np.array(rows)
    for t, j in zip(*np.nonzero(slot_row >= 0)):
        out[slot_row[t, j]] = x[t]
    return out


def sum_rows(rows, slot_row, prob=None):
    """(sum over j of prob[t, j] rows[slot_row[t, j]], the same sum of magnitudes)."""
    y = np.zeros((slot_row.shape[0], rows.shape[1]))
    size = np.zeros_like(y)
    for t, j in zip(*np.nonzero(slot_row >= 0)):
        v = rows[slot_row[t, j]] * (1.0 if prob is None else prob[t, j])
        y[t] += v
        size[t] += np.abs(v)
    return y, size


def sum_rows_backward(dy, rows, slot_row, prob, drows):
    """(drows with its slots' rows prob dy, dprob, the sums of magnitudes behind dprob)."""
    drows, dprob = np.array(drows), np.zeros(slot_row.shape)
    size = np.zeros_like(dprob)
    for t, j in zip(*np.nonzero(slot_row >= 0)):
        r = slot_row[t, j]
        drows[r] = prob[t, j] * dy[t]
        dprob[t, j] = (dy[t] * rows[r]).sum()
        size[t, j] = np.abs(dy[t] * rows[r]).sum()
    return drows, dprob, size


def philox4x32(counter, key, rounds=10):
    """The four 32-bit words of Philox 4x32 for a counter of four words and a
    key of two (Salmon, Moraes, Dror, Shaw, 2011)."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_mask(n, p, key, first):
    """Which of n elements are kept: word i % 4 at counter first + i / 4 (64 bits,
    wrapping) is at least round(p 2^32)."""
    limit, kept = round(p * 2.0 ** 32), []
    for q in range((n + 3) // 4):
        at = (first + q) & 0xFFFFFFFFFFFFFFFF
        kept += [w >= limit for w in philox4x32((at & 0xFFFFFFFF, at >> 32, 0, 0), (key & 0xFFFFFFFF, key >> 32 & 0xFFFFFFFF))]
    return np.array(kept[:n], dtype=bool)
