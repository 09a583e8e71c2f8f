"""CPU oracle of the paged 8-bit KV cache.

TEST INFRASTRUCTURE ONLY (same rules as the rest of ``oracle/``).

The pages of the method describe one sequence and one cache; a server keeps
the caches of many requests in pages of ``P`` tokens ([EAGLE blog] section
1.1: the accepted tokens of one verification forward are kept; [EAGLE-2
article]: every flattened row attends the prefix plus its ancestors).  Here:

* the values of the two 8-bit formats and rounding to them, from their
  definition (sign, exponent, mantissa; nearest, ties to the even code);
* the block map: pages returned and taken, request by request, on a stack;
* the commit: rows quantised page by page under a power-of-two scale;
* the attention: softmax over the tokens that are there, with the sums that
  bound what a kernel's roundings can do to it.
"""
import math
from typing import List, Optional, Tuple

import numpy as np

SCALE_EXP = 48
MAX_VALUE = {"e4m3": 448.0, "e5m2": 57344.0}


# ---------------------------------------------------------------------------
# the formats
# ---------------------------------------------------------------------------
def code_value(code: int, fmt: str) -> float:
    """What one 8-bit code stands for."""
    man_bits, bias = (3, 7) if fmt == "e4m3" else (2, 15)
    sign = -1.0 if code & 0x80 else 1.0
    exp, man = (code & 0x7F) >> man_bits, code & ((1 << man_bits) - 1)
    if fmt == "e4m3" and (code & 0x7F) == 0x7F:
        return math.nan
    if fmt == "e5m2" and exp == 31:
        return math.nan if man else sign * math.inf
    if exp == 0:
        return sign * man * 2.0 ** (1 - bias - man_bits)
    return sign * (1 + man / (1 << man_bits)) * 2.0 ** (exp - bias)


def decode(codes: np.ndarray, fmt: str) -> np.ndarray:
    table = np.array([code_value(c, fmt) for c in range(256)])
    return table[np.asarray(codes, np.uint8)]


def encode(x: np.ndarray, fmt: str) -> np.ndarray:
    """Nearest code, ties to the even code; past the largest value to it; NaN to the NaN code (sign as given by
    the canonical positive one)."""
    x = np.asarray(x, np.float64)
    top = 0x7E if fmt == "e4m3" else 0x7B
    vals = np.array([code_value(c, fmt) for c in range(top + 1)])  # ascending
    mag = np.abs(x)
    hi = np.clip(np.searchsorted(vals, mag), 1, top)
    a, b = vals[hi - 1], vals[hi]
    up = (b - mag < mag - a) | ((b - mag == mag - a) & (hi % 2 == 0))
    code = np.where(up, hi, hi - 1)
    code = np.where(mag >= vals[top], top, code)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def page_scale(amax: float, fmt: str) -> float:
    """The smallest 2^e >= amax / MAX within -48..48."""
    if not amax > 0:
        return 2.0 ** -SCALE_EXP
    e = -SCALE_EXP
    while e < SCALE_EXP and amax > MAX_VALUE[fmt] * 2.0 ** e:
        e += 1
    return 2.0 ** e


# ---------------------------------------------------------------------------
# block map
# ---------------------------------------------------------------------------
def block_map(prefix_len, new_len, n_blocks, block_table, free: List[int], page_size: int, max_new: int
              ) -> Tuple[np.ndarray, np.ndarray, List[int], np.ndarray, bool, bool]:
    """Returns (n_blocks', block_table', free stack', slot_map, a request was refused pages, an argument was bad)."""
    B, cols = block_table.shape
    n, table, free = np.array(n_blocks), np.array(block_table), list(free)
    slots = np.full((B, max_new), -1, np.int64)
    need = np.zeros(B, np.int64)
    good = np.zeros(B, bool)
    bad = False
    for b in range(B):
        if prefix_len[b] < 0:
            continue
        need[b] = -(-(int(prefix_len[b]) + int(new_len[b])) // page_size)
        good[b] = (new_len[b] >= 0 and (max_new == 0 or new_len[b] <= max_new) and 0 <= n[b] <= cols
                   and need[b] <= cols)
        bad |= not good[b]
    for b in range(B):
        if good[b]:
            for j in range(need[b], n[b]):
                free.append(int(table[b, j]))
                table[b, j] = -1
            n[b] = min(n[b], need[b])
    short = False
    for b in range(B):
        if not good[b]:
            continue
        missing = need[b] - n[b]
        if missing > 0 and (short or missing > len(free)):
            short = True
            continue
        for _ in range(missing):
            table[b, n[b]] = free.pop()
            n[b] += 1
        for i in range(new_len[b] if max_new else 0):
            pos = int(prefix_len[b]) + i
            slots[b, i] = int(table[b, pos // page_size]) * page_size + pos % page_size
    return n, table, free, slots, short, bad


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------
def kv_commit_paged(codes: np.ndarray, scale: np.ndarray, fmt: str, block_table: np.ndarray, tree: np.ndarray,
                    accept_len: np.ndarray, path: Optional[np.ndarray], prefix_len: np.ndarray
                    ) -> Tuple[np.ndarray, np.ndarray]:
    """One of K and V: codes [pages, Hkv, P, d] uint8, scale [pages, Hkv] fp32, tree [B, N, Hkv, d].  Returns the
    new codes and scales."""
    codes, scale = codes.copy(), scale.astype(np.float32).copy()
    Hkv, P = codes.shape[1], codes.shape[2]
    for b in range(tree.shape[0]):
        base = int(prefix_len[b])
        rows = int(accept_len[b]) + 1 if base >= 0 else 0
        got = {}  # block -> [(slot, tree row)]
        for i in range(rows):
            r = i if path is None else int(path[b, i])
            got.setdefault((base + i) // P, []).append(((base + i) % P, r))
        for blk, put in got.items():
            page = int(block_table[b, blk])
            first = put[0][0]
            for g in range(Hkv):
                x = np.stack([tree[b, r, g] for _, r in put]).astype(np.float64)
                fin = np.abs(x[np.isfinite(x)])
                s = page_scale(fin.max() if fin.size else 0.0, fmt)
                if first > 0:
                    old = float(scale[page, g])
                    s = max(old, s)
                    if s > old:
                        held = decode(codes[page, g, :first], fmt)
                        codes[page, g, :first] = encode(held * (old / s), fmt)
                for (slot, _), row in zip(put, x):
                    codes[page, g, slot] = encode(np.float32(row / s) if np.log2(s) % 1 else row / s, fmt)
                scale[page, g] = s
    return codes, scale


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def dequantised(codes: np.ndarray, scale: np.ndarray, fmt: str, table_row: np.ndarray, length: int) -> np.ndarray:
    """The cached rows of one sequence, [Hkv, length, d] float64."""
    P = codes.shape[2]
    rows = [decode(codes[table_row[j // P], :, j % P], fmt) * scale[table_row[j // P]].astype(np.float64)[:, None]
            for j in range(length)]
    return np.stack(rows, 1) if rows else np.zeros((codes.shape[1], 0, codes.shape[3]))


def paged_attention(q, kc, vc, k_tree, v_tree, keep_prefix, keep_tree, scale):
    """One sequence: q [N, Hq, d], kc/vc [Hkv, L, d], k/v_tree [N, Hkv, d], keep_prefix [L] and keep_tree [N, N] bool.

    Returns out [N, Hq, d], lse [Hq, N], and what bounds a kernel's error: the weighted magnitudes sum p |v| over the
    cached tokens and over the tree rows, [N, Hq, d] each, the largest sum |q||k| * scale of a row, [Hq, N], and the
    same for cached tokens with every |q| at its row's largest."""
    q = np.asarray(q, np.float64)
    N, Hq, d = q.shape
    G = Hq // k_tree.shape[1]
    L = kc.shape[1]
    out, lse = np.zeros((N, Hq, d)), np.full((Hq, N), -np.inf)
    abs_c, abs_t, reach, flat = np.zeros((N, Hq, d)), np.zeros((N, Hq, d)), np.zeros((Hq, N)), np.zeros((Hq, N))
    for h in range(Hq):
        g = h // G
        for i in range(N):
            jc, jt = np.flatnonzero(keep_prefix), np.flatnonzero(keep_tree[i])
            K = np.concatenate([kc[g][jc], k_tree[jt, g].astype(np.float64)])
            V = np.concatenate([vc[g][jc], v_tree[jt, g].astype(np.float64)])
            if not len(K):
                continue
            z = scale * (K @ q[i, h])
            top = z.max()
            p = np.exp(z - top)
            lse[h, i] = top + math.log(p.sum())
            p /= p.sum()
            out[i, h] = p @ V
            abs_c[i, h] = p[:len(jc)] @ np.abs(V[:len(jc)])
            abs_t[i, h] = p[len(jc):] @ np.abs(V[len(jc):])
            reach[h, i] = scale * (np.abs(K) @ np.abs(q[i, h])).max()
            if len(jc):
                flat[h, i] = scale * np.abs(q[i, h]).max() * np.abs(kc[g][jc]).sum(1).max()
    return out, lse, abs_c, abs_t, reach, flat
