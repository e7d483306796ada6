"""The serving operators in float64, from their definitions, for the tests.

Tolerances (derived; eps/2 is the largest relative error of one rounding):
  scores   a dot of d products in fp32 with any order and truncation: |dS| <= (d + 4) 2^-23 sum|q k| / sqrt d =: e
  row_sum  a mean of exponents: e, plus the exponential, logarithm and sums in fp32: 2^-20 + 2^-22 |row_sum|
  O        weights P / l move by 2 e + 2^-19 relatively; with bf16 inputs by 2^-8 more as P is rounded to bf16 for the tensor cores,
           and by up to 2^-8 again as l may be a sum of rounded P (a mean of factors within 2^-8 of 1);
           the result is rounded once (2^-8 of bf16, 2^-24 of fp32); sums of n terms in fp32 move by n 2^-24; all relative to
           sum_j w_j |V_j|
"""
import math

import numpy as np
import torch


def sequence(q, k, v, table, pos0):
    """One sequence in float64: q [L][H][d] at positions pos0 .., k, v [N][H_kv][d] at positions 0 ..
    Returns O, row_sum, sum w|V| and the largest sum|q k| / sqrt d of each row."""
    L, H, d = q.shape
    N, G, s = k.shape[0], H // k.shape[1], table.shape[1]
    O, A = torch.zeros_like(q), torch.zeros_like(q)
    R, E = torch.zeros((L, H), dtype=q.dtype, device=q.device), torch.zeros((L, H), dtype=q.dtype, device=q.device)
    i = torch.arange(pos0, pos0 + L, dtype=torch.float64, device=q.device)[:, None]
    j = torch.arange(N, dtype=torch.float64, device=q.device)[None]
    for h in range(H):
        c = torch.zeros((L, N), dtype=torch.float64, device=q.device)
        for delta, u in table[h].tolist():
            c += torch.floor((i + u) / delta) == torch.floor((j + u) / delta)
        c = torch.where(j <= i, c, 0.0)
        x = q[:, h] @ k[:, h // G].T / math.sqrt(d)
        x = torch.where(c > 0, x + torch.log(c), -math.inf)
        total = torch.logsumexp(x, 1)
        w = torch.exp(x - total[:, None])
        O[:, h], A[:, h] = w @ v[:, h // G], w @ v[:, h // G].abs()
        R[:, h] = total - math.log(s)
        E[:, h] = torch.where(c > 0, q[:, h].abs() @ k[:, h // G].abs().T / math.sqrt(d), 0.0).amax(1)
    return O, R, A, E


def check(O, R, want, dtype, what=""):
    """O [L][H][d], R [L][H] of a kernel against sequence()'s results."""
    wO, wR, A, E = want
    d, n = O.shape[-1], 4096
    e = (d + 4) * 2.0 ** -23 * E
    rel = 2 * e + 2.0 ** -19 + n * 2.0 ** -24 + (3 * 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24)
    off = ((O.double() - wO).abs() - rel[..., None] * A - 1e-30).max().item()
    assert off <= 0, f"{what}: O is {off} over its tolerance"
    roff = ((R.double() - wR).abs() - e - 2.0 ** -20 - 2.0 ** -22 * wR.abs()).max().item()
    assert roff <= 0, f"{what}: row_sum is {roff} over its tolerance"


def e4m3_grid():
    """The 127 non-negative e4m3 values in order (index = byte)."""
    return np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                     for e in range(16) for m in range(8)][:-1], dtype=np.float64)


def quantise(x):
    """Rows of a float64 array as (bytes, exponents): the definition, value by value. NaN and infinities: byte 0x7F."""
    flat = x.reshape(-1, x.shape[-1])
    out = np.zeros(flat.shape, dtype=np.uint8)
    exps = np.zeros(flat.shape[0], dtype=np.int64)
    grid = e4m3_grid()
    for r, row in enumerate(flat):
        fin = np.isfinite(row)
        top = np.abs(row[fin]).max(initial=0.0)
        e = -126
        while top > 448.0 * 2.0 ** e:
            e += 1
        y = np.abs(np.where(fin, row, 0.0)) * 2.0 ** -e
        hi = np.clip(np.searchsorted(grid, y), 0, len(grid) - 1)
        lo = np.maximum(hi - 1, 0)
        up, down = grid[hi] - y, y - grid[lo]
        b = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        b = np.where(grid[hi] == y, hi, b).astype(np.uint8)
        b = np.where(fin, b | (np.signbit(row).astype(np.uint8) << 7), 0x7F)
        out[r], exps[r] = b, e
    return out.reshape(x.shape), exps.reshape(x.shape[:-1])


def values(byte, exp):
    """The float64 values of e4m3 bytes (uint8 array) and row exponents."""
    grid = np.concatenate([e4m3_grid(), [np.nan]])
    v = grid[byte & 0x7F] * np.where(byte & 0x80, -1.0, 1.0)
    return v * (2.0 ** exp.astype(np.float64))[..., None]
