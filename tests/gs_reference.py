"""Plain definitions, in 64 bits, of the group-scaled 4-bit operators and the
expert routing, for the tests that compare kernels against them.

Half-step rounding units used in the tests' bounds: fp32 2^-24, bf16 2^-8.
"""
import numpy as np
import torch

U32 = 2.0 ** -24
UBF = 2.0 ** -8


def bf16_round(x32: np.ndarray) -> np.ndarray:
    """fp32 values rounded to bf16, nearest even, as float32."""
    return torch.from_numpy(np.ascontiguousarray(x32, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def quantise(w: np.ndarray, group: int, bf16_scale: bool):
    """(codes int8 [N, K], scales float32 [N, G]) of fp32 weights.  The fp64
    quotient of two fp32 numbers rounds to a half only when it is one: the
    quotient differs from a half by at least 2^-28 relative, if at all."""
    N, K = w.shape
    G = -(-K // group)
    codes = np.zeros((N, K), np.int8)
    scales = np.zeros((N, G), np.float32)
    for g in range(G):
        part = w[:, g * group:(g + 1) * group]
        s = (np.abs(part).max(1).astype(np.float32) / np.float32(7)).astype(np.float32)
        if bf16_scale:
            s = bf16_round(s)
        scales[:, g] = s
        d = s.astype(np.float64)[:, None]
        with np.errstate(divide="ignore", invalid="ignore"):
            c = np.where(d > 0, np.clip(np.rint(part.astype(np.float64) / d), -7, 7), 0)
        codes[:, g * group:(g + 1) * group] = c
    return codes, scales


def pack(codes: np.ndarray, ldp: int) -> np.ndarray:
    """Packed rows: code k in byte (k % 8) % 4 of word k // 8, nibble (k % 8) // 4."""
    out = np.zeros((codes.shape[0], ldp), np.uint8)
    for k in range(codes.shape[1]):
        out[:, 4 * (k // 8) + k % 4] |= ((codes[:, k].astype(np.int64) & 15) << (4 * (k % 8 // 4))).astype(np.uint8)
    return out


def linear(q, s_x, codes, scales, group):
    """(y, bound) in fp64: y = s_x * sum_g s_g * acc_g and the sum of |terms|."""
    M, K = q.shape
    y = np.zeros((M, codes.shape[0]))
    mag = np.zeros_like(y)
    for g in range(scales.shape[1]):
        k = slice(g * group, min(K, (g + 1) * group))
        part = (q[:, k].astype(np.float64) @ codes[:, k].astype(np.float64).T) * scales[:, g].astype(np.float64)
        y += part
        mag += np.abs(part)
    s = s_x.astype(np.float64)[:, None]
    return y * s, mag * np.abs(s)


def linear_bound(y, mag, G, bf16):
    """How far the kernels may be off, by counting roundings.  The integer
    sums of whole groups and their conversions are exact.  Each of the G
    multiply-adds and each addition of partial sums (fewer than G + 64: every
    partial sum holds a group) rounds a value of at most mag; two products
    follow.  A bf16 result adds half a step of the result,
    which is y plus that error."""
    e = (2 * G + 66) * U32 * mag * (1 + 1e-3)
    return e + UBF * (np.abs(y) + e) if bf16 else e


def plan(experts: np.ndarray, E: int):
    flat = experts.reshape(-1).astype(np.int64)
    keep = (flat >= 0) & (flat < E)
    order = [i for e in range(E) for i in np.nonzero(flat == e)[0]] if E <= 64 else \
        [i for i in np.argsort(np.where(keep, flat, E), kind="stable") if keep[i]]
    pos = np.full(flat.shape, -1, np.int32)
    pos[np.asarray(order, dtype=np.int64)] = np.arange(len(order))
    counts = np.bincount(flat[keep], minlength=E)
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), pos.reshape(experts.shape)
