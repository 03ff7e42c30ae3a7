"""Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011) in NumPy: what the dropout tests
compare with. It shares no code with the GPU path."""
import numpy as np

_LOW = np.uint64(0xFFFFFFFF)
_32 = np.uint64(32)


def words(index: np.ndarray, offset: int, key: int) -> np.ndarray:
    """The four words of each counter (index, offset): uint32 [n, 4]."""
    i = index.astype(np.uint64)
    c = [i & _LOW, i >> _32, np.full_like(i, offset & 0xFFFFFFFF), np.full_like(i, offset >> 32 & 0xFFFFFFFF)]
    k = [key & 0xFFFFFFFF, key >> 32 & 0xFFFFFFFF]
    for r in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> _32) ^ c[1] ^ np.uint64(k[0]), b & _LOW, (a >> _32) ^ c[3] ^ np.uint64(k[1]), a & _LOW]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1).astype(np.uint32)


def kept(n: int, seed: int, offset: int, limit: int, first: int = 0) -> np.ndarray:
    """Which of the elements 8 * first .. 8 * first + n - 1 stay."""
    w = words(first + np.arange(-(-n // 8), dtype=np.uint64), offset, seed)
    u = np.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:n]
    return u >= limit
