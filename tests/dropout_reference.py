"""Dropout's mask, from the generator's definition: Philox4x32-10 (Salmon,
Moraes, Dror and Shaw, SC 2011) in numpy, sixteen bits an element."""
import numpy as np


def philox4x32_10(counter, key):
    """Four uint32 words from counters [..., 4] and a key of two."""
    c = [np.asarray(counter)[..., i].astype(np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=-1).astype(np.uint32)


def threshold(p):
    return int(np.rint(float(np.float32(p)) * 65536.0))


def kept(n, p, seed, offset, first=0):
    """Whether the elements first .. first + n are kept (bool); first a multiple of 8."""
    octets = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    counter = np.empty((octets.size, 4), dtype=np.uint64)
    counter[:, 0], counter[:, 1] = octets & np.uint64(0xFFFFFFFF), octets >> np.uint64(32)
    counter[:, 2], counter[:, 3] = offset & 0xFFFFFFFF, offset >> 32
    w = philox4x32_10(counter, (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.stack([w & 0xFFFF, w >> 16], axis=-1).reshape(-1)  # words in order, the low half first
    return bits[:n] >= threshold(p)
