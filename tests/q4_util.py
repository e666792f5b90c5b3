"""Q4_0 blocks as the library lays them out, for the tests: codes in 32-bit
words of eight (word t * nb + b of a group of nb blocks holds elements
32 b + 8 t + {0..7}; element 8 t + 2 i at bit 4 i, element 8 t + 2 i + 1 at bit
16 + 4 i), weight rows in chunks of 256 elements (two groups of 128, then 8
fp16 scales), caches as a plane of codes, then a plane of scales."""
import numpy as np


def pack_groups(c, nb):
    """Codes [..., 32 nb] -> bytes [..., 16 nb]."""
    c = np.asarray(c, dtype=np.uint32)
    words = np.zeros(c.shape[:-1] + (4 * nb,), np.uint32)
    for e in range(32 * nb):
        b, r = divmod(e, 32)
        t, k = divmod(r, 8)
        words[..., t * nb + b] |= c[..., e] << np.uint32(4 * (k // 2) + 16 * (k % 2))
    return words.view(np.uint8)


def unpack_groups(raw, nb):
    words = np.ascontiguousarray(raw).view(np.uint32)
    out = np.zeros(words.shape[:-1] + (32 * nb,), np.uint8)
    for e in range(32 * nb):
        b, r = divmod(e, 32)
        t, k = divmod(r, 8)
        out[..., e] = (words[..., t * nb + b] >> np.uint32(4 * (k // 2) + 16 * (k % 2))) & 15
    return out


def pack_weights(c, d):
    """Codes [N][K], fp16 scales [N][K / 32] -> bytes [N][9 K / 16]."""
    n, k = c.shape
    out = np.zeros((n, k // 256, 144), np.uint8)
    out[:, :, :128] = pack_groups(c.reshape(n, k // 128, 128), 4).reshape(n, k // 256, 128)
    out[:, :, 128:] = np.ascontiguousarray(d).view(np.uint8).reshape(n, k // 256, 16)
    return out.reshape(n, -1)


def pack_cache(c, d):
    """Codes [n_seq][Hkv][n_ctx][hd], scales [..][hd / 32] -> the cache's bytes."""
    nb = c.shape[-1] // 32
    return np.concatenate([pack_groups(c, nb).reshape(-1), np.ascontiguousarray(d).view(np.uint8).reshape(-1)])


def unpack_cache(raw, n_seq, hkv, n_ctx, hd):
    n = n_seq * hkv * n_ctx
    c = unpack_groups(raw[:n * hd // 2].reshape(n, hd // 2), hd // 32).reshape(n_seq, hkv, n_ctx, hd)
    d = np.ascontiguousarray(raw[n * hd // 2:]).view(np.float16).reshape(n_seq, hkv, n_ctx, hd // 32)
    return c, d
