"""The layers of include/gclip_layer.h in binary64 on the CPU, from their
definitions: numpy arrays [rows, size] in, binary64 out."""
import numpy as np

LOW = np.uint64(0xFFFFFFFF)


def philox_words(counter, key):
    """Philox4x32-10 (Salmon et al., SC 2011): counter is four arrays of
    32-bit words, key two integers; four uint32 arrays."""
    c = [np.asarray(x, dtype=np.uint64) for x in counter]
    k = list(key)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & LOW,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & LOW]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return [x.astype(np.uint32) for x in c]


def dropout_threshold(p):
    return int(np.floor(65536.0 * p + 0.5))


def dropout_scale(p):
    """The factor of a kept element before its rounding to binary32."""
    t = dropout_threshold(p)
    return 65536.0 / (65536.0 - t) if t < 65536 else 0.0


def kept(rows, size, p, seed, step=0, site=0):
    """Truth values [rows, size]."""
    groups = -(-size // 8)
    r, g = np.meshgrid(np.arange(rows), np.arange(groups), indexing="ij")
    w = philox_words([g, r, np.full_like(g, site), np.full_like(g, step % (1 << 32))],
                     [seed & 0xFFFFFFFF, seed >> 32])
    u = np.empty((rows, groups, 8), dtype=np.uint32)
    for i in range(4):
        u[:, :, 2 * i] = w[i] & 0xFFFF
        u[:, :, 2 * i + 1] = w[i] >> 16
    return u.reshape(rows, groups * 8)[:, :size] >= dropout_threshold(p)


def statistics(x, eps):
    x = x.astype(np.float64)
    mean = x.sum(1) / x.shape[1]
    var = ((x - mean[:, None]) ** 2).sum(1) / x.shape[1]
    return mean, 1.0 / np.sqrt(var + eps)


def norm(x, weight, bias, eps):
    """(y, mean, rstd)"""
    mean, rstd = statistics(x, eps)
    return (x - mean[:, None]) * rstd[:, None] * weight + bias, mean, rstd


def norm_gradient(dy, x, mean, rstd, weight):
    """(dx, dweight, dbias)"""
    n = (x - mean[:, None]) * rstd[:, None]
    g = dy * weight
    size = x.shape[1]
    dx = rstd[:, None] * (g - g.sum(1, keepdims=True) / size - n * ((g * n).sum(1, keepdims=True) / size))
    return dx, (dy * n).sum(0), dy.sum(0)
