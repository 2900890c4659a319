"""The choice of candidates for the likeliest of a row, as k_logp makes it,
on the host: which inputs reach which of its ways."""
import numpy as np

CANDIDATES = 1024  # kCandidates: what a workgroup has room for
UNIT = {"f32": 4, "f16": 8, "bf16": 8}


def cut(rows, size, dtype):
    """(segments, turns, threads) of rows of more than 2048 columns."""
    units = -(-size // UNIT[dtype])
    most = -(-units // 256)
    if rows >= 1536 and units <= 64 * 64:
        return 1, -(-units // 64), 64
    if rows > 256:
        return 1, most, 256
    if units <= 1024 * max(8, rows // 8):
        return 1, -(-units // 1024), 1024
    wanted = min(64, 1024 // rows)
    turns = -(-most // wanted)
    return -(-most // turns), turns, 256


def candidates(x, top, dtype, turns, threads):
    """Of the columns of one workgroup: (whether the row is scarce, the columns
    that reach its threshold, those of them in other waves than the first, the
    first columns with nothing that can come)."""
    unit = UNIT[dtype]
    held = np.full(turns * threads * unit, -np.inf)
    held[:len(x)] = x
    lanes = held.reshape(turns, threads, unit)
    waves = lanes.max((0, 2)).reshape(-1, 64)  # the lanes' largest
    share = -(-top // len(waves))
    kth = lambda k: np.sort(waves, 1)[:, -k]  # noqa: E731
    least = max(kth(top).max(), kth(share).min())
    scarce = np.isneginf(least)
    reach = lanes > -np.inf if scarce else lanes >= least
    by_wave = reach.reshape(turns, -1, 64, unit).sum((0, 2, 3))
    return scarce, int(by_wave.sum()), int(by_wave[1:].sum()), int(np.isneginf(x[:top]).sum()) if scarce else 0


def allowed_in(waves, lanes, size, dtype, turns, threads):
    """The columns whose unit is one of the last `lanes` lanes of those waves of
    a workgroup of `threads`."""
    at = np.arange(size) // UNIT[dtype] % threads
    return np.isin(at // 64, list(waves)) & (at % 64 >= 64 - lanes)


# rows, columns, format, segments and threads of a row
CROWDED = [(300, 50304, "bf16", 1, 256), (257, 50304, "f32", 1, 256), (258, 262144, "bf16", 1, 256),
           (200, 131072, "bf16", 1, 1024), (256, 131072, "f32", 1, 1024), (9, 65536, "f16", 1, 1024),
           (2, 1 << 20, "bf16", 64, 256), (20, 600000, "f32", 49, 256), (1536, 16384, "f16", 1, 64)]


def crowded(rows, size, dtype):
    """Four rows of which a few lanes of every wave have all that can come, or
    of every wave but the first; the last two with 1024 and 1025 columns that
    reach the threshold."""
    segments, turns, threads = cut(rows, size, dtype)
    rng = np.random.default_rng([rows, size])
    x = np.full((4, size), -np.inf)
    waves = threads // 64
    few = 19 if waves == 1 else -(-20 // waves) - 1  # fewer than each wave's share
    spread = allowed_in(range(waves), few, size, dtype, turns, threads)
    behind = allowed_in(range(1, waves) if waves > 1 else (0,), 19, size, dtype, turns, threads)
    first = np.arange(size) < turns * threads * UNIT[dtype]
    for row, columns in enumerate((spread, behind)):
        if np.count_nonzero(columns & first) <= CANDIDATES:
            columns = behind
        x[row, columns] = rng.standard_normal(np.count_nonzero(columns))
    for row, n in ((2, CANDIDATES), (3, CANDIDATES + 1)):
        columns = np.flatnonzero(behind & first & (np.arange(size) >= 20))[:n - 20]
        x[row, columns] = rng.standard_normal(len(columns))
    return x
