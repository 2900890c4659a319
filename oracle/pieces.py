"""Functions of the rows of matrices, a piece of the rows at a time.

The rows of the layers and of the block operators have nothing to do with each
other, and a numpy expression of a large matrix mostly waits for its
temporaries' memory: pieces that stay in the caches, in a few threads, take a
fraction of the time and give the same bits."""
import contextvars
import functools
import os
from concurrent.futures import ThreadPoolExecutor

import numpy as np

ELEMENTS = 1 << 17  # of a piece
_THREADS = min(8, os.cpu_count() or 1)
_pool = None


def in_pieces(f, rows, size):
    """[f(first, last)] of the pieces of `rows` rows."""
    global _pool
    step = max(1, ELEMENTS // max(size, 1))
    if rows <= step:
        return [f(0, rows)]
    if _pool is None:
        _pool = ThreadPoolExecutor(_THREADS)
    # with the caller's numpy error state, which is a context's
    jobs = [_pool.submit(contextvars.copy_context().run, f, i, min(i + step, rows)) for i in range(0, rows, step)]
    return [j.result() for j in jobs]


def joined(parts):
    """Their results, one or several arrays each, one piece after another."""
    if len(parts) == 1:
        return parts[0]
    if isinstance(parts[0], tuple):
        return tuple(np.concatenate(p) for p in zip(*parts))
    return np.concatenate(parts)


def by_rows(*places):
    """A function of matrices and of vectors with an element for each row,
    which are its arguments number `places`."""
    def made(f):
        @functools.wraps(f)
        def whole(*args, **more):
            first = np.asarray(args[places[0]])
            if first.ndim == 0:
                return f(*args, **more)

            def piece(i, j):
                return f(*(a[i:j] if k in places else a for k, a in enumerate(args)), **more)
            return joined(in_pieces(piece, first.shape[0], first[0].size if first.shape[0] else 0))
        return whole
    return made
