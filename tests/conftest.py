import ctypes
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def keep_freed_memory():
    """Have malloc keep what is freed.  The oracles' temporaries are hundreds of
    MB each, which it would map anew and give back every time, a page fault for
    every page: log probabilities of 2100 x 20011 take 12 s so, and 2 s out of
    kept memory."""
    try:
        mallopt = ctypes.CDLL(None).mallopt
    except (AttributeError, OSError):
        return  # another C library: slower, no more
    mallopt(-4, 0)   # M_MMAP_MAX: nothing of its own mapping
    mallopt(-1, -1)  # M_TRIM_THRESHOLD: nothing is given back


def pytest_configure(config):
    keep_freed_memory()
    config.addinivalue_line("markers", "gpu: needs an MI355X (runs the HIP library through its C ABI)")
    config.addinivalue_line("markers", "slow: CPU test that takes more than a few seconds")
