"""Row-local functions on many rows.

The oracle's element-wise and per-row steps (norms, rotary embedding, activations, bf16
rounding) touch gigabytes of float64 at full workload sizes.  Taken a chunk of rows at a time
their temporaries stay in cache, and numpy releases the interpreter while it computes, so the chunks
run on all cores.  A row's result does not depend on the chunk it is in: the bits are those
of the plain call.
"""
import multiprocessing
import os
from concurrent.futures import ThreadPoolExecutor

import numpy as np

CHUNK_BYTES = 1 << 21
THREADS = None  # of by_rows; None: one per core (the one-thread timing sets 1)

_pool = None
_one_thread_pid = None


def one_blas_thread_in_a_worker():
    """In a process-pool worker, BLAS takes one thread: the pool has a worker per core.  To be called
    by the work itself, since a limit set when the worker starts, before numpy is loaded, finds no
    BLAS to limit (16 workers of 16 threads each on 16 cores took two to five times as long)."""
    global _one_thread_pid
    if _one_thread_pid == os.getpid() or multiprocessing.parent_process() is None:
        return
    _one_thread_pid = os.getpid()
    try:
        from threadpoolctl import threadpool_limits
    except ImportError:
        return
    threadpool_limits(1)


def _threads():
    global _pool
    n = THREADS or (len(os.sched_getaffinity(0)) if hasattr(os, "sched_getaffinity") else os.cpu_count() or 1)
    if _pool is None or _pool[0] != (os.getpid(), n):
        _pool = ((os.getpid(), n), ThreadPoolExecutor(n))
    return _pool[1]


def by_rows(f, *arrays):
    """f(*arrays) for an f that treats each row (first index, shared by all arrays) on its own
    and returns an array with as many rows, or a tuple of them."""
    n = len(arrays[0])
    step = max(1, CHUNK_BYTES // max(1, arrays[0][:1].nbytes))
    if n <= 4 * step:
        return f(*arrays)
    first = f(*(a[:step] for a in arrays))
    firsts = first if isinstance(first, tuple) else (first,)
    outs = [np.empty((n,) + o.shape[1:], o.dtype) for o in firsts]

    def put(i, res):
        for o, r in zip(outs, res if isinstance(res, tuple) else (res,)):
            o[i:i + step] = r

    put(0, first)
    run = map if THREADS == 1 else _threads().map
    list(run(lambda i: put(i, f(*(a[i:i + step] for a in arrays))), range(step, n, step)))
    return tuple(outs) if isinstance(first, tuple) else outs[0]
