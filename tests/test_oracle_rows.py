"""The oracle's row-chunked evaluation gives the bits of the plain call."""
import numpy as np
import pytest

from oracle import bf16, layer
from oracle.rows import CHUNK_BYTES, by_rows
from tests.oracle_pool import oracle_pool


@pytest.mark.parametrize("n", [0, 1, 5, 700, 3001])
def test_chunked_rows_have_the_plain_bits(n):
    rng = np.random.Generator(np.random.PCG64(n))
    h = 1600
    assert n < 700 or 4 * (CHUNK_BYTES // (h * 8)) < n  # the larger ones are cut
    x, u = rng.standard_normal((n, h)), rng.standard_normal((n, h))
    x[n // 2:n // 2 + 1, :3] = np.inf, np.nan, -np.inf
    r = rng.standard_normal(n)
    for f, a in ((lambda a, b: layer.silu(a) * b, (x, u)), (bf16._round_bf16, (x,)),
                 (lambda a, s: (a * s[:, None], a.sum(axis=1)), (x, r)),
                 (lambda a: a.reshape(len(a), 16, 100)[:, :, :50].copy(), (x,))):
        with np.errstate(invalid="ignore"):
            want, got = f(*a), by_rows(f, *a)
        for w, g in zip(want if isinstance(want, tuple) else (want,), got if isinstance(got, tuple) else (got,)):
            assert w.dtype == g.dtype and np.array_equal(w, g, equal_nan=True)
    bits = rng.integers(0, 0x7F80, size=(n, h), dtype=np.uint16)
    v = bf16.from_bits(bits)
    assert np.array_equal(v, bf16._from_bits(bits)) and np.array_equal(bf16.round_bf16(v), v)


def test_an_exception_in_a_chunk_reaches_the_caller():
    def f(a):
        if a[0, 0] > 500:
            raise ArithmeticError("row")
        return a
    x = np.repeat(np.arange(1000.0)[:, None], 5000, axis=1)
    with pytest.raises(ArithmeticError):
        by_rows(f, x)


def _blas_threads(args):
    from oracle import layer as oly
    if args is not None:
        oly.head_attention_fwd(args)
    from threadpoolctl import threadpool_info
    return max((i["num_threads"] for i in threadpool_info() if i.get("user_api") == "blas"), default=0)


def test_pool_workers_run_blas_on_one_thread():
    x = np.ones((8, 4))
    before = _blas_threads(None)
    with oracle_pool(2) as pmap:
        assert set(pmap(_blas_threads, [(x, x, x, 4)] * 4)) == {1}
    assert _blas_threads((x, x, x, 4)) == before  # and the caller's own BLAS keeps its threads


def test_one_thread_on_request(monkeypatch):
    import threading

    from oracle import rows
    seen = set()

    def f(a):
        seen.add(threading.get_ident())
        return a + 1
    x = np.zeros((4000, 1000))
    monkeypatch.setattr(rows, "THREADS", 1)
    assert (by_rows(f, x) == 1).all() and seen == {threading.get_ident()}
    monkeypatch.setattr(rows, "THREADS", 3)
    seen.clear()
    assert (by_rows(f, x) == 1).all() and 1 < len(seen) <= 4
