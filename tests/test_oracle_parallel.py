"""The oracle's process pool (CPU): what its workers start with."""

import os


def test_parallel_workers_start_with_one_blas_thread(monkeypatch):
    # numpy reads the limits when it is imported, so they must be in the environment a worker starts with
    from oracle.parallel import OraclePool

    monkeypatch.delenv("OPENBLAS_NUM_THREADS", raising=False)
    monkeypatch.setenv("OMP_NUM_THREADS", "5")
    with OraclePool(1) as pool:
        start = pool._pool.apply(eval, ("open('/proc/self/environ', 'rb').read()",)).split(b"\0")
    assert b"OPENBLAS_NUM_THREADS=1" in start and b"OMP_NUM_THREADS=1" in start
    assert os.environ["OMP_NUM_THREADS"] == "5" and "OPENBLAS_NUM_THREADS" not in os.environ
