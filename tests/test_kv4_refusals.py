"""Refusals of the four-bit caches' calls beside test_kv4's: no GPU is needed."""
import pytest

from test_kv4 import P, _lib, _write


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_block_drafter_gb300 import build
    build.build()


def test_write_refuses_caches_that_overlap():
    """Caches that share some of their memory, by one byte short of a whole cache or by all but one tile."""
    L = _lib()
    nb = L.dflash_kv4_cache_bytes(2, 64, 256)
    far = P + 64 * nb
    for over in (dict(cv=[P + nb - 16]), dict(cv=[P - nb + 16]), dict(cv=[P + 16]),
                 dict(batch=2, ck=[P, P + nb - 16], cv=[far, far + nb], at=[0, 100]),
                 dict(batch=2, ck=[P, P + nb], cv=[far, far + 128 * 36], at=[0, 200]),
                 dict(batch=3, ck=[P, P + 4 * nb, P + 8 * nb], cv=[far, far + nb, P + 7 * nb + 16], at=[0, 0, 0])):
        with pytest.raises(L.DflashError) as e:
            _write(L, **over)
        assert e.value.code == 2, over
    # side by side, and one cache in two places of the batch with other rows: the rest of the checks is reached
    for over in (dict(cv=[P + nb]), dict(batch=2, ck=[P + nb, P], cv=[far + nb, far], at=[0, 0]),
                 dict(batch=2, ck=[P, P], cv=[far, far], at=[0, 4])):
        n0 = L.dflash_launch_count()
        _write(L, **dict(over, n=0, at=[256] * over.get("batch", 1)))
        assert L.dflash_launch_count() == n0
