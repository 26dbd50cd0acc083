"""CPU checks of the binding: what its calls hand to the library, and what it needs to load."""

import ctypes
import sys
import threading

from mla_latent_kv_35_b200 import binding as B


def dims(cls=B.MLADims):
    return cls(4, 16, 32, 8, 16, 64, 64, 0.1, 10000.0, "bf16")


def n_heads_at(addr):
    return ctypes.cast(addr, ctypes.POINTER(B.Dims)).contents.n_heads


def test_two_first_calls_at_once_share_one_struct():
    """A second first call that comes in between finding no struct and keeping one: both calls hold the
    struct that is kept."""
    inner = []

    class Slow(B.MLADims):
        def c(self):
            if not inner:
                inner.append(None)
                inner[0] = B._addr(self)               # the other thread's whole call
            return super().c()
    d = dims(Slow)
    outer = B._addr(d)
    assert outer == inner[0] == B._addr(d)
    assert n_heads_at(outer) == 4


def test_first_calls_of_four_threads():
    old = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for _ in range(300):
            d, seen, go = dims(), [], threading.Barrier(4)

            def first():
                go.wait()
                seen.append(B._addr(d))
            ts = [threading.Thread(target=first) for _ in range(4)]
            for t in ts:
                t.start()
            for t in ts:
                t.join()
            assert len(seen) == 4 and set(seen) == {B._addr(d)}
    finally:
        sys.setswitchinterval(old)
