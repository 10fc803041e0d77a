"""What may change between a row exchange's arguments and its launch: the
session, on the CPU with validate_only sessions."""

import ctypes

import pytest
import torch

import rank_reductions_amd as rr
from rank_reductions_amd import rows
from test_rows_cpu import INVAL, NR, OK, R, embedding_calls, exchange_calls, route_call


@pytest.fixture
def lib():
    lib = rr.library()
    lib.rc_reset()
    yield lib
    lib.rc_reset()


def register(lib, ranks):
    cfg = rr.make_config(validate_only=True)
    assert lib.rc_register(ranks, ctypes.byref(cfg)) == OK


def session_id(lib):
    n = ctypes.c_int64(-1)
    assert lib.rc_session_id(ctypes.byref(n)) == OK
    return n.value


def statuses(lib, session, monkeypatch, older=False):
    """Every row exchange's status, with `session` in the descriptors."""
    got = {}
    for grad, fn in ((False, lib.rc_route), (True, lib.rc_route_grad)):
        args, (d, *keep) = route_call(grad)
        d.session = session
        if older:
            d.struct_size = rows.RcRouteDesc.session.offset
        got[fn.__name__] = fn(*args)
    for name, cls, calls in (("RcExchangeDesc", rows.RcExchangeDesc, exchange_calls),
                             ("RcEmbeddingDesc", rows.RcEmbeddingDesc, embedding_calls)):
        with monkeypatch.context() as m:
            class With(cls):
                def __init__(self, *a):
                    super().__init__(*a)
                    self.session = session
                    if older:
                        self.struct_size = cls.session.offset
            m.setattr(rows, name, With)
            got.update(calls(lib))
    return got


def test_calls_of_a_closed_session_are_refused(lib, monkeypatch):
    register(lib, R)
    first = session_id(lib)
    assert first > 0 and session_id(lib) == first
    assert set(statuses(lib, first, monkeypatch).values()) == {OK}, lib.rc_last_error()
    assert set(statuses(lib, 0, monkeypatch).values()) == {OK}
    for ranks in (R, R // 2, R * 2, 1):  # as many ranks, fewer and more
        lib.rc_reset()
        register(lib, ranks)
        assert session_id(lib) != first
        assert set(statuses(lib, first, monkeypatch).values()) == {INVAL}
        assert b"closed" in lib.rc_last_error()
    lib.rc_reset()
    assert set(statuses(lib, first, monkeypatch).values()) == {NR}
    assert lib.rc_session_id(None) == NR


def test_descriptors_without_a_session(lib, monkeypatch):
    """The size of a descriptor that ends before it: what lies there is not read."""
    register(lib, R)
    assert set(statuses(lib, 12345, monkeypatch, older=True).values()) == {OK}
    assert set(statuses(lib, 12345, monkeypatch).values()) == {INVAL}
