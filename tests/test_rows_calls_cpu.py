"""What may change between a row exchange's arguments and its launch - the
session, the lists - on the CPU with validate_only sessions."""

import ctypes
import weakref

import pytest
import torch

import rank_reductions_amd as rr
from rank_reductions_amd import rows
from test_rows_cpu import INVAL, NR, OK, R, embedding_calls, exchange_calls, route_call


MAX_EXPERTS = 1024  # RC_MAX_EXPERTS


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


def test_too_many_experts_are_refused_before_their_counts_are_allocated(lib):
    register(lib, 2)
    experts = [torch.zeros(3, 2, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)]
    for n in (MAX_EXPERTS + 2, 2**30, 2**31 - 2):
        with pytest.raises(rr.CollectiveError) as e:
            rr.dispatch_plan(experts, n)
        assert e.value.code == INVAL
    with pytest.raises(ValueError, match="CUDA"):  # as far as host tensors go
        rr.dispatch_plan(experts, MAX_EXPERTS)


class Drops:
    """A number; while it is read, the lists are emptied, as by another thread."""

    def __init__(self, value, *lists):
        self.value, self.lists, self.alive = value, lists, []

    def act(self):
        refs = [weakref.ref(t) for x in self.lists for t in x]
        for x in self.lists:
            x.clear()
        self.alive += [r() is not None for r in refs]

    def __float__(self):
        self.act()
        return float(self.value)

    def __index__(self):
        self.act()
        return int(self.value)


def test_tensors_live_until_the_call_returns(lib):
    register(lib, 2)
    f = lambda *n: [torch.zeros(*n), torch.zeros(*n)]
    i = lambda *n: [torch.zeros(*n, dtype=torch.int32), torch.zeros(*n, dtype=torch.int32)]
    ids, tables, dy, logits, experts, dw, out = i(3), f(5, 8), f(3, 8), f(3, 8), i(3, 1), f(3, 1), f(3, 8)
    calls = [
        (lambda n: rr.embedding(ids, tables, scale=n), ids, tables),
        (lambda n: rr.embedding_grad(ids, dy, 10, scale=n), ids, dy),
        (lambda n: rr.route(logits, 1, scale=n), logits),
        (lambda n: rr.route_grad(logits, experts, dw, scale=n), logits, experts, dw),
        (lambda n: rr.dispatch_plan(experts, n), experts),
    ]
    for call, *lists in calls:
        kept = [list(x) for x in lists]
        copies = [[t.clone() for t in x] for x in lists]
        for x, c in zip(lists, copies):
            x[:] = c
        del copies, c
        drops = Drops(2, *lists)
        with pytest.raises(ValueError, match="CUDA"):
            call(drops)
        assert drops.alive and all(drops.alive)
        for x, k in zip(lists, kept):
            x[:] = k


def test_streams_are_the_sessions_gpu_s(lib, monkeypatch):
    """A handle is taken for one of the session's GPU, whichever is current, and a
    stream of another GPU refused: neither becomes the current stream unseen."""
    rr.register(2, device=1, validate_only=True)
    x = [torch.zeros(3, 8), torch.zeros(3, 8)]
    made = []

    class Entered(Exception):
        pass

    def external(handle, device=None):
        made.append((handle, device))
        return "external"

    def stream(s):
        made.append(s)
        raise Entered

    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "stream", stream)

    class Stream:
        cuda_stream = 77

        def __init__(self, index):
            self.device = torch.device("cuda", index)

    with pytest.raises(Entered):
        rr.route(x, 2, stream=77)
    assert made == [(77, 1), "external"]
    made.clear()
    with pytest.raises(rr.CollectiveError) as e:
        rr.route(x, 2, stream=Stream(0))
    assert e.value.code == INVAL and not made
    right = Stream(1)
    with pytest.raises(Entered):
        rr.route(x, 2, stream=right)
    assert made == [right]
    rr.reset()
    with pytest.raises(rr.CollectiveError) as e:
        rr.route(x, 2, stream=right)
    assert e.value.code == NR
