"""Workspace's bookkeeping, on host buffers: what a captured graph holds stays allocated, a
capture gets no buffer that only its own replay would zero, and kinds of calls do not share
one."""
import gc
import weakref

import pytest
import torch

import int8_weight_quantized_int4_gb300 as q


@pytest.fixture
def capture(monkeypatch):
    """A switch: the number of the graph being captured, 0 for none."""
    now = [0]
    monkeypatch.setattr(q, "_capture_id", lambda index: now[0], raising=False)

    def switch(n):
        now[0] = n
    return switch


def host_workspace():
    ws = q.Workspace("cpu")
    ws._index = 0                       # as a device's, so that captures are asked for
    return ws


def test_growth_keeps_the_buffer_a_graph_was_captured_with(capture):
    ws = host_workspace()
    small, _ = ws.get_bytes(100)
    capture(1)
    assert ws.get_bytes(100)[0] is small
    capture(0)
    alive = weakref.ref(small)
    del small
    big, n = ws.get_bytes(1000)
    gc.collect()
    assert n == 1000 and ws.get_bytes(100)[0] is big
    assert alive() is not None and alive().data_ptr() != big.data_ptr()


def test_growth_without_a_capture_gives_the_buffer_back(capture):
    ws = host_workspace()
    alive = weakref.ref(ws.get_bytes(100)[0])
    ws.get_bytes(1000)
    gc.collect()
    assert alive() is None


def test_a_buffer_made_in_a_capture_serves_that_graph_only(capture):
    """Its zero-fill is a node of the graph: no other graph, and no eager call, may rely on it."""
    ws = host_workspace()
    capture(1)
    a, n = ws.get_bytes(100)
    assert n == 100 and not a.any() and ws.get_bytes(100)[0] is a
    a.fill_(1)
    capture(2)
    b, _ = ws.get_bytes(100)
    assert b is not a and not b.any()
    assert ws.get_bytes(200)[1] == 200
    capture(0)
    c, _ = ws.get_bytes(100)
    assert c is not a and c is not b and not c.any()
    capture(3)
    assert ws.get_bytes(100)[0] is c                             # one made before serves every graph
    assert ws.get_bytes(200)[1] == 200
    capture(0)
    assert ws.get_bytes(100)[0] is c


def test_kinds_of_calls_have_their_own_buffers():
    ws = host_workspace()
    ws._index = -1
    a, b = ws.get_bytes(100, "paged")[0], ws.get_bytes(100, "logprobs")[0]
    assert a is not b and ws.buf is b
    assert ws.get_bytes(50, "paged")[0] is a and ws.buf is a
    a.fill_(1)
    b.fill_(1)
    ws.zero()
    assert not a.any() and not b.any()
    assert ws.get_bytes(0, "paged") == (None, 0)


def test_every_kind_of_call_names_its_kind(monkeypatch):
    """One Workspace passed to calls of different kinds: none sees another's bytes.  (The calls
    end at the lookup, before any launch.)"""
    class Seen(Exception):
        pass
    kinds = []

    class Ws:
        def get(self, *a):
            kinds.append("gemm")
            raise Seen

        def get_bytes(self, need, kind="gemm"):
            kinds.append(kind)
            raise Seen
    monkeypatch.setattr(q, "_current_device", lambda: 0)
    for name in ("paged", "logprobs"):
        with pytest.raises(Seen):
            q._scratch(Ws(), 0, 0, name, lambda *a: 1)
    assert kinds == ["paged", "logprobs"]


def test_leading_zero_bytes_that_depend_on_the_call(capture):
    """A call leaves its own leading bytes zero and may write the others: a later call that needs
    more of them zero finds them so, whatever ran between, and graphs keep theirs."""
    ws = host_workspace()

    def call(need, zero):
        buf, n = ws.get_bytes(need, "topk", zero)
        assert n >= need and not buf[:zero].any(), (need, zero)
        buf[zero:need] = 7
        return buf
    a = call(1000, 300)
    assert call(200, 50) is a and call(1000, 300) is a and call(800, 290) is a and call(900, 600) is a
    capture(1)
    g1 = call(900, 600)
    own = call(900, 100)                                # a capture's own: its graph zero-fills it
    assert g1 is a and own is not a
    capture(0)
    b = call(500, 100)                                  # others leave the graph's buffer alone
    assert b is not a and call(900, 600) is a and call(500, 100) is b
    capture(2)
    assert call(900, 600) is a and call(500, 100) is b
    capture(0)
    assert call(500, 100) is b and call(400, 30) is not b and call(400, 30) is not a
