"""Copies of a Config or Router that was used: a copy, a deep copy, a pickle's other end
and an object of replaced fields each hand out the address of a C struct of their own,
with the fields' values, and never one that their original holds (which may be gone, or
in another process). CPU only."""
import copy
import ctypes
import dataclasses
import gc
import pickle

import pytest

from combine_ep_layout_10_amd import _ffi as F
from combine_ep_layout_10_amd import ops

OBJECTS = {
    "config": lambda: ops.Config(max_tokens=40, hidden=64, num_experts=8, num_topk=2, expert_alignment=16, idx_bits=32),
    "router": lambda: ops.Router(24, 3, ops.SCORE_SIGMOID, 4, 2, 2, True, 2.5, 32),
}
COPIES = {"copy": copy.copy, "deepcopy": copy.deepcopy, "replace": dataclasses.replace}
COPIES.update({"pickle%d" % p: lambda o, p=p: pickle.loads(pickle.dumps(o, p)) for p in range(pickle.HIGHEST_PROTOCOL + 1)})


def values(struct):
    return [getattr(struct, n) for n, _ in struct._fields_]


@pytest.mark.parametrize("how", sorted(COPIES))
@pytest.mark.parametrize("kind", sorted(OBJECTS))
def test_a_copy_has_its_own_struct(kind, how):
    o = OBJECTS[kind]()
    struct, address = o.c(), o.c_addr()
    if kind == "config":
        bound = o.recv_rows_bound()
    want = values(struct)
    new = COPIES[how](o)
    assert new == o and hash(new) == hash(o)
    assert new.c_addr() == ctypes.addressof(new.c()) != address
    assert values(new.c()) == want
    assert o.c() is struct and o.c_addr() == address  # the original's stays
    del o, struct
    gc.collect()
    read = type(new.c()).from_address(new.c_addr())
    assert values(read) == want
    if kind == "config":
        assert new.recv_rows_bound() == bound


@pytest.mark.parametrize("kind", sorted(OBJECTS))
def test_a_state_with_an_address_in_it(kind):
    """What an earlier version pickled held the address, too: it is not taken over."""
    o = OBJECTS[kind]()
    state = dict({f.name: getattr(o, f.name) for f in dataclasses.fields(o)}, _c_struct=o.c(), _c_addr=12345)
    new = type(o).__new__(type(o))
    if hasattr(new, "__setstate__"):
        new.__setstate__(state)
    else:
        vars(new).update(state)
    assert new == o and new.c_addr() == ctypes.addressof(new.c()) != 12345


def test_copies_of_unused_objects():
    """A copy of an object that was never used, and one whose struct alone was built."""
    for make in OBJECTS.values():
        for prepare in (lambda o: None, lambda o: o.c()):
            o = make()
            prepare(o)
            new = copy.deepcopy(o)
            assert new.c_addr() == ctypes.addressof(new.c())
            assert isinstance(new.c(), (F.ep_config, F.ep_router))


def test_two_threads_get_one_struct(monkeypatch):
    """Two first calls at once: a struct that another thread's replaced would leave its address dangling."""
    import threading
    for kind in sorted(OBJECTS):
        o = OBJECTS[kind]()
        both = threading.Barrier(2)
        build = type(o)._struct

        def slow(self):
            c = build(self)
            both.wait(10)  # both threads have built theirs
            return c

        monkeypatch.setattr(type(o), "_struct", slow)
        got = []
        threads = [threading.Thread(target=lambda: got.append(o.c_addr())) for _ in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert got == [ctypes.addressof(o.c())] * 2
