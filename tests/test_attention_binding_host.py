"""The binding of the cache and attention calls, without a GPU: the tensors are stand-ins with
addresses of their own, the library one that records its calls."""
import gc
import weakref

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl
from ternary_weight_linear_02_gb300 import attention


class Fake:
    """What the binding looks at of a tensor."""
    made = 0

    def __init__(self, *shape, dtype=torch.bfloat16, dense=True, device="cuda:0"):
        Fake.made += 1
        self.shape, self.dtype, self.device, self.dense = torch.Size(shape), dtype, torch.device(device), dense
        self.at, self.copies = 0x100000 * Fake.made, []

    @property
    def is_cuda(self):
        return self.device.type == "cuda"

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        st, n = [], 1 if self.dense else 2
        for s in reversed(self.shape):
            st.insert(0, n)
            n *= max(s, 1)
        return tuple(st) if i is None else st[i]

    def is_contiguous(self):
        return self.dense

    def contiguous(self):
        if self.dense:
            return self
        copy = Fake(*self.shape, dtype=self.dtype, device=self.device)
        self.copies.append(weakref.ref(copy, lambda r, at=copy.at: GONE.add(at)))
        return copy

    def data_ptr(self):
        return self.at


GONE = set()


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            gc.collect()
            gone = [a for a in args if isinstance(a, int) and a in GONE]
            assert not gone, f"{name} was given the address of a copy that is no longer held"
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    GONE.clear()
    lib = Library()
    monkeypatch.setattr(attention, "_ready", lib)
    monkeypatch.setattr(attention, "_stream", lambda dev: 0)
    monkeypatch.setattr(attention, "_ws_bytes", {})
    return lib


def cache(device="cuda:0", fmt="int8"):
    codes = [Fake(4, 2, 16, 64, dtype=torch.int8, device=device) for _ in "kv"]
    scales = [Fake(4, 2, 16, dtype=torch.float32, device=device) for _ in "kv"]
    return tl.KVCache(fmt, *codes, *scales)


def append(lib, **kw):
    a = dict(cache=cache(), k=Fake(3, 2, 64), v=Fake(3, 2, 64), slots=Fake(3, dtype=torch.int64), q=Fake(3, 8, 64),
             positions=Fake(3, dtype=torch.int64), table=Fake(9, 64, dtype=torch.float32), q_out=Fake(3, 8, 64))
    a.update(kw)
    c, k, v, s = (a.pop(n) for n in ("cache", "k", "v", "slots"))
    return tl.kv_append(c, k, v, s, **a)


def rope(lib, **kw):
    a = dict(x=Fake(3, 8, 64), positions=Fake(3, dtype=torch.int64), table=Fake(9, 64, dtype=torch.float32), out=Fake(3, 8, 64))
    a.update(kw)
    return tl.rope(a["x"], a["positions"], a["table"], out=a["out"])


def attend(lib, **kw):
    a = dict(q=Fake(2, 3, 8, 64), cache=cache(), page_table=Fake(2, 4, dtype=torch.int32), context_len=Fake(2, dtype=torch.int32),
             tree=Fake(2, 3, 3, dtype=torch.bool), out=Fake(2, 3, 8, 64))
    a.update(kw)
    return tl.tree_attention(a["q"], a["cache"], a["page_table"], a["context_len"], a["tree"], out=a["out"])


def strided(*shape, dtype):
    return Fake(*shape, dtype=dtype, dense=False)


@pytest.mark.parametrize("call,arg,shape,dtype", [
    (append, "slots", (3,), torch.int64), (append, "positions", (3,), torch.int64), (append, "k", (3, 2, 64), torch.bfloat16),
    (append, "v", (3, 2, 64), torch.bfloat16), (append, "q", (3, 8, 64), torch.bfloat16),
    (rope, "positions", (3,), torch.int64), (rope, "x", (3, 8, 64), torch.bfloat16),
    (attend, "q", (2, 3, 8, 64), torch.bfloat16), (attend, "page_table", (2, 4), torch.int32),
    (attend, "context_len", (2,), torch.int32), (attend, "tree", (2, 3, 3), torch.bool)])
def test_copies_live_until_the_call(lib, call, arg, shape, dtype):
    """A strided argument is copied; the copy's memory may not go back to the allocator, which would
    give it to the call's own output, before the work that reads it is enqueued."""
    t = strided(*shape, dtype=dtype)
    call(lib, **{arg: t})
    assert len(t.copies) == 1 and lib.calls[-1].startswith("ternary_")
