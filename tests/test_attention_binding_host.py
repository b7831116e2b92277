"""The binding of the cache and attention calls, without a GPU: the tensors are stand-ins with
addresses of their own, the library one that records its calls."""
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
HERE = [0]  # the current device


class On:
    """torch.cuda.device for the stand-ins."""

    def __init__(self, dev):
        self.index = torch.device(dev).index

    def __enter__(self):
        HERE.append(self.index)

    def __exit__(self, *exc):
        HERE.pop()


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            gone = [a for a in args if isinstance(a, int) and a in GONE]
            assert not gone, f"{name} was given the address of a copy that is no longer held"
            self.calls.append(name)
            self.where = (HERE[-1], args[-1])  # current device, stream
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    GONE.clear()
    lib = Library()
    monkeypatch.setattr(attention, "_ready", lib)
    monkeypatch.setattr(attention, "_stream", lambda dev: 1000 + dev.index)
    monkeypatch.setattr(attention, "_current_device", lambda: HERE[-1], raising=False)
    monkeypatch.setattr(torch.cuda, "device", On)
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
    kw.pop("cache", None)
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


ARGS = {append: dict(k=((3, 2, 64), torch.bfloat16), v=((3, 2, 64), torch.bfloat16), slots=((3,), torch.int64),
                     q=((3, 8, 64), torch.bfloat16), positions=((3,), torch.int64), table=((9, 64), torch.float32),
                     q_out=((3, 8, 64), torch.bfloat16)),
        rope: dict(x=((3, 8, 64), torch.bfloat16), positions=((3,), torch.int64), table=((9, 64), torch.float32),
                   out=((3, 8, 64), torch.bfloat16)),
        attend: dict(q=((2, 3, 8, 64), torch.bfloat16), page_table=((2, 4), torch.int32), context_len=((2,), torch.int32),
                     tree=((2, 3, 3), torch.bool), out=((2, 3, 8, 64), torch.bfloat16))}


def on(call, device):
    kw = {n: Fake(*shape, dtype=dt, device=device) for n, (shape, dt) in ARGS[call].items()}
    return dict(kw, cache=cache(device))


@pytest.mark.parametrize("call,arg", [(c, n) for c in ARGS for n in (*ARGS[c], "cache") if (c, n) != (rope, "cache")])
@pytest.mark.parametrize("device", ["cuda:1", "cpu"])
def test_a_tensor_on_another_device_is_refused(lib, call, arg, device):
    kw = on(call, "cuda:0")
    if arg == "cache":
        if device == "cpu":
            return  # refused when the cache is made
        kw["cache"] = cache(device)
    else:
        shape, dt = ARGS[call][arg]
        kw[arg] = Fake(*shape, dtype=dt, device=device)
    with pytest.raises(ValueError):
        call(lib, **kw)
    assert not any(n in ("ternary_rope", "ternary_kv_append", "ternary_tree_attention") for n in lib.calls)


def test_read_refuses_slots_on_another_device(lib):
    for device in ("cuda:1", "cpu"):
        with pytest.raises(ValueError):
            tl.kv_read(cache(), Fake(3, dtype=torch.int64, device=device))
    assert not lib.calls


@pytest.mark.parametrize("call", list(ARGS))
def test_the_tensors_device_is_the_current_one_during_the_call(lib, call):
    """A kernel launched on a device's default stream runs on the current device, whose pointers
    the tensors of another device are not."""
    for device in (0, 1):
        call(lib, **on(call, f"cuda:{device}"))
        assert lib.where == (device, 1000 + device)
        assert HERE == [0]


def test_workspace_sizes_kept_are_bounded(lib):
    """A page table that grows by a page at a time makes a new size each time."""
    for wide in range(1, 3000):
        attend(lib, page_table=Fake(2, wide, dtype=torch.int32))
    assert lib.calls.count("ternary_tree_attention") == 2999
    assert len(attention._ws_bytes) <= 1024
