"""Where the binding takes memory and on which device and stream it calls, with stand-ins
for device tensors and for the library (no GPU needed).

torch's allocator orders a block's uses only within the stream it was allocated on: a
block that an earlier call on the current stream has given back is handed out again at
once, while that call's kernels may still run.  So what a call on another stream works in
has to come from that stream."""
import contextlib
import ctypes

import pytest
import torch


class Fake:
    """What the binding asks of a device tensor."""

    def __init__(self, shape, dtype, device=1, took=None):
        self.t = torch.zeros(shape, dtype=dtype)
        self.shape, self.dtype, self.device, self.is_cuda = self.t.shape, dtype, torch.device("cuda", device), True
        self.nbytes, self.took, self.recorded = self.t.nbytes, took, []

    def get_device(self):
        return self.device.index

    def stride(self, *i):
        return self.t.stride(*i)

    def data_ptr(self):
        return self.t.data_ptr() or 16

    def is_contiguous(self):
        return True

    def record_stream(self, s):
        self.recorded.append(s)


class Stream:
    def __init__(self, n):
        self.cuda_stream = n


@pytest.fixture
def gpu(monkeypatch):
    """A machine of two devices with device 0 and its stream 100 current; `calls` lists the
    library's calls as (name, current device, stream)."""
    from depth_planed_kv_b200 import build as B
    B.build()
    from depth_planed_kv_b200 import ripe

    class State:
        device, current, taken, calls = 0, Stream(100), [], []
    st = State()

    @contextlib.contextmanager
    def stream(s):
        before, st.current = st.current, s
        yield
        st.current = before

    @contextlib.contextmanager
    def device(d):
        before, st.device = st.device, torch.device(d).index
        yield
        st.device = before

    def empty(shape, dtype=None, device=None):
        st.taken.append(Fake(shape, dtype, torch.device(device).index, st.current))
        return st.taken[-1]

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: st.device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: st.current)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: st.current.cuda_stream + d, raising=False)
    monkeypatch.setattr(torch, "empty", empty)

    def entry(name):
        def call(*a):
            s = a[-1].value if isinstance(a[-1], ctypes.c_void_p) else a[-1]
            st.calls.append((name, st.device, s))
            return 0
        monkeypatch.setattr(ripe._lib, name, call)
    for name in ("ripe_paged_attn", "ripe_paged_append", "ripe_sample", "ripe_accept"):
        entry(name)

    def bytes_(pages, H, n, out):
        ctypes.cast(out, ctypes.POINTER(ctypes.c_size_t))[0] = 4096
        return 0
    monkeypatch.setattr(ripe._lib, "ripe_paged_attn_workspace", bytes_)
    monkeypatch.setattr(ripe, "_work_bytes", {})
    st.ripe = ripe
    return st


def paged(gpu, stream, device=1, work=None):
    i32, bf = torch.int32, torch.bfloat16
    k, v = Fake((4, 2, 16, 64), bf, device), Fake((4, 2, 16, 64), bf, device)
    q, o = Fake((3, 4, 64), bf, device), Fake((3, 4, 64), bf, device)
    n = Fake((3, 2, 64), bf, device)
    batch = Fake((2, 2), i32, device), Fake((2,), i32, device), Fake((3,), i32, device)
    gpu.ripe.ripe_paged_append(n, n, k, v, *batch, stream=stream)
    gpu.ripe.ripe_paged_attn(q, k, v, *batch, o, max_ntok=2, work=work, stream=stream)


def test_work_space_of_another_stream_comes_from_that_stream(gpu):
    s = Stream(7)
    gpu.device = 1
    paged(gpu, s)
    assert [t.took for t in gpu.taken] == [s]
    assert gpu.current.cuda_stream == 100
    assert [c[2] for c in gpu.calls] == [7, 7]
    paged(gpu, None)
    assert gpu.taken[-1].took is gpu.current and [c[2] for c in gpu.calls[2:]] == [101, 101]
    paged(gpu, s, work=Fake((4096,), torch.uint8))   # the caller's own: nothing is taken
    assert len(gpu.taken) == 2


def test_outputs_of_another_stream_come_from_it_and_are_known_to_the_callers(gpu):
    s, mine = Stream(7), gpu.current
    gpu.device = 1
    out = gpu.ripe.ripe_sample(Fake((2, 10), torch.float32), Fake((2,), torch.float32), stream=s)
    assert [t.took for t in out] == [s, s] and all(t.recorded == [mine] for t in out)
    f = Fake((2, 3, 10), torch.float32)
    x = Fake((2, 3), torch.int32)
    out = gpu.ripe.ripe_accept(f, f, None, x, None, Fake((2, 3, 3), torch.float32), 1.0, stream=s)
    assert [t.took for t in out] == [s] * 3 and all(t.recorded == [mine] for t in out)
    assert [c[2] for c in gpu.calls] == [7, 7]
    out = gpu.ripe.ripe_sample(Fake((2, 10), torch.float32), Fake((2,), torch.float32))
    assert [t.took for t in out] == [mine, mine] and not any(t.recorded for t in out)


def test_calls_run_on_the_tensors_device(gpu):
    paged(gpu, None)
    gpu.ripe.ripe_sample(Fake((2, 10), torch.float32), Fake((2,), torch.float32))
    assert [c[1] for c in gpu.calls] == [1, 1, 1] and gpu.device == 0
    assert all(t.device.index == 1 for t in gpu.taken)


def test_tensors_of_two_devices_are_refused(gpu):
    with pytest.raises(AssertionError):
        gpu.ripe.ripe_sample(Fake((2, 10), torch.float32, 1), Fake((2,), torch.float32, 0))
    i32, bf = torch.int32, torch.bfloat16
    for other in range(5):
        dev = [1] * 5
        dev[other] = 0
        k = Fake((4, 2, 16, 64), bf)
        q, o = Fake((3, 4, 64), bf, dev[0]), Fake((3, 4, 64), bf, dev[1])
        batch = Fake((2, 2), i32, dev[2]), Fake((2,), i32, dev[3]), Fake((3,), i32, dev[4])
        with pytest.raises(AssertionError):
            gpu.ripe.ripe_paged_attn(q, k, k, *batch, o, max_ntok=2)
    assert not gpu.calls
