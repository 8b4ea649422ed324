"""Stand-ins for driving the torch binding without a GPU: CPU tensors that say they lie on a CUDA
device, a library whose entry points record their arguments, and a record of what was allocated
under which stream.  Both ways of marshalling (attention.py and csrc/marshal.c) read tensors
through their Python attributes, so both can be driven this way."""
import contextlib
import ctypes

import torch

I32, I64, F, P, S = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


class OnDevice(torch.Tensor):
    """A CPU tensor that says it lies on CUDA device `index`."""
    index = 0

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.index


class OnOther(OnDevice):
    index = 1


def on(t, index=0):
    return t.as_subclass(OnOther if index else OnDevice)


class Stream:
    """A side stream of a device."""

    def __init__(self, handle, index=0):
        self.cuda_stream, self.device = handle, torch.device("cuda", index)


SIGNATURES = dict(
    gdn_kv_append=[P] * 6 + [F] + [P] * 10,
    gdn_paged_attention=[P] * 11 + [S, P],
    gdn_shared_prefix_attention=[P] * 12 + [S, P],
    gdn_add_rmsnorm=[I64, I32, I32, P, P, P, F, P, P, P, I32, P],
)


class World:
    """The pretended machine: the current device and stream, calls made, tensors allocated."""

    def __init__(self, monkeypatch, shape_bytes):
        self.device, self.handle, self.calls, self.made = 0, 100, [], []
        real = {n: getattr(torch, n) for n in ("empty", "empty_like", "zeros")}

        def recording(name):
            def f(*args, **kw):
                kw.pop("device", None)
                t = on(real[name](*args, **kw), self.device)
                self.made.append((name, t.data_ptr(), t.nbytes, self.handle))
                return t
            return f

        for name in real:
            monkeypatch.setattr(torch, name, recording(name))

        @contextlib.contextmanager
        def stream(s):
            before = self.device, self.handle
            self.device, self.handle = s.device.index, s.cuda_stream
            yield
            self.device, self.handle = before

        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.device)
        monkeypatch.setattr(torch.cuda, "current_stream",
                            lambda device=None: Stream(self.handle, self.device))

        def entry(name, types):
            def call(*args):
                args = [a or 0 for a in args]
                if types[0] is P:
                    args[0] = ctypes.string_at(args[0], shape_bytes)
                self.calls.append((name, args))
                return 0
            return ctypes.CFUNCTYPE(ctypes.c_int, *types)(call)

        self.entries = {n: entry(n, t) for n, t in SIGNATURES.items()}

    def made_at(self, address):
        """(function, bytes, stream) of the allocation at this address."""
        return [(n, size, h) for n, a, size, h in self.made if a == address][-1]


class Library:
    """The recording entry points over the real library's size queries."""

    def __init__(self, world, real):
        self.__dict__.update(world.entries)
        self._real = real

    def __getattr__(self, name):
        return getattr(self._real, name)
