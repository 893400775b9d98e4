"""Tensors and streams that say they are on a GPU, for host-side tests of the checks that
the calls make before the library is entered."""
import torch


class OnDevice(torch.Tensor):
    dev = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.dev


def on_device(*shape, dtype=torch.bfloat16, dev=0):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)
    t.dev = dev
    return t


class Stream:
    cuda_stream = 0

    def __init__(self, dev=0):
        self.device_index = dev
