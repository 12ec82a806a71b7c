"""Argument checks and launch context shared by the operator bindings."""
from __future__ import annotations

import torch


def tensor(name: str, t, dtypes, shape=None, device=None, contiguous: bool = True):
    """t, if it is a CUDA tensor of one of the dtypes, of the shape, on the device."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a tensor of {' or '.join(str(d) for d in dtypes)}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda or (device is not None and t.device != device):
        raise TypeError(f"{name} must be on {device if device is not None else 'a CUDA device'}")
    return t


def launch_on(device: torch.device, stream):
    """Makes `device` and the launching stream current: what is allocated inside
    (outputs, workspaces) then belongs to the stream that uses it."""
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def pointer(t):
    return None if t is None else t.data_ptr()
