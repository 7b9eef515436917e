"""What the tensor helpers share: dtype codes, row layouts, and the device and
stream that a call runs on."""
from __future__ import annotations

import torch

from ._abi import DYT_BF16, DYT_F16, DYT_F32, lib

DTYPE_CODE = {torch.float32: DYT_F32, torch.bfloat16: DYT_BF16, torch.float16: DYT_F16}


def _code(t: torch.Tensor, what: str) -> int:
    try:
        return DTYPE_CODE[t.dtype]
    except KeyError:
        raise TypeError(f"{what}: dtype {t.dtype} is not supported (float32, bfloat16, float16)") from None


def _cuda_contig(t: torch.Tensor, what: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def row_pitch(t: torch.Tensor) -> int | None:
    """Elements between consecutive rows when t's leading dimensions collapse into
    one row index with a uniform pitch and its last dimension is dense; else None."""
    if t.dim() == 0:
        return None
    if t.dim() == 1:
        return t.shape[0] if t.shape[0] <= 1 or t.stride(0) == 1 else None
    shape, stride = t.shape, t.stride()
    N, ld = shape[-1], stride[-2]
    if N > 1 and stride[-1] != 1:
        return None
    n, step = shape[-2], ld  # of the last dimension with more than one step (others have no stride that matters)
    for i in range(len(shape) - 3, -1, -1):
        if shape[i] > 1:
            if n <= 1:
                ld = stride[i]
            elif stride[i] != n * step:  # dimension i must step over whole blocks of the next
                return None
            n, step = shape[i], stride[i]
    if ld < N and t.numel() > N:
        return None
    return ld if ld > N else N


def _rows(t: torch.Tensor, what: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    ld = row_pitch(t)
    if ld is None:
        raise ValueError(f"{what}: rows must be dense and evenly spaced (stride 1 along the last dimension)")
    return ld


def _stream(device, stream):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _current(index: int) -> int:
    """The current stream of a device, as the library takes it. (The raw handle: making a
    torch.cuda.Stream object for it costs as much as a launch, 2 to 3 us.)"""
    return torch._C._cuda_getCurrentRawStream(index)


def _pitch(t: torch.Tensor, what: str) -> int:
    """The row pitch of a CUDA tensor; contiguous ones need no look at their strides, and
    ordinary matrices one."""
    if t.is_contiguous() and t.dim():
        return t.shape[-1]
    if t.dim() == 2 and t.is_cuda:
        ld, inner = t.stride()
        if inner == 1 and ld >= t.shape[1]:
            return ld
    return _rows(t, what)


def _fresh(t: torch.Tensor) -> torch.Tensor:
    """An uninitialised contiguous tensor of t's shape, dtype and device. (empty_like of a
    contiguous tensor takes 1.3 us, empty_strided 1.4, torch.empty of its shape 3.3.)"""
    if t.is_contiguous():
        return torch.empty_like(t)
    if t.dim() == 2:
        return torch.empty_strided(t.shape, (t.shape[1], 1), dtype=t.dtype, device=t.device)
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _fresh_rows(rows: torch.Size, device: torch.device) -> torch.Tensor:
    """An uninitialised float32 value per row. (empty_strided takes 1.4 us, torch.empty of a shape 3.)"""
    if len(rows) == 1:
        return torch.empty_strided((rows[0],), (1,), dtype=torch.float32, device=device)
    return torch.empty(rows, dtype=torch.float32, device=device)


def _fresh_matrix(rows: torch.Size, n: int, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    """An uninitialised contiguous tensor of n values per row. (empty_strided takes 1.5 us, torch.empty of a
    shape 2.3 to 3.)"""
    if len(rows) == 1:
        return torch.empty_strided((rows[0], n), (n, 1), dtype=dtype, device=device)
    return torch.empty((*rows, n), dtype=dtype, device=device)


_sizes: dict = {}


def _bytes(name: str, index: int, *args: int) -> int:
    """The workspace size that the library's call `name` gives for args on device `index`, the current one: it depends
    on nothing else. (A question takes 0.7 us, a look here 0.2. 0 is no size to keep: it may stand for an error.)"""
    key = (name, index, args)
    n = _sizes.get(key)
    if n is None:
        n = getattr(lib, name)(*args)
        if n:
            if len(_sizes) >= 1024:
                _sizes.clear()
            _sizes[key] = n
    return n


def _scratch(n: int, device: torch.device) -> torch.Tensor:
    """An uninitialised workspace of at least n bytes."""
    return torch.empty_strided((n if n > 16 else 16,), (1,), dtype=torch.uint8, device=device)


def _elsewhere(index: int, stream: torch.cuda.Stream | None) -> bool:
    """Whether a call on the data of device `index` (a tensor's get_device()) has to
    switch the current device or stream (see _there)."""
    if index < 0:
        raise ValueError("the tensors must be CUDA tensors")
    return stream is not None or index != torch._C._cuda_getDevice()


def _there(t: torch.Tensor, stream: torch.cuda.Stream | None):
    """A context in which t's device is the current one and `stream`, if given, the
    current stream: what the call allocates then belongs to the stream that uses it."""
    if stream is None:
        return torch.cuda.device(t.device)
    if stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    return torch.cuda.stream(stream)


def _vector(t: torch.Tensor, what: str, n: int, index: int, dtypes) -> int:
    """The address of a contiguous tensor of n elements on device `index`."""
    if t.get_device() == index and t.dtype in dtypes and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != index:
        raise ValueError(f"{what} must be on cuda:{index}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: dtype {t.dtype} is not supported ({', '.join(str(d)[6:] for d in dtypes)})")
    if t.numel() != n:
        raise ValueError(f"{what} must have {n} elements, not {t.numel()}")
    raise ValueError(f"{what} must be contiguous")


def _like(t: torch.Tensor, what: str, x: torch.Tensor) -> int:
    """The row pitch of a tensor of x's shape, dtype and device."""
    if t.shape != x.shape or t.dtype != x.dtype or t.get_device() != x.get_device():
        raise ValueError(f"{what} must match its input in shape, dtype and device")
    return _pitch(t, what)


def _rows_of(x: torch.Tensor, what: str) -> tuple[int, int, int, int]:
    """(rows, elements of a row, row pitch, dtype code) of an input on the current device. (One look at each
    property: 0.5 us, through _pitch and _code 0.8.)"""
    shape = x.shape
    if not shape:
        raise ValueError(f"{what} must have at least one dimension")
    N, code = shape[-1], DTYPE_CODE.get(x.dtype)
    if code is None:
        _code(x, what)
    return x.numel() // N if N else 0, N, N if x.is_contiguous() else _pitch(x, what), code


def _workspace(ws: torch.Tensor, index: int) -> int:
    if ws.get_device() != index or not ws.is_contiguous() or ws.dtype != torch.uint8:
        raise ValueError(f"ws must be a contiguous uint8 tensor on cuda:{index}")
    return ws.data_ptr()
