"""``MX4``: vectors held as 4-bit codes (OCP Microscaling Formats v1.0, MXFP4: blocks of 32
values with one power-of-two scale) and the scores of queries against them, through
fgmm_mx4_encode / fgmm_mx4_decode / fgmm_mx4_scores (include/fgmm.h).  CUDA tensors only;
argument marshalling only.  Work runs on the current stream of the tensors' device."""
from __future__ import annotations

import ctypes
import threading

import torch

from . import _lib
from ._lib import LIB, check

_DTYPES = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}


_raw_stream = torch._C._cuda_getCurrentRawStream


def empty(n: int, d: int | None, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    """[n, d], or [n] without d (torch.empty takes half as long again)."""
    if d is not None:
        return torch.empty_strided((n, d), (d, 1), dtype=dtype, device=device)
    return torch.empty_strided((n,), (1,), dtype=dtype, device=device)


def call(fn, name: str, device: torch.device, *args) -> None:
    """fn(*args, current stream of `device`) with `device` as the current one."""
    i = device.index
    if i == torch.cuda.current_device():
        code = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            code = fn(*args, _raw_stream(i))
    if code:
        check(code, name)


_words: dict = {}   # the library's status word of each device: written only by a kernel that gave up
_reports: dict = {}   # how often each device's word has been found set, and cleared
_reports_lock = threading.Lock()


def _word(device: torch.device) -> torch.Tensor:
    """The device's status word.  Memory of the library, so that it does not matter what the first
    call is part of: a captured graph, another thread's first call, inference mode."""
    w = _words.get(device.index)
    if w is None:
        at = ctypes.c_void_p()
        with torch.cuda.device(device):
            check(LIB.fgmm_mx4_status_word(ctypes.byref(at)), "fgmm_mx4_status_word")
        with torch.inference_mode(False):
            w = torch.as_tensor(_Int32(at.value), device=device)
        _words[device.index] = w
    return w


class _Int32:
    """One int32 at a device address, for torch.as_tensor."""

    def __init__(self, at: int):
        self.__cuda_array_interface__ = {"shape": (1,), "typestr": "<i4", "data": (at, False),
                                         "version": 3}


def _rows(X: torch.Tensor, what: str):
    """(dtype code, rows, columns, row stride) of a 2-D tensor with contiguous rows."""
    if not (isinstance(X, torch.Tensor) and X.is_cuda and X.dim() == 2):
        raise ValueError(f"{what} must be a 2-D CUDA tensor")
    dt = _DTYPES.get(X.dtype)
    if dt is None:
        raise TypeError(f"{what} must be float32 or bfloat16")
    (n, d), (ld, one) = X.shape, X.stride()
    if d < 1:
        raise ValueError(f"{what} must have at least one dimension")
    if d > 1 and one != 1 or n > 1 and ld < d:
        raise ValueError(f"{what} rows must be contiguous and must not overlap")
    return dt, n, d, max(ld, d)


class MX4:
    """The rows of X [N, D] (float32 or bfloat16) as 4-bit codes: 4.25 bits a value.

    codes  : uint8 [N, ceil(D / 32) * 16], two codes a byte
    scales : uint8, tiles of 128 rows x 4 blocks as include/fgmm.h describes
    """

    def __init__(self, X: torch.Tensor):
        dt, N, D, ldx = _rows(X, "X")
        dev, nb = X.device, -(-D // _lib.MX4_BLOCK)
        self.shape, self._reports = (N, D), _reports.get(dev.index, 0)
        self.codes = empty(N, nb * 16, torch.uint8, dev)
        self.scales = empty(-(-N // 128) * -(-nb // 4) * 512, None, torch.uint8, dev)
        call(LIB.fgmm_mx4_encode, "fgmm_mx4_encode", dev, X.data_ptr(), dt, N, D, ldx,
             self.codes.data_ptr(), self.scales.data_ptr())

    @classmethod
    def from_codes(cls, codes: torch.Tensor, scales: torch.Tensor, D: int) -> "MX4":
        """Codes made earlier (kept by reference)."""
        if not (codes.is_cuda and scales.device == codes.device
                and codes.dtype == scales.dtype == torch.uint8 and codes.is_contiguous()
                and scales.is_contiguous() and codes.dim() == 2):
            raise ValueError("codes [N, bytes] and scales must be contiguous uint8 tensors on one GPU")
        N, nb = codes.shape[0], -(-D // _lib.MX4_BLOCK)
        if D < 1 or codes.shape[1] != nb * 16 or scales.numel() != -(-N // 128) * -(-nb // 4) * 512:
            raise ValueError("codes or scales have the wrong size for this D")
        self = cls.__new__(cls)
        self.shape, self.codes, self.scales = (N, D), codes, scales
        self._reports = _reports.get(codes.device.index, 0)
        return self

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()

    def decode(self, dtype: torch.dtype = torch.float32) -> torch.Tensor:
        """The rows that the codes stand for, [N, D], float32 or bfloat16 (exact in both; infinity where
        a scale of 2^126 or 2^127, which encoding never makes, takes a code beyond them)."""
        if dtype not in _DTYPES:
            raise TypeError("dtype must be float32 or bfloat16")
        N, D = self.shape
        dev = self.codes.device
        out = empty(N, D, dtype, dev)
        call(LIB.fgmm_mx4_decode, "fgmm_mx4_decode", dev, self.codes.data_ptr(),
             self.scales.data_ptr(), N, D, out.data_ptr(), _DTYPES[dtype], D)
        return out

    def scores(self, queries, alpha: float = 1.0, bias: torch.Tensor | None = None,
               dtype: torch.dtype = torch.float32) -> torch.Tensor:
        """alpha * queries @ rows.T + bias, [M, N].  queries: an MX4, or a [M, D] tensor, which
        is encoded first.  bias: float32 [N]."""
        N, D = self.shape
        dev = self.codes.device
        coded = isinstance(queries, MX4)
        if coded:
            (M, d), q_dev = queries.shape, queries.codes.device
        else:
            dt, M, d, ldq = _rows(queries, "queries")
            q_dev = queries.device
        if d != D:
            raise ValueError(f"queries have {d} dimensions, the codes {D}")
        if q_dev != dev:
            raise ValueError("queries and codes must be on one device")
        out_dt = _DTYPES.get(dtype)
        if out_dt is None:
            raise TypeError("dtype must be float32 or bfloat16")
        if bias is not None and not (bias.device == dev and bias.dtype == torch.float32
                                     and bias.shape == (N,) and bias.is_contiguous()):
            raise ValueError("bias must be a contiguous float32 [N] tensor on the codes' device")
        if coded:
            q_codes, q_scales = queries.codes.data_ptr(), queries.scales.data_ptr()
        else:
            nb = -(-D // _lib.MX4_BLOCK)
            split = -(-M * nb // 32) * 512    # (copies of scale tiles want their own 512 bytes)
            scratch = empty(split + -(-M // 128) * -(-nb // 4) * 512, None, torch.uint8, dev)
            q_codes = scratch.data_ptr()
            q_scales = q_codes + split
            call(LIB.fgmm_mx4_encode, "fgmm_mx4_encode", dev, queries.data_ptr(), dt, M, D, ldq,
                 q_codes, q_scales)
        out, word = empty(M, N, dtype, dev), _word(dev)
        call(LIB.fgmm_mx4_scores, "fgmm_mx4_scores", dev, q_codes, q_scales, M, self.codes.data_ptr(),
             self.scales.data_ptr(), N, D, alpha, None if bias is None else bias.data_ptr(),
             out.data_ptr(), out_dt, N, word.data_ptr())
        return out

    def status(self) -> int:
        """Synchronise with the current stream and return ERR_TIMEOUT if, since the last call on this
        MX4 (or since it was made), a bounded wait of any scores on its device expired; such scores
        are undefined.  The device has one status word: what one MX4 reads and clears, the others
        are told at their next call."""
        dev = self.codes.device
        word = _word(dev)
        with _reports_lock, torch.cuda.device(dev):
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the status cannot be read while a graph is captured")
            if int(word):
                word.zero_()
                torch.cuda.current_stream().synchronize()
                # counted after clearing: it covers what a kernel noted in between
                _reports[dev.index] = _reports.get(dev.index, 0) + 1
            reports = _reports.get(dev.index, 0)
            code = _lib.OK if reports == self._reports else _lib.ERR_TIMEOUT
            self._reports = reports
        return code

    def check_status(self):
        check(self.status(), "device status")
