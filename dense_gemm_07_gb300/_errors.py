"""The error raised for a nonzero status of the library."""
from __future__ import annotations

from . import _abi as abi


class GemmError(RuntimeError):
    """A nonzero gemm_status_t from the library."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {abi.gemm_status_string(status)} (status {status})")
