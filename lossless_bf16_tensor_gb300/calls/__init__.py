"""Loads _calls.so, the Python entry points of the gradient, adapter and vocabulary calls
(``calls.cpp``).  There is no fallback: importing this fails if the library has
not been built (``python -m lossless_bf16_tensor_gb300.build``)."""
from __future__ import annotations

import importlib.util
import os

import torch  # noqa: F401  (its libraries have to be loaded first)

from ..binding import LctError

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "_calls.so")

if not os.path.exists(PATH):
    raise ImportError("_calls.so is not built (run `python -m lossless_bf16_tensor_gb300.build`)")

_spec = importlib.util.spec_from_file_location("_calls", PATH)
calls = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(calls)
calls.set_error(LctError)
