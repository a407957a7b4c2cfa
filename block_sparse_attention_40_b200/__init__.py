"""Qwen Sparse Attention (QSA) on NVIDIA B200 (sm_100a).

The kernels and the C ABI live in ``csrc/`` and build into ``lib/libqsa.so`` (declared in
``include/qsa.h``).  ``binding`` is the thin ctypes layer that tests and benchmarks call;
``workloads`` draws the seeded synthetic inputs.
"""
from .binding import (KVCache, PagedKVCache, Decoder, DeltaExtend, Evictor, Prefill, QSAError,  # noqa: F401
                      compress, gated_deltanet, gated_deltanet_extend, gated_deltanet_step,
                      index_scores, last_device_error, load, prefill, prefill_select, topk,
                      version)
