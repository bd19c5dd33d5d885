"""sparse_paged_kv_gb300 -- the Locks decode-attention hot path on GB300 (sm_103a).

The compute lives in ``lib/libsparse_paged_kv.so`` (hand-written CUDA behind the
C ABI of ``include/locks.h``); ``binding`` marshals torch tensors into it and
``runtime`` bundles the buffers of one decode layer.
"""
from .binding import (LOCKS_KV_F8, LOCKS_KV_I4, LOCKS_KV_I8, LOCKS_SUMMARY_BF16,  # noqa: F401
                      LOCKS_SUMMARY_F32, LocksConfig, LocksError, LocksKvConfig,
                      LocksLibraryMissing, load_library, locks_build_summaries,
                      locks_dense_decode, locks_kv_decode, locks_kv_read, locks_kv_write,
                      locks_rope, locks_select, locks_sparse_decode, unpack_records)
