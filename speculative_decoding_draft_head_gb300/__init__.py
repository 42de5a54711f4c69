"""GB300-native DSpark draft-sample / schedule / verify hot path.

The compute lives in libdspark.so (CUDA for sm_103a, C ABI in include/dspark.h);
this package holds the build step, the ctypes binding and the seeded workload
generators.
"""
from .binding import (DSparkError, KVCache, Rotary, block_attention, draft_sample, kv_append, kv_append_rotary, kv_read,
                      load, read_device_flags, rotary, schedule_prefix, verify, version, window_attention,
                      workspace_bytes)

__all__ = ["DSparkError", "KVCache", "Rotary", "block_attention", "draft_sample", "kv_append", "kv_append_rotary", "kv_read",
           "load", "read_device_flags", "rotary", "schedule_prefix", "verify", "version", "window_attention",
           "workspace_bytes"]
