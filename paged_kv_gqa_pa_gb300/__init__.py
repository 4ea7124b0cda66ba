"""GB300-native paged-KV grouped-query decode attention.

The C ABI (include/pa.h, include/pa_q4.h) lives in libpa_gb300.so, built from csrc/ for sm_103a;
``binding`` and ``q4`` expose it to Python under the same names.  The library is loaded
on the first call, never at import, so ``workloads`` (the seeded input
generator) imports without a GPU.
"""
from .binding import (PAError, decode, load, new_workspace, pa_decode, pa_decode_partitions,
                      pa_decode_static, pa_get_error, pa_get_error_ex, pa_merge, pa_plan,
                      pa_plan_ex, pa_plan_t, pa_status_string, pa_version, prepare_decode)

from .q4 import (new_q4_cache, pa_extend_tables, pa_q4_decode, pa_q4_page_bytes, pa_q4_plan,
                 pa_q4_plan_t, pa_q4_read, pa_q4_write, pa_rope_axes, prepare_q4_decode,
                 q4_decode)

__all__ = ["PAError", "decode", "load", "new_workspace", "pa_decode", "pa_decode_partitions",
           "pa_decode_static", "pa_get_error", "pa_get_error_ex", "pa_merge", "pa_plan",
           "pa_plan_ex", "pa_plan_t", "pa_status_string", "pa_version", "prepare_decode",
           "new_q4_cache", "pa_extend_tables", "pa_q4_decode", "pa_q4_page_bytes", "pa_q4_plan",
           "pa_q4_plan_t", "pa_q4_read", "pa_q4_write", "pa_rope_axes", "prepare_q4_decode",
           "q4_decode"]
