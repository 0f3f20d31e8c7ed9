"""GB300 (sm_103a) implementation of R-KV's decode-time KV-cache compression
step: a C-ABI CUDA library (``librkv.so``, include/rkv.h) and its thin Python
binding (``rkv``).  ``cache`` binds what a decode loop does with a paged cache
between two compressions: rotary positions, appends (plain and at 4 bits) and
attention.  Synthetic workloads live in ``workloads``."""
from .cache import (Q4Cache, RopePlan, alloc_attention_workspace, alloc_q4_cache,  # noqa: F401
                    rkv_attention_workspace_size, rkv_paged_append, rkv_paged_attention,
                    rkv_q4_append, rkv_q4_attention, rkv_q4_read, rkv_rope_apply)
from .rkv import (RkvError, alloc_workspace, load, rkv_compress, rkv_compress_noalloc, rkv_gather,  # noqa: F401
                  rkv_get_device_status, rkv_score, rkv_select, rkv_timing_enable,
                  rkv_timing_read, rkv_workspace_init, rkv_workspace_size)
