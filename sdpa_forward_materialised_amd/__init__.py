"""MI355X-native materialised-probability SDPA forward.

``fwd(q, k, v, attn_mask=None, is_causal=False, scale=None, enable_gqa=False)``
returns ``(O, P, LSE)``: the attention output, the full probability map and
the float32 row log-sum-exp, computed by hand-written gfx950 HIP kernels in
``libsdpa_math.so`` (C ABI declared in ``include/sdpa_math.h``). This package
is argument marshalling only; torch supplies device memory and streams.

For serving (``include/sdpa_serve.h``): ``prompt_attention`` and
``key_weights`` over packed prompts without the probability map, and a paged
8-bit cache (``PagedCache``, ``new_cache``) with ``cache_append``,
``cache_attention`` and ``cache_evict``.
"""

from ._binding import (EXPORTS, LIB_PATH, PATHS, SdpaMathFunction, bwd, fwd, fwd_noalloc, fwd_varlen,  # noqa: F401
                       PreparedFwd, kernel_name, last_error, load_library, plan, prepare_fwd, probe_copy, probe_fill, sdpa_math, version)
from ._serving import (PagedCache, cache_append, cache_attention, cache_evict, key_weights, new_cache,  # noqa: F401
                       prompt_attention)

__all__ = ["fwd", "fwd_noalloc", "fwd_varlen", "bwd", "sdpa_math", "SdpaMathFunction", "plan", "kernel_name", "prepare_fwd", "PreparedFwd", "version", "last_error",
           "prompt_attention", "key_weights", "PagedCache", "new_cache", "cache_append", "cache_attention", "cache_evict",
           "load_library", "LIB_PATH", "PATHS", "EXPORTS"]
