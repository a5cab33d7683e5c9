"""Dynamic-vocabulary draft LM head (NanoSpec / MicroSpec) for GB300 (sm_103a).

The compute path is the C-ABI library ``libnanospec.so`` (include/nanospec.h,
include/nanospec_ops.h), built from ``csrc/`` by ``build.build()``; ``nanospec``
is the ctypes binding of the draft head, ``serving`` of the operators around it.
"""

from .nanospec import (  # noqa: F401
    EXPORTED,
    FLAG_BAD_ID,
    FLAG_OVERFLOW,
    FLAG_TIMEOUT,
    Handle,
    NanoSpecError,
    load_library,
)
from .serving import (  # noqa: F401
    FLAG_BAD_SEQ,
    FLAG_NO_PAGES,
    FLAG_SHARED_PAGE,
    KvPages,
    TokenLogprobs,
    attend_paged,
    attend_prompt,
    attend_shared,
    norm_rotate,
    ops_error,
    token_logprobs,
)
