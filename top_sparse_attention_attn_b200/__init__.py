"""Top-k index-selected sparse attention (forward + backward) for one NVIDIA B200.

The compute lives in libsparse_attn.so (CUDA, sm_100a) behind the C ABI of
include/sparse_attn.h; `_lib` is its ctypes binding and `api.SparseAttention`
a thin wrapper that marshals torch tensors into it; `kv8.Kv8Cache` and
`kv8.plan_pages` do the same for serving over a paged KV cache held in 8 bits.
"""

from . import _lib
from ._lib import SaError
from .api import SparseAttention, indexer_kl_grad
from .kv8 import Kv8Cache, PagePlan, plan_pages

__all__ = ["SparseAttention", "SaError", "_lib", "indexer_kl_grad", "Kv8Cache", "PagePlan", "plan_pages"]
