"""Paged KV-cache decode attention for GB300 (sm_103a).

* ``pa_decode``, ``pa_append_kv``, ``pa_copy_blocks``, ``pa_read_error`` --
  thin bindings of the C ABI in ``include/pa.h`` (libpa.so, CUDA kernels).
* ``pa_rope_append_kv``, ``pa_decode_tree``, ``pa_tree_verify``,
  ``pa_keep_kv`` -- a step of tree speculation over the cache: norms and rotary
  positions with the append, tree attention, the accepted path, and its tokens
  moved into place.  ``rope_inv_freq`` and ``tree_masks`` prepare their inputs.
* ``pa_append_kv_bs8``, ``pa_decode_bs8``, ``pa_decode_multi_bs8``,
  ``pa_copy_blocks_bs8``, ``pa_pack_blocks_bs8``, ``pa_unpack_blocks_bs8`` -- the
  8-bit cache with a scale for each block and KV head: quantising append, single
  tokens and chunks of any length over it, copy-on-write, and whole blocks from
  and to a 16-bit cache.  ``bs8_pool`` makes an empty pool.
* ``BlockManager`` -- host bookkeeping that builds block tables, slot
  mappings and copy-on-write copy lists.

The CUDA library is loaded on first use; without it every entry point raises.
"""

from ._lib import PagedAttentionError  # noqa: F401
from .block_manager import BlockManager  # noqa: F401
from .rope import rope_inv_freq  # noqa: F401
from .tree import tree_masks  # noqa: F401
from .ops import (  # noqa: F401
    make_shape,
    new_error_word,
    pa_append_kv,
    pa_copy_blocks,
    pa_append_kv_fp8,
    pa_copy_blocks_fp8,
    pa_decode,
    pa_decode_fp8,
    pa_decode_shared_prefix,
    pa_decode_multi,
    pa_decode_int4,
    pa_append_kv_int4,
    pa_copy_blocks_int4,
    int4_pool,
    pa_decode_workspace_bytes,
    pa_read_error,
    pa_set_decode_stall_ns,
    pa_decode_tree,
    pa_tree_verify,
    pa_keep_kv,
    pa_rope_append_kv,
    workspace_for,
    bs8_pool,
    bs8_scales,
    pa_append_kv_bs8,
    pa_copy_blocks_bs8,
    pa_decode_bs8,
    pa_decode_multi_bs8,
    pa_pack_blocks_bs8,
    pa_unpack_blocks_bs8,
)

__version__ = "0.1.0"
