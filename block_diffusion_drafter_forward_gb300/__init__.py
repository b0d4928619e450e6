"""GB300 (sm_103a) DFlash drafter gamma-block forward behind a C ABI (libdflash.so)."""
from . import _lib  # noqa: F401
from ._lib import (DflashError, dflash_attention_check, dflash_create, dflash_destroy, dflash_device_status,  # noqa: F401
                   dflash_fp8_layer, dflash_fp8_lm_head, dflash_gemm_bf16, dflash_gemm_bf16_noalloc, dflash_kv_layout, dflash_last_error, dflash_profile,
                   dflash_persistent, dflash_profile_read, dflash_propose, dflash_set_persistent, dflash_write_ctx_kv)
from ._lib import dflash_append_kv, dflash_attend, dflash_attend_workspace, dflash_extend_tables, dflash_extend_tables_ex, dflash_sample, dflash_take_status  # noqa: F401
from ._lib import dflash_append_kv_quant, dflash_attend_ex, dflash_draft_tree, dflash_keep_rows, dflash_read_kv_quant, dflash_rope_turns, dflash_rotate  # noqa: F401
from .drafter import Drafter, make_cfg  # noqa: F401
from .serve import PagedKV, QuantKV, Rope, RowPlan, TreePlan, draft_tree, extend_tables, sample, serve_status  # noqa: F401
