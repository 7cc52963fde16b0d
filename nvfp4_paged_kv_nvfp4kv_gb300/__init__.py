"""NVFP4 paged-KV attention decode / extend for GB300 (sm_103a).

The compute path is the C-ABI library libnvfp4kv.so (include/nvfp4kv.h),
built in-tree by ``build.build()``; this package only marshals arguments.
"""
from .api import (NvFp4KvError, PagedCache, Plan, default_sm_scale,  # noqa: F401
                  nvfp4kv_decode_attend, nvfp4kv_decode_merge, nvfp4kv_decode_plan,
                  nvfp4kv_decode_run, nvfp4kv_merge_states, nvfp4kv_quantize_append,
                  nvfp4kv_workspace_flags, nvfp4kv_decode_run_static,
                  nvfp4kv_static_workspace_flags,
                  nvfp4kv_decode_append_run, nvfp4kv_dequantize_paged)
from .step import (E4m3Cache, RopePlan, StepTable, nvfp4kv_build_page_table,  # noqa: F401
                   nvfp4kv_e4m3_append, nvfp4kv_e4m3_decode_run, nvfp4kv_norm_rope,
                   nvfp4kv_rope, nvfp4kv_rope_plan)
from .tree import (nvfp4kv_compact_tokens, nvfp4kv_copy_pages,  # noqa: F401
                   nvfp4kv_e4m3_compact_tokens, nvfp4kv_e4m3_copy_pages, nvfp4kv_fork_pages,
                   nvfp4kv_release_pages, nvfp4kv_tree_form, nvfp4kv_tree_masks,
                   nvfp4kv_tree_run)
