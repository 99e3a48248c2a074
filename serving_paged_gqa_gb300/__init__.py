"""Paged grouped-query decode attention for GB300 (sm_103a).

One decode step of attention over a block-table FP16 KV cache with three schedules (single-pass, rectangular
sequence split, compact device-built workqueue), a log-sum-exp merge, a device worklist builder and a host
roofline cost-model planner, all in libpkv.so (C ABI: include/pkv.h). This package is its Python binding. Prompts:
causal attention over packed sequences, their K/V into the FP16 pages or quantised into 4-bit pages, and the decode
step over 4-bit pages. Growing caches: tables of a step from the rows' lengths, attention of chunks of new tokens over the
pages, and a decode step over selected pages.
"""

from ._lib import (EXPORTS, LIB_PATH, PKV_MAX_BATCH, PKV_MAX_ROWS_IN_DECODE, PKV_MAX_SMS,  # noqa: F401
                   PKV_PLAN_INPUTS_AFTER_PREV,
                   PKV_PLAN_OVERLAP_PREV, PKV_PROMPT_WS_BYTES, PKV_Q4_BLOCK_BYTES, Prompt,
                   PKV_SESSION_GRAPHS, PKV_STATIC_SCRATCH_BYTES,
                   PKV_STATUS_BAD_LEN, PKV_STATUS_BAD_PAGE, PKV_STATUS_NO_PAGES, PKV_STATUS_TASKS, PKV_STATUS_TIMEOUT, PKV_VARIANT_SINGLE,
                   PKV_VARIANT_SPLIT, PKV_VARIANT_WORKQUEUE, VARIANT_NAMES, PkvError, load)
from .binding import (Plan, Policy, Problem, alloc_workspace, decode, make_problem, pkv_build_worklist,  # noqa: F401
                      pkv_check_problem, pkv_decode, pkv_decode_step, pkv_decode_step_append, pkv_decode_step_static,
                      pkv_merge, pkv_plan, pkv_plan_fixed, pkv_plan_launches, pkv_policy_default, pkv_read_status,
                      pkv_serve_step, pkv_step_input_layout, pkv_strerror, pkv_version, pkv_workspace_init, ServeSession,
                      ServeStep)
from .prompts import (make_prompt, pkv_check_prompt, pkv_prompt_append, pkv_prompt_attention,  # noqa: F401
                      pkv_q4_decode_step, pkv_q4_decode_step_append, pkv_q4_pool_bytes, pkv_q4_prompt_append, pkv_q4_read,
                      pkv_q4_workspace_bytes, prompt_append, prompt_attention, q4_decode, q4_problem, q4_prompt_append,
                      q4_read)
from .paged import (chunk_attention, page_bounds, pkv_chunk_attention, pkv_chunk_workspace_bytes,  # noqa: F401
                    pkv_page_bounds, pkv_select_pages, pkv_sparse_decode_step, pkv_sparse_workspace_bytes, pkv_tables_grow,
                    pkv_tables_release, select_pages, sparse_decode, sparse_problem, tables_grow, tables_release)
