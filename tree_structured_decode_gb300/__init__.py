"""Tree-structured decode attention on GB300 (sm_103a).

Thin Python binding over the C ABI of ``libtreeattn.so`` (declared in
``include/tree_attn.h``): argument marshalling only.  Every step of the
attention runs in the library's CUDA kernels; PyTorch supplies device memory
and streams.  There is no CPU fallback: if the library is missing, importing
the binding's entry points raises.

    plan = Plan(parent, node_kv_len, node_page_offsets, node_pages, num_pages,
                query_node, query_kv_end, n_q_heads, n_kv_heads, head_dim)
    out, lse = plan.run(q, k_pages, v_pages)

A decode loop whose lengths live on the GPU, so that one captured step serves
all steps, has ``extend_tables``, ``append_slots``, ``prefix_attention`` and
``sample``; they hold no state.
"""
from ._abi import (  # noqa: F401
    LIB_PATH,
    Options,
    PlanStats,
    TreeAttnError,
    load_library,
    status_string,
)
from .api import Plan, plan, run  # noqa: F401
from .batch import append_slots, extend_tables, prefix_attention, sample  # noqa: F401

__all__ = ["Plan", "plan", "run", "extend_tables", "append_slots", "prefix_attention", "sample",
           "Options", "PlanStats", "TreeAttnError",
           "load_library", "status_string", "LIB_PATH"]
