"""Sliding Tile Attention for NVIDIA B200 (sm_100a).

The compute path lives in libsta.so (C ABI: include/sta.h); ``sta`` is its thin
ctypes binding; ``window`` (causal sliding-window attention with sinks over
token sequences) and ``kv_cache`` (an 8-bit key/value cache and attention over
it) bind the token-sequence calls.  ``workloads`` holds the seeded synthetic problem shapes.
"""
from .sta import (Plan, Problem, StaError, sliding_tile_attention, sta_backward, sta_forward, sta_forward_host,
                  sta_permute,
                  sta_plan_create, sta_plan_destroy, sta_plan_kv_tiles, sta_plan_q_tiles,
                  sta_plan_workspace_size, sta_set_wait_limit_ns)
from .window import sliding_window_attention, window_backward, window_forward
from .kv_cache import KVCache

__all__ = ["Plan", "Problem", "StaError", "sliding_tile_attention", "sta_backward", "sta_forward", "sta_forward_host",
           "sta_permute",
           "sta_plan_create", "sta_plan_destroy", "sta_plan_kv_tiles", "sta_plan_q_tiles",
           "sta_plan_workspace_size", "sta_set_wait_limit_ns",
           "sliding_window_attention", "window_forward", "window_backward", "KVCache"]
