"""GB300 (sm_103a) GatedDeltaNet verify + commit for MTP speculative decoding.

The compute lives in ``libgdnspec.so`` (C ABI, ``include/gdnspec.h``);
``gdn`` is its ctypes binding, ``hybrid`` the binding of the operators a
Qwen3.5-style hybrid's step needs beside those layers (``include/gdnhybrid.h``),
``inputs`` the seeded synthetic workloads and ``build`` compiles the library
in-tree.  The bindings are imported lazily so that ``inputs`` and ``build`` work
before the library exists.
"""

__all__ = ["gdn", "hybrid", "inputs", "build"]


def __getattr__(name):
    if name in ("gdn_verify", "gdn_commit", "gdn_verify_commit", "gdn_verify_commit_static",
                "gdn_verify_deferred", "greedy_accept", "GdnArgs", "GdnPrevRows", "GdnError", "make_args",
                "make_prev", "work_bytes", "carry_bytes", "DeviceLayer", "REPLAY", "SNAPSHOT", "strerror"):
        from . import gdn

        return getattr(gdn, name)
    if name in ("gdn_page_map", "gdn_kv_append", "gdn_paged_attention", "gdn_sample_accept", "make_page_map_args",
                "make_kv_append_args", "make_paged_attention_args", "make_sample_accept_args", "paged_attention_work_bytes"):
        from . import hybrid

        return getattr(hybrid, name)
    raise AttributeError(name)
