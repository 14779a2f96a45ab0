"""P-EAGLE parallel drafting step on GB300 (sm_103a): Python binding of libpeagle.so."""
from .binding import (Drafter, Expanded, KvPool, PeError, pe_attn_decode,  # noqa: F401
                      pe_draft_forward, pe_expand_batch, pe_get_device_error, pe_kv_append,
                      pe_kv_evict, pe_lmhead_argmax, pe_linear, pe_set_kv_scores,
                      pe_set_trace)
