"""CPU oracle (fp64) for group-wise affine low-bit QMV.

TEST INFRASTRUCTURE ONLY: only tests/, __graft_entry__.smoke() and the
cpu_baseline leg of bench.py may import it.  It shares no code with the HIP
library.
"""
from .qmv_oracle import *  # noqa: F401,F403
from .qmv_oracle import (T5_MAX_BYTE, abs_mass, algorithmic_bytes, bits_of, check_close,
                         codes_of, dequant_f16, dequant_f64, effective_biases, pack_words,
                         qmv_brute, qmv_f64, qmv_reference, sym_ratio, t5_group_bytes,
                         t5_pack, t5_unpack, t5_unpack_scalar, tolerance, unpack_words,
                         unpack_words_scalar, weights_f64)
from .spec_oracle import spec_verify, spec_verify_scalar, target_tokens
from .kv_oracle import (PagesOracle, kv_append_f64, kv_attn_f64, kv_encode, kv_places, kv_sequence, kv_table,
                        rope_f64)
from .tree_oracle import (causal_context, kv_attn_seen_f64, kv_keep_f64, logprobs_f64, norm_f64, tree_above,
                          tree_accept, tree_context, tree_seen, tree_words)
