"""rans_entropy_coding_b200 -- indexed 64-bit rANS entropy coding on NVIDIA
B200 (sm_100a): the C-ABI library librans_b200 and its thin Python binding.

See include/rans_b200.h for the boundary.  Build the library with
``python -m rans_entropy_coding_b200.build``.
"""
from ._lib import (  # noqa: F401
    CHUNK_CONTIG, CHUNK_EXPLICIT, CHUNK_TILED, ERR_ARG, ERR_CAPACITY, ERR_CORRUPT, ERR_CUDA,
    FMT_ALIAS, FMT_RANS32_16, FMT_RANS64,
    ERR_INDEX, ERR_RANGE, ERR_TABLE, ERR_TIMEOUT, ERR_ZERO_FREQ, LIB_PATH, OK, SIGNATURES,
    SYM_INT16, SYM_INT32, SYM_UINT8, Chunking, RansError, Tables, Workspaces, aligned_empty,
    check, decode_to_values, decode_with_indexes, encode_from_scales, encode_with_indexes, lib,
    rans_alias_bytes, rans_alias_prepare, rans_build_cdfs_from_pmfs, rans_build_indexes, rans_decode_to_values,
    rans_encode_from_scales,
    rans_build_cdfs_from_scales, rans_chunking, rans_debug_divide, rans_debug_wait_timeout, rans_decode_with_indexes,
    rans_decode_workspace_bytes, rans_encode_with_indexes, rans_encode_with_indexes_noalloc,
    rans_encode_workspace_bytes,
    rans_gaussian_lengths, rans_get_status, rans_max_compressed_bytes, rans_num_streams,
    rans_tables, rans_tables_bytes, rans_tables_prepare, rans_tables_refresh,
    rans_tables_refresh_from_scales)
from ._lib import rans_adjust, rans_beams, rans_logits, rans_mxfp4, rans_state  # noqa: F401,E402
from .tokens import (  # noqa: F401,E402
    MAX_TOP, MAX_VOCAB, TOKEN_PRECISION, LogitAdjust, adjust_logits, decode_tokens,
    distill_loss, distill_loss_and_grad, encode_intervals, new_status, pack_mask,
    rans_adjust_logits, rans_decode_tokens, rans_distill, rans_distill_backward,
    rans_distill_forward, rans_encode_intervals, rans_token_intervals, rans_token_states,
    rans_token_states_finish, token_intervals, token_states)
from .mxfp4 import (  # noqa: F401,E402
    Mxfp4, mxfp4_logits, quantize_mxfp4, rans_mxfp4_codes_bytes, rans_mxfp4_logits,
    rans_mxfp4_logits_workspace_bytes, rans_mxfp4_product, rans_mxfp4_quantize,
    rans_mxfp4_scales_bytes, rans_mxfp4_values)
from .beams import (  # noqa: F401,E402
    MAX_BEAMS, MAX_CONTINUATIONS, MAX_STATES, BeamSearch, beam_select, rans_beam_advance,
    rans_beam_select, rans_beam_workspace_bytes, rans_reorder_states,
    rans_reorder_states_check, reorder_states)
from .interface import (  # noqa: F401,E402
    RansCoder, TokenCoder, from_byte_strings, to_byte_strings)
