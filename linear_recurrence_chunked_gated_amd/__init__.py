"""MI355X (gfx950) HIP implementation of one pipeline chunk of the gated
delta-rule recurrence (Gated DeltaNet), forward and backward, behind the C ABI
in include/sf_gdn.h.

    chunk_fwd(q, k, v, alpha, beta, S_in)            -> (o, S_out)
    chunk_bwd(q, k, v, alpha, beta, S_in, dO, dS_out)
                                 -> (dq, dk, dv, dalpha, dbeta, dS_in)
    chain_fwd / chain_bwd: consecutive chunks through their boundary states.
    gated_delta_chunk(q, k, v, alpha, beta, S_in)    -> (o, S_out), torch autograd
    short_conv(x, w, conv_in)                        -> (y, conv_out), torch autograd
    shortconv_fwd(x, w, conv_in)                     -> (y, conv_out)
    shortconv_bwd(x, w, conv_in, dy, dconv_out)      -> (dx, dw, dconv_in)
    recurrent_step(q, k, v, alpha, beta, state, slots, seq_start)  -> o, decoding
    shortconv_step(x, w, state, slots, seq_start)                  -> y, decoding
    gated_norm_fwd(x, gate, w) / gated_norm_bwd(x, gate, w, dy)
    residual_norm_fwd(x, r, w, s) / residual_norm_bwd(h, r, w, s, dy, dh)
    gated_norm(x, gate, w), residual_norm(x, r, w, s): the norms, torch autograd
    decay_chunk_fwd(q, k, v, decay, S_in, seq_start)               -> (o, S_out)
    decay_chunk_bwd(q, k, v, decay, S_in, dO, dS_out, seq_start)   -> (dq, dk, dv, dS_in)
    decay_chunk(q, k, v, decay, S_in, seq_start)                   -> (o, S_out), torch autograd
    decay_step(q, k, v, decay, state, slots, seq_start)            -> o, decoding
    qk_norm_rotary_fwd(q, k, pos, freq, wq, wk)                    -> (yq, yk)
    qk_norm_rotary_bwd(q, k, pos, freq, wq, wk, dyq, dyk)          -> (dq, dk, dwq, dwk)
    qk_norm_rotary(q, k, pos, freq, wq, wk)                        -> (yq, yk), torch autograd

Imports are lazy so that the input generator and the planner load without the
HIP library.
"""
__all__ = ["chunk_fwd", "chunk_bwd", "chain_fwd", "chain_bwd", "gated_delta_chunk", "short_conv",
           "shortconv_fwd", "shortconv_bwd", "recurrent_step", "shortconv_step", "gated_norm",
           "gated_norm_fwd", "gated_norm_bwd", "residual_norm", "residual_norm_fwd",
           "residual_norm_bwd", "decay_chunk", "decay_chunk_fwd", "decay_chunk_bwd", "decay_step",
           "qk_norm_rotary", "qk_norm_rotary_fwd", "qk_norm_rotary_bwd", "profile", "GDNError"]


def __getattr__(name):
    if name in ("chain_fwd", "chain_bwd"):
        from . import chain as module
    elif name in ("gated_delta_chunk", "short_conv", "gated_norm", "residual_norm", "decay_chunk",
                  "qk_norm_rotary"):
        from . import autograd as module
    elif name in __all__:
        from . import _lib as module
    else:
        raise AttributeError(name)
    globals()[name] = value = getattr(module, name)  # the next look-up finds it in the module
    return value
