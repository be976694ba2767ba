"""MI355X (gfx950) selective state-space scan: HIP kernels behind a C ABI.

    from selective_state_space_76_amd import conv1d_fwd, scan_fwd, state_update, conv1d_update
    u, conv_state = conv1d_fwd(x, conv_weight, conv_bias)          # the step that produces u
    out, h_last = scan_fwd(u, delta, A, B, C, D, z, delta_bias)    # prefill
    grads = scan_bwd(u, delta, A, B, C, D, z, delta_bias, dout=g)  # training backward
    out, h_last = selective_scan(u, delta, A, B, C, D, z, delta_bias)  # the same, under autograd
    u_t = conv1d_update(conv_state, x_t, conv_weight, conv_bias)   # decode
    y = state_update(h_last, u_t, delta_t, A, B_t, C_t, D, z_t, delta_bias)

and, for a training step around it:

    x = embedding(tokens, table, scale=s, channels_first=True)     # tokens to [B,E,L], under autograd
    u, conv_state = causal_conv1d(x, conv_weight, conv_bias)       # conv1d_fwd under autograd
    opt = AdamW(params, lr=1e-4, weight_decay=0.1, state_bits=8, max_grad_norm=1.0)
    opt.step()

and, for the rest of a residual block, with another recurrence to mix over time:

    y, hidden = layer_norm(branch, weight, bias, hidden, rms=True, p=0.1, seed=s)  # hidden + dropout(branch), normalised
    out, last = gated_recurrence(x, r, i, decay, r_bias, i_bias, z)                # one state per channel, gates per step
    out = dropout(branch, 0.1, s, call=1, residual=hidden)
    h_t = recurrence_update(last, x_t, r_t, i_t, decay, r_bias, i_bias, z_t)       # decode

The C ABI is include/ssm_scan.h; the library is libssmscan.so in this package,
built by `python -m selective_state_space_76_amd.build`.
"""
from ._lib import (SSMError, load, scan_fwd, scan_fwd_noalloc, state_update, conv1d_fwd, conv1d_update,  # noqa: F401
                   scan_bwd, bwd_workspace_size, workspace_size, checkpoints_shape, SSM_F32, SSM_BF16,
                   SSM_FLAG_ZOH, SSM_FLAG_REVERSE, LIB_PATH)
from .autograd import (SelectiveScanFn, causal_conv1d, dropout, embedding, gated_recurrence, layer_norm,  # noqa: F401
                       selective_scan)
from .block import (dropout_bwd, dropout_fwd, layer_norm_bwd, layer_norm_bwd_workspace_size, layer_norm_fwd,  # noqa: F401
                    recurrence_bwd, recurrence_bwd_workspace_size, recurrence_checkpoints_shape, recurrence_fwd,
                    recurrence_update, recurrence_workspace_size)
from .training import (AdamW, conv1d_bwd, conv1d_bwd_workspace_size, embedding_bwd,  # noqa: F401
                       embedding_bwd_workspace_size, embedding_fwd)

__all__ = ["scan_fwd", "scan_fwd_noalloc", "scan_bwd", "selective_scan", "SelectiveScanFn", "state_update", "conv1d_fwd",
           "conv1d_update", "workspace_size", "bwd_workspace_size", "checkpoints_shape", "load", "SSMError",
           "LIB_PATH", "embedding", "causal_conv1d", "conv1d_bwd", "conv1d_bwd_workspace_size", "embedding_fwd",
           "embedding_bwd", "embedding_bwd_workspace_size", "AdamW", "layer_norm",
           "layer_norm_fwd", "layer_norm_bwd", "layer_norm_bwd_workspace_size", "dropout", "dropout_fwd", "dropout_bwd",
           "gated_recurrence", "recurrence_fwd", "recurrence_bwd", "recurrence_update", "recurrence_checkpoints_shape",
           "recurrence_workspace_size", "recurrence_bwd_workspace_size"]
