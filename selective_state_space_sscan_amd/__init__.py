"""MI355X (gfx950) selective scan (Mamba S6): C-ABI library + thin Python binding.

``fwd`` / ``bidir`` call ``libsscan.so`` (``selective_scan`` /
``selective_scan_bidir``: the same with gradients through the backward entry points) (build it with
``python -m selective_state_space_sscan_amd.build``); ``inputs`` draws the seeded
synthetic workloads.  ``gated_delta`` (and ``delta_fwd`` / ``delta_step`` / ``delta_bwd``)
is the gated delta rule, ``gated_rms_norm`` and ``add_rms_norm`` the norms around a mixer.
``gated_recurrence`` (``rec_fwd`` / ``rec_step`` / ``rec_bwd``) is the gated recurrence with
one state per channel, ``pack8`` / ``unpack8`` hold activations in 8 bits, and
``add_layer_norm`` (``layer_norm`` / ``layer_norm_bwd``) is the layer norm of a residual sum.
"""
from .sscan import (SSCAN_BF16, SSCAN_F32, Kept8, Packed8, SScanError, add_layer_norm, add_norm,  # noqa: F401
                    add_norm_bwd, add_rms_norm, bidir, delta_bwd, delta_fwd, delta_step, delta_workspace_bytes, fwd,
                    gated_delta, gated_norm, gated_norm_bwd, gated_recurrence, gated_rms_norm, layer_norm,
                    layer_norm_bwd, load_library, pack8, rec_bwd, rec_fwd, rec_step, rec_workspace_bytes, run_inputs,
                    selective_scan, selective_scan_bidir, strerror, unpack8, workspace_bytes)

__all__ = ["fwd", "bidir", "run_inputs", "workspace_bytes", "load_library", "strerror", "SScanError",
           "SSCAN_F32", "SSCAN_BF16", "selective_scan", "selective_scan_bidir", "gated_delta", "delta_fwd", "delta_step",
           "delta_bwd", "delta_workspace_bytes", "gated_norm", "gated_norm_bwd", "gated_rms_norm", "add_norm",
           "add_norm_bwd", "add_rms_norm", "gated_recurrence", "rec_fwd", "rec_step", "rec_bwd", "rec_workspace_bytes",
           "pack8", "unpack8", "Packed8", "Kept8", "layer_norm", "layer_norm_bwd", "add_layer_norm"]
