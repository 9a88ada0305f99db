"""MI355X (gfx950) selective scan (Mamba S6): C-ABI library + thin Python binding.

``fwd`` / ``bidir`` call ``libsscan.so`` (``selective_scan`` /
``selective_scan_bidir``: the same with gradients through the backward entry points) (build it with
``python -m selective_state_space_sscan_amd.build``); ``inputs`` draws the seeded
synthetic workloads.  ``gated_delta`` (and ``delta_fwd`` / ``delta_step`` / ``delta_bwd``)
is the gated delta rule, ``gated_rms_norm`` and ``add_rms_norm`` the norms around a mixer.
"""
from .sscan import (SSCAN_BF16, SSCAN_F32, SScanError, add_norm, add_norm_bwd, add_rms_norm,  # noqa: F401
                    bidir, delta_bwd, delta_fwd, delta_step, delta_workspace_bytes, fwd, gated_delta,
                    gated_norm, gated_norm_bwd, gated_rms_norm, load_library, run_inputs, selective_scan,
                    selective_scan_bidir, strerror, workspace_bytes)

__all__ = ["fwd", "bidir", "run_inputs", "workspace_bytes", "load_library", "strerror", "SScanError",
           "SSCAN_F32", "SSCAN_BF16", "selective_scan", "selective_scan_bidir", "gated_delta", "delta_fwd", "delta_step",
           "delta_bwd", "delta_workspace_bytes", "gated_norm", "gated_norm_bwd", "gated_rms_norm", "add_norm",
           "add_norm_bwd", "add_rms_norm"]
