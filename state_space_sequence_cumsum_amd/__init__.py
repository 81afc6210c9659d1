"""MI355X-native (gfx950) Mamba-2 SSD chunked forward pass.

The compute path is libssd.so (hand-written HIP kernels behind the C ABI of
include/ssd.h); :mod:`.binding` marshals torch tensors into it, and :mod:`.block` those of
the operators around the forward (short convolution, selective scan, block norms), :mod:`.linattn`
those of linear attention with a decay for each head and of rotary positions.  Importing this
package does not load the library; the first call does, and raises if it is missing.
"""
from .binding import (FORWARD_EVENTS, SSD_BF16, SSD_F32, ForwardPlan, SsdError, SsdProblem, StepPlan, make_problem,
                      plan_candidates, problem_of, ssd_chunk_cumsum, ssd_chunk_out, ssd_forward,
                      ssd_forward_noalloc, ssd_plan, ssd_state_pass, ssd_step, ssd_status_string,
                      ssd_validate, ssd_workspace_bytes, ssd_workspace_bytes_planned,
                      ssd_workspace_layout, workspace_for, workspace_views)
from .block import (ConvProblem, ConvStepPlan, NormProblem, ScanProblem, ScanStepPlan, scan_problem,
                    ssd_conv, ssd_conv_step, ssd_norm, ssd_scan, ssd_scan_step,
                    ssd_scan_workspace_bytes)
from .linattn import (LinattnProblem, LinattnStepPlan, RotaryProblem, linattn_problem,
                      rotary_frequencies, ssd_linattn, ssd_linattn_backward,
                      ssd_linattn_backward_workspace_bytes, ssd_linattn_step,
                      ssd_linattn_workspace_bytes, ssd_rotary)
from .tune import autotune

__all__ = ["FORWARD_EVENTS", "SSD_BF16", "SSD_F32", "ForwardPlan", "SsdError", "SsdProblem", "StepPlan", "autotune",
           "make_problem", "plan_candidates", "problem_of", "ssd_workspace_bytes_planned",
           "ssd_chunk_cumsum", "ssd_chunk_out", "ssd_forward", "ssd_forward_noalloc", "ssd_plan", "ssd_state_pass", "ssd_step",
           "ssd_status_string", "ssd_validate", "ssd_workspace_bytes", "ssd_workspace_layout",
           "workspace_for", "workspace_views", "ConvProblem", "ConvStepPlan", "NormProblem",
           "ScanProblem", "ScanStepPlan", "scan_problem", "ssd_conv", "ssd_conv_step", "ssd_norm",
           "ssd_scan", "ssd_scan_step", "ssd_scan_workspace_bytes", "LinattnProblem", "LinattnStepPlan",
           "RotaryProblem", "linattn_problem", "rotary_frequencies", "ssd_linattn", "ssd_linattn_backward",
           "ssd_linattn_backward_workspace_bytes", "ssd_linattn_step",
           "ssd_linattn_workspace_bytes", "ssd_rotary"]
