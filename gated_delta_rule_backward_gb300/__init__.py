"""gated_delta_rule_backward_gb300: the gated delta rule (Gated DeltaNet / KDA) forward
and backward as hand-written CUDA for sm_103a behind a C ABI (``libgdn``).

Submodules:
  ``gdn``    -- the ctypes binding of ``libgdn`` (loads the CUDA library; raises if absent)
  ``decode`` -- the rule's serving form over a pool of states, and the moves of its states
  ``beam``   -- a beam search's selection over beams and vocabulary
  ``rms``    -- the root-mean-square norm with the residual's addition, forward and backward
  ``build``  -- compiles ``libgdn.so`` in-tree with nvcc for sm_103a
  ``synth``  -- seeded synthetic inputs (no recurrence arithmetic)
"""
