"""libm3ssm: the Mamba-3 SSM core recurrence (prefill scan and decode step)
and the other layers of a hybrid stack (gated recurrence, q/k norms with rotary
positions, causal attention) as hand-written HIP kernels for gfx950 behind a C
ABI."""
