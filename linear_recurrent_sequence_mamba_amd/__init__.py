"""libm3ssm: the Mamba-3 SSM core recurrence (prefill scan and decode step)
and the other layers of a hybrid stack (gated recurrence, gated delta rule, q/k
norms with rotary positions, causal attention, norms around a block) as
hand-written HIP kernels for gfx950 behind a C ABI."""
