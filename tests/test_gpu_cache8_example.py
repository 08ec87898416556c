"""examples/attention_step.py with the cache in 8 bits, at small sizes: batch_plan over many pages, LoRA
projections, the append, shared prompts and a captured step together, against 64-bit
arithmetic over keys and values rounded as the cache stores them.

Bar: 1e-2 for what the wide cache's test counts (test_gpu_attn_example.py), and what keys and
values add that become another code here than there.  A projection's value may be the next bf16,
a sixteenth of a code's step away, in at most half of the cases (the sums before the rounding differ by
less than a step); one in 16 of these is then the next code, and the step is (1/8) / m of a
value with m in [1, 2), rms 2^-3.5: together 2^-3.5 / sqrt(32) = 1.6e-2 of the values, and as
much of the scores, whose deviation is below 1 here: 2.2e-2."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("argv", [
    ["--requests", "5", "--adapters", "2", "--prompt", "70", "--steps", "40", "--d", "256", "--heads", "8", "--kv-heads",
     "2", "--head-dim", "64"],
    ["--requests", "40", "--adapters", "3", "--prompt", "390", "--steps", "33", "--d", "512", "--heads", "4",
     "--kv-heads", "2", "--head-dim", "128"]])
def test_example(argv, bits):
    from lora_serving_device_gb300 import build, lora
    build.build()
    lora.load()
    from examples import attention_step
    assert attention_step.main(argv + ["--bits", str(bits)]) < (3e-2 if bits == 8 else 1e-2)
