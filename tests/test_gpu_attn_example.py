"""The attention layer of examples/attention_step.py at small sizes: LoRA projections, the
append, shared prompts and a captured step together, against 64-bit arithmetic.

Bar: the output projection's bf16 rounding (2^-9 rms relative) beside the attention's, each
weight and value rounded at most twice before it: a relative Frobenius error below 1e-2."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("argv", [
    ["--requests", "5", "--adapters", "2", "--prompt", "70", "--steps", "3", "--d", "256", "--heads", "8", "--kv-heads",
     "2", "--head-dim", "64"],
    ["--requests", "40", "--adapters", "3", "--prompt", "390", "--steps", "9", "--d", "512", "--heads", "4",
     "--kv-heads", "2", "--head-dim", "128"]])
def test_example(argv):
    from lora_serving_device_gb300 import build, lora
    build.build()
    lora.load()
    from examples import attention_step
    assert attention_step.main(argv) < 1e-2
