"""The 8-bit cache's entry points used together."""
import importlib.util
import os

import pytest
import torch

import dsa_sparse_attention_step_gb300 as dsa

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("code", [torch.int8, torch.float8_e4m3fn])
def test_quant_decode_example(code):
    spec = importlib.util.spec_from_file_location(
        "quant_decode", os.path.join(ROOT, "examples", "quant_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for kw in (dict(), dict(prompts=(1, 64, 65, 200), steps=70)):
        worst, lost = example.main(code=code, **kw)
        # against what is held: f16 copies of the keys, 2^-11 of each, move a score by 2^-11
        # sum |q k| / sqrt(128) (some 2^-8), which with P's and the output's rounding (2^-11
        # and 2^-8 of values of at most 5) stays under 2^-4
        assert worst < 2.0**-4
        # a block's largest of 2048 normal values is below 6; INT8: a step of twice 6 / 127 at
        # most, off by half a step at each of some doublings, under one step in all; E4M3: 2^-4
        # of a value of unit root mean square, and codes below the normal ones
        assert lost < (12.0 / 127 if code == torch.int8 else 2.0**-4 + 2.0**-9)


def test_launch_count():
    """Each call counts the kernels it launches."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda:0")  # noqa: E731
    k, v = torch.zeros(2, 40, 2, 64, 64, dtype=torch.int8, device="cuda:0")
    cache = dsa.QuantCache(k, v, torch.ones(40, 2, 2, 4, device="cuda:0"))
    table = torch.arange(40, dtype=torch.int32, device="cuda:0")[None].contiguous()
    batch = dsa.Batch(i32([0, 1]), i32([100]), table, 40, [100], [1])
    x = torch.zeros(1, 4, 64, dtype=torch.float16, device="cuda:0")
    ws = torch.empty(dsa.dsa_quant_attention_workspace_size(batch, cache, 4), dtype=torch.uint8,
                     device="cuda:0")
    for call in (lambda: dsa.dsa_quant_append(cache, None, None, torch.tensor([99], device="cuda:0"),
                                              x, x[:, :2], x[:, 2:], x),
                 lambda: dsa.dsa_quant_read(batch, cache, x[:, :2], None),
                 lambda: dsa.dsa_quant_attention(batch, cache, x, 0.1, torch.empty_like(x), None, ws)):
        n = dsa.dsa_launch_count()
        call()
        assert dsa.dsa_launch_count() - n == 1
    torch.cuda.synchronize()
