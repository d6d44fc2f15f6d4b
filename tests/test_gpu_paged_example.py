"""The paged entry points used together, and beside the sparse step."""
import importlib.util
import os

import pytest
import torch

import dsa_sparse_attention_step_gb300 as dsa

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_dense_decode_example():
    spec = importlib.util.spec_from_file_location(
        "dense_decode", os.path.join(ROOT, "examples", "dense_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # turned q and k each rounded to bf16 move a score by up to 2 * 2^-8 * sum |q k| / sqrt(128)
    # (typically 8 such terms' spread, below 0.03), which with P's and the output's rounding
    # stays under 2^-4 for values of a few units
    assert example.main() < 2.0**-4
    assert example.main(prompts=(1, 64, 65, 200), steps=70) < 2.0**-4


def test_built_tables_drive_the_sparse_step():
    """A batch built on the GPU gives dsa_append_cache and dsa_decode the same
    results as the same tables from the host."""
    import dsa_inputs as di
    from gpu_helpers import GpuLayer
    layer = di.make_layer([3000, 700], n_q=[2, 1], seed=5, extra_pages=2)
    gl = GpuLayer(layer)
    want = gl.decode()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda:0")  # noqa: E731
    lens, new = layer.seq_lens_host, layer.q_counts_host
    host = layer.block_table
    pages = [-(-n // 64) for n in lens]
    free = torch.cat([host[b, :p].reshape(-1) for b, p in enumerate(pages)]).to(torch.int32).cuda()
    table = torch.zeros(len(lens), host.shape[1], dtype=torch.int32, device="cuda:0")
    q, s, taken, st = i32([0] * (len(lens) + 1)), i32([0] * len(lens)), i32([0]), i32([0])
    # everything enters at once, then the batch of the step: the last tokens of each
    dsa.dsa_build_tables(i32([0] * len(lens)), i32(lens), free, layer.num_pages, table, q, s,
                         pages_taken=taken, dev_status=st)
    assert int(taken.item()) == sum(pages) and int(st.item()) == 0
    dsa.dsa_build_tables(i32([a - b for a, b in zip(lens, new)]), i32(new), free[:0].contiguous(),
                         layer.num_pages, table, q, s, pages_taken=taken, dev_status=st)
    torch.cuda.synchronize()
    assert int(taken.item()) == 0 and int(st.item()) == 0
    gl.batch = dsa.Batch(q, s, table, layer.num_pages, lens, new)
    got = gl.decode()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_launch_count():
    """Each call counts the kernels it launches."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda:0")  # noqa: E731
    cache = dsa.KvCache(torch.zeros(40, 2, 64, 64, dtype=torch.float16, device="cuda:0"),
                        torch.zeros(40, 2, 64, 64, dtype=torch.float16, device="cuda:0"))
    table = torch.arange(40, dtype=torch.int32, device="cuda:0")[None].contiguous()

    def attention(length, hq):
        batch = dsa.Batch(i32([0, 1]), i32([length]), table, 40, [length], [1])
        q = torch.zeros(1, hq, 64, dtype=torch.float16, device="cuda:0")
        ws = torch.empty(dsa.dsa_paged_attention_workspace_size(batch, cache, hq),
                         dtype=torch.uint8, device="cuda:0")
        n = dsa.dsa_launch_count()
        dsa.dsa_paged_attention(batch, cache, q, 0.1, torch.empty_like(q), None, ws)
        return dsa.dsa_launch_count() - n
    assert attention(100, 4) == 1      # a cluster to each KV head
    n = dsa.dsa_launch_count()
    dsa.dsa_build_tables(i32([0]), i32([5]), i32([1]), 4, i32([[0]]), i32([0, 0]), i32([0]),
                         pages_taken=i32([0]))
    assert dsa.dsa_launch_count() - n == 1
    torch.cuda.synchronize()
