"""The README's example runs as it stands, and its serving step does what its comments say."""
import ast
import os
import re

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example(cuda_device):
    import torch
    dev, bf = cuda_device, torch.bfloat16
    B, Hq, H, Nk, d, block = 2, 8, 2, 6000, 128, 64
    text = open(os.path.join(ROOT, "README.md")).read()
    code = re.search(r"```python\n(.*?)```", text, re.S).group(1)
    gen = torch.Generator(device=dev).manual_seed(1)
    r = lambda *shape: torch.randn(*shape, generator=gen, device=dev).to(bf)
    nb = -(-Nk // block)
    f8 = torch.float8_e4m3fn
    env = {"q": r(B, Hq, 200, d), "k": r(B, H, 200, d), "v": r(B, H, 200, d), "do": r(B, Hq, 200, d),
           "k_cache": r(B, H, 300, d), "v_cache": r(B, H, 300, d), "q_new": r(B, Hq, 1, d), "k_new": r(B, H, 1, d),
           "v_new": r(B, H, 1, d), "k8": (r(B, H, Nk, d) * 60).to(f8), "v8": (r(B, H, Nk, d) * 60).to(f8),
           "ks": torch.full((B, H, nb), 2.0 ** -6, device=dev), "vs": torch.full((B, H, nb), 2.0 ** -6, device=dev),
           "lens": torch.tensor([6000, 5555], dtype=torch.int32, device=dev), "acc": torch.zeros(B, H, Nk, device=dev),
           "bounds": torch.zeros(B, H, nb, 2, d, device=dev).to(f8)}
    import exact_io_aware_44_b200 as fa
    fa.block_bounds(env["k8"], block, lens=env["lens"], bounds=env["bounds"])
    weighed = None
    for node in ast.parse(code).body:
        exec(compile(ast.Module([node], []), "README.md", "exec"), env)
        if "cache_weights" in ast.unparse(node):
            weighed = env["acc"].double().sum(-1)
    assert fa.get_status() == 0
    # a row's weights sum to one (each to 2^-16: scores of size up to 2^4 in fp32, exponentials)
    assert np.allclose(weighed.cpu().numpy(), Hq // H, rtol=2.0 ** -12)
    assert env["lens"].tolist() == [4096, 4096]
    fresh = fa.block_bounds(env["k8"], block, lens=env["lens"], bounds=env["bounds"].clone())
    assert torch.equal(fresh.view(torch.uint8), env["bounds"].view(torch.uint8))
