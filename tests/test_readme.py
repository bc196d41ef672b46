"""The example of the README's section on e4m3 experts: it defines what it uses, and runs."""
import ast
import builtins
import os
import re

import pytest
import torch

import routed_expert_ffn_route_gb300 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# what a user of that section has: the packed layer's config, blob and buffers (from the section
# before it), the experts' weights, the norm's weight, the residual stream, the attention's output
GIVEN = ["torch", "moe", "cfg", "packed", "ids", "w", "ws", "gate_up", "down", "norm_weight",
         "resid", "attention_out"]


def example():
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read()
    section = text[text.index("### Experts kept as e4m3 rows"):]
    return re.search(r"```python\n(.*?)```", section, re.S).group(1)


def test_the_example_defines_what_it_uses():
    known = set(GIVEN) | set(dir(builtins))
    for statement in ast.parse(example()).body:
        names = [n for n in ast.walk(statement) if isinstance(n, ast.Name)]
        used = {n.id for n in names if isinstance(n.ctx, ast.Load)}
        assert used <= known, f"undefined: {sorted(used - known)}"
        known |= {n.id for n in names if isinstance(n.ctx, ast.Store)}
        if isinstance(statement, (ast.Import, ast.ImportFrom)):
            known |= {a.asname or a.name for a in statement.names}


@pytest.mark.gpu
def test_the_example_runs():
    import gen
    from gen.device import build_packed_layer
    s = gen.LayerSpec("readme", hidden=512, inter=256, n_experts=16, top_k=8,
                      router="sigmoid_grouped", n_group=4, topk_group=2, rsf=2.5, bias_std=0.1)
    cfg, packed = build_packed_layer(s, 0, 0, "cuda", host_codes=True)
    T, d = 33, dict(device="cuda")
    torch.manual_seed(0)
    names = dict(torch=torch, moe=moe, cfg=cfg, packed=packed,
                 ids=torch.empty(T, 8, dtype=torch.int32, **d), w=torch.empty(T, 8, **d),
                 ws=torch.zeros(moe.moe_workspace_bytes(cfg, T), dtype=torch.uint8, **d),
                 gate_up=torch.randn(16, 512, 512, **d) / 23, down=torch.randn(16, 512, 256, **d) / 16,
                 norm_weight=(1 + 0.1 * torch.randn(512, **d)).bfloat16(),
                 resid=torch.randn(T, 512, **d).bfloat16(),
                 attention_out=torch.randn(T, 512, **d).bfloat16())
    before = names["resid"].clone()
    exec(example(), names)
    assert moe.moe_read_status(names["ws"]) == moe.MOE_OK
    assert bool((names["ids"] >= 0).all()) and bool((names["ids"] < 16).all())
    # the router saw the norm that the layer takes of the same residual: its codes, within an e4m3
    # rounding (2^-4, or 2^-10 of the scale near zero) and that of x to bf16
    codes = names["layer"].q[:T].float() * names["layer"].qs[:T]
    x = names["x"].float()
    assert bool(((codes - x).abs() <= x.abs() * (2 ** -4 + 2 ** -7)
                 + names["layer"].qs[:T] * 2 ** -9).all())
    out = names["resid"]
    assert out.shape == before.shape and bool(torch.isfinite(out.float()).all())
    assert not torch.equal(out, before)
