"""The DiT block with norms on both sides of its branches
(edit_dit_block_normed_forward) against its composition from the fp64 oracle's
parts, within the bars of the plain block: max |gpu - oracle| / max |oracle| of
1e-4 (fp32) and 2e-2 (bf16, fp32 accumulation)."""
import numpy as np
import pytest
import torch

import oracle.edit_oracle as O
from linear_compressed_attention_b200 import binding as bd
from linear_compressed_attention_b200.inputs import make_inputs

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-4, "bf16": 2e-2}
CFG = {
    "bf16": (dict(dtype="bf16", B=2, H=6, W=7, C=128, c_red=64, gn_groups=8, heads=2, seed=91, nonzero_affine=True),
             dict(n_cap=9, hidden=512)),
    "f32": (dict(dtype="f32", B=2, H=5, W=7, C=64, c_red=16, gn_groups=4, heads=2, seed=92, nonzero_affine=True),
            dict(n_cap=6, hidden=128)),
    "bf16_d72": (dict(dtype="bf16", B=1, H=12, W=10, C=1152, c_red=288, gn_groups=32, heads=16, seed=93,
                      nonzero_affine=True), dict(n_cap=50, hidden=4608)),
}


def norm(x, kind, eps, w):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdims=True)
    x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x if w is None else x * np.asarray(w, np.float64)


def block(d, H, W, heads, pre, post, w):
    f = lambda n: np.asarray(d[n], np.float64)  # noqa: E731
    m = f("sst")[None] + f("t6")
    sh_a, sc_a, g_a, sh_f, sc_f, g_f = (m[:, k][:, None, :] for k in range(6))
    eps, x, y = d["ln_eps"], f("x"), f("y")
    h1 = norm(x, pre, eps, w.get("pre_attn_w")) * (1 + sc_a) + sh_a
    a = O.linear(O.edit_forward(h1, H, W, d, heads), f("o_w"), f("o_b"))
    x1 = x + g_a * norm(a, post, eps, w.get("post_attn_w"))
    q, k, v = O.linear(x1, f("cq_w"), f("cq_b")), O.linear(y, f("ck_w"), f("ck_b")), O.linear(y, f("cv_w"), f("cv_b"))
    c = O.linear(O.sdpa(q, k, v, heads), f("co_w"), f("co_b"))
    x2 = x1 + norm(c, post, eps, w.get("post_cross_w"))
    h2 = norm(x2, pre, eps, w.get("pre_ffn_w")) * (1 + sc_f) + sh_f
    mlp = O.linear(O.gelu_tanh(O.linear(h2, f("fc1_w"), f("fc1_b"))), f("fc2_w"), f("fc2_b"))
    return x2 + g_f * norm(mlp, post, eps, w.get("post_ffn_w"))


@pytest.mark.parametrize("name", sorted(CFG))
@pytest.mark.parametrize("pre,post,weights", [("rms", "rms", True), ("layer", "layer", False), ("rms", "none", True),
                                              ("layer", "none", False)])
def test_normed_block_matches_composition(name, pre, post, weights):
    cfg, blk = CFG[name]
    d = make_inputs(**cfg, dit_block=blk)
    B, H, W, C, heads = cfg["B"], cfg["H"], cfg["W"], cfg["C"], cfg["heads"]
    rng = np.random.default_rng(5)
    w = {}
    if weights:
        for n in bd.DIT_NORM_WEIGHTS:
            if (pre if n.startswith("pre") else post) != "none":
                w[n] = torch.from_numpy((1 + 0.2 * rng.standard_normal(C)).astype(np.float32)).to(
                    torch.bfloat16).float().numpy()
    b = bd.DitBlock(d, B, H, W, blk["n_cap"], C, heads, cfg["dtype"], norms=(pre, post, w))
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", b.tdtype)  # noqa: E731
    x, y, t6 = dev(d["x"]), dev(d["y"]), dev(d["t6"])
    outs = [b.forward(x, y, t6).clone() for _ in range(2)]
    assert b.status() == 0
    assert torch.equal(*outs)
    ref = block(d, H, W, heads, pre, post, w)
    err = float(np.max(np.abs(outs[0].double().cpu().numpy() - ref)) / np.max(np.abs(ref)))
    assert err <= TOL[cfg["dtype"]], err
    if (pre, post) == ("layer", "none"):   # the plain block
        plain = bd.DitBlock(d, B, H, W, blk["n_cap"], C, heads, cfg["dtype"]).forward(x, y, t6)
        err = float(np.max(np.abs((outs[0].double() - plain.double()).cpu().numpy())) / np.max(np.abs(ref)))
        assert err <= TOL[cfg["dtype"]], err
