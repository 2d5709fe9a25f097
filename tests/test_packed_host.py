"""The packed-sequence entry points refuse bad arguments on the host with the
documented codes, before touching the device (no GPU here)."""
import ctypes

import numpy as np
import pytest
import torch

from linear_compressed_attention_b200 import binding as bd

NULL, SHAPE, ALIGN, DTYPE, WORKSPACE, UNSUPPORTED = -1, -2, -3, -4, -5, -8
P = ctypes.c_void_p


def attn(**kw):
    a = bd.PackedAttentionArgs()
    base = dict(dtype=1, heads=8, kv_heads=2, d=64, nseq=3, causal=1, max_k=100, scale=0.125, rows_q=50, rows_k=60,
                ldq=512, ldk=128, ldv=128, ldo=512, q_offsets=0x1000, k_offsets=0x2000, k_lens=0x3000,
                workspace=0x10000, workspace_bytes=1 << 40)
    for n, v in {**base, **kw}.items():
        setattr(a, n, v)
    return a


def attn_call(q=0x100000, k=0x200000, v=0x300000, out=0x400000, **kw):
    return bd.lib().edit_packed_attention_forward(P(q), P(k), P(v), ctypes.byref(attn(**kw)), P(out), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(heads=0), SHAPE), (dict(kv_heads=3), SHAPE), (dict(d=0), SHAPE),
    (dict(nseq=0), SHAPE), (dict(max_k=-1), SHAPE), (dict(rows_q=-1), SHAPE), (dict(rows_k=-5), SHAPE),
    (dict(d=60), UNSUPPORTED), (dict(d=136), UNSUPPORTED), (dict(heads=130, kv_heads=2), UNSUPPORTED),
    (dict(rows_q=1 << 31), UNSUPPORTED), (dict(rows_k=1 << 31), UNSUPPORTED),
    (dict(scale=0.0), UNSUPPORTED), (dict(scale=-1.0), UNSUPPORTED), (dict(scale=float("nan")), UNSUPPORTED),
    (dict(scale=float("inf")), UNSUPPORTED),
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(out=0), NULL), (dict(q_offsets=0), NULL),
    (dict(k_offsets=0), NULL), (dict(workspace=0), NULL),
    (dict(ldq=504), SHAPE), (dict(ldk=120), SHAPE), (dict(ldv=64), SHAPE), (dict(ldo=511), SHAPE),
    (dict(ldq=516), UNSUPPORTED), (dict(ldk=132), UNSUPPORTED),
    (dict(q=0x100008), ALIGN), (dict(out=0x400002), ALIGN), (dict(workspace=0x10010), ALIGN),
    (dict(q_offsets=0x1002), ALIGN), (dict(k_lens=0x3001), ALIGN),
    (dict(workspace_bytes=255), WORKSPACE),
])
def test_attention_refuses(kw, code):
    assert attn_call(**kw) == code


def test_attention_null_struct_and_workspace_query():
    L = bd.lib()
    assert L.edit_packed_attention_forward(P(1), P(1), P(1), None, P(1), None) == NULL
    assert L.edit_packed_attention_workspace_bytes(None) == 0
    assert bd.edit_packed_attention_workspace_bytes(attn(d=60)) == 0
    assert bd.edit_packed_attention_workspace_bytes(attn(rows_q=0)) > 0
    # a workspace for many rows serves every smaller call, split key lists included
    for heads, kv, d, nseq, max_k in ((32, 8, 128, 32, 8192), (8, 8, 64, 1, 100000), (3, 1, 72, 2, 5000)):
        kw = dict(heads=heads, kv_heads=kv, d=d, nseq=nseq, max_k=max_k)
        most = bd.edit_packed_attention_workspace_bytes(attn(rows_q=3000, **kw))
        need = [bd.edit_packed_attention_workspace_bytes(attn(rows_q=r, **kw)) for r in range(0, 3000, 7)]
        assert need == sorted(need) and need[-1] <= most
    # the split itself: few rows over a long cache take more than the status block
    assert bd.edit_packed_attention_workspace_bytes(attn(rows_q=1, nseq=1, max_k=100000)) > 4096

# For calls whose arguments are all in order and whose addresses are not: past the checks the launch fails for want of
# a device, with a code of its own; never run where there is one.
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")


@no_device
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("kv,group", [(1, 1), (2, 3), (8, 4), (1, 32), (1, 33), (2, 40), (1, 64)])
def test_attention_workspace_serves_every_smaller_call(dtype, kv, group):
    # group 33 to 64: a tile of the fp32 kernel holds one row, and its query met the plan of no rows first
    for nseq in (1, 3, 40):
        for max_k in (0, 257, 8192):
            kw = dict(dtype=dtype, heads=kv * group, kv_heads=kv, nseq=nseq, max_k=max_k, rows_k=0, ldq=kv * group * 64,
                      ldo=kv * group * 64, ldk=kv * 64, ldv=kv * 64, k=0, v=0)
            query = {n: v for n, v in kw.items() if n not in ("k", "v")}
            for most in (1, 4, 100, 700):
                room = bd.edit_packed_attention_workspace_bytes(attn(rows_q=most, **query))
                for rows in {1, 2, 3, most // 3, most // 2, most - 1, most}:
                    if 1 <= rows <= most:
                        assert attn_call(rows_q=rows, workspace_bytes=room, **kw) != WORKSPACE


def delta(**kw):
    a = bd.DeltaRuleArgs()
    base = dict(dtype=1, qk_heads=2, heads=4, d_k=64, d_v=72, nseq=3, qk_norm=1, scale=0.125, qk_eps=1e-6, rows=50,
                ldq=128, ldk=128, ldv=288, ldo=288, ldg=4, ldb=4, offsets=0x1000, workspace=0x10000,
                workspace_bytes=1 << 40)
    for n, v in {**base, **kw}.items():
        setattr(a, n, v)
    return a


def delta_call(q=0x100000, k=0x200000, v=0x300000, g=0x400000, beta=0x500000, si=0x600000, so=0x600000, out=0x700000,
               **kw):
    return bd.lib().edit_delta_rule_forward(P(q), P(k), P(v), P(g), P(beta), ctypes.byref(delta(**kw)), P(si), P(so),
                                            P(out), None)


def step_call(q=0x100000, k=0x200000, v=0x300000, g=0x400000, beta=0x500000, state=0x600000, out=0x700000, **kw):
    return bd.lib().edit_delta_rule_step(P(q), P(k), P(v), P(g), P(beta), ctypes.byref(delta(**kw)), P(state), P(out),
                                         None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=-1), DTYPE), (dict(heads=3), SHAPE), (dict(qk_heads=0), SHAPE), (dict(d_k=0), SHAPE),
    (dict(nseq=0), SHAPE), (dict(d_k=60), UNSUPPORTED), (dict(d_k=136), UNSUPPORTED), (dict(d_v=264), UNSUPPORTED),
    (dict(d_v=4), UNSUPPORTED),
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(g=0), NULL), (dict(beta=0), NULL), (dict(out=0), NULL),
    (dict(ldq=120), SHAPE), (dict(ldv=280), SHAPE), (dict(ldg=3), SHAPE), (dict(ldb=3), SHAPE),
    (dict(ldk=132), UNSUPPORTED), (dict(q=0x100004), ALIGN), (dict(g=0x400002), ALIGN), (dict(out=0x700008), ALIGN),
])
def test_delta_rule_refuses(kw, code):
    assert delta_call(**kw) == code
    assert step_call(**kw) == code


def test_delta_rule_refuses_more():
    assert delta_call(rows=-1) == SHAPE
    assert delta_call(rows=1 << 31) == UNSUPPORTED
    assert delta_call(offsets=0) == NULL
    assert delta_call(workspace=0) == NULL
    assert delta_call(workspace=0x10080) == ALIGN
    assert delta_call(workspace_bytes=8) == WORKSPACE
    assert delta_call(si=0x600008) == ALIGN
    assert delta_call(so=0x600004) == ALIGN
    assert step_call(state=0) == NULL
    assert step_call(state=0x600004) == ALIGN
    assert bd.edit_delta_rule_workspace_bytes(delta(d_k=60)) == 0
    sizes = [bd.edit_delta_rule_workspace_bytes(delta(rows=r)) for r in (0, 1, 64, 1000, 100000)]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    L = bd.lib()
    assert L.edit_delta_rule_forward(P(1), P(1), P(1), P(1), P(1), None, P(1), P(1), P(1), None) == NULL
    assert L.edit_delta_rule_step(P(1), P(1), P(1), P(1), P(1), None, P(1), P(1), None) == NULL


def norm_call(x=0x100000, y=0x200000, r=0x300000, h=0x400000, **kw):
    a = bd.BlockNormArgs()
    base = dict(dtype=1, norm_post=2, norm_pre=1, gate_act=0, C=128, samples=2, eps=1e-6, res_scale=1.0, rows=10,
                rows_per_sample=5, ldx=128, ldy=128, ldr=128, ldh=128, ld_mod=128, gate=0x500000, scale=0x510000,
                shift=0x520000, post_w=0x530000)
    for n, v in {**base, **kw}.items():
        setattr(a, n, v)
    return bd.lib().edit_block_norm_forward(P(x), P(y), ctypes.byref(a), P(r), P(h), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), DTYPE), (dict(C=0), SHAPE), (dict(samples=0), SHAPE), (dict(rows=-1), SHAPE),
    (dict(C=16385, ldx=16385), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(norm_post=3), UNSUPPORTED), (dict(norm_pre=-1), UNSUPPORTED), (dict(gate_act=2), UNSUPPORTED),
    (dict(norm_post=0), UNSUPPORTED), (dict(norm_pre=0, pre_b=0x10), UNSUPPORTED),
    (dict(x=0), NULL), (dict(r=0, h=0), NULL), (dict(h=0x300000), SHAPE),
    (dict(ldx=127), SHAPE), (dict(ldy=100), SHAPE), (dict(ldr=0), SHAPE), (dict(ldh=1), SHAPE), (dict(ld_mod=64), SHAPE),
    (dict(rows_per_sample=0), SHAPE), (dict(rows_per_sample=4), SHAPE),
    (dict(r=0x100000, ldr=256), SHAPE), (dict(h=0x200000, ldh=256), SHAPE), (dict(h=0x100000, ldh=256), SHAPE),
    (dict(r=0x200000, ldr=256), SHAPE),
    (dict(x=0x100001), ALIGN), (dict(gate=0x500001), ALIGN), (dict(offsets=0x1001), ALIGN),
    (dict(dtype=0, h=0x400002), ALIGN),
])
def test_block_norm_refuses(kw, code):
    assert norm_call(**kw) == code


def test_block_norm_null_struct_and_no_rows():
    assert bd.lib().edit_block_norm_forward(P(1), P(1), None, P(1), P(1), None) == NULL
    assert norm_call(rows=0) == 0     # nothing is enqueued


def test_dit_block_norms_refused():
    L, n = bd.lib(), bd.DitBlockNorms()
    w = bd.DitBlockWeights()
    s = bd.EditAttnWeights()
    s.dtype, s.c_red, s.gn_groups = 1, 288, 32
    for k, name in enumerate(bd.WEIGHT_NAMES):
        setattr(s, name, 0x10000 + 0x1000 * k)       # never dereferenced: validation fails first
    w.attn, w.hidden, w.ln_eps = s, 512, 1e-6
    for k, name in enumerate(bd.DIT_NAMES):
        setattr(w, name, 0x80000 + 0x1000 * k)
    w.workspace, w.workspace_bytes = 0x1000000, 1 << 40

    def call(norms=n, x=0x2000000):
        return L.edit_dit_block_normed_forward(P(x), P(0x3000000), P(0x4000000), 1, 64, 64, 300, 1152, 16,
                                               ctypes.byref(w), None if norms is None else ctypes.byref(norms),
                                               P(0x5000000), None)
    assert call(norms=None) == NULL
    assert call(x=0) == NULL
    n.norm_pre = 3
    assert call() == UNSUPPORTED
    n.norm_pre, n.norm_post = 1, -1
    assert call() == UNSUPPORTED
    n.norm_post, n.post_cross_w = 0, 0x6000000       # a post weight without a post norm
    assert call() == UNSUPPORTED
    n.norm_post, n.post_cross_w = 2, 0x6000008
    assert call() == ALIGN


@pytest.mark.parametrize("rows", [(1 << 31) - 511, (1 << 31) - 1])
def test_row_counts_whose_tiles_pass_32_bits_are_refused(rows):
    # the kernels step in whole tiles: an index past 2^31 - 1 would come back negative
    assert attn_call(rows_q=rows, dtype=0) == UNSUPPORTED
    assert attn_call(rows_k=rows, dtype=1) == UNSUPPORTED
    assert bd.edit_packed_attention_workspace_bytes(attn(rows_q=rows)) == 0
    assert bd.edit_packed_attention_workspace_bytes(attn(rows_q=(1 << 31) - 512)) > 0
    assert delta_call(rows=rows) == UNSUPPORTED
    assert bd.edit_delta_rule_workspace_bytes(delta(rows=rows)) == 0
    assert bd.edit_delta_rule_workspace_bytes(delta(rows=(1 << 31) - 512)) > 0


@pytest.mark.parametrize("scale", [2.0 ** 127, 3e38])
def test_scales_that_are_infinite_in_base_2_are_refused(scale):
    assert attn_call(scale=scale) == UNSUPPORTED


@pytest.mark.parametrize("weights", [dict(post_atn_w=np.ones(1152)), dict(post_ffn_w=np.ones(576)),
                                     dict(pre_attn_w=np.ones((2, 576)))])
def test_dit_block_norm_weights_of_another_name_or_shape_are_refused(weights):
    # a misspelt weight would be left out, a short one read past its end
    with pytest.raises(ValueError, match="norm weight"):
        bd.DitBlock({}, 1, 64, 64, 300, 1152, 16, norms=("layer", "rms", weights))


@pytest.mark.parametrize("rows_k", [-5, 0, 1 << 40])
def test_attention_workspace_query_does_not_read_the_keys(rows_k):
    # a caller sizes the workspace before it knows how many rows its cache will have
    assert bd.edit_packed_attention_workspace_bytes(attn(rows_k=rows_k)) == \
        bd.edit_packed_attention_workspace_bytes(attn()) > 0
