"""The gated delta rule through the C ABI against the token-by-token 64-bit
form, within the bounds of packed_ref.delta_rule."""
import os
import subprocess
import sys

import pytest
import torch

import packed_ref as R
from linear_compressed_attention_b200 import binding as bd
from packed_ref import float32_default  # noqa: F401

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def inputs(seed, dtype, rows, hq, h, dk, dv, rate=0.3, shared=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=g, device="cuda")
    q, k, v = n(rows, hq, dk), n(rows, hq, dk) + shared, n(rows, h, dv)
    return (q.to(DT[dtype]), k.to(DT[dtype]), v.to(DT[dtype]), -rate * n(rows, h).exp(), torch.sigmoid(2 * n(rows, h)))


def check(out, state, ref, at):
    o, s, ob, sb = ref
    n = at[-1]
    e = (out[:n].double() - o[:n]).norm(dim=-1)
    assert torch.isfinite(out[:n]).all()
    assert (e <= ob[:n]).all(), float((e / ob[:n]).max())
    if state is not None:
        e = (state.double() - s).flatten(2).norm(dim=-1)
        assert (e <= sb).all(), float((e / sb).max())


SHAPES = [(2, 4, 64, 64), (1, 2, 128, 128), (3, 3, 72, 72), (2, 2, 32, 96), (1, 3, 8, 256), (2, 2, 128, 40), (1, 1, 96, 64)]
LENS = {"ragged": [1, 64, 0, 65, 130, 63], "long": [515], "two": [127, 129], "ones": [1] * 9}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("hq,h,dk,dv", SHAPES)
def test_matches_token_by_token(dtype, lens, hq, h, dk, dv):
    at = offsets(LENS[lens])
    rows = at[-1] + 3
    q, k, v, g, beta = inputs(dk + dv, dtype, rows, hq, h, dk, dv)
    S = len(at) - 1
    state = torch.randn(S, h, dk, dv, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    op = bd.DeltaRule(hq, h, dk, dv, S, rows, dtype, scale=dk ** -0.5)
    ref = R.delta_rule(q, k, v, g, beta, at, state, dk ** -0.5, True)
    outs = []
    for _ in range(2):
        out, so = torch.full_like(v, 7.0), torch.full_like(state, 7.0)
        op.forward(q, k, v, g, beta, ints(at), state_in=state, state_out=so, out=out)
        assert op.status() == 0
        check(out, so, ref, at)
        assert (out[at[-1]:] == 7.0).all()
        outs.append((out, so))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    # from zeros, dropping the state; and in place
    out0 = op.forward(q, k, v, g, beta, ints(at), out=torch.full_like(v, 7.0))
    check(out0, None, R.delta_rule(q, k, v, g, beta, at, None, dk ** -0.5, True), at)
    same = state.clone()
    out1 = op.forward(q, k, v, g, beta, ints(at), state_in=same, state_out=same, out=torch.full_like(v, 7.0))
    assert torch.equal(out1, outs[0][0]) and torch.equal(same, outs[0][1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,h,dk,dv", SHAPES)
def test_step_is_one_token(dtype, hq, h, dk, dv):
    S = 5
    q, k, v, g, beta = inputs(7, dtype, S, hq, h, dk, dv)
    state = torch.randn(S, h, dk, dv, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    op = bd.DeltaRule(hq, h, dk, dv, S, 0, dtype, scale=0.7)
    ref = R.delta_rule(q, k, v, g, beta, list(range(S + 1)), state, 0.7, True)
    mine = state.clone()
    out = op.step(q, k, v, g, beta, mine)
    check(out, mine, ref, [0, S])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,h,dk,dv", [(16, 16, 128, 128), (8, 16, 72, 64), (16, 32, 8, 128), (16, 16, 40, 72)])
def test_step_of_many_sequences(dtype, hq, h, dk, dv):
    # enough states for the kernel that takes whole states (d_v 64 and 128); strided inputs
    S = 24
    q, k, v, g, beta = inputs(17, dtype, S, hq, h, dk, dv)
    g[3] = -float("inf")
    state = torch.randn(S, h, dk, dv, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    op = bd.DeltaRule(hq, h, dk, dv, S, 0, dtype, scale=0.7)
    ref = R.delta_rule(q, k, v, g, beta, list(range(S + 1)), state, 0.7, True)
    qk = torch.cat([q, k], 1)
    wide = torch.full((S, h + 1, dv), 3.0, device="cuda", dtype=v.dtype)
    for _ in range(2):
        mine = state.clone()
        op.step(qk[:, :hq], qk[:, hq:], v, g, beta, mine, out=wide[:, :h])
        assert (wide[:, h] == 3.0).all()
        check(wide[:, :h], mine, ref, [0, S])
    assert torch.equal(mine, (lambda m: (op.step(q, k, v, g, beta, m), m)[1])(state.clone()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_single_tokens_is_the_whole_sequence(dtype):
    hq, h, dk, dv = 2, 4, 64, 64
    lens = [100, 3]
    q, k, v, g, beta = inputs(8, dtype, 2 * 120, hq, h, dk, dv)
    at = [0, 120, 240]
    ref = R.delta_rule(q, k, v, g, beta, at, None, 0.125, True)
    op = bd.DeltaRule(hq, h, dk, dv, 2, 240, dtype)
    rows = [torch.arange(at[s], at[s] + lens[s], device="cuda") for s in range(2)]
    first = torch.cat(rows)
    state = torch.zeros(2, h, dk, dv, device="cuda")
    out = torch.zeros_like(v)
    out[first] = op.forward(q[first], k[first], v[first], g[first], beta[first], ints(offsets(lens)), state_out=state)
    for t in range(17):
        r = torch.tensor([at[s] + lens[s] + t for s in range(2)], device="cuda")
        out[r] = op.step(q[r], k[r], v[r], g[r], beta[r], state)
    for s in range(2):
        r = slice(at[s], at[s] + lens[s] + 17)
        assert ((out[r].double() - ref[0][r]).norm(dim=-1) <= ref[2][r] * 1.01).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[200], [65, 1]])
def test_without_the_norm_and_with_keys_alike(dtype, lens):
    # keys that nearly repeat: the triangular system of a chunk is far from the identity
    at = offsets(lens)
    q, k, v, g, beta = inputs(9, dtype, at[-1], 1, 2, 64, 64, rate=0.01, shared=3.0)
    op = bd.DeltaRule(1, 2, 64, 64, len(lens), at[-1], dtype)
    so = torch.zeros(len(lens), 2, 64, 64, device="cuda")
    out = op.forward(q, k, v, g, beta, ints(at), state_out=so)
    check(out, so, R.delta_rule(q, k, v, g, beta, at, None, 0.125, True), at)
    # unit keys given as they are
    kn = (k.float() / k.float().norm(dim=-1, keepdim=True) * 0.98).to(DT[dtype])
    qn = (q.float() / q.float().norm(dim=-1, keepdim=True)).to(DT[dtype])
    op = bd.DeltaRule(1, 2, 64, 64, len(lens), at[-1], dtype, qk_norm=False)
    out = op.forward(qn, kn, v, g, beta, ints(at), state_out=so)
    check(out, so, R.delta_rule(qn, kn, v, g, beta, at, None, 0.125, False), at)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forgetting_all_and_nothing(dtype):
    at = [0, 150]
    q, k, v, g, beta = inputs(10, dtype, 150, 1, 2, 64, 64)
    g = g.clone()
    g[40] = -float("inf")
    g[41, 0] = -1e30
    g[100:110] = 0.0
    beta = beta.clone()
    beta[20:30] = 0.0
    beta[120] = 1.0
    op = bd.DeltaRule(1, 2, 64, 64, 1, 150, dtype)
    so = torch.zeros(1, 2, 64, 64, device="cuda")
    out = op.forward(q, k, v, g, beta, ints(at), state_out=so)
    check(out, so, R.delta_rule(q, k, v, g, beta, at, None, 0.125, True), at)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_keys_and_queries(dtype):
    at = [0, 70]
    q, k, v, g, beta = inputs(11, dtype, 70, 1, 1, 64, 64)
    q[5] = 0
    k[7:9] = 0
    op = bd.DeltaRule(1, 1, 64, 64, 1, 70, dtype)
    out = op.forward(q, k, v, g, beta, ints(at))
    assert (out[5] == 0).all()
    check(out, None, R.delta_rule(q, k, v, g, beta, at, None, 0.125, True), at)


def test_strided_inputs():
    hq, h, d, n = 2, 4, 64, 140
    q0, k0, v0, g0, b0 = inputs(12, "bf16", n, hq, h, d, d)
    qkv = torch.cat([q0, k0, v0], 1)
    gb = torch.cat([g0, b0], 1)
    q, k, v = qkv[:, :hq], qkv[:, hq:2 * hq], qkv[:, 2 * hq:]
    op = bd.DeltaRule(hq, h, d, d, 1, n, "bf16")
    wide = torch.full((n, h + 2, d), 3.0, device="cuda", dtype=torch.bfloat16)
    op.forward(q, k, v, gb[:, :h], gb[:, h:], ints([0, n]), out=wide[:, :h])
    assert torch.equal(wide[:, :h], op.forward(q0, k0, v0, g0, b0, ints([0, n])))
    assert (wide[:, h:] == 3.0).all()


@pytest.mark.parametrize("at", [[0, 20, 10], [-3, 10, 20], [0, 10, 50], [2 ** 31 - 1, -2 ** 31, 7]])
def test_bad_offsets_are_recorded_and_stay_inside(at):
    for dtype in ("bf16", "f32"):
        q, k, v, g, beta = inputs(13, dtype, 20, 1, 2, 64, 64)
        guard = torch.full((24, 2, 64), 5.0, device="cuda", dtype=DT[dtype])
        op = bd.DeltaRule(1, 2, 64, 64, 2, 20, dtype)
        op.forward(q, k, v, g, beta, ints(at), out=guard[2:22])
        assert op.status() == -2
        assert (guard[:2] == 5.0).all() and (guard[22:] == 5.0).all()
        op.forward(q, k, v, g, beta, ints([0, 10, 20]), out=guard[2:22])
        assert op.status() == 0


def test_no_rows_copies_the_states():
    op = bd.DeltaRule(2, 4, 64, 64, 3, 0, "bf16")
    e = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    ev = torch.empty(0, 4, 64, device="cuda", dtype=torch.bfloat16)
    z = torch.empty(0, 4, device="cuda")
    s = torch.randn(3, 4, 64, 64, device="cuda")
    so = torch.zeros_like(s)
    op.forward(e, e, ev, z, z, ints([0, 0, 0, 0]), state_in=s, state_out=so)
    assert torch.equal(s, so)


def test_captured_call_replays_with_other_lengths():
    hq, h, d, n = 2, 4, 64, 300
    q, k, v, g, beta = inputs(14, "bf16", n, hq, h, d, d)
    at = ints([0, 100, n])
    out, so = torch.zeros_like(v), torch.zeros(2, h, d, d, device="cuda")
    op = bd.DeltaRule(hq, h, d, d, 2, n, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        op.forward(q, k, v, g, beta, at, state_out=so, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            op.forward(q, k, v, g, beta, at, state_out=so, out=out)
    torch.cuda.synchronize()
    other = bd.DeltaRule(hq, h, d, d, 2, n, "bf16")
    for now in ([0, 100, n], [0, 0, 77], [0, 299, n]):
        at.copy_(ints(now))
        out.fill_(2.0)
        graph.replay()
        torch.cuda.synchronize()
        s2 = torch.zeros_like(so)
        eager = other.forward(q, k, v, g, beta, at, state_out=s2, out=torch.full_like(v, 2.0))
        assert torch.equal(out, eager) and torch.equal(so, s2)
        check(out, so, R.delta_rule(q, k, v, g, beta, now, None, 0.125, True), now)


@pytest.mark.parametrize("S,h,lens", [(1, 2, [3000]), (2, 20, [1500, 1100]), (1, 40, [2100])])
def test_parts_of_long_sequences_and_states_in_place(S, h, lens):
    # few (sequence, head) pairs: a sequence's chunks are cut into parts that run side by side, more blocks than SMs in
    # some; the final states may go where the first ones are read
    at = offsets(lens)
    q, k, v, g, beta = inputs(21, "bf16", at[-1], h // 2, h, 128, 128, rate=0.02)
    state = torch.randn(S, h, 128, 128, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    op = bd.DeltaRule(h // 2, h, 128, 128, S, at[-1], "bf16")
    apart = torch.zeros_like(state)
    out = op.forward(q, k, v, g, beta, ints(at), state_in=state, state_out=apart)
    assert op.status() == 0
    for _ in range(3):
        same = state.clone()
        assert torch.equal(op.forward(q, k, v, g, beta, ints(at), state_in=same, state_out=same), out)
        assert torch.equal(same, apart)
    if h <= 4:
        check(out, apart, R.delta_rule(q, k, v, g, beta, at, state, 128 ** -0.5, True), at)


@pytest.mark.parametrize("at", [[0, 200, 100], [150, 20, 200], [-3, 100, 200], [0, 100, 500], [2 ** 31 - 1, -2 ** 31, 7]])
def test_bad_offsets_of_chunked_calls(at):
    # long enough for the chunked kernels: every slot they read lies in the workspace whatever the offsets are
    q, k, v, g, beta = inputs(23, "bf16", 200, 1, 2, 64, 64)
    guard = torch.full((204, 2, 64), 5.0, device="cuda", dtype=torch.bfloat16)
    op = bd.DeltaRule(1, 2, 64, 64, 2, 200, "bf16")
    op.workspace.zero_()
    so = torch.zeros(2, 2, 64, 64, device="cuda")
    op.forward(q, k, v, g, beta, ints(at), state_out=so, out=guard[2:202])
    assert op.status() == -2
    assert (guard[:2] == 5.0).all() and (guard[202:] == 5.0).all()
    out = op.forward(q, k, v, g, beta, ints([0, 100, 200]), state_out=so)
    assert op.status() == 0
    check(out, so, R.delta_rule(q, k, v, g, beta, [0, 100, 200], None, 0.125, True), [0, 100, 200])


WIDTHS_OF_WHOLE_STATES = """
import torch
from linear_compressed_attention_b200 import binding as bd
S, h, dv = 24, 16, 128
for dt, name in ((torch.bfloat16, "bf16"), (torch.float32, "f32")):
    q, k = (torch.ones(S, h, {dk}, device="cuda", dtype=dt) for _ in "qk")
    v = torch.ones(S, h, dv, device="cuda", dtype=dt)
    z, state = torch.zeros(S, h, device="cuda"), torch.zeros(S, h, {dk}, dv, device="cuda")
    out = bd.DeltaRule(h, h, {dk}, dv, S, 0, name, scale=1.0, qk_norm=False).step(q, k, v, z, z + 1, state)
    assert (state == 1).all() and (out == {dk}).all()
"""


@pytest.mark.parametrize("dk", [88, 96, 104])
def test_whole_states_in_a_process_that_ran_no_wider_ones(dk):
    # a state of 96 x 128 fills 48 KB of dynamic shared memory to the byte, and the kernel has static memory besides;
    # the limit is the process's: once raised for a wider state it would serve this one too
    root = os.path.dirname(os.path.dirname(os.path.abspath(bd.__file__)))
    subprocess.run([sys.executable, "-c", WIDTHS_OF_WHOLE_STATES.format(dk=dk)], cwd=root, check=True, timeout=300)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [24, 88, 96, 120])
def test_step_of_whole_states_of_other_widths(dtype, dk):
    S, hq, h, dv = 24, 8, 16, 128
    q, k, v, g, beta = inputs(31, dtype, S, hq, h, dk, dv)
    state = torch.randn(S, h, dk, dv, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    op = bd.DeltaRule(hq, h, dk, dv, S, 0, dtype, scale=0.7)
    mine = state.clone()
    out = op.step(q, k, v, g, beta, mine)
    check(out, mine, R.delta_rule(q, k, v, g, beta, list(range(S + 1)), state, 0.7, True), [0, S])


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("size", [1e-20, 1e-24, 1e-30, 1e-38])
def test_rows_of_tiny_values_in_chunks(size, which, norm):
    # rows whose sum of squares is 0 or subnormal in fp32 and whose values are not 0
    n, at = 200, [0, 200]
    q, k, v, g, beta = inputs(41, "bf16", n, 1, 2, 64, 64, rate=0.05)
    if not norm:
        q, k = ((0.98 * x.float() / x.float().norm(dim=-1, keepdim=True)).to(x.dtype) for x in (q, k))
    x = q if which == "q" else k
    for t in (0, 10, 70, 71, 72, 199):
        x[t] = (size * x[t].float()).to(x.dtype)
    x[100] = 0
    x[100, 0, 5] = size
    state = torch.randn(1, 2, 64, 64, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    op = bd.DeltaRule(1, 2, 64, 64, 1, n, "bf16", qk_norm=norm)
    so = torch.zeros_like(state)
    out = op.forward(q, k, v, g, beta, ints(at), state_in=state, state_out=so)
    check(out, so, R.delta_rule(q, k, v, g, beta, at, state, 0.125, norm), at)


def test_rows_of_huge_queries_in_chunks():
    # queries as given whose sum of squares is past fp32: their outputs are finite
    n, at = 130, [0, 130]
    q, k, v, g, beta = inputs(42, "bf16", n, 1, 2, 64, 64, rate=0.05)
    k = (0.98 * k.float() / k.float().norm(dim=-1, keepdim=True)).to(k.dtype)
    q[[3, 64, 129]] *= 1e21
    state = torch.randn(1, 2, 64, 64, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    op = bd.DeltaRule(1, 2, 64, 64, 1, n, "bf16", qk_norm=False)
    so = torch.zeros_like(state)
    out = op.forward(q, k, v, g, beta, ints(at), state_in=state, state_out=so)
    check(out, so, R.delta_rule(q, k, v, g, beta, at, state, 0.125, False), at)


LATE = [1e4, 1e6, 1e8, 1e30, float("inf"), -float("inf"), float("nan")]


def run_late(op, x, at, state):
    out, so = torch.zeros_like(x["v"]), torch.zeros_like(state)
    op.forward(x["q"], x["k"], x["v"], x["g"], x["beta"], ints(at), state_in=state, state_out=so, out=out)
    assert op.status() == 0
    return out, so


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", LATE)
@pytest.mark.parametrize("hq,h,dk,dv,n,t", [(1, 2, 64, 64, 200, 60), (2, 2, 128, 128, 200, 127), (1, 1, 72, 40, 130, 64),
                                            (1, 2, 128, 128, 1500, 1100)])
def test_a_value_reaches_no_token_before_it_and_no_other_column(dtype, bad, hq, h, dk, dv, n, t):
    q, k, v, g, beta = inputs(51, dtype, n, hq, h, dk, dv, rate=0.02)
    state = torch.randn(1, h, dk, dv, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    x = dict(q=q, k=k, v=v, g=g, beta=beta)
    op = bd.DeltaRule(hq, h, dk, dv, 1, n, dtype)
    clean, clean_state = run_late(op, x, [0, n], state)
    check(clean, clean_state, R.delta_rule(q, k, v, g, beta, [0, n], state, dk ** -0.5, True), [0, n])
    beta[t, 0] = 0.9
    clean, clean_state = run_late(op, x, [0, n], state)
    v[t, 0, 7] = bad
    out, so = run_late(op, x, [0, n], state)
    assert torch.equal(out[:t], clean[:t])
    other = [c for c in range(dv) if c != 7]
    assert torch.equal(out[:, 0][:, other], clean[:, 0][:, other]) and torch.equal(out[:, 1:], clean[:, 1:])
    assert torch.equal(so[0, 0][:, other], clean_state[0, 0][:, other]) and torch.equal(so[0, 1:], clean_state[0, 1:])
    if bad - bad != 0:                                   # and reaches every later token of its column
        assert (~torch.isfinite(out[t:, 0, 7])).all() and (~torch.isfinite(so[0, 0, :, 7])).all()
    else:
        check(out, so, R.delta_rule(q, k, v, g, beta, [0, n], state, dk ** -0.5, True), [0, n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what,bad", [("q", float("nan")), ("q", float("inf")), ("k", float("nan")), ("k", float("inf")),
                                      ("g", float("nan")), ("beta", float("nan")), ("beta", float("inf"))])
@pytest.mark.parametrize("t", [0, 5, 17, 40, 47, 63, 64, 100])
def test_what_is_not_finite_reaches_no_token_before_it(dtype, bad, what, t):
    n, h = 150, 2
    q, k, v, g, beta = inputs(52, dtype, n, 1, h, 64, 64, rate=0.02)
    state = torch.randn(1, h, 64, 64, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    x = dict(q=q, k=k, v=v, g=g, beta=beta)
    op = bd.DeltaRule(1, h, 64, 64, 1, n, dtype)
    clean, clean_state = run_late(op, x, [0, n], state)
    if what in "qk":
        x[what][t, 0, 9] = bad
    else:
        x[what][t, 0] = bad                              # of the first head only
    out, so = run_late(op, x, [0, n], state)
    assert torch.equal(out[:t], clean[:t])
    if what == "q":                                      # one token's output
        assert torch.equal(out[t + 1:], clean[t + 1:]) and torch.equal(so, clean_state)
        assert (~torch.isfinite(out[t])).all()
    else:
        heads = h if what == "k" else 1
        assert (~torch.isfinite(out[t:, :heads])).all() and (~torch.isfinite(so[:, :heads])).all()
        assert torch.equal(out[:, heads:], clean[:, heads:]) and torch.equal(so[:, heads:], clean_state[:, heads:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e3, 1e7, 1e20])
@pytest.mark.parametrize("t", [0, 3, 8, 40, 70])
def test_a_large_state_that_is_forgotten_is_gone(dtype, size, t):
    # tokens behind the one that forgets all are those of a sequence that starts there
    n, h = 140, 2
    q, k, v, g, beta = inputs(53, dtype, n, 1, h, 64, 64, rate=0.02)
    g[t] = -float("inf")
    state = size * torch.randn(1, h, 64, 64, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")
    op = bd.DeltaRule(1, h, 64, 64, 1, n, dtype)
    out, so = run_late(op, dict(q=q, k=k, v=v, g=g, beta=beta), [0, n], state)
    # (bounds of a state 0: what was forgotten has no part in them)
    o, s, ob, sb = R.delta_rule(q[t:], k[t:], v[t:], g[t:], beta[t:], [0, n - t], None, 0.125, True)
    check(out[t:], so, (o, s, ob, sb), [0, n - t])


def test_status_is_that_of_a_call():
    # the word lies in memory as it came until a forward call sets it; single tokens have none
    q, k, v, g, beta = inputs(61, "bf16", 2, 1, 1, 64, 64)
    op = bd.DeltaRule(1, 1, 64, 64, 2, 2, "bf16")
    op.workspace.fill_(0x5a)
    assert op.status() == 0
    op.step(q, k, v, g, beta, torch.zeros(2, 1, 64, 64, device="cuda"))
    assert op.status() == 0
    op.forward(q, k, v, g, beta, ints([0, 2, 1]))
    assert op.status() == -2
    op.forward(q, k, v, g, beta, ints([0, 1, 2]))
    assert op.status() == 0


def final_states(k, v, g, beta, at, state):
    """The final states in 64 bits and, per (sequence, head), the largest norm a state had on the way."""
    H, dk, dv = v.shape[1], k.shape[2], v.shape[2]
    kd = k.double() / (k.double().square().sum(-1, keepdim=True) + 1e-6).sqrt()
    kd, a, b, vd = kd.repeat_interleave(H // k.shape[1], 1), g.double().exp(), beta.double(), v.double()
    S, most = state.double().clone(), state.double().flatten(2).norm(dim=-1)
    for s in range(len(at) - 1):
        for t in range(at[s], at[s + 1]):
            S[s] *= a[t][:, None, None]
            u = b[t][:, None] * (vd[t] - torch.einsum("hk,hkv->hv", kd[t], S[s]))
            S[s] += kd[t][:, :, None] * u[:, None, :]
            most[s] = torch.maximum(most[s], S[s].flatten(1).norm(dim=-1))
    return S, most


@pytest.mark.parametrize("hq,h,dk,dv,lens", [(1, 2, 64, 64, [64]), (1, 2, 128, 128, [128, 70]), (2, 2, 72, 40, [200]),
                                             (1, 4, 128, 128, [1500])])
def test_states_of_chunks_keep_fp32_precision(hq, h, dk, dv, lens):
    # A chunk's three products each see an operand off by 2^-23 of its column's largest value, some 4.5 times the
    # column's mean size: 4.5 sqrt(3) 2^-23 = 9e-7 in norm, the roundings being independent; fp32 sums of up to 200 terms
    # add sqrt(200) 2^-24 = 8e-7; the triangular inverse of nearly orthogonal keys at most doubles it: 4e-6 of the
    # largest state for each chunk. An operand without its low half is off by 2^-12 of each value, 1e-4 in norm.
    at = offsets(lens)
    q, k, v, g, beta = inputs(71, "bf16", at[-1], hq, h, dk, dv, rate=0.01)
    state = torch.randn(len(lens), h, dk, dv, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda")
    op = bd.DeltaRule(hq, h, dk, dv, len(lens), at[-1], "bf16")
    so = torch.zeros_like(state)
    op.forward(q, k, v, g, beta, ints(at), state_in=state, state_out=so)
    ref, most = final_states(k, v, g, beta, at, state)
    chunks = torch.tensor([-(-n // 64) for n in lens], device="cuda")[:, None]
    e = (so.double() - ref).flatten(2).norm(dim=-1)
    assert (e <= 4e-6 * chunks * most).all(), float((e / most).max())


@pytest.mark.parametrize("S,h,lens", [(2, 20, [1500, 1100]), (1, 40, [2100])])
def test_parts_of_many_heads_match_the_64_bit_form(S, h, lens):
    # more blocks than SMs in each pass over the parts: some heads of the first and of the last blocks
    at = offsets(lens)
    q, k, v, g, beta = inputs(72, "bf16", at[-1], h // 2, h, 128, 128, rate=0.02)
    state = torch.randn(S, h, 128, 128, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda")
    op = bd.DeltaRule(h // 2, h, 128, 128, S, at[-1], "bf16")
    so = torch.zeros_like(state)
    out = op.forward(q, k, v, g, beta, ints(at), state_in=state, state_out=so)
    some = [0, h // 2, h - 2, h - 1]
    of = [i // 2 for i in some]
    ref = R.delta_rule(q[:, of], k[:, of], v[:, some], g[:, some], beta[:, some], at, state[:, some], 128 ** -0.5, True)
    check(out[:, some], so[:, some], ref, at)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("size", [0.0, 3e36])
def test_values_at_the_end_of_the_range_reach_no_token_before_them(sign, size):
    # the largest bf16 value, and what a state makes of it: finite in fp32 and past the largest bf16 value
    n, h, t = 64, 2, 40
    q, k, v, g, beta = inputs(54, "bf16", n, 1, h, 64, 64, rate=0.001)
    state = size * torch.randn(1, h, 64, 64, generator=torch.Generator(device="cuda").manual_seed(10), device="cuda")
    op = bd.DeltaRule(1, h, 64, 64, 1, n, "bf16")
    x = dict(q=q, k=k, v=v, g=g, beta=beta)
    clean, _ = run_late(op, x, [0, n], state)
    assert torch.isfinite(clean).all()
    v[t, 0, ::2] = sign * torch.finfo(torch.bfloat16).max
    out, _ = run_late(op, x, [0, n], state)
    assert torch.equal(out[:t], clean[:t]) and torch.equal(out[:, :, 1::2], clean[:, :, 1::2])
    assert torch.equal(out[:, 1:], clean[:, 1:])
