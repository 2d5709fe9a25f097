"""Packed softmax attention through the C ABI against its plain 64-bit form,
element by element within the bounds of packed_ref.attention."""
import numpy as np
import pytest
import torch

import packed_ref as R
from linear_compressed_attention_b200 import binding as bd
from packed_ref import float32_default  # noqa: F401

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def offsets(lens, start=0):
    at = [start]
    for n in lens:
        at.append(at[-1] + n)
    return at


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def draw(seed, dtype, rows, heads, d, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (gain * torch.randn(rows, heads, d, generator=g, device="cuda")).to(DT[dtype])


def run(dtype, heads, kv, d, lq, lk, causal, seed=0, gain=1.5, scale=None, behind=5):
    """A call with `behind` rows after the last sequence; checks every row."""
    q_at, k_at = offsets(lq), offsets(lk)
    q = draw(seed, dtype, q_at[-1] + behind, heads, d, gain)
    k, v = (draw(seed + i, dtype, k_at[-1] + behind, kv, d) for i in (1, 2))
    scale = d ** -0.5 if scale is None else scale
    op = bd.PackedAttention(heads, kv, d, len(lq), q.shape[0], max(lk), dtype, causal=causal, scale=scale)
    outs = []
    for _ in range(2):
        out = torch.full_like(q, 7.0)
        op.forward(q, k, v, ints(q_at), ints(k_at), out=out)
        assert op.status() == 0
        outs.append(out)
    assert torch.equal(*outs)
    ref, bound = R.attention(q, k, v, q_at, k_at, None, causal, scale)
    n = q_at[-1]
    assert torch.equal(outs[0][n:], torch.full_like(q[n:], 7.0))   # rows behind the last sequence
    err = (outs[0][:n].double() - ref[:n]).abs()
    assert torch.isfinite(outs[0][:n]).all()
    assert (err <= bound[:n]).all(), float((err / bound[:n]).max())


SHAPES = [
    # heads, kv_heads, d: shared heads 1, 2, 3, 4, 7, 8, 64; widths on and off the tile sizes
    (16, 16, 72), (8, 2, 64), (32, 8, 128), (6, 2, 80), (7, 1, 8), (8, 1, 128), (64, 1, 64), (3, 3, 96), (4, 2, 32),
    (2, 1, 104),
]
LENS = {
    "ragged": ([1, 130, 0, 63, 300, 64, 65], [1, 130, 0, 63, 300, 64, 65]),
    "more_keys": ([3, 1, 128, 40], [260, 1, 129, 1000]),
    "fewer_keys": ([70, 129, 5, 1], [3, 128, 0, 1]),          # causal: the first rows see nothing
    "one_each": ([1] * 40, list(range(40))),
}


@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads,kv,d", SHAPES)
def test_bf16(heads, kv, d, causal, lens):
    run("bf16", heads, kv, d, *LENS[lens], causal, seed=heads + d)


@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads,kv,d", [(4, 2, 64), (3, 1, 72), (2, 2, 128), (5, 5, 24)])
def test_f32(heads, kv, d, causal, lens):
    run("f32", heads, kv, d, *LENS[lens], causal, seed=heads + d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lq,lk", [([1], [4500]), ([2, 1], [3000, 777]), ([1] * 3, [0, 1, 2100]), ([9], [2049]), ([5], [2])])
def test_long_key_lists_are_split_and_joined(dtype, lq, lk):
    run(dtype, 8, 2, 64, lq, lk, True, seed=3)
    run(dtype, 3, 1, 72, lq, lk, False, seed=4)


def test_large_scores_and_negative_ones():
    # scores of hundreds: the running maximum has to move; and all of them far below zero
    run("bf16", 4, 2, 64, [200, 33], [700, 500], True, gain=60.0)
    run("f32", 4, 2, 64, [100, 33], [300, 200], True, gain=60.0)
    run("bf16", 4, 4, 64, [50], [400], False, gain=1e-3, scale=2.0)


def test_rising_scores_move_the_maximum_in_every_tile():
    # key j scores j / 2: every key tile brings a new maximum
    d, n = 64, 1500
    q = torch.zeros(300, 2, d, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(n, 2, d, device="cuda", dtype=torch.bfloat16)
    q[..., :2] = 1.0
    j = torch.arange(n, device="cuda")
    k[:, :, 0] = ((j // 8 * 8) / 2).to(torch.bfloat16)[:, None]       # (exact in bf16 up to the rounding shared by both sides)
    k[:, :, 1] = ((j % 8) / 2).to(torch.bfloat16)[:, None]
    v = draw(5, "bf16", n, 2, d)
    for causal in (False, True):
        op = bd.PackedAttention(2, 2, d, 1, 300, n, "bf16", causal=causal, scale=1.0)
        out = op.forward(q, k, v, ints([0, 300]), ints([0, n]))
        ref, bound = R.attention(q, k, v, [0, 300], [0, n], None, causal, 1.0)
        assert ((out.double() - ref).abs() <= bound).all()


def test_cache_filled_in_part_with_garbage_behind():
    S, cap, H, K, d = 5, 700, 8, 2, 128
    lens = [0, 1, 130, 700, 257]
    for nq in (1, 3):
        q = draw(9, "bf16", S * nq, H, d)
        k, v = draw(10, "bf16", S * cap, K, d), draw(11, "bf16", S * cap, K, d)
        for s, n in enumerate(lens):                     # what lies behind a cache's length is not used
            k[s * cap + n:(s + 1) * cap] = float("nan")
            v[s * cap + n:(s + 1) * cap] = float("inf")
        q_at, k_at = offsets([nq] * S), offsets([cap] * S)
        op = bd.PackedAttention(H, K, d, S, S * nq, cap, "bf16", causal=True)
        out = op.forward(q, k, v, ints(q_at), ints(k_at), ints(lens))
        assert op.status() == 0
        ref, bound = R.attention(q, k, v, q_at, k_at, lens, True, d ** -0.5)
        assert torch.isfinite(out).all()
        assert ((out.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(dtype, bad, where):
    H, K, d, n = 4, 2, 64, 300
    q, k, v = draw(20, dtype, n, H, d), draw(21, dtype, n, K, d), draw(22, dtype, n, K, d)
    clean_k, clean_v = k.clone(), v.clone()
    j = 150
    (k if where == "k" else v)[j, 1, 3] = bad
    op = bd.PackedAttention(H, K, d, 1, n, n, dtype, causal=True)
    out = op.forward(q, k, v, ints([0, n]), ints([0, n])).double()
    ref, bound = R.attention(q, clean_k, clean_v, [0, n], [0, n], None, True, d ** -0.5)
    ok = ((out - ref).abs() <= bound)
    assert ok[:, :2].all()                               # heads of the other key/value head
    assert ok[:j].all()                                  # rows before it
    if where == "v":                                     # only that column, in every row that sees it
        assert ok[:, :, [c for c in range(d) if c != 3]].all()
        seen = out[j:, 2:, 3]
        assert torch.isnan(seen).all() if bad != bad else (~torch.isfinite(seen)).all()
    elif bad != bad:
        assert torch.isnan(out[j:, 2:]).all()


def test_strided_slices_of_one_projection():
    H, K, d, n = 6, 2, 64, 211
    qkv = draw(30, "bf16", n, H + 2 * K, d)
    q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
    wide = torch.full((n, H + 1, d), 3.0, device="cuda", dtype=torch.bfloat16)
    op = bd.PackedAttention(H, K, d, 2, n, n, "bf16", causal=True)
    at = [0, 77, n]
    op.forward(q, k, v, ints(at), ints(at), out=wide[:, :H])
    ref, bound = R.attention(q, k, v, at, at, None, True, d ** -0.5)
    assert ((wide[:, :H].double() - ref).abs() <= bound).all()
    assert (wide[:, H] == 3.0).all()


def test_element_offsets_past_32_bits():
    # a cache whose last rows lie more than 2^31 elements in
    K, d, rows = 8, 128, (1 << 21) + 5000
    kv = torch.zeros(rows, K, d, device="cuda", dtype=torch.bfloat16)
    n = 400
    kv[-n:] = draw(40, "bf16", n, K, d)
    q = draw(41, "bf16", 2, 2 * K, d)
    op = bd.PackedAttention(2 * K, K, d, 2, 2, n, "bf16", causal=True)
    out = op.forward(q, kv, kv, ints([0, 1, 2]), ints([0, 0, rows]), ints([0, 0]))
    assert (out == 0).all()
    k_at = ints([rows - n, rows - n + 100, rows])
    out = op.forward(q, kv, kv, ints([0, 1, 2]), k_at)
    assert op.status() == 0
    ref, bound = R.attention(q, kv[-n:], kv[-n:], [0, 1, 2], [0, 100, n], None, True, d ** -0.5)
    assert ((out.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("q_at,k_at,lens,max_k", [
    ([0, 20, 10], [0, 30, 60], None, 64), ([-5, 10, 20], [0, 30, 60], None, 64), ([0, 10, 500], [0, 30, 60], None, 64),
    ([0, 10, 20], [0, 30, 61], None, 64), ([0, 10, 20], [40, 30, 60], None, 64), ([0, 10, 20], [0, 30, 60], [31, 5], 64),
    ([0, 10, 20], [0, 30, 60], [-1, 5], 64), ([0, 10, 20], [0, 30, 60], None, 29),
    ([0, 2 ** 31 - 1, -2 ** 31], [2 ** 31 - 1, -2 ** 31, 5], [2 ** 31 - 1, -2 ** 31], 64),
])
def test_bad_offsets_are_recorded_and_stay_inside(q_at, k_at, lens, max_k):
    # clamped in the kernels (packed_seq.cuh): nothing outside the rows given is touched
    for dtype in ("bf16", "f32"):
        q, k, v = draw(50, dtype, 20, 4, 64), draw(51, dtype, 60, 2, 64), draw(52, dtype, 60, 2, 64)
        guard = torch.full((24, 4, 64), 5.0, device="cuda", dtype=DT[dtype])
        op = bd.PackedAttention(4, 2, 64, 2, 20, max_k, dtype, causal=True)
        op.forward(q, k, v, ints(q_at), ints(k_at), None if lens is None else ints(lens), out=guard[2:22])
        assert op.status() == -2
        assert (guard[:2] == 5.0).all() and (guard[22:] == 5.0).all()
        # the word is set anew by the next call
        op.forward(q, k, v, ints([0, 10, 20]), ints([0, 20, 40]), ints([1, 2]), out=guard[2:22])
        assert op.status() == 0


def test_no_rows():
    op = bd.PackedAttention(4, 2, 64, 2, 10, 64, "bf16")
    e = torch.empty(0, 4, 64, device="cuda", dtype=torch.bfloat16)
    kv = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    assert op.forward(e, kv, kv, ints([0, 0, 0]), ints([0, 0, 0])).shape == (0, 4, 64)
    assert op.status() == 0
    q = draw(60, "bf16", 3, 4, 64)
    out = op.forward(q, kv, kv, ints([0, 1, 3]), ints([0, 0, 0]))   # no key at all
    assert (out == 0).all() and op.status() == 0


def test_captured_call_replays_with_other_lengths_on_another_stream():
    H, K, d, S, n = 8, 2, 64, 3, 400
    q, k, v = draw(70, "bf16", n, H, d), draw(71, "bf16", n, K, d), draw(72, "bf16", n, K, d)
    qo, ko = ints([0, 100, 250, n]), ints([0, 100, 250, n])
    out = torch.zeros_like(q)
    ops = [bd.PackedAttention(H, K, d, S, n, n, "bf16", causal=True) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops[0].forward(q, k, v, qo, ko, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ops[0].forward(q, k, v, qo, ko, out=out)
    torch.cuda.synchronize()
    for at in ([0, 100, 250, n], [0, 1, 1, 300], [0, 0, 399, n]):
        qo.copy_(ints(at))
        ko.copy_(ints(at))
        out.fill_(2.0)
        graph.replay()
        torch.cuda.synchronize()
        assert ops[0].status() == 0
        ref, bound = R.attention(q, k, v, at, at, None, True, d ** -0.5)
        m = at[-1]
        assert ((out[:m].double() - ref[:m]).abs() <= bound[:m]).all()
        assert (out[m:] == 2.0).all()
        eager = ops[1].forward(q, k, v, qo, ko, out=torch.full_like(q, 2.0))
        assert torch.equal(eager, out)


def test_two_calls_at_once_have_workspaces_of_their_own():
    H, K, d = 8, 2, 128
    lens = [3000]
    q, k, v = draw(80, "bf16", 1, H, d), draw(81, "bf16", 3000, K, d), draw(82, "bf16", 3000, K, d)
    ops = [bd.PackedAttention(H, K, d, 1, 1, 3000, "bf16", causal=True) for _ in range(2)]
    want = ops[0].forward(q, k, v, ints([0, 1]), ints([0, 3000])).clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    qo, ko = ints([0, 1]), ints([0, 3000])
    torch.cuda.synchronize()
    outs = [torch.zeros_like(q) for _ in range(2)]
    for _ in range(20):
        for op, s, o in zip(ops, streams, outs):
            op.forward(q, k, v, qo, ko, out=o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want) and lens


@pytest.mark.parametrize("S,heads,n,d", [(500, 16, 3, 32), (230, 16, 130, 64)])
def test_many_sequences(S, heads, n, d):
    # more items than a block finds at a time; short and longer row tiles, one of every seven sequences empty
    lens = [0 if s % 7 == 3 else n for s in range(S)]
    if n > 100:
        lens = [n + 21 if m else 0 for m in lens]
    run("bf16", heads, heads, d, lens, lens, True, seed=6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["k", "v"])
def test_new_tokens_do_not_see_what_comes_after_them(dtype, where):
    # three new tokens over a split cache; what is not finite lies in the last key, which only the last of them sees
    H, K, d, n = 8, 2, 64, 3001
    q, k, v = draw(90, dtype, 3, H, d), draw(91, dtype, n, K, d), draw(92, dtype, n, K, d)
    ref, bound = R.attention(q, k, v, [0, 3], [0, n], None, True, d ** -0.5)
    (k if where == "k" else v)[n - 1, 0, 5] = float("nan")
    op = bd.PackedAttention(H, K, d, 1, 3, n, dtype, causal=True)
    out = op.forward(q, k, v, ints([0, 3]), ints([0, n])).double()
    ok = (out - ref).abs() <= bound
    assert ok[:2].all() and ok[2, H // 2:].all()
    assert torch.isnan(out[2, :H // 2, 5]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [33, 64])
def test_many_heads_on_one_key_head_with_split_keys(dtype, heads):
    # more than 32 query heads a key/value head: one row a tile of the fp32 kernel; the workspace is the query's
    run(dtype, heads, 1, 64, [3], [4500], True, seed=7)
    run(dtype, heads, 1, 64, [1, 0, 2], [2100, 5, 3000], False, seed=8, behind=0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("n,nq,j", [(100, 100, 70), (200, 200, 20), (3001, 3, 2999), (3001, 3, 1500)])
def test_what_is_not_finite_reaches_rows_whose_weight_of_it_is_zero(dtype, bad, n, nq, j):
    # key j scores 400 below the others: its weight is 0 in fp32, in tiles with masked keys and in others alike
    H, K, d = 4, 2, 64
    q, k, v = draw(100, dtype, nq, H, d), draw(101, dtype, n, K, d), draw(102, dtype, n, K, d)
    q[..., 0], k[..., 0], k[j, :, 0] = 20.0, 0.0, -160.0
    ref, bound = R.attention(q, k, v, [0, nq], [0, n], None, True, d ** -0.5)
    v[j, 1, 3] = bad
    op = bd.PackedAttention(H, K, d, 1, nq, n, dtype, causal=True)
    out = op.forward(q, k, v, ints([0, nq]), ints([0, n])).double()
    first = max(0, j - (n - nq))                         # the first row that sees it
    ok = (out - ref).abs() <= bound
    assert ok[:first].all() and ok[:, :2].all() and ok[:, :, [c for c in range(d) if c != 3]].all()
    assert (~torch.isfinite(out[first:, 2:, 3])).all()
