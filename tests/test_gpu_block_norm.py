"""The block norm (norm after a branch, gate, residual, norm before the next)
through the C ABI against its plain 64-bit form, element by element within the
bounds of packed_ref.block_norm."""
import pytest
import torch

import packed_ref as R
from linear_compressed_attention_b200 import binding as bd
from packed_ref import float32_default  # noqa: F401

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rand(seed, dtype, *shape, mean=0.0, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (mean + gain * torch.randn(*shape, generator=g, device="cuda")).to(DT[dtype])


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check(got, ref, bound):
    e = (got.double() - ref).abs()
    assert (e <= bound).all(), float((e / bound).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [1, 8, 31, 256, 513, 1001, 1152, 1536, 2048, 2056, 2500, 4104, 16384, 16383])
@pytest.mark.parametrize("post,pre,act", [("rms", "layer", "linear"), ("layer", "rms", "tanh"), ("none", "none", "tanh"),
                                          ("none", "layer", "linear")])
def test_widths_and_kinds(dtype, C, post, pre, act):
    rows, at = 37, [0, 5, 5, 30]
    x, y = rand(1, dtype, rows, C, mean=0.3), rand(2, dtype, rows, C, mean=-0.5, gain=3.0)
    mod = rand(3, dtype, 3, 3, C, gain=0.5)
    kept = dict(gate0=rand(4, dtype, C, gain=0.1), scale0=rand(5, dtype, C, gain=0.1), shift0=rand(6, dtype, C, gain=0.1))
    if post != "none":
        kept |= dict(post_w=rand(7, dtype, C, mean=1.0, gain=0.2), post_b=rand(8, dtype, C, gain=0.2))
    if pre != "none":
        kept |= dict(pre_w=rand(9, dtype, C, mean=1.0, gain=0.2), pre_b=rand(10, dtype, C, gain=0.2))
    op = bd.BlockNorm(C, dtype, post=post, pre=pre, gate_act=act, eps=1e-5, res_scale=0.7, **kept)
    sample = torch.tensor([0] * 5 + [2] * 25, device="cuda")
    r, h = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    op.forward(x, y, gate=mod[:, 0], scale=mod[:, 1], shift=mod[:, 2], offsets=ints(at), r_out=r, h_out=h)
    ref = R.block_norm(x[:30], y[:30], sample, post, pre, act, 1e-5, 0.7,
                       kept | dict(gate=mod[:, 0], scale=mod[:, 1], shift=mod[:, 2]))
    check(r[:30], ref[0], ref[2])
    check(h[:30], ref[1], ref[3])
    assert (r[30:] == 9.0).all() and (h[30:] == 9.0).all()    # rows in no sample


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [64, 65, 3000])
def test_missing_parts_and_one_output(dtype, C):
    n = 24
    x, y, m = rand(11, dtype, n, C), rand(12, dtype, n, C), rand(13, dtype, 4, C)
    sample = torch.arange(n, device="cuda") // 6
    one = torch.zeros(n, dtype=torch.long, device="cuda")
    # no gate: 1; no samples' vectors at all
    r, h = bd.BlockNorm(C, dtype, post="rms", pre="rms").forward(x, y)
    ref = R.block_norm(x, y, one, "rms", "rms", "linear", 1e-6, 1.0, {})
    check(r, ref[0], ref[2])
    check(h, ref[1], ref[3])
    # no branch: the first norm of a block; no r
    r, h = bd.BlockNorm(C, dtype, pre="layer").forward(x, scale=m, shift=m, want_r=False)
    ref = R.block_norm(x, None, sample, "none", "layer", "linear", 1e-6, 1.0, dict(scale=m, shift=m))
    assert r is None
    check(h, ref[1], ref[3])
    # no h: the last residual; gates of equal shares of the rows
    r, h = bd.BlockNorm(C, dtype, post="layer", pre="none", gate_act="tanh").forward(x, y, gate=m, want_h=False)
    ref = R.block_norm(x, y, sample, "layer", "none", "tanh", 1e-6, 1.0, dict(gate=m))
    assert h is None
    check(r, ref[0], ref[2])
    # only a common gate
    g0 = rand(14, dtype, C)
    r, _ = bd.BlockNorm(C, dtype, gate0=g0).forward(x, y)
    check(r, *(R.block_norm(x, y, one, "none", "layer", "linear", 1e-6, 1.0, dict(gate0=g0))[i] for i in (0, 2)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [128, 129, 2304])
def test_in_place_and_strided(dtype, C):
    n = 50
    base = rand(15, dtype, n, 2 * C + 8)
    x, y = base[:, :C], base[:, C + 8:]
    op = bd.BlockNorm(C, dtype, post="rms", pre="layer", res_scale=0.5)
    want = op.forward(x.contiguous(), y.contiguous())
    r, h = op.forward(x, y)
    assert torch.equal(r, want[0]) and torch.equal(h, want[1])
    op.forward(x, y, r_out=x, h_out=y)          # r over x, h over y
    assert torch.equal(x, want[0]) and torch.equal(y, want[1])
    assert torch.equal(base[:, C:C + 8], rand(15, dtype, n, 2 * C + 8)[:, C:C + 8])


def test_rows_of_large_mean_keep_their_variance():
    # mean 1000, deviation 1: sums of squares would lose it in fp32
    x = rand(16, "f32", 9, 1152, mean=1000.0)
    _, h = bd.BlockNorm(1152, "f32", pre="layer").forward(x)
    z = torch.zeros(9, dtype=torch.long, device="cuda")
    ref = R.block_norm(x, None, z, "none", "layer", "linear", 1e-6, 1.0, {})
    check(h, ref[1], ref[3])
    assert (h.double() - ref[1]).abs().max() < 1e-3


def test_constant_and_zero_rows():
    x = torch.zeros(3, 256, device="cuda")
    x[1] = 4.0
    _, h = bd.BlockNorm(256, "f32", pre="layer").forward(x)
    assert (h == 0).all()
    _, h = bd.BlockNorm(256, "f32", pre="rms").forward(x)
    assert (h[0] == 0).all() and (h[1] - 1).abs().max() < 1e-5


def test_bad_offsets_stay_inside():
    x, y, m = rand(17, "bf16", 10, 64), rand(18, "bf16", 10, 64), rand(19, "bf16", 2, 64)
    op = bd.BlockNorm(64, "bf16")
    for at in ([5, 2, 30], [-4, 100, 3], [2 ** 31 - 1, -2 ** 31, 0], [20, 30, 40]):
        guard = torch.full((14, 64), 5.0, device="cuda", dtype=torch.bfloat16)
        op.forward(x, y, gate=m, offsets=ints(at), r_out=guard[2:12], want_h=False)
        torch.cuda.synchronize()
        assert (guard[:2] == 5.0).all() and (guard[12:] == 5.0).all()


def test_captured_call_and_no_rows():
    x, y, m = rand(20, "bf16", 40, 1152), rand(21, "bf16", 40, 1152), rand(22, "bf16", 2, 1152)
    op = bd.BlockNorm(1152, "bf16", post="rms", pre="rms")
    at = ints([0, 20, 40])
    r, h = torch.zeros_like(x), torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        op.forward(x, y, gate=m, offsets=at, r_out=r, h_out=h)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            op.forward(x, y, gate=m, offsets=at, r_out=r, h_out=h)
    torch.cuda.synchronize()
    at.copy_(ints([0, 3, 31]))
    r.fill_(4.0)
    graph.replay()
    torch.cuda.synchronize()
    want = op.forward(x, y, gate=m, offsets=at, r_out=torch.full_like(x, 4.0))
    assert torch.equal(r, want[0]) and (r[31:] == 4.0).all()
    e = x[:0]
    assert op.forward(e, e, gate=m, offsets=ints([0, 0, 0]))[0].shape == (0, 1152)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [64, 300, 504, 768, 1000, 1152, 1288, 1536, 1999, 2048, 2304])
def test_many_rows(dtype, C):
    # enough rows for every layout of a row over threads; samples that begin and end inside a block's rows, and none
    n, at = 1500, [4, 5, 5, 600, 1203, 1497]
    x, y = rand(31, dtype, n, C), rand(32, dtype, n, C, gain=2.0)
    mod = rand(33, dtype, 5, 3, C, gain=0.5)
    w = rand(34, dtype, C, mean=1.0, gain=0.2)
    op = bd.BlockNorm(C, dtype, post="layer", pre="rms", gate_act="tanh", post_w=w, pre_b=w)
    r, h = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    op.forward(x, y, gate=mod[:, 0], scale=mod[:, 1], shift=mod[:, 2], offsets=ints(at), r_out=r, h_out=h)
    sample = torch.bucketize(torch.arange(4, 1497, device="cuda"), torch.tensor(at[1:], device="cuda"), right=True)
    ref = R.block_norm(x[4:1497], y[4:1497], sample, "layer", "rms", "tanh", 1e-6, 1.0,
                       dict(post_w=w, pre_b=w, gate=mod[:, 0], scale=mod[:, 1], shift=mod[:, 2]))
    check(r[4:1497], ref[0], ref[2])
    check(h[4:1497], ref[1], ref[3])
    for t in (r, h):
        assert (t[:4] == 9.0).all() and (t[1497:] == 9.0).all()
    r2, h2 = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    op.forward(x, y, gate=mod[:, 0], scale=mod[:, 1], shift=mod[:, 2], offsets=ints(at), r_out=r2, h_out=h2)
    assert torch.equal(r, r2) and torch.equal(h, h2)


def test_one_sample_a_row():
    n, C = 900, 264
    x, y, m = rand(41, "bf16", n, C), rand(42, "bf16", n, C), rand(43, "bf16", n, C)
    r, h = bd.BlockNorm(C, "bf16", post="rms", pre="layer").forward(x, y, gate=m, scale=m, shift=m)
    ref = R.block_norm(x, y, torch.arange(n, device="cuda"), "rms", "layer", "linear", 1e-6, 1.0,
                       dict(gate=m, scale=m, shift=m))
    check(r, ref[0], ref[2])
    check(h, ref[1], ref[3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("rows", [37, 700])
@pytest.mark.parametrize("C", [64, 1001, 1152, 3000])
def test_values_that_are_not_finite_stay_in_their_row_or_sample(dtype, bad, rows, C):
    x, y = rand(61, dtype, rows, C), rand(62, dtype, rows, C)
    mod = rand(63, dtype, 3, 3, C)
    at = ints([0, 5, 20, rows])
    op = bd.BlockNorm(C, dtype, post="rms", pre="layer")

    def run():
        return op.forward(x, y, gate=mod[:, 0], scale=mod[:, 1], shift=mod[:, 2], offsets=at)
    clean = run()
    for t in (x, y):                                     # one row: the norm before the next branch spreads it over the row
        was = t[7, 3].clone()
        t[7, 3] = bad
        r, h = run()
        t[7, 3] = was
        others = [i for i in range(rows) if i != 7]
        assert torch.equal(r[others], clean[0][others]) and torch.equal(h[others], clean[1][others])
        assert not torch.isfinite(r[7, 3]) and torch.isnan(h[7]).all()
    for i in range(3):                                   # one value of one sample's gate, scale, shift
        was = mod[1, i, 3].clone()
        mod[1, i, 3] = bad
        r, h = run()
        mod[1, i, 3] = was
        others = [i for i in range(rows) if not 5 <= i < 20]
        assert torch.equal(r[others], clean[0][others]) and torch.equal(h[others], clean[1][others])
        assert (~torch.isfinite((r if i == 0 else h)[5:20, 3])).all()
        if i:                                            # that column only
            cols = [c for c in range(C) if c != 3]
            assert torch.equal(r, clean[0]) and torch.equal(h[5:20][:, cols], clean[1][5:20][:, cols])
