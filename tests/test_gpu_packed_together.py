"""The packed-sequence operators as a layer stack uses them: block norm, gated
delta rule, block norm, causal softmax attention over a cache, block norm, on
packed prompts of different lengths and then token by token, from projections
that are slices of one tensor. Each step is given what the step before it wrote,
and is held to its own 64-bit form on that."""
import pytest
import torch

import packed_ref as R
from linear_compressed_attention_b200 import binding as bd
from packed_ref import float32_default  # noqa: F401

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Stack:
    """Two mixers with norms between, weights drawn once."""

    def __init__(self, dtype, S, rows, cap):
        self.dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.H, self.K, self.d, self.C, self.S, self.cap = 4, 2, 64, 256, S, cap
        g = torch.Generator(device="cuda").manual_seed(3)

        def w(*s, gain=1.0):
            return (gain * torch.randn(*s, generator=g, device="cuda")).to(self.dt)
        C, H, K, d = self.C, self.H, self.K, self.d
        self.w_delta = w(C, (2 * K + H) * d, gain=C ** -0.5)
        self.w_gates = w(C, 2 * H, gain=C ** -0.5)
        self.w_attn = w(C, (H + 2 * K) * d, gain=C ** -0.5)
        self.n_w = (1 + 0.1 * torch.randn(C, generator=g, device="cuda")).to(self.dt)
        self.delta = bd.DeltaRule(K, H, d, d, S, rows, dtype)
        self.attn = bd.PackedAttention(H, K, d, S, rows, cap, dtype, causal=True)
        self.norm0 = bd.BlockNorm(C, dtype, pre="rms", pre_w=self.n_w)
        self.norm1 = bd.BlockNorm(C, dtype, post="rms", pre="rms", gate_act="tanh", res_scale=0.5, post_w=self.n_w,
                                  pre_w=self.n_w)
        self.state = torch.zeros(S, H, d, d, device="cuda")
        self.k = torch.full((S * cap, K, d), float("nan"), device="cuda", dtype=self.dt)   # an unused cache holds anything
        self.v = self.k.clone()
        self.len = [0] * S

    def check(self, got, ref, bound, what):
        e = (got.double() - ref).abs()
        assert torch.isfinite(got).all() and (e <= bound).all(), (what, float((e / bound).max()))

    def norm(self, op, x, y, gate, at, post, act, rho):
        sample = torch.repeat_interleave(torch.arange(self.S, device="cuda"), torch.diff(torch.tensor(at)).cuda())
        vec = dict(pre_w=self.n_w)
        if y is not None:
            vec |= dict(post_w=self.n_w, gate=gate)
        r, h = op.forward(x, y, gate=gate if y is not None else None, offsets=ints(at))
        ref = R.block_norm(x, y, sample, post, "rms", act, 1e-6, rho, vec)
        self.check(r, ref[0], ref[2], "r")
        self.check(h, ref[1], ref[3], "h")
        return r, h

    def forward(self, x, gate, lens, step):
        """x: the packed new rows of each sequence, lens of them."""
        H, K, d, S = self.H, self.K, self.d, self.S
        at = [0]
        for n in lens:
            at.append(at[-1] + n)
        x, h = self.norm(self.norm0, x, None, None, at, "none", "linear", 1.0)
        p = (h @ self.w_delta).view(-1, 2 * K + H, d)
        q, k, v = p[:, :K], p[:, K:2 * K], p[:, 2 * K:]
        ab = (h @ self.w_gates).float()
        g, beta = -0.2 * torch.nn.functional.softplus(ab[:, :H]), torch.sigmoid(ab[:, H:])
        before = self.state.clone()
        if step:
            o = self.delta.step(q, k, v, g, beta, self.state)
        else:
            o = self.delta.forward(q, k, v, g, beta, ints(at), state_in=self.state, state_out=self.state)
            assert self.delta.status() == 0
        ref, rs, ob, sb = R.delta_rule(q, k, v, g, beta, at, before, d ** -0.5, True)
        assert ((o.double() - ref).norm(dim=-1) <= ob).all()
        assert ((self.state.double() - rs).flatten(2).norm(dim=-1) <= sb).all()
        x, h = self.norm(self.norm1, x, o.reshape(-1, self.C), gate, at, "rms", "tanh", 0.5)
        p = (h @ self.w_attn).view(-1, H + 2 * K, d)
        for s in range(S):                    # the new keys and values go behind the sequence's cache
            b = s * self.cap + self.len[s]
            self.k[b:b + lens[s]] = p[at[s]:at[s + 1], H:H + K]
            self.v[b:b + lens[s]] = p[at[s]:at[s + 1], H + K:]
            self.len[s] += lens[s]
        k_at = [s * self.cap for s in range(S + 1)]
        o = self.attn.forward(p[:, :H], self.k, self.v, ints(at), ints(k_at), ints(self.len))
        assert self.attn.status() == 0
        ref, bound = R.attention(p[:, :H], self.k, self.v, at, k_at, self.len, True, d ** -0.5)
        self.check(o, ref, bound, "attention")
        return self.norm(self.norm1, x, o.reshape(-1, self.C), gate, at, "rms", "tanh", 0.5)[0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompts_then_tokens(dtype):
    lens = [70, 1, 133]
    st = Stack(dtype, 3, sum(lens), 160)
    g = torch.Generator(device="cuda").manual_seed(4)
    gate = torch.randn(3, 256, generator=g, device="cuda").to(st.dt)
    st.forward(torch.randn(sum(lens), 256, generator=g, device="cuda").to(st.dt), gate, lens, False)
    st.forward(torch.randn(7, 256, generator=g, device="cuda").to(st.dt), gate, [3, 4, 0], False)   # prompts go on
    for _ in range(3):
        st.forward(torch.randn(3, 256, generator=g, device="cuda").to(st.dt), gate, [1, 1, 1], True)


def test_objects_are_used_on_their_own_device(monkeypatch):
    # a workspace or kept weights of another device: refused, with every other tensor where it should be (one device is
    # visible here: the object is told that its memory lies on the next one)
    attn = bd.PackedAttention(2, 2, 64, 1, 4, 4, "bf16")
    delta = bd.DeltaRule(2, 2, 64, 64, 1, 4, "bf16")
    norm = bd.BlockNorm(64, "bf16", pre_w=torch.ones(64, device="cuda", dtype=torch.bfloat16))
    at = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    x = torch.ones(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    z = torch.zeros(4, 2, device="cuda")
    state = torch.zeros(1, 2, 64, 64, device="cuda")
    calls = [(attn, lambda: attn.forward(x, x, x, at, at)), (delta, lambda: delta.forward(x, x, x, z, z, at)),
             (delta, lambda: delta.step(x[:1], x[:1], x[:1], z[:1], z[:1], state)), (norm, lambda: norm.forward(x[:, 0]))]
    for op, call in calls:
        call()
        name = "devices" if op is norm else "device"
        with monkeypatch.context() as m:
            m.setattr(op, name, {1} if op is norm else 1)
            with pytest.raises(ValueError, match="device"):
                call()
