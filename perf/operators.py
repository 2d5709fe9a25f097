"""Measured cases of the packed-sequence operators: softmax attention over packed sequences, the gated delta rule
(whole sequences and single tokens) and the block norm (norm after a branch, gate, residual, norm before the next).

`run` computes an operator in its plain form (elementary torch operations, fp32 or fp64) or, with `own`, through this
package's entry points. A case's sequence lengths are made from its own seed, so that it stays a dict of plain values."""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # Prompts of a text encoder whose query heads share key/value heads, packed end to end, causal.
        dict(name="attn_prompts_causal", op="attention", dtype="bf16", heads=32, kv_heads=8, d=128, nseq=5, min_q=1500,
             max_q=4100, self_keys=True, causal=True, max_k=0, lens=11),
        # Image rows of the 1024 px layer (16 heads of 72) over captions of different lengths: cross-attention.
        dict(name="attn_captions_d72", op="attention", dtype="bf16", heads=16, kv_heads=16, d=72, nseq=4, min_q=4096,
             max_q=4096, self_keys=False, causal=False, max_k=333, lens=12),
        # One new token of each of 32 running requests over its key/value cache (8K slots each, used in part).
        dict(name="attn_new_tokens", op="attention", dtype="bf16", heads=32, kv_heads=8, d=128, nseq=32, min_q=1, max_q=1,
             self_keys=False, causal=True, max_k=8192, lens=13),
        # One short fp32 batch, odd lengths: the parity type.
        dict(name="attn_short_f32", op="attention", dtype="f32", heads=8, kv_heads=4, d=64, nseq=6, min_q=1, max_q=515,
             self_keys=True, causal=True, max_k=0, lens=14),
        # One long prompt through a delta-rule layer, 16 heads of 128.
        dict(name="delta_long_prompt", op="delta", dtype="bf16", qk_heads=16, heads=16, d_k=128, d_v=128, nseq=1,
             min_t=8192, max_t=8192, state=False, lens=15),
        # A packed batch of ragged prompts that go on from kept states; query/key heads shared by pairs.
        dict(name="delta_ragged_states", op="delta", dtype="bf16", qk_heads=12, heads=24, d_k=64, d_v=64, nseq=9, min_t=1,
             max_t=2500, state=True, lens=16),
        # fp32 inputs, odd lengths.
        dict(name="delta_short_f32", op="delta", dtype="f32", qk_heads=4, heads=8, d_k=64, d_v=72, nseq=3, min_t=60, max_t=400,
             state=True, lens=17),
        # One new token of each of 64 running requests.
        dict(name="delta_new_tokens", op="delta_step", dtype="bf16", qk_heads=16, heads=32, d_k=128, d_v=128, nseq=64),
        # One new token of a single request: latency.
        dict(name="delta_one_token", op="delta_step", dtype="bf16", qk_heads=8, heads=8, d_k=64, d_v=64, nseq=1),
        # The 4096 px layer's tokens between two branches of a block: gated LayerNorm'd branch, modulated LayerNorm.
        dict(name="norm_px4096", op="norm", dtype="bf16", rows=65536, C=1152, samples=1, post="layer", pre="layer",
             act="linear", affine=False),
        # Image and prompt tokens of the MM layer, fp32, RMS norms with weights and a tanh gate.
        dict(name="norm_mm_f32", op="norm", dtype="f32", rows=4429, C=1536, samples=3, post="rms", pre="rms", act="tanh",
             affine=True),
        # One token of 8 requests: latency; an odd width.
        dict(name="norm_new_tokens", op="norm", dtype="bf16", rows=8, C=1001, samples=8, post="rms", pre="rms", act="linear",
             affine=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attention", "decode", "delta", "delta_step", "norm"])
    if op == "attention":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        kv = rng.randint(1, 8)
        d = rng.choice([32, 64, 72, 80, 96, 128])
        self_keys = rng.random() < 0.6
        hi = _log_int(rng, 2, 600 if dtype == "f32" else 4000)
        return dict(op="attention", dtype=dtype, heads=kv * rng.randint(1, 4), kv_heads=kv, d=d, nseq=rng.randint(1, 4),
                    min_q=rng.randint(1, hi), max_q=hi, self_keys=self_keys, causal=rng.random() < 0.6,
                    max_k=0 if self_keys else _log_int(rng, 1, 1000), lens=rng.randrange(1 << 20))
    if op == "decode":
        kv = rng.randint(1, 8)
        return dict(op="attention", dtype="bf16", heads=kv * rng.randint(1, 8), kv_heads=kv, d=rng.choice([64, 72, 128]),
                    nseq=_log_int(rng, 1, 32), min_q=1, max_q=rng.randint(1, 3), self_keys=False, causal=True,
                    max_k=_log_int(rng, 16, 8000), lens=rng.randrange(1 << 20))
    if op == "delta":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        qk = rng.randint(1, 8)
        hi = _log_int(rng, 2, 400 if dtype == "f32" else 4000)
        return dict(op="delta", dtype=dtype, qk_heads=qk, heads=qk * rng.randint(1, 2), d_k=rng.choice([32, 64, 72, 128]),
                    d_v=rng.choice([32, 64, 72, 128]), nseq=rng.randint(1, 6), min_t=rng.randint(1, hi), max_t=hi,
                    state=rng.random() < 0.5, lens=rng.randrange(1 << 20))
    if op == "delta_step":
        qk = rng.randint(1, 16)
        return dict(op="delta_step", dtype=rng.choice(["bf16", "f32"]), qk_heads=qk, heads=qk * rng.randint(1, 2),
                    d_k=rng.choice([32, 64, 72, 128]), d_v=rng.choice([32, 64, 72, 128]), nseq=_log_int(rng, 1, 64))
    rows = _log_int(rng, 1, 60000)
    kinds = ["rms", "layer"]
    return dict(op="norm", dtype=rng.choice(["bf16", "f32"]), rows=rows, C=_log_int(rng, 16, 2000),
                samples=rng.randint(1, min(rows, 5)), post=rng.choice(kinds + ["none"]), pre=rng.choice(kinds),
                act=rng.choice(["linear", "tanh"]), affine=rng.random() < 0.5)


def _lengths(seed, n, lo, hi):
    """n lengths of lo..hi, the largest among them."""
    r = random.Random(seed)
    got = [r.randint(lo, hi) for _ in range(n)]
    got[r.randrange(n)] = hi
    return got


def _attention_lengths(c):
    lq = _lengths(c["lens"], c["nseq"], c["min_q"], c["max_q"])
    return lq, (lq if c["self_keys"] else _lengths(c["lens"] + 1, c["nseq"], 1, c["max_k"]))


def _offsets(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    st = dict(case=c)
    if c["op"] == "attention":
        lq, lk = _attention_lengths(c)
        # sequences with keys of their own keep them in a cache of max_k slots each, filled up to their lengths
        cap = [n if c["self_keys"] else c["max_k"] for n in lk]
        q_at, k_at = _offsets(lq), _offsets(cap)
        st.update(q=(1.5 * normal(q_at[-1], c["heads"], c["d"])).to(dt), k=normal(k_at[-1], c["kv_heads"], c["d"]).to(dt),
                  v=normal(k_at[-1], c["kv_heads"], c["d"]).to(dt), q_offsets=ints(q_at), k_offsets=ints(k_at),
                  k_lens=ints(lk), most_q=max(lq), most_k=max(lk))
        st["out"] = torch.zeros_like(st["q"])
        if own:
            from linear_compressed_attention_b200 import binding as bd
            st["op"] = bd.PackedAttention(c["heads"], c["kv_heads"], c["d"], c["nseq"], q_at[-1], max(lk), c["dtype"],
                                          causal=c["causal"], scale=c["d"] ** -0.5)
        return st
    if c["op"] in ("delta", "delta_step"):
        lengths = _lengths(c["lens"], c["nseq"], c["min_t"], c["max_t"]) if c["op"] == "delta" else [1] * c["nseq"]
        rows = sum(lengths)
        silu = torch.nn.functional.silu
        # queries and keys leave an activation and are normalised by the operator; decays of a few tokens to a few thousand
        rate = torch.exp(math.log(0.001) + (math.log(0.5) - math.log(0.001)) *
                         torch.rand(c["heads"], generator=gen, device="cuda"))
        st.update(q=silu(normal(rows, c["qk_heads"], c["d_k"])).to(dt), k=silu(normal(rows, c["qk_heads"], c["d_k"])).to(dt),
                  v=silu(normal(rows, c["heads"], c["d_v"])).to(dt),
                  g=-rate * torch.nn.functional.softplus(normal(rows, c["heads"])),
                  beta=torch.sigmoid(normal(rows, c["heads"])), offsets=ints(_offsets(lengths)), most=max(lengths))
        st["state"] = None
        if c["op"] == "delta_step" or c["state"]:
            st["state"] = 0.3 * normal(c["nseq"], c["heads"], c["d_k"], c["d_v"])
        st["out"] = torch.zeros_like(st["v"])
        st["state_out"] = torch.zeros(c["nseq"], c["heads"], c["d_k"], c["d_v"], device="cuda")
        if own:
            from linear_compressed_attention_b200 import binding as bd
            st["op"] = bd.DeltaRule(c["qk_heads"], c["heads"], c["d_k"], c["d_v"], c["nseq"], rows, c["dtype"],
                                    scale=c["d_k"] ** -0.5, qk_norm=True)
        return st
    C, n = c["C"], c["samples"]
    each = c["rows"] // n
    st.update(x=normal(c["rows"], C).to(dt), y=(2.0 * normal(c["rows"], C)).to(dt),
              offsets=ints([each * i for i in range(n)] + [c["rows"]]))
    st["mod"] = (0.5 * normal(n, 3, C)).to(dt)  # gate, scale, shift of each sample
    st["post_w"] = (1 + 0.2 * normal(C)).to(dt) if c["affine"] and c["post"] != "none" else None
    st["pre_w"] = (1 + 0.2 * normal(C)).to(dt) if c["affine"] else None
    st["r"], st["h"] = torch.zeros_like(st["x"]), torch.zeros_like(st["x"])
    if own:
        from linear_compressed_attention_b200 import binding as bd
        st["op"] = bd.BlockNorm(C, c["dtype"], post=c["post"], pre=c["pre"], gate_act=c["act"], eps=1e-6, res_scale=0.8,
                                post_w=st["post_w"], pre_w=st["pre_w"])
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    if own:
        if c["op"] == "attention":
            return st["op"].forward(st["q"], st["k"], st["v"], st["q_offsets"], st["k_offsets"], st["k_lens"],
                                    out=st["out"])
        if c["op"] == "delta":
            st["op"].forward(st["q"], st["k"], st["v"], st["g"], st["beta"], st["offsets"], state_in=st["state"],
                             state_out=st["state_out"], out=st["out"])
            return st["out"], st["state_out"]
        if c["op"] == "delta_step":
            st["op"].step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"], out=st["out"])
            return st["out"], st["state"]
        return st["op"].forward(st["x"], st["y"], gate=st["mod"][:, 0], scale=st["mod"][:, 1], shift=st["mod"][:, 2],
                                offsets=st["offsets"], r_out=st["r"], h_out=st["h"])
    return {"attention": _attention, "delta": _delta, "delta_step": _delta_step, "norm": _norm}[c["op"]](st)


def _pad_index(offsets, lens, most):
    """Rows of each sequence in a padded batch [nseq, most] (clamped to the sequence), and which of them are real."""
    i = torch.arange(most, device=offsets.device)
    lens, begin = lens.long(), offsets[:-1].long()
    return begin[:, None] + torch.minimum(i, (lens - 1).clamp(min=0)[:, None]), i < lens[:, None]


def _unpad_index(offsets, rows, most):
    """Where each packed row lies in the padded batch, flattened."""
    r = torch.arange(rows, device=offsets.device)
    s = torch.searchsorted(offsets[1:].long(), r, right=True)
    return s * most + (r - offsets[:-1].long()[s])


def _attention(st):
    """softmax(scale q k^T) v per sequence; causal: query i of a sequence sees keys up to i + len_k - len_q."""
    c = st["case"]
    S, H, K, d = c["nseq"], c["heads"], c["kv_heads"], c["d"]
    lq = (st["q_offsets"][1:] - st["q_offsets"][:-1]).long()
    lk = st["k_lens"].long()
    iq, _ = _pad_index(st["q_offsets"], lq, st["most_q"])
    ik, real_k = _pad_index(st["k_offsets"], lk, st["most_k"])
    q = st["q"].float()[iq].view(S, st["most_q"], K, H // K, d).permute(0, 2, 3, 1, 4)
    k, v = (t[ik].float().permute(0, 2, 1, 3) for t in (st["k"], st["v"]))
    s = (q.reshape(S, K, -1, d) @ k.transpose(-1, -2)).view(S, K, H // K, st["most_q"], st["most_k"])
    s *= d ** -0.5
    mask = real_k[:, None, :]
    if c["causal"]:
        last = torch.arange(st["most_q"], device=s.device) + (lk - lq)[:, None]
        mask = mask & (torch.arange(st["most_k"], device=s.device) <= last[:, :, None])
    s.masked_fill_(~mask[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(S, K, -1, st["most_k"]) @ v).view(S, K, H // K, st["most_q"], d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(-1, H, d)
    return o[_unpad_index(st["q_offsets"], st["q"].shape[0], st["most_q"])].to(st["q"].dtype)


def _unit(x):
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)


def _delta(st):
    """The gated delta rule in chunks of 64 tokens: within a chunk through the inverse of a unit triangular matrix, from
    chunk to chunk through the state."""
    c = st["case"]
    S, H, dk, dv, L = c["nseq"], c["heads"], c["d_k"], c["d_v"], 64
    N = -(-st["most"] // L)
    lens = (st["offsets"][1:] - st["offsets"][:-1]).long()
    at, real = _pad_index(st["offsets"], lens, N * L)
    share = H // c["qk_heads"]

    def chunks(x):  # [rows, heads, ...] -> [S, H, N, L, ...], zeros behind a sequence's end
        x = x[at] * real.view(S, N * L, *[1] * (x.dim() - 1))
        return x.view(S, N, L, *x.shape[2:]).movedim(3, 1)

    q, k = (chunks(_unit(st[n].float())).repeat_interleave(share, 1) for n in "qk")
    v, beta, g = chunks(st["v"].float()), chunks(st["beta"])[..., None], chunks(st["g"]).double()
    G = g.cumsum(-1)
    low = torch.ones(L, L, dtype=torch.bool, device=q.device).tril()
    decay = (G[..., :, None] - G[..., None, :]).masked_fill_(~low, -math.inf).exp_().float()
    a = (beta * (k @ k.transpose(-1, -2)) * decay).tril(-1).double().neg_()
    T = torch.eye(L, device=q.device, dtype=torch.float64) + a
    for _ in range(5):  # (I - a)^-1 = (I + a)(I + a^2)(I + a^4)..., a^64 = 0
        a = a @ a
        T = T + a @ T
    T = T.float()
    eG = G.exp().float()[..., None]
    U0, W = T @ (beta * v), T @ (beta * eG * k)
    P = (q @ k.transpose(-1, -2)) * decay
    to_end = (G[..., -1:] - G).exp().float()[..., None]
    kT, whole = (k * to_end).transpose(-1, -2), G[..., -1].exp().float()[..., None, None]
    s = torch.zeros(S, H, dk, dv, device=q.device) if st["state"] is None else st["state"]
    o = torch.empty_like(v)
    for n in range(N):  # the recurrence over the chunks
        u = U0[:, :, n] - W[:, :, n] @ s
        o[:, :, n] = (eG[:, :, n] * q[:, :, n]) @ s + P[:, :, n] @ u
        s = whole[:, :, n] * s + kT[:, :, n] @ u
    o = (o * dk ** -0.5).movedim(1, 3).reshape(S * N * L, H, dv)
    return o[_unpad_index(st["offsets"], st["v"].shape[0], N * L)].to(st["v"].dtype), s


def _delta_step(st):
    """One token: s = e^g s; s += k (beta (v - k^T s))^T; o = scale s^T q."""
    c = st["case"]
    share = c["heads"] // c["qk_heads"]
    q, k = (_unit(st[n].float()).repeat_interleave(share, 1)[..., None] for n in "qk")
    s = st["state"] * st["g"].exp()[..., None, None]
    u = st["beta"][..., None] * (st["v"].float() - (s * k).sum(-2))
    s = s + k * u[..., None, :]
    o = (s * q).sum(-2) * c["d_k"] ** -0.5
    st["state"].copy_(s)
    return o.to(st["v"].dtype), st["state"]


def _normed(x, kind, w):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    return x if w is None else x * w.float()


def _norm(st):
    """r = x + 0.8 act(gate) norm(y); h = norm(r) (1 + scale) + shift, the vectors of each row's sample."""
    c = st["case"]
    s = torch.searchsorted(st["offsets"][1:].long(), torch.arange(c["rows"], device="cuda"), right=True)
    gate, scale, shift = (st["mod"][:, i].float() for i in range(3))
    gate = gate.tanh() if c["act"] == "tanh" else gate
    r = st["x"].float() + 0.8 * gate[s] * _normed(st["y"].float(), c["post"], st["post_w"])
    h = _normed(r, c["pre"], st["pre_w"]) * (1 + scale[s]) + shift[s]
    return r.to(st["x"].dtype), h.to(st["x"].dtype)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "attention":
        lq, lk = _attention_lengths(c)
        if c["causal"]:  # query i sees max(0, i + lk - lq + 1) keys
            pairs = sum(sum(max(0, i + b - a + 1) for i in range(a)) for a, b in zip(lq, lk))
        else:
            pairs = sum(a * b for a, b in zip(lq, lk))
        return {"bytes": e * c["d"] * (2 * sum(lq) * c["heads"] + 2 * sum(lk) * c["kv_heads"]),
                "flops": 4 * c["d"] * c["heads"] * pairs}
    if c["op"] in ("delta", "delta_step"):
        rows = sum(_lengths(c["lens"], c["nseq"], c["min_t"], c["max_t"])) if c["op"] == "delta" else c["nseq"]
        states = 4 * c["nseq"] * c["heads"] * c["d_k"] * c["d_v"] * (2 if c.get("state", True) else 1)
        return {"bytes": rows * (2 * e * c["qk_heads"] * c["d_k"] + 2 * e * c["heads"] * c["d_v"] + 8 * c["heads"]) + states,
                "flops": 6 * rows * c["heads"] * c["d_k"] * c["d_v"]}
    return {"bytes": 4 * e * c["rows"] * c["C"] + 3 * e * c["samples"] * c["C"], "flops": 16 * c["rows"] * c["C"]}


# ---------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "attention":
        lq, lk = _attention_lengths(c)
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        share = c["heads"] // c["kv_heads"]
        for s, (a, b) in enumerate(zip(lq, lk)):
            q0, k0 = int(st["q_offsets"][s]), int(st["k_offsets"][s])
            seen = torch.ones(a, b, dtype=torch.bool, device="cuda")
            if c["causal"]:
                seen = seen.tril(b - a)
            for h in range(c["heads"]):
                q = st["q"][q0:q0 + a, h].double()
                k, v = (st[n][k0:k0 + b, h // share].double() for n in "kv")
                x = torch.where(seen, q @ k.T / math.sqrt(c["d"]), -math.inf)
                out[q0:q0 + a, h] = torch.nan_to_num(torch.softmax(x, -1), nan=0.0) @ v
        return out
    if c["op"] in ("delta", "delta_step"):
        step = c["op"] == "delta_step"
        share = c["heads"] // c["qk_heads"]
        q, k = ((t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt()).repeat_interleave(share, 1)
                for t in (st["q"].double(), st["k"].double()))
        v, alpha, beta = st["v"].double(), st["g"].double().exp(), st["beta"].double()
        n = c["nseq"]
        lengths = [1] * n if step else _lengths(c["lens"], n, c["min_t"], c["max_t"])
        begin = _offsets(lengths)
        state = torch.zeros(n, c["heads"], c["d_k"], c["d_v"], dtype=torch.float64, device="cuda")
        if st["state"] is not None:
            state += st["state"].double()
        out = torch.zeros(v.shape, dtype=torch.float64, device="cuda")
        for t in range(max(lengths)):  # token by token, every sequence that still has one
            live = [i for i in range(n) if t < lengths[i]]
            i = torch.tensor(live, device="cuda")
            r = torch.tensor([begin[j] + t for j in live], device="cuda")
            s = alpha[r][:, :, None, None] * state[i]
            u = beta[r][:, :, None] * (v[r] - torch.einsum("nhk,nhkv->nhv", k[r], s))
            s = s + torch.einsum("nhk,nhv->nhkv", k[r], u)
            out[r] = torch.einsum("nhk,nhkv->nhv", q[r], s) / math.sqrt(c["d_k"])
            state[i] = s
        return out, state

    def norm(x, kind, w):
        if kind == "none":
            return x
        mean = x.mean(-1, keepdim=True) if kind == "layer" else 0.0
        var = ((x - mean) ** 2).mean(-1, keepdim=True)
        x = (x - mean) / torch.sqrt(var + 1e-6)
        return x if w is None else x * w.double()

    at = st["offsets"].tolist()
    x, y, m = st["x"].double(), st["y"].double(), st["mod"].double()
    r, h = torch.empty_like(x), torch.empty_like(x)
    for i in range(c["samples"]):
        rows = slice(at[i], at[i + 1])
        gate = torch.tanh(m[i, 0]) if c["act"] == "tanh" else m[i, 0]
        r[rows] = x[rows] + 0.8 * gate * norm(y[rows], c["post"], st["post_w"])
        h[rows] = norm(r[rows], c["pre"], st["pre_w"]) * (1 + m[i, 1]) + m[i, 2]
    return r, h
