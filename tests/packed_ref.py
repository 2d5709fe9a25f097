"""Plain 64-bit forms of the packed-sequence operators, with the error bounds
their tests use. Bounds count: half a step of the output type (2^-8 of the
value for bf16, 2^-24 for fp32), half a step for each operand a kernel may
round to bf16, and (n + c) 2^-24 of the sum of absolute terms for an fp32 sum of
n terms."""
import math

import pytest
import torch

U32 = 2.0 ** -24


@pytest.fixture(autouse=True)
def float32_default():
    """fp32 for tensors made without a type, whatever another test module has set."""
    was = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(was)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def attention(q, k, v, q_at, k_at, k_lens, causal, scale):
    """Returns (out, bound), fp64 [rows, heads, d]; rows in no sequence NaN in out."""
    H, K, d = q.shape[1], k.shape[1], q.shape[2]
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    bf = q.dtype == torch.bfloat16
    for s in range(len(q_at) - 1):
        a, b = q_at[s + 1] - q_at[s], (k_at[s + 1] - k_at[s]) if k_lens is None else k_lens[s]
        rq = slice(q_at[s], q_at[s + 1])
        Q = q[rq].double()
        Kk, V = k[k_at[s]:k_at[s] + b].double(), v[k_at[s]:k_at[s] + b].double()
        for h in range(H):
            x = scale * Q[:, h] @ Kk[:, h * K // H].T
            dot = scale * Q[:, h].abs() @ Kk[:, h * K // H].abs().T   # for the error of a score
            if causal:
                hidden = torch.ones(a, b, dtype=torch.bool, device=q.device).triu(b - a + 1)
                x, dot = x.masked_fill(hidden, -math.inf), dot.masked_fill(hidden, 0.0)
            if b == 0:
                out[rq, h] = 0.0
                continue
            m = x.amax(-1, keepdim=True)
            p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
            tot = p.sum(-1, keepdim=True)
            p = torch.where(tot > 0, p / tot, torch.zeros_like(p))
            Vh = V[:, h * K // H]
            o = p @ Vh
            pv = p @ Vh.abs()
            # score error e_s: fp32 sum of d products and the exponent's own rounding; a weight is off by 2 e_s
            # (itself and the sum it is divided by), the sums over the keys by their count
            e_s = (d + 4) * U32 * dot.amax(-1, keepdim=True) + 4 * U32 * (x.masked_fill(x == -math.inf, 0.0).abs().amax(-1, keepdim=True))
            rel = 2 * e_s + (2 * b + 16) * U32 + 2.0 ** -20 * bf
            # bf16: a weight rounded for the product (2^-8 of sum p|v|) and, where the divisor sums rounded weights, 2^-8 of o
            out[rq, h] = o
            bound[rq, h] = half_step(q.dtype) * o.abs() + (rel + bf * half_step(q.dtype)) * pv + bf * half_step(q.dtype) * o.abs()
    return out, bound + 1e-30


def delta_rule(q, k, v, g, beta, at, state, scale, norm, eps=1e-6):
    """Token by token. Returns (out, final states, bound of |out error|_2 per (row, head), bound of |state error|_F)."""
    Hq, H, dk, dv = q.shape[1], v.shape[1], q.shape[2], v.shape[2]
    n = len(at) - 1
    bf = q.dtype == torch.bfloat16
    qd, kd = q.double(), k.double()
    if norm:
        qd = qd / (qd.square().sum(-1, keepdim=True) + eps).sqrt()
        kd = kd / (kd.square().sum(-1, keepdim=True) + eps).sqrt()
    qd, kd = qd.repeat_interleave(H // Hq, 1), kd.repeat_interleave(H // Hq, 1)
    vd, bd = v.double(), beta.double()
    gd = g.double().clamp(min=-200.0)
    out = torch.full(v.shape, float("nan"), dtype=torch.float64, device=v.device)
    ob = torch.zeros(v.shape[:2], dtype=torch.float64, device=v.device)
    S = torch.zeros(n, H, dk, dv, dtype=torch.float64, device=v.device)
    if state is not None:
        S += state.double()
    E = torch.zeros(n, H, dtype=torch.float64, device=v.device)
    # one step's own error, relative to the state and value it handles: fp32 sums over d_k (and over a 64-token chunk);
    # bf16 inputs may run on operands split into two bf16 halves, 2^-16 of each of the three products in a row
    c = (dk + 64 + 16) * U32 + bf * 3 * 2.0 ** -16
    for s in range(n):
        us, before = [], []
        for t in range(at[s], at[s + 1]):
            a = gd[t].exp()
            kt, qt = kd[t], qd[t]
            S[s] = a[:, None, None] * S[s]
            u = bd[t][:, None] * (vd[t] - torch.einsum("hk,hkv->hv", kt, S[s]))
            kn, qn = kt.norm(dim=-1), qt.norm(dim=-1)
            size = S[s].flatten(1).norm(dim=1)
            # (I - beta k k^T) does not expand for |k| <= 1, 0 <= beta <= 1, the only case with a bound here
            E[s] = a * E[s] + c * (size + kn * bd[t] * (vd[t].norm(dim=-1) + kn * size))
            S[s] = S[s] + kt[:, :, None] * u[:, None, :]
            out[t] = scale * torch.einsum("hk,hkv->hv", qt, S[s])
            us.append(u.norm(dim=-1))
            before.append(size + E[s])
            ob[t] = half_step(q.dtype) * out[t].norm(dim=-1) + scale * qn * (E[s] + c * S[s].flatten(1).norm(dim=1))
        if bf and us:  # the products that give the output may take state, scores and values rounded to bf16
            r = slice(at[s], at[s + 1])
            G, un, n_t = gd[r].cumsum(0), torch.stack(us), len(us)          # [T, H]
            lag = torch.arange(n_t, device=v.device)[:, None] - torch.arange(n_t, device=v.device)
            near = ((lag >= 0) & (lag < 64))[None]                          # a chunk's tokens up to this one
            D = torch.where(near, G.T[:, :, None] - G.T[:, None, :], -math.inf).exp() * un.T[:, None, :]   # [H, t, j]
            qk = torch.einsum("thk,jhk->htj", qd[r], kd[r]).abs()
            qn = qd[r].norm(dim=-1)
            ob[r] += scale * 2.0 ** -8 * (qn * torch.stack(before) + 2.1 * (D * qk).sum(-1).T)
            # a chunk's first state decays to `size` in the bound above only if no value left it since: add what the
            # chunk's own tokens may have taken out
            ob[r] += scale * 2.0 ** -8 * qn * (D * kd[r].norm(dim=-1).T[:, None, :]).sum(-1).T
    return out, S, ob + 1e-30, E + 1e-30


def block_norm(x, y, sample, post, pre, act, eps, rho, vec):
    """vec: dict of the optional vectors (gate, scale, shift per sample). Returns (r, h, bound r, bound h)."""
    u = half_step(x.dtype)
    C = x.shape[1]
    acc = (C + 32) * U32   # fp32 sums over a row

    def get(n):
        return None if vec.get(n) is None else vec[n].double()

    def norm(z, e, kind, w, b):
        """z and a bound e of its error -> the normed row and the bound of its error."""
        if kind == "none":
            return z, e
        mean = z.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(z[:, :1])
        zc = z - mean
        var = zc.square().mean(-1, keepdim=True)
        rstd = 1 / torch.sqrt(var + eps)
        em = acc * z.abs().mean(-1, keepdim=True) * (kind == "layer") + e.mean(-1, keepdim=True) + U32 * z.abs()
        ez = e + em
        # relative error of rstd: half of var's
        ev = 0.5 * (2 * (zc.abs() * ez).mean(-1, keepdim=True) * rstd ** 2 + acc) + 8 * U32
        n = zc * rstd
        en = ez * rstd + n.abs() * ev
        if w is not None:
            n, en = n * w, en * w.abs()
        if b is not None:
            n = n + b
        return n, en + 4 * U32 * n.abs()

    xd = x.double()
    r, er = xd, torch.zeros_like(xd)
    if y is not None:
        n, en = norm(y.double(), torch.zeros_like(xd), post, get("post_w"), get("post_b"))
        gate = None
        for key in ("gate0", "gate"):
            if get(key) is not None:
                gv = get(key)[sample] if key == "gate" else get(key)[None]
                gate = gv if gate is None else gate + gv
        gate = torch.ones_like(xd[:1]) if gate is None else (gate.tanh() if act == "tanh" else gate)
        r = xd + rho * gate * n
        er = abs(rho) * (gate.abs() * en + 16 * U32 * (gate.abs() + 1e-3) * n.abs()) + 2 * U32 * r.abs()
    n, en = norm(r, er, pre, get("pre_w"), get("pre_b"))
    sc, sh = torch.ones_like(xd[:1]), torch.zeros_like(xd[:1])
    for key in ("scale0", "scale"):
        if get(key) is not None:
            sc = sc + (get(key)[sample] if key == "scale" else get(key)[None])
    for key in ("shift0", "shift"):
        if get(key) is not None:
            sh = sh + (get(key)[sample] if key == "shift" else get(key)[None])
    h = n * sc + sh
    eh = en * sc.abs() + 4 * U32 * (n.abs() * (1 + sc.abs()) + sh.abs())
    return r, h, er + u * r.abs() + 1e-30, eh + u * (h.abs() + eh) + 1e-30
