"""Measured calls of the decayed linear attention, the rotary positions and the layer norm.

The three are the parts of one attention layer without a softmax: q and k are turned by their
positions, the decayed linear attention mixes the values, and its unnormalized outputs go
through a layer norm.

Operators and their plain forms (per head h with decay g = exp(log_decay[h])):

  prefill  o_t = scale (g^(t+1) q_t S_0 + sum_{s<=t} g^(t-s) (q_t . k_s) v_s) over packed
           sequences, and the state S_T = g^T S_0 + sum_s g^(T-1-s) k_s v_s^T
  decode   S <- g S + k v^T, o = scale q S for one token of every sequence, S in place
  train    o as in prefill (no state) and the gradients of sum(dO * o)
  rotary   the pairs (a, b) of the first `rot` coordinates become
           m (a cos x - b sin x), m (a sin x + b cos x), x = position * rate; the others are copied
  rotary_grad  the gradient of the same: x -> -x
  norm     y = (x - mean) / sqrt(var + eps) * w + b over the last axis
  norm_train   the same and the gradients of sum(dy * y)
"""

import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
C = 128                                              # rows of a plain form's block
EPS = 1e-5


def listed():
    bf = "bf16"
    return [
        # one new token of one sequence of the 340M layer's 16 heads of width 64: pure latency
        dict(name="decay_decode_b1", kind="decode", B=1, H=16, dk=64, dv=64, dtype=bf),
        # one new token for a serving batch of 512 sequences: the state is streamed
        dict(name="decay_decode_b512", kind="decode", B=512, H=16, dk=64, dv=64, dtype=bf),
        # a small packed batch of prompts, one of them empty, that continue cached states
        dict(name="decay_prefill_packed", kind="prefill", lengths="1,0,77,512,130,1303", H=16,
             dk=64, dv=64, dtype=bf, initial=True),
        # one long prompt
        dict(name="decay_prefill_131k", kind="prefill", lengths="131072", H=16, dk=64, dv=64,
             dtype=bf, initial=False),
        # four prompts of 16k tokens with wide heads
        dict(name="decay_prefill_wide", kind="prefill", lengths="16384,16384,16384,16384", H=16,
             dk=128, dv=128, dtype=bf, initial=False),
        # the attention of a training step at 8 x 4096 tokens
        dict(name="decay_train_4k", kind="train", B=8, T=4096, H=16, dk=64, dv=64, dtype=bf),
        # a small training step in fp32 with odd sizes
        dict(name="decay_train_fp32", kind="train", B=2, T=1001, H=3, dk=40, dv=72, dtype="fp32"),
        # q and k of one new token for each of 512 sequences, at far positions
        dict(name="rotary_decode", kind="rotary", B=512, T=1, H=16, Hk=16, D=64, rot=64, dtype=bf,
             interleaved=False, far=131072, scaling="parts"),
        # q and k of one long prompt, positions scaled past the trained length
        dict(name="rotary_prompt_131k", kind="rotary", B=1, T=131072, H=16, Hk=16, D=64, rot=64,
             dtype=bf, interleaved=False, far=0, scaling="parts"),
        # the gradient for neighbouring pairs in a part of the head, fp32, fewer key heads
        dict(name="rotary_grad_part", kind="rotary_grad", B=2, T=1777, H=12, Hk=4, D=80, rot=48,
             dtype="fp32", interleaved=True, far=0, scaling="none"),
        # the outputs of one decoded token for 512 sequences, all heads together
        dict(name="norm_decode", kind="norm", rows=512, N=1024, dtype=bf),
        # the outputs of a training step's 8 x 4096 tokens, forward and backward
        dict(name="norm_train_32k", kind="norm_train", rows=32768, N=1024, dtype=bf),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "prefill", "prefill", "train", "rotary", "rotary_grad", "norm",
                       "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind in ("norm", "norm_train"):
        N = _log(rng, 8, 8192)
        return dict(kind=kind, rows=_log(rng, 1, max(1, min(65536, (1 << 25) // N))), N=N,
                    dtype=dtype)
    H = _log(rng, 1, 32)
    if kind in ("rotary", "rotary_grad"):
        D = 8 * rng.randint(2, 16)
        return dict(kind=kind, B=(B := _log(rng, 1, 64)), T=_log(rng, 1, max(1, (1 << 19) // (B * H))),
                    H=H, Hk=rng.choice([h for h in range(1, H + 1) if H % h == 0]), D=D,
                    rot=rng.choice([D, D, 2 * rng.randint(1, D // 2)]), dtype=dtype,
                    interleaved=rng.random() < 0.5, far=rng.choice([0, 1000, 500000]),
                    scaling=rng.choice(["none", "linear", "parts"]))
    dk, dv = 8 * rng.randint(2, 16), 8 * rng.randint(2, 16)
    if kind == "decode":
        return dict(kind=kind, B=_log(rng, 1, max(1, (1 << 25) // (H * dk * dv))), H=H, dk=dk, dv=dv,
                    dtype=dtype)
    if kind == "train":
        B = _log(rng, 1, 8)
        return dict(kind=kind, B=B, T=_log(rng, 1, (1 << 18) // (B * H)), H=H, dk=dk, dv=dv, dtype=dtype)
    n = _log(rng, 1, 40)
    lengths = [rng.choice([0, 1, 64]) if rng.random() < 0.2 else _log(rng, 2, max(3, (1 << 19) // (n * H)))
               for _ in range(n)]
    lengths[rng.randrange(n)] = _log(rng, 2, 4096)
    return dict(kind=kind, lengths=",".join(map(str, lengths)), H=H, dk=dk, dv=dv, dtype=dtype,
                initial=rng.random() < 0.5)


def _rates(case):
    """Radians a token of each pair, fp64, and the magnitude: rotary frequencies of base 10000, for 8
    times the trained length either slowed down alike or, by parts, the slower turning pairs only."""
    rot = case["rot"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["scaling"] == "none":
        return f, 1.0
    if case["scaling"] == "linear":
        return f / 8, 1.0
    turns = 16384 * f / (2 * math.pi)                # over the trained length
    keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
    return f / 8 * (1 - keep) + f * keep, 0.1 * math.log(8.0) + 1


def _blocks(lengths):
    """Rows of the plain form's blocks of C tokens (the row behind the last where a block ends
    early), each block's sequence, first position, and length."""
    rows, seq, pos, size, at, total = [], [], [], [], 0, sum(lengths)
    for i, n in enumerate(lengths):
        for p in range(0, n, C):
            m = min(C, n - p)
            rows += [at + p + j if j < m else total for j in range(C)]
            seq.append(i), pos.append(p), size.append(m)
        at += n
    return [torch.tensor(x, dtype=torch.int64) for x in (rows, seq, pos, size)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    kind, dtype = case["kind"], BF16 if case["dtype"] == "bf16" else F32

    def normal(*shape, to=dtype):
        return torch.randn(*shape, generator=g, device=dev).to(to)

    s = dict(kind=kind, case=case)
    if kind in ("norm", "norm_train"):
        rows, N = case["rows"], case["N"]
        s.update(x=normal(rows, N) + 0.5, w=normal(N, to=F32) * 0.1 + 1, b=normal(N, to=F32) * 0.1)
        if kind == "norm_train":
            s["dy"] = normal(rows, N)
        return s
    H = case["H"]
    if kind in ("rotary", "rotary_grad"):
        B, T, D = case["B"], case["T"], case["D"]
        rates, magnitude = _rates(case)
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device=dev)
        s.update(q=normal(B, T, H, D), k=normal(B, T, case["Hk"], D), rates=rates.to(dev),
                 magnitude=magnitude, positions=start + torch.arange(T, device=dev))
        return s
    dk, dv = case["dk"], case["dv"]
    # decays from 1 - 2^-3 to 1 - 2^-10 over the heads, as of layers with windows of 8 to 1000 tokens
    x = torch.arange(H, dtype=torch.float64) / max(1, H - 1)
    s.update(log_decay=torch.log1p(-(2.0 ** -(3 + 7 * x))).float().to(dev), scale=dk ** -0.5)
    if kind == "decode":
        B = case["B"]
        s.update(q=normal(B, 1, H, dk), k=normal(B, 1, H, dk), v=normal(B, 1, H, dv),
                 state=normal(B, H, dk, dv, to=F32) * 4)
        return s
    lengths = [case["T"]] * case["B"] if kind == "train" else [int(n) for n in case["lengths"].split(",")]
    B, T = (case["B"], case["T"]) if kind == "train" else (1, sum(lengths))
    rows, seq, pos, size = (x.to(dev) for x in _blocks(lengths))
    n = torch.tensor(lengths, dtype=torch.int64, device=dev)
    s.update(q=normal(B, T, H, dk), k=normal(B, T, H, dk), v=normal(B, T, H, dv),
             rows=rows, seq=seq, pos=pos, size=size, n=n, initial=None)
    if kind == "train":
        s["dO"] = normal(B, T, H, dv)
    else:
        s["cu"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).int()
        if case["initial"]:
            s["initial"] = normal(len(lengths), H, dk, dv, to=F32) * 4
    return s


# ---- plain forms -------------------------------------------------------------------------

def _plain_decay(s, q, k, v, initial):
    """fp32 q, k, v [tokens][H][d] -> o [tokens][H][dv] and the states after the last tokens, by blocks
    of C tokens; every power of the decay is taken in 64 bits."""
    H, NB, ld = q.shape[1], s["seq"].numel(), s["log_decay"].double()[:, None, None]
    i = torch.arange(C, device=q.device)

    def blocked(x):                                  # -> [H][NB][C][d], zeros behind a sequence
        x = torch.cat([x, x.new_zeros(1, *x.shape[1:])])
        return x.index_select(0, s["rows"]).view(NB, C, H, -1).permute(2, 0, 1, 3).contiguous()

    def power(e, keep):                              # g^e where keep, else 0
        return torch.exp(ld * e.double().clamp(min=0)).where(keep, 0.0).float()

    Q, K, V = blocked(q), blocked(k), blocked(v)
    seq, pos, size, n = s["seq"], s["pos"], s["size"], s["n"]
    inside = power(i[:, None] - i, i[:, None] >= i)                              # [H][C][C]
    o = torch.matmul(torch.matmul(Q, K.transpose(-1, -2).contiguous()) * inside[:, None], V)
    left = size[:, None] - 1 - i                                                 # tokens of the block behind
    sums = torch.matmul((K * power(left, left >= 0)[..., None]).transpose(-1, -2).contiguous(), V)
    flat = sums.flatten(2)                                                       # [H][NB][dk dv]
    gap = pos[:, None] - pos - size
    entry = torch.matmul(power(gap, (seq[:, None] == seq) & (gap >= 0)), flat)
    rest = n[:, None] - pos - size
    final = torch.matmul(power(rest, torch.arange(n.numel(), device=q.device)[:, None] == seq), flat)
    if initial is not None:
        first = initial.permute(1, 0, 2, 3).flatten(2)                           # [H][N][dk dv]
        entry = entry + first[:, seq] * power(pos[:, None], pos[:, None] >= 0)
        final = final + first * power(n[:, None], n[:, None] >= 0)
    step = power(i[:, None] + 1, i[:, None] >= 0)                                # [H][C][1]
    o = (o + torch.matmul(Q * step[:, None], entry.view_as(sums))) * s["scale"]
    out = q.new_zeros(q.shape[0] + 1, H, v.shape[2])
    out = out.index_copy(0, s["rows"], o.permute(1, 2, 0, 3).reshape(-1, H, v.shape[2]))[:-1]
    return out, final.view(H, n.numel(), q.shape[2], v.shape[2]).permute(1, 0, 2, 3).contiguous()


def _plain_rotary(x, s, sign):
    case, rot = s["case"], s["case"]["rot"]
    angle = s["positions"].double()[..., None] * s["rates"]                      # [B][T][rot / 2]
    m = s["magnitude"]
    cos, sin = (m * angle.cos()).float()[:, :, None], (m * sign * angle.sin()).float()[:, :, None]
    y = x.float()
    turned, rest = y[..., :rot], y[..., rot:]
    if case["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = turned[..., : rot // 2], turned[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, rest], -1).to(x.dtype)


def _plain_norm(x, w, b):
    x = x.float()
    d = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    return d * r, r, (d * r) * w + b


def run(s):
    kind = s["kind"]
    if own:
        return _run_own(s, kind)
    if kind in ("norm", "norm_train"):
        hat, r, y = _plain_norm(s["x"], s["w"], s["b"])
        y = y.to(s["x"].dtype)
        if kind == "norm":
            return y
        dy = s["dy"].float()
        t = dy * s["w"]
        dx = (t - t.mean(-1, keepdim=True) - hat * (t * hat).mean(-1, keepdim=True)) * r
        return y, dx.to(y.dtype), (dy * hat).sum(0), dy.sum(0)
    if kind in ("rotary", "rotary_grad"):
        sign = 1.0 if kind == "rotary" else -1.0
        return _plain_rotary(s["q"], s, sign), _plain_rotary(s["k"], s, sign)
    if kind == "decode":
        q, k, v = (s[x].float()[:, 0] for x in "qkv")
        s["state"].mul_(torch.exp(s["log_decay"].double()).float()[:, None, None])
        s["state"].add_(k[..., None] * v[..., None, :])
        o = (q[..., None] * s["state"]).sum(-2) * s["scale"]
        return o[:, None].to(s["q"].dtype), s["state"]
    q, k, v = (s[x].float().flatten(0, 1) for x in "qkv")
    if kind == "prefill":
        o, final = _plain_decay(s, q, k, v, s["initial"])
        return o.view_as(s["v"]).to(s["q"].dtype), final
    leaves = [x.requires_grad_() for x in (q.clone(), k.clone(), v.clone())]
    o, _ = _plain_decay(s, *leaves, None)
    grads = torch.autograd.grad(o, leaves, s["dO"].float().flatten(0, 1))
    back = lambda x, like: x.detach().view_as(like).to(like.dtype)  # noqa: E731
    return back(o, s["v"]), back(grads[0], s["q"]), back(grads[1], s["k"]), back(grads[2], s["v"])


def _run_own(s, kind):
    import kernelized_psd_feature_amd as kata

    if kind == "norm":
        return kata.fwd_layer_norm(s["x"], s["w"], s["b"], eps=EPS)
    if kind == "norm_train":
        y, mean, rstd = kata.fwd_layer_norm(s["x"], s["w"], s["b"], eps=EPS, return_stats=True)
        return (y, *kata.bwd_layer_norm(s["dy"], s["x"], s["w"], mean, rstd))
    if kind in ("rotary", "rotary_grad"):
        return kata.rotary(s["q"], s["k"], s["rates"], positions=s["positions"],
                           interleaved=s["case"]["interleaved"], magnitude=s["magnitude"],
                           inverse=kind == "rotary_grad")
    if kind == "decode":
        return kata.decode_decay(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"]), s["state"]
    if kind == "prefill":
        return kata.fwd_decay(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                              initial_state=s["initial"], cu_seqlens=s["cu"], return_state=True)
    o = kata.fwd_decay(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"])
    return (o, *kata.bwd_decay(s["q"], s["k"], s["v"], s["dO"], s["log_decay"], scale=s["scale"])[:3])


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    kind, e = case["kind"], 2 if case["dtype"] == "bf16" else 4
    if kind in ("norm", "norm_train"):
        rows, N = case["rows"], case["N"]
        if kind == "norm":
            return {"bytes": 2 * rows * N * e + 8 * N, "flops": 8 * rows * N}
        return {"bytes": 4 * rows * N * e + 16 * N, "flops": 20 * rows * N}
    H = case["H"]
    if kind in ("rotary", "rotary_grad"):
        tokens = case["B"] * case["T"]
        heads = H + case["Hk"]
        return {"bytes": 2 * tokens * heads * case["D"] * e + 8 * tokens + 4 * case["rot"],
                "flops": 3 * tokens * heads * case["rot"]}
    dk, dv = case["dk"], case["dv"]
    if kind == "decode":
        B = case["B"]
        return {"bytes": B * H * (8 * dk * dv + (2 * dk + 2 * dv) * e) + 4 * H, "flops": 5 * B * H * dk * dv}
    if kind == "train":
        # q, k, v, dO in; o, dq, dk, dv out; the recurrences of o, dq, dk and dv
        rows = case["B"] * case["T"] * H
        return {"bytes": rows * (4 * dk + 4 * dv) * e + 4 * H, "flops": 16 * rows * dk * dv}
    lengths = [int(n) for n in case["lengths"].split(",")]
    states = len(lengths) * H * dk * dv * 4
    return {"bytes": sum(lengths) * H * (2 * dk + 2 * dv) * e + states * (2 if case["initial"] else 1) + 4 * H,
            "flops": 4 * sum(lengths) * H * dk * dv}


# ---- the definitions in 64 bits ------------------------------------------------------------

def _pairs(a, b, c, ld, later):
    """sum over pairs, by the definition: row t of a [H][n][d], rows s of b and c, weight
    g^|t-s| for s <= t, or for s >= t where `later`."""
    n, step = a.shape[1], 2048
    out = a.new_zeros(a.shape[0], n, c.shape[2])
    for t0 in range(0, n, step):
        t = torch.arange(t0, min(n, t0 + step), device=a.device)
        for s0 in range(t0 if later else 0, n if later else t0 + 1, step):
            u = torch.arange(s0, min(n, s0 + step), device=a.device)
            far = (u - t[:, None] if later else t[:, None] - u).double()
            w = torch.exp(ld[:, None, None] * far.clamp(min=0)) * (far >= 0)
            w *= torch.bmm(a[:, t0:t0 + step], b[:, s0:s0 + step].transpose(1, 2).contiguous())
            out[:, t0:t0 + step] += torch.bmm(w, c[:, s0:s0 + step])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("norm", "norm_train"):
        x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
        mean = x.sum(-1, keepdim=True) / case["N"]
        sd = torch.sqrt(((x - mean) ** 2).sum(-1, keepdim=True) / case["N"] + EPS)
        hat = (x - mean) / sd
        if kind == "norm":
            return hat * w + b
        dy = s["dy"].double()
        n, wdy = case["N"], s["dy"].double() * w
        dx = (n * wdy - wdy.sum(-1, keepdim=True) - hat * (wdy * hat).sum(-1, keepdim=True)) / (n * sd)
        return hat * w + b, dx, (dy * hat).sum(0), dy.sum(0)
    if kind in ("rotary", "rotary_grad"):
        angle = s["positions"].double()[:, :, None, None] * s["rates"]
        z = torch.polar(torch.full_like(angle, s["magnitude"]), angle if kind == "rotary" else -angle)
        out = []
        for x in (s["q"].double(), s["k"].double()):
            rot, half = case["rot"], case["rot"] // 2
            a = slice(0, rot, 2) if case["interleaved"] else slice(0, half)
            b = slice(1, rot, 2) if case["interleaved"] else slice(half, rot)
            turned = torch.complex(x[..., a], x[..., b]) * z
            y = x.clone()
            y[..., a], y[..., b] = turned.real, turned.imag
            out.append(y)
        return tuple(out)
    ld, scale = s["log_decay"].double(), s["scale"]
    if kind == "decode":
        q, k, v = (s[x].double()[:, 0] for x in "qkv")
        state = s["state"].double() * torch.exp(ld)[:, None, None] + torch.einsum("bhi,bhj->bhij", k, v)
        return (torch.einsum("bhi,bhij->bhj", q, state) * scale)[:, None], state
    q, k, v = (s[x].double().transpose(1, 2) for x in "qkv")                     # [B][H][T][d]
    if kind == "train":
        dO = s["dO"].double().transpose(1, 2)
        if case["B"] * case["H"] * case["T"] ** 2 > 1 << 34:
            return None
        per = [(_pairs(q[b], k[b], v[b], ld, False), _pairs(dO[b], v[b], k[b], ld, False),
                _pairs(v[b], dO[b], q[b], ld, True), _pairs(k[b], q[b], dO[b], ld, True))
               for b in range(case["B"])]
        return tuple((torch.stack(x) * scale).transpose(1, 2) for x in zip(*per))
    outs, states, at = [], [], 0
    for i, n in enumerate(int(n) for n in case["lengths"].split(",")):
        Q, K, V = (x[0, :, at:at + n] for x in (q, k, v))
        at += n
        o = _pairs(Q, K, V, ld, False)
        t = torch.arange(n, device=o.device, dtype=torch.float64)
        state = torch.matmul((K * torch.exp(ld[:, None] * (n - 1 - t))[..., None]).transpose(1, 2).contiguous(), V)
        if s["initial"] is not None:
            first = s["initial"][i].double()
            o = o + torch.matmul(Q * torch.exp(ld[:, None] * (t + 1))[..., None], first)
            state = state + first * torch.exp(ld * n)[:, None, None]
        outs.append(o * scale), states.append(state)
    return torch.cat(outs, 1).transpose(0, 1)[None], torch.stack(states)
