"""The operators of the linear attention layer, as cases to time and compare.

Two operators, in each direction that a user runs them:

* ``rope``: the norm of every query and key head with the position rotation in the same
  pass (forward and backward);
* ``linattn``: causal linear attention with one decay per head, over prompts (forward and
  backward) and for single tokens (the decode step).

With ``own`` false, ``run`` computes a case from elementary torch operations in 32 bits,
rounded once at the end.  With ``own`` true it calls the library.
"""
import functools
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def _rope(name, B, T, Hq, Hk, D, rot, dtype, *, backward=False, interleaved=False, positions=False,
          ragged=0, fused=True):
    return dict(name=name, op="rope_backward" if backward else "rope", B=B, T=T, Hq=Hq, Hk=Hk, D=D, rot=rot,
                dtype=dtype, interleaved=interleaved, positions=positions, ragged=ragged, fused=fused)


def _attn(name, B, T, H, D, dtype, *, backward=False, ragged=0, resumed=False, fused=False):
    return dict(name=name, op="linattn_backward" if backward else "linattn", B=B, T=T, H=H, D=D, dtype=dtype,
                ragged=ragged, resumed=resumed, fused=fused)


def _decode(name, B, H, D, dtype, *, slots=0):
    return dict(name=name, op="decode", B=B, H=H, D=D, dtype=dtype, slots=slots)


def listed():
    return [
        # one token of eight sequences, each at its own position: a serving step, all latency
        _rope("rope decode 8x1", 8, 1, 16, 16, 128, 128, "bf16", positions=True),
        # the LM shape's queries and keys, read out of the fused projection
        _rope("rope lm 8x4096", 8, 4096, 16, 16, 128, 128, "bf16"),
        # its gradient, with four key heads to sixteen query heads
        _rope("rope back lm 8x4096 16/4", 8, 4096, 16, 4, 128, 128, "bf16", backward=True),
        # the gradient of the recommendation shape in fp32: short ragged histories, half the head rotated
        _rope("rope back rec 512x200 f32", 512, 200, 2, 2, 32, 16, "f32", backward=True, interleaved=True, ragged=20),
        # the LM shape's prompt: heads enough to fill the card
        _attn("linattn lm 8x4096", 8, 4096, 16, 128, "bf16", fused=True),
        # one long prompt: few heads, a long axis
        _attn("linattn long 65536", 1, 65536, 32, 128, "bf16"),
        # the recommendation shape: many short ragged sequences of small heads
        _attn("linattn rec 512x200", 512, 200, 2, 32, "bf16", ragged=20),
        # fp32 at the sweep shape, resumed from a state, an odd length
        _attn("linattn f32 4x1021", 4, 1021, 4, 64, "f32", resumed=True),
        # training at the LM shape
        _attn("linattn back lm 8x4096", 8, 4096, 16, 128, "bf16", backward=True),
        # training on segments of a longer text: a state comes in and its gradient goes out
        _attn("linattn back 4x1000 d64", 4, 1000, 4, 64, "bf16", backward=True, resumed=True),
        # single tokens of eight sequences: latency
        _decode("decode 8 d128", 8, 16, 128, "bf16"),
        # single tokens of a large batch whose states lie in a pool of slots
        _decode("decode 256 d128 slots", 256, 16, 128, "bf16", slots=288),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "rope_backward", "linattn", "linattn", "linattn_backward", "decode"])
    D = rng.choice([16, 32, 64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "decode":
        H = _spread(rng, 1, 32)
        B = _spread(rng, 1, min(1024, max(1, (1 << 26) // (H * D * D))))
        return {k: v for k, v in _decode("", B, H, D, dtype, slots=rng.choice([0, B + B // 8 + 1])).items() if k != "name"}
    H = _spread(rng, 1, 32)
    # at most 2^28 elements of q in bf16 (the long prompt's size), 2^25 for training and in fp32
    most = (1 << 28) if op in ("rope", "linattn") and dtype == "bf16" else (1 << 25)
    tokens = max(1, most // (H * D))
    T = _spread(rng, 1, min(tokens, 65536))
    B = _spread(rng, 1, max(1, min(tokens // T, 512)))
    ragged = rng.choice([0, 0, 1]) * max(1, T // 8)
    if op in ("rope", "rope_backward"):
        Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0])
        rot = rng.choice([D, D, D // 2])
        c = _rope("", B, T, H, Hk, D, rot, dtype, backward=op == "rope_backward", interleaved=rng.random() < 0.4,
                  positions=rng.random() < 0.4, ragged=ragged, fused=rng.random() < 0.6)
    else:
        c = _attn("", B, T, H, D, dtype, backward=op == "linattn_backward", ragged=ragged,
                  resumed=rng.random() < 0.4, fused=rng.random() < 0.4)
    return {k: v for k, v in c.items() if k != "name"}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    def unit(*shape):
        x = normal(*shape)
        return x.mul_(torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS)).to(dt)

    B, D = case["B"], case["D"]
    s = dict(case)
    if case["op"] == "decode":
        H, N = case["H"], max(case["slots"], case["B"])
        s.update(q=unit(B, H, D), k=unit(B, H, D), v=normal(B, H, D).to(dt), state=normal(N, H, D, D) * 2, slot=None)
        if case["slots"]:
            s["slot"] = torch.randperm(N, generator=g, device="cuda")[:B].to(torch.int32)
        s.update(log_decay=_slopes(case["H"], g), scale=1.0)
        return s
    T = case["T"]
    s["lens"] = None
    if case["ragged"]:
        s["lens"] = torch.randint(case["ragged"], T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    if case["op"] in ("rope", "rope_backward"):
        Hq, Hk, rot = case["Hq"], case["Hk"], case["rot"]
        if case["fused"]:   # one projection of queries, keys and values for each token
            x = normal(B, T, Hq + 2 * Hk, D, dtype=dt)
            s["q"], s["k"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
        else:
            s["q"], s["k"] = normal(B, T, Hq, D, dtype=dt), normal(B, T, Hk, D, dtype=dt)
        s["qw"], s["kw"] = 1 + 0.2 * normal(D), 1 + 0.2 * normal(D)
        P = T if not case["positions"] else T + 4096
        freq = torch.exp(torch.arange(rot // 2, device="cuda", dtype=torch.float64) * (-2 * math.log(10000.0) / rot))
        angle = torch.arange(P, device="cuda", dtype=torch.float64)[:, None] * freq
        s["table"] = torch.cat([angle.cos(), angle.sin()], -1).to(torch.float32)
        s["pos"] = None
        if case["positions"]:
            first = torch.randint(0, 4097, (B, 1), generator=g, device="cuda", dtype=torch.int32)
            s["pos"] = (first + torch.arange(T, device="cuda", dtype=torch.int32)).contiguous()
        s["scales"] = (D ** -0.5, 1.0)
        if case["op"] == "rope_backward":
            s["dq"], s["dk"] = normal(B, T, Hq, D, dtype=dt), normal(B, T, Hk, D, dtype=dt)
        return s
    H = case["H"]
    s["q"], s["k"] = unit(B, T, H, D), unit(B, T, H, D)
    s["v"] = normal(B, T, 3, H, D, dtype=dt)[:, :, 2] if case["fused"] else normal(B, T, H, D, dtype=dt)
    s.update(log_decay=_slopes(H, g), scale=1.0, state=normal(B, H, D, D) if case["resumed"] else None)
    if case["op"] == "linattn_backward":
        s["d_out"] = normal(B, T, H, D, dtype=dt)
        s["d_state"] = normal(B, H, D, D) if case["resumed"] else None
    return s


def _slopes(H, g):
    """One decay a head, from a few tokens' memory to a few thousand's: exp(-slope)."""
    at = (torch.arange(H, device="cuda") + torch.rand(H, generator=g, device="cuda")) / H
    return -torch.exp(math.log(0.5) + at * math.log(2.0 ** -11))


# ---- the plain forms ----

def _live(T, lens, B, device):
    """[B,T]: the tokens that are there."""
    t = torch.arange(T, device=device)
    return (t < lens[:, None]) if lens is not None else torch.ones(B, T, dtype=torch.bool, device=device)


def _there(s):
    """The tokens that have a position, and that position."""
    B, T = s["B"], s["T"]
    live = _live(T, s["lens"], B, s["q"].device)
    pos = s["pos"].long() if s["pos"] is not None else torch.arange(T, device=s["q"].device).expand(B, T)
    live = live & (pos >= 0) & (pos < s["table"].shape[0])
    return live, pos.clamp(0, s["table"].shape[0] - 1)


def _turn(y, table, interleaved, back=False):
    """The rotation of y [B,T,H,D] by table [B,T,1,rot] (cosines, then sines), or its inverse."""
    rot = table.shape[-1]
    c, z = table[..., :rot // 2], table[..., rot // 2:]
    z = -z if back else z
    x, rest = y[..., :rot], y[..., rot:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:])
    p, r = a * c - b * z, b * c + a * z
    x = torch.stack([p, r], -1).flatten(-2) if interleaved else torch.cat([p, r], -1)
    return torch.cat([x, rest], -1)


def _norm_turn(x, w, scale, s, live, table):
    x = torch.where(live, x.float(), 0.0)
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (w * scale)
    return torch.where(live, _turn(y, table, s["interleaved"]), 0.0).to(TYPES[s["dtype"]])


def _norm_turn_back(dy, x, w, scale, s, live, table):
    x, dy = torch.where(live, x.float(), 0.0), torch.where(live, dy.float(), 0.0)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    u, n = _turn(dy, table, s["interleaved"], back=True) * scale, x * r
    dw = (u * n).sum((0, 1, 2))
    u = u * w
    return (r * (u - n * (u * n).mean(-1, keepdim=True))).to(TYPES[s["dtype"]]), dw


def _decayed(x, y, z, ld):
    """sum over j <= i of exp((i - j) ld) (x_i . y_j) z_j for x, y, z [B,H,T,D]: within chunks, and
    between them through the chunks' sums of z y^T."""
    B, H, T, D = x.shape
    C = min(128, T)
    N = -(-T // C)
    x, y, z = (torch.nn.functional.pad(a, (0, 0, 0, N * C - T)).reshape(B, H, N, C, D) for a in (x, y, z))
    i = torch.arange(C, device=x.device)
    ld = ld[:, None, None]

    def powers(n):                       # exp(n ld), zero where n is negative
        return torch.where(n >= 0, torch.exp(n.clamp_min(0) * ld), 0.0)

    inside = (x @ y.transpose(-1, -2)) * powers(i[:, None] - i)[:, None] @ z
    sums = z.transpose(-1, -2) @ (y * powers((C - 1 - i)[:, None])[:, None])
    n = torch.arange(N, device=x.device)
    before = (powers(C * (n[:, None] - 1 - n)) @ sums.reshape(B, H, N, D * D)).reshape(B, H, N, D, D)
    before = (x * powers((i + 1)[:, None])[:, None]) @ before.transpose(-1, -2)
    return (inside + before).reshape(B, H, N * C, D)[:, :, :T]


def _heads_first(a, live):
    return torch.where(live, a.float(), 0.0).transpose(1, 2)


def _attn_plain(s):
    live = _live(s["T"], s["lens"], s["B"], s["q"].device)[:, :, None, None]
    q, k, v = (_heads_first(s[n], live) for n in ("q", "k", "v"))
    ld, t = s["log_decay"], torch.arange(s["T"], device=q.device)
    left = live.sum(1).reshape(-1, 1, 1) - 1 - t                                   # [B,1,T]: tokens that follow
    w = torch.where(left >= 0, torch.exp(left.clamp_min(0) * ld[:, None]), 0.0)
    o = _decayed(q, k, v, ld)
    state = v.transpose(-1, -2) @ (k * w[..., None])
    if s["state"] is not None:
        o = o + torch.exp((t + 1) * ld[:, None])[..., None] * (q @ s["state"].transpose(-1, -2))
        state = state + torch.exp(live.sum(1).reshape(-1, 1) * ld)[..., None, None] * s["state"]
    return (o * s["scale"]).transpose(1, 2).to(TYPES[s["dtype"]]).contiguous(), state


def _attn_plain_back(s):
    live = _live(s["T"], s["lens"], s["B"], s["q"].device)[:, :, None, None]
    q, k, v, do = (_heads_first(s[n], live) for n in ("q", "k", "v", "d_out"))
    do = do * s["scale"]
    ld, t = s["log_decay"], torch.arange(s["T"], device=q.device)
    dq = _decayed(do, v, k, ld)
    dk, dv = (_decayed(a.flip(2), b.flip(2), c.flip(2), ld).flip(2) for a, b, c in ((v, do, q), (k, q, do)))
    grown = torch.exp((t + 1) * ld[:, None])[..., None]
    got = {"initial_state": None}
    if s["state"] is not None:
        left = live.sum(1).reshape(-1, 1, 1) - 1 - t
        w = torch.where(left >= 0, torch.exp(left.clamp_min(0) * ld[:, None]), 0.0)[..., None]
        dq = dq + grown * (do @ s["state"])
        dk, dv = dk + w * (v @ s["d_state"]), dv + w * (k @ s["d_state"].transpose(-1, -2))
        got["initial_state"] = (do.transpose(-1, -2) @ (q * grown)
                                + torch.exp(live.sum(1).reshape(-1, 1) * ld)[..., None, None] * s["d_state"])
    dt = TYPES[s["dtype"]]
    got.update({n: a.transpose(1, 2).to(dt).contiguous() for n, a in (("q", dq), ("k", dk), ("v", dv))})
    return got


def _decode_plain(s):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    old = s["state"] if s["slot"] is None else s["state"][s["slot"].long()]
    new = torch.exp(s["log_decay"])[:, None, None] * old + v[..., None] * k[..., None, :]
    o = (new * q[..., None, :]).sum(-1) * s["scale"]
    if s["slot"] is None:
        s["state"].copy_(new)
    else:
        s["state"][s["slot"].long()] = new
    return o.to(TYPES[s["dtype"]]), s["state"]


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    if s["op"] == "decode":
        return _decode_plain(s)
    if s["op"] == "linattn":
        return _attn_plain(s)
    if s["op"] == "linattn_backward":
        return _attn_plain_back(s)
    live, pos = _there(s)
    live, table = live[:, :, None, None], s["table"][pos][:, :, None]
    if s["op"] == "rope":
        return (_norm_turn(s["q"], s["qw"], s["scales"][0], s, live, table),
                _norm_turn(s["k"], s["kw"], s["scales"][1], s, live, table))
    dq, dqw = _norm_turn_back(s["dq"], s["q"], s["qw"], s["scales"][0], s, live, table)
    dk, dkw = _norm_turn_back(s["dk"], s["k"], s["kw"], s["scales"][1], s, live, table)
    return {"q": dq, "k": dk, "q_weight": dqw, "k_weight": dkw}


@functools.cache
def _library():
    from linear_recurrent_sequence_causal_gb300 import linattn
    return linattn


def _run_own(s):
    linattn = _library()
    if s["op"] == "decode":
        out = linattn.prism_linattn_decode_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"],
                                                slots=s["slot"])
        return out, s["state"]
    if s["op"] == "linattn":
        return linattn.prism_linattn_forward(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                                             initial_state=s["state"], seq_lens=s["lens"])
    if s["op"] == "linattn_backward":
        return linattn.prism_linattn_backward(s["q"], s["k"], s["v"], s["log_decay"], s["d_out"], scale=s["scale"],
                                              initial_state=s["state"], d_final_state=s["d_state"],
                                              seq_lens=s["lens"])
    how = dict(q_weight=s["qw"], k_weight=s["kw"], q_scale=s["scales"][0], k_scale=s["scales"][1], eps=EPS,
               positions=s["pos"], seq_lens=s["lens"], interleaved=s["interleaved"])
    if s["op"] == "rope":
        return linattn.prism_qk_norm_rope(s["q"], s["k"], s["table"], **how)
    return linattn.prism_qk_norm_rope_backward(s["q"], s["k"], s["table"], s["dq"], s["dk"], **how)


# ---- what a pass cannot do without ----

def work(case):
    n = 2 if case["dtype"] == "bf16" else 4
    B, D = case["B"], case["D"]
    if case["op"] == "decode":
        H = case["H"]
        return {"bytes": B * H * (2 * D * D * 4 + 4 * D * n), "flops": B * H * 5 * D * D}
    T = case["T"]
    t = B * (T if not case["ragged"] else (case["ragged"] + T) / 2)   # tokens that are there, on average
    if case["op"] in ("rope", "rope_backward"):
        rows, table = case["Hq"] + case["Hk"], T * case["rot"] * 4
        if case["op"] == "rope":
            return {"bytes": (t + B * T) * rows * D * n + table, "flops": t * rows * D * 7}
        return {"bytes": (2 * t + B * T) * rows * D * n + table, "flops": t * rows * D * 16}
    H = case["H"]
    state = B * H * D * D * 4 * (2 if case["resumed"] else 1)
    # the recurrence itself: an update and a product of the state for each token
    if case["op"] == "linattn":
        return {"bytes": (3 * t + B * T) * H * D * n + state, "flops": t * H * 4 * D * D}
    return {"bytes": (4 * t + 3 * B * T) * H * D * n + (3 * B * H * D * D * 4 if case["resumed"] else 0),
            "flops": t * H * 10 * D * D}


# ---- the definition, in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _decode_exact(s)
    if case["op"] == "linattn":
        return _attn_exact(s)
    if case["op"] == "linattn_backward":
        return _attn_back_exact(s)
    if case["op"] == "rope":
        with torch.no_grad():
            return tuple(_rope_exact(s[n].double(), s[n + "w"].double(), c, s) for n, c in zip("qk", s["scales"]))
    got = {}
    for n, c in zip("qk", s["scales"]):
        x, w = s[n].double().requires_grad_(), s[n + "w"].double().requires_grad_()
        y = _rope_exact(x, w, c, s)
        got[n], got[n + "_weight"] = torch.autograd.grad(y, (x, w), s["d" + n].double())
    return got


def _rope_exact(x, w, scale, s):
    """Each pair of a head's normed vector as a complex number, turned by its angle."""
    B, T, H, D = x.shape
    table = s["table"].double()
    rot = table.shape[1]
    turn = torch.complex(table[:, :rot // 2], table[:, rot // 2:])
    pos = s["pos"].long() if s["pos"] is not None else torch.arange(T, device=x.device)[None].expand(B, T)
    turn = turn[pos][:, :, None]
    y = scale * w * x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt()
    pairs = y[..., :rot].unflatten(-1, (rot // 2, 2) if s["interleaved"] else (2, rot // 2))
    at = -1 if s["interleaved"] else -2
    z = torch.complex(pairs.select(at, 0), pairs.select(at, 1)) * turn
    y = torch.cat([torch.stack([z.real, z.imag], at).flatten(-2), y[..., rot:]], -1)
    if s["lens"] is not None:
        gone = torch.arange(T, device=x.device) >= s["lens"][:, None]
        y = y.masked_fill(gone[..., None, None], 0.0)
    return y


def _attn_exact(s):
    """Token by token: S = exp(ld) S + v k^T, o = scale S q."""
    B, T, H, D = s["q"].shape
    decay = s["log_decay"].double().exp()[:, None, None]
    S = torch.zeros(B, H, D, D, dtype=torch.float64, device="cuda") if s["state"] is None else s["state"].double()
    out = torch.zeros(B, T, H, D, dtype=torch.float64, device="cuda")
    lens = s["lens"][:, None, None, None] if s["lens"] is not None else None
    for t in range(T):
        new = torch.addcmul(decay * S, s["v"][:, t].double()[..., None], s["k"][:, t].double()[..., None, :])
        o = torch.matmul(new, s["q"][:, t].double()[..., None])[..., 0]
        if lens is not None:
            new, o = torch.where(t < lens, new, S), torch.where(t < lens[..., 0], o, 0.0)
        S = new
        out[:, t] = o
    return out * s["scale"], S


def _attn_back_exact(s):
    """Token by token: the states forwards for dq, their gradients backwards for dk and dv."""
    B, T, H, D = s["q"].shape
    decay = s["log_decay"].double().exp()[:, None, None]
    zero = torch.zeros(B, H, D, D, dtype=torch.float64, device="cuda")
    lens = s["lens"][:, None, None, None] if s["lens"] is not None else None
    dq, dk, dv = (torch.zeros(B, T, H, D, dtype=torch.float64, device="cuda") for _ in range(3))
    S = zero if s["state"] is None else s["state"].double()
    G = zero if s["d_state"] is None else s["d_state"].double()
    for t in range(T):
        S = torch.addcmul(decay * S, s["v"][:, t].double()[..., None], s["k"][:, t].double()[..., None, :])
        dq[:, t] = torch.matmul(S.transpose(-1, -2), s["d_out"][:, t].double()[..., None])[..., 0] * s["scale"]
    for t in reversed(range(T)):
        here = torch.addcmul(G, s["d_out"][:, t].double()[..., None], s["q"][:, t].double()[..., None, :], value=s["scale"])
        dv[:, t] = torch.matmul(here, s["k"][:, t].double()[..., None])[..., 0]
        dk[:, t] = torch.matmul(here.transpose(-1, -2), s["v"][:, t].double()[..., None])[..., 0]
        G = decay * here if lens is None else torch.where(t < lens, decay * here, G)
    if lens is not None:
        gone = torch.arange(T, device="cuda") >= s["lens"][:, None]
        dq, dk, dv = (a.masked_fill(gone[..., None, None], 0.0) for a in (dq, dk, dv))
    return {"q": dq, "k": dk, "v": dv, "initial_state": G if s["state"] is not None else None}


def _decode_exact(s):
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    at = torch.arange(s["B"], device="cuda") if s["slot"] is None else s["slot"].long()
    state = s["state"].double()
    state[at] = torch.einsum("h,bhvk->bhvk", s["log_decay"].double().exp(), state[at]) + torch.einsum("bhv,bhk->bhvk", v, k)
    return torch.einsum("bhvk,bhk->bhv", state[at], q) * s["scale"], state
