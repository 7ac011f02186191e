"""The operators of the gated recurrent layer, as cases to time and compare.

Two operators, in each direction that a user runs them:

* ``scan``: the gated linear recurrence with a gate for every channel and token, over prompts
  (forward and backward) and for single tokens (the decode step);
* ``norm``: layer norm over a token's whole width (forward and backward).

With ``own`` false, ``run`` computes a case from elementary torch operations in 32 bits,
rounded once at the end.  With ``own`` true it calls the library.
"""
import functools
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
CHUNK = 64          # the forward pass leaves the state before every 64th token to the backward pass


def _scan(name, B, T, D, dtype, *, backward=False, gated=True, ragged=0, resumed=False, fused=False):
    return dict(name=name, op="scan_backward" if backward else "scan", B=B, T=T, D=D, dtype=dtype, gated=gated,
                ragged=ragged, resumed=resumed, fused=fused)


def _decode(name, B, D, dtype, *, gated=True, slots=0, fused=False):
    return dict(name=name, op="decode", B=B, D=D, dtype=dtype, gated=gated, slots=slots, fused=fused)


def _norm(name, B, T, D, dtype, *, backward=False, affine=True, ragged=0):
    return dict(name=name, op="norm_backward" if backward else "norm", B=B, T=T, D=D, dtype=dtype, affine=affine,
                ragged=ragged)


def listed():
    return [
        # the LM shape's prompts, values and both gates read out of one projection
        _scan("scan lm 8x4096", 8, 4096, 2048, "bf16", fused=True),
        # one long prompt, whose write gate is what the forget gate leaves
        _scan("scan long 65536", 1, 65536, 4096, "bf16", gated=False),
        # the recommendation shape: many short ragged histories of a narrow layer
        _scan("scan rec 512x200", 512, 200, 64, "bf16", ragged=20),
        # fp32 at the sweep shape, resumed from a state, an odd length
        _scan("scan f32 4x1021", 4, 1021, 256, "f32", resumed=True),
        # training at the LM shape
        _scan("scan back lm 8x4096", 8, 4096, 2048, "bf16", backward=True, fused=True),
        # training on ragged segments of longer texts in fp32: a state comes in and its gradient goes out
        _scan("scan back f32 4x1000", 4, 1000, 256, "f32", backward=True, gated=False, resumed=True, ragged=125),
        # single tokens of eight sequences: latency
        _decode("decode 8", 8, 2048, "bf16", fused=True),
        # single tokens of a large batch whose states lie in a pool of slots
        _decode("decode 512 slots", 512, 4096, "bf16", slots=576),
        # the norm in front of a serving step: eight rows, all latency
        _norm("norm decode 8x1", 8, 1, 2048, "bf16"),
        # the norm of the LM shape's tokens
        _norm("norm lm 8x4096", 8, 4096, 2048, "bf16"),
        # its gradient, the weights' and the biases' sums over all tokens among it
        _norm("norm back lm 8x4096", 8, 4096, 2048, "bf16", backward=True),
        # the gradient at the recommendation shape in fp32: short rows, a part of them padding
        _norm("norm back rec 512x200 f32", 512, 200, 64, "f32", backward=True, ragged=20),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_backward", "scan_backward", "decode", "norm", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = 8 * _spread(rng, 2, 1024)
    if op == "decode":
        B = _spread(rng, 1, min(1024, (1 << 21) // D))
        c = _decode("", B, D, dtype, gated=rng.random() < 0.6, slots=rng.choice([0, B + B // 8 + 1]),
                    fused=rng.random() < 0.5)
    else:
        # at most the long prompt's elements, fewer for training and in fp32
        tokens = max(1, ((1 << 28) if op == "scan" and dtype == "bf16" else (1 << 25)) // D)
        T = _spread(rng, 1, min(tokens, 65536))
        B = _spread(rng, 1, max(1, min(tokens // T, 512)))
        ragged = rng.choice([0, 0, 1]) * max(1, T // 8)
        if op in ("norm", "norm_backward"):
            c = _norm("", B, T, D, dtype, backward=op == "norm_backward", affine=rng.random() < 0.8, ragged=ragged)
        else:
            c = _scan("", B, T, D, dtype, backward=op == "scan_backward", gated=rng.random() < 0.6, ragged=ragged,
                      resumed=rng.random() < 0.4, fused=rng.random() < 0.5)
    return {k: v for k, v in c.items() if k != "name"}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    B, D = case["B"], case["D"]
    s = dict(case)
    if case["op"] in ("norm", "norm_backward"):
        T = case["T"]
        # tokens of a residual stream: channels that stand apart from the others
        s["x"] = (normal(B, T, D, dtype=dt) * (1 + normal(D).abs()) + normal(D)).to(dt)
        s["w"], s["b"] = (1 + 0.2 * normal(D), 0.2 * normal(D)) if case["affine"] else (None, None)
        s["lens"] = _lens(case, g)
        if case["op"] == "norm_backward":
            s["dy"] = normal(B, T, D, dtype=dt)
        return s
    shape = (B, D) if case["op"] == "decode" else (B, case["T"], D)
    if case["fused"]:   # one projection of values and gates for each token
        x = normal(*shape[:-1], 3 if case["gated"] else 2, D, dtype=dt)
        s["x"], s["f"] = x[..., 0, :], x[..., 1, :]
        s["i"] = x[..., 2, :] if case["gated"] else None
    else:
        s["x"], s["f"] = normal(*shape, dtype=dt), normal(*shape, dtype=dt)
        s["i"] = normal(*shape, dtype=dt) if case["gated"] else None
    # channels that remember a token or two and channels that remember a thousand
    s["f"] += (7 * torch.rand(D, generator=g, device="cuda")).to(dt)
    if case["op"] == "decode":
        N = max(case["slots"], B)
        s.update(state=normal(N, D), slot=None)
        if case["slots"]:
            s["slot"] = torch.randperm(N, generator=g, device="cuda")[:B].to(torch.int32)
        return s
    s["lens"] = _lens(case, g)
    s["state"] = normal(B, D) if case["resumed"] else None
    if case["op"] == "scan_backward":
        s["d_out"] = normal(*shape, dtype=dt)
        s["d_state"] = normal(B, D) if case["resumed"] else None
        # what the forward pass has left: the state before the tokens 0, 64, 128, ...
        first = s["state"] if case["resumed"] else torch.zeros(B, D, device="cuda")
        h = _states(s)[2]
        s["states"] = torch.cat([first[:, None], h[:, CHUNK - 1:-1:CHUNK]], 1).contiguous()
    return s


def _lens(case, g):
    if not case["ragged"]:
        return None
    return torch.randint(case["ragged"], case["T"] + 1, (case["B"],), generator=g, device="cuda", dtype=torch.int32)


# ---- the plain forms ----

def _live(s):
    """[B,T,1]: the tokens that are there."""
    t = torch.arange(s["T"], device=s["x"].device)
    if s["lens"] is None:
        return torch.ones(s["B"], s["T"], 1, dtype=torch.bool, device=t.device)
    return (t < s["lens"][:, None])[..., None]


def _running(a, u):
    """r_t = a_t r_(t-1) + u_t along dim 1, from zero: spans of 1, 2, 4, ... tokens joined."""
    n, T = 1, a.shape[1]
    while n < T:
        u = torch.cat([u[:, :n], u[:, n:] + a[:, n:] * u[:, :-n]], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return u


def _gates(f, i):
    """sigmoid(f) and the write gate: sigmoid(i), or 1 - sigmoid(f)."""
    return 1 / (1 + torch.exp(-f.float())), 1 / (1 + torch.exp(f.float() if i is None else -i.float()))


def _states(s):
    """Gates and states of every token; padding keeps the state."""
    live = _live(s)
    a, w = _gates(s["f"], s["i"])
    a = torch.where(live, a, 1.0)
    u = torch.where(live, w * s["x"].float(), 0.0)
    if s["state"] is not None:
        u[:, 0] += a[:, 0] * s["state"]
    return a, w, _running(a, u)


def _scan_plain(s):
    h = _states(s)[2]
    return torch.where(_live(s), h, 0.0).to(TYPES[s["dtype"]]), h[:, -1].contiguous()


def _scan_plain_back(s):
    live, dt = _live(s), TYPES[s["dtype"]]
    a, w, h = _states(s)
    x = s["x"].float()
    before = torch.cat([s["states"][:, :1], h[:, :-1]], 1)
    d = torch.where(live, s["d_out"].float(), 0.0)
    if s["d_state"] is not None:
        d[:, -1] += s["d_state"]
    # G_t = d_t + a_(t+1) G_(t+1): the same recurrence from the other end, the gates a token on
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    G = _running(after.flip(1), d.flip(1)).flip(1)
    got = {"x": w * G, "forget": G * (before if s["gated"] else before - x) * a * (1 - a)}
    if s["gated"]:
        got["input_gate"] = G * x * w * (1 - w)
    got = {n: torch.where(live, y, 0.0).to(dt) for n, y in got.items()}
    got.setdefault("input_gate", None)
    got["initial_state"] = a[:, 0] * G[:, 0] if s["resumed"] else None
    return got


def _decode_plain(s):
    a, w = _gates(s["f"], s["i"])
    at = torch.arange(s["B"], device="cuda") if s["slot"] is None else s["slot"].long()
    h = a * s["state"][at] + w * s["x"].float()
    s["state"][at] = h
    return h.to(TYPES[s["dtype"]]), s["state"]


def _centred(s):
    """The live tokens' x - mean, and 1 / sqrt(variance + eps)."""
    x = torch.where(_live(s), s["x"].float(), 0.0)
    x = x - x.mean(-1, keepdim=True)
    return x, torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _norm_plain(s):
    x, r = _centred(s)
    y = x * r
    if s["affine"]:
        y = y * s["w"] + s["b"]
    return torch.where(_live(s), y, 0.0).to(TYPES[s["dtype"]])


def _norm_plain_back(s):
    x, r = _centred(s)
    n = x * r
    dy = torch.where(_live(s), s["dy"].float(), 0.0)
    g = dy * s["w"] if s["affine"] else dy
    dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    return {"x": torch.where(_live(s), dx, 0.0).to(TYPES[s["dtype"]]),
            "weight": (dy * n).sum((0, 1)) if s["affine"] else None, "bias": dy.sum((0, 1)) if s["affine"] else None}


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_plain(s):
    return {"scan": _scan_plain, "scan_backward": _scan_plain_back, "decode": _decode_plain, "norm": _norm_plain,
            "norm_backward": _norm_plain_back}[s["op"]](s)


@functools.cache
def _library():
    from linear_recurrent_sequence_causal_gb300 import gated
    return gated


def _run_own(s):
    gated, op = _library(), s["op"]
    if op == "scan":
        return gated.prism_gated_scan_forward(s["x"], s["f"], input_gate=s["i"], initial_state=s["state"],
                                              seq_lens=s["lens"])
    if op == "scan_backward":
        return gated.prism_gated_scan_backward(s["x"], s["f"], s["states"], s["d_out"], input_gate=s["i"],
                                               d_final_state=s["d_state"], seq_lens=s["lens"],
                                               want_initial_state=s["resumed"])
    if op == "decode":
        out = gated.prism_gated_scan_decode_step(s["x"], s["f"], s["state"], input_gate=s["i"], slots=s["slot"])
        return out, s["state"]
    if op == "norm":
        return gated.prism_layer_norm(s["x"], weight=s["w"], bias=s["b"], eps=EPS, seq_lens=s["lens"])
    return gated.prism_layer_norm_backward(s["x"], s["dy"], weight=s["w"], bias=s["b"], eps=EPS, seq_lens=s["lens"])


# ---- what a pass cannot do without ----

def work(case):
    n = 2 if case["dtype"] == "bf16" else 4
    B, D = case["B"], case["D"]
    if case["op"] == "decode":
        return {"bytes": B * D * ((4 if case["gated"] else 3) * n + 8), "flops": B * D * (12 if case["gated"] else 8)}
    T = case["T"]
    t = B * (T if not case["ragged"] else (case["ragged"] + T) / 2)   # tokens that are there, on average
    if case["op"] == "norm":
        return {"bytes": (t + B * T) * D * n + (8 * D if case["affine"] else 0), "flops": t * D * 8}
    if case["op"] == "norm_backward":
        return {"bytes": (2 * t + B * T) * D * n + (12 * D if case["affine"] else 0), "flops": t * D * 15}
    inputs = 3 if case["gated"] else 2
    state = B * D * 4 * (2 if case["resumed"] else 1)
    if case["op"] == "scan":
        return {"bytes": (inputs * t + B * T) * D * n + state, "flops": t * D * 4 * inputs}
    left = t / CHUNK * D * 4 + (state if case["resumed"] else 0)
    return {"bytes": ((inputs + 1) * t + inputs * B * T) * D * n + left, "flops": t * D * 9 * inputs}


# ---- the definition, in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_backward"):
        return _norm_exact(s)
    with torch.no_grad():
        return {"scan": _scan_exact, "scan_backward": _scan_back_exact, "decode": _decode_exact}[case["op"]](s)


def _rates(f, i):
    keep = torch.sigmoid(f.double())
    return keep, torch.sigmoid(-f.double() if i is None else i.double())


def _tokens(s):
    """For each token the gates, the value and whether each sequence has it."""
    for t in range(s["T"]):
        keep, write = _rates(s["f"][:, t], None if s["i"] is None else s["i"][:, t])
        yield t, keep, write, s["x"][:, t].double(), None if s["lens"] is None else (t < s["lens"])[:, None]


def _scan_exact(s):
    """Token by token: h = a h + w x."""
    B, T, D = s["x"].shape
    h = torch.zeros(B, D, dtype=torch.float64, device="cuda") if s["state"] is None else s["state"].double()
    out = torch.zeros(B, T, D, dtype=torch.float64, device="cuda")
    for t, keep, write, x, there in _tokens(s):
        new = torch.addcmul(write * x, keep, h)
        if there is None:
            out[:, t] = h = new
        else:
            h = torch.where(there, new, h)
            out[:, t] = new.masked_fill_(~there, 0.0)
    return out, h


def _scan_back_exact(s):
    """Token by token: the states forwards, then what reaches each of them, backwards."""
    B, T, D = s["x"].shape
    zero = torch.zeros(B, D, dtype=torch.float64, device="cuda")
    h = zero if s["state"] is None else s["state"].double()
    before = torch.empty(B, T, D, dtype=torch.float64, device="cuda")
    for t, keep, write, x, there in _tokens(s):
        before[:, t] = h
        h = torch.addcmul(write * x, keep, h) if there is None else torch.where(there, torch.addcmul(write * x, keep, h), h)
    dx, df, di = (torch.zeros(B, T, D, dtype=torch.float64, device="cuda") for _ in range(3))
    flow = zero if s["d_state"] is None else s["d_state"].double()
    for t in reversed(range(T)):
        keep, write = _rates(s["f"][:, t], None if s["i"] is None else s["i"][:, t])
        G, x = flow + s["d_out"][:, t].double(), s["x"][:, t].double()
        there = None if s["lens"] is None else (t < s["lens"])[:, None]
        G = G if there is None else G.masked_fill(~there, 0.0)
        dx[:, t] = G * write
        if s["gated"]:
            df[:, t] = G * before[:, t] * keep * (1 - keep)
            di[:, t] = G * x * write * (1 - write)
        else:
            df[:, t] = G * (before[:, t] - x) * keep * write
        flow = G * keep if there is None else torch.where(there, G * keep, flow)
    return {"x": dx, "forget": df, "input_gate": di if s["gated"] else None,
            "initial_state": flow if s["resumed"] else None}


def _decode_exact(s):
    keep, write = _rates(s["f"], s["i"])
    at = torch.arange(s["B"], device="cuda") if s["slot"] is None else s["slot"].long()
    state = s["state"].double()
    state[at] = keep * state[at] + write * s["x"].double()
    return state[at], state


def _norm_exact(s):
    """The operator on the live tokens alone, its gradient by differentiation."""
    B, T, D = s["x"].shape
    there = (torch.ones(B, T, dtype=torch.bool, device="cuda") if s["lens"] is None
             else torch.arange(T, device="cuda") < s["lens"][:, None])
    x = s["x"][there].double()
    leaves = [x] + ([s["w"].double(), s["b"].double()] if s["affine"] else [])
    back = s["op"] == "norm_backward"
    with torch.set_grad_enabled(back):
        for leaf in leaves:
            leaf.requires_grad_(back)
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        y = (x - mean) / (var + EPS).sqrt()
        if s["affine"]:
            y = y * leaves[1] + leaves[2]
        got = torch.autograd.grad(y, leaves, s["dy"][there].double()) if back else [y]
    whole = torch.zeros(B, T, D, dtype=torch.float64, device="cuda")
    whole[there] = got[0]
    if not back:
        return whole
    return {"x": whole, "weight": got[1] if s["affine"] else None, "bias": got[2] if s["affine"] else None}
