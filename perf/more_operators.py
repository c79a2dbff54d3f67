"""The operators of selective state space layers: the packed scan with its short convolution, the step of
decoding requests, and the root-mean-square norm (residual, gate, 8-bit codes) around them.

``listed`` and ``draw`` give cases, ``prepare`` a case's inputs, ``run`` one pass: in elementary torch
operations, or, where ``own`` is set, through the library's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TOP = {"e4m3": 448.0, "int8": 127.0}
CHUNK = 64                   # tokens of a chunk of the plain form


# ------------------------------------------------------------------ cases --

def listed():
    """The chat wave (32 x 1,024 tokens), the long prompts (4 x 8,192) with 16 groups and 32 heads of 128 on 128, ragged
    prompts of 17 to 2,048 tokens and batches of 32 and 64 decoding requests are this repository's workloads; heads of 64,
    one or eight groups and the widths of the norm are generic."""
    return [
        # one short prompt alone: latency
        dict(name="scan short prompt", op="scan", n=1, lo=100, hi=100, H=16, G=1, P=64, N=128, conv=True, init=False, ckpt=0, mix=1),
        # ragged prompts that continue cached prefixes, states kept every 256 tokens
        dict(name="scan ragged prefixes", op="scan", n=8, lo=17, hi=2048, H=64, G=8, P=64, N=128, conv=True, init=True, ckpt=256, mix=2),
        # a chat wave from nothing
        dict(name="scan chat wave", op="scan", n=32, lo=1024, hi=1024, H=64, G=1, P=64, N=128, conv=True, init=False, ckpt=0, mix=3),
        # long prompts whose rows are convolved already
        dict(name="scan long prompts", op="scan", n=4, lo=8192, hi=8192, H=32, G=16, P=128, N=128, conv=False, init=False, ckpt=0, mix=4),
        # one user alone: the smallest decode call
        dict(name="step one request", op="step", n=1, n_tok=1, H=64, G=1, P=64, N=128, snap=False, mix=5),
        # a decode batch
        dict(name="step batch", op="step", n=64, n_tok=1, H=64, G=8, P=64, N=128, snap=False, mix=6),
        # verification of drafted tokens, every state kept
        dict(name="step 4 tokens kept", op="step", n=16, n_tok=4, H=32, G=2, P=128, N=64, snap=True, mix=7),
        # a decode step's residual and norm, codes for the next projection
        dict(name="norm decode rows", op="norm", rows=32, dim=4096, groups=1, res="bf16", gate="none", code="e4m3", block=0, mix=8),
        # a pass's residual and norm, codes with a scale per 128 channels
        dict(name="norm pass rows", op="norm", rows=32768, dim=4096, groups=1, res="bf16", gate="none", code="e4m3", block=128, mix=9),
        # an odd width with the residual stream in 32 bits
        dict(name="norm odd width", op="norm", rows=1000, dim=2777, groups=1, res="fp32", gate="none", code="", block=0, mix=10),
        # the gated norm over each head that follows the delta-rule scan
        dict(name="norm gate after", op="norm", rows=8192, dim=4096, groups=32, res="", gate="after", code="", block=0, mix=11),
        # the gated norm over groups that follows the state space scan, codes for the output projection
        dict(name="norm gate first int8", op="norm", rows=1024, dim=4096, groups=8, res="", gate="first", code="int8", block=0, mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, mix = rng.choice(["scan", "scan", "step", "norm"]), rng.randrange(1 << 20)
    if op == "norm":
        groups = rng.choice([1, 1, 2, 8, 32])
        gate = rng.choice(["none", "first", "after"])
        code = rng.choice(["", "e4m3", "int8"])
        block = rng.choice([0, 128]) if code else 0
        if groups > 1:
            dim = groups * rng.choice([32, 64, 128, 256, 512])
        else:
            dim = _log(rng, 1, 16384)
        if block:
            dim = max(128, dim // 128 * 128)
            groups = 1 if dim % groups or (groups > 1 and dim // groups not in (32, 64, 128, 256, 512)) else groups
        return dict(op=op, rows=_log(rng, 1, min(32768, (1 << 26) // dim)), dim=dim, groups=groups, res=rng.choice(["", "bf16", "fp32"]),
                    gate=gate, code=code, block=block, mix=mix)
    G, P, N = rng.choice([1, 1, 2, 4, 8]), rng.choice([32, 64, 64, 128]), rng.choice([32, 64, 128, 128])
    H = G * rng.choice([1, 2, 3, 4, 6, 8, 16])
    while H * P > 8192:
        P //= 2
    if op == "step":
        n_tok, snap = rng.choice([1, 1, 1, 2, 3, 4]), rng.random() < 0.3
        most = min(64, 64 * 4096 // (H * P * (n_tok if snap else 1)))
        return dict(op=op, n=_log(rng, 1, most), n_tok=n_tok, H=H, G=G, P=P, N=N, snap=snap, mix=mix)
    n = _log(rng, 1, 32)
    hi = _log(rng, 1, min(8192, 4096 * 32768 // (n * max(H * P, 4096))))
    return dict(op=op, n=n, lo=rng.randint(1, hi), hi=hi, H=H, G=G, P=P, N=N, conv=rng.random() < 0.7, init=rng.random() < 0.5,
                ckpt=rng.choice([0, 64, 100, 512]), mix=mix)


def _lens(case):
    r = random.Random(case["mix"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]


def _ckpts(case):
    """Positions in the pack: every `ckpt` tokens of each prompt."""
    out, at = [], 0
    for x in _lens(case):
        if case["ckpt"]:
            out += range(at + case["ckpt"], at + x + 1, case["ckpt"])
        at += x
    return out


def _dims(case):
    """(inner width H P, conv width, width of one projected row [z | x | B | C | dt])."""
    inner = case["H"] * case["P"]
    conv = inner + 2 * case["G"] * case["N"]
    return inner, conv, inner + conv + (case["H"] + 7) // 8 * 8


# ----------------------------------------------------------------- inputs --

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _layer(g, case, s):
    """A layer's constants: decays between 1 and 16, steps between 0.001 and 0.1 at a raw step of 0."""
    H, (_, conv, _) = case["H"], _dims(case)
    rand = lambda *n: torch.rand(*n, generator=g, device=DEV)
    s["A"] = -(1.0 + 15.0 * rand(H))
    dt = torch.exp(rand(H) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    s["dt_bias"] = dt + torch.log(-torch.expm1(-dt))
    s["D"] = 1.0 + 0.1 * torch.randn(H, generator=g, device=DEV)
    s["w"] = rand(conv, 4) - 0.5
    s["bias"] = 0.2 * (rand(conv) - 0.5)


def _rows(g, case, t, s):
    """Rows of one merged projection, in bf16: the columns of x, B, C and of the raw steps."""
    inner, conv, width = _dims(case)
    row = torch.randn(t, width, generator=g, device=DEV).bfloat16()
    s["row"] = row
    s["xbc"], s["dt"] = row[:, inner:inner + conv], row[:, inner + conv:inner + conv + case["H"]]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    randn = lambda *n: torch.randn(*n, generator=g, device=DEV)
    s = dict(case=case, op=case["op"])
    if case["op"] == "norm":
        t, d = case["rows"], case["dim"]
        chan = torch.ones(d, device=DEV)
        chan[::64] = 8.0                                       # channels that stand out, as in a residual stream
        s["x"] = (randn(t, d) * chan).bfloat16()
        s["z"] = randn(t, d).bfloat16() if case["gate"] != "none" else None
        s["res"] = (randn(t, d) * chan).to(torch.bfloat16 if case["res"] == "bf16" else torch.float32) if case["res"] else None
        s["w"] = 1.0 + 0.1 * randn(d)
        s["res_out"] = torch.empty_like(s["res"]) if case["res"] else None
        s["out"] = torch.empty(t, d, dtype=torch.bfloat16, device=DEV)
        if case["code"]:
            s["codes"] = torch.empty(t, d, dtype=torch.float8_e4m3fn if case["code"] == "e4m3" else torch.int8, device=DEV)
            s["scales"] = torch.empty(t, d // case["block"] if case["block"] else 1, device=DEV)
        return s
    H, P, N, n = case["H"], case["P"], case["N"], case["n"]
    inner, conv, _ = _dims(case)
    _layer(g, case, s)
    if case["op"] == "step":
        pool, nt = n + 3, case["n_tok"]
        _rows(g, case, n * nt, s)
        s["state"], s["window"] = 0.5 * randn(pool, H, P, N), randn(pool, 3, conv).bfloat16()
        s["slot"] = torch.randperm(pool, generator=g, device=DEV)[:n].to(torch.int32)
        s["slot_host"] = s["slot"].cpu().numpy()
        s["out"] = torch.empty(n * nt, H, P, dtype=torch.bfloat16, device=DEV)
        s["snap"] = torch.empty(n, nt, H, P, N, device=DEV) if case["snap"] else None
        return s
    lens = _lens(case)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    t = cu[-1]
    _rows(g, case, t, s)
    if not case["conv"]:                                       # what a convolution before would have left in these columns
        s["xbc"].copy_(torch.nn.functional.silu(s["xbc"].float()))
    s["init"] = 0.5 * randn(n, H, P, N) if case["init"] else None
    s["window_in"] = randn(n, 3, conv).bfloat16() if case["conv"] and case["init"] else None
    ck = _ckpts(case)
    s.update(cu=_i32(cu), cu_host=np.array(cu, dtype=np.int32), ck=_i32(ck), ck_host=np.array(ck, dtype=np.int32), n_max=max(lens))
    s["out"] = torch.empty(t, H, P, dtype=torch.bfloat16, device=DEV)
    s["final"] = torch.empty(n, H, P, N, device=DEV)
    s["kept"] = torch.empty(len(ck), H, P, N, device=DEV)
    s["window_out"] = torch.empty(n, 3, conv, dtype=torch.bfloat16, device=DEV) if case["conv"] else None
    s["window_kept"] = torch.empty(len(ck), 3, conv, dtype=torch.bfloat16, device=DEV) if case["conv"] and ck else None
    return s


# --------------------------------------------------- the library's calls --

_lib = None


def _gdn():
    global _lib
    if _lib is None:
        import gated_deltanet_prefill_varlen_amd as lib
        _lib = lib
    return _lib


def _handle(s):
    """The layer's shape and the scan's workspace: made once, kept by the program."""
    if "handle" not in s:
        gdn, c = _gdn(), s["case"]
        if s["op"] == "norm":
            s["handle"] = gdn.make_norm(c["dim"], groups=c["groups"], eps=1e-5, gate_first=c["gate"] == "first",
                                        scale_block=c["block"])
        else:
            s["handle"] = gdn.make_ssm(c["H"], c["G"], c["P"], c["N"])
        if s["op"] == "scan":
            size = gdn.gdn_ssm_prefill_workspace(s["handle"], s["cu_host"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s["handle"]


def _run_own(s):
    gdn, c, h = _gdn(), s["case"], _handle(s)
    if s["op"] == "scan":
        with_conv = dict(conv_weight=s["w"], conv_bias=s["bias"], conv_state_in=s["window_in"], conv_state_out=s["window_out"],
                         conv_ckpt=s["window_kept"]) if c["conv"] else {}
        gdn.gdn_ssm_prefill_packed(h, s["cu"], s["cu_host"], s["xbc"], s["dt"], s["A"], s["out"], dt_bias=s["dt_bias"], D=s["D"],
                                   init_state=s["init"], final_state=s["final"], ckpt_positions=s["ck"], ckpt_positions_host=s["ck_host"],
                                   ckpt_buf=s["kept"], workspace=s["workspace"], **with_conv)
        return _all(s["out"], s["final"], s["kept"], s["window_out"], s["window_kept"])
    if s["op"] == "step":
        gdn.gdn_ssm_decode(h, c["n_tok"], s["xbc"], s["dt"], s["A"], s["state"], s["out"], dt_bias=s["dt_bias"], D=s["D"],
                           conv_weight=s["w"], conv_bias=s["bias"], conv_state=s["window"], slot=s["slot"], slot_host=s["slot_host"],
                           snapshots=s["snap"])
        return _all(s["out"], s["state"], s["window"], s["snap"])
    codes = dict(codes=s["codes"], scales=s["scales"]) if c["code"] else dict(out=s["out"])
    gdn.gdn_rms_norm(h, s["x"], s["w"], residual=s["res"], residual_out=s["res_out"], gate=s["z"], **codes)
    if c["code"] == "int8":                                    # the values that the codes stand for
        nb = s["scales"].shape[1]
        out = s["out"].view(c["rows"], nb, -1)
        torch.mul(s["codes"].view(c["rows"], nb, -1), s["scales"][:, :, None], out=out)
        return _all(s["out"], s["scales"], s["res_out"])
    return _all(s["codes"], s["scales"], s["res_out"]) if c["code"] else _all(s["out"], s["res_out"])


# --------------------------------------------------------- the plain form --

def _all(*v):
    return [x for x in v if x is not None]


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))


def _conv(s, ext):
    """silu(bias + the four taps) over rows that start with the three before the first: [.., 3 + L, C] -> [.., L, C]."""
    w, n = s["w"], ext.shape[-2] - 3
    y = s["bias"] + w[:, 0] * ext[..., 0:n, :] + w[:, 1] * ext[..., 1:n + 1, :] + w[:, 2] * ext[..., 2:n + 2, :] + w[:, 3] * ext[..., 3:n + 3, :]
    return _silu(y)


def _run_scan(s):
    c = s["case"]
    H, G, P, N, n = c["H"], c["G"], c["P"], c["N"], c["n"]
    inner, conv, _ = _dims(c)
    cu = s["cu"].long()
    new = cu[1:] - cu[:-1]
    nc = -(-s["n_max"] // CHUNK)
    i = torch.arange(nc * CHUNK, device=DEV)[None, :]
    at = cu[:-1, None] + torch.minimum(i, new[:, None] - 1)
    real = i < new[:, None]
    raw = torch.where(real[..., None], s["xbc"][at], 0).float()                              # [n, L, C], zeros past each end
    if c["conv"]:
        before = s["window_in"].float() if s["window_in"] is not None else raw.new_zeros(n, 3, conv)
        ext = torch.cat([before, raw], 1)
        u = torch.where(real[..., None], _conv(s, ext), 0.0)
    else:
        u = raw
    x = u[..., :inner].reshape(n, nc, CHUNK, H, P).permute(0, 1, 3, 2, 4)                   # [n, nc, H, c, P]
    B = u[..., inner:inner + G * N].reshape(n, nc, CHUNK, G, N).permute(0, 1, 3, 2, 4)
    C = u[..., inner + G * N:].reshape(n, nc, CHUNK, G, N).permute(0, 1, 3, 2, 4)
    dt = torch.where(real[..., None], _softplus(s["dt"][at].float() + s["dt_bias"]), 0.0)
    dt = dt.reshape(n, nc, CHUNK, H).transpose(2, 3)                                         # [n, nc, H, c]
    cum = torch.cumsum(dt.double() * s["A"].double()[:, None], -1)                           # sums of many steps: 64 bits
    # inside a chunk
    seen = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    decay = (cum[..., :, None] - cum[..., None, :]).masked_fill_(~seen, float("-inf")).exp_().float()
    scores = torch.matmul(C, B.transpose(3, 4).contiguous()).repeat_interleave(H // G, 2)
    xdt = (x * dt[..., None]).contiguous()
    y = torch.matmul(scores.mul_(decay), xdt)
    # each chunk's own state, and the states that enter the chunks
    w = (cum[..., -1:] - cum).exp_().float()
    Bh, Ch = B.repeat_interleave(H // G, 2), C.repeat_interleave(H // G, 2)
    local = torch.matmul((xdt * w[..., None]).transpose(3, 4).contiguous(), Bh)              # [n, nc, H, P, N]
    total = torch.cumsum(torch.cat([cum.new_zeros(n, 1, H), cum[..., -1]], 1), 1)            # [n, nc + 1, H]
    far = (total[:, :, None] - total[:, None, :]).permute(0, 3, 1, 2)                        # [n, H, to, from]
    order = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=DEV).tril()
    far = far.masked_fill(~order, float("-inf")).exp_().float()
    first = s["init"] if s["init"] is not None else local.new_zeros(n, H, P, N)
    parts = torch.cat([first[:, None], local], 1).permute(0, 2, 1, 3, 4).reshape(n, H, nc + 1, P * N)
    states = torch.matmul(far, parts).reshape(n, H, nc + 1, P, N)
    enter = states[:, :, :-1].transpose(1, 2)                                                # [n, nc, H, P, N]
    y = y.add_(torch.matmul(Ch, enter.transpose(3, 4).contiguous()).mul_(cum.exp().float()[..., None])).add_(x * s["D"][:, None, None])
    out = y.permute(0, 1, 3, 2, 4).reshape(n, nc * CHUNK, H, P)[real].bfloat16()
    final = states[:, :, -1]
    # the state after some tokens: that of the chunk's start and the tokens up to there
    p = s["ck"].long()
    who = torch.searchsorted(cu, p) - 1
    last = p - cu[who] - 1
    ch, off = last // CHUNK, last % CHUNK
    cc = cum[who, ch]                                                                        # [k, H, c]
    upto = torch.gather(cc, 2, off[:, None, None].expand(-1, H, 1))
    w = (upto - cc).masked_fill_(torch.arange(CHUNK, device=DEV) > off[:, None, None], float("-inf")).exp_().float()
    kept = torch.matmul((xdt[who, ch] * w[..., None]).transpose(2, 3).contiguous(), Bh[who, ch])
    kept.add_(states[who, :, ch].mul_(upto.exp().float()[..., None]))
    if not c["conv"]:
        return [out, final, kept]
    three = torch.arange(3, device=DEV)
    rows = torch.arange(n, device=DEV)[:, None]
    window = ext[rows, new[:, None] + three].bfloat16()
    windows = ext[who[:, None], (last + 1)[:, None] + three].bfloat16() if s["window_kept"] is not None else None
    return _all(out, final, kept, window, windows)


def _step(s, u, dt, state):
    """One token of every request: x, B, C in u [n, C], its steps dt [n, H]; (y [n, H, P], the next state)."""
    c = s["case"]
    H, G, P, N, n = c["H"], c["G"], c["P"], c["N"], c["n"]
    inner = H * P
    x = u[:, :inner].reshape(n, H, P)
    B = u[:, inner:inner + G * N].reshape(n, G, 1, N).repeat_interleave(H // G, 1)
    C = u[:, inner + G * N:].reshape(n, G, 1, N).repeat_interleave(H // G, 1)
    state = state * torch.exp(dt * s["A"])[..., None, None] + (x * dt[..., None])[..., None] * B
    return (state * C).sum(-1) + x * s["D"][:, None], state


def _run_step(s):
    c = s["case"]
    n, nt, H = c["n"], c["n_tok"], c["H"]
    slot = s["slot"].long()
    ext = torch.cat([s["window"][slot], s["xbc"].reshape(n, nt, -1)], 1)
    u = _conv(s, ext.float())
    dt = _softplus(s["dt"].reshape(n, nt, H).float() + s["dt_bias"])
    state, ys, snaps = s["state"][slot], [], []
    for i in range(nt):
        y, state = _step(s, u[:, i], dt[:, i], state)
        ys.append(y)
        snaps.append(state)
    s["state"][slot] = state
    s["window"][slot] = ext[:, nt:]
    out = torch.stack(ys, 1).reshape(n * nt, H, c["P"]).bfloat16()
    return _all(out, s["state"], s["window"], torch.stack(snaps, 1) if c["snap"] else None)


def _run_norm(s):
    c = s["case"]
    t, d, groups = c["rows"], c["dim"], c["groups"]
    r = s["x"].float()
    if s["res"] is not None:
        r = r + s["res"].float()
    y = r
    if c["gate"] == "first":
        y = y * _silu(s["z"].float())
    y = y.reshape(t, groups, d // groups)
    y = (y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-5)).reshape(t, d) * s["w"]
    if c["gate"] == "after":
        y = y * _silu(s["z"].float())
    res_out = r.to(s["res"].dtype) if s["res"] is not None else None
    if not c["code"]:
        return _all(y.bfloat16(), res_out)
    y = y.reshape(t, d // c["block"] if c["block"] else 1, -1)
    top = TOP[c["code"]]
    scales = y.abs().amax(-1, keepdim=True) / top
    code = torch.clamp(y / scales, -top, top)
    if c["code"] == "e4m3":
        return _all(code.reshape(t, d).to(torch.float8_e4m3fn), scales[..., 0], res_out)
    return _all((code.round() * scales).reshape(t, d).bfloat16(), scales[..., 0], res_out)


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "scan":
        return _run_scan(state)
    return _run_step(state) if state["op"] == "step" else _run_norm(state)


# ------------------------------------------------------------------- work --

def work(case):
    if case["op"] == "norm":
        t, d = case["rows"], case["dim"]
        res = {"": 0, "bf16": 4, "fp32": 8}[case["res"]]
        out = 1 if case["code"] else 2
        scales = 4 * t * (d // case["block"] if case["block"] else 1) if case["code"] else 0
        return {"bytes": t * d * (2 + res + (2 if case["gate"] != "none" else 0) + out) + scales + 4 * d, "flops": t * d * 8}
    H, P, N, n = case["H"], case["P"], case["N"], case["n"]
    inner, conv, _ = _dims(case)
    state, layer = 4 * H * P * N, 4 * 3 * H
    if case["op"] == "step":
        t = n * case["n_tok"]
        moved = n * (2 * state + 2 * 6 * conv) + (t * state if case["snap"] else 0)
        return {"bytes": moved + t * 2 * (conv + H + inner) + layer + 20 * conv, "flops": t * H * P * (6 * N + 4) + 10 * t * conv}
    t, k = sum(_lens(case)), len(_ckpts(case))
    windows = 6 * conv * (n + k + (n if case["init"] else 0)) + 20 * conv if case["conv"] else 0
    return {"bytes": t * 2 * (conv + H + inner) + state * (n + k + (n if case["init"] else 0)) + windows + layer,
            "flops": t * H * P * (6 * N + 4) + (10 * t * conv if case["conv"] else 0)}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    """The operators' definition in 64 bits, token by token."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        t, d, groups = case["rows"], case["dim"], case["groups"]
        r = s["x"].double() + (s["res"].double() if s["res"] is not None else 0.0)
        gate = s["z"].double() * torch.sigmoid(s["z"].double()) if s["z"] is not None else 1.0
        y = (r * gate if case["gate"] == "first" else r).view(t, groups, -1)
        norm = torch.linalg.vector_norm(y, dim=-1, keepdim=True)
        y = (y * torch.rsqrt(norm ** 2 * groups / d + 1e-5)).view(t, d) * s["w"].double()
        if case["gate"] == "after":
            y = y * gate
        res = r if s["res"] is not None else None
        if not case["code"]:
            return _all(y, res)
        y = y.view(t, s["scales"].shape[1], -1)
        step = y.abs().amax(-1) / TOP[case["code"]]
        q = y / step[..., None]
        if case["code"] == "e4m3":
            return _all(q.float().to(torch.float8_e4m3fn).double().view(t, d), step, res)
        return _all((torch.round(q) * step[..., None]).view(t, d), step, res)
    H, G, P, N, n = case["H"], case["G"], case["P"], case["N"], case["n"]
    inner, conv, _ = _dims(case)
    per, wide = H // G, s["xbc"].double()
    dt_all = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=1e9)
    A, D = s["A"].double(), s["D"].double()

    def convolved(ext):
        y = torch.nn.functional.conv1d(ext.t()[None].contiguous(), s["w"].double()[:, None, :], s["bias"].double(), groups=conv)[0].t()
        return y * torch.sigmoid(y)

    def advance(state, u, dt):
        """state [m, H, P, N] in place by one token (u [m, conv], dt [m, H]); its output."""
        b = u[:, inner:inner + G * N].view(-1, G, 1, N).expand(-1, G, per, N).reshape(-1, H, 1, N)
        c = u[:, inner + G * N:].view(-1, G, 1, N).expand(-1, G, per, N).reshape(-1, H, N, 1)
        x = u[:, :inner].view(-1, H, P)
        state.mul_(torch.exp(A * dt)[..., None, None]).addcmul_((dt[..., None] * x)[..., None], b)
        return torch.matmul(state, c)[..., 0] + D[:, None] * x

    if case["op"] == "step":
        nt, slot = case["n_tok"], s["slot"].long()
        ext = torch.cat([s["window"][slot].double(), wide.view(n, nt, conv)], 1)
        u = torch.stack([convolved(ext[r]) for r in range(n)])
        state, out, snaps = s["state"].double()[slot], [], []
        for i in range(nt):
            out.append(advance(state, u[:, i], dt_all.view(n, nt, H)[:, i]))
            snaps.append(state.clone())
        pool, window = s["state"].double(), s["window"].double()
        pool[slot], window[slot] = state, ext[:, nt:]
        return _all(torch.stack(out, 1).reshape(n * nt, H, P), pool, window, torch.stack(snaps, 1) if case["snap"] else None)
    if case["n"] * case["H"] * P * N * s["n_max"] > 2e11:
        return None
    lens, cu = _lens(case), s["cu_host"].tolist()
    parts = [wide[a:b] for a, b in zip(cu, cu[1:])]
    if case["conv"]:
        before = s["window_in"].double() if s["window_in"] is not None else torch.zeros(n, 3, conv, dtype=torch.float64, device=DEV)
        ext = [torch.cat([before[r], parts[r]]) for r in range(n)]
        parts = [convolved(e) for e in ext]
    order = sorted(range(n), key=lambda r: -lens[r])           # longest first: those still running are the first rows
    state = s["init"].double()[order] if s["init"] is not None else torch.zeros(n, H, P, N, dtype=torch.float64, device=DEV)
    u = torch.zeros(n, max(lens), conv, dtype=torch.float64, device=DEV)
    dt = torch.zeros(n, max(lens), H, dtype=torch.float64, device=DEV)
    out = torch.zeros(n, max(lens), H, P, dtype=torch.float64, device=DEV)
    for k, r in enumerate(order):
        u[k, :lens[r]], dt[k, :lens[r]] = parts[r], dt_all[cu[r]:cu[r + 1]]
    ck, kept, home = _ckpts(case), {}, {}
    for p in ck:
        r = max(i for i in range(n) if cu[i] < p)
        home.setdefault(p - cu[r], []).append((order.index(r), p))
    for i in range(max(lens)):
        m = sum(x > i for x in lens)
        out[:m, i] = advance(state[:m], u[:m, i], dt[:m, i])
        for k, p in home.get(i + 1, []):
            kept[p] = state[k].clone()
    back = [order.index(r) for r in range(n)]
    y = torch.cat([out[back[r], :lens[r]] for r in range(n)])
    keep = torch.stack([kept[p] for p in ck]) if ck else torch.empty(0, H, P, N, dtype=torch.float64, device=DEV)
    if not case["conv"]:
        return [y, state[back], keep]
    window = torch.stack([e[-3:] for e in ext])
    windows = None
    if ck:
        who = [max(i for i in range(n) if cu[i] < p) for p in ck]
        windows = torch.stack([ext[r][p - cu[r]:p - cu[r] + 3] for r, p in zip(who, ck)])
    return _all(y, state[back], keep, window, windows)
