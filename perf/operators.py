"""The operators of a selective state-space layer, each in its plain form and as the library's
kernels: the selective scan over prompts (``selective_scan``) and its gradient
(``selective_scan_bwd``), its form for single tokens (``selective_state_update``), the gradient
of the short causal convolution before it (``causal_conv1d_bwd``, with ``causal_conv1d``), and
the channels-last group norm with an activation or a gate after it (``group_norm``,
``group_norm_bwd``).

With ``own`` false, ``run`` computes the plain form: elementary torch operations in fp32, each
output rounded once at the end.  The scan is a recurrence over tokens, so its plain form has a
loop over them: everything but the recurrence itself (one fused multiply-add per token) is done
for a block of tokens at once.  With ``own`` true, ``run`` calls the library.

A case is a dict of plain values; ``op`` names the path it times:
  scan        prompt: y and the final states of a dense or packed batch
  train_scan  forward and backward of the same
  step        one token for each of ``batch`` sequences, the states in a pool of lines
  train_conv  the short convolution forward and backward
  norm        group norm forward
  train_norm  group norm forward and backward
``lens`` (a text of comma-separated lengths) makes a packed batch; without it the batch is
``batch`` sequences of ``tokens`` tokens.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128  # tokens whose decays and inputs the plain scan forms at once
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --- the cases ------------------------------------------------------------------------------

def listed():
    return [
        # the first words of a conversation, fp32, an odd channel count, a carried state
        dict(name="scan-short-f32", op="scan", dtype="f32", batch=1, tokens=129, lens="",
             channels=1000, groups=1, dstate=16, gate=False, state=True),
        # a serving batch of prompts of unlike lengths, packed; one of them a single token
        dict(name="scan-packed", op="scan", dtype="bf16", batch=1, tokens=12454,
             lens="2048,1999,2041,1537,1801,2003,1,1024", channels=4096, groups=1, dstate=16,
             gate=True, state=True),
        # one long prompt alone: few rows, a long axis
        dict(name="scan-long", op="scan", dtype="bf16", batch=1, tokens=8192, lens="",
             channels=4096, groups=1, dstate=16, gate=True, state=False),
        # a small fp32 training step, B and C shared by two groups of channels
        dict(name="train-scan-f32", op="train_scan", dtype="f32", batch=2, tokens=257, lens="",
             channels=768, groups=2, dstate=16, gate=True, state=True),
        # a training step of ordinary size
        dict(name="train-scan", op="train_scan", dtype="bf16", batch=8, tokens=2048, lens="",
             channels=4096, groups=1, dstate=16, gate=True, state=False),
        # one user's next token: the latency of one call
        dict(name="step-1", op="step", dtype="bf16", batch=1, channels=4096, groups=1,
             dstate=16, gate=True),
        # the decode batch, one token for each of 256 sequences
        dict(name="step-256", op="step", dtype="bf16", batch=256, channels=4096, groups=1,
             dstate=16, gate=True),
        # the convolution's step on a packed fp32 batch with sequences shorter than its width
        dict(name="train-conv-packed", op="train_conv", dtype="f32", batch=1, tokens=1190,
             lens="1,2,333,100,517,3,234", channels=1000, width=3, act=True),
        # the convolution before a wide layer, a quarter of the 16 x 8192 batch
        dict(name="train-conv", op="train_conv", dtype="bf16", batch=4, tokens=8192, lens="",
             channels=12288, width=4, act=True),
        # the gated norm of every token's heads after the scan of a prompt
        dict(name="norm-tokens", op="norm", dtype="bf16", batch=16384, positions=1,
             channels=4096, groups=32, act=True, gate=True),
        # a small odd feature map, fp32
        dict(name="norm-map-f32", op="norm", dtype="f32", batch=2, positions=63, channels=320,
             groups=32, act=True, gate=False),
        # a training step over feature maps: statistics over thousands of positions
        dict(name="train-norm-map", op="train_norm", dtype="bf16", batch=8, positions=4096,
             channels=512, groups=32, act=True, gate=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges: lengths from one token on, channel counts that are no
    multiple of a vector, small and large states, groups, both types."""
    op = rng.choice(["scan", "train_scan", "step", "train_conv", "norm", "train_norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("scan", "train_scan", "step"):
        groups = rng.choice([1, 1, 2, 4])
        channels = groups * _log_int(rng, 16, 4096 // groups)
        dstate = rng.choice([4, 8, 12, 16, 16, 32, 64] if op != "step" else
                            [4, 8, 12, 16, 16, 32, 64, 128])
        case = dict(op=op, dtype=dtype, channels=channels, groups=groups, dstate=dstate,
                    gate=rng.random() < 0.7)
        if op == "step":
            case["batch"] = max(1, min(_log_int(rng, 1, 256),
                                       256 * 4096 * 16 // (channels * dstate)))
            return case
        case["state"] = rng.random() < 0.5
        longest = _log_int(rng, 1, 2048)
        most = 8 * 2048 * 4096 * 16 // (channels * dstate * longest)  # sequences of that length
        n = max(1, min(_log_int(rng, 1, 32), most, 16384 // longest + 1))
        if n > 1 and rng.random() < 0.5:
            lens = [rng.randint(max(1, longest // 2), longest) for _ in range(n - 1)] + [longest]
            rng.shuffle(lens)
            case.update(batch=1, tokens=sum(lens), lens=",".join(map(str, lens)))
        else:
            case.update(batch=n, tokens=longest, lens="")
        return case
    if op == "train_conv":
        channels = 8 * _log_int(rng, 1, 1536)
        total = max(1, min(_log_int(rng, 1, 32768), 4 * 8192 * 12288 // channels))
        case = dict(op=op, dtype=dtype, channels=channels, width=rng.choice([2, 3, 4, 4]),
                    act=rng.random() < 0.8)
        if total > 3 and rng.random() < 0.5:
            n = _log_int(rng, 1, min(total, 64))
            cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
            case.update(batch=1, tokens=total, lens=",".join(map(str, lens)))
        else:
            n = _log_int(rng, 1, min(total, 32))
            case.update(batch=n, tokens=max(1, total // n), lens="")
        return case
    groups = rng.choice([1, 4, 8, 16, 32, 32])
    channels = groups * _log_int(rng, 1, 4096 // groups)
    most = 16384 * 4096 // channels
    if rng.random() < 0.5:
        batch, positions = _log_int(rng, 1, min(16384, most)), 1
    else:
        positions = _log_int(rng, 2, min(16384, most))
        batch = _log_int(rng, 1, max(1, min(32, most // positions)))
    act = rng.random() < 0.8
    return dict(op=op, dtype=dtype, batch=batch, positions=positions, channels=channels,
                groups=groups, act=act, gate=act and rng.random() < 0.4)


# --- their inputs ---------------------------------------------------------------------------

def _lens(case):
    return [int(t) for t in case["lens"].split(",")] if case["lens"] else None


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32) * std + mean

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev, dtype=torch.float32)

    s = dict(case=case)
    op, D = case["op"], case["channels"]
    if op in ("scan", "train_scan", "step"):
        G, S = case["groups"], case["dstate"]
        lead = (case["batch"], case["tokens"]) if op != "step" else (case["batch"],)
        # the time steps' usual start: softplus(dt_bias) log-uniform in [0.001, 0.1]; decay rates
        # 1 .. S, spread a little as training does
        first = torch.exp(uniform(D) * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = first + torch.log(-torch.expm1(-first))
        s["A"] = -torch.arange(1, S + 1, device=dev, dtype=torch.float32) * torch.exp(
            normal(D, S, std=0.2))
        s["D"] = normal(D, std=0.1, mean=1.0)
        s["x"] = normal(*lead, D).to(dt)
        s["dt"] = normal(*lead, D, std=0.5).to(dt)
        # B and C are slices of one projection, behind the low-rank input of dt
        rank = (D + 15) // 16
        proj = normal(*lead, rank + 2 * G * S).to(dt)
        s["B"] = proj[..., rank:rank + G * S].unflatten(-1, (G, S))
        s["C"] = proj[..., rank + G * S:].unflatten(-1, (G, S))
        # the gate is the second half of the layer's input projection
        s["z"] = normal(*lead, 2 * D).to(dt)[..., D:] if case["gate"] else None
        if op == "step":
            # a pool of lines: every sequence reads one and writes another
            n = case["batch"]
            s["pool"] = normal(2 * n + 3, D, S, std=0.5)
            lines = torch.randperm(2 * n + 3, generator=gen, device=dev)[:2 * n].to(torch.int32)
            s["read"], s["write"] = lines[:n].contiguous(), lines[n:].contiguous()
            return s
        lens = _lens(case)
        n = len(lens) if lens else case["batch"]
        s["longest"] = max(lens) if lens else case["tokens"]
        s["cu"] = None
        if lens:
            s["cu"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
        s["h0"] = normal(n, D, S, std=0.5) if case["state"] else None
        if op == "train_scan":
            s["dy"] = normal(*lead, D).to(dt)
            s["dht"] = normal(n, D, S, std=0.5) if case["state"] else None
        return s
    if op == "train_conv":
        W = case["width"]
        s["x"] = normal(case["batch"], case["tokens"], D).to(dt)
        s["dy"] = normal(case["batch"], case["tokens"], D).to(dt)
        s["weight"] = normal(D, W, std=W ** -0.5)
        s["bias"] = normal(D, std=0.1)
        lens = _lens(case)
        s["cu"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32) if lens else None
        return s
    shape = (case["batch"], D) if case["positions"] == 1 else (case["batch"], case["positions"], D)
    # a mean that is not zero, and groups of unlike scale
    scale = torch.exp(normal(D, std=0.5))
    s["x"] = (normal(*shape, mean=0.3) * scale).to(dt)
    s["weight"], s["bias"] = normal(D, std=0.1, mean=1.0), normal(D, std=0.1)
    s["gate"] = normal(*shape).to(dt) if case["gate"] else None
    if op == "train_norm":
        s["dy"] = normal(*shape).to(dt)
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


# --- the library's calls --------------------------------------------------------------------

def _run_own(s):
    import gated_deltanet_chunked_02_amd as gdn
    case = s["case"]
    op = case["op"]
    if op in ("scan", "train_scan"):
        common = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True,
                      initial_state=s["h0"], cu_seqlens=s["cu"])
        args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
        y, ht = gdn.selective_scan(*args, **common)
        if op == "scan":
            return dict(y=y, ht=ht)
        dx, ddt, dA, dB, dC, dD, dz, dbias, dh0 = gdn.selective_scan_bwd(
            *args, s["dy"], dht=s["dht"], **common)
        return dict(y=y, ht=ht, dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=dD, dz=dz, dbias=dbias,
                    dh0=dh0)
    if op == "step":
        y = gdn.selective_state_update(
            s["pool"], s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
            dt_bias=s["dt_bias"], dt_softplus=True, cache_indices=s["read"],
            out_indices=s["write"])
        return dict(y=y, pool=s["pool"])
    if op == "train_conv":
        act = "silu" if case["act"] else None
        y = gdn.causal_conv1d(s["x"], s["weight"], s["bias"], cu_seqlens=s["cu"], activation=act)
        dx, dweight, dbias, _ = gdn.causal_conv1d_bwd(
            s["x"], s["weight"], s["dy"], bias=s["bias"], cu_seqlens=s["cu"], activation=act)
        return dict(y=y, dx=dx, dweight=dweight, dbias=dbias)
    act = "silu" if case["act"] else None
    y, mean, rstd = gdn.group_norm(s["x"], case["groups"], s["weight"], s["bias"], eps=1e-5,
                                   activation=act, gate=s["gate"])
    if op == "norm":
        return dict(y=y, mean=mean, rstd=rstd)
    dx, dweight, dbias, dgate = gdn.group_norm_bwd(
        s["dy"], s["x"], case["groups"], mean, rstd, weight=s["weight"], bias=s["bias"],
        activation=act, gate=s["gate"])
    return dict(y=y, mean=mean, rstd=rstd, dx=dx, dweight=dweight, dbias=dbias, dgate=dgate)


# --- the plain form: elementary torch operations in fp32 --------------------------------------

def _run_plain(s):
    op = s["case"]["op"]
    if op in ("scan", "train_scan"):
        return _plain_scan(s)
    if op == "step":
        return _plain_step(s)
    if op == "train_conv":
        return _plain_conv(s)
    return _plain_norm(s)


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _plain_scan(s):
    case, dtype = s["case"], s["x"].dtype
    D, G, S = case["channels"], case["groups"], case["dstate"]
    cu, L = s["cu"], s["longest"]
    A = s["A"].reshape(G, D // G, S)
    if cu is None:
        mask, at = None, None
    else:  # [sequence, position] -> token; padded positions take no step (their dt is zero)
        at = torch.arange(L, device=cu.device)[:, None] + cu[:-1].long()[None, :]
        mask = at < cu[1:].long()[None, :]
        at = torch.where(mask, at, 0)

    def rows(t):  # [L, N, ...] fp32
        return (t.transpose(0, 1) if at is None else t[0][at]).float()

    def back(t):  # the tokens of [L, N, ...], in the inputs' order
        if at is None:
            return t.transpose(0, 1).contiguous()
        out = t.new_empty((case["tokens"],) + t.shape[2:])
        out[at[mask]] = t[mask]
        return out[None]

    x, z = rows(s["x"]), rows(s["z"]) if s["z"] is not None else None
    raw = rows(s["dt"]) + s["dt_bias"]
    step = _softplus(raw)
    if mask is not None:
        step = step * mask[..., None]
    N = x.shape[1]
    heads = lambda t: t.reshape(t.shape[:2] + (G, D // G, 1))  # noqa: E731
    Bm, Cm = rows(s["B"])[:, :, :, None], rows(s["C"])[:, :, :, None]
    train = case["op"] == "train_scan"
    h = torch.zeros(N, G, D // G, S, device=x.device) if s["h0"] is None else \
        s["h0"].reshape(N, G, D // G, S)
    h0 = h
    inner = torch.empty_like(x)
    states = []
    for b in range(0, L, BLOCK):
        d = heads(step[b:b + BLOCK])
        decay = torch.exp(d * A)
        hs = (d * heads(x[b:b + BLOCK])) * Bm[b:b + BLOCK]
        for i in range(hs.shape[0]):
            h = torch.addcmul(hs[i], decay[i], h, out=hs[i])
        inner[b:b + BLOCK] = (hs * Cm[b:b + BLOCK]).sum(-1).reshape(d.shape[0], N, D)
        if train:
            states.append(hs)
    pre = inner + x * s["D"]
    y = pre if z is None else pre * z * torch.sigmoid(z)
    out = dict(y=back(y).to(dtype), ht=h.reshape(N, D, S).clone())
    if not train:
        return out

    dy = rows(s["dy"])
    if mask is not None:
        dy = dy * mask[..., None]
    dz = None
    if z is not None:
        sig = torch.sigmoid(z)
        dz = dy * pre * sig * (1.0 + z * (1.0 - sig))
        dy = dy * z * sig
    dx, dstep = dy * s["D"], torch.empty_like(step)
    dA = torch.zeros_like(A)
    dB = torch.empty(L, N, G, S, device=x.device)
    dC = torch.empty_like(dB)
    carry = torch.zeros_like(h) if s["dht"] is None else s["dht"].reshape(h.shape)
    for k in range(len(states) - 1, -1, -1):
        b = k * BLOCK
        e = min(b + BLOCK, L)
        hs = states[k]
        d, xs, dys = heads(step[b:e]), heads(x[b:e]), heads(dy[b:e])
        decay = torch.exp(d * A)
        g = dys * Cm[b:e]
        g[-1] += carry
        for i in range(e - b - 2, -1, -1):
            torch.addcmul(g[i], decay[i + 1], g[i + 1], out=g[i])
        carry = decay[0] * g[0]
        before = torch.cat([(states[k - 1][-1] if k else h0)[None], hs[:-1]])
        q = g * decay * before
        dA += (q * d).sum((0, 1))
        gB = (g * Bm[b:e]).sum(-1, keepdim=True)
        dstep[b:e] = ((q * A).sum(-1, keepdim=True) + xs * gB).reshape(e - b, N, D)
        dx[b:e] += (d * gB).reshape(e - b, N, D)
        dB[b:e] = (g * (d * xs)).sum(3)
        dC[b:e] = (hs * dys).sum(3)
    if mask is not None:
        dstep = dstep * mask[..., None]
    ddt = dstep * torch.sigmoid(raw)
    out.update(dx=back(dx).to(dtype), ddt=back(ddt).to(dtype), dA=dA.reshape(D, S),
               dB=back(dB).to(dtype), dC=back(dC).to(dtype), dD=(dy * x).sum((0, 1)),
               dz=None if dz is None else back(dz).to(dtype), dbias=ddt.sum((0, 1)),
               dh0=carry.reshape(N, D, S) if s["h0"] is not None else None)
    return out


def _plain_step(s):
    case = s["case"]
    D, G, S, n = case["channels"], case["groups"], case["dstate"], case["batch"]
    heads = lambda t: t.reshape(n, G, D // G, 1)  # noqa: E731
    x = s["x"].float()
    step = _softplus(s["dt"].float() + s["dt_bias"])
    h = s["pool"][s["read"].long()].reshape(n, G, D // G, S)
    h = torch.exp(heads(step) * s["A"].reshape(G, D // G, S)) * h + \
        heads(step * x) * s["B"].float()[:, :, None]
    y = (h * s["C"].float()[:, :, None]).sum(-1).reshape(n, D) + x * s["D"]
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    s["pool"][s["write"].long()] = h.reshape(n, D, S)
    return dict(y=y.to(s["x"].dtype), pool=s["pool"])


def _plain_conv(s):
    case, dtype = s["case"], s["x"].dtype
    W, C = case["width"], case["channels"]
    x, dy = s["x"].float().reshape(-1, C), s["dy"].float().reshape(-1, C)
    n = x.shape[0]
    token = torch.arange(n, device=x.device)
    if s["cu"] is None:
        pos = token % case["tokens"]
    else:
        cu = s["cu"].long()
        pos = token - cu[torch.searchsorted(cu, token, right=True) - 1]
    w = s["weight"]
    reach = [(pos >= j)[:, None] for j in range(W)]  # whether token t - j is of t's sequence

    def shifted(j):  # x[t - j], zero before the sequence
        return torch.roll(x, j, 0) * reach[j]

    u = s["bias"] + sum(w[:, W - 1 - j] * shifted(j) for j in range(W))
    if case["act"]:
        sig = torch.sigmoid(u)
        y, du = u * sig, dy * sig * (1.0 + u * (1.0 - sig))
    else:
        y, du = u, dy
    dx = sum(torch.roll(du * reach[j], -j, 0) * w[:, W - 1 - j] for j in range(W))
    dweight = torch.stack([(du * shifted(W - 1 - i)).sum(0) for i in range(W)], 1)
    shape = s["x"].shape
    return dict(y=y.reshape(shape).to(dtype), dx=dx.reshape(shape).to(dtype), dweight=dweight,
                dbias=du.sum(0))


def _plain_norm(s):
    case, dtype = s["case"], s["x"].dtype
    n, P, C, G = case["batch"], case["positions"], case["channels"], case["groups"]
    x = s["x"].float().reshape(n, P, G, C // G)
    mean = x.mean((1, 3), keepdim=True)
    rstd = torch.rsqrt((x - mean).square().mean((1, 3), keepdim=True) + 1e-5)
    w = s["weight"].reshape(G, C // G)
    hat = (x - mean) * rstd
    u = hat * w + s["bias"].reshape(G, C // G)
    gate = s["gate"].float().reshape(x.shape) if s["gate"] is not None else None
    v = gate if gate is not None else u
    sig = torch.sigmoid(v) if case["act"] else None
    a = v * sig if case["act"] else v
    y = u * a if gate is not None else a
    shape = s["x"].shape
    out = dict(y=y.reshape(shape).to(dtype), mean=mean.reshape(n, G), rstd=rstd.reshape(n, G))
    if case["op"] == "norm":
        return out
    dy = s["dy"].float().reshape(x.shape)
    slope = sig * (1.0 + v * (1.0 - sig)) if case["act"] else torch.ones_like(v)
    dgate = None
    if gate is not None:
        dgate = dy * u * slope
        du = dy * a
    else:
        du = dy * slope
    dhat = du * w
    dx = rstd * (dhat - dhat.mean((1, 3), keepdim=True) -
                 hat * (dhat * hat).mean((1, 3), keepdim=True))
    out.update(dx=dx.reshape(shape).to(dtype), dweight=(du * hat).sum((0, 1)).reshape(C),
               dbias=du.sum((0, 1)).reshape(C),
               dgate=None if dgate is None else dgate.reshape(shape).to(dtype))
    return out


# --- the definition in 64 bits, its gradients by differentiating it ---------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("scan", "train_scan"):
        return _exact_scan(s, case)
    if op == "step":
        return _exact_step(s, case)
    if op == "train_conv":
        return _exact_conv(s, case)
    return _exact_norm(s, case)


def _double(t, grad=False):
    return None if t is None else t.double().contiguous().requires_grad_(grad)


def _silu64(t):
    return t / (1.0 + torch.exp(-t))


def _exact_scan(s, case):
    D, G, S = case["channels"], case["groups"], case["dstate"]
    train = case["op"] == "train_scan"
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0")
    v = {k: _double(s[k], train) for k in names}
    ends = s["cu"].tolist() if s["cu"] is not None else None
    per = D // G
    with torch.set_grad_enabled(train):
        delta = torch.logaddexp(v["dt"] + v["dt_bias"], torch.zeros((), device="cuda",
                                                                    dtype=torch.float64))
        ys, hts = [], []
        if ends is None:
            runs = [[(t.unbind(1)) for t in (delta, v["x"], v["B"], v["C"])]]
            firsts = [v["h0"]]
        else:  # one sequence after another
            cut = [t[0].split([b - a for a, b in zip(ends, ends[1:])])
                   for t in (delta, v["x"], v["B"], v["C"])]
            runs = [[p[i][None].unbind(1) for p in cut] for i in range(len(ends) - 1)]
            firsts = [None if v["h0"] is None else v["h0"][i:i + 1] for i in range(len(runs))]
        for (ds, xs, bs, cs), h in zip(runs, firsts):
            if h is None:
                h = torch.zeros(ds[0].shape[0], D, S, device="cuda", dtype=torch.float64)
            seq = []
            for dl, xt, bt, ct in zip(ds, xs, bs, cs):
                Bt = bt.repeat_interleave(per, 1)
                Ct = ct.repeat_interleave(per, 1)
                h = torch.exp(dl[..., None] * v["A"]) * h + Bt * (dl * xt)[..., None]
                seq.append(torch.matmul(h[:, :, None, :], Ct[..., None])[..., 0, 0])
            ys.append(torch.stack(seq, 1))
            hts.append(h)
        inner = ys[0] if ends is None else torch.cat(ys, 1)
        y = inner + v["D"] * v["x"]
        if v["z"] is not None:
            y = y * _silu64(v["z"])
        ht = hts[0] if ends is None else torch.cat(hts)
        if not train:
            return dict(y=y, ht=ht)
        loss = (y * s["dy"].double()).sum()
        if s["dht"] is not None:
            loss = loss + (ht * s["dht"].double()).sum()
        have = [k for k in names if v[k] is not None]
        g = dict(zip(have, torch.autograd.grad(loss, [v[k] for k in have])))
    return dict(y=y.detach(), ht=ht.detach(), dx=g["x"], ddt=g["dt"], dA=g["A"], dB=g["B"],
                dC=g["C"], dD=g["D"], dz=g.get("z"), dbias=g["dt_bias"], dh0=g.get("h0"))


def _exact_step(s, case):
    D, G, S = case["channels"], case["groups"], case["dstate"]
    v = {k: _double(s[k]) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "pool")}
    per = D // G
    delta = torch.log1p(torch.exp(v["dt"] + v["dt_bias"]))
    h = torch.exp(torch.einsum("bd,ds->bds", delta, v["A"])) * v["pool"][s["read"].long()]
    h = h + v["B"].repeat_interleave(per, 1) * (delta * v["x"])[..., None]
    y = (h * v["C"].repeat_interleave(per, 1)).sum(-1) + v["D"] * v["x"]
    if v["z"] is not None:
        y = y * _silu64(v["z"])
    pool = v["pool"].clone()
    pool[s["write"].long()] = h
    return dict(y=y, pool=pool)


def _exact_conv(s, case):
    W = case["width"]
    x, dy = s["x"].double(), s["dy"].double()
    x.requires_grad_()
    w, bias = _double(s["weight"], True), _double(s["bias"], True)
    lens = _lens(case)
    parts = [x] if lens is None else x.split(lens, 1)
    ys = []
    for p in parts:
        padded = torch.nn.functional.pad(p, (0, 0, W - 1, 0))
        z = bias
        for i in range(W):
            z = z + padded[:, i:i + p.shape[1]] * w[:, i]
        ys.append(_silu64(z) if case["act"] else z)
    y = torch.cat(ys, 1)
    dx, dweight, dbias = torch.autograd.grad((y * dy).sum(), (x, w, bias))
    return dict(y=y.detach(), dx=dx, dweight=dweight, dbias=dbias)


def _exact_norm(s, case):
    n, C, G = case["batch"], case["channels"], case["groups"]
    train = case["op"] == "train_norm"
    x, gate = _double(s["x"], train), _double(s["gate"], train)
    w, bias = _double(s["weight"], train), _double(s["bias"], train)
    f = _silu64 if case["act"] else lambda t: t  # noqa: E731
    with torch.set_grad_enabled(train):
        grouped = x.reshape(n, -1, G, C // G).transpose(1, 2).flatten(2)
        mean = grouped.sum(-1) / grouped.shape[-1]
        var = (grouped ** 2).sum(-1) / grouped.shape[-1] - mean ** 2
        rstd = (var + 1e-5) ** -0.5
        wide = lambda t: t.repeat_interleave(C // G, 1).reshape(  # noqa: E731
            (n,) + (1,) * (x.dim() - 2) + (C,))
        u = (x - wide(mean)) * wide(rstd) * w + bias
        y = u * f(gate) if gate is not None else f(u)
        out = dict(y=y.detach(), mean=mean.detach(), rstd=rstd.detach())
        if train:
            have = [t for t in (x, w, bias, gate) if t is not None]
            g = torch.autograd.grad((y * s["dy"].double()).sum(), have)
            out.update(dx=g[0], dweight=g[1], dbias=g[2], dgate=g[3] if gate is not None else None)
    return out


# --- what a pass cannot do without ------------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, C = case["op"], case["channels"]
    if op in ("scan", "train_scan", "step"):
        G, S = case["groups"], case["dstate"]
        tokens = case["batch"] * (case["tokens"] if op != "step" else 1)
        lens = _lens(case) if op != "step" else None
        n = len(lens) if lens else case["batch"]
        params = 4 * (C * S + 2 * C)
        # x, dt, z, y; B, C; the parameters; exp counted as one operation
        wide = 4 if case["gate"] else 3
        if op == "step":
            # the state read and written; a pool line that no sequence names is not touched
            return dict(bytes=e * tokens * (wide * C + 2 * G * S) + params + 8 * n * C * S,
                        flops=7 * tokens * C * S)
        states = 4 * n * C * S * (2 if case["state"] else 1)
        fwd = dict(bytes=e * tokens * (wide * C + 2 * G * S) + params + states,
                   flops=7 * tokens * C * S)
        if op == "scan":
            return fwd
        # dy in; dx, ddt, dz, dB, dC, the parameters' gradients out; dht in and dh0 out
        more = e * tokens * ((4 if case["gate"] else 3) * C + 2 * G * S) + params + \
            (8 * n * C * S if case["state"] else 0)
        return dict(bytes=fwd["bytes"] + more, flops=fwd["flops"] + 15 * tokens * C * S)
    if op == "train_conv":
        n, W = case["batch"] * case["tokens"], case["width"]
        return dict(bytes=4 * e * n * C + 8 * C * (W + 1), flops=(6 * W + 12) * n * C)
    n = case["batch"] * case["positions"]
    wide = 3 if case["gate"] else 2
    fwd = dict(bytes=e * n * C * wide + 8 * C + 8 * case["batch"] * case["groups"],
               flops=12 * n * C)
    if op == "norm":
        return fwd
    return dict(bytes=fwd["bytes"] + e * n * C * (3 if case["gate"] else 2) + 8 * C,
                flops=30 * n * C)
