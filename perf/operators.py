"""The operators around training and deploying a pruned layer, as a program calls them, and their plain forms.

* 8-bit deployment.  Values are e4m3 with one power-of-two scale (e8m0) for each block of 128: activations have a scale
  for every token and 128 consecutive input channels, weights one for every 128 x 128 block.
  - quant8:        activations to 8 bits, with the layer's input-channel permutation applied on the way
  - quant8_weight: the permuted and N:M-masked weight to 8 bits
  - mm8:           Y = X W^T of two 8-bit operands with their scales
  - linear8:       the deployed layer on plain activations (quant8 and mm8 in one call)
* Training the logits of many layers together.
  - clip:  the 2-norm over all gradients, and every gradient times min(1, max_norm / (norm + 1e-6))
  - adamw: the same factor, applied inside one AdamW update of all layers

`own` false: plain torch operations; true: the library's calls.
"""
import math

import torch

own = False

GROUP = 128          # channels (and weight rows) that share one scale
E4M3_MAX = 448.0
BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
OPT = dict(lr=5e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
STEP = 7             # the 1-based AdamW step that is taken


def listed():
    return [
        # one decoded token through a 7B attention projection
        dict(name="linear8 token 4096x4096", op="linear8", tokens=1, cin=4096, cout=4096, block=64, x=BF16, y=F32),
        # a prompt through the 7B down projection
        dict(name="linear8 prompt 11008x4096", op="linear8", tokens=2048, cin=11008, cout=4096, block=64, x=BF16, y=BF16),
        # a ragged batch of requests on a small layer with odd sizes
        dict(name="mm8 ragged 1120x1000", op="mm8", tokens=333, cin=1120, cout=1000, y=F32),
        # the calibration tokens of a 13B block through its gate projection: the largest product
        dict(name="mm8 calibration 5120x13824", op="mm8", tokens=4096, cin=5120, cout=13824, y=F32),
        # the activations of a 7B layer's calibration batch, permuted in blocks of 64
        dict(name="quant8 activations 2048x4096", op="quant8", tokens=2048, cin=4096, block=64, x=BF16),
        # a few decoded tokens, float32, no permutation, a short last group
        dict(name="quant8 few tokens f32", op="quant8", tokens=5, cin=1120, block=0, x=F32),
        # a 13B down projection after hardening: permuted, pruned 2:4
        dict(name="quant8_weight 5120x13824", op="quant8_weight", cout=5120, cin=13824, block=64, n=2, m=4, x=BF16),
        # a small float32 layer as it is, ragged in both directions
        dict(name="quant8_weight ragged f32", op="quant8_weight", cout=1000, cin=1120, block=0, n=0, m=0, x=F32),
        # the logit gradients of one 4096-channel layer
        dict(name="clip one layer", op="clip", count=1, size=4096 * 64, wide=4096 * 64, odd=0, scale=1e-3, limit=1.0, x=F32),
        # those of all 224 layers of a 7B model
        dict(name="clip 7B model", op="clip", count=224, size=4096 * 64, wide=11008 * 64, odd=0, scale=1e-3, limit=1.0, x=F32),
        # the update of one layer's logits
        dict(name="adamw one layer", op="adamw", count=1, size=4096 * 64, wide=4096 * 64, odd=0, scale=1e-3, limit=1.0, x=F32),
        # the update of all 280 layers of a 13B model
        dict(name="adamw 13B model", op="adamw", count=280, size=5120 * 64, wide=13824 * 64, odd=0, scale=1e-3, limit=1.0, x=F32),
    ]


def _log(rng, lo, hi, mult=1):
    """A multiple of `mult` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / mult)) * mult))


def draw(rng):
    op = rng.choice(["linear8", "linear8", "mm8", "quant8", "quant8_weight", "clip", "adamw"])
    x = rng.choice([BF16, BF16, F32])
    if op in ("clip", "adamw"):
        size = _log(rng, 64, 1 << 20)
        count = _log(rng, 1, max(1, min(300, (96 << 20) // size)))
        odd = rng.choice([0, 0, 1, 3])
        return dict(op=op, count=count, size=size if odd else -(-size // 8) * 8, wide=(size if odd else -(-size // 8) * 8) * rng.choice([1, 2]), odd=odd,
                    scale=rng.choice([1e-6, 1e-3, 1.0]), limit=rng.choice([1.0, 1.0, 1e6]), x=x if op == "clip" else F32)
    block = rng.choice([0, 32, 64, 64, 128, 256])
    mult = max(32, block)
    cin = _log(rng, 256, 13824 // mult * mult, mult)
    cout = _log(rng, 64, 13824, 8)
    if op == "quant8":
        return dict(op=op, tokens=_log(rng, 1, 4096), cin=cin, block=block, x=x)
    if op == "quant8_weight":
        if cin * cout > 5120 * 13824:
            cout = 5120 * 13824 // cin // 8 * 8
        n, m = rng.choice([(0, 0), (2, 4), (2, 4), (4, 8), (1, 4)])
        return dict(op=op, cout=cout, cin=cin, block=block, n=n, m=m, x=x)
    tokens = _log(rng, 1, 4096) if rng.random() < 0.6 else rng.randint(1, 64)
    while tokens * cin * cout > 4096 * 5120 * 13824:
        tokens //= 2
    y = rng.choice([BF16, F32])
    if op == "mm8":
        return dict(op=op, tokens=tokens, cin=cin, cout=cout, y=y)
    return dict(op=op, tokens=tokens, cin=cin, cout=cout, block=block, x=x, y=y)


def groups(n):
    return -(-n // GROUP)


def sizes(case):
    """The lengths of a clip or adamw case's tensors: seven to a model's layer, the last of them wide."""
    return [(case["wide"] if i % 7 == 6 else case["size"]) + (i % 5) * case["odd"] for i in range(case["count"])]


def work(case):
    op = case["op"]
    e = 2 if case.get("x") == BF16 else 4
    if op == "clip":
        n = sum(sizes(case))
        return dict(bytes=2 * n * e + 4, flops=3 * n)
    if op == "adamw":
        n = sum(sizes(case))
        return dict(bytes=28 * n + 4, flops=16 * n)
    cin = case["cin"]
    if op == "quant8":
        t = case["tokens"]
        return dict(bytes=t * cin * (e + 1) + t * groups(cin) + (4 * cin if case["block"] else 0), flops=2 * t * cin)
    cout = case["cout"]
    weight = cout * cin + groups(cout) * groups(cin)
    perm = 4 * cin if case.get("block") else 0
    if op == "quant8_weight":
        return dict(bytes=cout * cin * e + weight + perm + (cout * cin // 8 if case["m"] else 0), flops=2 * cout * cin)
    t, ey = case["tokens"], 2 if case["y"] == BF16 else 4
    x = t * cin + t * groups(cin) if op == "mm8" else t * cin * e + perm
    return dict(bytes=weight + x + t * cout * ey, flops=2 * t * cin * cout)


# --------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _outliers(g, cin):
    """A factor for each channel: one in a hundred stands out, as in trained layers."""
    return torch.where(torch.rand(cin, generator=g, device="cuda") < 0.01, 5.0, 1.0)


def _perm(g, cin, block):
    if not block:
        return None
    return torch.rand(cin // block, block, generator=g, device="cuda").argsort(1).to(torch.int32)


def _mask(g, rows, cols, n, m):
    """Packed bits of a mask that keeps n of every m columns of each row: column j is bit j % 32 of word j / 32."""
    r = torch.rand(rows, cols // m, m, generator=g, device="cuda").argsort(2)
    keep = (r < n).view(rows, cols // 32, 32).to(torch.int64)
    bits = (keep << torch.arange(32, device="cuda")).sum(2)
    return torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)


def _operand8(g, rows, cin, scale_rows, std):
    """An 8-bit operand as a quantiser leaves it: values up to the top of e4m3's range, scales around the data's size."""
    q = (_normal(g, rows, cin) * 110.0).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    near = round(math.log2(std / 110.0)) + 127
    s = torch.randint(near - 1, near + 3, (scale_rows, groups(cin)), generator=g, device="cuda", dtype=torch.uint8)
    return q, s.view(torch.float8_e8m0fnu)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("clip", "adamw"):
        ns = sizes(case)
        dt = DTYPES[case["x"]]
        # the tensors of a model lie one after another in one buffer, as a flat gradient store keeps them
        flat = (_normal(g, sum(ns)) * case["scale"]).to(dt)
        s["g"] = flat
        s["max_norm"] = case["scale"] * case["limit"]      # a limit of 1e6 leaves every gradient as it is
        if op == "clip":
            s["out"] = torch.empty_like(flat)
            if own:
                from learnable_channel_permutation_b200 import binding as b
                s["list"] = b.GradList(list(flat.split(ns)), out=list(s["out"].split(ns)))
            return s
        s["L"] = _normal(g, sum(ns)) * 1e-3
        s["m"] = _normal(g, sum(ns)) * (case["scale"] * 0.1)
        s["v"] = _normal(g, sum(ns)).square() * case["scale"] ** 2
        if own:
            from learnable_channel_permutation_b200 import binding as b
            s["list"] = b.AdamwList(*[list(s[k].split(ns)) for k in ("L", "g", "m", "v")])
            s["opt"] = b.adamw_params(**OPT)
        return s
    cin = case["cin"]
    if op == "quant8_weight":
        s["W"] = (_normal(g, case["cout"], cin) * (0.02 * _outliers(g, cin))).to(DTYPES[case["x"]])
        s["perm"] = _perm(g, cin, case["block"])
        s["mask"] = _mask(g, case["cout"], cin, case["n"], case["m"]) if case["m"] else None
        return s
    if op in ("quant8", "linear8"):
        s["X"] = (_normal(g, case["tokens"], cin) * _outliers(g, cin)).to(DTYPES[case["x"]])
        s["perm"] = _perm(g, cin, case["block"])
    else:
        s["Xq"], s["Xs"] = _operand8(g, case["tokens"], cin, case["tokens"], 1.0)
    if op != "quant8":
        s["Wq"], s["Ws"] = _operand8(g, case["cout"], cin, groups(case["cout"]), 0.02)
    return s


# ------------------------------------------------------------------ plain form

def _permuted(X, perm):
    """Column bB + i of X goes to column bB + perm[b][i]."""
    if perm is None:
        return X
    nb, B = perm.shape
    dst = (perm.long() + torch.arange(nb, device=X.device)[:, None] * B).reshape(-1)
    out = torch.empty_like(X)
    out[:, dst] = X
    return out


def _quantise(blocks, dim):
    """e4m3 values and e8m0 scales of float32 `blocks` that share a scale along `dim`: the smallest power of two that
    brings the block's largest magnitude to at most 448 (1 for a block of zeros; NaN for one with an infinity or NaN)."""
    amax = blocks.abs().amax(dim, keepdim=True)
    frac, e = torch.frexp(amax)                       # amax = frac 2^e with frac in [1/2, 1); 448 = 7/8 * 2^9
    k = (e - 9 + (frac > 0.875).int()).clamp(min=-127)
    k = torch.where(amax == 0, torch.zeros_like(k), k)
    bad = ~torch.isfinite(amax)
    k = torch.where(bad, torch.zeros_like(k), k)
    q = blocks * ((127 - k) << 23).view(torch.float32)   # 2^-k, a normal number for every k in [-127, 120]
    q = torch.where(bad, torch.full_like(q, math.nan), q).to(torch.float8_e4m3fn)
    byte = torch.where(bad, torch.full_like(k, 255), k + 127).to(torch.uint8)
    return q, byte.view(torch.float8_e8m0fnu)


def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[1], 0, rows - x.shape[0]))


def _plain_quant8(X, perm):
    T, cin = X.shape
    G = groups(cin)
    x = _pad(_permuted(X, perm).float(), T, G * GROUP).view(T, G, GROUP)
    q, s = _quantise(x, 2)
    return q.view(T, -1)[:, :cin].contiguous(), s.view(T, G)


def _plain_quant8_weight(W, perm, mask):
    cout, cin = W.shape
    w = _permuted(W, perm).float()
    if mask is not None:
        keep = (mask[:, :, None] >> torch.arange(32, device=W.device, dtype=torch.int32)) & 1
        w = torch.where(keep.view(cout, cin) != 0, w, torch.zeros((), device=W.device))
    R, G = groups(cout), groups(cin)
    w = _pad(w, R * GROUP, G * GROUP).view(R, GROUP, G, GROUP).transpose(1, 2).reshape(R, G, GROUP * GROUP)
    q, s = _quantise(w, 2)
    q = q.view(R, G, GROUP, GROUP).transpose(1, 2).reshape(R * GROUP, G * GROUP)
    return q[:cout, :cin].contiguous(), s.view(R, G)


def _plain_mm8(Xq, Xs, Wq, Ws, y):
    cout, cin = Wq.shape
    x = Xq.float() * Xs.float().repeat_interleave(GROUP, 1)[:, :cin]
    w = Wq.float() * Ws.float().repeat_interleave(GROUP, 0)[:cout].repeat_interleave(GROUP, 1)[:, :cin]
    return (x @ w.t()).to(DTYPES[y])


def _plain_factor(flat, max_norm):
    """The norm and the clipping factor, summed in 64 bits."""
    norm = flat.float().square().sum(dtype=torch.float64).sqrt()
    return norm.float().view(1), (max_norm / (norm + 1e-6)).clamp(max=1.0).float()


def _plain_adamw(s):
    norm, factor = _plain_factor(s["g"], s["max_norm"])
    g = s["g"] * factor
    b1, b2 = OPT["beta1"], OPT["beta2"]
    s["m"].mul_(b1).add_(g * (1 - b1))
    s["v"].mul_(b2).add_(g * g * (1 - b2))
    den = s["v"].sqrt() * (1 / math.sqrt(1 - b2 ** STEP)) + OPT["eps"]
    s["L"].mul_(1 - OPT["lr"] * OPT["weight_decay"]).sub_(s["m"] / den * (OPT["lr"] / (1 - b1 ** STEP)))
    return norm


# ------------------------------------------------------------------------ run

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from learnable_channel_permutation_b200 import binding as b
        if op == "quant8":
            q, sc = b.quant8(s["X"], s["perm"])
            return dict(q=q, scales=sc)
        if op == "quant8_weight":
            q, sc = b.quant8_weight(s["W"], s["perm"], s["mask"])
            return dict(q=q, scales=sc)
        if op == "mm8":
            return dict(Y=b.mm8(s["Xq"], s["Xs"], s["Wq"], s["Ws"], out_dtype=DTYPES[case["y"]]))
        if op == "linear8":
            return dict(Y=b.linear8(s["Wq"], s["Ws"], s["X"], s["perm"], out_dtype=DTYPES[case["y"]]))
        if op == "clip":
            return dict(norm=s["list"].clip(s["max_norm"]), g=s["out"])
        norm = s["list"].run(s["opt"], STEP, s["max_norm"])
        return dict(norm=norm, L=s["L"], m=s["m"], v=s["v"])
    if op == "quant8":
        q, sc = _plain_quant8(s["X"], s["perm"])
        return dict(q=q, scales=sc)
    if op == "quant8_weight":
        q, sc = _plain_quant8_weight(s["W"], s["perm"], s["mask"])
        return dict(q=q, scales=sc)
    if op == "mm8":
        return dict(Y=_plain_mm8(s["Xq"], s["Xs"], s["Wq"], s["Ws"], case["y"]))
    if op == "linear8":
        q, sc = _plain_quant8(s["X"], s["perm"])
        return dict(Y=_plain_mm8(q, sc, s["Wq"], s["Ws"], case["y"]))
    if op == "clip":
        norm, factor = _plain_factor(s["g"], s["max_norm"])
        torch.mul(s["g"].float(), factor, out=s["out"])
        return dict(norm=norm, g=s["out"])
    norm = _plain_adamw(s)
    return dict(norm=norm, L=s["L"], m=s["m"], v=s["v"])


# ---------------------------------------------------------------------- exact

def _power_64(k):
    """2^k in float64, from its bits."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _e4m3_64(x):
    """Nearest e4m3 value of float64 x, ties to even: three fraction bits, no exponent below -6."""
    _, e = torch.frexp(x)
    step = _power_64((e - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _values_64(v, group_max):
    """(e4m3 values, scale) of float64 v given the largest magnitude of every value's block."""
    part, e = torch.frexp(torch.where(group_max > 0, group_max, torch.full_like(group_max, E4M3_MAX)) / E4M3_MAX)
    k = torch.where(part > 0.5, e, e - 1).clamp(min=-127)          # the exponent of the next power of two upwards
    scale = _power_64(k)
    return _e4m3_64(v / scale), scale


def _columns_64(x, perm):
    if perm is None:
        return x
    nb, B = perm.shape
    src = torch.argsort(perm.long(), 1) + torch.arange(nb, device=x.device)[:, None] * B
    return x[:, src.reshape(-1)]


def _rows_64(X, perm):
    x = _columns_64(X.double(), perm)
    top = torch.stack([c.abs().amax(1) for c in x.split(GROUP, 1)], 1)
    q, scale = _values_64(x, top.repeat_interleave(GROUP, 1)[:, : x.shape[1]])
    return q, scale, scale[:, ::GROUP]


def _dequantised_64(q, s, per_row):
    q = q.double()
    col = torch.arange(q.shape[1], device=q.device) // GROUP
    row = torch.arange(q.shape[0], device=q.device)
    return q * s.float().double()[row if per_row else row // GROUP][:, col]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant8":
        q, _, scales = _rows_64(s["X"], s["perm"])
        return dict(q=q, scales=scales)
    if op == "quant8_weight":
        w = _columns_64(s["W"].double(), s["perm"])
        if s["mask"] is not None:
            j = torch.arange(w.shape[1], device=w.device)
            w = w * ((s["mask"].long()[:, j // 32] >> (j % 32)) & 1)
        top = torch.stack([torch.stack([t.abs().max() for t in r.split(GROUP, 1)]) for r in w.split(GROUP, 0)])
        every = top.repeat_interleave(GROUP, 0)[: w.shape[0]].repeat_interleave(GROUP, 1)[:, : w.shape[1]]
        q, scale = _values_64(w, every)
        return dict(q=q, scales=scale[::GROUP, ::GROUP])
    if op in ("mm8", "linear8"):
        if op == "mm8":
            x = _dequantised_64(s["Xq"], s["Xs"], True)
        else:
            q, scale, _ = _rows_64(s["X"], s["perm"])
            x = q * scale
        return dict(Y=torch.einsum("tk,ok->to", x, _dequantised_64(s["Wq"], s["Ws"], False)))
    g = s["g"].double()
    norm = torch.sqrt(torch.dot(g, g)).view(1)
    factor = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    if op == "clip":
        return dict(norm=norm, g=g * factor)
    g = g * factor
    m = OPT["beta1"] * s["m"].double() + (1 - OPT["beta1"]) * g
    v = OPT["beta2"] * s["v"].double() + (1 - OPT["beta2"]) * g ** 2
    mh, vh = m / (1 - OPT["beta1"] ** STEP), v / (1 - OPT["beta2"] ** STEP)
    L = s["L"].double()
    L = L - OPT["lr"] * OPT["weight_decay"] * L - OPT["lr"] * mh / (vh.sqrt() + OPT["eps"])
    return dict(norm=norm, L=L, m=m, v=v)
