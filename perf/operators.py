"""Operators of the fine-tuning step, as cases to measure.

Two families: the AdamW step over many tensors at once (FP32 or 8-bit states, with the
global gradient norm that clips it), and the low-rank adapters of many requests at once
beside a shared projection (forward for serving, forward and backward for training).

``run`` computes each in its plain form (elementary torch operations in 32 bits) or,
where ``own`` is true, through the package.  The numerics of both are those of
``include/qf.h``.

Sizes: the projections of ``workloads`` (hidden 4096, K/V 1024, gate/up 14336, the MoE
experts' 768 x 2048) and generic ragged ones.
"""
import random

import torch

own = False

DEV = "cuda"
BLOCK = 256             # elements behind one scale of the 8-bit states
E4M3_MAX = 448.0
LR, BETA1, BETA2, EPS, DECAY = 2e-4, 0.9, 0.95, 1e-8, 0.1
STEP = 1000             # the step number: far enough in that both moments are warm
MAX_NORM = 1.0
TIED = "16777216*1,4194304*2,58720256*2"      # Q; K, V; gate, up
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # One attention layer's rank-16 adapter factors (A and B of Q, K, V, O): the smallest
        # step, where the number of launches counts.
        {"name": "adamw_adapters", "op": "adamw", "sizes": "65536*6,16384*2", "bits": 32,
         "p": "bf16", "g": "bf16", "clip": True, "copy": False, "amax": False},
        # Full-parameter training of a layer's tied projections: FP32 masters, FP32 states, the
        # BF16 copy for the next forward pass and the tie groups' new amax.
        {"name": "adamw_layer_32", "op": "adamw", "sizes": TIED, "bits": 32,
         "p": "f32", "g": "bf16", "clip": False, "copy": True, "amax": True},
        # The same layer with 8-bit states and no copy (the fake-quant pass reads FP32).
        {"name": "adamw_layer_8", "op": "adamw", "sizes": TIED, "bits": 8,
         "p": "f32", "g": "bf16", "clip": False, "copy": False, "amax": True},
        # 48 experts of an MoE layer, three matrices each, clipped by the global norm.
        {"name": "adamw_experts_32", "op": "adamw", "sizes": "1572864*144", "bits": 32,
         "p": "f32", "g": "f32", "clip": True, "copy": False, "amax": False},
        # Norm weights, biases and odd-sized leftovers beside one matrix: ragged ends.
        {"name": "adamw_ragged_8", "op": "adamw",
         "sizes": "4096*24,1*3,257*5,12289*4,100003*3,1048577*2,16777215*1", "bits": 8,
         "p": "f32", "g": "f32", "clip": False, "copy": True, "amax": False},
        # One token of one request: the latency of decoding with an adapter.
        {"name": "lora_one_token", "op": "lora", "tokens": 1, "requests": 1, "cols": 4096,
         "rows": 4096, "adapters": 1, "rank": "16", "bare": 0},
        # A decoding batch: 64 requests of one token, 24 adapters of mixed ranks, some requests
        # without one.
        {"name": "lora_decode", "op": "lora", "tokens": 64, "requests": 64, "cols": 4096,
         "rows": 14336, "adapters": 24, "rank": "8,16,64", "bare": 5},
        # Prompts and decoding tokens in one batch, ragged lengths, the down projection.
        {"name": "lora_prefill", "op": "lora", "tokens": 8191, "requests": 37, "cols": 14336,
         "rows": 4096, "adapters": 11, "rank": "16,32", "bare": 4},
        # A training step of one adapter on the gate projection: forward and backward.
        {"name": "lora_train", "op": "lora_train", "tokens": 8192, "requests": 1, "cols": 4096,
         "rows": 14336, "adapters": 1, "rank": "16", "bare": 0},
        # Several adapters trained side by side on the query projection, ragged sequences.
        {"name": "lora_train_many", "op": "lora_train", "tokens": 16381, "requests": 29,
         "cols": 4096, "rows": 4096, "adapters": 8, "rank": "64,8,20", "bare": 3},
        # A short step of an expert-sized projection.
        {"name": "lora_train_short", "op": "lora_train", "tokens": 517, "requests": 3,
         "cols": 2048, "rows": 768, "adapters": 2, "rank": "32", "bare": 0},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    """AdamW: 1 to 200 tensors of 1 to 2^25 elements, at most 2^27 in all.  Adapters: 1 to
    16384 tokens, 1 to 64 requests (each token its own in a decoding batch), 256 to 14336
    columns (multiples of 16) and rows (multiples of 8), 1 to 24 adapters, ranks 1 to 128."""
    if rng.random() < 0.45:
        kinds, left, parts = rng.randint(1, 5), 1 << 27, []
        for _ in range(kinds):
            size = _log(rng, 1, 1 << 25)
            if rng.random() < 0.5:
                size = max(64, size // 64 * 64)
            count = max(1, min(_log(rng, 1, 40), left // size))
            left = max(1, left - size * count)
            parts.append("%d*%d" % (min(size, left), count) if size > left else "%d*%d" % (size, count))
        p = rng.choice(["f32", "f32", "bf16"])
        return {"op": "adamw", "sizes": ",".join(parts), "bits": rng.choice([8, 32]), "p": p,
                "g": rng.choice(["f32", "bf16"]), "clip": rng.random() < 0.5,
                "copy": p == "f32" and rng.random() < 0.5, "amax": rng.random() < 0.5}
    cols, rows = _log(rng, 16, 896) * 16, _log(rng, 32, 1792) * 8
    ranks = ",".join(str(rng.choice([1, 4, 8, 12, 16, 16, 32, 64, _log(rng, 1, 128)]))
                     for _ in range(rng.randint(1, 3)))
    train = rng.random() < 0.45
    if not train and rng.random() < 0.4:                      # decoding: one token a request
        tokens = requests = _log(rng, 1, 256)
    else:
        tokens = _log(rng, 1, 8192 if train else 16384)
        requests = min(tokens, _log(rng, 1, 64))
    adapters = _log(rng, 1, 24)
    return {"op": "lora_train" if train else "lora", "tokens": tokens, "requests": requests,
            "cols": cols, "rows": rows, "adapters": adapters, "rank": ranks,
            "bare": rng.randint(0, requests // 4)}


# ---------------------------------------------------------------- shapes of a case

def _sizes(case):
    pairs = [s.split("*") for s in case["sizes"].split(",")]
    return [int(n) for n, count in pairs for _ in range(int(count))]


def _ranks(case):
    have = [int(r) for r in case["rank"].split(",")]
    return [have[i % len(have)] for i in range(case["adapters"])]


def _requests(case):
    """The requests' lengths and adapters (-1: none), the same for every seed."""
    t, r, n = case["tokens"], case["requests"], case["adapters"]
    rng = random.Random("%d %d %d" % (t, r, n))
    cuts = sorted(rng.sample(range(1, t), r - 1)) if r > 1 else []
    lengths = [b - a for a, b in zip([0] + cuts, cuts + [t])]
    adapters = [-1] * case["bare"] + [rng.randrange(n) for _ in range(r - case["bare"])]
    rng.shuffle(adapters)
    return lengths, adapters


def work(case):
    """Each input once, each output once."""
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        p, g = (4 if case[k] == "f32" else 2 for k in ("p", "g"))
        states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        per = 2 * p + g + states + (2 if case["copy"] else 0)
        return {"bytes": n * per, "flops": n * (18 + (2 if case["clip"] else 0))}
    lengths, adapters = _requests(case)
    k, n, ranks = case["cols"], case["rows"], _ranks(case)
    live = sum(length for length, a in zip(lengths, adapters) if a >= 0)
    rank_tokens = sum(length * ranks[a] for length, a in zip(lengths, adapters) if a >= 0)
    used = sum(ranks[a] for a in set(a for a in adapters if a >= 0))
    factors = 2 * used * (k + n)
    total = 4 * case["tokens"] + factors + live * (2 * k + 4 * n)          # x; y read, written
    flops = 2 * rank_tokens * (k + n)
    if case["op"] == "lora_train":
        total += factors + live * (2 * k + 2 * n + 4 * k)                   # x, gy; gx read, written
        total += 2 * sum(ranks) * (k + n)                                   # the factors' gradients
        flops += 4 * rank_tokens * (k + n)
    return {"bytes": max(total, 1), "flops": flops}


# ---------------------------------------------------------------- inputs

def _padded(sizes):
    return [(n + BLOCK - 1) // BLOCK * BLOCK for n in sizes]


def _views(flat, sizes):
    out, at = [], 0
    for n, room in zip(sizes, _padded(sizes)):
        out.append(flat[at:at + n])
        at += room
    return out


def _encode(x, lift):
    """Blocks of 256 in E4M3 with an FP32 scale each (see ``_adamw_plain``)."""
    x = x.view(-1, BLOCK)
    scale = x.abs().amax(1, keepdim=True) / x.new_full((1, 1), E4M3_MAX)
    scale = torch.where(scale < 2.0 ** -126, 0.0, scale)
    inv = torch.where(scale == 0, 0.0, 1.0 / scale)
    codes = (x * inv).to(torch.float8_e4m3fn).view(torch.uint8)
    if lift:      # a positive second moment keeps the smallest code above zero
        codes = torch.where((codes == 0) & (x > 0) & (scale > 0), 1, codes).to(torch.uint8)
    return codes.view(-1), scale.view(-1)


def _decode(codes, scale):
    return codes.view(torch.float8_e4m3fn).float().view(-1, BLOCK) * scale.view(-1, 1)


def _prepare_adamw(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    sizes = _sizes(case)
    room = sum(_padded(sizes))
    live = torch.zeros(room, dtype=torch.bool, device=DEV)
    ends = torch.tensor([[a, a + n] for a, n in zip(_starts(sizes), sizes)], device=DEV)
    edge = torch.zeros(room + 1, dtype=torch.int32, device=DEV)
    edge.index_add_(0, ends[:, 0], torch.ones(len(sizes), dtype=torch.int32, device=DEV))
    edge.index_add_(0, ends[:, 1], -torch.ones(len(sizes), dtype=torch.int32, device=DEV))
    live = edge.cumsum(0)[:room] > 0

    def normal(std):
        x = torch.empty(room, device=DEV).normal_(0.0, std, generator=gen)
        return x.mul_(live)

    p = normal(0.02).to(TYPES[case["p"]])
    # gradients: most of them small, a few entries (the rows of rare tokens) zero throughout
    g = normal(1e-3)
    g.mul_(torch.rand(room, device=DEV, generator=gen) > 0.01)
    g = g.to(TYPES[case["g"]])
    m, r = normal(3e-4), normal(1e-3).abs_()
    s = {"case": case, "sizes": sizes, "p": p, "g": g}
    if case["bits"] == 32:
        s["m"], s["v"] = m, r.square_()
    else:
        s["m"], s["ms"] = _encode(m, False)
        s["v"], s["vs"] = _encode(r, True)
    s["w"] = torch.zeros(room, dtype=torch.bfloat16, device=DEV) if case["copy"] else None
    s["amax"] = torch.zeros(2, device=DEV) if case["amax"] else None
    s["norm"] = torch.zeros(2, device=DEV) if case["clip"] else None
    return s


def _starts(sizes):
    at, out = 0, []
    for n in _padded(sizes):
        out.append(at)
        at += n
    return out


def _groups(sizes):
    """The first three tensors share one scale, the rest another."""
    return [0 if i < 3 else 1 for i in range(len(sizes))]


def _prepare_lora(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    t, k, n, ranks = case["tokens"], case["cols"], case["rows"], _ranks(case)

    def normal(rows, cols, std):
        return torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV).normal_(
            0.0, std, generator=gen)

    x = normal(t, k, 1.0)
    x[:, :: max(1, k // 64)] *= 8                             # a few loud channels
    lengths, adapters = _requests(case)
    index = torch.repeat_interleave(torch.tensor(adapters, dtype=torch.int32),
                                    torch.tensor(lengths)).to(DEV)
    s = {"case": case, "x": x, "y": normal(t, n, 1.0), "index": index,
         "adapters": [(normal(n, r, 0.05), normal(r, k, k ** -0.5), 16.0 / (8 + r))
                      for r in ranks]}
    if case["op"] == "lora_train":
        s["gy"], s["gx"] = normal(t, n, 1e-3), normal(t, k, 2e-4)
    return s


def prepare(case, seed):
    return _prepare_adamw(case, seed) if case["op"] == "adamw" else _prepare_lora(case, seed)


# ---------------------------------------------------------------- plain forms

def _adamw_plain(s):
    """p, m and v of one step.  Decided in binary32, one rounding per operation, so that the
    8-bit codes next to a rounding border are decided alike everywhere."""
    case = s["case"]
    g = s["g"].float()
    if case["clip"]:
        norm = s["g"].double().square().sum().sqrt()
        s["norm"].copy_(torch.stack([norm, torch.clamp(MAX_NORM / norm, max=1.0)]))
        g = g * s["norm"][1]
    if case["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m = _decode(s["m"], s["ms"]).view(-1)
        r = _decode(s["v"], s["vs"]).view(-1)
        v = r * r
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    root = v.sqrt()
    denom = root * ((1 - BETA2 ** STEP) ** -0.5) + EPS
    p = s["p"].float() * (1 - LR * DECAY) - (m / denom) * (LR / (1 - BETA1 ** STEP))
    s["p"].copy_(p)
    if case["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        for name, x, lift in (("m", m, False), ("v", root, True)):
            codes, scale = _encode(x, lift)
            s[name].copy_(codes)
            s[name + "s"].copy_(scale)
    if case["copy"]:
        s["w"].copy_(s["p"])
    if case["amax"]:
        first = sum(_padded(s["sizes"][:3]))
        s["amax"].copy_(torch.stack([s["p"][:first].abs().max().float(),
                                     s["p"][first:].abs().max().float() if first < s["p"].numel()
                                     else s["amax"].new_zeros(())]))


def _adamw_outputs(s):
    out = {k: s[k] for k in ("p", "w", "amax", "norm") if s[k] is not None}
    if s["case"]["bits"] == 32:
        out["m"], out["v"] = s["m"], s["v"]
    else:      # the values that the codes stand for: m, and the root of v
        out["m"], out["root_v"] = _decode(s["m"], s["ms"]), _decode(s["v"], s["vs"])
    return out


def _lora_plain(s):
    """All adapters as one of their summed rank; each token keeps its own columns."""
    case, index = s["case"], s["index"].long()
    ranks = torch.tensor(_ranks(case), device=DEV)
    owner = torch.repeat_interleave(torch.arange(case["adapters"], device=DEV), ranks)
    scale = torch.tensor([a[2] for a in s["adapters"]], device=DEV)[owner]
    b = torch.cat([a[0] for a in s["adapters"]], 1).float()
    a = torch.cat([a[1] for a in s["adapters"]], 0).float()
    mine = torch.where(index.view(-1, 1) == owner, scale, 0.0)
    x = s["x"].float()
    u = x @ a.t() * mine
    s["y"].copy_(s["y"].float() + u @ b.t())
    if case["op"] == "lora":
        return s["y"]
    gy = s["gy"].float()
    v = gy @ b * mine
    s["gx"].copy_(s["gx"].float() + v @ a)
    ga = (v.t() @ x).bfloat16()
    gb = (gy.t() @ u).bfloat16()
    return {"y": s["y"], "gx": s["gx"], "ga": list(ga.split(_ranks(case), 0)),
            "gb": [w.contiguous() for w in gb.split(_ranks(case), 1)]}


def _adamw_own(s):
    """The calls are marshalled once, as a training loop does: the buffers stay."""
    import fp4_fake_quant_b200 as qf
    case = s["case"]
    if "call" not in s:
        sizes = s["sizes"]
        views = {k: _views(s[k], sizes) for k in ("p", "g", "m", "v")}
        more = {}
        if case["bits"] == 8:
            at = [[a // BLOCK, (a + room) // BLOCK] for a, room in zip(_starts(sizes), _padded(sizes))]
            more = {"m_scales": [s["ms"][i:j] for i, j in at], "v_scales": [s["vs"][i:j] for i, j in at]}
        if case["copy"]:
            more["copies"] = _views(s["w"], sizes)
        if case["amax"]:
            more["groups"], more["group_amax"] = _groups(sizes), s["amax"]
        if case["clip"]:
            s["norm_call"] = qf.prepare_grad_norm(views["g"], s["norm"], max_norm=MAX_NORM,
                                                  workspace=qf.alloc_grad_norm_workspace(DEV))
            more["grad_scale"] = s["norm"][1:]
        s["call"] = qf.prepare_adamw(views["p"], views["g"], views["m"], views["v"], lr=LR,
                                     betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, **more)
    if case["clip"]:
        s["norm_call"]()
    s["call"](STEP)


def _lora_own(s):
    import fp4_fake_quant_b200 as qf
    case = s["case"]
    train = case["op"] == "lora_train"
    if "u" not in s:
        one = case["adapters"] == 1 and not case["bare"]       # every token has the adapter
        s["plan"] = None if one else qf.alloc_lora_plan(case["tokens"], case["adapters"], DEV)
        s["u"] = qf.alloc_lora_u(case["tokens"], s["adapters"])
        if not one:
            s["plan_call"] = qf.prepare_lora_plan(s["index"], case["adapters"], s["plan"])
        s["call"] = qf.prepare_lora_apply(s["x"], s["adapters"], s["y"], s["u"], plan=s["plan"])
        if train:
            s["ga"] = [torch.empty_like(a) for _, a, _ in s["adapters"]]
            s["gb"] = [torch.empty_like(b) for b, _, _ in s["adapters"]]
            s["back"] = qf.prepare_lora_apply_backward(
                s["x"], s["gy"], s["adapters"], s["u"], s["gx"], s["ga"], s["gb"],
                plan=s["plan"], workspace=qf.alloc_lora_workspace(case["tokens"], s["adapters"]))
    if s["plan"] is not None:
        s["plan_call"]()
    s["call"]()
    if not train:
        return s["y"]
    s["back"]()
    return {"y": s["y"], "gx": s["gx"], "ga": s["ga"], "gb": s["gb"]}


def run(state):
    if state["case"]["op"] == "adamw":
        _adamw_own(state) if own else _adamw_plain(state)
        return _adamw_outputs(state)
    return _lora_own(state) if own else _lora_plain(state)


# ---------------------------------------------------------------- from the definition

def _adamw_exact(case, seed):
    s = _prepare_adamw(case, seed)
    n = s["p"].numel()
    out = {k: torch.empty(n, dtype=torch.float64, device=DEV) for k in ("p", "m", "v")}
    norm = sum(float(g.double().square().sum()) for g in s["g"].split(1 << 24)) ** 0.5
    scale = min(1.0, MAX_NORM / norm) if case["clip"] and norm > 0 else 1.0
    for at in range(0, n, 1 << 24):
        cut = slice(at, min(n, at + (1 << 24)))
        if case["bits"] == 32:
            m, v = s["m"][cut].double(), s["v"][cut].double()
        else:
            rows = slice(cut.start // BLOCK, cut.stop // BLOCK)
            m, v = (s[k][cut].view(torch.float8_e4m3fn).double().view(-1, BLOCK)
                    * s[k + "s"][rows].double().view(-1, 1) for k in ("m", "v"))
            m, v = m.view(-1), v.view(-1).square()
        g = s["g"][cut].double() * scale
        m = torch.lerp(g, m, BETA1)
        v = torch.lerp(g.square(), v, BETA2)
        step = (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)).sqrt() + EPS) \
            + DECAY * s["p"][cut].double()
        out["p"][cut], out["m"][cut], out["v"][cut] = s["p"][cut].double() - LR * step, m, v
    if case["copy"]:
        out["w"] = out["p"]
    if case["amax"]:
        # of the weights as they are kept: rounding to their type keeps the order
        first, p = sum(_padded(s["sizes"][:3])), out["p"].to(TYPES[case["p"]]).double()
        out["amax"] = torch.stack([p[:first].abs().max(), p[first:].abs().max()
                                   if first < n else p.new_zeros(())])
    if case["clip"]:
        out["norm"] = torch.tensor([norm, scale], dtype=torch.float64)
    if case["bits"] == 8:
        # what an 8-bit code stands for jumps by a sixteenth at each rounding border, and the
        # definition decides on which side a value is in 32 bits: there is no value in 64
        out["m"] = out["root_v"] = None
        del out["v"]
    return out


def _lora_exact(case, seed):
    s = _prepare_lora(case, seed)
    if sum(_ranks(case)) * case["tokens"] * (case["cols"] + case["rows"]) > 4e12:
        return None
    train = case["op"] == "lora_train"
    y = s["y"].double()
    gx = s["gx"].double() if train else None
    gas, gbs = [], []
    for i, (b, a, scale) in enumerate(s["adapters"]):
        rows = (s["index"] == i).nonzero().view(-1)
        a, b, x = a.double(), b.double(), s["x"][rows].double()
        y[rows] += scale * ((x @ a.t()) @ b.t())
        if train:
            gy = s["gy"][rows].double()
            gx[rows] += scale * ((gy @ b) @ a)
            gas.append(scale * (gy @ b).t() @ x)
            gbs.append(scale * gy.t() @ (x @ a.t()))
    return {"y": y, "gx": gx, "ga": gas, "gb": gbs} if train else y


def exact(case, seed):
    return _adamw_exact(case, seed) if case["op"] == "adamw" else _lora_exact(case, seed)
