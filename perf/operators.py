"""Cases, plain forms and exact values of the operators that train the MoE layer.

Four operators follow one another in a training step of the layer, around its forward and
backward passes:

* ``balance``          counts, load-balancing loss and router z-loss with their gradient;
* ``router_backward``  that gradient taken through the linear router, onto the layer's gradients;
* ``grad_norm``        the global norm of many gradients and the clipping scale;
* ``adamw``            one AdamW step over many tensors, its moments in 32 or in 8 bits.

Every case names its operator in ``op``. Layer shapes are those of this repository's workloads
(``synthetic.py``), or small odd ones.
"""
import math

import torch

own = False

ALPHA, Z_COEF = 1e-2, 1e-3
LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.999, 1e-8, 0.1
MAX_NORM = 1.0
BLOCK = 128           # elements that share a scale where moments are held in 8 bits
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a test-sized batch: what a step costs where only latency counts
        dict(name="balance tiny", op="balance", T=64, N=8, k=2, mask="none", zipf=False, grad=True),
        # evaluation of a padded batch: the loss and the counts without a gradient, odd sizes
        dict(name="balance eval odd", op="balance", T=5001, N=100, k=3, mask="tail", zipf=False,
             grad=False),
        # a training batch of the fine-grained layer, skewed loads, padded sequences
        dict(name="balance fine-grained", op="balance", T=16384, N=256, k=8, mask="tail", zipf=True,
             grad=True),
        # a test-sized layer's router, gradients written
        dict(name="router tiny", op="router_backward", T=64, d=128, N=8, add=False),
        # the 32-expert layer's router at its training batch, added onto the layer's gradients
        dict(name="router 32 experts", op="router_backward", T=16384, d=2880, N=32, add=True),
        # the fine-grained layer's router at its training batch: the largest
        dict(name="router fine-grained", op="router_backward", T=16384, d=7168, N=256, add=True),
        # clipping of a test-sized layer
        dict(name="norm tiny", op="grad_norm", layers=1, N=8, d=128, F=256, glu=True, grads="fp32"),
        # clipping of one 32-expert layer's gradients as the backward pass leaves them (fp32)
        dict(name="norm 32 experts", op="grad_norm", layers=1, N=32, d=2880, F=2880, glu=True,
             grads="fp32"),
        # the update of a test-sized layer, everything in fp32
        dict(name="adamw tiny", op="adamw", layers=1, N=8, d=128, F=256, glu=True, params="fp32",
             grads="fp32", bits=32, step=10, clip=False),
        # many small odd tensors at once (256 of them), moments in 8 bits
        dict(name="adamw 256 tensors 8-bit", op="adamw", layers=64, N=5, d=64, F=64, glu=True,
             params="bf16", grads="bf16", bits=8, step=1000, clip=True),
        # the top-1 layer in mixed precision: bf16 weights with fp32 masters and fp32 moments
        dict(name="adamw top-1 masters", op="adamw", layers=1, N=64, d=1024, F=4096, glu=False,
             params="master", grads="fp32", bits=32, step=1000, clip=True),
        # the same layer in as little memory as it takes: bf16 weights alone, 8-bit moments
        dict(name="adamw top-1 8-bit", op="adamw", layers=1, N=64, d=1024, F=4096, glu=False,
             params="bf16", grads="fp32", bits=8, step=1000, clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "router_backward", "grad_norm", "adamw", "adamw"])
    if op == "balance":
        N = _log(rng, 1, 256)
        return dict(op=op, T=_log(rng, 1, 16384), N=N, k=rng.randint(1, min(8, N)),
                    mask=rng.choice(["none", "tail", "tail", "sparse"]), zipf=rng.random() < 0.5,
                    grad=rng.random() < 0.75)
    if op == "router_backward":
        return dict(op=op, T=_log(rng, 1, 16384), d=64 * _log(rng, 1, 112), N=_log(rng, 1, 256),
                    add=rng.random() < 0.5)
    case = dict(op=op, layers=_log(rng, 1, 24), N=_log(rng, 1, 48), d=64 * _log(rng, 1, 20),
                F=64 * _log(rng, 1, 20), glu=rng.random() < 0.5, grads=rng.choice(["fp32", "bf16"]))
    while sum(_expert_sizes(case)) > 200_000_000:
        case["layers" if case["layers"] > 1 else "N"] //= 2
    if op == "adamw":
        case.update(params=rng.choice(["fp32", "bf16", "master"]), bits=rng.choice([32, 8]),
                    step=_log(rng, 2, 100000), clip=rng.random() < 0.5)
    return case


# ----------------------------------------------------------------------------------- inputs
def _gen(seed, part):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1_000_003 + part)
    return g


def _randn(shape, seed, part, std=1.0):
    return torch.randn(shape, generator=_gen(seed, part), device="cuda").mul_(std)


def _rand(shape, seed, part):
    return torch.rand(shape, generator=_gen(seed, part), device="cuda")


def _prepare_balance(c, seed):
    T, N, k = c["T"], c["N"], c["k"]
    logits = _randn((T, N), seed, 1)
    if c["zipf"]:
        rank = torch.arange(1, N + 1, device="cuda", dtype=torch.float32)
        logits += torch.log_softmax(-1.1 * rank.log(), 0)
    idx = logits.topk(k, dim=1).indices.to(torch.int32)
    mask = None
    if c["mask"] == "sparse":  # nearly all of the batch is padding
        mask = (_rand((T,), seed, 2) < 0.05).to(torch.uint8)
        mask[T // 2] = 1
    elif c["mask"] == "tail":  # sequences of 512 positions, each padded from a length of its own
        lengths = 128 + (_rand((T // 512 + 1,), seed, 2) * 385).long()
        mask = (torch.arange(T, device="cuda") % 512 < lengths.repeat_interleave(512)[:T])
        mask = mask.to(torch.uint8)
    s = dict(logits=logits, idx=idx, mask=mask,
             counts=torch.empty(N, dtype=torch.int32, device="cuda"),
             tokens=torch.empty(1, dtype=torch.int32, device="cuda"),
             prob_mean=torch.empty(N, device="cuda"), loss=torch.empty(3, device="cuda"),
             d_logits=torch.empty(T, N, device="cuda") if c["grad"] else None)
    if own:
        import sparse_mixture_experts_11_b200 as moe
        s["dims"] = moe.make_dims(T, 64, N, k, 64)
        s["ws"] = moe.new_workspace(s["dims"])
    return s


def _prepare_router(c, seed):
    T, d, N = c["T"], c["d"], c["N"]
    # a softmax's gradient, zero on a tenth of the tokens (padding)
    p = torch.softmax(2.0 * _randn((T, N), seed, 1), 1)
    u = _randn((T, N), seed, 2)
    dL = p * (u - (p * u).sum(1, keepdim=True)) / T
    if N == 1:
        dL = u / T
    dL[_rand((T,), seed, 3) < 0.1] = 0
    s = dict(x=_randn((T, d), seed, 4).to(torch.bfloat16), w=_randn((N, d), seed, 5, d ** -0.5),
             d_logits=dL, add=c["add"])
    size = dL.norm()
    # what the layer's own backward pass left there, of the same size as what is added
    s["d_x"] = _randn((T, d), seed, 6) * (size / math.sqrt(T * d))
    s["d_w"] = _randn((N, d), seed, 7) * (size / math.sqrt(N))
    s["d_b"] = _randn((N,), seed, 8) * (size / math.sqrt(N))
    if own:
        import sparse_mixture_experts_11_b200 as moe
        s["dims"] = moe.make_dims(T, d, N, 1, 64)
        s["ws"] = moe.new_router_backward_workspace(s["dims"])
    return s


def _router_sizes(c):
    return [c["N"] * c["d"], c["N"]] * c["layers"]


def _expert_sizes(c):
    rows = 2 * c["F"] if c["glu"] else c["F"]
    return [c["N"] * rows * c["d"], c["N"] * c["d"] * c["F"]] * c["layers"]


def _group(sizes, params, grads, bits, step, N, seed, part):
    """Tensors of one kind, each a part of one buffer that begins at a multiple of BLOCK elements;
    what lies between them is zero."""
    begin, end = [], 0
    for n in sizes:
        begin.append(end)
        end += -(-n // BLOCK) * BLOCK
    # the places that lie between the tensors; each is zeroed below (there are few of them)
    gaps = torch.cat([torch.arange(b + n, b + -(-n // BLOCK) * BLOCK) for b, n in zip(begin, sizes)])
    gaps = gaps.cuda()
    g = dict(sizes=sizes, begin=begin, bits=bits)
    w = _randn((end,), seed, part, 0.02)
    grad = _randn((end,), seed, part + 1, 1e-3)
    for b, n in zip(begin, sizes):
        if N > 4:
            grad[b:b + n // N] = 0  # an expert that no token chose
    w[gaps] = 0
    grad[gaps] = 0
    g["grad"] = grad if grads == "fp32" else grad.to(torch.bfloat16)
    if params is None:
        return g
    g["master"] = w if params == "master" else None
    g["param"] = w if params == "fp32" else w.to(torch.bfloat16)
    m = _randn((end,), seed, part + 2, 2.3e-4)
    r = 1e-3 * (0.5 + _rand((end,), seed, part + 3)) * math.sqrt(1 - BETA2 ** (step - 1))
    m[gaps] = 0
    r[gaps] = 0
    if bits == 32:
        g.update(m=m, v=r.square_(), ms=None, vs=None)
    else:
        for name, scale, t in (("m", "ms", m), ("v", "vs", r)):
            a = t.view(-1, BLOCK).abs().amax(1) / 448
            g[name] = (t.view(-1, BLOCK) / a.clamp(min=1e-30)[:, None]).to(torch.float8_e4m3fn).view(-1)
            g[scale] = a
    return g


def _prepare_tensors(c, seed):
    step = c.get("step", 1)
    s = dict(step=step, adamw=c["op"] == "adamw", seed=seed & M32)
    s["router"] = _group(_router_sizes(c), "fp32" if s["adamw"] else None, "fp32", 32, step, c["N"],
                         seed, 10)
    s["experts"] = _group(_expert_sizes(c), c.get("params"), c["grads"], c.get("bits", 32), step,
                          c["N"], seed, 20)
    # tensors in the order of the layers: router weight, router bias, gate and up, down
    s["router"]["index"] = [4 * (i // 2) + i % 2 for i in range(2 * c["layers"])]
    s["experts"]["index"] = [4 * (i // 2) + 2 + i % 2 for i in range(2 * c["layers"])]
    s["router"]["decay"], s["experts"]["decay"] = 0.0, DECAY
    for g in (s["router"], s["experts"]):
        blocks = torch.tensor([-(-n // BLOCK) for n in g["sizes"]])
        first = (blocks.cumsum(0) - blocks).repeat_interleave(blocks)
        g["at"] = ((torch.arange(int(blocks.sum())) - first) * BLOCK).cuda()
        g["of"] = torch.tensor(g["index"]).repeat_interleave(blocks).cuda()
    s["scale"] = torch.tensor([0.37], device="cuda") if c.get("clip") else None
    s["norm"], s["clip"] = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    if own:
        import sparse_mixture_experts_11_b200 as moe
        every = [None] * (4 * c["layers"])
        for g in (s["router"], s["experts"]):
            for j, b, n in zip(g["index"], g["begin"], g["sizes"]):
                part = lambda t: None if t is None else t[b:b + n]  # noqa: E731,B023
                scales = lambda t: None if t is None else t[b // BLOCK:b // BLOCK + -(-n // BLOCK)]  # noqa: E731,B023
                every[j] = (moe.adamw_tensor(part(g["param"]), part(g["grad"]), part(g["m"]), part(g["v"]),
                                             master=part(g["master"]), m_scale=scales(g["ms"]),
                                             v_scale=scales(g["vs"]), weight_decay=g["decay"])
                            if s["adamw"] else part(g["grad"]))
        if s["adamw"]:
            s["plan"] = moe.adamw_plan(every)
        else:
            s["plan"] = moe.grad_plan(every)
            s["ws"] = moe.new_grad_norm_workspace()
    return s


def prepare(case, seed):
    if case["op"] == "balance":
        s = _prepare_balance(case, seed)
    elif case["op"] == "router_backward":
        s = _prepare_router(case, seed)
    else:
        s = _prepare_tensors(case, seed)
    s["op"] = case["op"]
    return s


# ------------------------------------------------------------------------------ plain forms
def _plain_balance(s):
    L, idx, N = s["logits"], s["idx"], s["logits"].shape[1]
    valid = torch.ones_like(L[:, 0]) if s["mask"] is None else (s["mask"] != 0).float()
    n = valid.sum().clamp(min=1)
    m = L.amax(1, keepdim=True)
    e = (L - m).exp()
    total = e.sum(1, keepdim=True)
    p = e / total * valid[:, None]
    lse = (m + total.log())[:, 0] * valid
    chosen = (idx[:, :, None] == torch.arange(N, device=L.device, dtype=idx.dtype)).sum(1)
    counts = (chosen * (valid != 0)[:, None]).sum(0)
    prob_mean = p.sum(0) / n
    f = counts / n
    balance = ALPHA * N * (f * prob_mean).sum()
    z = Z_COEF * lse.square().sum() / n
    out = dict(counts=counts.to(torch.int32), tokens=valid.sum().to(torch.int32).view(1),
               prob_mean=prob_mean, loss=torch.stack([balance + z, balance, z]))
    if s["d_logits"] is not None:
        inner = f - (p * f).sum(1, keepdim=True)
        out["d_logits"] = p * (ALPHA * N / n * inner + (2 * Z_COEF / n * lse)[:, None])
    return out


def _plain_router(s):
    dL = s["d_logits"]
    d_w, d_x, d_b = dL.t() @ s["x"].float(), dL @ s["w"], dL.sum(0)
    if s["add"]:
        for mine, more in ((s["d_w"], d_w), (s["d_x"], d_x), (s["d_b"], d_b)):
            mine += more
        return dict(d_w=s["d_w"], d_x=s["d_x"], d_b=s["d_b"])
    return dict(d_w=d_w, d_x=d_x, d_b=d_b)


def _plain_norm(s):
    total = s["router"]["grad"].float().square().sum(dtype=torch.float64)
    total = total + s["experts"]["grad"].float().square().sum(dtype=torch.float64)
    norm = total.sqrt().float().view(1)
    return dict(norm=norm, scale=(MAX_NORM / (norm + 1e-6)).clamp(max=1))


def _mix(x):
    """Mixes 32-bit numbers (held in int64): xors of shifts and odd products."""
    x = x ^ (x >> 16)
    x = (x * 0x2F5A6B1D) & M32
    x = x ^ (x >> 15)
    x = (x * 0xB4C3D7A9) & M32
    return x ^ (x >> 16)


def _random(g, seed, step):
    """Two words of random bits for every element, from its place in its tensor, the tensor's
    place in the list, the step and the seed. No tensor here has 2**32 elements or more."""
    key = _mix(_mix((g["of"] * 0x632BE5AB + seed) & M32) + ((step * 0x9E3779B1) & M32) & M32)
    i = g["at"][:, None] + torch.arange(BLOCK, device=key.device)
    h = _mix((i * 0x9E3779B1 + key[:, None]) & M32)
    return h, (h * 0xD1B54A35 + key[:, None]) & M32


def _to_e4m3(x, bits20):
    """Rounds to E4M3 (at most 448) up with the probability of what is cut off."""
    y = x.abs()
    small = y < 2.0 ** -6   # the subnormal codes: one step wide each, like the next eight
    y = torch.where(small, y + 2.0 ** -6, y)
    code = ((y.view(torch.int32) + bits20) >> 20) - (120 << 3) - 8 * small
    return code.clamp(max=126) + 128 * (x < 0)


def _pack_e4m3(code):
    return code.to(torch.uint8).view(torch.float8_e4m3fn).view(-1)


def _plain_group(g, s):
    step, eight = s["step"], g["bits"] == 8
    w = g["master"] if g["master"] is not None else g["param"].float()
    grad = g["grad"].float()
    if s["scale"] is not None:
        grad = grad * s["scale"]
    m, v = g["m"], g["v"]
    if eight:
        m = (m.float().view(-1, BLOCK) * g["ms"][:, None]).view(-1)
        v = (v.float().view(-1, BLOCK) * g["vs"][:, None]).square().view(-1)
    m = BETA1 * m + (1 - BETA1) * grad
    v = BETA2 * v + (1 - BETA2) * grad * grad
    r = v.sqrt()
    w = w * (1 - LR * g["decay"]) - LR / (1 - BETA1 ** step) * m / (r / math.sqrt(1 - BETA2 ** step) + EPS)
    alone = g["param"].dtype == torch.bfloat16 and g["master"] is None
    if eight or alone:
        h, h2 = _random(g, s["seed"], step)
    if eight:
        for name, scale, t, bits in (("m", "ms", m, h & 0xFFFF), ("v", "vs", r, h >> 16)):
            t = t.view(-1, BLOCK)
            top = t.abs().amax(1, keepdim=True)
            flat = top < 2.0 ** -96
            code = _to_e4m3(torch.where(flat, 0, t * (448 / top)), ((bits << 4) + 8).to(torch.int32))
            if name == "v":  # a second moment that is not zero stays so
                code = torch.where((t > 0) & ~flat, code.clamp(min=1), code)
            g[name].copy_(_pack_e4m3(torch.where(flat, 0, code)))
            g[scale].copy_(torch.where(flat, 0, top / 448)[:, 0])
    else:
        g["m"].copy_(m)
        g["v"].copy_(v)
    if alone:
        up = w.view(torch.int32) + (h2 >> 16).to(torch.int32).view(-1)
        g["param"].copy_((up & -65536).view(torch.float32))
    else:
        if g["master"] is not None:
            g["master"].copy_(w)
        g["param"].copy_(w)


def _tensors_out(s):
    return [[g[k] for k in ("param", "master", "m", "v", "ms", "vs") if g[k] is not None]
            for g in (s["router"], s["experts"])]


def run(s):
    if s["op"] == "balance":
        if not own:
            return _plain_balance(s)
        import sparse_mixture_experts_11_b200 as moe
        moe.balance_loss(s["dims"], s["logits"], s["idx"], s["mask"], s["counts"], s["tokens"],
                         s["prob_mean"], s["loss"], s["d_logits"], s["ws"], alpha=ALPHA, z_coef=Z_COEF)
        out = {k: s[k] for k in ("counts", "tokens", "prob_mean", "loss")}
        return out if s["d_logits"] is None else dict(out, d_logits=s["d_logits"])
    if s["op"] == "router_backward":
        if not own:
            return _plain_router(s)
        import sparse_mixture_experts_11_b200 as moe
        moe.router_backward(s["dims"], s["x"], s["w"], s["d_logits"], s["d_x"], s["d_w"], s["d_b"],
                            s["ws"], accumulate=s["add"])
        return dict(d_w=s["d_w"], d_x=s["d_x"], d_b=s["d_b"])
    if s["op"] == "grad_norm":
        if not own:
            return _plain_norm(s)
        import sparse_mixture_experts_11_b200 as moe
        moe.grad_norm(s["plan"], MAX_NORM, s["norm"], s["clip"], s["ws"])
        return dict(norm=s["norm"], scale=s["clip"])
    if own:
        import sparse_mixture_experts_11_b200 as moe
        moe.adamw_step(s["plan"], s["step"], lr=LR, betas=(BETA1, BETA2), eps=EPS, seed=s["seed"],
                       grad_scale=s["scale"])
    else:
        _plain_group(s["router"], s)
        _plain_group(s["experts"], s)
    return _tensors_out(s)


# ------------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "balance":
        T, N, k = c["T"], c["N"], c["k"]
        moved = T * N * 4 * (2 if c["grad"] else 1) + T * k * 4 + 8 * N + 16
        return dict(bytes=moved + (T if c["mask"] != "none" else 0), flops=T * N * (12 if c["grad"] else 6))
    if c["op"] == "router_backward":
        T, N, d = c["T"], c["N"], c["d"]
        outs = (T * d + N * d + N) * 4
        return dict(bytes=T * N * 4 + T * d * 2 + N * d * 4 + outs * (2 if c["add"] else 1),
                    flops=4 * T * N * d + T * N)
    router, experts = sum(_router_sizes(c)), sum(_expert_sizes(c))
    grad = 4 if c["grads"] == "fp32" else 2
    if c["op"] == "grad_norm":
        return dict(bytes=router * 4 + experts * grad, flops=2 * (router + experts))
    weights = dict(fp32=8, bf16=4, master=10)[c["params"]]
    moments = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
    return dict(bytes=router * 28 + int(experts * (grad + weights + moments)),
                flops=16 * (router + experts))


# ------------------------------------------------------------------------- the definition
def _exact_balance(s):
    L, N = s["logits"].double(), s["logits"].shape[1]
    keep = torch.ones(len(L), dtype=torch.bool, device=L.device) if s["mask"] is None else s["mask"].bool()
    n = int(keep.sum())
    counts = torch.bincount(s["idx"][keep].flatten().long(), minlength=N)
    out = dict(counts=None, tokens=None, prob_mean=torch.zeros(N, dtype=torch.float64, device="cuda"),
               loss=torch.zeros(3, dtype=torch.float64, device="cuda"))
    d_logits = torch.zeros_like(L)
    if n:
        R = L[keep].requires_grad_()
        mean = R.softmax(1).mean(0)
        balance = ALPHA * N * torch.dot(counts.double() / n, mean)
        z = Z_COEF * R.logsumexp(1).pow(2).mean()
        d_logits[keep] = torch.autograd.grad(balance + z, R)[0]
        out.update(prob_mean=mean.detach(), loss=torch.stack([balance + z, balance, z]).detach())
    return dict(out, d_logits=d_logits) if s["d_logits"] is not None else out


def _exact_router(s):
    dL = s["d_logits"].double()
    before = {k: s[k].double() if s["add"] else 0 for k in ("d_w", "d_x", "d_b")}
    return dict(d_w=torch.einsum("tn,td->nd", dL, s["x"].double()) + before["d_w"],
                d_x=torch.einsum("tn,nd->td", dL, s["w"].double()) + before["d_x"],
                d_b=torch.einsum("tn->n", dL) + before["d_b"])


def _exact_norm(s):
    norm = torch.linalg.vector_norm(torch.stack(
        [torch.linalg.vector_norm(s[g]["grad"], dtype=torch.float64) for g in ("router", "experts")]))
    return dict(norm=norm.view(1), scale=(MAX_NORM / (norm.view(1) + 1e-6)).clamp(max=1.0))


def _step_up(x, digits, lowest, u):
    """|x| on the grid of `digits` binary digits after the first (none finer than 2**lowest), up
    where the part cut off and u in [0, 1) make one step."""
    e = torch.frexp(x)[1].double() - 1
    grid = torch.exp2(torch.clamp(e - digits, min=float(lowest)))
    return torch.floor(x.abs() / grid + u) * grid * torch.sign(x)


def _exact_group(g, s):
    t, scale = s["step"], 1.0 if s["scale"] is None else s["scale"].double()
    grad = g["grad"].double() * scale
    m, v = g["m"].double(), g["v"].double()
    if g["bits"] == 8:
        m = m * g["ms"].double().repeat_interleave(BLOCK)
        v = (v * g["vs"].double().repeat_interleave(BLOCK)).pow(2)
    m += (1 - BETA1) * (grad - m)
    v += (1 - BETA2) * (grad.pow_(2) - v)
    del grad
    w = (g["param"] if g["master"] is None else g["master"]).double()
    w -= LR * g["decay"] * w
    w -= LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt_() + EPS)
    bits = None
    if g["bits"] == 8 or (g["master"] is None and g["param"].dtype == torch.bfloat16):
        bits = _random(g, s["seed"], t)
    out = []
    if g["param"].dtype == torch.bfloat16 and g["master"] is None:
        out.append(_step_up(w, 7, -133, (bits[1] >> 16).view(-1).double() / 65536))
    else:
        out.append(w)
    if g["master"] is not None:
        out.append(w)
    if g["bits"] == 32:
        return out + [m, v]
    codes, scales = [], []
    for x, b in ((m, bits[0] & 0xFFFF), (v.sqrt_(), bits[0] >> 16)):
        top = x.view(-1, BLOCK).abs().amax(1)
        top = torch.where(top < 2.0 ** -96, 0, top)
        rel = torch.where(top[:, None] > 0, x.view(-1, BLOCK) * 448 / top[:, None], 0).view(-1)
        c = _step_up(rel, 3, -9, (b.view(-1).double() * 16 + 8) / 2 ** 20).clamp(-448, 448)
        if codes:
            c = torch.where(rel > 0, c.clamp(min=2.0 ** -9), c)
        codes.append(c)
        scales.append(top / 448)
    return out + codes + scales


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "balance":
        return _exact_balance(s)
    if s["op"] == "router_backward":
        return _exact_router(s)
    if s["op"] == "grad_norm":
        return _exact_norm(s)
    return [_exact_group(s["router"], s), _exact_group(s["experts"], s)]
