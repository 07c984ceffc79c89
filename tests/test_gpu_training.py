"""The training operators on the GPU against the float64 oracle (oracle/moe_training.py).

Tolerances, in units of u = 2^-24 (half a step of fp32):
* balance loss: a probability is exp(L - max) / sum. The difference's rounding gives exp a relative
  error of |L - max| u (logits here span less than 40), expf is within 2 steps, the sum over N adds
  at most 13 roundings and the division 2: below 60 u for numerator and denominator together.
  Summing T probabilities adds at most 100 roundings in the kernel's order. PROB = 200 u.
  A gradient is p times a difference of terms: its error is held to 200 u of the sum of their
  magnitudes. The logsumexp has |lse| u + 60 u absolute, squared in z.
* router backward: a sum of n products in fp32 is within (n + 8) u of the sum of the magnitudes, in
  whatever order; on tensor cores the three-term operands leave out products below 2^-24 of
  their factors (3 of them: 6 u more) and an addition may truncate (2 u). BOUND = (2 n + 32) u.
* AdamW: m' has 3 roundings, v' 4; the update's square root and quotient are approximations within 2
  steps each, 16 u in all, and p' rounds twice more.
"""
import numpy as np
import pytest
import torch

import oracle
import sparse_mixture_experts_11_b200 as moe
import synthetic
from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(*shape, seed=0, std=1.0):
    return torch.randn(shape, generator=gen(seed), device="cuda") * std


# ---------------------------------------------------------------- balance loss
def run_balance(L, idx, mask, alpha=0.01, z=0.001, d_loss=None, grad=True, ws=None):
    T, N = L.shape
    k = idx.shape[1]
    dims = moe.make_dims(T, 64, N, k, 64)
    ws = moe.new_workspace(dims) if ws is None else ws
    guard = 8  # rows behind the gradient that must stay
    d = torch.full((T + guard, N), 7.0, device="cuda")
    out = dict(counts=torch.full((N,), -1, dtype=torch.int32, device="cuda"),
               n=torch.full((1,), -1, dtype=torch.int32, device="cuda"),
               pm=torch.full((N,), float("nan"), device="cuda"), loss=torch.full((3,), float("nan"), device="cuda"))
    moe.balance_loss(dims, L, idx, mask, out["counts"], out["n"], out["pm"], out["loss"],
                     d[:T] if grad else None, ws, alpha=alpha, z_coef=z, d_loss=d_loss)
    torch.cuda.synchronize()
    assert bool((d[T:] == 7.0).all())
    assert grad or bool((d == 7.0).all())
    out["d"] = d[:T]
    return out


def check_balance(L, idx, mask, alpha=0.01, z=0.001, d_loss=1.0, out=None):
    want = oracle.balance_loss(H.f64(L), idx.cpu().numpy(), None if mask is None else mask.cpu().numpy(),
                               alpha, z, d_loss)
    N = L.shape[1]
    assert np.array_equal(out["counts"].cpu().numpy(), want["counts"])
    assert int(out["n"]) == want["n_tokens"]
    np.testing.assert_allclose(H.f64(out["pm"]), want["prob_mean"], rtol=200 * U, atol=1e-30)
    # the output is fp32: a lse^2 / n past 3.4e38 (a counted row of the type's lowest value has
    # lse^2 = 1.2e77) is infinite there, which is the expected value rounded to fp32
    with np.errstate(over="ignore"):
        want_loss = want["loss"].astype(np.float32).astype(np.float64)
    np.testing.assert_allclose(H.f64(out["loss"]), want_loss, rtol=500 * U, atol=1e-30)
    n = max(1, want["n_tokens"])
    f = want["counts"] / n
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        Ld = H.f64(L)
        keep = np.ones(len(Ld), bool) if mask is None else mask.cpu().numpy() != 0
        p = np.zeros_like(Ld)
        lse = np.zeros(len(Ld))
        rows = keep & np.isfinite(Ld).any(1)
        e = np.exp(Ld[rows] - Ld[rows].max(1, keepdims=True))
        p[rows] = e / e.sum(1, keepdims=True)
        lse[rows] = Ld[rows].max(1) + np.log(e.sum(1))
    size = abs(d_loss) * p * (alpha * N / n * (f + (p @ f)[:, None]) + (2 * z / n * (np.abs(lse) + 1))[:, None])
    err = np.abs(H.f64(out["d"]) - want["d_logits"])
    assert (err <= 200 * U * size + 1e-37).all(), float((err / (size + 1e-37)).max() / U)


@pytest.mark.parametrize("T,N,k,masked", [
    (1, 1, 1, False), (1, 256, 8, False), (2, 7, 3, True), (64, 8, 2, False), (65, 8, 2, True), (33, 16, 4, True),
    (127, 12, 5, True), (129, 20, 2, False), (1000, 100, 3, True), (512, 64, 8, True), (513, 64, 8, True),
    (300, 33, 1, False), (300, 65, 2, True), (700, 129, 8, True), (4099, 255, 8, True), (2500, 128, 4, True),
    (4096, 64, 1, False), (4097, 64, 1, True), (16384, 256, 8, True), (40000, 3, 2, True), (9000, 9, 8, False)])
def test_balance_loss_matches_oracle(T, N, k, masked):
    L = randn(T, N, seed=T + N, std=3.0)
    idx = L.topk(k, 1).indices.to(torch.int32)
    mask = (torch.rand(T, generator=gen(T), device="cuda") < 0.7).to(torch.uint8) * 3 if masked else None
    out = run_balance(L, idx, mask)
    check_balance(L, idx, mask, out=out)
    again = run_balance(L, idx, mask)
    for key in out:
        assert torch.equal(out[key], again[key]), key
    plain = run_balance(L, idx, mask, grad=False)
    for key in ("counts", "n", "pm", "loss"):
        assert torch.equal(out[key], plain[key]), key


@pytest.mark.parametrize("T,N", [(50, 8), (6000, 37)])
def test_balance_loss_every_token_masked(T, N):
    L = torch.full((T, N), float("nan"), device="cuda")
    idx = torch.zeros((T, 2), dtype=torch.int32, device="cuda")
    out = run_balance(L, idx, torch.zeros(T, dtype=torch.uint8, device="cuda"))
    assert int(out["n"]) == 0
    for key in ("counts", "pm", "loss", "d"):
        assert torch.count_nonzero(out[key]) == 0, key


@pytest.mark.parametrize("T,N,k", [(200, 8, 2), (5000, 50, 2)])
def test_balance_loss_padding_and_infinities(T, N, k):
    """Masked rows may hold anything; -inf logits have probability zero; a row of -inf adds nothing;
    ids outside the experts are not counted."""
    L = randn(T, N, seed=5, std=3.0)
    idx = L.topk(k, 1).indices.to(torch.int32)
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    mask[::3] = 0
    L[0] = float("nan")
    L[3] = float("inf")
    L[6, 1] = -float("inf")
    L[1::7, 2] = -float("inf")
    L[5] = -float("inf")
    L[8] = torch.finfo(torch.float32).min
    idx[4, 0] = -1
    idx[7, 1] = N
    idx[10, 0] = 2 ** 31 - 1
    out = run_balance(L, idx, mask)
    check_balance(L, idx, mask, out=out)
    assert torch.count_nonzero(out["d"][::3]) == 0 and torch.count_nonzero(out["d"][5]) == 0


def test_balance_loss_upstream_gradient_and_coefficients():
    L = randn(300, 24, seed=8, std=2.0)
    idx = L.topk(3, 1).indices.to(torch.int32)
    for d_loss, alpha, z in ((torch.tensor([512.0], device="cuda"), 0.02, 0.0),
                             (torch.tensor(0.25, device="cuda"), 0.0, 0.01),
                             (torch.tensor([-3.0], device="cuda"), 1.0, 1.0)):
        out = run_balance(L, idx, None, alpha, z, d_loss)
        check_balance(L, idx, None, alpha, z, float(d_loss), out=out)


def test_balance_loss_agrees_with_router_stats():
    T, N, k = 3000, 40, 4
    L = randn(T, N, seed=2)
    idx = L.topk(k, 1).indices.to(torch.int32)
    out = run_balance(L, idx, None, z=0.0)
    dims = moe.make_dims(T, 64, N, k, 64)
    picks, pm = torch.empty(N, dtype=torch.int32, device="cuda"), torch.empty(N, device="cuda")
    aux, drop = torch.empty(1, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    moe.router_stats(dims, L, idx, torch.zeros_like(idx), picks, pm, aux, drop, moe.new_workspace(dims))
    assert torch.equal(picks, out["counts"])
    torch.testing.assert_close(pm, out["pm"], rtol=400 * U, atol=0)
    torch.testing.assert_close(aux[0], out["loss"][1], rtol=1000 * U, atol=0)


def test_balance_loss_gradient_against_differences():
    """The kernel's own loss, moved along the gradient of one token: fp32 differences of a loss of
    size ~1 with a step that changes it by ~1e-2 are good to 1e-4 of the change."""
    T, N, k = 40, 8, 2
    L = randn(T, N, seed=12)
    idx = L.topk(k, 1).indices.to(torch.int32)
    base = run_balance(L, idx, None, 1.0, 0.1)
    d = base["d"].double()
    h = 0.02 / float(d.norm())
    up = run_balance((L.double() + h * d).float(), idx, None, 1.0, 0.1)["loss"].double()[0]
    dn = run_balance((L.double() - h * d).float(), idx, None, 1.0, 0.1)["loss"].double()[0]
    # third-order term: h^2 |d|^2 / 6 of the slope's size, 1e-4; rounding of two losses 1e-6 / 2e-2
    assert abs(float((up - dn) / (2 * h)) / float(d.square().sum()) - 1) < 5e-3


# ---------------------------------------------------------------- router backward
def run_router(T, d, N, accumulate, which=("d_x", "d_w_router", "d_logit_bias"), seed=0, scale=1.0):
    x = randn(T, d, seed=seed + 1).to(torch.bfloat16)
    w = randn(N, d, seed=seed + 2, std=d ** -0.5)
    g = randn(T, N, seed=seed + 3, std=scale) * torch.exp(2 * randn(T, N, seed=seed + 4))
    dims = moe.make_dims(T, d, N, 1, 64)
    ws = moe.new_router_backward_workspace(dims)
    ws[256:] = 0xFF  # only the status word has to start at zero
    outs, old = {}, {}
    for i, (name, shape) in enumerate((("d_x", (T, d)), ("d_w_router", (N, d)), ("d_logit_bias", (N,)))):
        t = torch.full((shape[0] * (shape[1] if len(shape) > 1 else 1) + 64,), float("nan"), device="cuda")
        body = t[:-64].view(shape)
        if accumulate:
            body.copy_(randn(*shape, seed=seed + 5 + i))
        t[-64:] = 3.0
        outs[name], old[name] = t, (H.f64(body) if accumulate else 0.0)
    view = lambda n, shape: outs[n][:-64].view(shape) if n in which else None
    moe.router_backward(dims, x, w, g, view("d_x", (T, d)), view("d_w_router", (N, d)),
                        view("d_logit_bias", (N,)), ws, accumulate=accumulate)
    torch.cuda.synchronize()
    assert moe.read_device_error(ws) == moe.OK
    for t in outs.values():
        assert bool((t[-64:] == 3.0).all())
    shapes = {"d_x": (T, d), "d_w_router": (N, d), "d_logit_bias": (N,)}
    return x, w, g, {n: outs[n][:-64].view(shapes[n]) for n in outs}, old


def check_router(T, d, N, x, w, g, outs, old, which):
    X, W, G = H.f64(x), H.f64(w), H.f64(g)
    want = oracle.router_backward(X, W, G)
    size = oracle.router_backward(np.abs(X), np.abs(W), np.abs(G))
    for name, n in (("d_x", N), ("d_w_router", T), ("d_logit_bias", T)):
        if name not in which:
            continue
        o = want[name] + old[name]
        err = np.abs(H.f64(outs[name]) - o)
        bound = (2 * n + 32) * U * (size[name] + np.abs(old[name])) + 1e-37
        assert (err <= bound).all(), (name, float((err / bound).max()))
        # errors of many roundings add up like a random walk: far below the bound in norm
        assert np.linalg.norm(err) <= 2e-6 * np.linalg.norm(o) + 1e-30, (name, np.linalg.norm(err) / np.linalg.norm(o))


ROUTER_CASES = [(1, 64, 1), (1, 128, 256), (3, 64, 5), (64, 128, 8), (65, 192, 7), (130, 2880, 32),
                (257, 1024, 64), (512, 448, 130), (1000, 320, 33), (700, 7168, 17), (4096, 1024, 64),
                (2049, 640, 256), (5000, 256, 100), (16384, 512, 31), (8192, 4096, 8),
                (2001, 2880, 7), (1537, 448, 130), (300, 576, 200), (16384, 64, 256), (260, 4096, 40),
                (64, 4096, 256), (101, 5760, 130), (3000, 2880, 9), (5003, 4096, 5), (2999, 1024, 37)]


@pytest.mark.parametrize("T,d,N", ROUTER_CASES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_router_backward_matches_oracle(T, d, N, accumulate):
    x, w, g, outs, old = run_router(T, d, N, accumulate)
    which = ("d_x", "d_w_router", "d_logit_bias")
    check_router(T, d, N, x, w, g, outs, old, which)
    again = run_router(T, d, N, accumulate)[3]
    for name in which:
        assert torch.equal(outs[name], again[name]), name


@pytest.mark.parametrize("T,d,N", [(130, 192, 7), (4096, 1024, 64)])
@pytest.mark.parametrize("which", [("d_x",), ("d_w_router",), ("d_logit_bias",), ("d_x", "d_logit_bias"), ()])
def test_router_backward_some_outputs(T, d, N, which):
    x, w, g, outs, old = run_router(T, d, N, False, which)
    check_router(T, d, N, x, w, g, outs, old, which)
    for name in outs:
        if name not in which:
            assert bool(torch.isnan(outs[name]).all()), name


@pytest.mark.parametrize("scale", [1e-12, 1e12])
def test_router_backward_other_magnitudes(scale):
    for T, d, N in ((100, 128, 9), (4096, 1024, 40)):
        r = run_router(T, d, N, False, seed=3, scale=scale)
        check_router(T, d, N, *r[:5], ("d_x", "d_w_router", "d_logit_bias"))


def test_router_backward_zero_gradient():
    T, d, N = 4096, 1024, 64
    dims = moe.make_dims(T, d, N, 1, 64)
    dx, dw, db = (torch.full(s, 5.0, device="cuda") for s in ((T, d), (N, d), (N,)))
    args = (dims, randn(T, d).to(torch.bfloat16), randn(N, d), torch.zeros(T, N, device="cuda"))
    ws = moe.new_router_backward_workspace(dims)
    moe.router_backward(*args, dx, dw, db, ws, accumulate=True)
    assert all(bool((t == 5.0).all()) for t in (dx, dw, db))
    moe.router_backward(*args, dx, dw, db, ws)
    assert all(torch.count_nonzero(t) == 0 for t in (dx, dw, db))


@pytest.mark.parametrize("N", [20, 50, 200])
def test_router_backward_timeout_is_reported(N):
    """With a wait limit far too short the tensor-core kernels may stop early: they drain what they
    issued and say so, and the context and the next call are as before. An attempt to wait suspends
    the thread for a while and the limit is looked at after a failed one, so a kernel whose every wait
    ends within the attempt finishes, with the right results and no error."""
    T, d = 4096, 2048
    dims = moe.make_dims(T, d, N, 1, 64)
    ws = moe.new_router_backward_workspace(dims)
    x, w, g = randn(T, d).to(torch.bfloat16), randn(N, d), randn(T, N)
    outs = [torch.zeros(s, device="cuda") for s in ((T, d), (N, d), (N,))]
    moe.debug_set_wait_timeout_ns(1)
    try:
        moe.router_backward(dims, x, w, g, *outs, ws)
        torch.cuda.synchronize()
    finally:
        moe.debug_set_wait_timeout_ns(0)
    old = dict(d_x=0.0, d_w_router=0.0, d_logit_bias=0.0)
    status = moe.read_device_error(ws)
    assert status in (moe.OK, moe.ERR_TIMEOUT)
    if status == moe.OK:
        check_router(T, d, N, x, w, g, dict(zip(old, outs)), old, tuple(old))
    moe.router_backward(dims, x, w, g, *outs, ws)
    torch.cuda.synchronize()
    assert moe.read_device_error(ws) == moe.OK
    check_router(T, d, N, x, w, g, dict(zip(old, outs)), old, tuple(old))


def test_balance_loss_bool_mask():
    L = randn(100, 8, seed=1)
    idx = L.topk(2, 1).indices.to(torch.int32)
    mask = torch.rand(100, generator=gen(2), device="cuda") < 0.5
    a, b = run_balance(L, idx, mask), run_balance(L, idx, mask.to(torch.uint8))
    for k in a:
        assert torch.equal(a[k], b[k]), k


# ---------------------------------------------------------------- gradient norm
@pytest.mark.parametrize("sizes", [[], [0], [1], [5, 0, 3], [128] * 300, [1 << 20, 7, 12345], [3] * 2500,
                                   [33_000_001]])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, "mixed"])
def test_grad_norm_matches_oracle(sizes, dtype):
    grads = []
    for i, n in enumerate(sizes):
        t = torch.float32 if dtype == "mixed" and i % 2 else torch.bfloat16 if dtype == "mixed" else dtype
        grads.append(randn(n, seed=i % 50, std=0.1).to(t))
    ws = moe.new_grad_norm_workspace()
    plan = moe.grad_plan(grads)
    norm, scale = torch.full((2,), -1.0, device="cuda"), torch.full((2,), -1.0, device="cuda")
    for max_norm in (1.0, 1e9, float("inf")):
        for _ in range(2):  # the workspace is left as it was found
            moe.grad_norm(plan, max_norm, norm[:1], scale[:1], ws)
            want, ws_scale = oracle.grad_norm([H.f64(g) for g in grads], max_norm)
            # eight squares in fp32 (8 u), fp64 from there; the square root halves it
            assert abs(float(norm[0]) - want) <= 8 * U * want
            assert abs(float(scale[0]) - ws_scale) <= 16 * U
    assert float(norm[1]) == float(scale[1]) == -1.0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30])
def test_grad_norm_not_finite(bad):
    g = randn(10_000)
    g[777] = bad
    norm, scale = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    moe.grad_norm(moe.grad_plan([randn(50), g]), 1.0, norm, scale, moe.new_grad_norm_workspace())
    assert not np.isfinite(float(norm)) and np.isnan(float(scale))


# ---------------------------------------------------------------- AdamW
KINDS = [(p, g, b) for p in ("fp32", "master", "bf16") for g in (torch.float32, torch.bfloat16) for b in (32, 8)]


def make_tensor(n, kind, seed, fresh=False):
    params, gdtype, bits = kind
    w = randn(n, seed=seed, std=0.02)
    t = dict(param=w if params == "fp32" else w.to(torch.bfloat16), master=w.clone() if params == "master" else None,
             grad=(randn(n, seed=seed + 1, std=1e-3) * torch.exp(randn(n, seed=seed + 2))).to(gdtype))
    t["grad"][: n // 5] = 0
    t.update(moe.new_adamw_state(w, bits))
    if not fresh:
        m, r = randn(n, seed=seed + 3, std=2e-4), randn(n, seed=seed + 4, std=1e-3).abs()
        if bits == 32:
            t["m"], t["v"] = m, r.square()
        else:
            code, s = oracle.quantise_moment(H.f64(m), np.full(n, 32768), False)
            t["m"] = torch.tensor(code, device="cuda").to(torch.float8_e4m3fn)
            t["m_scale"] = torch.tensor(s, device="cuda").float()
            code, s = oracle.quantise_moment(H.f64(r), np.full(n, 32768), True)
            t["v"] = torch.tensor(code, device="cuda").to(torch.float8_e4m3fn)
            t["v_scale"] = torch.tensor(s, device="cuda").float()
    return t


def descriptor(t, wd=0.0):
    return moe.adamw_tensor(t["param"], t["grad"], t["m"], t["v"], master=t["master"],
                            m_scale=t.get("m_scale"), v_scale=t.get("v_scale"), weight_decay=wd)


def snapshot(t):
    return {k: None if v is None else H.f64(v.float()) for k, v in t.items()}


def check_adamw(before, t, kind, **hyper):
    params, _, bits = kind
    start = before["master"] if params == "master" else before["param"]
    want = oracle.adamw(start, before["grad"], before["m"], before["v"], bits=bits, m_scale=before.get("m_scale"),
                        v_scale=before.get("v_scale"), bf16_alone=params == "bf16", **hyper)
    after = snapshot(t)
    b1, b2 = hyper.get("betas", (0.9, 0.999))
    g = before["grad"] * hyper.get("grad_scale", 1.0)
    n = g.size
    p_tol = 16 * U * np.abs(want["update"]) + 4 * U * np.abs(start)
    # m' cancels where b1 m and (1 - b1) g do: its error in the update goes by their magnitudes
    m_old = before["m"] * (np.repeat(before["m_scale"], 128)[:n] if bits == 8 else 1.0)
    m_tol = 6 * U * (b1 * np.abs(m_old) + (1 - b1) * np.abs(g)) + 1e-44
    with np.errstate(divide="ignore", invalid="ignore"):
        ratio = np.where(want["m_exact"] != 0, np.abs(want["update"] / want["m_exact"]), 0)
    small = np.abs(want["v_exact"]) < 1e-37  # subnormal v: held absolutely through eps
    p_tol = p_tol + ratio * m_tol + np.where(small, 1e-3 * np.abs(want["update"]), 0)
    if params == "bf16":
        err = np.abs(after["param"] - want["param"])
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want["param"]), 2.0 ** -126))) - 7)
        # where p' lies within its error of a border, a neighbour is right too
        assert (err <= 2 * step).all() and (err > 0).sum() <= 2e-3 * n + 3
        assert (np.abs(after["param"] - want["param_exact"]) <= step * 1.001 + p_tol).all()
    else:
        got = after["master"] if params == "master" else after["param"]
        assert (np.abs(got - want["param"]) <= p_tol).all()
        if params == "master":
            assert torch.equal(t["param"], t["master"].to(torch.bfloat16))
    if bits == 32:
        assert (np.abs(after["m"] - want["m"]) <= m_tol).all()
        assert (np.abs(after["v"] - want["v"]) <= 8 * U * want["v"] + 1e-44).all()
    else:
        # the scale is the largest |m'| of the block / 448, and m' is known to m_tol, not to a part of
        # itself: b1 m and (1 - b1) g may cancel (a block of one element did, to 1e-3 of either).
        # The magnitudes' errors bound that of their maximum; the product with 1 / 448 rounds twice
        pad = np.zeros(len(want["m_scale"]) * 128)
        pad[:n] = m_tol
        s_tol = pad.reshape(-1, 128).max(1) / 448 + 4 * U * want["m_scale"]
        assert (np.abs(after["m_scale"] - want["m_scale"]) <= s_tol).all()
        np.testing.assert_allclose(after["v_scale"], want["v_scale"], rtol=10 * U, atol=0)
        for name in ("m", "v"):
            differ = after[name] != want[name]
            # the value before rounding has an error of ~10 u of 448 / spacing steps at most
            assert differ.sum() <= 1e-3 * n + 3, (name, int(differ.sum()))
            gap = np.maximum(np.abs(want[name]) / 8, 2.0 ** -9) * 1.01
            assert (np.abs(after[name] - want[name]) <= gap).all()
    return want


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: f"{k[0]}-{str(k[1])[6:]}-{k[2]}")
@pytest.mark.parametrize("n", [1, 3, 4, 127, 128, 129, 300, 5000, 100_003])
def test_adamw_matches_oracle(kind, n):
    for fresh, step in ((True, 1), (False, 100)):
        t = make_tensor(n, kind, seed=n, fresh=fresh)
        before = snapshot(t)
        plan = moe.adamw_plan([descriptor(t, 0.1)])
        moe.adamw_step(plan, step, lr=1e-3, seed=9)
        torch.cuda.synchronize()
        check_adamw(before, t, kind, step=step, lr=1e-3, seed=9, weight_decay=float(np.float32(0.1)))


def test_adamw_many_tensors_at_once():
    """800 tensors (three launches) of every kind and odd sizes, with a clipping scale; the memory
    behind each stays."""
    n_t = 800
    flat = {}
    ts, kinds, before = [], [], []
    for i in range(n_t):
        n = [1, 77, 128, 1000, 0, 4099, 256][i % 7]
        kind = KINDS[i % len(KINDS)]
        t = make_tensor(n, kind, seed=i)
        for k in ("param", "master", "m", "v", "m_scale", "v_scale"):
            if t.get(k) is not None:  # move into a larger buffer with a guard behind
                buf = torch.zeros(t[k].numel() + 32, dtype=torch.float32, device="cuda").to(t[k].dtype)
                buf[t[k].numel():] = 1.5
                buf[: t[k].numel()] = t[k]
                t[k] = buf[: t[k].numel()]
                flat[(i, k)] = buf
        ts.append(t)
        kinds.append(kind)
        before.append(snapshot(t))
    scale = torch.tensor([0.37], device="cuda")
    plan = moe.adamw_plan([descriptor(t, 0.01 * (i % 3)) for i, t in enumerate(ts)])
    moe.adamw_step(plan, 7, lr=3e-4, betas=(0.8, 0.95), eps=1e-6, seed=123456789, grad_scale=scale)
    torch.cuda.synchronize()
    for i in range(n_t):
        if ts[i]["param"].numel():
            check_adamw(before[i], ts[i], kinds[i], step=7, index=i, lr=3e-4, betas=(0.8, 0.95), eps=1e-6,
                        seed=123456789, grad_scale=float(scale), weight_decay=float(np.float32(0.01 * (i % 3))))
    for (i, k), buf in flat.items():
        assert bool((buf[ts[i][k].numel():].float() == 1.5).all()), (i, k)


@pytest.mark.parametrize("kind", [("fp32", torch.float32, 32), ("bf16", torch.bfloat16, 8)])
def test_adamw_leaves_the_step_out(kind):
    t = make_tensor(1000, kind, seed=1)
    before = snapshot(t)
    plan = moe.adamw_plan([descriptor(t)])
    for bad in (float("nan"), float("inf")):
        moe.adamw_step(plan, 3, grad_scale=torch.tensor([bad], device="cuda"))
    for s in (0, -5):
        moe.adamw_step(plan, torch.tensor([s], dtype=torch.int32, device="cuda"))
    after = snapshot(t)
    for k in before:
        assert before[k] is None or np.array_equal(before[k], after[k]), k


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: f"{k[0]}-{str(k[1])[6:]}-{k[2]}")
def test_adamw_keeps_a_nan(kind):
    """Without grad_scale a NaN gradient is not left out: its element's parameter becomes NaN (and
    stays it), no other parameter does, and a block's 8-bit moments become NaN by their scale."""
    n, at = 1000, [0, 129, 131, 701, 999]
    t = make_tensor(n, kind, seed=1)
    t["grad"][at] = float("nan")
    plan = moe.adamw_plan([descriptor(t)])
    moe.adamw_step(plan, 1, seed=5)
    for name in ("param", "master"):
        if t[name] is not None:
            assert torch.isnan(t[name]).nonzero().flatten().tolist() == at
    if kind[2] == 8:
        for name in ("m_scale", "v_scale"):
            assert torch.isnan(t[name]).nonzero().flatten().tolist() == sorted({i // 128 for i in at})
    else:
        for name in ("m", "v"):
            assert torch.isnan(t[name]).nonzero().flatten().tolist() == at
    t["grad"].zero_()
    moe.adamw_step(plan, 2, seed=5)
    assert bool(torch.isnan(t["param"][at]).all())


def test_adamw_step_and_rate_on_the_device_replayed():
    """A captured step with the step number, rate and scale on the device, replayed, equals steps
    called one by one with numbers."""
    kind = ("bf16", torch.float32, 8)
    a, b = make_tensor(3000, kind, seed=4), make_tensor(3000, kind, seed=4)
    pa, pb = moe.adamw_plan([descriptor(a, 0.1)]), moe.adamw_plan([descriptor(b, 0.1)])
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    lr, scale = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step.add_(1)
        moe.adamw_step(pa, step, lr=lr, seed=5, grad_scale=scale)
    for i in range(4):
        lr.fill_(1e-3 / (i + 1))
        scale.fill_(1.0 - 0.1 * i)
        graph.replay()
        moe.adamw_step(pb, i + 1, lr=float(np.float32(1e-3 / (i + 1))), seed=5,
                       grad_scale=torch.tensor([1.0 - 0.1 * i], device="cuda"))
    torch.cuda.synchronize()
    assert int(step) == 4
    for k in ("param", "m", "v", "m_scale", "v_scale"):
        x, y = a[k].float(), b[k].float()
        # the bias corrections are formed by pow on the device and on the host: an ulp apart
        assert float((x != y).float().mean()) < 5e-3 and torch.allclose(x, y, rtol=0.13, atol=2e-4), k


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: f"{k[0]}-{str(k[1])[6:]}-{k[2]}")
def test_adamw_bit_by_bit(kind):
    """Every fp32 operation is rounded by itself in the order of the formulas: the same lines in fp32
    tensor operations give the same bits, over several steps."""
    n, lr, b1, b2, eps, wd, seed = 128 * 20000, 3e-4, 0.9, 0.999, 1e-8, 0.1, 11
    t = make_tensor(n, kind, seed=21)
    t["grad"] = t["grad"].float().to(kind[1])
    scale = torch.tensor([0.37], device="cuda")
    w = (t["master"] if kind[0] == "master" else t["param"].float()).clone()
    m, v = t["m"].clone(), t["v"].clone()
    ms, vs = (t["m_scale"].clone(), t["v_scale"].clone()) if kind[2] == 8 else (None, None)
    plan = moe.adamw_plan([descriptor(t, wd)])

    def codes(x, words, keep):
        top = x.view(-1, 128).abs().amax(1, keepdim=True)
        x = x.view(-1, 128) * (448 / top)
        y = x.abs()
        small = y < 2.0 ** -6
        y = torch.where(small, y + 2.0 ** -6, y)
        c = ((y.view(torch.int32) + words.view(-1, 128) * 16 + 8) >> 20) - 960 - 8 * small
        c = c.clamp(max=126)
        c = torch.where(x > 0, c.clamp(min=1), c) if keep else c
        return (c + 128 * (x < 0)).to(torch.uint8).view(torch.float8_e4m3fn).view(-1), (top / 448)[:, 0]

    for step in (5, 6, 7):
        moe.adamw_step(plan, step, lr=lr, betas=(b1, b2), eps=eps, seed=seed, grad_scale=scale)
        um, uv, up = (torch.tensor(u, dtype=torch.int32, device="cuda") for u in oracle.random_bits(n, seed, step, 0))
        g = t["grad"].float() * scale
        m32 = m.float() if ms is None else (m.float().view(-1, 128) * ms[:, None]).view(-1)
        v32 = v.float() if vs is None else (v.float().view(-1, 128) * vs[:, None]).square().view(-1)
        m32 = b1 * m32 + (1 - b1) * g
        v32 = b2 * v32 + (1 - b2) * g * g
        r = v32.sqrt()
        # the quotient on the host: the framework's elementwise division is not to nearest everywhere
        f = np.float32
        inv = f(1) / f(np.sqrt(1 - b2 ** step))
        upd = f(lr / (1 - b1 ** step)) * m32.cpu().numpy() / (r.cpu().numpy() * inv + f(eps))
        w = w.cpu().numpy() * f(1 - lr * float(f(wd))) - upd
        assert w.dtype == f
        w = torch.tensor(w, device="cuda")
        if kind[2] == 8:
            m, ms = codes(m32, um, False)
            v, vs = codes(r, uv, True)
            assert torch.equal(t["m_scale"], ms) and torch.equal(t["v_scale"], vs)
        else:
            m, v = m32, v32
        assert torch.equal(t["m"].float(), m.float()) and torch.equal(t["v"].float(), v.float())
        if kind[0] == "bf16":
            w = ((w.view(torch.int32) + up) & -65536).view(torch.float32)
            assert torch.equal(t["param"].float(), w)
        else:
            assert torch.equal(t["master"] if kind[0] == "master" else t["param"], w)


def test_adamw_moments_in_8_bits_keep_their_expectation():
    """From one state and 400 seeds: the mean of the stored second moment's root is its exact value.
    A value's spread is at most half a spacing (2^-4 of it): the mean of 400 is within 5 x
    2^-4 / 2 / 20 of it, and over all elements together within 2^-4 / (2 sqrt(400 n)) x 5."""
    kind, n, seeds = ("fp32", torch.float32, 8), 512, 400
    total = np.zeros(n)
    for s in range(seeds):
        t = make_tensor(n, kind, seed=77)
        before = snapshot(t)
        moe.adamw_step(moe.adamw_plan([descriptor(t)]), 50, seed=s)
        after = snapshot(t)
        total += after["v"] * np.repeat(after["v_scale"], 128)
    want = oracle.adamw(before["param"], before["grad"], before["m"], before["v"], bits=8, step=50,
                        m_scale=before["m_scale"], v_scale=before["v_scale"])
    r = np.sqrt(want["v_exact"])
    rel = (total / seeds - r) / r
    large = r > 2.0 ** -6 * np.repeat(want["v_scale"], 128)
    assert large.mean() > 0.9
    assert np.abs(rel[large]).max() < 5 * 2.0 ** -4 / 2 / 20 * 2
    assert abs(rel[large].mean()) < 5 * 2.0 ** -4 / (2 * np.sqrt(seeds * large.sum())) + 1e-5


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_past_2_32_bytes(bits):
    """A tensor whose elements pass 32-bit offsets: its last blocks are updated like a small one's."""
    n = (1 << 32) + 1000 if bits == 8 else (1 << 31) + 1000
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    st = moe.new_adamw_state(p, bits)
    tail = 3000
    p[-tail:] = randn(tail, seed=1, std=0.02).to(torch.bfloat16)
    g[-tail:] = randn(tail, seed=2, std=1e-3).to(torch.bfloat16)
    g[0] = 1e-3
    start, grad = H.f64(p[-tail:]), H.f64(g[-tail:])
    moe.adamw_step(moe.adamw_plan([moe.adamw_tensor(p, g, st["m"], st["v"], m_scale=st.get("m_scale"),
                                                    v_scale=st.get("v_scale"))]), 1, lr=1e-3, seed=3)
    torch.cuda.synchronize()
    m = 0.1 * grad
    upd = 1e-3 * (m / 0.1) / (np.abs(grad) * np.sqrt(0.001) / np.sqrt(0.001) + 1e-8)
    up = oracle.random_bits(tail, 3, 1, 0, first=n - tail)[2]
    want = oracle.round_up_by_chance(start - upd, 7, -133, up / 65536.0)
    got = H.f64(p[-tail:])
    assert (got != want).sum() <= 0.002 * tail + 3
    assert float(p[0]) < 0 and torch.count_nonzero(p[1:1000]) == 0
    if bits == 32:
        assert np.abs(H.f64(st["m"][-tail:]) - m).max() <= 4 * U * np.abs(m).max()


# ---------------------------------------------------------------- together
def train_step(T, d, N, k, F, act, seed=0, stream=None):
    """Forward, balance loss, backward, the loss's gradient through the router, norm and update."""
    inp = synthetic.make_custom_inputs(T, d, N, F, act, seed=seed, device="cuda")
    cap = oracle.capacity_from_factor(1.25, T, N)
    dims = moe.make_dims(T, d, N, k, F, act, cap)
    rows = 2 * F if act == "swiglu" else F
    f32 = lambda *s: torch.full(s, float("nan"), device="cuda")
    b = dict(fws=moe.new_workspace(dims, forward=True), bws=moe.new_backward_workspace(dims),
             rws=moe.new_router_backward_workspace(dims), nws=moe.new_grad_norm_workspace(),
             out=torch.empty_like(inp["x"]), dx=f32(T, d), dwr=f32(N, d), db=f32(N), dgu=f32(N, rows, d),
             ddn=f32(N, d, F), counts=torch.empty(N, dtype=torch.int32, device="cuda"),
             n=torch.empty(1, dtype=torch.int32, device="cuda"), pm=f32(N), loss=f32(3), dl=f32(T, N),
             norm=f32(1), scale=f32(1), step=torch.zeros(1, dtype=torch.int32, device="cuda"))
    bias = torch.zeros(N, device="cuda")
    g = synthetic.make_grad_output(T, d, seed=seed, device="cuda")
    lay = moe.forward_layout(dims, b["fws"])
    view = lambda p, n, dt: b["fws"][p - b["fws"].data_ptr():][: n * 4].view(dt)
    logits, idx = view(lay.logits, T * N, torch.float32).view(T, N), view(lay.topk_idx, T * k, torch.int32).view(T, k)
    stage = b["fws"][lay.stage_ws - b["fws"].data_ptr():][: lay.stage_ws_bytes]
    ps = [inp["w_router"], bias, inp["w_gate_up"], inp["w_down"]]
    gs = [b["dwr"], b["db"], b["dgu"], b["ddn"]]
    st = [moe.new_adamw_state(p, 32 if i < 2 else 8) for i, p in enumerate(ps)]
    plan = moe.adamw_plan([moe.adamw_tensor(p, q, s["m"], s["v"], m_scale=s.get("m_scale"), v_scale=s.get("v_scale"),
                                            weight_decay=0.1) for p, q, s in zip(ps, gs, st)])
    gplan = moe.grad_plan(gs)

    def go():
        b["step"].add_(1)
        moe.forward_into(dims, inp["x"], ps[0], bias, ps[2], ps[3], inp["x"], b["out"], b["fws"], stream)
        moe.balance_loss(dims, logits, idx, None, b["counts"], b["n"], b["pm"], b["loss"], b["dl"], stage,
                         alpha=1.0, z_coef=0.1, stream=stream)
        moe.backward_into(dims, inp["x"], ps[0], ps[2], ps[3], b["fws"], g, b["dx"], b["dwr"], b["db"], b["dgu"],
                          b["ddn"], b["bws"], stream)
        moe.router_backward(dims, inp["x"], ps[0], b["dl"], b["dx"], b["dwr"], b["db"], b["rws"], accumulate=True,
                            stream=stream)
        moe.grad_norm(gplan, 1.0, b["norm"], b["scale"], b["nws"], stream)
        moe.adamw_step(plan, b["step"], lr=1e-3, seed=seed, grad_scale=b["scale"], stream=stream)
    return go, dims, inp, g, b, ps, st, logits, idx, stage


@pytest.mark.parametrize("T,d,N,k,F,act", [(200, 128, 8, 2, 128, "swiglu"), (300, 192, 5, 1, 64, "gelu"),
                                           (4096, 1024, 64, 2, 64, "gelu")])
def test_training_step_end_to_end(T, d, N, k, F, act):
    go, dims, inp, g, b, ps, st, logits, idx, stage = train_step(T, d, N, k, F, act)
    start = [H.f64(p) for p in ps]
    go()
    torch.cuda.synchronize()
    assert moe.read_device_error(stage) == moe.read_device_error(b["bws"]) == moe.read_device_error(b["rws"]) == 0
    L, I = H.f64(logits), idx.cpu().numpy()
    aux = oracle.balance_loss(L, I, None, 1.0, 0.1)
    np.testing.assert_allclose(H.f64(b["loss"]), aux["loss"], rtol=500 * U)
    x = H.f64(inp["x"])
    want = oracle.moe_layer_backward(x, start[0], start[2], start[3], H.f64(g), top_k=k, act=act,
                                     capacity=dims.capacity, logits=L)
    more = oracle.router_backward(x, start[0], aux["d_logits"])
    grads = [want["d_w_router"] + more["d_w_router"], want["d_logit_bias"] + more["d_logit_bias"],
             want["d_w_gate_up"], want["d_w_down"]]
    # the layer's backward pass has bf16 operands: the bars of its own test (1e-2, 3e-2)
    for got, o in ((b["dx"], want["dx"] + more["d_x"]), (b["dwr"], grads[0]), (b["db"], grads[1])):
        err = np.abs(H.f64(got) - o)
        assert err.sum() / np.abs(o).sum() <= 1e-2 and err.max() <= 3e-2 * np.abs(o).max()
    norm = np.sqrt(sum((q ** 2).sum() for q in grads))
    assert abs(float(b["norm"]) - norm) <= 1e-2 * norm
    # the update, from the GPU's own gradients
    for i, (p, q) in enumerate(zip(ps, (b["dwr"], b["db"], b["dgu"], b["ddn"]))):
        eight = i >= 2
        z = np.zeros(p.numel())
        o = oracle.adamw(start[i].reshape(-1), H.f64(q).reshape(-1), z, z, step=1, index=i, lr=1e-3, weight_decay=0.1,
                         grad_scale=float(b["scale"]), seed=0, bits=8 if eight else 32,
                         m_scale=np.zeros(-(-p.numel() // 128)), v_scale=np.zeros(-(-p.numel() // 128)),
                         bf16_alone=eight)
        got = H.f64(p).reshape(-1)
        if eight:
            assert (got != o["param"]).mean() <= 2e-3
        else:
            assert np.abs(got - o["param"]).max() <= 1e-3 * 1e-5 + 4 * U * np.abs(got).max()


@pytest.mark.parametrize("shape", [(300, 128, 8, 2, 64, "swiglu"), (2100, 1024, 64, 2, 64, "gelu")])
def test_training_step_replayed_on_a_side_stream_equals_calls(shape):
    go, *_, b1, p1, s1, _, _, _ = train_step(*shape, seed=3)
    go()
    go()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    go2, *_, b2, p2, s2, _, _, _ = train_step(*shape, seed=3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go2()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, c in zip(p1, p2):
        assert torch.equal(a, c)
    for a, c in zip(s1, s2):
        for k in a:
            assert torch.equal(a[k].float(), c[k].float()), k
    assert torch.equal(b1["loss"], b2["loss"]) and int(b2["step"]) == 2


# ---------------------------------------------------------------- balance loss, far logits
@pytest.mark.parametrize("z", [0.0, 1e-3, 1.0])
@pytest.mark.parametrize("T,N,k", [(3, 256, 8), (200, 8, 2), (5000, 50, 2), (6001, 100, 3)])
@pytest.mark.parametrize("value", [torch.finfo(torch.float32).min, -1e20, 1e20, -3e14, 2e14])
def test_balance_loss_of_far_logits(T, N, k, z, value):
    """Counted rows whose logsumexp has a square past fp32's range: with the z-loss off they add
    nothing, with it on they add the mean of the squares wherever that is an fp32 number."""
    L = randn(T, N, seed=T, std=3.0)
    idx = L.topk(k, 1).indices.to(torch.int32)
    L[1] = value
    L[T - 1] = value / 3
    out = run_balance(L, idx, None, z=z)
    assert z > 0 or (float(out["loss"][2]) == 0 and bool(torch.isfinite(out["loss"]).all()))
    check_balance(L, idx, None, z=z, out=out)
    plain = run_balance(L, idx, None, z=z, grad=False)
    assert torch.equal(out["loss"], plain["loss"])


# ---------------------------------------------------------------- AdamW, a rate that is not finite
@pytest.mark.parametrize("kind", [("fp32", torch.float32, 32), ("master", torch.bfloat16, 32), ("bf16", torch.float32, 8)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_adamw_leaves_the_step_out_for_a_bad_rate(kind, bad):
    """A rate read on the device cannot be refused by the call as a number is: the step is left out."""
    t = make_tensor(1000, kind, seed=2)
    before = snapshot(t)
    plan = moe.adamw_plan([descriptor(t, 0.1)])
    rate = torch.tensor([bad], device="cuda")
    moe.adamw_step(plan, 3, lr=rate)
    moe.adamw_step(plan, torch.tensor([3], dtype=torch.int32, device="cuda"), lr=rate)
    after = snapshot(t)
    for k in before:
        assert before[k] is None or np.array_equal(before[k], after[k]), k
    moe.adamw_step(plan, 3, lr=rate.fill_(1e-3))
    assert not np.array_equal(before["param"], snapshot(t)["param"])


@pytest.mark.parametrize("T,d,N", [(5000, 64, 256), (4700, 64, 210), (4097, 64, 255)])
def test_balance_loss_where_the_workspace_holds_fewer_rows(T, d, N):
    """Sizes at which the region that the stages share has a row for fewer CTAs than there are SMs:
    nothing behind the workspace is written, and the result is as good."""
    dims = moe.make_dims(T, d, N, 2, 64, capacity=T * 2 // N)
    n = moe.workspace_bytes(dims)
    buf = torch.zeros(n + 4096, dtype=torch.uint8, device="cuda")
    buf[n:] = 77
    L = randn(T, N, seed=N, std=3.0)
    idx = L.topk(2, 1).indices.to(torch.int32)
    out = dict(counts=torch.empty(N, dtype=torch.int32, device="cuda"), n=torch.empty(1, dtype=torch.int32, device="cuda"),
               pm=torch.empty(N, device="cuda"), loss=torch.empty(3, device="cuda"), d=torch.empty(T, N, device="cuda"))
    for _ in range(2):  # the counter is left as it was found
        moe.balance_loss(dims, L, idx, None, out["counts"], out["n"], out["pm"], out["loss"], out["d"], buf[:n], z_coef=1e-3)
        torch.cuda.synchronize()
        check_balance(L, idx, None, out=out)
    assert bool((buf[n:] == 77).all())


def test_router_backward_workspace_of_a_longer_batch():
    """A workspace made for 1443 tokens serves 1436, which by itself takes more token ranges."""
    N, d = 256, 7168
    n = moe.router_backward_workspace_bytes(moe.make_dims(1443, d, N, 1, 64))
    buf = torch.zeros(n + 4096, dtype=torch.uint8, device="cuda")
    buf[n:] = 77
    for T in (1443, 1436, 70, 1):
        x, w, g = randn(T, d, seed=T).to(torch.bfloat16), randn(N, d, seed=1, std=d ** -0.5), randn(T, N, seed=2)
        outs = {k: torch.full(s, float("nan"), device="cuda") for k, s in
                (("d_x", (T, d)), ("d_w_router", (N, d)), ("d_logit_bias", (N,)))}
        moe.router_backward(moe.make_dims(T, d, N, 1, 64), x, w, g, *outs.values(), buf[:n])
        torch.cuda.synchronize()
        assert moe.read_device_error(buf[:n]) == moe.OK
        check_router(T, d, N, x, w, g, outs, dict.fromkeys(outs, 0.0), tuple(outs))
    assert bool((buf[n:] == 77).all())


@pytest.mark.parametrize("T,d,N", [(16384, 2880, 8), (16384, 2880, 64), (16384, 1024, 256)])
@pytest.mark.parametrize("which", ["d_x", "d_w_router"])
def test_router_backward_wait_limit_runs_out(T, d, N, which):
    """Batches whose TMA copies and chains take far longer than an attempt to wait: with a limit of 1 ns
    each of the two kernels gives up, says so and drains; the next call is right."""
    dims = moe.make_dims(T, d, N, 1, 64)
    ws = moe.new_router_backward_workspace(dims)
    x, w, g = randn(T, d, seed=1).to(torch.bfloat16), randn(N, d, seed=2), randn(T, N, seed=3)
    outs = dict.fromkeys(("d_x", "d_w_router", "d_logit_bias"))
    outs[which] = torch.zeros((T, d) if which == "d_x" else (N, d), device="cuda")
    moe.debug_set_wait_timeout_ns(1)
    try:
        moe.router_backward(dims, x, w, g, *outs.values(), ws)
        torch.cuda.synchronize()
    finally:
        moe.debug_set_wait_timeout_ns(0)
    assert moe.read_device_error(ws) == moe.ERR_TIMEOUT
    moe.router_backward(dims, x, w, g, *outs.values(), ws)
    torch.cuda.synchronize()
    assert moe.read_device_error(ws) == moe.OK
    check_router(T, d, N, x, w, g, outs, dict.fromkeys(outs, 0.0), (which,))


# ---------------------------------------------------------------- router backward, the stated precision
@pytest.mark.parametrize("T,d,N", [(300, 576, 40), (16384, 512, 31), (4096, 1024, 64), (2048, 1024, 256), (8192, 2880, 8)])
@pytest.mark.parametrize("operands", ["wide", "cancelling", "columns"])
def test_router_backward_stated_precision(T, d, N, operands):
    """The bound of include/moe.h, element by element, and its figure in norm, on operands that strain
    them: magnitudes spread over 40 binades; rows of dL that add up to zero against rows of W_r with a
    large common part; columns of W_r 2^-30 below the others. The largest d_x floor is the derived
    (N 2^-37 + 2^-38) sum, at N = 256 just over half of the stated 2^-28."""
    X, W, G = randn(T, d, seed=1).to(torch.bfloat16), randn(N, d, seed=2), randn(T, N, seed=3)
    if operands == "wide":
        W = W * torch.exp2(-(torch.arange(d, device="cuda") % 41).float())
        G = G * torch.exp2(-(torch.arange(N, device="cuda") % 31).float())
    elif operands == "columns":
        W[:, ::3] *= 2.0 ** -30
    else:
        p = torch.softmax(2 * G, 1)
        u = randn(T, N, seed=4)
        G = p * (u - (p * u).sum(1, keepdim=True))
        W = W + 100 * randn(1, d, seed=5)
        X = (X.float() + 10).to(torch.bfloat16)
    dims = moe.make_dims(T, d, N, 1, 64)
    ws = moe.new_router_backward_workspace(dims)
    outs = {k: torch.full(s, float("nan"), device="cuda") for k, s in
            (("d_x", (T, d)), ("d_w_router", (N, d)), ("d_logit_bias", (N,)))}
    moe.router_backward(dims, X, W, G, *outs.values(), ws)
    torch.cuda.synchronize()
    assert moe.read_device_error(ws) == moe.OK
    x, w, g = H.f64(X), H.f64(W), H.f64(G)
    want, size = oracle.router_backward(x, w, g), oracle.router_backward(np.abs(x), np.abs(w), np.abs(g))
    for name, n in (("d_x", N), ("d_w_router", T), ("d_logit_bias", T)):
        err = np.abs(H.f64(outs[name]) - want[name])
        bound = (2 * n + 32) * U * size[name]
        if name == "d_x":
            bound = bound + 2.0 ** -28 * (np.abs(g) @ np.abs(w).max(1))[:, None]
        assert (err <= bound + 1e-37).all(), (name, float((err / (bound + 1e-37)).max()))
        assert np.linalg.norm(err) <= 1e-6 * np.linalg.norm(size[name]), (name, np.linalg.norm(err) / np.linalg.norm(size[name]))


def test_adamw_second_moment_in_8_bits_over_many_steps():
    """Mean of v over 1000 steps after 3000, moments in 8 bits against fp32 on the same Gaussian
    gradients. A rounding of r = sqrt(v) that moves by d between codes h apart adds h |d| to E[r^2], with
    |d| = (1 - beta2) |g^2 - v| / (2 r) and a decay of 1 - beta2: in equilibrium (h / r) E|z^2 - 1| / 2 of
    v, E|z^2 - 1| = 0.968 and h / r in [1/16, 1/8], hence 3.0 to 6.1 %; the block's scale moves every
    code by as much again at most. So the excess lies above zero and below 12.2 %. The elements differ
    by a factor of 2 at most, singly: the mean of 4096 is good to 1 %."""
    n, first, last = 4096, 3000, 4000
    p8, p32, g = (torch.zeros(n, device="cuda") for _ in range(3))
    s8, s32 = moe.new_adamw_state(p8, 8), moe.new_adamw_state(p32, 32)
    plan = moe.adamw_plan([moe.adamw_tensor(p8, g, s8["m"], s8["v"], m_scale=s8["m_scale"], v_scale=s8["v_scale"]),
                           moe.adamw_tensor(p32, g, s32["m"], s32["v"])])
    rng, total8, total32 = gen(5), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    for t in range(1, last + 1):
        g.normal_(0.0, 1e-3, generator=rng)
        moe.adamw_step(plan, t, lr=0.0, seed=1)
        if t > first:
            total8 += (s8["v"].float().view(-1, 128) * s8["v_scale"][:, None]).square().view(-1)
            total32 += s32["v"]
    excess = float((total8 / total32).mean()) - 1
    assert 0 < excess < 0.122 + 0.01
    # fp32 moments themselves: the mean of g^2, whose 4e6 values over ~1000 independent steps vary by 0.1 %
    assert abs(float(total32.mean()) / (last - first) / 1e-6 - 1) < 0.05
