"""The training operators on the host (no GPU): the oracle against differences and against the
definition of an unbiased rounding, and the refusals of the C ABI and of the binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import sparse_mixture_experts_11_b200 as moe

P = ctypes.c_void_p
BIG = 1 << 30


# ---------------------------------------------------------------- oracle
@pytest.mark.parametrize("masked", [False, True])
def test_oracle_balance_gradient_against_differences(masked):
    rng = np.random.default_rng(3)
    T, N, k = 9, 6, 2
    L = rng.normal(size=(T, N)) * 2
    idx = np.argsort(-L, 1)[:, :k]  # the choice itself is held while the logits move
    mask = (rng.random(T) < 0.6) if masked else None
    f = lambda M: oracle.balance_loss(M, idx, mask, 0.3, 0.2)["loss"][0]
    got = oracle.balance_loss(L, idx, mask, 0.3, 0.2, d_loss=1.5)["d_logits"]
    h = 1e-6
    for t in range(T):
        for e in range(N):
            up, dn = L.copy(), L.copy()
            up[t, e] += h
            dn[t, e] -= h
            # central differences: error h^2 f''' / 6 + rounding eps / h, both below 1e-9 here
            assert abs(got[t, e] - 1.5 * (f(up) - f(dn)) / (2 * h)) < 1e-8


def test_oracle_balance_agrees_with_the_layers_oracle():
    rng = np.random.default_rng(4)
    L = rng.normal(size=(50, 7))
    idx = np.argsort(-L, 1)[:, :3].astype(np.int32)
    b = oracle.balance_loss(L, idx, None, 0.01)
    s = oracle.router_statistics(L, idx, np.zeros_like(idx), 0.01)
    assert np.array_equal(b["counts"], s["picks"])
    assert abs(b["loss"][1] - s["aux_loss"]) < 1e-15 and b["loss"][2] == 0
    from oracle.moe_backward import aux_loss_backward
    np.testing.assert_allclose(b["d_logits"], aux_loss_backward(L, idx, 0.01), rtol=0, atol=1e-17)


def test_oracle_router_gradient_against_differences():
    rng = np.random.default_rng(5)
    x, w, g = rng.normal(size=(5, 4)), rng.normal(size=(3, 4)), rng.normal(size=(5, 3))
    f = lambda x, w, b: float((g * (x @ w.T + b)).sum())  # linear: differences are exact
    r = oracle.router_backward(x, w, g)
    b = np.zeros(3)
    for name, a in (("d_x", x), ("d_w_router", w), ("d_logit_bias", b)):
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + 0.5
            up = f(x, w, b)
            a[i] = old - 0.5
            dn = f(x, w, b)
            a[i] = old
            assert abs(r[name][i] - (up - dn)) < 1e-12


def test_oracle_rounding_keeps_the_expectation():
    """Over all 2^16 random words the mean of a rounded value is the value, to half a word's
    weight (2^-17 of the spacing) and rounding in float64; every result is a neighbour."""
    u = (np.arange(65536) * 16 + 8) / 2.0 ** 20
    for x in (1.03, 2.0, 447.9, 0.017, 2.0 ** -7 + 1e-4, 3e-4, 1.99999, 0.015624):
        e = max(math.floor(math.log2(x)) - 3, -9)
        r = oracle.round_up_by_chance(np.full(65536, x), 3, -9, u)
        assert np.all(np.abs(r - x) < 2.0 ** e)
        assert abs(r.mean() - x) <= 2.0 ** e * 2.0 ** -16
        codes = torch.tensor(r).to(torch.float8_e4m3fn).double().numpy()
        assert np.array_equal(codes, r)  # every result is an E4M3 value


def test_oracle_random_words_are_even_and_independent():
    um, uv, up = oracle.random_bits(1 << 18, 7, 3, 2)
    n = um.size
    for a in (um, uv, up):
        # mean of n uniform words: standard deviation 2^16 / sqrt(12 n); 5 of them
        assert abs(a.mean() - 32767.5) < 5 * 65536 / math.sqrt(12 * n)
    for a, b in ((um, uv), (um, up), (uv, up), (um[1:], um[:-1]), (uv[1:], um[:-1])):
        assert abs(np.corrcoef(a, b)[0, 1]) < 5 / math.sqrt(n)
    other = oracle.random_bits(1 << 12, 7, 4, 2)[0], oracle.random_bits(1 << 12, 7, 3, 3)[0]
    for a in other:
        assert (a == um[:1 << 12]).mean() < 0.01


# ---------------------------------------------------------------- refusals, C ABI
def _dims(**kw):
    base = dict(T=16, d_model=128, n_experts=8, top_k=2, d_ff=128, act=0, capacity=16)
    base.update(kw)
    return moe.Dims(**base)


def _balance(d, logits=P(16), idx=P(16), mask=None, alpha=0.1, z=0.0, d_loss=None, counts=P(16),
             n=P(16), pm=P(16), loss=P(16), dl=P(16), ws=P(256), nb=BIG):
    return moe._lib.moe_balance_loss(ctypes.byref(d), logits, idx, mask, alpha, z, d_loss, counts, n, pm,
                                     loss, dl, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), moe.ERR_INVALID), (dict(idx=None), moe.ERR_INVALID),
    (dict(counts=None), moe.ERR_INVALID), (dict(n=None), moe.ERR_INVALID),
    (dict(pm=None), moe.ERR_INVALID), (dict(loss=None), moe.ERR_INVALID),
    (dict(ws=None), moe.ERR_INVALID), (dict(alpha=float("nan")), moe.ERR_INVALID),
    (dict(z=float("inf")), moe.ERR_INVALID), (dict(logits=P(20)), moe.ERR_UNSUPPORTED),
    (dict(dl=P(8)), moe.ERR_UNSUPPORTED), (dict(mask=P(3)), moe.ERR_UNSUPPORTED),
    (dict(nb=300), moe.ERR_WORKSPACE)])
def test_balance_loss_refusals(kw, status):
    assert _balance(_dims(), **kw) == status


def test_balance_loss_bad_dims_and_empty_batch():
    assert _balance(_dims(n_experts=300)) == moe.ERR_UNSUPPORTED
    assert _balance(_dims(top_k=9)) == moe.ERR_INVALID
    assert _balance(_dims(T=-1)) == moe.ERR_INVALID
    assert _balance(_dims(T=0), None, None, None, counts=None, ws=None, nb=0) == moe.OK


def _router(d, x=P(16), w=P(16), dl=P(16), dx=P(16), dw=P(16), db=P(16), acc=0, ws=P(256), nb=BIG):
    return moe._lib.moe_router_backward(ctypes.byref(d), x, w, dl, dx, dw, db, acc, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), moe.ERR_INVALID), (dict(w=None), moe.ERR_INVALID), (dict(dl=None), moe.ERR_INVALID),
    (dict(ws=None), moe.ERR_INVALID), (dict(acc=2), moe.ERR_INVALID), (dict(x=P(2)), moe.ERR_UNSUPPORTED),
    (dict(db=P(4)), moe.ERR_UNSUPPORTED), (dict(nb=8), moe.ERR_WORKSPACE)])
def test_router_backward_refusals(kw, status):
    assert _router(_dims(), **kw) == status


def test_router_backward_bad_dims_and_empty_batch():
    assert _router(_dims(d_model=100)) == moe.ERR_UNSUPPORTED
    assert _router(_dims(T=0), None, None, None, None, None, None, 0, None, 0) == moe.OK
    n = ctypes.c_size_t(0)
    assert moe._lib.moe_router_backward_workspace_bytes(ctypes.byref(_dims(T=0)), ctypes.byref(n)) == moe.OK
    assert moe._lib.moe_router_backward_workspace_bytes(ctypes.byref(_dims()), None) == moe.ERR_INVALID


def _norm(items, max_norm=1.0, norm=P(16), scale=P(16), ws=P(256), nb=BIG, n=None):
    a = (moe.GradTensor * max(1, len(items)))(*items)
    return moe._lib.moe_grad_norm(a, len(items) if n is None else n, max_norm, norm, scale, ws, nb, None)


def test_grad_norm_refusals():
    ok = moe.GradTensor(16, 5, 0)
    for bad in (0.0, -1.0, float("nan")):
        assert _norm([ok], max_norm=bad) == moe.ERR_INVALID
    assert _norm([ok], norm=None) == moe.ERR_INVALID
    assert _norm([ok], scale=None) == moe.ERR_INVALID
    assert _norm([ok], ws=None) == moe.ERR_INVALID
    assert _norm([ok], n=-1) == moe.ERR_INVALID
    assert moe._lib.moe_grad_norm(None, 1, 1.0, P(16), P(16), P(256), BIG, None) == moe.ERR_INVALID
    assert _norm([moe.GradTensor(None, 5, 0)]) == moe.ERR_INVALID
    assert _norm([ok, moe.GradTensor(16, -1, 0)]) == moe.ERR_INVALID
    assert _norm([moe.GradTensor(16, 5, 2)]) == moe.ERR_INVALID
    assert _norm([moe.GradTensor(18, 5, 1)]) == moe.ERR_UNSUPPORTED
    assert _norm([ok], nb=256) == moe.ERR_WORKSPACE


def _adam(n=None, config=None, **kw):
    t = dict(param=16, master=None, grad=16, m=16, v=16, m_scale=None, v_scale=None, numel=5, param_dtype=0,
             grad_dtype=0, state_bits=32, weight_decay=0.0)
    c = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, seed=0, step_dev=None, lr_dev=None,
             grad_scale=None)
    c.update(config or {})
    t.update(kw)
    a = (moe.AdamWTensor * 1)(moe.AdamWTensor(**t))
    return moe._lib.moe_adamw_step(a, 1 if n is None else n, ctypes.byref(moe.AdamWConfig(**c)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), moe.ERR_INVALID), (dict(numel=-1), moe.ERR_INVALID), (dict(param=None), moe.ERR_INVALID),
    (dict(grad=None), moe.ERR_INVALID), (dict(m=None), moe.ERR_INVALID), (dict(v=None), moe.ERR_INVALID),
    (dict(param_dtype=2), moe.ERR_INVALID), (dict(grad_dtype=-1), moe.ERR_INVALID),
    (dict(state_bits=16), moe.ERR_INVALID), (dict(state_bits=8, m_scale=16), moe.ERR_INVALID),
    (dict(state_bits=8, v_scale=16), moe.ERR_INVALID), (dict(master=16), moe.ERR_INVALID),
    (dict(weight_decay=float("nan")), moe.ERR_INVALID), (dict(grad=20), moe.ERR_UNSUPPORTED),
    (dict(m=17, state_bits=8, m_scale=16, v_scale=16), moe.ERR_UNSUPPORTED),
    (dict(master=8, param_dtype=1), moe.ERR_UNSUPPORTED),
    (dict(state_bits=8, m_scale=18, v_scale=16), moe.ERR_UNSUPPORTED),
    (dict(config=dict(eps=1e-60)), moe.ERR_INVALID), (dict(config=dict(eps=1e60)), moe.ERR_INVALID),
    (dict(config=dict(step=0)), moe.ERR_INVALID), (dict(config=dict(eps=0.0)), moe.ERR_INVALID),
    (dict(config=dict(beta1=1.0)), moe.ERR_INVALID), (dict(config=dict(beta2=-0.1)), moe.ERR_INVALID),
    (dict(config=dict(lr=float("inf"))), moe.ERR_INVALID), (dict(config=dict(eps=float("nan"))), moe.ERR_INVALID),
])
def test_adamw_refusals(kw, status):
    assert _adam(**kw) == status


def test_adamw_nothing_to_do_needs_no_device():
    assert _adam(n=0) == moe.OK
    assert _adam(numel=0, param=None, grad=None, m=None, v=None) == moe.OK
    c = moe.AdamWConfig(1e-3, 0.9, 0.999, 1e-8, 1, 0, None, None, None)
    assert moe._lib.moe_adamw_step(None, 0, ctypes.byref(c), None) == moe.OK
    assert moe._lib.moe_adamw_step(None, 1, ctypes.byref(c), None) == moe.ERR_INVALID
    assert moe._lib.moe_adamw_step(None, 0, None, None) == moe.ERR_INVALID


# ---------------------------------------------------------------- refusals, binding
def test_binding_refuses_before_any_call():
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)
    with pytest.raises(ValueError, match="fp32 or bf16"):
        moe.adamw_tensor(z(4, dt=torch.float16), z(4), z(4), z(4))
    with pytest.raises(ValueError, match="m and v"):
        moe.adamw_tensor(z(4), z(4), z(4), z(4, dt=torch.bfloat16))
    with pytest.raises(ValueError, match="8-bit moments"):
        moe.adamw_tensor(z(4), z(4), z(4), z(4), m_scale=z(1))
    with pytest.raises(ValueError, match="bf16 param"):
        moe.adamw_tensor(z(4), z(4), z(4), z(4), master=z(4))
    with pytest.raises(ValueError, match="elements"):
        moe.adamw_tensor(z(4), z(5), z(4), z(4))
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.adamw_tensor(z(4), z(4), z(4), z(4))
    with pytest.raises(ValueError, match="fp32 or bf16"):
        moe.grad_plan([z(4, dt=torch.float16)])
    with pytest.raises(ValueError, match="bits"):
        moe.new_adamw_state(z(4), bits=4)
    s = moe.new_adamw_state(z(3, 43), bits=8)
    assert s["m"].dtype == torch.float8_e4m3fn and s["m_scale"].shape == (2,) and s["v"].numel() == 129


def test_binding_names_the_argument_at_fault(monkeypatch):
    """The calls' own checks on the host: what is wrong is named before the library is entered."""
    monkeypatch.setattr(moe, "_device", lambda: 0)
    d = _dims()
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)
    args = [z(16, 8), z(16, 2, dt=torch.int32), None, z(8, dt=torch.int32), z(1, dt=torch.int32), z(8), z(3), None]
    with pytest.raises(ValueError, match="ws must be a CUDA tensor"):
        moe.balance_loss(d, *args, z(10, dt=torch.uint8))
    with pytest.raises(ValueError, match="ws is required"):
        moe.balance_loss(d, *args, None)
    with pytest.raises(ValueError, match="ws must be"):
        moe.router_backward(d, z(16, 128, dt=torch.bfloat16), z(8, 128), z(16, 8), None, None, None, z(10))
    for call in (lambda: moe._arg(z(4), 0, "a", torch.float32, (4,)), lambda: moe._arg(z(4), -1, "a", torch.int32, (4,)),
                 lambda: moe._arg(None, 0, "a", torch.float32, (4,)), lambda: moe._arg(z(4, 4).t(), -1, "a", torch.float32, (4, 4))):
        with pytest.raises(ValueError, match="^a "):
            call()


@pytest.mark.parametrize("call", [
    lambda: _balance(_dims(), n=P(18)), lambda: _balance(_dims(), d_loss=P(17)),
    lambda: _norm([moe.GradTensor(16, 5, 0)], norm=P(18)), lambda: _norm([moe.GradTensor(16, 5, 0)], scale=P(33)),
    lambda: _adam(config=dict(step_dev=18)), lambda: _adam(config=dict(lr_dev=17)),
    lambda: _adam(config=dict(grad_scale=19))])
def test_misaligned_scalars_are_refused(call):
    """One-element arguments need their type's alignment: an access to any other address would fault."""
    assert call() == moe.ERR_UNSUPPORTED


@pytest.mark.parametrize("T,d,N,k,F,stage,forward", [
    (4096, 128, 256, 8, 64, 240128, 34452224), (5000, 64, 256, 2, 64, 164352, 10599168),
    (6000, 128, 93, 1, 64, 103936, 7790080), (8192, 128, 256, 8, 64, 282112, 68704000),
    (5000, 64, 210, 8, 64, 135680, 25566464)])
def test_balance_loss_leaves_workspace_sizes_alone(T, d, N, k, F, stage, forward):
    """The sizes of the layer's calls from before there was a balance loss: a workspace of that size
    is still enough for every one of them, and for the balance loss."""
    dims = moe.Dims(T=T, d_model=d, n_experts=N, top_k=k, d_ff=F, act=0, capacity=max(1, T * k // N))
    assert moe.workspace_bytes(dims) == stage and moe.forward_workspace_bytes(dims) == forward
    assert _balance(dims, nb=stage) != moe.ERR_WORKSPACE and _balance(dims, nb=stage - 1) == moe.ERR_WORKSPACE


@pytest.mark.parametrize("N,d", [(256, 7168), (256, 5120), (32, 2880), (8, 128), (64, 1024), (5, 64), (130, 448)])
def test_router_backward_workspace_serves_shorter_batches(N, d):
    """The size for a batch is enough for every shorter one: what a call needs itself is not monotone
    in T (fewer, longer token ranges, or the other path). Every length up to 3000, then a spread."""
    lengths = list(range(1, 3001)) + [3001 + 211 * i + i * i for i in range(200)] + [2 ** i + j for i in range(12, 21) for j in (-1, 0, 1)]
    last = 0
    for T in sorted(lengths):
        dims = _dims(T=T, n_experts=N, top_k=1, d_model=d)
        size = moe.router_backward_workspace_bytes(dims)
        assert size >= last, (T, size, last)
        last = size
        assert _router(dims, nb=size) != moe.ERR_WORKSPACE


def test_router_backward_workspace_is_not_much_more_than_needed():
    """At the layers' training batches the size stays what the call itself needs: 4 N and 4 d N bytes a
    token range, 10 bytes a logit, 4 a token and 4 a weight."""
    for T, N, d, ranges, planes in ((16384, 256, 7168, 5, 1), (16384, 32, 2880, 12, 3)):
        need = T * (10 * N + 4) + 4 * N * d * (1 + ranges * planes) + 592 * N * 4 + 4096
        assert moe.router_backward_workspace_bytes(_dims(T=T, n_experts=N, top_k=1, d_model=d)) <= need
