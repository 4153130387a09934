"""GPU tests of gptq_qk_norm_rope and its gradients against the fp64 reference.

Bounds, from the kernels' arithmetic in fp32 (u = 2^-24): the sum of squares is a chain of 16 and a
tree of at most 5 additions, so r = (mean + eps)^-1/2 is off by at most (16 + 5 + 2) / 2 u and 3 more
for the division and the reciprocal root: 15 u.  n = x r w adds 2: 17 u.  The rotation adds 3 roundings to
each product, so |y - y0| <= 20 u (|n_a cos| + |n_b sin|), doubled here for second-order terms.
Backward: dn 3 u of D = |dy_a cos| + |dy_b sin|; the mean of g x has a chain of 16 + 5 and 4 more; r^3 is off
by 47 u; |dx - dx0| <= 22 u r |w| D + (47 + 29) u |x| r^3 mean(|w| D |x|).  dw: each term 20 u, and a chain of
the terms a lane sums, 10 butterfly and wave steps, 32 + 16 partial sums.
"""

import numpy as np
import pytest

from attnhelp import H, U, close, on_device, rotation, values
from gpuhelp import say, to_dev, torch_dev
from oracle import attn_ref as R

pytestmark = pytest.mark.gpu


def _inputs(tokens, qh, kh, dim, rot, bf16, seed, weight=True):
    rng = np.random.default_rng(seed)
    q, k = values(rng, (tokens, qh, dim), bf16), values(rng, (tokens, kh, dim), bf16)
    w = [values(rng, (dim,), bf16, 0.2) + 0.0 for _ in range(2)] if weight else [None, None]
    cos, sin = rotation(rng, 97, rot)
    return q, k, w, cos, sin, rng.integers(0, 97, tokens).astype(np.int32), rng


def _dev(w, bf16):
    return None if w is None else on_device(w[None, None], bf16)[0, 0]


def _rope(cos, sin, inter, eps):
    import post_weight_quantization_03_amd as g
    return g.Rope(to_dev(cos), to_dev(sin), inter, eps) if cos.shape[1] else g.Rope(None, None, inter, eps)


def _mag(x, w, cos, sin, pos, inter, eps):
    """|n_a cos| + |n_b sin| of each element."""
    c, s = np.abs(cos.astype(np.float64))[pos][:, None], np.abs(sin.astype(np.float64))[pos][:, None]
    n = np.abs(R.norm(x, w, eps))
    # the magnitudes turn like the values, with every sign positive
    half = c.shape[-1]
    y = n.copy()
    a = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if inter else (slice(0, half), slice(half, 2 * half))
    y[..., a[0]] = n[..., a[0]] * c + n[..., a[1]] * s
    y[..., a[1]] = n[..., a[0]] * s + n[..., a[1]] * c
    return y


FORMS = [
    # tokens, q heads, k heads, dim, rot, interleaved, bf16, layout
    (1, 32, 8, 128, 128, False, True, "slice"),
    (1, 1, 1, 16, 16, False, False, "plain"),
    (5, 3, 2, 64, 32, True, True, "plain"),
    (7, 2, 1, 96, 96, False, False, "odd"),
    (3, 5, 0, 256, 64, False, True, "odd"),
    (4, 0, 2, 512, 512, True, False, "plain"),
    (2, 3, 1, 320, 160, False, True, "heads first"),
    (33, 7, 1, 80, 0, False, False, "slice"),
    (700, 40, 8, 128, 128, False, True, "slice"),   # four heads a lane group
    (700, 37, 9, 128, 64, True, True, "plain"),     # and head counts that are not multiples of 4
]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("weight", [True, False])
def test_forward(form, weight):
    import post_weight_quantization_03_amd as g
    tokens, qh, kh, dim, rot, inter, bf16, layout = form
    say(f"norm_rope {form} weight={weight}")
    torch, _ = torch_dev()
    eps = 1e-5
    q, k, w, cos, sin, pos, _ = _inputs(tokens, qh, kh, dim, rot, bf16, 11, weight)
    st = to_dev(np.zeros(1, np.int32))
    qo, ko = g.gptq_qk_norm_rope(on_device(q, bf16, layout) if qh else None, on_device(k, bf16, layout) if kh else None,
                                 to_dev(pos), _rope(cos, sin, inter, eps), _dev(w[0], bf16), _dev(w[1], bf16),
                                 d_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for name, x, ww, y in (("q", q, w[0], qo), ("k", k, w[1], ko)):
        if y is None:
            continue
        want = R.norm_rope(x, ww, cos, sin, pos, inter, eps)
        bound = 40 * U * _mag(x, ww, cos, sin, pos, inter, eps) + (H if bf16 else U) * np.abs(want) + 1e-40
        close(name, y.float().cpu().numpy(), want, bound)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("weight", [True, False])
def test_backward(form, weight):
    import post_weight_quantization_03_amd as g
    tokens, qh, kh, dim, rot, inter, bf16, layout = form
    say(f"norm_rope backward {form} weight={weight}")
    torch, _ = torch_dev()
    eps = 1e-5
    q, k, w, cos, sin, pos, rng = _inputs(tokens, qh, kh, dim, rot, bf16, 12, weight)
    dy = [values(rng, x.shape, bf16) for x in (q, k)]
    put = lambda x: on_device(x, bf16, layout) if x.shape[1] else None  # noqa: E731
    got = g.gptq_qk_norm_rope_backward(put(dy[0]), put(dy[1]), put(q), put(k), to_dev(pos), _rope(cos, sin, inter, eps),
                                       _dev(w[0], bf16) if qh else None, _dev(w[1], bf16) if kh else None)
    again = g.gptq_qk_norm_rope_backward(put(dy[0]), put(dy[1]), put(q), put(k), to_dev(pos),
                                         _rope(cos, sin, inter, eps), _dev(w[0], bf16) if qh else None,
                                         _dev(w[1], bf16) if kh else None)
    torch.cuda.synchronize()
    for a, b in zip(got, again):
        assert (a is None and b is None) or torch.equal(a, b)  # the order of every sum is fixed
    for name, x, ww, d, dx, dw in (("q", q, w[0], dy[0], got[0], got[2]), ("k", k, w[1], dy[1], got[1], got[3])):
        if dx is None:
            continue
        want, want_w = R.norm_rope_backward(d, x, ww, cos, sin, pos, inter, eps)
        D = _mag(d, None, cos, sin, pos, inter, eps)  # magnitudes do not care for the angle's sign
        bound = (H if bf16 else U) * np.abs(want) + 1e-40
        if ww is None:
            close("d" + name, dx.float().cpu().numpy(), want, bound + 6 * U * D)
            continue
        r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        gm = np.abs(ww) * D
        bound = bound + 44 * U * r * gm + 152 * U * np.abs(x) * r ** 3 * (gm * np.abs(x)).mean(-1, keepdims=True)
        close("d" + name, dx.float().cpu().numpy(), want, bound)
        groups = 256 // (1 << max(0, (dim // 16 - 1)).bit_length())
        items = tokens * x.shape[1]
        chain = -(-items // (groups * min(512, -(-items // groups)))) + 10 + 48
        close("d" + name + "_weight", dw.cpu().numpy(), want_w,
              2 * (20 + chain) * U * (D * np.abs(x) * r).sum((0, 1)) + 1e-40)


def test_gradient_against_differences_on_the_device():
    """A loss sum(y dy) in fp32 through the forward kernel, against the backward kernel's dx and dw.
    Differences of step h: the loss, a sum of about 500 terms of size 1, is off by some 500 * 40 u * 4, so the
    quotient by up to 5e-3 / h * 1e-1 and by h^2 of the curvature: h = 2^-6 leaves 3e-2."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    q, _, w, cos, sin, pos, rng = _inputs(2, 2, 0, 128, 128, False, 13)
    w0 = 1.0 + 0.1 * w[0]
    dy = values(rng, q.shape, False)
    rope = _rope(cos, sin, False, 1e-5)

    def loss(x, ww):
        y, _ = g.gptq_qk_norm_rope(on_device(x, False), None, to_dev(pos), rope, _dev(ww, False))
        return float((y.double().cpu().numpy() * dy).sum())

    dx, _, dw, _ = g.gptq_qk_norm_rope_backward(on_device(dy, False), None, on_device(q, False), None, to_dev(pos), rope,
                                                _dev(w0, False))
    dx, dw = dx.cpu().numpy(), dw.cpu().numpy()
    h = 2.0 ** -6
    for idx in [(0, 0, 0), (0, 1, 70), (1, 0, 127), (1, 1, 31)]:
        e = np.zeros_like(q)
        e[idx] = h
        assert abs((loss(q + e, w0) - loss(q - e, w0)) / (2 * h) - dx[idx]) < 3e-2
    for i in (0, 64, 127):
        e = np.zeros(128)
        e[i] = h
        assert abs((loss(q, w0 + e) - loss(q, w0 - e)) / (2 * h) - dw[i]) < 3e-2


def test_in_place_and_on_another_stream():
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    q, k, w, cos, sin, pos, _ = _inputs(50, 8, 2, 128, 128, True, 14)
    rope, p = _rope(cos, sin, False, 1e-6), to_dev(pos)
    dq, dk, wq, wk = on_device(q, True, "slice"), on_device(k, True), _dev(w[0], True), _dev(w[1], True)
    a, b = g.gptq_qk_norm_rope(dq, dk, p, rope, wq, wk)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c, d = g.gptq_qk_norm_rope(dq, dk, p, rope, wq, wk, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, c) and torch.equal(b, d)
    g.gptq_qk_norm_rope(dq, dk, p, rope, wq, wk, q_out=dq, k_out=dk)
    assert torch.equal(a, dq) and torch.equal(b, dk)


def test_positions_out_of_range_are_raised_and_touch_no_other_token():
    import post_weight_quantization_03_amd as g
    torch, _ = torch_dev()
    q, k, w, cos, sin, pos, _ = _inputs(6, 4, 2, 128, 128, True, 15)
    args = on_device(q, True), on_device(k, True)
    rope = _rope(cos, sin, False, 1e-6)
    good, _ = g.gptq_qk_norm_rope(*args, to_dev(pos), rope)
    for bad in (-1, 97, 2 ** 31 - 1, -2 ** 31):
        p = pos.copy()
        p[3] = bad
        st = to_dev(np.zeros(1, np.int32))
        y, _ = g.gptq_qk_norm_rope(*args, to_dev(p), rope, d_status=st)
        assert int(st) == g.GPTQ_EINVAL
        for t in (0, 1, 2, 4, 5):
            assert torch.equal(y[t], good[t])


def test_values_that_are_not_finite_stay_in_their_head():
    import post_weight_quantization_03_amd as g
    torch, _ = torch_dev()
    q, k, w, cos, sin, pos, _ = _inputs(4, 4, 1, 128, 128, True, 16)
    rope, p = _rope(cos, sin, False, 1e-6), to_dev(pos)
    good, _ = g.gptq_qk_norm_rope(on_device(q, True), None, p, rope, _dev(w[0], True))
    x = on_device(q, True)
    x[1, 2, 5] = float("nan")
    x[2, 0, 7] = float("inf")
    y, _ = g.gptq_qk_norm_rope(x, None, p, rope, _dev(w[0], True))
    assert torch.isnan(y[1, 2]).all() and torch.isnan(y[2, 0]).any()
    keep = torch.ones((4, 4), dtype=torch.bool)
    keep[1, 2] = keep[2, 0] = False
    assert torch.equal(y[keep.to(y.device)], good[keep.to(y.device)])


def test_backward_of_no_tokens_gives_zero_weight_gradients():
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    e = torch.empty((0, 4, 128), dtype=torch.bfloat16, device=dev)
    w = torch.ones(128, dtype=torch.bfloat16, device=dev)
    _, _, dw, _ = g.gptq_qk_norm_rope_backward(e, None, e, None, torch.empty(0, dtype=torch.int32, device=dev),
                                               g.Rope(None, None), w)
    assert torch.equal(dw, torch.zeros(128, device=dev))
