"""The block norm and 4-bit oracles against finite differences, torch.autograd and
closed forms (no GPU needed)."""
import numpy as np
import pytest
import torch

from oracle import block_norm_oracle as bno
from oracle import w4_oracle as w4o

CASES = [(5, 12, True, 2, "tanh", True), (4, 6, True, 1, "sigmoid", True), (6, 8, False, 6, "none", True),
         (3, 5, True, 0, "none", False), (7, 9, False, 3, "sigmoid", False), (4, 7, None, 0, "none", True)]


def draw(T, d, post, gate_rows, nxt, seed=0):
    g = np.random.default_rng(seed)
    v = {"x": g.normal(size=(T, d)), "y": None if post is None else g.normal(size=(T, d)),
         "post_gain": g.normal(size=d) if post else None,
         "gate": g.normal(size=(-(-T // gate_rows), d)) if gate_rows else None,
         "next_gain": g.normal(size=d) if nxt else None}
    return v, g.normal(size=(T, d)), (g.normal(size=(T, d)) if nxt else None)


def value(v, gate_rows, kind, d_out, dh):
    out, h, _, _ = bno.forward(v["x"], v["y"], v["post_gain"], v["gate"], gate_rows, kind, 0.9, 0.7, 1e-3,
                               v["next_gain"])
    return (out * d_out).sum() + (0.0 if h is None else (h * dh).sum())


@pytest.mark.parametrize("T,d,post,gate_rows,kind,nxt", CASES)
def test_backward_matches_differences(T, d, post, gate_rows, kind, nxt):
    v, d_out, dh = draw(T, d, post, gate_rows, nxt)
    out = bno.forward(v["x"], v["y"], v["post_gain"], v["gate"], gate_rows, kind, 0.9, 0.7, 1e-3, None)[0]
    got = bno.backward(out, v["y"], v["post_gain"], v["gate"], gate_rows, kind, 0.9 if post is not None else 1.0, 0.7,
                       1e-3, v["next_gain"], d_out, dh)
    names = {"x": "dx", "y": "dy", "post_gain": "d_post_gain", "gate": "dgate", "next_gain": "d_next_gain"}
    step = 1e-5
    for name, grad in names.items():
        if v[name] is None:
            assert grad not in got
            continue
        flat, want = v[name].reshape(-1), got[grad][0].reshape(-1)
        for i in range(flat.size):
            was = flat[i]
            flat[i] = was + step
            up = value(v, gate_rows, kind, d_out, dh)
            flat[i] = was - step
            down = value(v, gate_rows, kind, d_out, dh)
            flat[i] = was
            # central differences: the third derivative's term, and 64-bit rounding over the step
            assert abs((up - down) / (2 * step) - want[i]) <= 1e-7 * (1 + abs(want[i])), (name, i)


def test_forward_matches_torch():
    v, _, _ = draw(6, 16, True, 3, True, seed=4)
    t = {k: torch.from_numpy(a) for k, a in v.items()}
    n = torch.nn.functional.rms_norm(t["y"], (16,), t["post_gain"], eps=1e-3)
    out = 0.9 * t["x"] + 0.7 * torch.tanh(t["gate"]).repeat_interleave(3, 0) * n
    h = torch.nn.functional.rms_norm(out, (16,), t["next_gain"], eps=1e-3)
    got = bno.forward(v["x"], v["y"], v["post_gain"], v["gate"], 3, "tanh", 0.9, 0.7, 1e-3, v["next_gain"])
    assert np.allclose(got[0], out.numpy(), rtol=1e-13, atol=1e-13)
    assert np.allclose(got[1], h.numpy(), rtol=1e-13, atol=1e-13)


def test_combine_skips_missing_slots():
    y_perm = np.arange(12.0).reshape(4, 3)
    y, size = bno.combine(y_perm, [[0, -1], [3, 1], [-1, 9]], [[0.5, 9.0], [-1.0, 2.0], [1.0, 1.0]])
    assert np.array_equal(y, [[0, .5, 1], [-3, -2, -1], [0, 0, 0]])
    assert np.array_equal(size, [[0, .5, 1], [15, 18, 21], [0, 0, 0]])


def test_bf16_rounding_matches_torch():
    g = np.random.default_rng(1)
    a = np.concatenate([g.normal(size=4096), g.normal(size=4096) * 1e-38, [0.0, -0.0, 1.00390625, 1.01171875]])
    a = a.astype(np.float32)
    want = torch.from_numpy(a).to(torch.bfloat16).float().numpy()
    assert np.array_equal(w4o.round_bf16(a).view(np.uint32), want.view(np.uint32))


def test_quantize_by_hand():
    # largest magnitude 7: scale 1, codes are the rounded values + 8, halves to even
    w = np.array([[7.0, -7.0, 0.5, 1.5, -2.5, 6.4999, 0.0, 3.0] + [0.0] * 24])
    q, s = w4o.quantize(w, 32)
    assert s.tolist() == [[1.0]]
    assert q[0, :8].tolist() == [15, 1, 8, 10, 6, 14, 8, 11]
    assert w4o.values(q, s, 32)[0, :8].tolist() == [7, -7, 0, 2, -2, 6, 0, 3]
    q, s = w4o.quantize(np.zeros((2, 40)), 32)
    assert np.all(q == 8) and np.all(s == 0) and s.shape == (2, 2)


def test_quantize_error_is_half_a_step():
    g = np.random.default_rng(2)
    w = g.normal(size=(5, 160))
    for group in (32, 64, 128):
        q, s = w4o.quantize(w, group)
        step = s[:, np.arange(160) // group]
        # |w| <= 7 s (1 + 2^-8) for s rounded down by at most half a bf16 step
        assert np.all(np.abs(w4o.values(q, s, group) - w) <= step * (0.5 + 7 * 2 ** -8))


def test_products_are_the_matrix_product():
    g = np.random.default_rng(3)
    q, s = g.integers(0, 16, size=(6, 96)), g.random(size=(6, 3))
    x = g.normal(size=(4, 96))
    y, sx, swx = w4o.products(x, q, s, 32)
    for t in range(4):
        for r in range(6):
            terms = [s[r, c // 32] * (q[r, c] - 8.0) * x[t, c] for c in range(96)]
            assert abs(y[t, r] - sum(terms)) < 1e-12
            assert abs(swx[t, r] - sum(abs(v) for v in terms)) < 1e-12
            assert abs(sx[t, r] - sum(abs(s[r, c // 32] * x[t, c]) for c in range(96))) < 1e-12
