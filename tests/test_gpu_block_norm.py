"""The norms around a block on the GPU, forward and backward, against the float64 oracle.

Tolerance of every element, from its size S (block_norm_oracle: the same sums with every
term's magnitude), u = 2^-24:

    |g - o| <= half |o| + (160 + n) u S

half is half a step of the output's type (bf16 2^-8; float32 2^-24, in the second part).
A float32 term carries: 2 factors' statistics, each a sum of d squares kept in at most
32 sequential steps a lane (d <= 16,384 over its team) and 10 joining ones, halved by the
root and one rounding for it: 2 * 23; the sum inside a norm's Jacobian, 42 more; the gate's
function, whose exponential is within 2 and which is within 8 altogether, twice: 16; and
under 16 products and sums: 120 in all, 160 with second-order terms.  n = 0, except the
sums over tokens: n terms added one after another at most, n = T.  A bf16 sum y of expert
rows is not rounded in between, its k <= 8 additions are within the 40 spare.
"""
import numpy as np
import pytest
import torch

from mixture_experts_layer_16_amd import binding as B
from mixture_experts_layer_16_amd import workloads as W
from oracle import block_norm_oracle as bno
from parity_util import bits_equal, f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32


def check(g, o, size, dt, what, n=0):
    g, o, size = f64(g).reshape(o.shape), np.asarray(o), np.asarray(size)
    half = 2.0 ** -8 if g is not None and dt == BF else 0.0
    bound = half * np.abs(o) + (160 + n) * U * size + 1e-40
    err = np.abs(g - o)
    assert np.all(np.isfinite(g)), f"{what}: not finite"
    worst = (err / bound).max()
    assert worst <= 1, f"{what}: {worst:.3g} times its bound (error {err.max():.3e})"


def draw(T, d, dt, branch="y", post=True, gate_rows=0, nxt=True, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * std

    v = dict(x=rnd(T, d, std=2.0).to(dt), y=None, y_perm=None, slot_row=None, topk_w=None, post_gain=None, gate=None,
             next_gain=None)
    if branch == "y":
        v["y"] = rnd(T, d, std=0.5).to(dt)
    elif branch:
        k = branch
        v["y_perm"] = rnd(T * k, d).to(dt)
        sr = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k)
        sr = torch.where(torch.rand(T, k, generator=g, device=DEV) < 0.2, -1, sr)
        sr[0] = -1                         # a token none of whose experts is here
        v["slot_row"], v["topk_w"] = sr, torch.rand(T, k, generator=g, device=DEV)
    if post:
        v["post_gain"] = 1 + rnd(d, std=0.2)
    if gate_rows:
        v["gate"] = rnd(-(-T // gate_rows), d).to(dt)
    if nxt:
        v["next_gain"] = 1 + rnd(d, std=0.2)
    return v, rnd(T, d).to(dt), rnd(T, d).to(dt) if nxt else None


def oracle_forward(v, gate_rows, act, rs=0.9, bs=0.7, eps=1e-6):
    y = size = None
    if v["y"] is not None:
        y = f64(v["y"])
    elif v["y_perm"] is not None:
        y, size = bno.combine(f64(v["y_perm"]), v["slot_row"].cpu().numpy(), f64(v["topk_w"]))
    return bno.forward(f64(v["x"]), y, f64(v["post_gain"]), f64(v["gate"]), gate_rows, act, rs, bs, eps,
                       f64(v["next_gain"]), size), y, size


def forward(v, gate_rows=0, act="none", rs=0.9, bs=0.7, eps=1e-6, **kw):
    return B.moe_block_norm(**v, gate_rows=gate_rows, gate_act=act, res_scale=rs, branch_scale=bs, eps=eps, **kw)


def run_case(T, d, dt, branch, post, gate_rows, act, nxt, seed=0):
    print(f"[block norm] T={T} d={d} {dt} branch={branch} post={post} gate_rows={gate_rows} {act} next={nxt}", flush=True)
    v, d_out, dh = draw(T, d, dt, branch, post, gate_rows, nxt, seed)
    got = forward(v, gate_rows, act, want_y=isinstance(branch, int))
    torch.cuda.synchronize()
    (out, h, so, sh), y, ysize = oracle_forward(v, gate_rows, act)
    if branch:
        check(got.out, out, so, dt, "out")
    else:
        assert got.out is None
    if nxt:
        check(got.h, h, sh, dt, "h")
    else:
        assert got.h is None
    yk = v["y"]
    if isinstance(branch, int):
        check(got.y_out, y, ysize, dt, "y_out")
        yk = got.y_out

    # backward from what the forward wrote
    kept = got.out if branch else v["x"]
    rs = 0.9 if branch else 1.0
    b = B.moe_block_norm_backward(d_out, dh, out=kept, y=yk, post_gain=v["post_gain"], gate=v["gate"],
                                  gate_rows=gate_rows, gate_act=act, next_gain=v["next_gain"], res_scale=rs,
                                  branch_scale=0.7)
    torch.cuda.synchronize()
    want = bno.backward(f64(kept), f64(yk), f64(v["post_gain"]), f64(v["gate"]), gate_rows, act, rs, 0.7, 1e-6,
                        f64(v["next_gain"]), f64(d_out), f64(dh))
    for name in ("dx", "dy", "d_post_gain", "dgate", "d_next_gain"):
        g = getattr(b, name)
        assert (g is None) == (name not in want), name
        if g is not None:
            rows = name in ("dx", "dy") or (name == "dgate" and gate_rows == 1)
            assert g.dtype == (dt if rows else FP)
            check(g, *want[name], g.dtype, name, 0 if rows else T)


WIDTHS = [64, 128, 192, 256, 320, 512, 576, 1024, 1088, 1536, 1600, 2048, 2112, 2496, 3136, 4096, 4160, 6144, 6208, 8192, 8256, 16384]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("d", WIDTHS)
def test_every_width(d, dt):
    run_case(37, d, dt, "y", True, 10, "tanh", True, seed=d)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 255, 1000])
def test_row_counts(T, dt):
    run_case(T, 192, dt, "y", True, T, "sigmoid", True, seed=T)
    run_case(T, 1088, dt, "y", True, 1, "tanh", True, seed=T)


@pytest.mark.parametrize("branch", [None, "y", 1, 2, 3, 8])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate_rows,act", [(0, "none"), (1, "none"), (4, "sigmoid"), (77, "tanh")])
@pytest.mark.parametrize("nxt", [False, True])
def test_every_combination(branch, post, gate_rows, act, nxt):
    if branch is None and (post or gate_rows or not nxt):
        pytest.skip("no branch: only the norm before a block")
    run_case(41, 576, BF, branch, post, gate_rows, act, nxt, seed=3)


@pytest.mark.parametrize("gate_rows", [1, 2, 3, 7, 700, 1699, 5999, 6000, 6001, 10 ** 12, 2 ** 63 - 1])
def test_gate_groups_over_many_teams(gate_rows):
    # narrow rows, a few a team: groups lie inside, straddle and span teams
    run_case(6000, 64, BF, "y", True, gate_rows, "tanh", True, seed=9)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("gate_rows", [0, 1, 5, 9, 31, 65, 200, 4001])
@pytest.mark.parametrize("d", [64, 128, 256, 448, 512])
def test_several_teams_a_wavefront(d, gate_rows, dt):
    # teams of 8 to 64 lanes; workgroups whose teams share a gate group, and that do not, and a
    # last one with teams that have no rows
    run_case(4001, d, dt, "y", True, gate_rows, "tanh" if gate_rows else "none", True, seed=d + gate_rows)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 2, 63, 300])
def test_several_teams_a_wavefront_from_expert_rows(T, d):
    run_case(T, d, BF, 3, True, 7, "sigmoid", True, seed=T)


@pytest.mark.parametrize("d", [64, 192, 512])
def test_narrow_rows_past_the_caches(d):
    # more than 32 MB a tensor, and more rows than teams
    T = (33 << 20) // (2 * d) + 5
    run_case(T, d, BF, "y", True, 1000, "sigmoid", True, seed=d)


@pytest.mark.parametrize("gate_rows", [3, 130, 1500])
def test_gate_groups_of_wide_rows(gate_rows):
    run_case(1501, 2112, FP, "y", True, gate_rows, "sigmoid", True, seed=10)


def test_gradients_match_differences():
    # central differences of the kernel's own float32 forward, summed against random
    # gradients in 64 bits.  A direction of step e moves the value by e <g, v>; the forward's
    # rounding (at most 160 u of each output's size) over 2e and the third derivative (e^2)
    # bound the quotient's error
    v, d_out, dh = draw(9, 128, FP, "y", True, 4, True, seed=21)
    got = forward(v, 4, "tanh")
    b = B.moe_block_norm_backward(d_out, dh, out=got.out, y=v["y"], post_gain=v["post_gain"], gate=v["gate"],
                                  gate_rows=4, gate_act="tanh", next_gain=v["next_gain"], res_scale=0.9,
                                  branch_scale=0.7)
    e = 2.0 ** -6

    def value(w):
        n = forward(w, 4, "tanh")
        return float((n.out.double() * d_out.double()).sum() + (n.h.double() * dh.double()).sum())

    (_, _, so, sh), _, _ = oracle_forward(v, 4, "tanh")
    noise = 160 * U * float((so * np.abs(f64(d_out))).sum() + (sh * np.abs(f64(dh))).sum()) / e
    for name, grad in (("x", b.dx), ("y", b.dy), ("post_gain", b.d_post_gain), ("gate", b.dgate),
                       ("next_gain", b.d_next_gain)):
        gen = torch.Generator(device=DEV).manual_seed(5)
        way = torch.randn(v[name].shape, generator=gen, device=DEV)
        way = way / way.norm() * 4
        moved = [dict(v, **{name: v[name] + s * e * way}) for s in (1, -1)]
        slope = (value(moved[0]) - value(moved[1])) / (2 * e)
        want = float((grad.double() * way.double()).sum())
        # third derivative: |way|^3 = 64 times derivatives of order 1 of values of order |d_out| + |dh|
        third = e * e * 64 * float((d_out.double() ** 2).sum() + (dh.double() ** 2).sum()) ** 0.5
        print(f"[differences] {name} {slope:.6f} {want:.6f} bound {noise + third:.6f}", flush=True)
        assert abs(slope - want) <= noise + third, name


def test_only_one_gradient_given():
    v, d_out, dh = draw(20, 192, BF, "y", True, 0, True, seed=1)
    n = forward(v)
    kw = dict(out=n.out, y=v["y"], post_gain=v["post_gain"], next_gain=v["next_gain"], branch_scale=0.7)
    b = B.moe_block_norm_backward(None, dh, **kw)
    zero = B.moe_block_norm_backward(torch.zeros_like(dh), dh, **kw)
    for name in ("dx", "dy", "d_post_gain", "d_next_gain"):
        assert bits_equal(getattr(b, name), getattr(zero, name)), name


@pytest.mark.parametrize("dt", [BF, FP])
def test_over_the_input(dt):
    v, d_out, dh = draw(70, 1088, dt, "y", True, 16, True, seed=2)
    a = forward(v, 16, "tanh")
    x = v["x"].clone()
    over = forward(dict(v, x=x), 16, "tanh", out=x)
    assert over.out is x and bits_equal(x, a.out) and bits_equal(over.h, a.h)
    kw = dict(out=a.out, y=v["y"], post_gain=v["post_gain"], gate=v["gate"], gate_rows=16, gate_act="tanh",
              next_gain=v["next_gain"])
    want = B.moe_block_norm_backward(d_out, dh, **kw)
    g = d_out.clone()
    b = B.moe_block_norm_backward(g, dh, dx=g, **kw)
    assert b.dx is g
    for name in ("dx", "dy", "d_post_gain", "dgate", "d_next_gain"):
        assert bits_equal(getattr(b, name), getattr(want, name)), name


@pytest.mark.parametrize("d", [64, 128, 256, 576])       # 64 to 256: rows that share a wavefront
def test_rows_of_zeros_and_of_nan_stay_theirs(d):
    v, d_out, dh = draw(6, d, BF, "y", True, 0, True, seed=6)
    clean = forward(v)
    w = dict(v, x=v["x"].clone(), y=v["y"].clone())
    w["y"][1] = 0
    w["x"][2], w["y"][2] = 0, 0
    w["y"][4, 3] = float("nan")
    w["x"][5, 7] = float("inf")
    n = forward(w)
    assert bits_equal(n.out[[0, 3]], clean.out[[0, 3]]) and bits_equal(n.h[[0, 3]], clean.h[[0, 3]])
    assert torch.equal(n.out[1].float(), (0.9 * w["x"][1].float()).to(BF).float())
    assert not n.out[2].any() and not n.h[2].any()
    assert n.out[4].isnan().all() and n.h[4].isnan().all()
    assert n.out[5, 7].isinf()
    kw = dict(y=v["y"], post_gain=v["post_gain"], next_gain=v["next_gain"])
    a = B.moe_block_norm_backward(d_out, dh, out=clean.out, **kw)
    bad = d_out.clone()
    bad[4, 0] = float("nan")
    b = B.moe_block_norm_backward(bad, dh, out=clean.out, **kw)
    rows = [0, 1, 2, 3, 5]
    assert bits_equal(b.dx[rows], a.dx[rows]) and bits_equal(b.dy[rows], a.dy[rows])


def test_slots_outside_the_rows_are_skipped():
    v, _, _ = draw(9, 192, BF, 4, True, 0, True, seed=8)
    want = forward(v, want_y=True)
    w = dict(v, slot_row=torch.where(v["slot_row"] < 0, torch.tensor(36, dtype=torch.int32, device=DEV),
                                     v["slot_row"]))
    got = forward(w, want_y=True)
    w["slot_row"] = torch.where(v["slot_row"] < 0, torch.tensor(2 ** 31 - 1, dtype=torch.int32, device=DEV),
                                v["slot_row"])
    far = forward(w, want_y=True)
    for n in (got, far):
        assert bits_equal(n.out, want.out) and bits_equal(n.h, want.h) and bits_equal(n.y_out, want.y_out)


def test_the_combine_inside_is_moe_combine():
    v, _, _ = draw(50, 1024, BF, 8, False, 0, False, seed=11)
    n = forward(v, want_y=True, rs=0.0, bs=1.0)
    y = B.moe_combine(v["y_perm"], v["slot_row"], v["topk_w"])
    assert bits_equal(n.y_out, y)


def test_results_are_reproducible():
    v, d_out, dh = draw(5000, 1024, BF, "y", True, 1300, True, seed=12)
    n = forward(v, 1300, "sigmoid")
    kw = dict(out=n.out, y=v["y"], post_gain=v["post_gain"], gate=v["gate"], gate_rows=1300, gate_act="sigmoid",
              next_gain=v["next_gain"])
    a, b = (B.moe_block_norm_backward(d_out, dh, **kw) for _ in range(2))
    for name in ("dx", "dy", "d_post_gain", "dgate", "d_next_gain"):
        assert bits_equal(getattr(a, name), getattr(b, name)), name


def test_offsets_past_32_bits():
    # 2.16e9 elements a tensor, compared on rows at both ends and around 2^31 elements
    T, d = 131900, 16384
    print(f"[block norm] T={T} d={d}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(T, d, dtype=BF, device=DEV)
    for i in range(0, T, 8192):
        n = min(8192, T - i)
        x[i:i + n] = torch.randn(n, d, generator=g, device=DEV).to(BF)
    post, nxt = (1 + 0.2 * torch.randn(d, generator=g, device=DEV) for _ in range(2))
    gate = torch.randn(2, d, generator=g, device=DEV).to(BF)
    n = B.moe_block_norm(x, x, post_gain=post, next_gain=nxt, gate=gate, gate_rows=131000, gate_act="tanh")
    rows = torch.tensor([0, 1, 130999, 131000, 131071, 131072, 131073, T - 1], device=DEV)
    xs, table = f64(x[rows]), f64(gate)[[0, 0, 0, 1, 1, 1, 1, 1]]
    out, h, so, sh = bno.forward(xs, xs, f64(post), table, 1, "tanh", 1.0, 1.0, 1e-6, f64(nxt))
    check(n.out[rows], out, so, BF, "out")
    check(n.h[rows], h, sh, BF, "h")
    b = B.moe_block_norm_backward(n.h, x, out=n.out, y=x, post_gain=post, next_gain=nxt, gate=gate, gate_rows=131000,
                                  gate_act="tanh")
    want = bno.backward(f64(n.out[rows]), xs, f64(post), table, 1, "tanh", 1.0, 1.0, 1e-6, f64(nxt), f64(n.h[rows]), xs)
    check(b.dx[rows], *want["dx"], BF, "dx")
    check(b.dy[rows], *want["dy"], BF, "dy")


def replays_match(calls, outs, expected):
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            for c in calls:
                c()
    torch.cuda.current_stream().wait_stream(s)
    junk = torch.randn(1 << 20, device=DEV)
    for i in range(4):
        for o in outs:
            o.fill_(float("nan"))
        junk.mul_(1.0001)
        g.replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, expected):
            assert bits_equal(o, e), f"replay {i} differs"
    return g


def test_graph_replays_and_streams_match_eager():
    v, d_out, dh = draw(900, 1088, BF, "y", True, 200, True, seed=13)
    F = B.BlockNorm(**v, gate_rows=200, gate_act="tanh", branch_scale=0.7)
    R = B.BlockNormBackward(d_out, dh, out=F.out, y=v["y"], post_gain=v["post_gain"], gate=v["gate"], gate_rows=200,
                            gate_act="tanh", next_gain=v["next_gain"], branch_scale=0.7)
    F(), R()
    torch.cuda.synchronize()
    outs = [F.out, F.h, R.dx, R.dy, R.d_post_gain, R.dgate, R.d_next_gain]
    expected = [o.clone() for o in outs]
    other = torch.cuda.Stream()
    for o in outs:
        o.fill_(float("nan"))
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        F(), R()
    torch.cuda.current_stream().wait_stream(other)
    torch.cuda.synchronize()
    for o, e in zip(outs, expected):
        assert bits_equal(o, e)
    replays_match([F, R], outs, expected)


def test_a_training_block_runs_together():
    """norm -> routed layer -> norm, gate and residual, and back, against float64 end to end."""
    from oracle import moe_layer_backward_oracle as lbo
    from oracle import moe_oracle as orc
    T, d, E, k, F = 120, 128, 8, 2, 64
    wl = W.Workload("block", T, d, E, k, F, FP)
    inp = W.make_inputs(wl, device=DEV, seed=4)
    x = inp["x"]
    g = torch.Generator(device=DEV).manual_seed(8)
    g1, g2, g3 = (1 + 0.1 * torch.randn(d, generator=g, device=DEV) for _ in range(3))
    gate = torch.randn(1, d, generator=g, device=DEV)
    pre = B.moe_block_norm(x, next_gain=g1)
    L = B.moe_layer_forward(pre.h, inp["w_router"], None, inp["w_gate"], inp["w_up"], inp["w_down"], k,
                            want_routing=True, want_y_perm=True)
    post = B.moe_block_norm(x, L.y, post_gain=g2, gate=gate, gate_rows=T, gate_act="tanh", next_gain=g3)
    d_out, dh = torch.randn(2, T, d, generator=g, device=DEV)
    pb = B.moe_block_norm_backward(d_out, dh, out=post.out, y=L.y, post_gain=g2, gate=gate, gate_rows=T,
                                   gate_act="tanh", next_gain=g3)
    LB = B.moe_layer_backward(pre.h, inp["w_router"], inp["w_gate"], inp["w_up"], inp["w_down"], L.topk_ids, L.topk_w,
                              L.y_perm, pb.dy)
    fb = B.moe_block_norm_backward(pb.dx, LB.dx, out=x, next_gain=g1)
    torch.cuda.synchronize()

    X, G1, G2, G3, GT = (f64(t) for t in (x, g1, g2, g3, gate))
    Wr, Wg, Wu, Wd = (f64(inp[n]) for n in ("w_router", "w_gate", "w_up", "w_down"))
    H = bno.forward(X, None, None, None, 0, "none", 1, 1, 1e-6, G1)[1]
    ref = orc.layer_forward(H, Wr, None, Wg, Wu, Wd, k, ids=L.topk_ids.cpu().numpy(), weights=f64(L.topk_w))
    out, h, _, _ = bno.forward(X, ref["y"], G2, GT, T, "tanh", 1, 1, 1e-6, G3)
    wb = bno.backward(out, ref["y"], G2, GT, T, "tanh", 1, 1, 1e-6, G3, f64(d_out), f64(dh))
    lb = lbo.layer_backward(H, Wr, Wg, Wu, Wd, L.topk_ids.cpu().numpy(), f64(L.topk_w), ref["y_perm"],
                            wb["dy"][0])
    fw = bno.backward(X, None, None, None, 0, "none", 1, 1, 1e-6, G1, wb["dx"][0], lb["dx"])
    # the framework's float32 rule, ten layers of it: the routed layer's own outputs are held to
    # 1e-5 of their largest value, and its errors pass through two norms and the layer's Jacobian
    for name, a, o in (("out", post.out, out), ("h", post.h, h), ("dx", fb.dx, fw["dx"][0]),
                       ("dgate", pb.dgate, wb["dgate"][0]), ("d_post_gain", pb.d_post_gain, wb["d_post_gain"][0]),
                       ("d_first_gain", fb.d_next_gain, fw["d_next_gain"][0])):
        err = np.abs(f64(a) - o).max()
        assert err <= 1e-4 * np.abs(o).max(), (name, err, np.abs(o).max())
