"""4-bit weights on the GPU: quantisation, layout, and the products, against the float64 oracle.

Tolerance of a product's element y = sum_c s (q - 8) x (u = 2^-24, half = half a step of
the output's type: bf16 2^-8, float32 2^-24):

    |g - y| <= half |y| + 48 u P + (C/128 + 8) u sum|s (q - 8) x| + 2^-23 sum|s (q - 8) x|

P is what a group's partial sums are at most.  With bf16 activations the codes enter the
sums as 128 + q or 16 + q with the offset taken out inside a group: P = A sum|s x|,
A = 136 + 143.  With float32 ones they enter as q - 8: P = sum|s (q - 8) x|.  32 products
of an MFMA and at most 12 MFMAs that follow one another round each partial sum, 48 in all.
The groups' totals are then added C/128 times and over four wavefronts.  Float32 activations
are three bf16 numbers whose sum is within 2^-24 of them; 2^-23 holds that and the
second plane's 2^-16 of the hidden activations is counted where they are.
"""
import numpy as np
import pytest
import torch

from mixture_experts_layer_16_amd import binding as B
from oracle import w4_oracle as w4o
from parity_util import bits_equal, f64
from test_gpu_block_norm import replays_match

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def packed(n, R, C, group, seed=0, scale=None):
    """(W4Weights, codes [n, R, C], scales [n, R, groups]) with random codes"""
    g = gen(seed)
    q = torch.randint(0, 16, (n, R, C), generator=g, device=DEV, dtype=torch.uint8)
    s = (torch.rand(n, R, -(-C // group), generator=g, device=DEV) + 0.1).to(BF) if scale is None else \
        torch.full((n, R, -(-C // group)), scale, device=DEV, dtype=BF)
    w = B.moe_w4_pack((q[..., 0::2] | q[..., 1::2] << 4).contiguous(), s, group)
    return w, q.cpu().numpy().astype(np.float64), f64(s)


def product_bound(x, q, s, group, dt):
    """(y, error of the float32 evaluation)"""
    y, sx, swx = w4o.products(x, q, s, group)
    return y, 48 * U * (279.0 * sx if dt == BF else swx) + (q.shape[-1] / 128 + 8) * U * swx + 2.0 ** -23 * swx


def check(g, o, err, dt, what):
    g = f64(g)
    bound = (2.0 ** -8 if dt == BF else U) * np.abs(o) + err + 1e-40
    assert np.all(np.isfinite(g)), f"{what}: not finite"
    worst = (np.abs(g - o) / bound).max()
    assert worst <= 1, f"{what}: {worst:.3g} times its bound"


# ---- quantisation and layout ------------------------------------------------

@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,R,C", [(1, 1, 32), (1, 16, 128), (3, 15, 96), (2, 17, 160), (1, 515, 1024), (2, 33, 416)])
def test_quantize_gives_the_oracles_values(n, R, C, group, dt):
    print(f"[quantize] {n} {R} {C} {group} {dt}", flush=True)
    w = torch.randn(n, R, C, generator=gen(R + C), device=DEV)
    w[0, 0, :32] = 0
    w[-1, -1, :8] = torch.tensor([7.0, -7.0, 0.5, 1.5, -2.5, 3.5, -0.5, 0.0], device=DEV)
    w[-1, -1, 8:32] = 0
    w = w.to(dt)
    got = B.moe_w4_quantize(w, group)
    q, s = w4o.quantize(f64(w), group)
    want = torch.from_numpy(w4o.values(q, s, group))
    assert bits_equal(got.dequantize(FP).cpu() + 0.0, want.to(FP) + 0.0)     # 12 bits: exact in float32
    assert torch.equal(got.dequantize(BF).cpu(), want.to(BF))
    # and the same buffers as the oracle's codes and scales packed, what pads them included
    q, s = torch.from_numpy(q).to(DEV, torch.uint8), torch.from_numpy(s).to(DEV, BF)
    same = B.moe_w4_pack(q[..., 0::2] | q[..., 1::2] << 4, s, group)
    assert torch.equal(got.codes, same.codes) and bits_equal(got.scales, same.scales)


def test_quantize_next_to_a_half_goes_by_the_exact_quotient():
    # float32 weights one step to either side of (k + 1/2) s
    s = np.float32(7.0 / 7)
    base = np.array([k + 0.5 for k in range(-7, 7)], np.float32) * s
    w = np.zeros((3, 32), np.float32)
    w[:, 0] = 7
    w[0, 1:15], w[1, 1:15], w[2, 1:15] = base, np.nextafter(base, np.float32(99)), np.nextafter(base, np.float32(-99))
    # other scales, exact in bf16: small, subnormal ones (bf16 2^-130) and large
    w = np.concatenate([w] + [w * np.float32(f) for f in (2.0 ** -20, 1.7109375, 2.0 ** -100, 2.0 ** 120)]
                       + [(w.astype(np.float64) * 2.0 ** -126).astype(np.float32)])
    got = B.moe_w4_quantize(torch.from_numpy(w).to(DEV), 32).dequantize(FP)
    q, sc = w4o.quantize(w, 32)
    assert np.array_equal(f64(got)[0], w4o.values(q, sc, 32))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,R,C", [(1, 1, 32), (2, 16, 128), (3, 31, 96), (1, 100, 672)])
def test_pack_holds_the_codes_and_scales(n, R, C, group):
    w, q, s = packed(n, R, C, group, seed=3)
    assert np.array_equal(f64(w.dequantize(FP)), w4o.values(q, s, group))
    RT, KT = -(-R // 16), -(-C // 128)
    NG = -(-KT * (128 // group) // 4) * 4
    assert w.codes.numel() == n * RT * KT * 1024 and w.scales.numel() == n * RT * 16 * NG
    # rows and columns past the matrix: every word of theirs is code 8, every scale 0
    nib = w.codes.cpu().numpy()
    nib = np.stack([nib & 15, nib >> 4], -1).reshape(n, RT, KT, 64, 4, 8)
    lane, word = np.meshgrid(np.arange(64), np.arange(4), indexing="ij")
    row, col = lane % 16, word * 32 + lane // 16 * 8
    for rt in range(RT):
        for kt in range(KT):
            out = (rt * 16 + row >= R) | (kt * 128 + col >= C)
            assert np.all(nib[:, rt, kt][:, out] == 8)
    sc = f64(w.scales).reshape(n, RT * 16, NG)
    assert not sc[:, R:].any() and not sc[:, :, -(-C // group):].any()


# ---- one matrix -------------------------------------------------------------

@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("T,C,R,group", [
    (1, 32, 1, 32), (1, 128, 16, 128), (2, 96, 17, 64), (15, 160, 31, 32), (16, 1024, 33, 128), (17, 416, 100, 64),
    (33, 1600, 48, 128), (64, 640, 129, 32), (96, 2048, 515, 128), (1, 6144, 700, 128), (5, 5024, 64, 32),
    (130, 288, 260, 64)])
def test_matvec(T, C, R, group, dt):
    print(f"[matvec] T={T} C={C} R={R} group={group} {dt}", flush=True)
    w, q, s = packed(1, R, C, group, seed=T + R)
    x = torch.randn(T, C, generator=gen(7), device=DEV).to(dt)
    y, err = product_bound(f64(x), q[0], s[0], group, dt)
    check(B.moe_w4_matvec(x, w), y, err, dt, "y")


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("code", [0, 7, 8, 15])
def test_matvec_of_one_code(code, dt):
    # whole numbers below 2^24 throughout: the product is exact in float32
    C, R = 1024, 48
    q = torch.full((1, R, C // 2), code * 17, dtype=torch.uint8, device=DEV)
    s = torch.full((1, R, C // 128), 0.5, dtype=BF, device=DEV)
    x = torch.randint(-8, 9, (3, C), generator=gen(5), device=DEV).to(dt)
    y = B.moe_w4_matvec(x, B.moe_w4_pack(q, s, 128))
    want = (0.5 * (code - 8) * x.double().sum(1, keepdim=True)).expand(3, R).to(dt)
    assert torch.equal(y, want)


@pytest.mark.parametrize("dt", [BF, FP])
def test_matvec_picks_every_weight(dt):
    # unit vectors: each column of W comes back as it is
    C, R, group = 288, 40, 32
    w, q, s = packed(1, R, C, group, seed=9)
    y = B.moe_w4_matvec(torch.eye(C, device=DEV).to(dt), w)
    assert torch.equal(y.t().contiguous(), w.dequantize(dt)[0])


def test_a_token_with_nan_or_infinity_leaves_the_others():
    w, _, _ = packed(1, 100, 640, 64, seed=2)
    x = torch.randn(20, 640, generator=gen(1), device=DEV).to(BF)
    clean = B.moe_w4_matvec(x, w)
    x[3, 5], x[17, 600], x[9, 1] = float("nan"), float("inf"), -float("inf")
    y = B.moe_w4_matvec(x, w)
    rows = [t for t in range(20) if t not in (3, 9, 17)]
    assert bits_equal(y[rows], clean[rows])
    assert y[[3, 9, 17]].isnan().all()


def test_matvec_rows_do_not_depend_on_the_batch():
    w, _, _ = packed(1, 200, 1024, 128, seed=4)
    x = torch.randn(37, 1024, generator=gen(2), device=DEV).to(BF)
    y = B.moe_w4_matvec(x, w)
    for t in (0, 15, 16, 36):
        assert bits_equal(B.moe_w4_matvec(x[t:t + 1].contiguous(), w), y[t:t + 1])


# ---- the experts ------------------------------------------------------------

def experts(E, d, F, group, seed=0):
    # scales such that the products stay near one
    out = []
    for i, (R, C) in enumerate(((F, d), (F, d), (d, F))):
        w, q, s = packed(E, R, C, group, seed=seed + i)
        k = float(2.0 ** np.floor(np.log2(0.4 / np.sqrt(C))))
        w.scales.mul_(k)                  # a power of two: exact
        out.append((w, q, s * k))
    return out


def ffn_bound(x, ws, e, group, dt):
    (_, qg, sg), (_, qu, su), (_, qd, sd) = ws
    g, eg = product_bound(x, qg[e], sg[e], group, dt)
    u, eu = product_bound(x, qu[e], su[e], group, dt)
    h = w4o.silu(g) * u
    # |silu'| <= 1.1; the exponential, the quotient and two products: 8 u; the planes: 2^-16 or 2^-24
    eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(w4o.silu(g)) * eu + (8 * U + (2.0 ** -16 if dt == BF else U)) * np.abs(h)
    y, ey = product_bound(h, qd[e], sd[e], group, dt)
    return y, ey + eh @ np.abs(w4o.values(qd[e], sd[e], group)).T


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("d,F,group,counts", [
    (64, 64, 32, [1]), (128, 64, 128, [3, 0, 1]), (192, 320, 64, [0, 0, 17, 0, 2, 1, 0]),
    (512, 256, 128, [16, 15, 33, 0, 1, 100]), (320, 192, 32, [1] * 70), (256, 128, 128, [0, 5] * 40 + [40])])
def test_grouped_ffn(d, F, group, counts, dt):
    print(f"[w4 ffn] d={d} F={F} group={group} E={len(counts)} {dt}", flush=True)
    E, N, T = len(counts), sum(counts), 50
    ws = experts(E, d, F, group, seed=d)
    x = torch.randn(T, d, generator=gen(3), device=DEV).to(dt)
    a_rows = torch.randint(0, T, (N,), generator=gen(4), device=DEV).to(torch.int32)
    off = offsets_of(counts)
    y = B.moe_w4_grouped_ffn(x, off, *(w[0] for w in ws), a_rows=a_rows)
    xs, lo = f64(x)[a_rows.cpu().numpy()], 0
    for e, c in enumerate(counts):
        if c:
            want, err = ffn_bound(xs[lo:lo + c], ws, e, group, dt)
            check(y[lo:lo + c], want, err, dt, f"expert {e}")
        lo += c
    # the same rows copied beforehand: the same bits
    flat = B.moe_w4_grouped_ffn(x[a_rows.long()].contiguous(), off, *(w[0] for w in ws))
    assert bits_equal(flat, y)


def test_rows_behind_the_last_expert_stay():
    counts = [3, 0, 20, 2]
    ws = [w[0] for w in experts(4, 128, 64, 64, seed=1)]
    x = torch.randn(40, 128, generator=gen(3), device=DEV).to(BF)
    y = torch.full((40, 128), 7.0, dtype=BF, device=DEV)
    B.moe_w4_grouped_ffn(x, offsets_of(counts), *ws, y_perm=y)
    assert (y[25:] == 7).all() and not (y[:25] == 7).all(1).any()
    again = B.moe_w4_grouped_ffn(x[:25].contiguous(), offsets_of(counts), *ws)
    assert bits_equal(again, y[:25])
    none = torch.full((40, 128), 7.0, dtype=BF, device=DEV)
    B.moe_w4_grouped_ffn(x, offsets_of([0, 0, 0, 0]), *ws, y_perm=none)
    assert (none == 7).all()


@pytest.mark.parametrize("raw", [[-5, 3, 2, 50, 1000, 7], [9, 9, 9, 9, 9, 9], [2 ** 31 - 1, 0, 0, 4, 5, 6],
                                 [-2 ** 31, -7, 12, 12, 3, 2 ** 31 - 1], [30, 20, 10, 5, 1, 0]])
def test_offsets_that_are_not_consistent_stay_inside(raw):
    # each bound is the running maximum clamped to the rows, as moe_grouped_ffn takes them
    E, rows = 5, 40
    ws = experts(E, 128, 64, 32, seed=2)
    x = torch.randn(rows, 128, generator=gen(3), device=DEV).to(BF)
    y = torch.full((rows + 16, 128), 7.0, dtype=BF, device=DEV)
    B.moe_w4_grouped_ffn(x, torch.tensor(raw, dtype=torch.int32, device=DEV), *(w[0] for w in ws), y_perm=y[:rows])
    b = np.clip(np.maximum.accumulate(raw), 0, rows)
    for e in range(E):
        if b[e + 1] > b[e]:
            want, err = ffn_bound(f64(x)[b[e]:b[e + 1]], ws, e, 32, BF)
            check(y[b[e]:b[e + 1]], want, err, BF, f"expert {e}")
    assert (y[:b[0]] == 7).all() and (y[b[-1]:] == 7).all()


def test_gather_map_is_clamped():
    ws = [w[0] for w in experts(2, 64, 64, 32, seed=2)]
    x = torch.randn(10, 64, generator=gen(3), device=DEV).to(BF)
    rows = torch.tensor([-1, 4, 10, 2 ** 31 - 1, -2 ** 31, 9], dtype=torch.int32, device=DEV)
    y = B.moe_w4_grouped_ffn(x, offsets_of([4, 2]), *ws, a_rows=rows)
    z = B.moe_w4_grouped_ffn(x, offsets_of([4, 2]), *ws, a_rows=rows.clamp(0, 9))
    assert bits_equal(y, z)


def test_more_experts_than_a_scan_step():
    E = 1024
    counts = [(e * 7) % 3 if e % 5 else 0 for e in range(E)]
    counts[-1] = 19
    ws = experts(E, 64, 64, 32, seed=6)
    x = torch.randn(sum(counts), 64, generator=gen(3), device=DEV).to(BF)
    y = B.moe_w4_grouped_ffn(x, offsets_of(counts), *(w[0] for w in ws))
    lo = 0
    for e, c in enumerate(counts):
        if c and e % 37 < 3 or e == E - 1:
            want, err = ffn_bound(f64(x[lo:lo + c]), ws, e, 32, BF)
            check(y[lo:lo + c], want, err, BF, f"expert {e}")
        lo += c


def test_matches_the_grouped_ffn_on_the_same_weights():
    # moe_grouped_ffn on the dequantised weights, which bf16 holds exactly here (codes times a
    # power of two); it rounds h to bf16, this does not: 2^-8 of |h| more, through W_d
    E, d, F, group, counts = 6, 256, 128, 64, [10, 0, 3, 90, 1, 20]
    ws = []
    for i, (R, C) in enumerate(((F, d), (F, d), (d, F))):
        ws.append(packed(E, R, C, group, seed=i, scale=2.0 ** -6))
    x = torch.randn(sum(counts), d, generator=gen(3), device=DEV).to(BF)
    off = offsets_of(counts)
    y = B.moe_w4_grouped_ffn(x, off, *(w[0] for w in ws))
    z = B.moe_grouped_ffn(x, off, *(w[0].dequantize(BF) for w in ws))
    lo = 0
    for e, c in enumerate(counts):
        if c:
            want, err = ffn_bound(f64(x[lo:lo + c]), ws, e, group, BF)
            W = [w4o.values(w[1][e], w[2][e], group) for w in ws]
            xs = f64(x[lo:lo + c])
            h = w4o.silu(xs @ W[0].T) * (xs @ W[1].T)
            tol = 2 * 2.0 ** -8 * np.abs(want) + 2 * err + 2.0 ** -8 * (np.abs(h) @ np.abs(W[2]).T)
            assert np.all(np.abs(f64(y[lo:lo + c]) - f64(z[lo:lo + c])) <= tol), e
        lo += c


def test_replays_reproduce_and_two_graphs_do_not_meet():
    counts = [4, 0, 18, 1]
    ws = [w[0] for w in experts(4, 256, 128, 128, seed=8)]
    a, b = (torch.randn(23, 256, generator=gen(s), device=DEV).to(FP) for s in (1, 2))
    one, two = (B.W4GroupedFfn(x, offsets_of(counts), *ws) for x in (a, b))
    mv = B.W4Matvec(a, B.moe_w4_quantize(torch.randn(70, 256, generator=gen(5), device=DEV), 32))
    want = [one().clone(), two().clone(), mv().clone()]
    torch.cuda.synchronize()
    g1 = replays_match([one, mv], [one.y_perm, mv.y], [want[0], want[2]])
    g2 = replays_match([two], [two.y_perm], [want[1]])
    side = torch.cuda.Stream()
    for _ in range(3):                    # both in flight at once
        for o in (one.y_perm, two.y_perm, mv.y):
            o.fill_(float("nan"))
        side.wait_stream(torch.cuda.current_stream())
        g1.replay()
        with torch.cuda.stream(side):
            g2.replay()
        torch.cuda.synchronize()
        assert bits_equal(one.y_perm, want[0]) and bits_equal(two.y_perm, want[1]) and bits_equal(mv.y, want[2])


def test_a_decode_step_runs_together():
    """previous block's combine, norm, gate and residual -> router -> 4-bit experts -> the next block's norm"""
    from oracle import block_norm_oracle as bno
    T, d, E, k, F, group = 6, 256, 16, 4, 128, 64
    g = gen(31)

    def rnd(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * std

    ws = experts(E, d, F, group, seed=40)
    x, w_router = rnd(T, d).to(BF), rnd(E, d, std=d ** -0.5).to(BF)
    y_perm = rnd(T * k, d).to(BF)
    slot_row = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k)
    topk_w = torch.softmax(rnd(T, k), 1)
    g1, g2, g3 = (1 + rnd(d, std=0.1) for _ in range(3))
    first = B.moe_block_norm(x, y_perm=y_perm, slot_row=slot_row, topk_w=topk_w, post_gain=g1, next_gain=g2)
    ids, w, _ = B.moe_route(first.h, w_router, k, want_logits=False)
    off, row_token, slots, _ = B.moe_permute(first.h, ids, E, copy_rows=False)
    rows = B.moe_w4_grouped_ffn(first.h, off, *(q[0] for q in ws), a_rows=row_token)
    last = B.moe_block_norm(first.out, y_perm=rows, slot_row=slots, topk_w=w, post_gain=g1, next_gain=g3)
    torch.cuda.synchronize()
    # in float64 from what each call was given
    H, ids, slots = f64(first.h), ids.cpu().numpy(), slots.cpu().numpy()
    want, size = np.zeros((2, T * k, d))
    for t in range(T):
        for j in range(k):
            want[slots[t, j]], size[slots[t, j]] = (v[0] for v in ffn_bound(H[t:t + 1], ws, ids[t, j], group, BF))
    assert np.all(np.abs(f64(rows) - want) <= 2.0 ** -8 * np.abs(want) + size)
    y, ysize = bno.combine(f64(rows), slots, f64(w))
    out, h, so, sh = bno.forward(f64(first.out), y, f64(g1), None, 0, "none", 1, 1, 1e-6, f64(g3), ysize)
    for got, o, s in ((last.out, out, so), (last.h, h, sh)):
        assert np.all(np.abs(f64(got) - o) <= 2.0 ** -8 * np.abs(o) + 160 * U * s)
