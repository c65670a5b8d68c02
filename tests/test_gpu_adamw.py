"""GPU parity of the AdamW operators against the plain reference.

Tolerances. The moments and the 8-bit codes have a pinned order of float32
roundings: they are compared bit for bit. A weight W' = W - lr (wd W + u) is
formed from those moments in float32: the direction u by two bias factors
(expm1 of a rounded float32 argument, rsqrt), three products, one fused
multiply-add and one division, each off by at most a few 2^-24 of itself (16 of
them at most together: expm1 and rsqrt 2 each, their arguments and roundings 4,
sqrt 1, the rest 5), then two fused multiply-adds and the rounding of lr. So
|W' - exact| <= 2^-24 (2 |W'| + 20 lr (|u| + wd |W|)), plus half a bf16 step
(2^-8 relative) where W is bf16.
"""
import math

import numpy as np
import pytest
import torch

import matrix_aware_sign_b200 as S
import oracle as O
import workloads as WL
from matrix_aware_sign_b200 import checkpoint as C
from oracle import adamw_oracle as A
from tests.gpu_util import dev, host, rel_fro

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
B1, B2, EPS, LR, WD = 0.9, 0.999, 1e-8, 1e-3, 0.1
U = 2.0 ** -24
# one entry, below / at / above a lane's eight and a block's 256, odd matrices, several blocks
SHAPES = [(1,), (2,), (7,), (8,), (9,), (255,), (256,), (257,), (3, 5), (17, 131), (1000,), (2, 3, 43), (64, 96), ()]


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy() if t.dtype == torch.float8_e4m3fn else t.cpu().numpy()


def f64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


class Reference:
    """The run of one tensor, from float32 inputs, in the reference's arithmetic."""

    def __init__(self, w, m, v, eight, index=0, seed=0, wd=WD, lr_scale=1.0, bf16=False, master=False):
        self.w, self.m, self.v, self.eight = w.copy(), m.copy(), v.copy(), eight
        self.index, self.seed, self.wd, self.ls, self.bf16, self.master = index, seed, wd, lr_scale, bf16, master
        if eight:
            self.cm, self.bm = A.encode(m)
            self.cr, self.br = A.encode(A.f32(np.sqrt(v)))

    def step(self, g, t, lr=LR, scale=None):
        """Moves the moments; returns (exact W', tolerance)."""
        if self.eight:
            self.m, r = A.decode(self.cm, self.bm), A.decode(self.cr, self.br)
            self.v = r * r
        self.m, self.v, r = A.moments(self.m, self.v, g, B1, B2, scale)
        u = A.direction(self.m, r, t, B1, B2, EPS)
        lr = lr * self.ls
        w = self.w - lr * (self.wd * self.w + u)
        tol = U * (2 * np.abs(w) + 20 * lr * (np.abs(u) + self.wd * np.abs(self.w)))
        if self.eight:
            rnd = A.rounding_bits(g.size, self.index, self.seed, t)
            self.cm, self.bm = A.encode(self.m, rnd)
            self.cr, self.br = A.encode(r, rnd)
        return w, tol

    def check(self, opt, i, w, tol):
        """Compares tensor i of opt, and takes over its weights (so that steps are compared one by one)."""
        stepped = opt.master[i] if self.master else opt.W[i]
        got = f64(stepped)
        t = tol + (2.0 ** -8 * np.abs(w) if self.bf16 and not self.master else 0.0)
        fine = np.isfinite(w)
        assert np.all(np.abs(got - w)[fine] <= t[fine]), (i, np.max((np.abs(got - w) / t)[fine]))
        assert np.array_equal(np.isfinite(got), fine)
        if self.master:
            assert torch.equal(opt.W[i], stepped.to(BF16))
        if self.eight:
            assert np.array_equal(bits(opt.m[i]).reshape(-1), self.cm)
            assert np.array_equal(bits(opt.v[i]).reshape(-1), self.cr)
            assert np.array_equal(opt.scales[i].cpu().numpy(), np.stack([self.bm, self.br], 1))
        else:
            assert np.array_equal(f64(opt.m[i]), self.m, equal_nan=True)
            assert np.array_equal(f64(opt.v[i]), self.v, equal_nan=True)
        self.w = got


def draw_tensor(rng, shape, sigma=1e-3):
    n = int(np.prod(shape, dtype=np.int64))
    size = sigma * np.exp(rng.standard_normal(n))
    g = rng.standard_normal(n) * size
    m = 0.3 * rng.standard_normal(n) * size
    v = size * size * rng.uniform(0.3, 1.3, n)
    w = 0.02 * rng.standard_normal(n)
    return tuple(A.f32(x) for x in (w, g, m, v))


def make(shapes, eight, wdt, gdt, master, seed=0, t=0, rng_seed=5, **kw):
    """(opt, G, references, gradients as the kernels see them)."""
    rng = np.random.default_rng(seed)
    W, G, M, V, sc, refs, gs = [], [], [], [], [], [], []
    for i, s in enumerate(shapes):
        w, g, m, v = draw_tensor(rng, s)
        wt = torch.from_numpy(w.astype(np.float32)).to(wdt).cuda().reshape(s)
        gt = torch.from_numpy(g.astype(np.float32)).to(gdt).cuda().reshape(s)
        ref = Reference(f64(wt), m, v, eight, i, rng_seed, bf16=wdt == BF16, master=master)
        if eight:
            M.append(torch.from_numpy(ref.cm).cuda().view(torch.float8_e4m3fn).reshape(s))
            V.append(torch.from_numpy(ref.cr).cuda().view(torch.float8_e4m3fn).reshape(s))
            sc.append(torch.from_numpy(np.stack([ref.bm, ref.br], 1)).cuda())
        else:
            M.append(torch.from_numpy(m.astype(np.float32)).cuda().reshape(s))
            V.append(torch.from_numpy(v.astype(np.float32)).cuda().reshape(s))
        W.append(wt)
        G.append(gt)
        refs.append(ref)
        gs.append(f64(gt))
    opt = S.AdamW(W, m=M, v=V, scales=sc if eight else None, master=True if master else None, weight_decay=WD,
                  seed=rng_seed, t=t, **kw)
    return opt, G, refs, gs


def step_refs(opt, refs, gs, t, **kw):
    for i, (r, g) in enumerate(zip(refs, gs)):
        r.check(opt, i, *r.step(g, t, **kw))


# ------------------------------------------------------------------ the step
@pytest.mark.parametrize("gdt", [F32, BF16])
@pytest.mark.parametrize("wdt,master", [(F32, False), (BF16, False), (BF16, True)])
@pytest.mark.parametrize("eight", [False, True])
def test_three_steps_of_every_shape(eight, wdt, master, gdt):
    opt, G, refs, gs = make(SHAPES, eight, wdt, gdt, master)
    for t in (1, 2, 3):
        S.adamw_step(opt, G, LR, B1, B2, EPS)
        assert opt.t == t
        step_refs(opt, refs, gs, t)


@pytest.mark.parametrize("eight", [False, True])
def test_float32_step_against_the_formula_in_64_bits(eight):
    """Without the pinned roundings: m' = b1 m + (1-b1) g has five roundings (both factors, both products, the sum), so
    it is within 3 U of the sum of its terms' magnitudes; v' (positive terms, one product more) within 5 U of itself."""
    opt, G, refs, gs = make([(4099,)], eight, F32, F32, False, t=9)
    r = refs[0]
    m, v = r.m, r.v
    if eight:
        m, v = A.decode(r.cm, r.bm), A.decode(r.cr, r.br) ** 2
    w, m64, v64 = A.step64(r.w, gs[0], m, v, 10, LR, B1, B2, EPS, WD)
    S.adamw_step(opt, G, LR, B1, B2, EPS)
    u = (r.w - w) / LR
    # the direction inherits m's error, at most 3 U (|b1 m| + |c1 g|), over a root within 3 U of itself
    root = np.sqrt(v64) / math.sqrt(1 - B2 ** 10) + EPS
    inherited = 3 * U * (B1 * np.abs(m) + (1 - B1) * np.abs(gs[0])) / (1 - B1 ** 10) / root + 3 * U * np.abs(u)
    assert np.all(np.abs(f64(opt.W[0]) - w) <= U * (2 * np.abs(w) + 20 * LR * (np.abs(u) + WD)) + LR * inherited)
    if not eight:
        assert np.all(np.abs(f64(opt.m[0]) - m64) <= 3 * U * (B1 * np.abs(m) + (1 - B1) * np.abs(gs[0])))
        assert np.all(np.abs(f64(opt.v[0]) - v64) <= 5 * U * v64)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("t", [0, 1, 999, 10 ** 6, 2 ** 33 + 5])
def test_late_steps(eight, t):
    """Bias corrections and the rounding's counter (step's low word) far into a run."""
    opt, G, refs, gs = make([(300,), (5, 7)], eight, F32, F32, False, t=t)
    S.adamw_step(opt, G, LR, B1, B2, EPS)
    step_refs(opt, refs, gs, t + 1)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("betas", [(0.0, 0.999), (0.9, 0.0), (0.95, 0.9999), (0.0, 0.0)])
def test_other_betas(eight, betas):
    opt, G, refs, gs = make([(513,)], eight, F32, F32, False, t=3)
    S.adamw_step(opt, G, LR, *betas, EPS)
    r, g = refs[0], gs[0]
    m, v = (A.decode(r.cm, r.bm), A.decode(r.cr, r.br) ** 2) if eight else (r.m, r.v)
    m, v, root = A.moments(m, v, g, *betas)
    u = A.direction(m, root, 4, *betas, EPS)
    w = r.w - LR * (WD * r.w + u)
    assert np.all(np.abs(f64(opt.W[0]) - w) <= U * (2 * np.abs(w) + 20 * LR * (np.abs(u) + WD * np.abs(r.w))))
    if eight:
        rnd = A.rounding_bits(g.size, 0, r.seed, 4)
        assert np.array_equal(bits(opt.m[0]), A.encode(m, rnd)[0]) and np.array_equal(bits(opt.v[0]), A.encode(root, rnd)[0])
    else:
        assert np.array_equal(f64(opt.m[0]), m) and np.array_equal(f64(opt.v[0]), v)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("wdt,gdt", [(F32, BF16), (BF16, F32)])
def test_column_ranges_and_odd_addresses(eight, wdt, gdt):
    """W and G as column ranges of wider matrices (aligned and not), moments at odd addresses: the rest of every buffer
    stays as it was."""
    rng = np.random.default_rng(8)
    cases = [((33, 64), 96, 0, 32, 0), ((33, 64), 96, 8, 16, 0), ((9, 37), 41, 3, 1, 3), ((5, 64), 65, 0, 1, 1), ((1, 700), 704, 3, 4, 0)]
    for rows_cols, ld, w_off, g_off, odd in cases:
        r, c = rows_cols
        w, g, m, v = draw_tensor(rng, (r, c))
        wide = lambda off: max(ld, off + c)  # noqa: E731
        wbuf = torch.full((r + 1, wide(w_off) + 8), 7.0, dtype=wdt, device="cuda")
        gbuf = torch.full((r + 1, wide(g_off) + 8), 9.0, dtype=gdt, device="cuda")
        W, G = wbuf[:r, w_off:w_off + c], gbuf[:r, g_off:g_off + c]
        W.copy_(torch.from_numpy(w.astype(np.float32)).reshape(r, c))
        G.copy_(torch.from_numpy(g.astype(np.float32)).reshape(r, c))
        n, wref, gref = r * c, f64(W.contiguous()), f64(G.contiguous())
        ref = Reference(wref, m, v, eight, 0, 2, bf16=wdt == BF16)
        kind = torch.float8_e4m3fn if eight else F32
        mbuf, vbuf = (torch.full((n + odd + 5,), 3.0, dtype=F32, device="cuda").to(kind) for _ in range(2))
        M, V = (b[odd:odd + n] for b in (mbuf, vbuf))
        if eight:
            M.view(torch.uint8).copy_(torch.from_numpy(ref.cm))
            V.view(torch.uint8).copy_(torch.from_numpy(ref.cr))
        else:
            M.copy_(torch.from_numpy(m))
            V.copy_(torch.from_numpy(v))
        sbuf = torch.full((-(-n // 256) + 2, 2), 77, dtype=torch.uint8, device="cuda")
        sc = sbuf[1:-1]
        sc.copy_(torch.from_numpy(np.stack([ref.bm, ref.br], 1)) if eight else sc)
        opt = S.AdamW([W], m=[M.view(r, c)], v=[V.view(r, c)], scales=[sc] if eight else None, weight_decay=WD, seed=2)
        S.adamw_step(opt, [G], LR, B1, B2, EPS)
        ref.check(opt, 0, *ref.step(gref, 1))
        keep = wbuf.clone()
        keep[:r, w_off:w_off + c] = 7.0
        assert torch.all(keep == 7.0) and torch.all(gbuf[r:] == 9.0)
        three = torch.full((1,), 3.0, device="cuda").to(kind).float()
        for b in (mbuf, vbuf):
            assert torch.all(b[:odd].float() == three) and torch.all(b[odd + n:].float() == three)
        assert torch.all(sbuf[0] == 77) and torch.all(sbuf[-1] == 77)


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("w_off,g_off", [(1, 0), (0, 1), (3, 5)])
def test_long_tensors_off_their_vector_addresses(w_off, g_off, eight, master):
    """Several tiles each: a flat tensor, rows of odd length, rows of a whole number of vectors at an odd offset, a single
    column; W, G or both off the addresses that vectors need. Entries beside the tensors stay as they were."""
    rng = np.random.default_rng(17)
    wdt, gdt = (BF16, F32) if master else (F32, BF16)
    W, G, refs, gs, bufs = [], [], [], [], []
    for i, (r, c, ld) in enumerate([(1, 5003, 5010), (37, 133, 140), (61, 64, 80), (1500, 1, 6), (3, 1100, 1104)]):
        w, g, _, _ = draw_tensor(rng, (r, c))
        wb = torch.full((r, ld + 3), 7.0, dtype=wdt, device="cuda")
        gb = torch.full((r, ld + 5), 9.0, dtype=gdt, device="cuda")
        W.append(wb[:, w_off:w_off + c])
        G.append(gb[:, g_off:g_off + c])
        W[i].copy_(torch.from_numpy(w.astype(np.float32)).reshape(r, c))
        G[i].copy_(torch.from_numpy(g.astype(np.float32)).reshape(r, c))
        bufs.append((wb, c))
        refs.append(Reference(f64(W[i].contiguous()), np.zeros(r * c), np.zeros(r * c), eight, i, 4, bf16=master, master=master))
        gs.append(f64(G[i].contiguous()))
    opt = S.AdamW(W, bits=8 if eight else 32, master=master, weight_decay=WD, seed=4)
    plan = S.AdamWPlan(opt, G, B1, B2, EPS)
    for t in (1, 2):
        plan.run(LR)
        step_refs(opt, refs, gs, t)
    for (wb, c) in bufs:
        assert torch.all(wb[:, :w_off] == 7.0) and torch.all(wb[:, w_off + c:] == 7.0)


@pytest.mark.parametrize("eps", [1e-8, 1e-15, 1e-30])
@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.0, 0.999), (0.9, 0.0)])
@pytest.mark.parametrize("size", [1e-3, 1e-17, 1e-19])
def test_small_eps_and_small_gradients(size, betas, eps):
    """Second moments down to float32's subnormal range beside an eps of any size, 8-bit moments, whole tiles."""
    n = 2048
    g = A.f32(np.random.default_rng(3).standard_normal(n) * size * np.exp2(np.repeat([0, -20, -3, 0], 512)))
    opt = S.AdamW([torch.ones(n, device="cuda")], bits=8, seed=2)
    S.adamw_step(opt, [dev(g.astype(np.float32))], LR, *betas, eps)
    m, v, r = A.moments(np.zeros(n), np.zeros(n), g, *betas)
    rnd = A.rounding_bits(n, 0, 2, 1)
    for x, t, col in ((m, opt.m[0], 0), (r, opt.v[0], 1)):
        c, b = A.encode(x, rnd)
        assert np.array_equal(bits(t), c) and np.array_equal(opt.scales[0].cpu().numpy()[:, col], b)
    u = A.direction(m, r, 1, *betas, eps)
    w = 1.0 - LR * u
    assert np.all(np.abs(f64(opt.W[0]) - w) <= U * (2 * np.abs(w) + 20 * LR * np.abs(u)))


@pytest.mark.parametrize("b2", [0.999, 0.999999])
@pytest.mark.parametrize("eps", [1e-12, 1e-10, 1e-9, 1e-8])
def test_small_roots_beside_eps(eps, b2):
    """Gradients near 2^-59 in the tiles of ordinary ones: their second moments are subnormal, and the bias correction
    (32 and 1000 times the root in the first step) lifts the root towards eps. W starts at 0, so the step is all it holds."""
    n = 2048
    rng = np.random.default_rng(4)
    g = rng.standard_normal(n) * 1e-3
    g[::7] = np.exp2(rng.uniform(-62, -57, g[::7].size)) * rng.choice([-1.0, 1.0], g[::7].size)
    g = A.f32(g)
    opt = S.AdamW([torch.zeros(n, device="cuda")], bits=8, seed=2)
    S.adamw_step(opt, [dev(g.astype(np.float32))], LR, B1, b2, eps)
    m, v, r = A.moments(np.zeros(n), np.zeros(n), g, B1, b2)
    assert np.any((v > 0) & (v < 2.0 ** -126))
    u = A.direction(m, r, 1, B1, b2, eps)
    w = -LR * u
    assert np.all(np.abs(f64(opt.W[0]) - w) <= U * (2 * np.abs(w) + 20 * LR * np.abs(u)))


@pytest.mark.parametrize("eight", [False, True])
def test_two_weights_in_one_matrix(eight):
    """Column halves of one matrix as two weights of a call."""
    rng = np.random.default_rng(4)
    both = dev(rng.standard_normal((24, 80)).astype(np.float32))
    W = [both[:, :32], both[:, 32:]]
    before = [f64(w.contiguous()) for w in W]
    G = [dev(rng.standard_normal(w.shape).astype(np.float32)) for w in W]
    opt = S.AdamW(W, bits=8 if eight else 32, weight_decay=WD, seed=5)
    S.adamw_step(opt, G, LR, B1, B2, EPS)
    for i in (0, 1):
        ref = Reference(before[i], 0 * before[i], 0 * before[i], eight, i, 5)
        ref.check(opt, i, *ref.step(f64(G[i]), 1))


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("eight", [False, True])
def test_many_tensors_mixed_types_and_empty_ones(eight, planned):
    """More tensors than a launch holds, of every combination of types, empty ones and a long one among them: each tensor
    keeps its own place in the lists (the rounding's key), its own decay and learning-rate factor. Planned: the tables in
    memory, some hundred tensors each."""
    rng = np.random.default_rng(6)
    W, G, M, refs, gs, wd, ls = [], [], [], [], [], [], []
    for i in range(700):
        n = 0 if i % 50 == 7 else 40_000 + i if i in (100, 401) else int(rng.integers(1, 600))
        wdt, gdt = (F32, BF16)[int(rng.integers(2))], (F32, BF16)[int(rng.integers(2))]
        w, g, m, v = draw_tensor(rng, (n,))
        W.append(torch.from_numpy(w.astype(np.float32)).to(wdt).cuda())
        G.append(torch.from_numpy(g.astype(np.float32)).to(gdt).cuda())
        M.append(W[-1].float() if wdt == BF16 and rng.random() < 0.5 and n else None)
        wd.append(float(np.float32(rng.uniform(0, 0.2))))
        ls.append(float(np.float32(rng.uniform(0, 2))))
        refs.append(Reference(f64(W[-1]), np.zeros(n), np.zeros(n), eight, i, 9, wd[-1], ls[-1], wdt == BF16, M[-1] is not None))
        gs.append(f64(G[-1]))
    opt = S.AdamW(W, bits=8 if eight else 32, master=M, weight_decay=wd, lr_scale=ls, seed=9, device_step=True)
    plan = S.AdamWPlan(opt, G, B1, B2, EPS) if planned else None
    for t in (1, 2):
        plan.run(LR) if planned else S.adamw_step(opt, G, LR, B1, B2, EPS)
        assert opt.d_t.tolist() == [t, 0]
        for i, (r, g) in enumerate(zip(refs, gs)):
            if g.size:
                r.check(opt, i, *r.step(g, t))


def test_a_plan_of_two_thousand_tensors():
    """One type, lengths from one entry to several tiles: the guide's parts hold more than 32 tensors and less than one."""
    rng = np.random.default_rng(9)
    ns = [int(x) for x in np.exp(rng.uniform(0, 5, 1000))] + [70_000] + [int(x) for x in np.exp(rng.uniform(0, 9, 1000))]
    W = [torch.randn(n, device="cuda") for n in ns]
    G = [torch.randn(n, device="cuda") for n in ns]
    for b in (32, 8):
        one = S.AdamW([w.clone() for w in W], bits=b, weight_decay=WD, seed=3)
        two = S.AdamW([w.clone() for w in W], bits=b, weight_decay=WD, seed=3)
        S.AdamWPlan(one, G, B1, B2, EPS).run(LR)
        S.adamw_step(two, G, LR, B1, B2, EPS)
        for k in ("W", "m", "v", "scales"):
            for x, y in zip(getattr(one, k) or [], getattr(two, k) or []):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    for i in (0, 999, 1000, 2000):  # and some of them against the reference
        g, z = f64(G[i]), np.zeros(ns[i])
        m, v, r = A.moments(z, z, g, B1, B2)
        c, byte = A.encode(m, A.rounding_bits(ns[i], i, 3, 1))
        assert np.array_equal(bits(one.m[i]), c) and np.array_equal(one.scales[i][:, 0].cpu().numpy(), byte)


def test_only_empty_tensors():
    w = [torch.zeros(0, device="cuda"), torch.zeros(0, 5, device="cuda")]
    opt = S.AdamW(w, device_step=True)
    S.adamw_step(opt, [torch.zeros_like(x) for x in w], LR)
    assert opt.t == 1
    host_opt = S.AdamW(w)
    S.adamw_step(host_opt, [torch.zeros_like(x) for x in w], LR)
    assert host_opt.t == 1


@pytest.mark.parametrize("eight", [False, True])
def test_zero_gradients_and_moments_only_decay(eight):
    w = torch.randn(1000, device="cuda")
    opt = S.AdamW([w.clone()], bits=8 if eight else 32, weight_decay=WD)
    S.adamw_step(opt, [torch.zeros(1000, device="cuda")], LR)
    exact = f64(w) * (1 - LR * WD)
    assert np.all(np.abs(f64(opt.W[0]) - exact) <= 3 * U * np.abs(exact))
    assert not bits(opt.m[0]).any() and not bits(opt.v[0]).any()
    assert eight is False or not opt.scales[0].any()


@pytest.mark.parametrize("eight", [False, True])
def test_extreme_gradients(eight):
    """Blocks of very large, very small and mixed gradients; moments that underflow in a block."""
    n = 6 * 256
    g = np.random.default_rng(1).standard_normal(n)
    g[:256] *= 1e-30
    g[256:512] *= 1e18
    g[512:768] *= np.exp2(np.linspace(-60, 0, 256))
    g[768] = 1e15
    g[1024:1280] = 0
    g[1030] = 1e-38
    g = A.f32(g)
    opt = S.AdamW([torch.zeros(n, device="cuda")], bits=8 if eight else 32, seed=1)
    ref = Reference(np.zeros(n), np.zeros(n), np.zeros(n), eight, 0, 1, wd=0.0)
    G = [dev(g.astype(np.float32))]
    for t in (1, 2):
        S.adamw_step(opt, G, LR, B1, B2, EPS)
        w, tol = ref.step(g, t)
        # float32's own spacing near zero (products and quotients below 2^-126) beside the relative errors
        ref.check(opt, 0, w, tol + 2.0 ** -140)


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("size", [2.0 ** -44, 1e-9, 1e-3, 1.0, 7e4, 1e7, 1e15])
def test_small_codes_beside_large_ones(size, odd):
    """Blocks whose moments span all that a block can hold (2^16) and more, codes of every size: of 4 steps, the later ones
    without gradients but for the blocks' largest. Sizes on either side of what the form for whole tiles takes."""
    n = 8 * 256 + 77
    rng = np.random.default_rng(6)
    g = A.f32(size * rng.choice([-1.0, 1.0], n) * np.exp2(rng.uniform(-26, 0, n)))
    g[::256] = A.f32(size)
    only = np.where(np.arange(n) % 256 == 0, g, 0.0)
    buf = [torch.zeros(n + 1, dtype=torch.uint8, device="cuda") for _ in range(2)]
    m, v = (b[odd:odd + n].view(torch.float8_e4m3fn) for b in buf)
    opt = S.AdamW([torch.zeros(n, device="cuda")], m=[m], v=[v], seed=8,
                  scales=[torch.zeros(-(-n // 256), 2, dtype=torch.uint8, device="cuda")])
    ref = Reference(np.zeros(n), np.zeros(n), np.zeros(n), True, 0, 8, wd=0.0)
    for t in range(1, 5):
        S.adamw_step(opt, [dev((g if t == 1 else only).astype(np.float32))], LR, B1, B2, EPS)
        w, tol = ref.step(g if t == 1 else only, t)
        ref.check(opt, 0, w, tol + 2.0 ** -140)
        small = (ref.cr & 127) < 8
        assert small.any() and (ref.cm[small] != 0).any()


@pytest.mark.parametrize("small", [1.0, 2.0 ** -20, 2.0 ** -45, 2.0 ** -60, 2.0 ** -75, 1e-30, 0.0])
@pytest.mark.parametrize("large", [2e4, 2e5, 1e9, 3e11, 1e13, 2.0 ** 62])
def test_large_gradients_beside_small_ones(large, small):
    """Tiles with moments beyond what a single factor brings to the codes' patterns, beside moments of any smaller size: in
    the same block, and in the tile's other block. W starts at 0, so the step is all it holds."""
    n = 4 * 512
    rng = np.random.default_rng(7)
    g = rng.standard_normal(n) * large
    g[0:256:3] = rng.standard_normal(g[0:256:3].size) * small     # the same block
    g[512 + 256:1024] = rng.standard_normal(256) * small          # the tile's other block
    g = A.f32(g)
    opt = S.AdamW([torch.zeros(n, device="cuda")], bits=8, seed=2)
    ref = Reference(np.zeros(n), np.zeros(n), np.zeros(n), True, 0, 2, wd=0.0)
    for t in (1, 2, 3):
        S.adamw_step(opt, [dev(g.astype(np.float32))], LR, B1, B2, EPS)
        w, tol = ref.step(g, t)
        ref.check(opt, 0, w, tol + 2.0 ** -140)


@pytest.mark.parametrize("odd", [0, 1])
def test_moments_too_small_to_be_held_have_no_signs(odd):
    """A block of first moments below 2^-119 is held as code 0 (not 0x80) for negative ones, too, at any address."""
    n = 4 * 256 + 5
    g = np.zeros(n)
    g[[3, 300, n - 1]] = -1e-38
    g[700:] = 0.01
    g[701] = -1e-30  # and one whose block is held: code 0x80, its sign
    g = A.f32(g)
    buf = [torch.zeros(n + 1, dtype=torch.uint8, device="cuda") for _ in range(2)]
    m, v = (b[odd:odd + n].view(torch.float8_e4m3fn) for b in buf)
    opt = S.AdamW([torch.zeros(n, device="cuda")], m=[m], v=[v], seed=1,
                  scales=[torch.zeros(-(-n // 256), 2, dtype=torch.uint8, device="cuda")])
    ref = Reference(np.zeros(n), np.zeros(n), np.zeros(n), True, 0, 1, wd=0.0)
    S.adamw_step(opt, [dev(g.astype(np.float32))], LR, B1, B2, EPS)
    w, tol = ref.step(g, 1)
    assert not ref.cm[:512].any() and ref.cm[701] == 0x80
    ref.check(opt, 0, w, tol + 2.0 ** -140)


@pytest.mark.parametrize("eight", [False, True])
def test_non_finite_gradients_stay_where_they_are(eight):
    """A NaN or an infinity spoils its own weight and moments (8 bits: the moments of its block) and nothing else."""
    n = 4 * 256 + 11
    rng = np.random.default_rng(2)
    w, g, _, _ = draw_tensor(rng, (n,))
    g[300], g[700] = math.nan, math.inf
    opt = S.AdamW([dev(w.astype(np.float32))], bits=8 if eight else 32, weight_decay=WD, seed=3)
    S.adamw_step(opt, [dev(g.astype(np.float32))], LR, B1, B2, EPS)
    bad = np.zeros(n, bool)
    bad[[300, 700]] = True
    got = f64(opt.W[0])
    assert np.array_equal(np.isfinite(got), ~bad)
    g0 = np.where(bad, 0, g)
    m, v, r = A.moments(np.zeros(n), np.zeros(n), g0, B1, B2)
    if eight:
        rnd = A.rounding_bits(n, 0, 3, 1)
        spoilt = (np.arange(n) // 256 == 1) | (np.arange(n) // 256 == 2)
        assert opt.scales[0].cpu().numpy()[1:3].tolist() == [[255, 255]] * 2
        for x, t in ((m, opt.m[0]), (r, opt.v[0])):
            c, _ = A.encode(x, rnd)
            assert np.array_equal(bits(t)[~spoilt], c[~spoilt]) and not bits(t)[spoilt].any()
    else:
        assert np.array_equal(f64(opt.m[0])[~bad], m[~bad]) and np.array_equal(f64(opt.v[0])[~bad], v[~bad])


# ------------------------------------------------------------------ device-side arguments
@pytest.mark.parametrize("eight", [False, True])
def test_gradient_factor_and_learning_rate_from_the_device(eight):
    opt, G, refs, gs = make([(600,), (3, 70)], eight, BF16, BF16, True, device_step=True)
    coef, lr = torch.tensor([0.37], device="cuda"), torch.tensor([0.02], device="cuda")
    S.adamw_step(opt, G, lr, B1, B2, EPS, grad_scale=coef)
    lr32 = float(lr.double())
    step_refs(opt, refs, gs, 1, lr=lr32, scale=0.37)
    plan = S.AdamWPlan(opt, G, B1, B2, EPS, lr=lr, grad_scale=coef)
    lr.fill_(0.005)
    coef.fill_(2.5)
    plan.run()
    step_refs(opt, refs, gs, 2, lr=float(lr.double()), scale=2.5)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("device_step", [False, True])
def test_a_skipped_step_changes_nothing(eight, device_step):
    opt, G, refs, gs = make([(600,), (3, 70)], eight, BF16, F32, True, device_step=device_step)
    everything = lambda: [x.clone() for k in (opt.W, opt.m, opt.v, opt.master, opt.scales or []) for x in k]  # noqa: E731
    before = everything()
    skip = torch.ones(1, dtype=torch.int32, device="cuda")
    S.adamw_step(opt, G, LR, B1, B2, EPS, skip_if=skip)
    for a, b in zip(before, everything()):
        assert np.array_equal(bits(a), bits(b)) if a.dtype != BF16 else torch.equal(a, b)
    assert opt.t == (0 if device_step else 1)
    skip.zero_()
    S.adamw_step(opt, G, LR, B1, B2, EPS, skip_if=skip)
    step_refs(opt, refs, gs, 1 if device_step else 2)


@pytest.mark.parametrize("eight", [False, True])
def test_captured_steps_count_on(eight):
    """A step captured once and replayed equals the same number of eager steps, bit for bit; a plan's first run may be
    the captured one."""
    a = make([(700,), (33, 40), (1,)], eight, BF16, BF16, True, device_step=True)
    b = make([(700,), (33, 40), (1,)], eight, BF16, BF16, True, device_step=True)
    lr = torch.tensor([LR], device="cuda")
    plan = S.AdamWPlan(a[0], a[1], B1, B2, EPS, lr=lr)
    norm = S.GradNorm(a[1], 0.01)
    clipped = S.AdamWPlan(a[0], a[1], B1, B2, EPS, lr=lr, grad_scale=norm.coef, skip_if=norm.skip)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
        norm.run()
        clipped.run()
    out, skip = torch.zeros(2, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(3):
        graph.replay()
        S.adamw_step(b[0], b[1], lr, B1, B2, EPS)
        ws = S.smuon_grad_norm(b[1], 0.01, out, skip)
        S.adamw_step(b[0], b[1], lr, B1, B2, EPS, grad_scale=out[1:], skip_if=skip)
        torch.cuda.synchronize()
        del ws
    assert a[0].t == b[0].t == 6
    for k in ("W", "m", "v", "master", "scales"):
        for x, y in zip(getattr(a[0], k) or [], getattr(b[0], k) or []):
            assert torch.equal(x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x,
                               y.view(torch.uint8) if y.dtype == torch.float8_e4m3fn else y)
    assert torch.equal(norm.out, out)


@pytest.mark.parametrize("eight", [False, True])
def test_a_captured_step_with_copies_and_a_fork(eight):
    """One graph: the gradients copied in, the norm, then the step on a second stream that joins before the conversion,
    copies on either side of each. Replayed with new gradients it equals the eager calls; parameters may require gradients."""
    rng = np.random.default_rng(11)
    shapes = [(3000,), (40, 64), (7,)] + [(65,)] * 20
    w0 = [dev((0.02 * rng.standard_normal(s)).astype(np.float32)) for s in shapes]
    src = [torch.zeros(s, device="cuda") for s in shapes]

    def build():
        W = [torch.nn.Parameter(w.clone()) for w in w0]
        G = [torch.zeros_like(w) for w in w0]
        opt = S.AdamW(W, bits=8 if eight else 32, weight_decay=WD, seed=3, device_step=True)
        other = S.AdamW(W, bits=32 if eight else 8, device_step=True)
        norm = S.GradNorm(G, 0.5)
        plan = S.AdamWPlan(opt, G, B1, B2, EPS, grad_scale=norm.coef, skip_if=norm.skip)
        return W, G, opt, other, norm, plan, torch.zeros(shapes[0], device="cuda")

    def body(W, G, opt, other, norm, plan, out, side):
        for g, s in zip(G, src):
            g.copy_(s)
        norm.run()
        norm.skip.add_(0)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            plan.run(LR)
        torch.cuda.current_stream().wait_stream(side)
        S.adamw_convert(opt, other)
        out.copy_(W[0].detach())

    a, b = build(), build()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body(*a, side)
    for step in range(3):
        for s in src:
            s.normal_(std=0.1)
        if step == 1:
            src[1][3, 3] = math.inf
        graph.replay()
        body(*b, side)
        torch.cuda.synchronize()
        assert a[2].t == b[2].t == a[3].t == b[3].t == (1, 1, 2)[step]
        assert torch.equal(a[6], b[6]) and torch.equal(a[4].out[1:], b[4].out[1:])
        for x, y in zip(a[2:4], b[2:4]):
            for k in ("W", "m", "v", "scales"):
                for p, q in zip(getattr(x, k) or [], getattr(y, k) or []):
                    assert torch.equal(p.detach().view(torch.uint8), q.detach().view(torch.uint8))


def test_steps_on_another_stream():
    opt, G, refs, gs = make([(70000,), (33, 40)], True, F32, F32, False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        S.adamw_step(opt, G, LR, B1, B2, EPS)
    S.adamw_step(opt, G, LR, B1, B2, EPS, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for i, (r, g) in enumerate(zip(refs, gs)):
        w, tol = r.step(g, 1)
        r.w = w
        w2, tol2 = r.step(g, 2)
        r.check(opt, i, w2, tol + tol2 + U * np.abs(w2))


def test_a_plan_runs_on_another_stream_at_once():
    """A plan's table is uploaded on the stream that was current at its creation; the first run elsewhere waits for it
    (here behind a queue of copies), and so does the norm's."""
    shapes = [(300 + i,) for i in range(40)]
    a, b = (make(shapes, True, F32, F32, False) for _ in range(2))
    big = torch.randn(1 << 27, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        big.mul_(1.0)
    plan, norm = S.AdamWPlan(a[0], a[1], B1, B2, EPS), S.GradNorm(a[1], 1.0)
    plan.run(LR, stream=side)
    norm.run(stream=side)
    with torch.cuda.stream(side):
        plan.run(LR)
        norm.run()
    for _ in range(2):
        S.adamw_step(b[0], b[1], LR, B1, B2, EPS)
    torch.cuda.synchronize()
    want, _ = A.grad_norm(b[3], 1.0)
    assert abs(float(norm.norm) - want) <= 6 * U * want
    for k in ("W", "scales"):
        assert all(torch.equal(x, y) for x, y in zip(getattr(a[0], k), getattr(b[0], k)))
    for k in ("m", "v"):
        assert all(np.array_equal(bits(x), bits(y)) for x, y in zip(getattr(a[0], k), getattr(b[0], k)))


def test_a_plan_made_on_a_side_stream_runs_on_the_default_one():
    a, b = (make([(300 + i,) for i in range(40)], False, F32, F32, False) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    big = torch.randn(1 << 27, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            big.mul_(1.0)
        plan, norm = S.AdamWPlan(a[0], a[1], B1, B2, EPS), S.GradNorm(a[1], 1.0)
    plan.run(LR)
    norm.run()
    S.adamw_step(b[0], b[1], LR, B1, B2, EPS)
    torch.cuda.synchronize()
    for k in ("W", "m", "v"):
        assert all(torch.equal(x, y) for x, y in zip(getattr(a[0], k), getattr(b[0], k)))
    assert abs(float(norm.norm) - A.grad_norm(a[3], 1.0)[0]) <= 6 * U * float(norm.norm)


def test_a_plan_is_complete_when_it_is_made():
    """A plan made behind a queue of work: its table has arrived when the constructor returns (checked before anything
    runs on it), so a capture begun by hand, which waits for nothing, may be replayed at once."""
    shapes = [(300 + i,) for i in range(40)]
    a, b = (make(shapes, True, F32, F32, False, device_step=True) for _ in range(2))
    big = torch.randn(1 << 27, device="cuda")
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            big.mul_(1.0)
        plan = S.AdamWPlan(a[0], a[1], B1, B2, EPS)
        assert side.query()
        for _ in range(20):
            big.mul_(1.0)
        norm = S.GradNorm(a[1], 1.0)
        assert side.query()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(other):
        graph.capture_begin()
        plan.run(LR)
        norm.run()
        graph.capture_end()
        graph.replay()
    S.adamw_step(b[0], b[1], LR, B1, B2, EPS)
    torch.cuda.synchronize()
    for k in ("W", "m", "v", "scales"):
        for x, y in zip(getattr(a[0], k), getattr(b[0], k)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    want, _ = A.grad_norm(a[3], 1.0)
    assert abs(float(norm.norm) - want) <= 6 * U * want


def test_events_order_what_a_kernel_reads():
    """A stream that waits for another one's event between two of these kernels (the first of which lets the next begin
    early): the second reads what the other stream wrote before the event."""
    n = 1 << 20
    g, ones = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    big = torch.randn(1 << 27, device="cuda")
    first, norm = S.GradNorm([ones], 1.0), S.GradNorm([g], 1.0)
    opt = S.AdamW([torch.zeros(n, device="cuda")])
    step = S.AdamWPlan(opt, [g], B1, 0.0, EPS)
    side = torch.cuda.Stream()
    for i in range(1, 9):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(10):
                big.mul_(1.0)
            g.fill_(float(i))
            ready = torch.cuda.Event()
            ready.record()
        first.run()
        torch.cuda.current_stream().wait_event(ready)
        norm.run()
        step.run(0.0)
        torch.cuda.synchronize()
        assert float(norm.norm) == i * 1024.0 and float(opt.v[0][n - 1]) == float(i * i)


@pytest.mark.parametrize("eight", [False, True])
def test_one_gradient_for_two_weights(eight):
    opt, G, refs, gs = make([(700,), (700,), (9, 40)], eight, F32, BF16, False)
    G[1], gs[1] = G[0], gs[0]
    S.adamw_step(opt, G, LR, B1, B2, EPS)
    step_refs(opt, refs, gs, 1)


def test_plans_are_prepared_before_a_capture():
    w, g = [torch.zeros(8, device="cuda")], [torch.ones(8, device="cuda")]
    opt = S.AdamW(w, device_step=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="capture"):
            S.AdamWPlan(opt, g)
        S.adamw_step(opt, g, LR)
    graph.replay()
    graph.replay()
    assert opt.t == 2


def test_two_graphs_with_a_plan_each():
    """Two captured steps on two states, replayed at the same time on two streams: plans share nothing."""
    sets = [make([(50_001,), (130, 64)] + [(33,)] * 20, True, BF16, F32, True, seed=i, device_step=True) for i in (0, 1)]
    twins = [make([(50_001,), (130, 64)] + [(33,)] * 20, True, BF16, F32, True, seed=i, device_step=True) for i in (0, 1)]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for opt, G, _, _ in sets:
        norm = S.GradNorm(G, 0.5)
        plan = S.AdamWPlan(opt, G, B1, B2, EPS, grad_scale=norm.coef, skip_if=norm.skip)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            norm.run()
            plan.run(LR)
        graphs.append((g, norm, plan))
    torch.cuda.synchronize()
    for _ in range(4):
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (opt, _, _, _), (other, G, _, _) in zip(sets, twins):
        out, skip = torch.zeros(2, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        for _ in range(4):
            keep = S.smuon_grad_norm(G, 0.5, out, skip)
            S.adamw_step(other, G, LR, B1, B2, EPS, grad_scale=out[1:], skip_if=skip)
        torch.cuda.synchronize()
        del keep
        assert opt.t == other.t == 4
        for k in ("W", "m", "v", "master", "scales"):
            for x, y in zip(getattr(opt, k), getattr(other, k)):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("eight", [False, True])
def test_offsets_beyond_32_bits(eight):
    """More than 2^31 entries in one tensor: its start, the 2^31 border and its end against the reference, and the norm."""
    rows, cols = 2, (1 << 30) + 777
    n = rows * cols
    if torch.cuda.mem_get_info()[0] < (14 if eight else 27) * n // 2 + (2 << 30):
        pytest.skip("needs more free memory")
    W = torch.full((rows, cols), 0.5, dtype=BF16, device="cuda")
    G = torch.full((rows, cols), 2.0 ** -9, dtype=BF16, device="cuda")
    flat_w, flat_g = W.view(-1), G.view(-1)
    places = [0, (1 << 31) - 512, (1 << 31), (n // 256 - 1) * 256]
    rng = np.random.default_rng(1)
    for p in places:
        size = min(512, n - p)
        flat_g[p:p + size] = dev((rng.standard_normal(size) * 1e-2).astype(np.float32)).to(BF16)
    opt = S.AdamW([W], bits=8 if eight else 32, weight_decay=WD, seed=6)
    S.adamw_step(opt, [G], LR, B1, B2, EPS)
    for p in places:
        size = min(512, n - p)
        g, z = f64(flat_g[p:p + size]), np.zeros(size)
        m, v, r = A.moments(z, z, g, B1, B2)
        w = 0.5 - LR * (WD * 0.5 + A.direction(m, r, 1, B1, B2, EPS))
        assert np.all(np.abs(f64(flat_w[p:p + size]) - w) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(w))
        sl = slice(p, p + size)
        if eight:
            rnd = A.rounding_bits(size, 0, 6, 1, first=p)
            for x, t, col in ((m, opt.m[0], 0), (r, opt.v[0], 1)):
                c, b = A.encode(x, rnd)
                assert np.array_equal(bits(t.view(-1)[sl]), c)
                assert np.array_equal(opt.scales[0][p // 256:p // 256 + b.size, col].cpu().numpy(), b)
        else:
            assert np.array_equal(f64(opt.m[0].view(-1)[sl]), m) and np.array_equal(f64(opt.v[0].view(-1)[sl]), v)
    norm = S.GradNorm([G], 1.0)
    norm.run()
    # the places' gradients in place of as many of 2^-9
    taken = sum(min(512, n - p) for p in places)
    want = math.sqrt(sum(float((f64(flat_g[p:p + min(512, n - p)]) ** 2).sum()) for p in places) + (n - taken) * 2.0 ** -18)
    assert abs(float(norm.norm) - want) <= 6 * U * want


@pytest.mark.parametrize("eight", [False, True])
def test_weights_beyond_32_bits_are_stepped(eight):
    """A learning rate that moves bf16 weights by many of their steps: every place differs from where it was, at the start,
    at the 2^31 border, in between and at the end."""
    n = (1 << 31) + 1554
    if torch.cuda.mem_get_info()[0] < (14 if eight else 27) * n // 2 + (2 << 30):
        pytest.skip("needs more free memory")
    W = torch.full((2, n // 2), 0.5, dtype=BF16, device="cuda")
    G = torch.full((2, n // 2), 2.0 ** -9, dtype=BF16, device="cuda")
    flat_w, flat_g = W.view(-1), G.view(-1)
    places = [0, (1 << 30) + 512, (1 << 31) - 512, 1 << 31, (n // 256 - 1) * 256]
    rng = np.random.default_rng(1)
    for p in places:
        size = min(512, n - p)
        flat_g[p:p + size] = dev((rng.standard_normal(size) * 1e-2).astype(np.float32)).to(BF16)
    opt = S.AdamW([W], bits=8 if eight else 32, weight_decay=WD, seed=6)
    S.adamw_step(opt, [G], 0.25, B1, B2, EPS)
    for p in places:
        size = min(512, n - p)
        g, z = f64(flat_g[p:p + size]), np.zeros(size)
        m, _, r = A.moments(z, z, g, B1, B2)
        u = A.direction(m, np.asarray(r), 1, B1, B2, EPS)
        w = 0.5 - 0.25 * (WD * 0.5 + u)
        got = f64(flat_w[p:p + size])
        assert np.all(np.abs(got - w) <= 2.0 ** -8 * np.abs(w) + U * (2 * np.abs(w) + 20 * 0.25 * (np.abs(u) + WD * 0.5)))
        assert np.all(np.abs(got - 0.5) > 0.1)
    # all the others had one gradient (whose direction is 1 but for eps, 5e-6 of it)
    w = 0.5 - 0.25 * (WD * 0.5 + 1)
    for p in places:
        flat_w[p:p + 512] = w
    assert all(bool(((part.float() - w).abs() <= (2.0 ** -8 + 2.0 ** -14) * w).all()) for part in flat_w.split(1 << 28))


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("cols,ld,off", [(704, (1 << 30) + 16, 0), (701, (1 << 30) + 5, 3)])
def test_rows_more_than_32_bits_apart(cols, ld, off, eight):
    """W and G as three rows whose last begins beyond 2^31 entries, on vector addresses and off them; the norm of such
    gradients; nothing else in W's buffer changes."""
    total = 2 * ld + cols + off
    if torch.cuda.mem_get_info()[0] < 6 * total:
        pytest.skip("needs more free memory")
    wbuf, gbuf = (torch.zeros(total, dtype=BF16, device="cuda") for _ in range(2))
    W, G = (b.as_strided((3, cols), (ld, 1), off) for b in (wbuf, gbuf))
    w, g, _, _ = draw_tensor(np.random.default_rng(3), (3, cols))
    W.copy_(torch.from_numpy(w.astype(np.float32)).reshape(3, cols))
    G.copy_(torch.from_numpy(g.astype(np.float32)).reshape(3, cols))
    ref = Reference(f64(W.contiguous()), np.zeros(3 * cols), np.zeros(3 * cols), eight, 0, 6, bf16=True)
    opt = S.AdamW([W], bits=8 if eight else 32, weight_decay=WD, seed=6)
    check_norm([G], 1.0)
    S.adamw_step(opt, [G], LR, B1, B2, EPS)
    ref.check(opt, 0, *ref.step(f64(G.contiguous()), 1))
    W.zero_()
    assert not any(bool(part.any()) for part in wbuf.split(1 << 28))


def test_results_do_not_depend_on_the_split():
    """The same tensors in one call, one by one in calls of their own (32 bits), and prepared: equal bits."""
    shapes = [(257,), (40, 41), (3000,)]
    a, b, c = (make(shapes, False, F32, F32, False) for _ in range(3))
    S.adamw_step(a[0], a[1], LR, B1, B2, EPS)
    S.AdamWPlan(b[0], b[1], B1, B2, EPS).run(LR)
    for i in range(3):
        one = S.AdamW([c[0].W[i]], m=[c[0].m[i]], v=[c[0].v[i]], weight_decay=WD)
        S.adamw_step(one, [c[1][i]], LR, B1, B2, EPS)
    for other in (b, c):
        for k in ("W", "m", "v"):
            assert all(torch.equal(x, y) for x, y in zip(getattr(a[0], k), getattr(other[0], k)))


# ------------------------------------------------------------------ conversion
def test_convert_both_ways():
    shapes = SHAPES + [(0,), (70001,)]
    opt32, _, refs, _ = make(shapes, False, F32, F32, False, t=41)
    opt32.m[-1][5], opt32.v[-1][600] = math.nan, math.inf
    opt8 = S.AdamW([w.clone() for w in opt32.W], bits=8)
    S.adamw_convert(opt32, opt8)
    assert opt8.t == 41
    for i in range(len(shapes)):
        for x, codes, col in ((f64(opt32.m[i]), opt8.m[i], 0), (A.f32(np.sqrt(f64(opt32.v[i]))), opt8.v[i], 1)):
            c, b = A.encode(x)
            assert np.array_equal(bits(codes).reshape(-1), c) and np.array_equal(opt8.scales[i].cpu().numpy()[:, col], b)
    back = S.AdamW([w.clone() for w in opt32.W])
    S.adamw_convert(opt8, back)
    for i in range(len(shapes)):
        sc = opt8.scales[i].cpu().numpy()
        m, r = A.decode(bits(opt8.m[i]).reshape(-1), sc[:, 0]), A.decode(bits(opt8.v[i]).reshape(-1), sc[:, 1])
        assert np.array_equal(f64(back.m[i]), m, equal_nan=True)
        assert np.array_equal(f64(back.v[i]), A.f32(r * r), equal_nan=True)
    again = S.AdamW([w.clone() for w in opt32.W], bits=8)
    S.adamw_convert(back, again)
    # What 8 bits hold converts to the same values (v's root is exact), though not always to the same codes: a block's
    # largest y in [248, 256) rounds to 256, so the second conversion takes the next exponent for the block. There every
    # value of at least 2^-6 units still has its three mantissa bits; smaller ones are rounded to its 2^-9 units again.
    for i in range(len(shapes)):
        s1, s2 = opt8.scales[i].cpu().numpy(), again.scales[i].cpu().numpy()
        for c1, c2, col in ((opt8.m[i], again.m[i], 0), (opt8.v[i], again.v[i], 1)):
            x, y = A.decode(bits(c1).reshape(-1), s1[:, col]), A.decode(bits(c2).reshape(-1), s2[:, col])
            unit = np.repeat(np.exp2(s2[:, col].astype(float) - 127), 256)[:x.size]
            large = np.abs(x) >= 2.0 ** -6 * unit
            assert np.array_equal(np.isnan(x), np.isnan(y)) and np.array_equal(x[large], y[large])
            small = ~large & ~np.isnan(x)
            assert np.all(np.abs(x - y)[small] <= 2.0 ** -10 * unit[small])


@pytest.mark.parametrize("odd", [0, 1])
def test_convert_keeps_roots_that_are_not_zero(odd):
    n = 700
    v = A.f32(np.exp2(np.random.default_rng(3).uniform(-60, 0, n)))
    v[5] = 0.0
    src = S.AdamW([torch.zeros(n, device="cuda")], m=[torch.ones(n, device="cuda")], v=[dev(v.astype(np.float32))])
    buf = [torch.zeros(n + 1, dtype=torch.uint8, device="cuda") for _ in range(2)]
    m8, v8 = (b[odd:odd + n].view(torch.float8_e4m3fn) for b in buf)
    dst = S.AdamW(src.W, m=[m8], v=[v8], scales=[torch.zeros(3, 2, dtype=torch.uint8, device="cuda")])
    S.adamw_convert(src, dst)
    c, b = A.encode(A.f32(np.sqrt(v)).view(A.Roots))
    assert np.array_equal(bits(v8), c) and np.array_equal(dst.scales[0][:, 1].cpu().numpy(), b)
    assert c[5] == 0 and (np.delete(c, 5) >= 1).all() and (c == 1).sum() > 100


def test_convert_at_odd_addresses_and_counts():
    n = 777
    m, v = torch.randn(n + 3, device="cuda")[3:], torch.rand(n + 1, device="cuda")[1:]
    w = torch.zeros(n, device="cuda")
    src = S.AdamW([w], m=[m], v=[v], t=7, device_step=True)
    cm, cv = (torch.zeros(n + 7, dtype=torch.uint8, device="cuda") for _ in range(2))
    dst = S.AdamW([w], m=[cm[3:n + 3].view(torch.float8_e4m3fn)], v=[cv[1:n + 1].view(torch.float8_e4m3fn)],
                  scales=[torch.zeros(4, 2, dtype=torch.uint8, device="cuda")], device_step=True)
    S.adamw_convert(src, dst)
    assert dst.t == 7
    assert np.array_equal(cm[3:n + 3].cpu().numpy(), A.encode(f64(m))[0])
    assert np.array_equal(cv[1:n + 1].cpu().numpy(), A.encode(A.f32(np.sqrt(f64(v))))[0])
    assert not cm[:3].any() and not cm[n + 3:].any() and not cv[:1].any() and not cv[n + 1:].any()


# ------------------------------------------------------------------ gradient norm
def norm_of(G, max_norm, **kw):
    out = torch.full((2,), -1.0, device="cuda")
    skip = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    S.smuon_grad_norm(G, max_norm, out, skip, status=status, **kw)
    torch.cuda.synchronize()
    return float(out[0]), float(out[1]), int(skip), int(status)


def check_norm(G, max_norm):
    """Eight squares by fused multiply-adds: 8 roundings of at most U each on positive terms, so the sum is within 8 U and
    its root within 4 U; one rounding of the result (half a step: U, or 2^-150 below 2^-126, where float32's numbers are
    2^-149 apart) and of the factor."""
    want, coef = A.grad_norm([f64(g.contiguous()) for g in G], max_norm)
    got, c, skip, status = norm_of(G, max_norm)
    assert abs(got - want) <= 6 * U * want + 2.0 ** -150 and abs(c - coef) <= 6 * U * coef, (got, want)
    assert skip == 0 and status == 0


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 255, 256, 257, 2049, 70001, 3_000_001])
def test_norm_of_one_tensor(n, dt):
    G = [torch.randn(n, device="cuda").to(dt)]
    for max_norm in (1e-3, 1e9, math.inf):
        check_norm(G, max_norm)


def test_norm_of_many_tensors_with_strides():
    g = torch.Generator(device="cuda").manual_seed(1)
    G = []
    for i in range(1100):
        n = 0 if i == 50 else int(torch.randint(1, 900, (1,)).item())
        G.append(torch.randn(n, device="cuda", generator=g).to(BF16 if i % 3 else F32))
    big = torch.randn(65, 129, device="cuda", generator=g)
    G += [big[:, 1:38], torch.randn(64, 128, device="cuda", generator=g)[:, 64:], torch.randn(12, 10, device="cuda").to(BF16)[:, 1:2],
          torch.randn(1001, device="cuda", generator=g)[1:]]
    check_norm(G, 1.0)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("r,c,ld,off", [(1, 9001, 9001, 1), (300, 37, 41, 0), (40, 256, 264, 8), (40, 256, 264, 4), (5000, 1, 3, 1)])
def test_norm_off_the_vector_addresses(r, c, ld, off, dt):
    buf = torch.randn(r * ld + off + 8, device="cuda").to(dt)
    buf[:off] = math.nan
    check_norm([buf[off:off + r * ld].view(r, ld)[:, :c]], 1.0)


@pytest.mark.parametrize("size", [1e-42, 1e-30, 1e-22, 1e17, 1e19, 1e30])
def test_norm_of_small_and_large_gradients(size):
    """Squares beyond float32's range, up and down; one of ordinary size would drown them, so they are alone. The
    smallest are subnormal float32 numbers (exact in float64)."""
    x = (np.random.default_rng(0).standard_normal(5000) * size).astype(np.float32)
    check_norm([dev(x)], size)
    check_norm([torch.cat([dev(x), torch.zeros(300, device="cuda")])], size)


def test_norm_of_nothing_and_of_zeros():
    assert norm_of([torch.zeros(0, device="cuda")], 1.0)[:3] == (0.0, 1.0, 0)
    assert norm_of([torch.zeros(5000, device="cuda")], 1.0)[:3] == (0.0, 1.0, 0)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 3e38])
def test_norm_that_float32_does_not_hold(bad):
    G = [torch.randn(3000, device="cuda"), torch.full((3000,), 1.0, device="cuda")]
    G[1][1234] = bad
    if bad == 3e38:
        G[1][1235] = 3e38
    norm, coef, skip, status = norm_of(G, 1.0)
    assert coef == 0.0 and skip == 1 and status == S.DEV_NONFINITE_NORM
    assert math.isnan(norm) if math.isnan(bad) else norm == math.inf


def test_norm_is_the_same_every_time():
    G = [torch.randn(n, device="cuda") for n in (1_000_003, 17, 65536)]
    a = S.GradNorm(G, 1.0)
    a.run()
    first = a.out.clone()
    for _ in range(5):
        a.run()
        assert torch.equal(a.out, first)
    out = torch.zeros(2, device="cuda")
    S.smuon_grad_norm(G, 1.0, out)
    assert torch.equal(out, first)


def test_norm_on_another_stream_takes_its_workspace_there():
    """The workspace that the call makes for itself comes from the memory of the stream it runs on."""
    G = [torch.randn(3000, device="cuda")]
    out, side = torch.zeros(2, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream, handle in ((side, side.cuda_stream), (side.cuda_stream, side.cuda_stream), (None, 0)):
        ws = S.smuon_grad_norm(G, 1.0, out, stream=stream)
        torch.cuda.synchronize()
        of = [seg["stream"] for seg in torch.cuda.memory_snapshot()
              if seg["address"] <= ws.data_ptr() < seg["address"] + seg["total_size"]]
        assert of == [handle]
        want, _ = A.grad_norm([f64(G[0])], 1.0)
        assert abs(float(out[0]) - want) <= 6 * U * want
        out.zero_()
        torch.cuda.synchronize()


# ------------------------------------------------------------------ a run of them together
@pytest.mark.parametrize("eight", [False, True])
def test_training_steps_beside_sign_muon(eight):
    """Matrices by Sign-Muon, the other parameters by a clipped AdamW step, one of the steps with a gradient that is not
    finite: it is skipped, the others follow the reference; stopped and resumed, the run goes on bit for bit."""
    rng = np.random.default_rng(12)
    mats, others = [(64, 96), (128, 64)], [(500, 64), (64,), (64,), (192,)]
    Wm = [dev(0.02 * rng.standard_normal(s).astype(np.float32)) for s in mats]
    mom = [torch.zeros(s, device="cuda") for s in mats]
    Um = [torch.zeros(s, dtype=BF16, device="cuda") for s in mats]
    Gm = [torch.zeros(s, device="cuda") for s in mats]
    wm_ref = [host(w).astype(np.float64) for w in Wm]
    mom_ref = [np.zeros(s) for s in mats]
    Wo = [dev((0.02 * rng.standard_normal(s)).astype(np.float32)).to(BF16) for s in others]
    Go = [torch.zeros(s, dtype=BF16, device="cuda") for s in others]
    opt = S.AdamW(Wo, bits=8 if eight else 32, master=True, weight_decay=[WD, 0.0, 0.0, 0.0], seed=21, device_step=True)
    refs = [Reference(f64(opt.master[i]), 0 * f64(w), 0 * f64(w), eight, i, 21, WD if i == 0 else 0.0, bf16=True, master=True)
            for i, w in enumerate(Wo)]
    norm = S.GradNorm(Go, 0.5)
    plan = S.AdamWPlan(opt, Go, B1, B2, EPS, grad_scale=norm.coef, skip_if=norm.skip)
    ns = S.NsPlan(mom, Um, *WL.QUINTIC, 5, G=Gm, beta=0.9, flags=S.NS_SPLIT_BF16)
    upd = S.UpdatePlan(Wm, 0.01, U=[[u] for u in Um], M=1)
    saved, t = None, 0
    for step in range(5):
        gm = [rng.standard_normal(s).astype(np.float32) for s in mats]
        go = [torch.from_numpy((0.1 * rng.standard_normal(s)).astype(np.float32)).to(BF16) for s in others]
        if step == 2:
            go[1][3] = math.nan
        for d, s in zip(Gm + Go, [torch.from_numpy(x) for x in gm] + go):
            d.copy_(s)
        ns.run()
        upd.run()
        norm.run()
        plan.run(LR)
        for i in range(len(mats)):
            mom_ref[i] = 0.9 * mom_ref[i] + gm[i]
            u = O.newton_schulz(mom_ref[i], *WL.QUINTIC, 5)
            assert rel_fro(host(Um[i]), u) < 1e-2
            wm_ref[i] = wm_ref[i] - 0.01 * O.sign_extract(host(Um[i]))
            np.testing.assert_allclose(host(Wm[i]), wm_ref[i], atol=(step + 1) * 2.0 ** -24)
        if step == 2:
            assert int(norm.skip) == 1
            continue
        t += 1
        want, coef = A.grad_norm([f64(g) for g in go], 0.5)
        assert abs(float(norm.norm) - want) <= 6 * U * want and abs(float(norm.coef) - coef) <= 6 * U * coef
        step_refs(opt, refs, [f64(g) for g in go], t, scale=float(norm.coef.double()))
        if step == 1:
            saved = C.snapshot(opt)
    assert opt.t == t == 4
    # resumed from the second step's snapshot in fresh buffers with the same gradients
    fresh = S.AdamW([torch.zeros_like(w) for w in Wo], bits=8 if eight else 32, master=True,
                    weight_decay=[WD, 0.0, 0.0, 0.0], seed=21, device_step=True)
    C.restore(fresh, saved)
    a, b = S.AdamW([w.clone() for w in Wo], bits=8 if eight else 32, master=True, weight_decay=[WD, 0.0, 0.0, 0.0],
                   seed=21, device_step=True), fresh
    C.restore(a, saved)
    for _ in range(2):
        S.adamw_step(a, Go, LR, B1, B2, EPS)
        S.AdamWPlan(b, Go, B1, B2, EPS).run(LR)
    assert a.t == b.t == 4
    for k in ("W", "m", "v", "master", "scales"):
        for x, y in zip(getattr(a, k) or [], getattr(b, k) or []):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_binding_refuses_what_is_not_one_device_or_one_value():
    w = [torch.zeros(8, device="cuda")]
    opt = S.AdamW(w)
    with pytest.raises(ValueError, match="CUDA device"):
        S.adamw_step(opt, [torch.zeros(8)], LR)
    with pytest.raises(ValueError, match="shape"):
        S.adamw_step(opt, [torch.zeros(4, 2, device="cuda")], LR)
    with pytest.raises(ValueError):
        S.adamw_step(opt, [torch.zeros(8, device="cuda")] * 2, LR)
    with pytest.raises(ValueError, match="grad_scale"):
        S.adamw_step(opt, [torch.zeros(8, device="cuda")], LR, grad_scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="skip_if"):
        S.adamw_step(opt, [torch.zeros(8, device="cuda")], LR, skip_if=torch.ones(1, device="cuda"))
    with pytest.raises(S.SmuonError, match="lr"):
        S.adamw_step(opt, [torch.zeros(8, device="cuda")], -1.0)
    with pytest.raises(S.SmuonError, match="lr"):
        S.adamw_step(opt, [torch.zeros(8, device="cuda")], math.nan)
    with pytest.raises(S.SmuonError, match="overlap"):
        S.adamw_step(opt, [w[0]], LR)
    with pytest.raises(S.SmuonError, match="overlap"):
        S.adamw_step(S.AdamW([w[0], w[0]]), [torch.zeros(8, device="cuda")] * 2, LR)
    plan = S.AdamWPlan(opt, [torch.zeros(8, device="cuda")])
    with pytest.raises(ValueError, match="lr"):
        plan.run()
    assert opt.t == 0 and not w[0].any()
