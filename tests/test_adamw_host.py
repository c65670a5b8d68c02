"""AdamW operators without a GPU: the oracle against things other than itself
(the method's formula in exact fractions, PyTorch's E4M3 casts, the repository's
counter generator), the rounding's mean, and the host checks of every entry
point: bad arguments are refused before a device would be touched."""
import ctypes
import importlib.util
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import matrix_aware_sign_b200 as S
from matrix_aware_sign_b200 import checkpoint as C
from oracle import adamw_oracle as A
from workloads import counter_rng as CR

ADDR = 1 << 20  # fake, aligned device addresses: only looked at, never read


# ------------------------------------------------------------------ oracle pins
def test_step_against_fractions():
    """Two steps of one weight against the formula evaluated in fractions (the square root to 60 bits)."""
    b1, b2, lr, eps, wd = Fraction(9, 10), Fraction(99, 100), Fraction(1, 100), Fraction(1, 10 ** 6), Fraction(1, 10)
    w, m, v = Fraction(1, 2), Fraction(0), Fraction(0)
    wo, mo, vo = 0.5, 0.0, 0.0
    root = lambda q: Fraction(math.isqrt(q.numerator * q.denominator << 200), q.denominator << 100)  # noqa: E731
    for t, g in ((1, Fraction(1, 4)), (2, Fraction(-3, 8))):
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        w = w - lr * (wd * w + (m / (1 - b1 ** t)) / (root(v / (1 - b2 ** t)) + eps))
        wo, mo, vo = A.step64(wo, float(g), mo, vo, t, float(lr), float(b1), float(b2), float(eps), float(wd))
        for got, want in ((wo, w), (mo, m), (vo, v)):
            assert abs(got - float(want)) <= 1e-14 * abs(float(want))


def test_first_step_is_the_sign_times_lr():
    """From zero moments, with eps far below |g|, step 1 moves every weight by lr against its gradient's sign."""
    g = np.array([3.0, -2e-5, 1e4])
    w, _, _ = A.step64(np.zeros(3), g, 0 * g, 0 * g, 1, 0.01, 0.9, 0.999, 1e-16, 0.0)
    np.testing.assert_allclose(w, -0.01 * np.sign(g), rtol=1e-10)


def test_moments_round_every_operation_once():
    """The float32 moments equal numpy's float32 arithmetic operation by operation."""
    rng = np.random.default_rng(3)
    m, g = rng.standard_normal((2, 5000)).astype(np.float32)
    v = rng.random(5000).astype(np.float32)
    f = np.float32
    b1, c1, b2, c2, s = f(0.9), f(1 - 0.9), f(0.999), f(1 - 0.999), f(0.37)
    mo, vo, ro = A.moments(m, v, g, 0.9, 0.999, 0.37)
    gs = s * g
    want_v = b2 * v + c2 * (gs * gs)
    for got, want in ((mo, b1 * m + c1 * gs), (vo, want_v), (ro, np.sqrt(want_v))):
        assert np.array_equal(got.astype(np.float32), want)


def test_codes_are_torchs_e4m3():
    """Code values and rounding to nearest against PyTorch's float8_e4m3fn casts."""
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(A.code_values(), ref)
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.standard_normal(4000) * np.exp2(rng.uniform(-12, 6, 4000)), ref[np.isfinite(ref)] / 2,
                        (np.arange(200) - 100) * 2.0 ** -10]).astype(np.float32)
    y = y[np.abs(y) < 256]
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(A._nearest_code(y.astype(np.float64)), want)


@pytest.mark.parametrize("scale", [1.0, 1e-20, 1e20, 2.0 ** -118, 3e38])
def test_round_trip_error_is_half_a_step(scale):
    """To nearest, a value is off by at most 2^-4 of itself, or half a step (2^-10) of the smallest codes."""
    x = (np.random.default_rng(1).standard_normal(700) * np.exp2(np.random.default_rng(2).uniform(-20, 0, 700)))
    x = A.f32(x / np.abs(x).max() * scale)
    codes, byte = A.encode(x)
    back = A.decode(codes, byte)
    unit = np.repeat(np.exp2(byte.astype(float) - 127), 256)[:700]
    bound = np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * unit)
    # a block whose largest magnitude is below 2^-119 (byte 0) is held as zeros by definition: off by the value itself
    zeros = np.repeat(byte == 0, 256)[:700]
    assert np.all(np.abs(x[zeros]) < 2.0 ** -119) and not back[zeros].any()
    assert np.all((np.abs(back - x) <= bound)[~zeros])


def test_special_blocks():
    x = np.zeros(4 * 256)
    x[5] = 1e-37            # block 0: below 2^-119
    x[256 + 9] = math.nan   # block 1
    x[512 + 1] = -math.inf  # block 2
    x[768] = 2.0 ** -119    # block 3: the smallest that is held
    codes, byte = A.encode(A.f32(x))
    assert list(byte) == [0, 255, 255, 1] and not codes[:768].any()
    back = A.decode(codes, byte)
    assert np.all(back[:256] == 0) and np.isnan(back[256:768]).all() and back[768] == 2.0 ** -119


def test_random_rounding_has_the_value_as_its_mean():
    """Over all 2^16 values of the random bits the mean of the decoded codes is the value, but for the four
    bits below the random ones (less than 2^-16 of a code step): for codes of full precision."""
    rnd = np.arange(65536, dtype=np.uint32)
    for x in (1.0, 1.03, -1.9999, 0.37, 5.3e-3):
        got = []
        for first in range(0, 65536, 255):
            r = rnd[first:first + 255]
            block = np.full(256, 1.5)  # sets the block's exponent
            block[1:1 + r.size] = x
            bits = np.zeros(256, np.uint32)
            bits[1:1 + r.size] = r
            c, b = A.encode(A.f32(block), bits)
            got.append(A.decode(c, b)[1:1 + r.size])
        got = np.concatenate(got)
        step = 2.0 ** (math.frexp(abs(x))[1] - 4)
        assert abs(np.mean(got) - float(np.float32(x))) <= 2.0 ** -16 * step * 1.001


def test_random_rounding_has_the_value_as_its_mean_at_every_size():
    """The same down to 2^-17 of the block's largest, where codes are 2^-9 units apart (a unit: 1 / 128 to 1 / 256 of the
    block's largest; here 1 / 192): off by less than 2^-16 of a code step, as above, and by the rounding to 2^-29 units."""
    rnd = np.arange(65536, dtype=np.uint32)
    unit = 2.0 ** -7
    for x in [1.5 * 1.37 * 2.0 ** -k for k in range(1, 18)] + [-1.1e-4, 3.3 * 2.0 ** -16, 2.0 ** -17]:
        got = []
        for first in range(0, 65536, 255):
            r = rnd[first:first + 255]
            block = np.full(256, 1.5)
            block[1:1 + r.size] = x
            bits = np.zeros(256, np.uint32)
            bits[1:1 + r.size] = r
            c, b = A.encode(A.f32(block), bits)
            assert b[0] == 120
            got.append(A.decode(c, b)[1:1 + r.size])
        got = np.concatenate(got)
        step = max(2.0 ** (math.frexp(abs(x))[1] - 4), 2.0 ** -9 * unit)
        assert abs(np.mean(got) - float(np.float32(x))) <= 2.0 ** -16 * step * 1.001 + 2.0 ** -30 * unit, x
        assert np.ptp(got) == (step if len(set(got)) > 1 else 0) and np.all(np.abs(got - x) <= step)


def test_moments_in_8_bits_decay_as_they_would_in_float32():
    """255 entries whose gradients have ceased, beside one whose moments stay: over 400 steps the mean root falls by
    b2^200, the mean first moment to nothing, at every size down to the smallest codes. The rounding leaves a mean
    alone. A root that was a code of at most 16 steps moves by f <= 16 (1 - sqrt(b2)) = 0.008 steps and is rounded with
    variance f (1 - f), so after 400 roundings the mean of 255 is within six times sqrt(400 * 0.008 / 255) = 0.67 code
    steps (2^-9 units, or 2^-3 of the value at most) of its expectation."""
    rng = np.random.default_rng(5)
    b1, b2, steps = 0.9, 0.999, 400
    for k in (3, 9, 12, 13, 14, 15):
        x = np.full(256, 1.5)
        x[1:] = 1.9 * 1.5 * 2.0 ** -k
        m, r = x.copy(), x.copy()
        for _ in range(steps):
            noise = rng.integers(0, 65536, 256)
            m, r = A.f32(b1 * m), A.f32(np.sqrt(b2) * r)
            m[0] = r[0] = 1.5
            m, r = A.decode(*A.encode(m, noise)), A.decode(*A.encode(r, noise))
        step = max(2.0 ** -3 * x[1], 2.0 ** -9 * 2.0 ** -7)
        assert abs(r[1:].mean() - x[1] * b2 ** (steps / 2)) <= 6 * math.sqrt(steps * 0.008 / 255) * step, k
        assert np.abs(m[1:]).mean() <= x[1] * b1 ** steps + 2.0 ** -9 * 2.0 ** -7, k


def test_roots_that_are_not_zero_stay():
    """Whatever the random bits, and to nearest: a root below the smallest code gets it, zero stays zero, a block that is
    too small to be held is held as zeros; first moments are rounded as they are."""
    x = np.zeros(512)
    x[:4] = 1.5, 1e-9, 0.0, 2.0 ** -17
    x[256:] = 2.0 ** -120
    _, _, r = A.moments(np.zeros(512), x * x, np.zeros(512), 0.5, 1 - 2.0 ** -30)
    for rnd in (None, np.zeros(512, np.uint32), np.full(512, 65535, np.uint32)):
        c, b = A.encode(r, rnd)
        assert list(c[1:3]) == [1, 0] and c[3] >= 1 and not c[4:].any() and b[1] == 0
        m, _ = A.encode(np.asarray(r), rnd)
        # 1e-9 is 6.6e-5 of the smallest code's 2^-16 (a unit is 2^-7): the largest random number alone brings it there
        assert m[1] == (rnd is not None and rnd[1] == 65535) and m[0] == c[0]


def test_no_first_moment_is_held_over_a_root_of_zero():
    """300 steps in 8 bits of entries whose gradients are 1e-5 of their block's largest: m' is not zero only where a gradient
    was not, and there v' is not zero either, so no direction has eps alone for its denominator."""
    rng = np.random.default_rng(2)
    cm = cr = np.zeros(256, np.uint8)
    bm = br = np.zeros(1, np.uint8)
    for t in range(1, 301):
        g = rng.standard_normal(256) * 1e-5
        g[0] = rng.standard_normal()
        m, r = A.decode(cm, bm), A.decode(cr, br)
        m, v, r = A.moments(m, r * r, A.f32(g), 0.9, 0.999)
        rnd = rng.integers(0, 65536, 256)
        (cm, bm), (cr, br) = A.encode(m, rnd), A.encode(r, rnd)
        assert not np.any(((cm & 127) > 0) & (cr == 0)), t


def test_rounding_bits_come_from_the_repositorys_generator():
    """Word i of the Philox block of group e / 8 serves entries 2i (low half) and 2i + 1 (high half)."""
    got = A.rounding_bits(40, 6, 11, 5)
    for grp in range(5):
        words = CR.philox4x32_10(np.array([grp, 0, 5, 1], np.uint32), np.array([11, 6], np.uint32))
        want = [h for w in words for h in (int(w) & 0xFFFF, int(w) >> 16)]
        assert list(got[8 * grp:8 * grp + 8]) == want


# ------------------------------------------------------------------ host checks
@pytest.fixture(scope="module")
def L():
    return S.lib()


def _mats(*ms):
    return (S.SmuonMat * len(ms))(*ms)


def _m(k, rows=4, cols=8, ld=None, dt=S.F32, off=0):
    return S.SmuonMat(ADDR * (k + 1) + off, rows, cols, cols if ld is None else ld, dt)


def _state(W=None, m=None, v=None, master=None, scales=None, n=1, t=0, wd=None, ls=None, seed=0, d_t=None):
    keep = (_mats(W or _m(0)), _mats(m or _m(1)), _mats(v or _m(2)), _mats(master) if master else None,
            (ctypes.c_void_p * 1)(scales) if scales else None,
            (ctypes.c_float * 1)(wd) if wd is not None else None, (ctypes.c_float * 1)(ls) if ls is not None else None)
    st = S.AdamWState(n, seed, keep[0], keep[3], keep[1], keep[2], keep[4], keep[6], keep[5], t, d_t)
    st._keep = keep
    return st


E8 = dict(m=_m(1, dt=S.E4M3), v=_m(2, dt=S.E4M3))

REFUSED = {
    "no tensors": (dict(n=0), {}, -1, b"n_tensors"),
    "negative t": (dict(t=-1), {}, -1, b"t < 0"),
    "W int8": (dict(W=_m(0, dt=S.I8)), {}, -3, b"W[0]"),
    "m bf16": (dict(m=_m(1, dt=S.BF16)), {}, -3, b"m[0]"),
    "m 8 bit, v not": (dict(m=_m(1, dt=S.E4M3), scales=ADDR * 9), {}, -3, b"v[0]"),
    "8 bit without scales": (E8, {}, -1, b"scales"),
    "odd scales": (dict(E8, scales=ADDR * 9 + 1), {}, -1, b"2-byte"),
    "m shorter": (dict(m=_m(1, rows=3)), {}, -2, b"number of entries"),
    "m strided": (dict(m=_m(1, ld=12)), {}, -2, b"contiguous"),
    "master of f32": (dict(master=_m(5)), {}, -3, b"not BF16"),
    "master shorter": (dict(W=_m(0, dt=S.BF16), master=_m(5, rows=2)), {}, -2, b"master[0]"),
    "negative decay": (dict(wd=-0.1), {}, -1, b"weight_decay[0]"),
    "nan lr scale": (dict(ls=math.nan), {}, -1, b"lr_scale[0]"),
    "negative rows": (dict(W=_m(0, rows=-1)), {}, -2, b"W[0]"),
    "rows too far apart": ({}, dict(G=_m(3, ld=1 << 39)), -2, b"2^40"),
    "W null": (dict(W=S.SmuonMat(None, 4, 8, 8, S.F32)), {}, -1, b"NULL"),
    "W misaligned": (dict(W=_m(0, off=2)), {}, -1, b"aligned"),
    "G shape": ({}, dict(G=_m(3, rows=8, cols=4)), -2, b"G[0]"),
    "G e4m3": ({}, dict(G=_m(3, dt=S.E4M3)), -3, b"G[0]"),
    "G ld": ({}, dict(G=_m(3, ld=7)), -2, b"ld"),
    "G null": ({}, dict(G=None), -1, b"G is NULL"),
    "beta1": ({}, dict(beta1=1.0), -1, b"beta1"),
    "beta2 nan": ({}, dict(beta2=math.nan), -1, b"beta2"),
    "eps 0": ({}, dict(eps=0.0), -1, b"eps"),
    "m is W": (dict(m=_m(0)), {}, -1, b"overlap"),
    "v reaches into m": (dict(v=_m(1, off=64)), {}, -1, b"overlap"),
    "G is m": ({}, dict(G=_m(1)), -1, b"overlap"),
    "scales in v": (dict(E8, scales=ADDR * 3 + 30), {}, -1, b"overlap"),
    "d_t in W": (dict(d_t=ADDR + 8), {}, -1, b"overlap"),
    "d_t misaligned": (dict(d_t=ADDR * 9 + 4), {}, -1, b"d_t"),
    "skip misaligned": ({}, dict(skip=ADDR * 9 + 2), -1, b"4-byte"),
}


@pytest.mark.parametrize("name", list(REFUSED))
def test_step_and_plan_refuse(L, name):
    st_kw, call_kw, code, word = REFUSED[name]
    st = _state(**st_kw)
    a = dict(G=_m(3), lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, skip=None)
    a.update(call_kw)
    G = None if a["G"] is None else _mats(a["G"])
    assert L.adamw_step(ctypes.byref(st), G, a["lr"], a["beta1"], a["beta2"], a["eps"], None, None, a["skip"], None) == code
    assert word in L.smuon_last_error(), L.smuon_last_error()
    h = ctypes.c_void_p(1)
    assert L.adamw_plan_create(ctypes.byref(st), G, a["beta1"], a["beta2"], a["eps"], None, None, a["skip"], ADDR * 30,
                               4096, None, ctypes.byref(h)) == code
    assert not h.value
    assert st.t == st_kw.get("t", 0)


def test_tensors_that_share_memory(L):
    """Two weights may be column ranges of one matrix; ranges that meet are refused, and so is one tensor listed twice."""
    def call(w0, w1, n=32):
        W, keep = _mats(w0, w1), []
        e = [_mats(_m(4 + k, rows=w0.rows, cols=w0.cols), _m(8 + k, rows=w1.rows, cols=w1.cols)) for k in range(3)]
        keep += e
        st = S.AdamWState(2, 0, W, None, e[0], e[1], None, None, None, 0, None)
        return L.adamw_step(ctypes.byref(st), e[2], 1e-3, 0.9, 0.999, 1e-8, None, None, None, None)

    halves = _m(0, cols=8, ld=16), _m(0, cols=8, ld=16, off=32)
    without_gpu = () if torch.cuda.is_available() else (-6, -4)
    if without_gpu:  # past every check of arguments: only the device is missing
        assert call(*halves) in without_gpu
        assert b"overlap" not in L.smuon_last_error()
    for bad in ((halves[0], _m(0, cols=8, ld=16, off=28)), (halves[0], _m(0, cols=9, ld=16, off=32)),
                (halves[0], _m(0, cols=8, ld=18, off=32)), (halves[0], halves[0]), (_m(0), _m(0, off=4 * 31)),
                (_m(0, rows=1, cols=100), _m(0, rows=1, cols=1, off=396))):
        assert call(*bad) == -1 and b"overlap" in L.smuon_last_error(), bad



WIDE = dict(W=_m(0, cols=8, ld=16))  # rows of 32 bytes, 64 apart
BETWEEN_ROWS = {  # what lies where, and whether it reaches from the gap behind a row into the next row
    "d_t": (WIDE, dict(d_t=ADDR + 56), True),
    "d_t in the gap": (WIDE, dict(d_t=ADDR + 40), False),
    "scales": (dict(WIDE, **E8, scales=ADDR + 62), {}, False),  # one block: two bytes, the gap's last
    "scales of two blocks": (dict(W=_m(0, rows=40, cols=8, ld=16), m=_m(1, rows=40, dt=S.E4M3), v=_m(2, rows=40, dt=S.E4M3),
                                  scales=ADDR + 62), dict(rows=40), True),
    "m": (dict(WIDE, m=S.SmuonMat(ADDR + 48, 4, 8, 8, S.F32)), {}, True),
    "m in a wide gap": (dict(W=_m(0, cols=8, ld=80), m=S.SmuonMat(ADDR + 64, 4, 8, 8, S.F32)), {}, False),
    "one row of m": (dict(WIDE, m=S.SmuonMat(ADDR + 48, 1, 32, 32, S.F32)), {}, True),
}


@pytest.mark.parametrize("name", list(BETWEEN_ROWS))
def test_memory_between_the_rows_of_a_strided_weight(L, name):
    """Whatever starts behind a row is refused where it reaches the next one, and taken where it does not."""
    st_kw, more, meets = BETWEEN_ROWS[name]
    st = _state(**st_kw, **{k: v for k, v in more.items() if k == "d_t"})
    if not meets and torch.cuda.is_available():
        pytest.skip("would run on made-up addresses")
    code = L.adamw_step(ctypes.byref(st), _mats(_m(3, rows=more.get("rows", 4))), 1e-3, 0.9, 0.999, 1e-8, None, None, None, None)
    if meets:
        assert code == -1 and b"overlap" in L.smuon_last_error()
    else:  # past every check of arguments: only the device is missing
        assert code in (-6, -4) and b"overlap" not in L.smuon_last_error()


@pytest.mark.parametrize("which", ["d_lr", "d_grad_scale", "d_skip_if"])
@pytest.mark.parametrize("at", [ADDR + 4, ADDR * 2 + 124, ADDR * 3, ADDR * 9, ADDR * 10 + 12])
def test_scalars_in_written_memory(L, which, at):
    """Every CTA reads them while others write: refused in W, m, v, scales and the device count."""
    st = _state(**E8, scales=ADDR * 9, d_t=ADDR * 10) if at >= ADDR * 9 else _state()
    d = {k: (at if k == which else None) for k in ("d_lr", "d_grad_scale", "d_skip_if")}
    assert L.adamw_step(ctypes.byref(st), _mats(_m(3)), 1e-3, 0.9, 0.999, 1e-8, *d.values(), None) == -1
    assert which.encode() in L.smuon_last_error() and b"overlap" in L.smuon_last_error()

def test_execute_refuses_other_plans(L):
    st = _state()
    assert L.adamw_execute(None, ctypes.byref(st), 1e-3, None) == -1
    assert L.smuon_grad_norm_execute(None, None) == -1


def test_convert_refuses(L):
    a, b = _state(), _state(W=_m(4), m=_m(5), v=_m(6))
    e = _state(W=_m(7), m=_m(8, dt=S.E4M3), v=_m(9, dt=S.E4M3), scales=ADDR * 20)
    call = lambda x, y: L.adamw_convert(ctypes.byref(x), ctypes.byref(y), None)  # noqa: E731
    assert call(a, b) == -3
    assert call(e, e) == -3
    other = _state(W=_m(7, rows=5), m=_m(8, rows=5, dt=S.E4M3), v=_m(9, rows=5, dt=S.E4M3), scales=ADDR * 20)
    assert call(a, other) == -2
    inside = _state(W=_m(7), m=_m(1, dt=S.E4M3), v=_m(9, dt=S.E4M3), scales=ADDR * 20)
    assert call(a, inside) == -1 and b"overlap" in L.smuon_last_error()
    counted = _state(W=_m(7), m=_m(8, dt=S.E4M3), v=_m(9, dt=S.E4M3), scales=ADDR * 20, d_t=ADDR * 21)
    assert call(a, counted) == -1 and b"count" in L.smuon_last_error()
    many = S.AdamWState(2, 0, a.W, None, a.m, a.v, None, None, None, 0, None)
    many.n_tensors = 0
    assert call(many, e) == -1


def test_norm_refuses(L):
    G = _mats(_m(0), _m(1, dt=S.BF16))
    size = ctypes.c_size_t(0)
    assert L.smuon_grad_norm_workspace_bytes(G, 2, ctypes.byref(size)) == 0 and size.value >= 16
    ok = dict(G=G, n=2, max_norm=1.0, out=ADDR * 4, skip=None, ws=ADDR * 5, size=size.value)

    def call(**kw):
        a = dict(ok, **kw)
        return L.smuon_grad_norm(a["G"], a["n"], a["max_norm"], a["out"], a["skip"], a["ws"], a["size"], None, None)

    assert call(G=None) == -1 and call(n=0) == -1 and call(out=None) == -1 and call(out=ADDR + 2) == -1
    assert call(max_norm=0.0) == -1 and call(max_norm=math.nan) == -1 and call(max_norm=-1.0) == -1
    assert call(ws=None) == -5 and call(ws=ADDR + 8) == -5 and call(size=8) == -5
    assert call(G=_mats(_m(0, dt=S.I8)), n=1) == -3
    assert call(G=_mats(_m(0, ld=3)), n=1) == -2
    h = ctypes.c_void_p(1)
    assert L.smuon_grad_norm_plan_create(G, 2, -1.0, ADDR * 4, None, ADDR * 5, size.value, None, None,
                                         ctypes.byref(h)) == -1
    assert not h.value


def test_workspaces(L):
    """A norm's holds its table (two places of 40 bytes a tensor) and a sum for each of at most 592 CTAs; a step's plan 96 bytes a
    tensor. A plan refuses one that is missing, misaligned or too small."""
    size = ctypes.c_size_t(0)
    for n in (1, 512, 5000):
        G = _mats(*[_m(k, rows=1, cols=1) for k in range(n)])
        assert L.smuon_grad_norm_workspace_bytes(G, n, ctypes.byref(size)) == 0 and size.value >= 592 * 8 + 80 * n
    none = _mats(S.SmuonMat(None, 0, 5, 5, S.F32))
    assert L.smuon_grad_norm_workspace_bytes(none, 1, ctypes.byref(size)) == 0
    assert L.smuon_grad_norm_workspace_bytes(none, 1, None) == -1
    st, h = _state(), ctypes.c_void_p()
    assert L.adamw_plan_workspace_bytes(ctypes.byref(st), ctypes.byref(size)) == 0 and size.value >= 96
    assert L.adamw_plan_workspace_bytes(None, ctypes.byref(size)) == -1
    for ws, n in ((None, 4096), (ADDR * 30 + 16, 4096), (ADDR * 30, 95)):
        assert L.adamw_plan_create(ctypes.byref(st), _mats(_m(3)), 0.9, 0.999, 1e-8, None, None, None, ws, n, None,
                                   ctypes.byref(h)) == -5


def test_binding_refuses_before_the_library():
    w = [torch.zeros(4, 8), torch.zeros(5)]
    with pytest.raises(ValueError, match="CUDA"):
        S.AdamW(w)
    with pytest.raises(ValueError, match="CUDA"):
        S.GradNorm(w, 1.0)
    with pytest.raises(ValueError):
        S.AdamW(w, bits=16)
    with pytest.raises(ValueError):
        S.AdamW(w, m=[torch.zeros(4, 8), torch.zeros(5)])
    z8 = [torch.zeros(4, 8).to(torch.float8_e4m3fn), torch.zeros(5).to(torch.float8_e4m3fn)]
    with pytest.raises(ValueError, match="scales"):
        S.AdamW(w, m=z8, v=z8)
    with pytest.raises(ValueError, match="scales"):
        S.AdamW(w, m=z8, v=z8, scales=[torch.zeros(1, 2, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)])


def test_tensor_descriptions():
    d = lambda t: (lambda m: (m.rows, m.cols, m.ld, m.dtype))(S.tensor(t))  # noqa: E731
    assert d(torch.zeros(())) == (1, 1, 1, S.F32)
    assert d(torch.zeros(7)) == (1, 7, 7, S.F32)
    assert d(torch.zeros(2, 3, 5, dtype=torch.bfloat16)) == (6, 5, 5, S.BF16)
    assert d(torch.zeros(4, 10)[:, 2:5]) == (4, 3, 10, S.F32)
    assert d(torch.zeros(0, 5)) == (0, 0, 0, S.F32)
    assert d(torch.zeros(3, 1).to(torch.float8_e4m3fn)) == (3, 1, 1, S.E4M3)
    for bad in (torch.zeros(4, 5).t(), torch.zeros(2, 4, 4)[:, :, :2], torch.zeros(4).expand(3, 4), torch.zeros(4)[::2]):
        with pytest.raises(ValueError):
            S.tensor(bad)
    with pytest.raises(ValueError):
        S.tensor(torch.zeros(3, dtype=torch.float16))


def test_checkpoint_knows_the_state():
    """A snapshot names every tensor of an AdamW state, and refuses another seed."""
    class Fake(S.AdamW):
        def __init__(self, seed):  # the fields that a checkpoint reads, on the CPU
            self.W, self.master = [torch.ones(3)], None
            self.m, self.v = [torch.ones(3).to(torch.float8_e4m3fn)], [torch.ones(3).to(torch.float8_e4m3fn)]
            self.scales, self.d_t = [torch.ones(1, 2, dtype=torch.uint8)], None
            self.state = S.AdamWState(1, seed)
            self.state.t = 4

    a, b = Fake(3), Fake(3)
    snap = C.snapshot(a)
    assert set(snap["tensors"]) == {"W.0", "m.0", "v.0", "scales.0"}
    b.state.t, b.W[0][:] = 0, 9.0
    C.restore(b, snap)
    assert b.state.t == 4 and torch.equal(b.W[0], a.W[0])
    with pytest.raises(ValueError, match="seed"):
        C.restore(Fake(4), snap)


def test_a_plan_asks_its_own_device_for_a_capture(monkeypatch):
    """What counts is whether the stream of the plan's device is capturing, whichever device is current."""
    class Device:
        current = 0

        def __init__(self, device):
            self.to = device.index

        def __enter__(self):
            self.back, Device.current = Device.current, self.to

        def __exit__(self, *_):
            Device.current = self.back

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: Device.current == 1)
    with pytest.raises(ValueError, match="capture"):
        S._Prepared()._uploading(torch.device("cuda:1"))
    assert Device.current == 0
    with S._Prepared()._uploading(torch.device("cuda:0")):
        assert Device.current == 0


def test_the_current_stream_without_pytorchs_short_ways(monkeypatch):
    """On a PyTorch without these private names the public calls give the current stream's handle, to every operator."""
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: type("Stream", (), {"cuda_stream": 100 + index}))
    spec = importlib.util.spec_from_file_location("binding_again", S.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    assert again._current_device() == 3 and again._stream(None) == 103 and again._stream(7) == 7
